"""Experts whose keys are equal, or nearly so, where the last of the k are chosen: the numbers of the formula in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu

MASKS = [-1e4, -65504.0, -1e9, -1e20, -1e30]


def chosen(x, k, scoring, bias=None, groups=1, top_groups=None, group_best=2):
    """(The experts by the definition, with keys in 64 bits; rows that 64 bits leave open).  No logit here is infinite or NaN.

    Of rows left open: a score in 64 bits is off by at most (E + 8) 2^-53 (exponentials, a sum of E terms, a quotient), a key
    and a sum of two by 2^-53 of their size more; so worths that are nearer than (2 E + 16) 2^-53 (1 + the largest key), as
    those that are equal in exact arithmetic, lie in the order of these roundings, unless their terms are the same."""
    x = x.double().cpu()
    T, E = x.shape
    near_0 = torch.exp(-x.abs())
    s = torch.softmax(x, -1) if scoring == "softmax" else torch.where(x < 0, near_0, 1.0) / (1 + near_0)
    key = x if bias is None else s + bias.double().cpu()
    left_open = torch.zeros(T, dtype=torch.bool)
    if top_groups is not None and top_groups < groups:
        of = x if bias is None and group_best == 1 else s if bias is None else key
        terms = of.view(T, groups, -1).topk(min(group_best, E // groups), -1).values
        worth = terms.sum(-1)
        ranks = torch.sort(worth, dim=-1, descending=True, stable=True)
        last = ranks.indices[:, top_groups:]
        shut = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, last, True)
        key = key.masked_fill(shut.repeat_interleave(E // groups, 1), -torch.inf)
        if bias is not None or group_best == 2:
            slack = (2 * E + 16) * 2.0**-53 * (1 + of.abs().amax(-1, keepdim=True))
            near = (worth - ranks.values[:, top_groups - 1:top_groups]).abs() < slack
            apart = terms.masked_fill(~near[..., None], -torch.inf).amax(1) != terms.masked_fill(~near[..., None], torch.inf).amin(1)
            left_open = (near & shut).any(-1) & apart.any(-1)
    return torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :k].to(torch.int32), left_open


def check(x, k, scoring, bias=None, every_row=False, **more):
    x = x.cuda()
    bias = None if bias is None else bias.cuda()
    got = binding.route_experts(x, k, scoring, bias=bias, **more)[0].cpu()
    want, left_open = chosen(x, k, scoring, bias, **more)
    left_open &= not every_row
    wrong = (got != want).any(-1) & ~left_open
    assert not wrong.any(), (int(wrong.sum()), got[wrong][0].tolist(), want[wrong][0].tolist())
    assert left_open.double().mean() <= 0.1  # (that the rows are held to something)


def tied(E, k, low, high, rest, dtype):
    """k and k + 1 times `low` with `high` behind them, and once between them, at several places; the others are `rest`."""
    rows = []
    for n in (k, k + 1, 2 * k + 1):
        for first in (0, 1, E // 2):
            if first + n + 1 > E:
                continue
            for at in {first + n, E - 1, first + n // 2}:
                row = [rest - 0.25 * (e % 7) for e in range(E)]
                row[first:first + n] = [low] * n
                row[at] = high
                rows.append(row)
    return torch.tensor(rows, dtype=torch.float64).to(dtype)


@pytest.mark.parametrize("k", [1, 2, 8])
@pytest.mark.parametrize("E", [24, 64, 256])
def test_a_better_one_behind_equal_ones(E, k):
    """By its logit (nothing else chooses without a bias), and by scores that 32 bits do not tell apart."""
    for scoring in ("softmax", "sigmoid"):
        check(tied(E, k, 0.0, 1e-7, -10.0, torch.float32), k, scoring)
        check(tied(E, k, 1.0, 1.0 + 2.0**-7, -60.0, torch.bfloat16), k, scoring)
        check(tied(E, k, 1.0, 1.0 + 2.0**-23, -1.0, torch.float32), k, scoring)
    for bias in (torch.zeros(E), torch.full((E,), 0.5)):
        for low, high in ((16.0, 16.125), (14.0, 14.0625), (20.0, 21.0)):
            check(tied(E, k, low, high, -3.0, torch.bfloat16), k, "sigmoid", bias)
        x = tied(E, k, -12.0, -11.9375, -14.0, torch.bfloat16)
        x[:, 5] = 5.0  # an expert with nearly all of the softmax
        check(x, k, "softmax", bias)
        check(x, min(k + 1, E), "softmax", bias)


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_a_better_one_behind_equal_ones_in_open_groups(scoring, best):
    for k in (1, 2, 4):
        more = dict(groups=8, top_groups=3, group_best=best)
        check(tied(64, k, 0.0, 1e-7, -10.0, torch.float32), k, scoring, **more)
        check(tied(64, k, 16.0, 16.125, -3.0, torch.bfloat16), k, scoring, torch.zeros(64), **more)


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E", [8, 64, 256])
def test_finite_masks(E, dtype, mask):
    """Masked experts beside repeated logits (bf16 repeats them by itself), which their mask must not push together."""
    g = torch.Generator().manual_seed(E)
    x = (1.5 * torch.randn(2000, E, generator=g)).to(torch.bfloat16).to(dtype)
    x[torch.rand(2000, E, generator=g) < 0.3] = mask
    x[:100, 2:] = mask  # fewer than k are left
    x[-1] = torch.tensor([0.0, 0.0, 1.0, 0.5, 5.0, 6.0, 6.0] + [mask] * (E - 7)).to(dtype)
    bias = 0.2 * torch.randn(E, generator=g)
    for scoring in ("softmax", "sigmoid"):
        for k in (1, 2, 8):
            check(x, k, scoring)
            check(x, k, scoring, torch.zeros(E))
            check(x, k, scoring, bias)
        check(x, 2, scoring, groups=4, top_groups=2, group_best=1)
        check(x, 2, scoring, bias, groups=4, top_groups=2, group_best=1)


def test_repeated_logits():
    """Few different values: every token has ties at its last place."""
    g = torch.Generator().manual_seed(7)
    for E, k in ((16, 2), (64, 8), (200, 6)):
        x = torch.randint(-3, 4, (3000, E), generator=g).to(torch.bfloat16) * 0.125 + 14
        for scoring in ("softmax", "sigmoid"):
            for bias in (None, torch.zeros(E), 0.25 * torch.randint(0, 2, (E,), generator=g).float()):
                check(x, k, scoring, bias)
                check(x, k, scoring, bias, groups=8, top_groups=4)


@pytest.mark.parametrize("offset", [-3e3, -4096.0, -5e3, -2e4, -1e9, 1e4, 1e9, 1e30])
def test_rows_far_from_zero(offset):
    """Of logits as large as the masked ones nothing is left out of the comparison."""
    g = torch.Generator().manual_seed(3)
    x = (20 * torch.randn(500, 64, generator=g).double() + offset).float()
    x[::2, ::3] -= abs(offset)  # half of the rows in two parts
    for scoring in ("softmax", "sigmoid"):
        for k in (1, 8):
            check(x, k, scoring)
        check(x, 2, scoring, groups=8, top_groups=2, group_best=1)
    check(x, 8, "softmax", (0.1 * torch.randn(64, generator=g)))
    bias = (20 * torch.randn(64, generator=g).double() + offset).float()
    check(torch.randn(500, 64, generator=g), 8, "sigmoid", bias)
