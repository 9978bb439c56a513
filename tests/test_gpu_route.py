"""Routing to experts against the formula in fp64, the experts number for number.

Bounds of the weights: an fp32 exponential is off by 2 units in the last place and by its argument's rounding,
(|x| + 4) 2^-24 relative with |x| <= the logits' spread; a sum of up to 512 terms by 48 2^-24, a division and the scale by
2^-24 each.  With s the spread: (2 s + 64) 2^-24 relative, 2^-120 absolute."""
import math
import random

import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu


def reference(x, k, scoring, bias, groups, top_groups, group_best, renormalize, scale):
    """(experts, weights) of rows x, a token at a time in Python's 64-bit floats."""
    E = x.shape[1]
    bias = [0.0] * E if bias is None else bias.double().tolist()
    experts, weights = [], []
    for row, exact in zip(x.double().cpu().tolist(), x.float().cpu().tolist()):
        row = [-math.inf if v != v else min(v, torch.finfo(torch.float32).max) for v in row]
        top = max(row)
        if scoring == "softmax":
            e = [math.exp(v - top) if v > -math.inf else 0.0 for v in row]
            total = math.fsum(e)
            s = [v / total if total else 0.0 for v in e]
        else:
            s = [1 / (1 + math.exp(-v)) if v > 0 else (math.exp(v) / (1 + math.exp(v)) if v > -math.inf else 0.0) for v in row]
        key = [a + b if v > -math.inf and a + b == a + b else -math.inf for a, b, v in zip(s, bias, row)]
        rank = key if any(bias) else row
        open_groups = range(groups)
        if top_groups < groups:
            size = E // groups
            if group_best == 1 and not any(bias):
                worth = [max(row[g * size:(g + 1) * size]) for g in range(groups)]
            else:
                worth = []
                for g in range(groups):
                    best = sorted((v for v in key[g * size:(g + 1) * size] if v > -math.inf), reverse=True)[:group_best]
                    worth.append(sum(best) if best else -math.inf)
            open_groups = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
        live = sorted((e for e in range(E) if e // (E // groups) in open_groups), key=lambda e: (-rank[e], e))[:k]
        w = [s[e] for e in live]
        if renormalize:
            # ratios of scores of any size, from their logarithms (softmax: less the one that all share)
            log = [row[e] if scoring == "softmax" else min(row[e], 0.0) - math.log1p(math.exp(-abs(row[e]))) for e in live]
            best = max(log)
            w = [math.exp(v - best) if v > -math.inf else 0.0 for v in log]
            total = math.fsum(w)
            w = [v / total if total else 0.0 for v in w]
        experts.append(live)
        weights.append([scale * v for v in w])
    return torch.tensor(experts, dtype=torch.int32), torch.tensor(weights, dtype=torch.float64)


def check(x, k, scoring="softmax", bias=None, groups=1, top_groups=None, group_best=2, renormalize=True, scale=1.0):
    experts, weights = binding.route_experts(x, k, scoring, bias=bias, groups=groups, top_groups=top_groups,
                                             group_best=group_best, renormalize=renormalize, scale=scale)
    want_e, want_w = reference(x, k, scoring, bias, groups, top_groups or groups, group_best, renormalize, scale)
    assert experts.dtype == torch.int32 and weights.dtype == torch.float32
    assert torch.equal(experts.cpu(), want_e)
    finite = x.float()[torch.isfinite(x.float())]
    spread = float(finite.max() - finite.min()) if len(finite) else 0.0
    bound = (2 * min(spread, 200.0) + 64) * 2.0**-24 * want_w.abs() + 2.0**-120
    assert ((weights.double().cpu() - want_w).abs() <= bound).all()
    return experts, weights


def logits(T, E, dtype, seed=0, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(T, E, generator=g, device="cuda")).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (3, 8, 8), (17, 60, 4), (9, 33, 32), (70, 256, 8), (5, 384, 6),
                                   (300, 64, 2), (2, 512, 32), (33, 511, 7)])
def test_plain(T, E, k, scoring, dtype):
    x = logits(T, E, dtype)
    check(x, k, scoring)
    check(x, k, scoring, renormalize=False, scale=2.5)
    g = torch.Generator(device="cuda").manual_seed(1)
    check(x, k, scoring, bias=0.2 * torch.randn(E, generator=g, device="cuda"))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 4, 1, 4), (96, 3, 2, 8), (32, 32, 5, 5),
                                            (510, 17, 3, 32), (40, 5, 5, 4), (504, 9, 1, 8), (24, 8, 7, 3)])
def test_groups(E, groups, top, k, biased, scoring):
    g = torch.Generator(device="cuda").manual_seed(2)
    bias = 0.3 * torch.randn(E, generator=g, device="cuda") if biased else None
    for best in (1, 2):
        for dtype in (torch.bfloat16, torch.float32):
            check(logits(45, E, dtype, 3), k, scoring, bias, groups, top, best)


def test_equal_keys_go_to_the_lowest_number():
    for bias in (None, torch.zeros(64, device="cuda"), torch.full((64,), 0.5, device="cuda")):
        x = torch.zeros(4, 64, device="cuda")
        x[1, 40:] = 1.0
        x[2, ::3] = -2.0
        x[3, 5] = x[3, 63] = 9.0
        for scoring in ("softmax", "sigmoid"):
            e, _ = check(x, 8, scoring, bias)
            assert e[0].tolist() == list(range(8)) and e[1].tolist() == list(range(40, 48))
            check(x, 8, scoring, bias, groups=8, top_groups=2)


def test_keys_that_32_bits_do_not_tell_apart():
    """Biases that make the keys of neighbours differ by some 2^-30: 32 bits would choose by rounding."""
    rng = random.Random(5)
    E = 128
    for scoring in ("sigmoid", "softmax"):
        x = logits(64, E, torch.float32, 7, 0.5)
        # row 0's scores and the bias add up to nearly the same everywhere
        s = torch.sigmoid(x[0].double()) if scoring == "sigmoid" else torch.softmax(x[0].double(), -1)
        bias = (0.75 - s).float()
        x[1:] = x[0]
        for i in range(1, 64):
            j = rng.randrange(E)
            x[i, j] += rng.choice([-1, 1]) * 2.0**-rng.randint(12, 22)
        check(x, 8, scoring, bias)
        check(x, 4, scoring, bias, groups=16, top_groups=3)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_masked_infinite_and_far_logits(scoring):
    x = logits(12, 64, torch.float32, 9)
    x[0, :] = -math.inf           # nothing left
    x[1, 3:] = -math.inf          # fewer than k left
    x[2, 7] = math.nan
    x[3, [5, 50]] = math.inf
    x[4, :32] = -math.inf         # whole groups out
    x[5] *= 40.0                  # beyond exp's range
    x[6] -= 150.0                 # sigmoids that 32 bits do not hold
    x[7] = torch.finfo(torch.float32).min
    x[8, ::2] = -math.inf
    x[9, 1:] = -1000.0
    bias = torch.linspace(-0.4, 0.4, 64, device="cuda")
    rows = [i for i in range(12) if not (scoring == "sigmoid" and i == 6)]
    for b in (None, bias):
        for groups, top in ((1, 1), (8, 3), (4, 2)):
            check(x[rows], 8, scoring, b, groups, top)
            check(x[rows], 8, scoring, b, groups, top, group_best=1, renormalize=False)
    if scoring == "sigmoid":
        check(x[6:7], 8, scoring)  # ratios of exponentials, whatever their size
    bias[10], bias[11], bias[12] = math.inf, -math.inf, math.nan
    e, w = binding.route_experts(x[rows], 8, scoring, bias=bias)
    assert (e[rows.index(10), 0] == 10) and not bool(((e == 11) | (e == 12))[rows.index(10)].any())
    assert torch.isfinite(w).all()


def test_strided_rows_and_alignment():
    x = logits(40, 200, torch.bfloat16, 11)
    for first in (0, 1, 3, 8):
        check(x[:, first:first + 64], 4)
        check(x.float()[::3, first:first + 96], 8, "sigmoid")


def test_many_tokens():
    """Against the same rows in a small call, which the tests above hold against the formula."""
    x = logits(20000, 128, torch.bfloat16, 13)
    bias = 0.1 * torch.randn(128, device="cuda")
    e, w = binding.route_experts(x, 8, "sigmoid", bias=bias, groups=8, top_groups=4)
    some = torch.arange(0, 20000, 997, device="cuda")
    check(x[some], 8, "sigmoid", bias, 8, 4)
    e1, w1 = binding.route_experts(x[some], 8, "sigmoid", bias=bias, groups=8, top_groups=4)
    assert torch.equal(e[some], e1) and torch.equal(w[some], w1)


def test_no_tokens():
    e, w = binding.route_experts(torch.zeros(0, 16, device="cuda"), 4)
    assert e.shape == (0, 4) and w.shape == (0, 4)


def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    for bad in (dict(k=0), dict(k=33), dict(k=4, groups=5), dict(k=4, groups=64), dict(k=9, groups=8, top_groups=1),
                dict(k=4, groups=8, top_groups=9), dict(k=4, groups=8, top_groups=0), dict(k=4, group_best=3)):
        with pytest.raises(binding.QmmError):
            binding.route_experts(x, **bad)
    with pytest.raises(ValueError):
        binding.route_experts(x, 4, "tanh")
    with pytest.raises(ValueError):
        binding.route_experts(x, -1)
    with pytest.raises(ValueError):
        binding.route_experts(x, 4, bias=torch.zeros(63, device="cuda"))
    with pytest.raises(ValueError):
        binding.route_experts(x.t(), 4)
    with pytest.raises(ValueError):
        binding.route_experts(x.cpu(), 4)
    with pytest.raises(TypeError):
        binding.route_experts(x.half(), 4)
    with pytest.raises(binding.QmmError):
        binding.route_experts(torch.zeros(2, 513, device="cuda"), 4)


def test_feeds_the_gathered_product():
    """The chosen experts' products, weighted: the index list as route_experts leaves it."""
    T, E, k, K, N = 3, 16, 4, 256, 48
    g = torch.Generator(device="cuda").manual_seed(17)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    wq = torch.randint(-2**31, 2**31, (E, N, K // 8), generator=g, device="cuda").to(torch.int32)
    s = (0.01 + 0.01 * torch.rand(E, N, K // 64, generator=g, device="cuda")).half()
    b = (-8 * s.float()).half()
    experts, weights = binding.route_experts(logits(T, E, torch.float32, 19), k)
    lhs = torch.arange(T, dtype=torch.int32, device="cuda").repeat_interleave(k)
    y = binding.gather_small_m(x, wq, s, b, lhs, experts.view(-1), 4, 64, out_dtype=torch.float32)
    for t in range(T):
        for j in range(k):
            e = int(experts[t, j])
            one = binding.small_m(x[t:t + 1], wq[e].contiguous(), s[e].contiguous(), b[e].contiguous(), 4, 64,
                                  out_dtype=torch.float32)
            bound = 1e-3 * (x[t].float().abs().sum() * 0.02 * 8)  # both within 1e-3 of sum |x w|
            assert ((y[t * k + j] - one[0]).abs() <= bound).all()
    assert binding.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_masked_by_the_lowest_value(scoring, dtype):
    """Experts masked by the type's lowest value are off the scale of the others, which keep their order."""
    x = logits(48, 96, dtype, 17)
    x[::2, ::2] = torch.finfo(dtype).min
    x[1::4, 5:] = torch.finfo(dtype).min  # fewer than k left: the lowest numbers of the masked
    x[3] = -math.inf
    x[3, 4] = torch.finfo(dtype).min
    for b in (None, torch.linspace(-0.4, 0.4, 96, device="cuda")):
        check(x, 8, scoring, b)
        check(x, 8, scoring, b, groups=8, top_groups=3, group_best=1, renormalize=False)
