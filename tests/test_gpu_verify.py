"""qmm_verify_draft against its definition in fp64.  Whole numbers are equal wherever no decision of the definition is
closer than 1e-5 (relative): fp32 probabilities are off by a few 1e-7."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu

NEAR = 1e-5


def row(x):
    x = np.where(np.isnan(x), -np.inf, x)
    return x, int(np.argmax(x))


def choose(w, e):
    """(token, whether it is clear) of the largest w/e."""
    r = np.where(w > 0, w / e, 0.0)
    t = int(np.argmax(r))
    second = np.max(np.delete(r, t)) if len(r) > 1 else 0.0
    return t, second < r[t] * (1 - NEAR)


def reference(x, d, q, u, e, T, n_draft):
    """(tokens, accepted, clear) of one sequence."""
    k = len(d)
    n_draft = k if n_draft is None else min(max(n_draft, 0), k)
    clear = True
    for n in range(k + 1):
        z, best = row(x[n])
        drafted = n < n_draft
        if not T > 0 or not np.isfinite(z[best]):
            if drafted and np.isfinite(z[best]) and d[n] == best:
                continue
            return list(d[:n]) + [best], n, clear
        with np.errstate(invalid="ignore"):
            p = np.where(z > -np.inf, np.exp((z - z[best]) / T), 0.0)
        p /= p.sum()
        valid = drafted and 0 <= d[n] < len(p)
        if valid:
            qd = u[n] * (1.0 if q is None else q[n][d[n]])
            clear &= abs(qd - p[d[n]]) > NEAR * p[d[n]]
            if qd < p[d[n]]:
                continue
        if drafted:
            w = p - q[n] if q is not None else np.where(np.arange(len(p)) == d[n], 0.0, p)
            if q is not None:
                # a difference of nearly equal numbers is known to fewer digits
                t, _ = choose(np.maximum(w, 0.0), e)
                if (w > 0).any():
                    clear &= w[t] > 1e-2 * p[t]
            w = np.maximum(w, 0.0)
            if not (w > 0).any():
                w = p
        else:
            w = p
        t, sure = choose(w, e)
        return list(d[:n]) + [t], n, clear and sure


def check(x, d, q, u, e, T, lens=None, need=0.9, **kw):
    """Tensors on the GPU; at least `need` of the sequences must be clear."""
    tokens, accepted = binding.verify_draft(x, d, q, u, e, T, draft_lens=lens, **kw)
    torch.cuda.synchronize()
    tokens, accepted = tokens.cpu().numpy(), accepted.cpu().numpy()
    B, rows, _ = x.shape
    sure = 0
    for b in range(B):
        want, n, clear = reference(x[b].double().cpu().numpy(), d[b].cpu().numpy(),
                                   None if q is None else q[b].double().cpu().numpy(), u[b].double().cpu().numpy(),
                                   e[b].double().cpu().numpy(), float(T[b]), None if lens is None else int(lens[b]))
        sure += clear
        if clear:
            want = want + [-1] * (rows - len(want))
            assert accepted[b] == n and list(tokens[b]) == want, (b, n, want, accepted[b], list(tokens[b]))
    assert sure >= need * B
    return tokens, accepted


def problem(B, k, V, dtype=torch.float32, seed=0, near=0.7, greedy=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 2.5 * torch.randn(B, k + 1, V, generator=g, device="cuda")
    q = torch.softmax(x[:, :k] + near * torch.randn(B, k, V, generator=g, device="cuda"), -1)
    d = (q / torch.empty_like(q).exponential_(generator=g)).argmax(-1).to(torch.int32)
    x = x.to(dtype)
    if greedy:  # half of the drafts are the target's choice
        best = x[:, :k].float().argmax(-1).to(torch.int32)
        d = torch.where(torch.rand(B, k, generator=g, device="cuda") < 0.7, best, d)
    u = torch.rand(B, k, generator=g, device="cuda")
    e = torch.empty(B, V, device="cuda").exponential_(generator=g).clamp_(min=1e-20)
    T = 0.5 + torch.rand(B, generator=g, device="cuda")
    return x, d, q, u, e, torch.zeros_like(T) if greedy else T


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,k,V", [(1, 1, 1), (3, 2, 2), (5, 1, 33), (40, 7, 1000), (8, 5, 32000), (2, 3, 151937),
                                   (70, 4, 517), (300, 1, 64), (3, 31, 257)])
def test_drawn(B, k, V, dtype):
    check(*problem(B, k, V, dtype, seed=V + B), need=0.7)


@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("B,k,V,dtype", [(24, 6, 40000, torch.float32), (24, 5, 70001, torch.bfloat16)])
def test_rows_read_in_turn(B, k, V, dtype, greedy):
    """More than 16 MB of logits: rounds of two rows, the last one of a single row or ending before it."""
    x, d, q, u, e, T = problem(B, k, V, dtype, seed=5, greedy=greedy)
    assert x.numel() * x.element_size() > 16 << 20
    best = x[:, :k].float().argmax(-1).to(torch.int32)
    d = torch.where(torch.rand(B, k, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda") < 0.8, best, d)
    lens = torch.arange(B, device="cuda", dtype=torch.int32) % (k + 1)
    check(x, d, None, u, e, T, need=0.7)
    check(x, d, None, u * 1e-30, e, T, lens, need=0.7)
    check(x, d, None, torch.full_like(u, 0.999999), e, T, need=0.7)


@pytest.mark.parametrize("B,k,V", [(20, 7, 1000), (4, 5, 32001)])
def test_ragged_and_certain_drafts(B, k, V):
    x, d, q, u, e, T = problem(B, k, V, seed=2)
    lens = torch.arange(-1, B - 1, device="cuda", dtype=torch.int32) % (k + 3) - 1
    check(x, d, q, u, e, T, lens, need=0.7)
    check(x, d, None, u, e, T, lens, need=0.7)
    check(x, d, None, u, e, T, need=0.7)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_greedy(dtype):
    x, d, q, u, e, T = problem(40, 6, 5003, dtype, seed=3, greedy=True)
    x[:, :, 4000] = x.float().amax(-1).to(dtype)  # a tie: the lower index wins
    d = torch.where(torch.rand(40, 6, device="cuda") < 0.8, x[:, :6].float().argmax(-1).to(torch.int32), d)
    _, accepted = check(x, d, q, u, e, T, need=1.0)
    check(x, d, None, u, e, -torch.ones_like(T), need=1.0)
    assert accepted.max() > 0


def test_mixed_temperatures():
    x, d, q, u, e, T = problem(30, 4, 999, seed=4)
    T[::3] = 0.0
    T[1] = float("nan")
    check(x, d, q, u, e, T, need=0.7)


def test_everything_accepted_or_refused():
    x, d, q, u, e, T = problem(16, 5, 3001, seed=5)
    _, accepted = check(x, d, q, torch.zeros_like(u), e, T, need=0.7)
    assert (accepted == 5).all()
    x2 = x.clone()
    for b in range(16):
        x2[b, 0, int(d[b, 0])] = -float("inf")
    _, accepted = check(x2, d, q, u, e, T, need=0.7)
    assert (accepted == 0).all()


def test_equal_distributions():
    """q = p bit for bit in the definition's eyes: all accepted with u < 1; nothing is left if one were refused."""
    x, d, q, u, e, T = problem(8, 3, 64, seed=6)
    q = torch.zeros_like(q)
    q.scatter_(2, d.long()[..., None], 1.0)
    x = torch.full_like(x, -float("inf"))
    x[:, :3].scatter_(2, d.long()[..., None], 0.0)
    x[:, 3, 5] = 1.0
    tokens, accepted = binding.verify_draft(x, d, q, u * 0.99, e, T)
    assert (accepted == 3).all() and (tokens[:, 3] == 5).all()
    tokens, accepted = binding.verify_draft(x, d, q, torch.ones_like(u), e, T)  # u = 1: refused, and p - q = 0
    assert (accepted == 0).all() and torch.equal(tokens[:, 0], d[:, 0])


def test_unusable_rows_and_nan():
    x, d, q, u, e, T = problem(7, 3, 300, seed=7)
    x[0, 0] = -float("inf")
    x[1, 1] = float("nan")
    x[2, 0, 17] = float("inf")
    x[2, 0, 11] = float("inf")
    x[3, 0, 5:250] = float("nan")
    x[4, :, ::2] = -float("inf")
    x[5, 3] = float("nan")
    check(x, d, q, u, e, T, need=0.5)
    check(x, d, q, u, e, torch.zeros_like(T), need=0.5)


def test_drafts_outside_the_vocabulary():
    x, d, q, u, e, T = problem(6, 3, 300, seed=8)
    d[0, 0], d[1, 0], d[2, 0] = -1, 300, 2**31 - 1
    for qq in (q, None):
        tokens, accepted = check(x, d, qq, u, e, T, need=0.5)
        assert (accepted[:3] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_offsets_streams(dtype):
    """Rows further apart than V, at an odd offset; another stream."""
    x, d, q, u, e, T = problem(5, 3, 1001, dtype, seed=9)
    pad = torch.full((5, 4, 1111), float("nan"), device="cuda").to(dtype)
    view = pad[:, :, 7:1008]
    view.copy_(x)
    a = check(x, d, q, u, e, T, need=0.5)
    b = check(view, d, q, u, e, T, need=0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = check(view, d, q, u, e, T, need=0.5, stream=side)
    for other in (b, c):
        assert np.array_equal(a[0], other[0]) and np.array_equal(a[1], other[1])


def test_no_drafts():
    x, d, q, u, e, T = problem(4, 1, 700, seed=10)
    x = x[:, :1].contiguous()
    tokens, accepted = check(x, d[:, :0].contiguous(), q[:, :0].contiguous(), u[:, :0].contiguous(), e, T, need=0.5)
    assert (accepted == 0).all() and tokens.shape == (4, 1)


def test_repeats_are_equal():
    args = problem(30, 5, 20000, torch.bfloat16, seed=11)
    first = binding.verify_draft(*args)
    for _ in range(3):
        again = binding.verify_draft(*args)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_acceptance_follows_the_probabilities():
    """Over many sequences the next token of a refused or accepted draft is distributed as the target's p."""
    V, B = 8, 60000
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.tensor([0.3, -1.0, 0.8, 0.0, 1.2, -0.5, 0.1, 0.4], device="cuda").expand(B, 2, V).contiguous()
    q1 = torch.softmax(torch.tensor([1.0, 0.0, 0.2, -0.3, 0.1, 0.9, -2.0, 0.0], device="cuda"), -1)
    q = q1.expand(B, 1, V).contiguous()
    d = (q / torch.empty_like(q).exponential_(generator=g)).argmax(-1).to(torch.int32)
    u = torch.rand(B, 1, generator=g, device="cuda")
    e = torch.empty(B, V, device="cuda").exponential_(generator=g).clamp_(min=1e-20)
    tokens, _ = binding.verify_draft(x, d, q, u, e, torch.ones(B, device="cuda"))
    freq = torch.bincount(tokens[:, 0].long(), minlength=V).double() / B
    p = torch.softmax(x[0, 0].double(), -1)
    assert ((freq - p).abs() <= 5 * (p * (1 - p) / B).sqrt()).all()  # five standard deviations


def test_refusals():
    x, d, q, u, e, T = problem(4, 3, 100)
    with pytest.raises(TypeError):
        binding.verify_draft(x.half(), d, q, u, e, T)
    with pytest.raises(ValueError):
        binding.verify_draft(x, d.long(), q, u, e, T)
    with pytest.raises(ValueError):
        binding.verify_draft(x, d, q[:, :2], u, e, T)
    with pytest.raises(ValueError):
        binding.verify_draft(x, d, q, u, e[:, :50], T)
    with pytest.raises(ValueError):
        binding.verify_draft(x.transpose(1, 2), d, q, u, e, T)
    with pytest.raises(ValueError):
        binding.verify_draft(x.cpu(), d, q, u, e, T)
    y, d2, q2, u2, e2, T2 = problem(1, 32, 40)
    with pytest.raises(binding.QmmError):
        binding.verify_draft(y, d2, q2, u2, e2, T2)
