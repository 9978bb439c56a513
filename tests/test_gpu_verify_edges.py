"""qmm_verify_draft at the ends of its arguments' ranges."""
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding
from test_gpu_verify import check, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [0, 3])
@pytest.mark.parametrize("T", [1e-30, 1e-38, 4.4e-39, 4.1e-39, 1e-39, 1e-40, 1.5e-45])
def test_small_temperatures(T, k):
    """All the weight on the largest logit, down to the smallest denormal: log2(e) / T passes fp32's range on the way."""
    x, d, q, u, e, t = problem(12, max(k, 1), 900, seed=20)
    x, d, q, u = x[:, :k + 1].contiguous(), d[:, :k].contiguous(), q[:, :k].contiguous(), u[:, :k].contiguous()
    best = x.argmax(-1)
    if k:
        d[::2, 0] = best[::2, 0].int()  # accepted wherever they are offered and uniform * q < 1
    t = torch.full_like(t, T)
    assert (t > 0).all()
    none = torch.zeros(12, dtype=torch.int32, device="cuda")
    for qq, lens in ((q, None), (None, None), (q, none), (None, none)):
        tokens, accepted = check(x, d, qq, u, e, t, lens, need=0.9)
        assert (tokens[:, 0] >= 0).all() and (tokens < 900).all()
        if k and lens is None:
            assert (accepted[::2] >= 1).all()


@pytest.mark.parametrize("V", [5, 900, 40001])
def test_noise_that_is_no_positive_number(V):
    """Counts as +inf: where all of a row is, the lowest token with a weight is taken; else one whose noise is a number."""
    x, d, q, u, e, t = problem(9, 3, V, seed=21)
    none = torch.zeros(9, dtype=torch.int32, device="cuda")
    nan, inf = float("nan"), float("inf")
    e[0], e[1], e[2] = nan, -1.0, inf
    e[3, ::2], e[4, 1:], e[5, 1:] = nan, nan, -0.5
    as_inf = torch.where(e >= 0, e, inf)
    for qq, uu, lens in ((q, u, None), (q, torch.full_like(u, 0.999999), None), (None, u, None), (q, u, none), (None, u, none)):
        tokens, accepted = binding.verify_draft(x, d, qq, uu, e, t, draft_lens=lens)
        again = binding.verify_draft(x, d, qq, uu, as_inf, t, draft_lens=lens)
        assert torch.equal(tokens, again[0]) and torch.equal(accepted, again[1])
        last = tokens.gather(1, accepted[:, None].long())[:, 0]
        assert ((last >= 0) & (last < V)).all(), last
        if lens is not None:
            assert (last[:3] == 0).all() and (last[3] % 2 == 1 if V > 5 else True) and (last[4:6] == 0).all()
