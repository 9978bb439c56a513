"""qmm_verify_draft at the ends of its arguments' ranges."""
import pytest

torch = pytest.importorskip("torch")

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
