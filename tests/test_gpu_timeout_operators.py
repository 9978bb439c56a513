"""A bounded wait of the operators around the product that runs out, without a GPU fault: with QMM_TEST_INJECT=short_wait a
barrier waits for 16 bytes more than its copies bring, for 100 us.  All copies land; the call returns with a status bit,
and the next one is right."""
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding
import test_gpu_matmul_mx as mx
from test_gpu_paged import Cache, check, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("D,M,Hq,lens", [(128, 1, 8, [40000]), (128, 8, 8, [300, 41]), (64, 4, 16, [900] * 3), (256, 2, 4, [5000])])
def test_attention(monkeypatch, D, M, Hq, lens, dtype):
    """The worker of the list's first piece gives up on it, waits for the others that it has asked for, and asks for no more."""
    c = Cache(lens, 2, D, 16, dtype, seed=7)
    q = queries(len(lens), M, Hq, D)
    want, _ = check(c, q)
    monkeypatch.setenv("QMM_TEST_INJECT", "short_wait")
    out = binding.paged_attention(q, *c.args())
    torch.cuda.synchronize()
    assert binding.device_status() == 1
    assert out.shape == want.shape
    monkeypatch.delenv("QMM_TEST_INJECT")
    again, _ = check(c, q)
    assert torch.equal(again, want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(8, 300, 1024), (4, 1000, 512), (200, 256, 1024)])
def test_matmul(monkeypatch, M, N, K, fmt):
    """The first CTA's products wait in vain for their first stage (which no later one uses again); so does the end of its
    copies."""
    x, w = mx.matrix(M, K, fmt, 1), mx.matrix(N, K, fmt, 2)
    want = mx.check(x, w, fmt, torch.float32)
    monkeypatch.setenv("QMM_TEST_INJECT", "short_wait")
    y = binding.matmul_mx(*x, *w, fmt, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert binding.device_status() == 1 | 4
    assert y.shape == want.shape
    monkeypatch.delenv("QMM_TEST_INJECT")
    assert torch.equal(mx.check(x, w, fmt, torch.float32), want)
