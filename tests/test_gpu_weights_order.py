"""Weights made by one call and read by the next on the stream, with nothing in between: the products copy weights ahead of
their wait for the preceding kernel, so the kernels that write weights complete before their dependents start."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
@pytest.mark.parametrize("M", [1, 8, 16])
@pytest.mark.parametrize("N,K", [(48, 64), (256, 1024), (5120, 5120), (1000, 4128)])
def test_quantised_weights(N, K, M, fmt):
    """Two matrices in turn through one buffer of codes and scales; a wrong order would read the other one's."""
    g = torch.Generator(device="cuda").manual_seed(N + M)
    ws = [torch.randn(N, K, generator=g, device="cuda").bfloat16() for _ in range(2)]
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    want = []
    for w in ws:
        codes, scales = binding.quantize_mx(w, fmt)
        torch.cuda.synchronize()
        want.append(binding.small_m_mx(x, codes, scales, fmt))
    torch.cuda.synchronize()
    n = 40
    ys = torch.zeros(n, *want[0].shape, device="cuda", dtype=want[0].dtype)
    out = torch.empty_like(codes), torch.empty_like(scales)
    torch.cuda.synchronize()
    for i in range(n):
        binding.quantize_mx(ws[i & 1], fmt, out=out)
        binding.small_m_mx(x, *out, fmt, out=ys[i])
    torch.cuda.synchronize()
    for i in range(n):
        assert torch.equal(ys[i], want[i & 1]), i


def test_a_call_between():
    """The product that reads the weights starts while the one before it still waits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    N = K = 2048
    ws = [torch.randn(N, K, generator=g, device="cuda").bfloat16() for _ in range(3)]
    x = torch.randn(4, K, generator=g, device="cuda").bfloat16()
    first = binding.quantize_mx(ws[2], "mxfp4")
    torch.cuda.synchronize()
    want = []
    for w in ws[:2]:
        q = binding.quantize_mx(w, "mxfp4")
        torch.cuda.synchronize()
        want.append(binding.small_m_mx(binding.small_m_mx(x, *first, "mxfp4"), *q, "mxfp4"))
    torch.cuda.synchronize()
    out = torch.empty_like(q[0]), torch.empty_like(q[1])
    mid = torch.empty_like(want[0])
    ys = torch.zeros(40, *mid.shape, device="cuda", dtype=mid.dtype)
    torch.cuda.synchronize()
    for i in range(40):
        binding.quantize_mx(ws[i & 1], "mxfp4", out=out)
        binding.small_m_mx(x, *first, "mxfp4", out=mid)
        binding.small_m_mx(mid, *out, "mxfp4", out=ys[i])
    torch.cuda.synchronize()
    for i in range(40):
        assert torch.equal(ys[i], want[i & 1]), i


@pytest.mark.parametrize("kind", ["q4_0", "q4_1", "q8_0"])
def test_converted_weights(kind):
    N, K = 1024, 2048
    blocks = [torch.from_numpy(synth.make_ggml_blocks(seed, N, K, kind).reshape(-1)).cuda() for seed in (1, 2)]
    x = torch.from_numpy(synth.make_x(5, K)[:4].copy().view(np.int16)).cuda().view(torch.bfloat16)
    want, ys = [], []
    for b in blocks:
        wq, s, z, bits = binding.from_ggml(kind, b, N, K)
        torch.cuda.synchronize()
        want.append(binding.small_m(x, wq, s, z, bits, 32))
    torch.cuda.synchronize()
    for i in range(20):
        wq, s, z, bits = binding.from_ggml(kind, blocks[i & 1], N, K)
        ys.append(binding.small_m(x, wq, s, z, bits, 32))
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        assert torch.equal(y, want[i & 1]), i
