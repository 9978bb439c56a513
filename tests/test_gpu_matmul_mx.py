"""qmm_matmul_mx against fp64 products of the decoded matrices.

Products of codes and scales are exact and sums are fp32 in an order that is
not fixed by the definition, in at most K/16 + 64 roundings or truncations of
partial sums bounded by A = sum |x w|: |y - y_ref| <= (K/16 + 64) 2^-23 A, where
A is within fp32's range.  A bf16 output adds half a unit in its last place."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from qmm_harness import bf16_half_ulp
from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
VALUES = torch.cat([VALUES, -VALUES])


def matrix(rows, K, fmt, seed, lo=None, hi=None):
    g = 16 if fmt == "nvfp4" else 32
    r = np.random.default_rng(seed)
    codes = torch.from_numpy(r.integers(0, 2**32, (rows, K // 8), dtype=np.uint32).view(np.int32)).cuda()
    lo, hi = (lo, hi) if lo is not None else ((0x18, 0x48) if fmt == "nvfp4" else (118, 130))
    return codes, torch.from_numpy(r.integers(lo, hi, (rows, K // g), dtype=np.uint8)).cuda()


def decode(codes, scales, fmt):
    place = torch.arange(8, device="cuda", dtype=torch.int32) * 4
    c = ((codes[..., None] >> place) & 15).reshape(codes.shape[0], scales.shape[1], -1)
    s = scales.view(torch.float8_e4m3fn).double() if fmt == "nvfp4" else torch.exp2(scales.double() - 127)
    if fmt != "nvfp4":
        s[scales == 255] = float("nan")
    return (VALUES.cuda()[c.long()] * s[..., None]).reshape(codes.shape[0], -1)


def check(x, w, fmt, out_dtype, **kw):
    y = binding.matmul_mx(*x, *w, fmt, out_dtype=out_dtype, **kw)
    torch.cuda.synchronize()
    xv, wv = decode(*x, fmt), decode(*w, fmt)
    ref, scale = xv @ wv.t(), xv.abs() @ wv.abs().t()
    K = xv.shape[1]
    err = (y.double() - ref).abs().cpu().numpy()
    bound = (K / 16 + 64) * 2.0**-23 * scale.cpu().numpy()
    if out_dtype == torch.bfloat16:
        bound = bound + bf16_half_ulp(y.double().cpu().numpy())
    bound[~(scale < 3e38).cpu().numpy()] = np.inf  # sums of magnitudes past fp32's range: anything may come out
    err = np.nan_to_num(err, nan=np.inf)
    assert y.dtype == out_dtype and np.all(err <= bound), (fmt, tuple(y.shape), K, float((err - bound).max()))
    assert binding.device_status() == 0
    return y


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 100, 128, 129, 200, 256, 257, 500])
def test_rows(M, fmt):
    N, K = 392, 1056
    check(matrix(M, K, fmt, M), matrix(N, K, fmt, 1000 + M), fmt, torch.float32)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("N,K", [(1, 32), (2, 64), (127, 96), (128, 128), (129, 160), (130, 256), (255, 288), (257, 544),
                                 (300, 2048), (33, 5120), (640, 8160)])
def test_columns_and_lengths(N, K, fmt, out_dtype):
    for M in (5, 70, 300):
        check(matrix(M, K, fmt, N + K), matrix(N, K, fmt, N * K + 1), fmt, out_dtype)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_many_tiles(fmt):
    check(matrix(700, 512, fmt, 1), matrix(20011, 512, fmt, 2), fmt, torch.bfloat16)
    check(matrix(3001, 320, fmt, 3), matrix(1500, 320, fmt, 4), fmt, torch.bfloat16)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("K", [512, 768, 1536, 2560])
def test_stages_of_a_tile(K, fmt):
    """Several tiles a CTA, of 2, 3, 6 and 10 stages; scales that start where a pair of stages may, and where not."""
    x, w = matrix(700, K, fmt, K), matrix(20011, K, fmt, K + 1)
    y = check(x, w, fmt, torch.bfloat16)
    for step in (1, 8, 16):
        moved = torch.zeros(x[1].numel() + 16, dtype=torch.uint8, device="cuda")[step:step + x[1].numel()].view(x[1].shape)
        moved.copy_(x[1])
        assert torch.equal(binding.matmul_mx(x[0], moved, *w, fmt), y)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_scale_range(fmt):
    """Small and large scales, the subnormal ones among them."""
    lo, hi = (0, 0x7F) if fmt == "nvfp4" else (64, 190)
    check(matrix(40, 256, fmt, 1, lo, hi), matrix(150, 256, fmt, 2, lo, hi), fmt, torch.float32)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_nan_scales_stay_in_their_row(fmt):
    x, w = matrix(20, 512, fmt, 5), matrix(200, 512, fmt, 6)
    x[1][3, 2] = 0x7F if fmt == "nvfp4" else 255
    w[1][150, 1] = 0x7F if fmt == "nvfp4" else 255
    y = binding.matmul_mx(*x, *w, fmt, out_dtype=torch.float32)
    want = torch.zeros(20, 200, dtype=torch.bool, device="cuda")
    want[3], want[:, 150] = True, True
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(4, 256, 4096), (200, 300, 1024)])
def test_repeats_are_equal_and_nothing_else_is_written(M, N, K, fmt):
    x, w = matrix(M, K, fmt, 7), matrix(N, K, fmt, 8)
    y0 = check(x, w, fmt, torch.float32)
    buf = torch.full((M * N + 512,), 7.5, device="cuda")
    out = buf[256:256 + M * N].view(M, N)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.matmul_mx(*x, *w, fmt, out=out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, y0)
    assert (buf[:256] == 7.5).all() and (buf[256 + M * N:] == 7.5).all()


def test_agrees_with_the_few_row_product():
    """The same weights through small_m_mx with the activations' values."""
    x = torch.randn(16, 2048, device="cuda").to(torch.bfloat16)
    w = torch.randn(512, 2048, device="cuda").to(torch.bfloat16)
    for fmt in ("mxfp4", "nvfp4"):
        values = torch.empty_like(x)
        xq = binding.quantize_mx(x, fmt, values=values)
        wq = binding.quantize_mx(w, fmt)
        a = check(xq, wq, fmt, torch.float32)
        b = binding.small_m_mx(values, *wq, fmt, out_dtype=torch.float32)
        scale = decode(*xq, fmt).abs() @ decode(*wq, fmt).abs().t()
        assert ((a - b).abs() <= 1e-4 * scale).all()


def test_in_a_graph():
    x, w = matrix(48, 1024, "nvfp4", 9), matrix(640, 1024, "nvfp4", 10)
    y0 = check(x, w, "nvfp4", torch.bfloat16)
    out = torch.zeros_like(y0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.matmul_mx(*x, *w, "nvfp4", out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y0)


def test_refusals():
    x, w = matrix(4, 64, "mxfp4", 1), matrix(8, 64, "mxfp4", 2)
    with pytest.raises(ValueError):
        binding.matmul_mx(*x, *w, "mxfp8")
    with pytest.raises(ValueError):
        binding.matmul_mx(*x, *w, "nvfp4")  # scales of the wrong group size
    with pytest.raises(ValueError):
        binding.matmul_mx(x[0], x[1][:, :1], *w, "mxfp4")
    with pytest.raises(TypeError):
        binding.matmul_mx(*x, *w, "mxfp4", out_dtype=torch.float16)
    with pytest.raises(ValueError):
        binding.matmul_mx(*x, *w, "mxfp4", out=torch.empty(8, 4, device="cuda"))
    assert binding.matmul_mx(x[0][:0], x[1][:0], *w, "mxfp4").shape == (0, 8)
    assert (binding.matmul_mx(x[0][:, :0], x[1][:, :0], w[0][:, :0], w[1][:, :0], "mxfp4") == 0).all()
