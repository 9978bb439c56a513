"""qmm_quantize_mx against the formats' definition in numpy: codes, scale bytes
and values are equal bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8 * 2.0**-6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest(a, grid):
    """Index of the nearest of the ascending magnitudes, ties to the even index, beyond the last to the last."""
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    mid = 0.5 * (grid[hi - 1] + grid[hi])
    return np.where((a > mid) | ((a == mid) & (hi % 2 == 0)), hi, hi - 1)


def bf16_round(v):
    """Nearest even into bf16, returned as the 16-bit patterns of a torch CPU tensor."""
    return torch.from_numpy(v).to(torch.float32).to(torch.bfloat16)


def reference(x, fmt):
    """(codes [R, K], scale bytes [R, K/g], values [R, K] fp64) of x (fp64 values of the inputs)."""
    _, bits, g = binding.MX_FORMATS[fmt]
    grid = E4M3 if bits == 8 else E2M1
    R, K = x.shape
    x = x.reshape(R, K // g, g)
    bad = ~np.isfinite(x).all(-1)
    clean = np.where(bad[..., None], 0.0, x)
    a = np.abs(clean).max(-1)
    if fmt == "nvfp4":
        byte = nearest((a.astype(np.float32) / np.float32(6)).astype(np.float64), E4M3)
        s = E4M3[byte]
        byte = np.where(bad, 0x7F, byte)
    else:
        e = np.where(a > 0, np.frexp(np.where(a > 0, a, 1.0))[1] - 1, -1000) - (8 if bits == 8 else 2)
        byte = np.clip(e + 127, 0, 254)
        s = np.ldexp(1.0, byte - 127)
        byte = np.where(bad, 255, byte)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s[..., None] > 0, clean / s[..., None], 0.0)
    mag = nearest(np.abs(y), grid)
    neg = np.signbit(x) & ~bad[..., None]
    codes = np.where(bad[..., None], 0, mag + neg * (1 << (bits - 1)))
    values = np.where(bad[..., None], np.nan, np.where(neg, -1.0, 1.0) * grid[mag] * s[..., None])
    return codes.reshape(R, K), byte.astype(np.uint8), values.reshape(R, K)


def check(x, fmt, **kw):
    """x: a CUDA tensor [R, K]."""
    values = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
    codes, scales = binding.quantize_mx(x, fmt, values=values, **kw)
    torch.cuda.synchronize()
    bits = binding.MX_FORMATS[fmt][1]
    rc, rs, rv = reference(x.double().cpu().numpy(), fmt)
    got = binding.unpack(codes.cpu().numpy().view(np.uint32), x.shape[1], bits)
    assert np.array_equal(scales.cpu().numpy(), rs), fmt
    assert np.array_equal(got, rc), fmt
    want = bf16_round(rv)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(values.cpu()), nan)
    assert torch.equal(values.cpu().view(torch.int16)[~nan], want.view(torch.int16)[~nan]), fmt
    return codes, scales


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
@pytest.mark.parametrize("shape", [(1, 32), (3, 32), (7, 96), (129, 160), (33, 4128), (1000, 544)])
def test_random(shape, fmt, dtype):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    x = torch.randn(shape, generator=g, device="cuda") * torch.exp(3 * torch.randn(shape[1], generator=g, device="cuda"))
    check(x.to(dtype), fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
def test_ties_and_every_scale(fmt):
    """Rows of every binade of bf16, each element a multiple of 1/16 of the largest: quotients meet the midpoints."""
    e = torch.arange(-133, 128, device="cuda", dtype=torch.float64)
    base = torch.tensor([1.0, 1.125, 1.25, 1.5, 1.75, 1.9921875], dtype=torch.float64, device="cuda")
    top = (base[None, :] * torch.exp2(e)[:, None]).reshape(-1, 1)
    step = torch.arange(32, device="cuda", dtype=torch.float64) / 16 - 1
    x = (top * step).to(torch.float32).to(torch.bfloat16)
    check(x, fmt)
    check(x.float(), fmt)


@pytest.mark.parametrize("fmt", ["nvfp4"])
def test_fp32_next_to_ties(fmt):
    """fp32 inputs one unit in the last place beside midpoint * scale."""
    s = torch.tensor(E4M3[8:120], dtype=torch.float32, device="cuda")
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    m = (s[:, None] * mids).repeat(1, 2)
    x = torch.cat([6 * s[:, None], m, torch.zeros_like(s)[:, None]], 1)
    up = torch.nextafter(x, torch.full_like(x, float("inf")))
    down = torch.nextafter(x, torch.zeros_like(x))
    up[:, 0] = down[:, 0] = 6 * s
    check(torch.cat([torch.cat([up, -down], 1), torch.cat([x, down], 1)]), fmt)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
def test_special_values(fmt, dtype):
    x = torch.randn(12, 64, generator=torch.Generator().manual_seed(5))
    x[0] = 0.0
    x[1] = -0.0
    x[2, 3] = float("nan")
    x[3, 40] = float("inf")
    x[4, 0] = -float("inf")
    x[5] *= 1e-38
    x[6] *= 1e-40
    x[7] *= 3e37
    x[8] = torch.where(torch.arange(64) % 2 == 0, -1e-30, 1.0)
    x[9, ::16] = 3e38
    x[10] *= 2.0**-9
    x[11] *= 1e-3
    check(x.to(dtype).cuda(), fmt)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "mxfp8"])
def test_strides_and_offsets(fmt, dtype):
    """Rows at any distance, first element at any element offset."""
    g = torch.Generator(device="cuda").manual_seed(3)
    flat = torch.randn(40000, generator=g, device="cuda").to(dtype)
    for ld, off in ((96, 1), (97, 0), (104, 8), (200, 3), (112, 2)):
        check(torch.as_strided(flat, (101, 96), (ld, 1), off), fmt)


def test_other_stream_and_given_outputs():
    x = torch.randn(257, 1024, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    out = torch.full((257, 128), -1, dtype=torch.int32, device="cuda"), torch.zeros(257, 64, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    codes, scales = check(x, "nvfp4", out=out, stream=side)
    assert codes is out[0] and scales is out[1]
    check(x, "nvfp4", stream=side.cuda_stream)


def test_feeds_the_product():
    """Codes and scales are what small_m_mx reads: X = I picks out the values."""
    w = torch.randn(48, 64, device="cuda").to(torch.bfloat16)
    for fmt in ("mxfp4", "nvfp4", "mxfp8"):
        values = torch.empty_like(w)
        codes, scales = binding.quantize_mx(w, fmt, values=values)
        eye = torch.eye(64, device="cuda").to(torch.bfloat16)
        y = torch.cat([binding.small_m_mx(eye[i:i + 16].contiguous(), codes, scales, fmt) for i in range(0, 64, 16)])
        assert torch.equal(y.t(), values), fmt


def test_refusals():
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.quantize_mx(x.half(), "mxfp4")
    with pytest.raises(ValueError):
        binding.quantize_mx(x[:, :48].contiguous(), "mxfp4")
    with pytest.raises(ValueError):
        binding.quantize_mx(x.t(), "mxfp4")
    with pytest.raises(ValueError):
        binding.quantize_mx(x, "mxfp4", values=torch.empty(4, 64, device="cuda"))
    with pytest.raises(ValueError):
        binding.quantize_mx(x.cpu(), "mxfp4")
    with pytest.raises(KeyError):
        binding.quantize_mx(x, "fp4")
    codes, scales = binding.quantize_mx(x[:0], "mxfp4")
    assert codes.shape == (0, 8) and scales.shape == (0, 2)
