"""Adapters beside a projection against the formula in fp64.

Bounds: h = A x is an fp32 sum of K exact products, off by at most (K + 8) 2^-24 sum|a x|; it enters the second product with
16 bits (2^-16) where y is bf16 and 24 (2^-23 with its scale's rounding) where y is fp32; that one's R products and the base
add (R + 8) 2^-24 of their sizes, y its rounding, 2^-8 (bf16) or 2^-24 relative."""
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu


def problem(ids, L, R, K, N, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = len(ids)

    def randn(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)

    return dict(base=randn(T, N).to(dtype), x=randn(T, K), a=randn(L, R, K, std=max(K, 1)**-0.5), b=randn(L, N, R, std=R**-0.5),
                adapters=torch.tensor(ids, dtype=torch.int32, device="cuda"),
                scales=0.5 + torch.rand(L, generator=g, device="cuda"))


def check(p, **more):
    base = p["base"].clone()
    got = binding.lora_add(**p, **more)
    torch.cuda.synchronize()
    T, N = base.shape
    L, R, K = p["a"].shape
    f32 = base.dtype == torch.float32
    want, bound = base.double(), torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for i in range(L):
        t = torch.nonzero(p["adapters"] == i)[:, 0]
        if len(t) == 0:
            continue
        x, a, b = p["x"][t].double(), p["a"][i].double(), p["b"][i].double()
        s = 1.0 if p["scales"] is None else float(p["scales"][i].double())
        h, size = x @ a.t(), x.abs() @ a.abs().t()
        dh = abs(s) * ((K + 8) * 2.0**-24 * size + (2.0**-23 if f32 else 2.0**-16) * h.abs())
        want[t] += s * (h @ b.t())
        bound[t] = dh @ b.abs().t() + (R + 8) * 2.0**-24 * (abs(s) * (h.abs() @ b.abs().t()) + base[t].double().abs())
        bound[t] += (2.0**-24 if f32 else 2.0**-8) * want[t].abs()
    assert got.dtype == base.dtype
    assert ((got.double() - want).abs() <= bound).all(), float(((got.double() - want).abs() - bound).max())
    alone = p["adapters"] < 0
    assert torch.equal(got[alone], base[alone])
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,K,N", [(8, 64, 48), (16, 256, 1), (24, 136, 77), (64, 5120, 640), (128, 1024, 1000), (40, 8, 33),
                                   (16, 2056, 4099), (8, 4096, 8200)])
def test_formula(R, K, N, dtype):
    check(problem([2, 0, 0, -1, 1, 2, 2], 3, R, K, N, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [[1], [1] * 9, [16, 3, 17], [64, 65, 63, 1], [200, 1, 1, 130], [5] * 40, [300] * 4, [2000, 3]])
def test_requests(rows, dtype):
    """Rows of requests one after another, on adapters that some share."""
    ids = [(-1 if r % 5 == 4 else r * 3 % 7) for r, n in enumerate(rows) for _ in range(n)]
    check(problem(ids, 7, 16, 320, 272, dtype, seed=len(ids)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R", [16, 24, 32, 64, 96, 128])
def test_many_rows_an_adapter(R, dtype):
    """Tiles of 16, 32 or 64 rows, full and not."""
    check(problem([0] * 130 + [-1] * 40 + [1] * 65 + [2] * 3 + [0] * 31, 3, R, 448, 600, dtype, seed=R))


@pytest.mark.parametrize("T,L", [(50, 64), (333, 5), (1500, 100), (5000, 40), (700, 1), (600, 5000)])
def test_rows_in_any_order(T, L):
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, L, (T,), generator=g).tolist()
    check(problem(ids, L, 32, 192, 200, seed=1))


def test_no_adapter_at_all():
    for ids in ([-1] * 5, [-7] * 300, [-2**31, -1]):
        check(problem(ids, 2, 16, 64, 100))


def test_no_adapters_loaded():
    p = problem([-1, -1], 1, 16, 64, 100)
    p["a"], p["b"], p["scales"] = p["a"][:0], p["b"][:0], p["scales"][:0]
    got = binding.lora_add(**p)
    assert torch.equal(got, p["base"])


def test_a_number_out_of_range_counts_as_none():
    p = problem([0, 1, 0], 2, 16, 64, 100)
    want = check(p)
    p["adapters"][1] = 2
    got = binding.lora_add(**p)
    torch.cuda.synchronize()
    assert binding.device_status() == 8
    assert torch.equal(got[1], p["base"][1]) and torch.equal(got[[0, 2]], want[[0, 2]])
    ids = [0] * 400 + [2**31 - 1] + [1] * 100
    p = problem([max(0, min(i, 1)) for i in ids], 2, 16, 64, 100)
    want = check(p)
    p["adapters"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    got = binding.lora_add(**p)
    torch.cuda.synchronize()
    assert binding.device_status() == 8
    assert torch.equal(got[400], p["base"][400]) and torch.equal(got[:400], want[:400]) and torch.equal(got[401:], want[401:])


def test_without_scales_and_a_sum_of_no_products():
    p = problem([0, 1, -1], 2, 8, 64, 100)
    p["scales"] = None
    check(p)
    p = problem([0, 1, -1], 2, 8, 0, 100)
    assert torch.equal(binding.lora_add(**p), p["base"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ids", [[1, 0, -1, 1], [0] * 70 + [-1] * 9 + [1] * 200])
def test_in_place_and_strided(ids, dtype):
    """One part of a fused projection's columns, updated where it is; the other columns stay."""
    p = problem(ids, 2, 16, 128, 200, dtype)
    want = check(p)
    T = len(ids)
    for first, width in ((0, 200), (3, 333), (8, 300)):
        wide = torch.full((T, first + width), 5.0, device="cuda").to(dtype)
        part = wide[:, first:first + 200]
        part.copy_(p["base"])
        x = torch.full((T, 160), float("nan"), device="cuda").to(torch.bfloat16)
        x[:, 16:144] = p["x"]
        q = {**p, "base": part, "x": x[:, 16:144]}
        got = binding.lora_add(**q, out=part)
        assert got.data_ptr() == part.data_ptr() and torch.equal(got, want)
        assert (wide[:, :first] == 5.0).all() and (wide[:, first + 200:] == 5.0).all()
        # and out of a strided base into rows of its own
        part.copy_(p["base"])
        assert torch.equal(binding.lora_add(**q), want)


def test_what_is_not_finite_stays_in_its_row():
    p = problem([0, 1, 0, -1], 2, 16, 128, 100)
    want = check(p)
    p["x"][1, 7] = float("nan")
    p["x"][3] = float("nan")  # no adapter: not read
    got = binding.lora_add(**p)
    assert torch.isnan(got[1]).all() and torch.equal(got[[0, 2, 3]], want[[0, 2, 3]])
    p = problem([0, 1, 0, 1], 2, 16, 128, 100)
    want = check(p)
    p["a"][0] = float("inf")
    p["b"][0, 50] = float("nan")
    got = binding.lora_add(**p)
    assert torch.equal(got[[1, 3]], want[[1, 3]])


def test_some_of_the_rows():
    """The same rows with more or fewer others, which changes how they are tiled, and repeated exactly."""
    p = problem([0, 1, 2, 0, 1, 1] * 60, 3, 32, 512, 300, seed=3)
    want = check(p)
    assert torch.equal(binding.lora_add(**p), want)
    for rows in ([0], [5], list(range(3)), list(range(100, 290))):
        check({**p, "base": p["base"][rows], "x": p["x"][rows], "adapters": p["adapters"][rows]})


def test_workspace():
    """One that is reused, holding NaN."""
    for T in (7, 300):
        p = problem([0, 1, -1, 1, 0, 2, 1] * (T // 7), 3, 16, 512, 300, torch.float32, seed=4)
        want = check(p)
        ws = torch.full((binding.lora_workspace(len(p["x"]), 3, 16),), 255, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            assert torch.equal(binding.lora_add(**p, workspace=ws), want)
        with pytest.raises(binding.QmmError):
            binding.lora_add(**p, workspace=ws[:-256])


def test_refusals():
    p = problem([0, 1, -1], 2, 16, 64, 100)
    dev = dict(device="cuda")
    for bad, kind in ((dict(a=p["a"][:, :12], b=p["b"][..., :12].contiguous()), ValueError), (dict(b=p["b"][:1]), ValueError),
                      (dict(a=p["a"][:, :4].contiguous(), b=p["b"][..., :4].contiguous()), binding.QmmError),
                      (dict(a=torch.zeros(2, 136, 64, **dev).bfloat16(), b=torch.zeros(2, 100, 136, **dev).bfloat16()), binding.QmmError),
                      (dict(a=torch.zeros(2, 16, 60, **dev).bfloat16(), x=torch.zeros(3, 60, **dev).bfloat16()), binding.QmmError),
                      (dict(x=p["x"][:2]), ValueError), (dict(adapters=p["adapters"].long()), ValueError),
                      (dict(scales=torch.ones(3, **dev)), ValueError), (dict(base=p["base"].half()), TypeError),
                      (dict(x=p["x"].float()), TypeError), (dict(out=p["base"].float()), ValueError),
                      (dict(out=p["base"][:2]), ValueError), (dict(x=p["x"].t()), ValueError), (dict(adapters=p["adapters"].cpu()), ValueError),
                      (dict(x=torch.zeros(3, 72, **dev).bfloat16()[:, 4:68]), binding.QmmError)):
        with pytest.raises(kind):
            binding.lora_add(**{**p, **bad})


def test_nothing_to_do():
    p = problem([], 2, 16, 64, 100)
    assert binding.lora_add(**p).shape == (0, 100)
    p = problem([0, 1], 2, 16, 64, 0)
    assert binding.lora_add(**p).shape == (2, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 96, 128])
@pytest.mark.parametrize("N", [1, 31, 601, 604])
def test_rows_of_any_width(N, R, dtype):
    """Tiles of 16, 32 or 64 rows, whose columns are no whole pieces of 16 bytes."""
    p = problem([0] * 130 + [-1] * 41 + [1] * 65 + [2] * 3 + [0] * 31, 3, R, 256, N, dtype, seed=R + N)
    want = check(p)
    got = p["base"].clone()
    assert torch.equal(binding.lora_add(**{**p, "base": got}, out=got), want)
