"""Rotation of queries and keys into the paged cache against the formula in fp64.

Bounds: an angle is off by pi 2^-25 (its 24 bits of half a turn) and 2^-31, its sine and cosine by 2 units in the last place
more, together 2^-22; two products and a sum add 3 2^-24; so a turned element is off by
(|x1| + |x2|) |factor| (2^-22 + 2^-22) and its output's rounding: eps / 2 of its type (bf16 2^-8, E4M3 2^-4, for E4M3
2^-10 below its normal range).  Values and what is not turned are exact (E4M3: rounded once)."""
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def problem(lens, rows, M, Hq, Hkv, D, page, dtype=torch.bfloat16, rot=None, seed=0, base=1e4, extra=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    counts = [-(-max(n, 0) // page) for n in lens]
    total = sum(counts) + extra
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(counts) + 1), -3, dtype=torch.int32, device="cuda")
    for b, n in enumerate(counts):
        table[b, :n], perm = perm[:n], perm[n:]
    rot = D if rot is None else rot
    x = torch.randn(B, M, Hq + 2 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = x.split([Hq, Hkv, Hkv], 2)
    mark = torch.full((total, page, Hkv, D), 7.0, device="cuda").to(dtype)
    return dict(q=q, k_new=k, v_new=v, k_cache=mark, v_cache=mark.clone(), block_table=table,
                lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                inv_freq=base ** (-torch.arange(0, rot, 2, device="cuda").float() / rot) if rot else torch.zeros(0, device="cuda"),
                q_lens=None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda"))


def turned(x, theta, interleaved, factor):
    """(turned x, |x1| + |x2| of every element's pair) in fp64; x [.., heads, D], theta [.., R]."""
    x = x.double()
    R = theta.shape[-1]
    c, s = torch.cos(theta)[..., None, :], torch.sin(theta)[..., None, :]
    y, size = x.clone(), torch.zeros_like(x)
    first = slice(0, 2 * R, 2) if interleaved else slice(0, R)
    second = slice(1, 2 * R, 2) if interleaved else slice(R, 2 * R)
    a, b = x[..., first], x[..., second]
    y[..., first] = factor * (a * c - b * s)
    y[..., second] = factor * (b * c + a * s)
    size[..., first] = size[..., second] = abs(factor) * (a.abs() + b.abs())
    return y, size


def check(p, positions=None, sections=None, interleaved=False, factor=1.0, k_scale=1.0, v_scale=1.0, out=None, stream=None):
    B, M, Hq, D = p["q"].shape
    e8 = p["k_cache"].dtype == E4M3
    page = p["k_cache"].shape[1]
    q_in = p["q"].clone()
    got = binding.rope_append(p["q"], p["k_new"], p["v_new"], p["k_cache"], p["v_cache"], p["block_table"], p["lengths"],
                              p["inv_freq"], q_lens=p["q_lens"], positions=positions, sections=sections,
                              interleaved=interleaved, factor=factor, k_scale=k_scale, v_scale=v_scale, out=out, stream=stream)
    torch.cuda.synchronize()
    L = p["lengths"].long()
    m = p["q_lens"].long().clamp(0, M) if p["q_lens"] is not None else torch.full_like(L, M)
    i = torch.arange(M, device="cuda")
    pos = L[:, None] - m[:, None] + i
    R = len(p["inv_freq"])
    if positions is None:
        where = pos[..., None].expand(B, M, R)
    elif positions.dim() == 2:
        where = positions.long()[..., None].expand(B, M, R)
    else:
        where = torch.cat([positions[a].long()[..., None].expand(B, M, n) for a, n in enumerate(sections)], -1)
    theta = where.double() * p["inv_freq"].double()
    real = (i < m[:, None])[..., None, None]
    y, size = turned(q_in, theta, interleaved, factor)
    y, size = torch.where(real, y, 0.0), torch.where(real, size, 0.0)
    assert ((got.double() - y).abs() <= 2.0**-21 * size + 2.0**-8 * y.abs()).all()
    assert torch.equal(got[..., 2 * R:][real.expand_as(got)[..., 2 * R:]], q_in[..., 2 * R:][real.expand_as(got)[..., 2 * R:]])
    assert (got[~real.expand_as(got)] == 0).all()
    # the cache: what the rows name, and nothing else
    y, size = turned(p["k_new"], theta, interleaved, factor)
    for cache, new, slack, scale in ((p["k_cache"], y, size, k_scale), (p["v_cache"], p["v_new"].double(), 0 * size, v_scale)):
        want = torch.full(cache.shape, 7.0, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(want)
        for b in range(B):
            for r in range(int(m[b])):
                at = int(pos[b, r])
                if at < 0:
                    continue
                pg = int(p["block_table"][b, at // page])
                if not 0 <= pg < cache.shape[0]:
                    continue
                z = new[b, r]
                if e8:
                    z, sl = (z / scale).clamp(-448, 448), slack[b, r] / scale
                    bound[pg, at % page] = 2.0**-21 * sl + torch.maximum(2.0**-4 * z.abs(), torch.tensor(2.0**-10, device="cuda"))
                else:
                    bound[pg, at % page] = 2.0**-21 * slack[b, r] + 2.0**-8 * z.abs() * (slack[b, r] > 0)
                want[pg, at % page] = z
        assert ((cache.double() - want).abs() <= bound).all()
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,rot,page", [(8, 2, 64, 64, 16), (4, 4, 128, 128, 1), (6, 1, 128, 32, 24), (2, 2, 256, 256, 7),
                                               (32, 8, 128, 64, 64), (3, 1, 256, 16, 5)])
def test_formula(Hq, Hkv, D, rot, page, interleaved, dtype):
    check(problem([90, 5, 3, 33], [3, 5, 1, 4], 5, Hq, Hkv, D, page, dtype, rot), interleaved=interleaved, k_scale=0.0625,
          v_scale=0.125)


@pytest.mark.parametrize("lens,rows,M", [([1], None, 1), ([0], [0], 4), ([4, 2, 0], [4, 4, 0], 4), ([700], None, 300),
                                         ([40] * 9, list(range(9)), 8), ([9, 9], [-3, 20], 4), ([1100, 20], [1000, 20], 1000)])
def test_rows_and_lengths(lens, rows, M):
    """Rows before the sequence's start are dropped (their queries are turned all the same), rows behind m_b are 0."""
    check(problem(lens, rows, M, 4, 2, 64, 16))
    assert binding.device_status() == 0


def test_nothing_turns():
    p = problem([20, 7], [3, 2], 3, 4, 2, 64, 16, rot=0)
    check(p)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Angles of thousands and millions of turns: 32-bit angles would be off by radians."""
    p = problem([40, 30, 20], None, 4, 4, 2, 128, 16, base=1e6)
    for far in (131071, 10**6 + 1, 2**31 - 1, 0, -5, -2**31):
        p["k_cache"].fill_(7.0), p["v_cache"].fill_(7.0)
        check(p, positions=torch.full((3, 4), far, dtype=torch.int32, device="cuda"), interleaved=interleaved)


def test_frequencies_of_any_size():
    """p f has at most 53 bits here, so that the reference's product is exact too."""
    p = problem([40, 30], None, 4, 2, 2, 128, 16)
    p["inv_freq"] = torch.tensor([0.0, 1.0, 1e-38, 1e-42, 2.0**-126, 0.99999994, 1.5, 3.25, 1000.7, 1e6, 2.0**20, 7e5, -0.3, -1e-3,
                                  6.2831855, 3.1415927], device="cuda").repeat(4)
    check(p, positions=torch.randint(0, 4096, (2, 4), device="cuda", dtype=torch.int32), factor=-1.25)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("sections", [(16, 24, 24), (0, 64, 0), (64, 0, 0, 0), (1, 2, 3, 58), (30, 34)])
def test_axes(sections, dtype):
    p = problem([50, 20, 11], [6, 4, 1], 6, 4, 2, 128, 16, dtype)
    pos = torch.randint(0, 100000, (len(sections), 3, 6), device="cuda", dtype=torch.int32)
    for interleaved in (False, True):
        p["k_cache"].copy_(torch.full(p["k_cache"].shape, 7.0, device="cuda").to(dtype))
        p["v_cache"].copy_(torch.full(p["v_cache"].shape, 7.0, device="cuda").to(dtype))
        check(p, positions=pos, sections=sections, interleaved=interleaved, k_scale=0.5, v_scale=0.5)


def test_in_place_and_strided():
    """Queries that are a slice of one projection's output, turned where they are."""
    for interleaved in (False, True):
        p = problem([33, 8, 50], [4, 2, 3], 4, 8, 2, 128, 16, seed=3)
        want = check(p, interleaved=interleaved)
        p["k_cache"].fill_(7.0), p["v_cache"].fill_(7.0)
        kv = p["k_new"].clone(), p["v_new"].clone()
        got = check(p, interleaved=interleaved, out=p["q"])
        assert torch.equal(got, want) and got.data_ptr() == p["q"].data_ptr()
        assert torch.equal(kv[0], p["k_new"]) and torch.equal(kv[1], p["v_new"])


def test_other_orders_of_the_cache():
    p = problem([60, 17], [5, 3], 5, 4, 2, 64, 16)
    for name in ("k_cache", "v_cache"):
        c = p[name]
        p[name] = c.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) if name == "k_cache" else \
            c.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3)
    check(p)


def test_bad_pages_and_lengths():
    p = problem([40, 30], None, 4, 4, 2, 64, 16)
    p["block_table"][0, 2] = 10**6
    check(p)
    assert binding.device_status() == 32
    p = problem([40, 30], None, 4, 4, 2, 64, 16)
    p["lengths"][1] = 10**6  # clamped to what the table holds, whose last page is none
    binding.rope_append(p["q"], p["k_new"], p["v_new"], p["k_cache"], p["v_cache"], p["block_table"], p["lengths"], p["inv_freq"])
    torch.cuda.synchronize()
    assert binding.device_status() == 32
    assert (p["k_cache"] == 7.0).sum() == p["k_cache"].numel() - 4 * 2 * 64


def test_matches_kv_append_without_rotation():
    p = problem([40, 30], [4, 2], 4, 4, 2, 128, 16, E4M3, rot=0)
    k, v = p["k_cache"].clone(), p["v_cache"].clone()
    check(p, k_scale=0.25, v_scale=0.5)
    binding.kv_append(p["k_new"], p["v_new"], k, v, p["block_table"], p["lengths"], p["q_lens"], 0.25, 0.5)
    assert torch.equal(k.view(torch.uint8), p["k_cache"].view(torch.uint8))
    assert torch.equal(v.view(torch.uint8), p["v_cache"].view(torch.uint8))


def test_infinities_and_nan_stay_in_their_pairs():
    p = problem([20], None, 2, 2, 1, 64, 16)
    p["q"][0, 0, 0, 3] = float("nan")
    p["k_new"][0, 1, 0, 5] = float("inf")
    got = binding.rope_append(p["q"], p["k_new"], p["v_new"], p["k_cache"], p["v_cache"], p["block_table"], p["lengths"], p["inv_freq"])
    bad = torch.nonzero(~torch.isfinite(got.float())).tolist()
    assert bad == [[0, 0, 0, 3], [0, 0, 0, 35]]
    assert int((~torch.isfinite(p["k_cache"].float())).sum()) == 2


def test_refusals():
    p = problem([40, 30], None, 4, 4, 2, 64, 16)

    def call(**changes):
        a = {**p, **changes}
        return binding.rope_append(a.pop("q"), a.pop("k_new"), a.pop("v_new"), a.pop("k_cache"), a.pop("v_cache"),
                                   a.pop("block_table"), a.pop("lengths"), a.pop("inv_freq"), **a)

    dev = dict(device="cuda")
    pos = torch.zeros(2, 4, dtype=torch.int32, **dev)
    for bad, kind in ((dict(inv_freq=torch.ones(12, **dev)), binding.QmmError), (dict(inv_freq=torch.ones(40, **dev)), binding.QmmError),
                      (dict(inv_freq=torch.ones(32, **dev).double()), ValueError), (dict(sections=(32,)), ValueError),
                      (dict(positions=pos[:1]), ValueError), (dict(positions=pos.long()), ValueError),
                      (dict(positions=pos.expand(3, 2, 4).contiguous()), ValueError),
                      (dict(positions=pos.expand(2, 2, 4).contiguous(), sections=(10, 10)), binding.QmmError),
                      (dict(positions=pos.expand(2, 2, 4).contiguous(), sections=(40, -8)), ValueError),
                      (dict(positions=pos.expand(5, 2, 4).contiguous(), sections=(8, 8, 8, 4, 4)), ValueError),
                      (dict(factor=float("inf")), binding.QmmError), (dict(q=p["q"].float()), TypeError),
                      (dict(q=p["q"][:, :3]), ValueError), (dict(out=torch.zeros(2, 4, 4, 64, **dev)), TypeError),
                      (dict(out=p["q"][:1]), ValueError), (dict(k_cache=p["k_cache"].half(), v_cache=p["v_cache"].half()), TypeError),
                      (dict(lengths=p["lengths"].long()), ValueError), (dict(inv_freq=torch.ones(32)), ValueError)):
        with pytest.raises(kind):
            call(**bad)
    torch.cuda.synchronize()
    assert (p["k_cache"] == 7.0).all()
