"""The paged key-value cache: append bit for bit, attention against the formula in fp64.

Bounds of the attention, from its roundings: a score is an fp32 sum of D exact
products, off by at most d = (D + 8) 2^-24 scale sum|q k|; probabilities enter
the second product with 8 bits (relative 2^-8 with the roundings of exp and of
the sums), so with P = sum_j p_j |v_j| the output is off by at most
(2^-8 + 2 d) P + 2^-9 |o| (the last for the bf16 output), and the log-sum-exp by
d + 2^-20 (2 + |lse|)."""
import math

import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu


class Cache:
    """A paged cache with its dense twin.  Every slot that no sequence owns, and every place past a sequence's length,
    holds NaN; ``order`` is the dimensions' order in memory."""

    def __init__(self, lens, Hkv, D, page, dtype=torch.bfloat16, order=(0, 1, 2, 3), seed=0, extra=3, k_scale=1.0,
                 v_scale=1.0, std=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.D, self.page, self.dtype = lens, D, page, dtype
        self.k_scale, self.v_scale = k_scale, v_scale
        counts = [-(-n // page) for n in lens]
        total = sum(counts) + extra
        shape = (total, page, Hkv, D)
        perm = torch.randperm(total, generator=g, device="cuda").tolist()
        self.table = torch.full((len(lens), max(counts) + 1), -7, dtype=torch.int32, device="cuda")

        def pages():
            mem = torch.full([shape[i] for i in order], float("nan"), device="cuda").to(dtype)
            return mem.permute([order.index(i) for i in range(4)])

        self.k, self.v = pages(), pages()
        self.dense = []
        for b, n in enumerate(lens):
            mine, perm = perm[:counts[b]], perm[counts[b]:]
            self.table[b, :counts[b]] = torch.tensor(mine, dtype=torch.int32, device="cuda")
            kv = []
            for cache, s in ((self.k, k_scale), (self.v, v_scale)):
                x = (std * torch.randn(n, Hkv, D, generator=g, device="cuda") / s).to(torch.bfloat16)
                x = x if dtype == torch.bfloat16 else x.float().clamp(-448, 448).to(dtype)
                j = torch.arange(n, device="cuda")
                if n:
                    at = torch.tensor(mine, device="cuda")[j // page], j % page
                    raw = cache if dtype == torch.bfloat16 else cache.view(torch.uint8)
                    raw[at] = x if dtype == torch.bfloat16 else x.view(torch.uint8)
                kv.append(x.double() * (s if dtype != torch.bfloat16 else 1.0))
            self.dense.append(kv)
        self.lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def args(self):
        return self.k, self.v, self.table, self.lengths

    def scales(self):
        return dict(k_scale=self.k_scale, v_scale=self.v_scale)


def reference(q, c, rows, scale, window, sinks):
    """(out, lse, bound of out, bound of lse) in fp64."""
    B, M, Hq, D = q.shape
    o = torch.zeros(B, M, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, M, Hq), -math.inf, dtype=torch.float64, device="cuda")
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    for b, n in enumerate(c.lens):
        k, v = c.dense[b]
        Hkv = k.shape[1]
        for i in range(rows[b]):
            p = n - rows[b] + i
            j = torch.arange(max(0, p + 1), device="cuda")
            if window:
                j = j[(j > p - window) | (j < sinks)]
            if len(j) == 0:
                continue
            qq = q[b, i].double().view(Hkv, Hq // Hkv, D)
            x = torch.einsum("hgd,thd->hgt", qq, k[j]) * scale
            d = ((D + 8) * 2.0**-24 * abs(scale) * torch.einsum("hgd,thd->hgt", qq.abs(), k[j].abs())).amax(-1).reshape(Hq)
            w = torch.softmax(x, -1)
            lse[b, i] = torch.logsumexp(x, -1).reshape(Hq)
            o[b, i] = torch.einsum("hgt,thd->hgd", w, v[j]).reshape(Hq, D)
            P = torch.einsum("hgt,thd->hgd", w, v[j].abs()).reshape(Hq, D)
            bo[b, i] = (2.0**-8 + 2 * d[:, None]) * P + 2.0**-9 * o[b, i].abs() + 1e-30
            bl[b, i] = d + 2.0**-20 * (2 + lse[b, i].abs())
    return o, lse, bo, bl


def check(c, q, rows=None, scale=None, window=0, sinks=0, **kw):
    B, M, _, D = q.shape
    q_lens = torch.tensor(rows, dtype=torch.int32, device="cuda") if rows is not None else None
    out, lse = binding.paged_attention(q, *c.args(), q_lens=q_lens, scale=scale, window=window, sinks=sinks,
                                       return_lse=True, **c.scales(), **kw)
    torch.cuda.synchronize()
    o, l, bo, bl = reference(q, c, rows or [M] * B, D ** -0.5 if scale is None else scale, window, sinks)
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert (out[empty] == 0).all()
    eo, el = (out.double() - o).abs(), (lse.double() - l).abs()[~empty]
    assert (eo <= bo).all(), float((eo / bo.clamp(min=1e-300)).max())
    assert (el <= bl[~empty]).all(), float((el / bl[~empty]).max())
    assert binding.device_status() == 0
    return out, lse


def queries(B, M, Hq, D, seed=1):
    return torch.randn(B, M, Hq, D, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("M,Hq,Hkv", [(1, 1, 1), (1, 8, 2), (1, 40, 8), (2, 7, 1), (3, 24, 4), (5, 4, 4), (8, 32, 8),
                                      (16, 8, 8), (16, 8, 1), (11, 10, 2), (16, 16, 1)])
def test_heads_and_rows(M, Hq, Hkv, D, dtype):
    lens = [max(M, 1), 63, 64, 65, 130, 700, M + 1]
    c = Cache(lens, Hkv, D, 16, dtype, seed=M * Hq, k_scale=0.25, v_scale=0.5)
    check(c, queries(len(lens), M, Hq, D))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("page", [1, 7, 16, 24, 64, 100, 256])
def test_pages(page, dtype):
    lens = [1, 5, page, page + 1, 3 * page - 1, 333]
    c = Cache(lens, 2, 128, page, dtype, seed=page, k_scale=0.125, v_scale=0.125)
    check(c, queries(len(lens), 3, 8, 128), rows=[1, 3, 1, 2, 3, 0])


@pytest.mark.parametrize("lens", [[1], [2], [20000], [1, 20000, 3], [5000] * 3, [64] * 100, list(range(1, 300))])
def test_lengths(lens):
    c = Cache(lens, 2, 128, 32, seed=len(lens))
    check(c, queries(len(lens), 1, 8, 128))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("page", [16, 12])
@pytest.mark.parametrize("M,Hq,D", [(1, 16, 128), (2, 32, 128), (4, 64, 64), (16, 16, 64), (1, 8, 256), (4, 32, 256)])
def test_many_tiles_per_sm(M, Hq, D, page, dtype):
    """Long lists: every stage of an SM's ring is refilled many times, and queues of unequal speed run beside each other."""
    c = Cache([40000, 9000, 31000], 8, D, page, dtype, seed=M, k_scale=0.5, v_scale=0.5)
    check(c, queries(3, M, Hq, D), rows=[M, 1, M])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (16, 4), (63, 0), (64, 64), (65, 1), (100, 130),
                                          (300, 5), (5000, 4), (1000000, 7)])
def test_window_and_sinks(window, sinks, dtype):
    lens = [1, 17, 64, 65, 200, 1111, 3000]
    c = Cache(lens, 2, 64, 16, dtype, seed=window + sinks, k_scale=0.5, v_scale=0.25)
    check(c, queries(len(lens), 4, 16, 64), rows=[1, 4, 4, 3, 4, 2, 4], window=window, sinks=sinks)


def test_rows_that_see_nothing():
    """Length 0, fewer tokens than new rows, no new rows."""
    c = Cache([0, 3, 40, 8], 2, 128, 16)
    check(c, queries(4, 8, 4, 128), rows=[8, 8, 0, 8])
    check(c, queries(4, 1, 4, 128), rows=[1, 1, 0, 1])


def test_all_empty():
    c = Cache([0, 0], 2, 128, 16)
    check(c, queries(2, 2, 4, 128))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("M,Hq", [(3, 2), (8, 8), (16, 16), (16, 32)])
def test_nonfinite_values_a_row_does_not_see(M, Hq, dtype):
    """A later draft row's key and value are NaN / inf: the earlier rows are as if they were not there."""
    c = Cache([70, 150, 64], 2, 128, 16, dtype, seed=3)
    q = queries(3, M, Hq, 128)
    o0, l0 = check(c, q)
    for b, n in enumerate(c.lens):
        page, slot = int(c.table[b, (n - 1) // 16]), (n - 1) % 16
        c.k[page, slot] = float("nan")
        c.v[page, slot, 0] = float("nan")
        c.v[page, slot, 1] = float("inf") if dtype == torch.bfloat16 else float("nan")
    o1, l1 = binding.paged_attention(q, *c.args(), return_lse=True)
    assert torch.equal(o0[:, :-1], o1[:, :-1]) and torch.equal(l0[:, :-1], l1[:, :-1])
    assert torch.isnan(o1[:, -1]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_infinite_value_behind_the_window(dtype):
    """The token that left the window of the later rows only: the first row sees its infinity, the others do not."""
    bad = float("inf") if dtype == torch.bfloat16 else float("nan")
    c = Cache([200], 1, 64, 16, dtype, seed=4)
    q = queries(1, 4, 4, 64)
    o0, _ = check(c, q, window=50)
    first = 200 - 4 + 1 - 50  # the oldest token that row 0 sees
    c.v[int(c.table[0, first // 16]), first % 16] = bad
    o1 = binding.paged_attention(q, *c.args(), window=50)
    assert torch.equal(o0[:, 1:], o1[:, 1:])
    assert not torch.isfinite(o1[:, 0]).any()


def test_large_scores_and_scales():
    c = Cache([900], 2, 128, 16, std=8.0)
    check(c, queries(1, 2, 8, 128) * 4)
    check(c, queries(1, 2, 8, 128), scale=0.0)
    check(c, queries(1, 2, 8, 128), scale=-0.05)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("order", [(0, 2, 1, 3), (2, 0, 1, 3), (1, 0, 2, 3)])
def test_memory_orders(order, dtype):
    lens = [100, 33]
    c = Cache(lens, 4, 64, 16, dtype, order)
    check(c, queries(2, 2, 8, 64))


def test_strided_queries_and_other_stream():
    """q is a slice of a fused projection's output; the call runs on another stream with its own workspace."""
    c = Cache([100, 33, 600], 2, 128, 16)
    fused = torch.randn(3, 4, 8 + 2 + 2, 128, device="cuda").bfloat16()
    q = fused[:, :, :8]
    o, l = check(c, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    need = binding.lib().qmm_paged_attention_workspace(3, 4, 8, 2, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    o2, l2 = binding.paged_attention(q, *c.args(), return_lse=True, stream=side, workspace=ws)
    o3 = binding.paged_attention(q, *c.args(), stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(l, l2) and torch.equal(o, o3)


def test_repeats_are_equal():
    c = Cache([3000, 10, 777], 2, 128, 16)
    q = queries(3, 8, 16, 128)
    first = binding.paged_attention(q, *c.args())
    for _ in range(4):
        assert torch.equal(first, binding.paged_attention(q, *c.args()))


def test_offsets_past_32_bits():
    """Pages more than 2^31 elements apart: strides and page numbers in 64 bits."""
    page, Hkv, D = 64, 8, 256
    total = 2**31 // (page * Hkv * D) + 40
    big = torch.zeros(total, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    c = Cache([200, 150], Hkv, D, page)
    at = torch.tensor([total - 1, 3, total - 9, total - 2, 0, total - 30, 7], device="cuda")
    kb, vb = big, torch.zeros_like(big)
    table = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
    used = 0
    for b, n in enumerate(c.lens):
        for j in range(-(-n // page)):
            kb[at[used]], vb[at[used]] = c.k[int(c.table[b, j])], c.v[int(c.table[b, j])]
            table[b, j] = int(at[used])
            used += 1
    c.k, c.v, c.table = kb, vb, table
    check(c, queries(2, 2, 16, D))


def test_bad_pages_and_lengths_are_reported():
    c = Cache([100, 40], 2, 128, 16)
    q = queries(2, 1, 4, 128)
    o0 = binding.paged_attention(q, *c.args())
    good = c.table.clone()
    c.table[0, 2] = 10**6
    o1 = binding.paged_attention(q, *c.args())
    assert binding.device_status() == 32
    assert torch.equal(o0[1], o1[1]) and torch.isfinite(o1).all() and not torch.equal(o0[0], o1[0])
    c.table = good
    c.lengths = torch.tensor([-5, 10**9], dtype=torch.int32, device="cuda")
    c.table[1] = c.table[0, 0]
    binding.paged_attention(q, *c.args())
    assert binding.device_status() == 32
    binding.kv_append(torch.zeros(2, 1, 2, 128, device="cuda").bfloat16(), torch.zeros(2, 1, 2, 128, device="cuda").bfloat16(),
                      c.k, c.v, torch.full_like(c.table, -1), torch.tensor([1, 1], dtype=torch.int32, device="cuda"))
    assert binding.device_status() == 32


# ----------------------------------------------------------------- append
@pytest.mark.parametrize("dtype,scale", [(torch.bfloat16, 1.0), (torch.float8_e4m3fn, 1.0), (torch.float8_e4m3fn, 0.3)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("M,page", [(1, 16), (5, 1), (16, 24), (3, 64)])
def test_append(M, page, D, dtype, scale):
    lens, rows = [M, 40, 2, 17, 1], [M, max(1, M - 1), M, 0, 1]
    for order in ((0, 1, 2, 3), (0, 2, 1, 3)):
        c = Cache(lens, 3, D, page, dtype, order, seed=M)
        raw = (lambda t: t.view(torch.uint8)) if dtype != torch.bfloat16 else (lambda t: t.view(torch.int16))
        want = [raw(c.k).clone(), raw(c.v).clone()]
        fused = 30 * torch.randn(5, M, 9, D, device="cuda").bfloat16()
        fused[0, 0, 3, :4] = torch.tensor([0.0, -0.0, 1e30, -1e-30]).bfloat16()
        new = fused[:, :, 3:6], fused[:, :, 6:9]
        for w, x in zip(want, new):
            for b, (n, m) in enumerate(zip(lens, rows)):
                for i in range(m):
                    p = n - m + i
                    if p < 0:
                        continue
                    y = x[b, i]
                    if dtype != torch.bfloat16:
                        y = (y.float() / torch.tensor(scale, device="cuda")).clamp(-448, 448).to(dtype)
                    w[int(c.table[b, p // page]), p % page] = raw(y.contiguous())
        binding.kv_append(*new, *c.args(), q_lens=torch.tensor(rows, dtype=torch.int32, device="cuda"), k_scale=scale,
                          v_scale=scale)
        torch.cuda.synchronize()
        assert torch.equal(raw(c.k), want[0]) and torch.equal(raw(c.v), want[1])
        assert binding.device_status() == 0


def test_append_then_attend():
    """The new rows arrive in two steps; attention over them equals attention over the whole."""
    c = Cache([50, 90], 2, 128, 16)
    new = [torch.stack([c.dense[b][kv][-4:] for b in range(2)]).bfloat16() for kv in (0, 1)]
    q = queries(2, 4, 8, 128)
    want, _ = check(c, q)
    for b, n in enumerate(c.lens):
        for j in range(n - 4, n):
            c.k[int(c.table[b, j // 16]), j % 16] = float("nan")
            c.v[int(c.table[b, j // 16]), j % 16] = float("nan")
    binding.kv_append(*new, *c.args())
    assert torch.equal(want, binding.paged_attention(q, *c.args()))


def test_refusals():
    c = Cache([50, 90], 2, 128, 16)
    q = queries(2, 4, 8, 128)
    call = binding.paged_attention
    for bad, err in (((q[:, :, :7].contiguous(), *c.args()), binding.QmmError),      # heads no multiple
                     ((queries(2, 17, 8, 128), *c.args()), binding.QmmError),        # too many rows
                     ((q.float(), *c.args()), TypeError),
                     ((q, c.k.half(), c.v.half(), c.table, c.lengths), TypeError),
                     ((q, c.k, c.v[1:], c.table, c.lengths), ValueError),
                     ((q, c.k, c.v, c.table.long(), c.lengths), ValueError),
                     ((q, c.k, c.v, c.table, c.lengths[:1]), ValueError),
                     ((q[..., :64].contiguous(), *c.args()), ValueError),
                     ((q.cpu(), *c.args()), ValueError),
                     ((q.transpose(1, 2).contiguous().transpose(1, 2), *c.args()), ValueError)):
        with pytest.raises(err):
            call(*bad)
    with pytest.raises(binding.QmmError):
        call(q, *c.args(), window=-1)
    with pytest.raises(binding.QmmError):  # head size
        call(queries(1, 1, 2, 32), *Cache([5], 2, 32, 16).args())
    f8 = Cache([50], 2, 128, 16, torch.float8_e4m3fn)
    with pytest.raises(binding.QmmError):
        call(q[:1], *f8.args(), k_scale=0.0)
    with pytest.raises(ValueError):
        binding.kv_append(q, q, *c.args())  # heads do not match
