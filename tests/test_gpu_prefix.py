"""Attention behind a shared prefix against the formula in fp64.

Bounds, from its roundings: a score is an fp32 sum of D exact products, off by at most d = (D + 8) 2^-24 scale sum|q k|;
probabilities enter the second product with 16 bits (2^-16) after an exponential (2^-21), and sums of up to some hundred
terms in a chain (tiles of 128, then parts) add 2^-16; so with P = sum_j p_j |v_j| the output is off by at most
(2^-14 + 2 d) P + 2^-8 |o| (the last for the bf16 output), and the log-sum-exp by d + 2^-16 + 2^-20 |lse|.
An E4M3 cache's probabilities enter that product in fp16, 11 bits, whose rounding is off by at most eps / 2 = 2^-11 of each:
(2^-11 + 2^-14 + 2 d) P there."""
import math

import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding
from test_gpu_paged import Cache, queries

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


class Shared:
    """A cache of a prefix and of the sequences' own tokens behind it; everything that nobody owns is NaN."""

    def __init__(self, pages, own, Hkv, D, page, dtype=torch.bfloat16, **more):
        self.P, self.own = pages * page, own
        self.c = Cache([self.P] + own, Hkv, D, page, dtype, **more)
        self.k, self.v = self.c.k, self.c.v
        self.prefix = self.c.table[0, :pages].contiguous()
        self.table = self.c.table[1:]
        self.lengths = torch.tensor([n + self.P for n in own], dtype=torch.int32, device="cuda")

    def args(self):
        return self.k, self.v, self.prefix, self.table, self.lengths


def reference(q, s, rows, scale):
    B, M, Hq, D = q.shape
    o = torch.zeros(B, M, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, M, Hq), -math.inf, dtype=torch.float64, device="cuda")
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    k0, v0 = s.c.dense[0]
    Hkv = k0.shape[1]
    for b, n in enumerate(s.own):
        m = rows[b]
        if m == 0:
            continue
        k, v = (torch.cat(x).permute(1, 2, 0) for x in zip((k0, v0), s.c.dense[b + 1]))  # [Hkv, D, tokens]
        qq = q[b, :m].double().view(m, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        last = torch.arange(s.P + n - m, s.P + n, device="cuda").repeat_interleave(Hq // Hkv)
        unseen = torch.arange(s.P + n, device="cuda") > last[:, None]
        x = (scale * (qq @ k)).masked_fill(unseen, -math.inf)
        d = ((D + 8) * 2.0**-24 * abs(scale) * (qq.abs() @ k.abs())).masked_fill(unseen, 0).amax(-1)
        p = torch.softmax(x, -1)

        def back(t):
            return t.view(Hkv, m, Hq // Hkv, -1).permute(1, 0, 2, 3).reshape(m, Hq, -1)

        o[b, :m] = back(p @ v.transpose(1, 2))
        lse[b, :m] = back(torch.logsumexp(x, -1))[..., 0]
        weight = 2.0**-14 + (2.0**-11 if s.k.dtype == E4M3 else 0.0)
        bo[b, :m] = back((weight + 2 * d)[..., None] * (p @ v.abs().transpose(1, 2))) + 2.0**-8 * o[b, :m].abs()
        bl[b, :m] = back(d)[..., 0] + 2.0**-16 + 2.0**-20 * lse[b, :m].abs()
    return o, lse, bo, bl


def check(q, s, rows=None, scale=None, **more):
    B, M, Hq, D = q.shape
    q_lens = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    size = binding.shared_prefix_attention_workspace(B, M, Hq, s.k.shape[2], D)
    workspace = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read before it is written
    out, lse = binding.shared_prefix_attention(q, *s.args(), q_lens=q_lens, scale=scale, return_lse=True, workspace=workspace,
                                               **s.c.scales(), **more)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    rows = [M] * B if rows is None else rows
    rows = [r if s.own[b] > 0 or s.P == 0 else 0 for b, r in enumerate(rows)]
    o, l, bo, bl = reference(q, s, rows, 1 / math.sqrt(D) if scale is None else scale)
    assert ((out.double() - o).abs() <= bo).all(), float(((out.double() - o).abs() - bo).max())
    seen = l > -math.inf
    assert torch.equal(lse > -math.inf, seen)
    assert ((lse.double() - l)[seen].abs() <= bl[seen]).all()
    return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("pages,page,own,M,Hq,Hkv,D", [
    (4, 16, [3, 20, 1], 1, 4, 2, 64), (1, 1, [1], 1, 1, 1, 64), (9, 16, [5, 40], 5, 8, 2, 128), (1, 128, [16, 16], 16, 8, 1, 128),
    (40, 24, [100, 7, 33, 64], 4, 8, 8, 128), (130, 1, [9, 3], 3, 6, 2, 128), (3, 500, [700, 10], 2, 32, 8, 64),
    (20, 64, [30, 31], 2, 8, 2, 256), (7, 20, [70] * 5, 7, 14, 2, 256), (33, 32, [16] * 20, 16, 16, 1, 128),
    (11, 8, [16] * 9, 16, 112, 7, 64)])
def test_formula(pages, page, own, M, Hq, Hkv, D, dtype):
    s = Shared(pages, own, Hkv, D, page, dtype, seed=1, k_scale=0.5, v_scale=0.25)
    q = queries(len(own), M, Hq, D)
    check(q, s)


@pytest.mark.parametrize("B,M,G", [(1, 1, 1), (3, 5, 1), (8, 16, 1), (43, 3, 1), (16, 16, 1), (5, 13, 2), (20, 13, 1), (64, 8, 4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
def test_rows_around_tiles(B, M, G, dtype):
    """Rows that end in and between tiles of 128 (1 .. 2048 of them), some of them padding."""
    rows = [1 + (3 * b + M) % M for b in range(B)]
    s = Shared(19, [M + 5 * b % 40 for b in range(B)], 2, 128, 16, dtype, seed=2)
    q = queries(B, M, 2 * G, 128)
    check(q, s, rows)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("tokens", [1, 63, 64, 65, 127, 128, 129, 255, 256, 383, 1000, 2049, 5000])
def test_prefix_lengths(tokens, D):
    """Pages of one token: a prefix of any length."""
    s = Shared(tokens, [4, 9], 1, D, 1, seed=tokens)
    check(queries(2, 2, 4, D), s)


def test_long():
    s = Shared(300, [1, 40, 1000], 4, 128, 64, seed=3)
    check(queries(3, 1, 16, 128), s)
    s = Shared(300, [8] * 33, 1, 64, 64, E4M3, seed=4)
    check(queries(33, 8, 8, 64), s)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
def test_many_sequences(dtype):
    """More than a CTA lists the first rows of (rows that do not exist are computed then, and not written)."""
    own = [1 + b % 7 for b in range(430)]
    s = Shared(11, own, 1, 64, 16, dtype, seed=13)
    check(queries(430, 2, 2, 64), s, [min(1 + b % 2, own[b]) for b in range(430)])


def test_empty_prefix_and_empty_sequences():
    s = Shared(0, [5, 30, 17], 2, 128, 16)
    check(queries(3, 4, 4, 128), s, [4, 4, 1])
    s = Shared(6, [5, 0, 30, 0], 2, 128, 16)
    s.lengths[1] = s.lengths[3] = 0  # padding of the batch
    out, lse = check(queries(4, 4, 4, 128), s, [4, 4, 0, 2])
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


def test_no_own_pages():
    """No sequence has a row: nothing seen, nothing read."""
    s = Shared(6, [0, 0], 2, 128, 16)
    s.lengths.zero_()
    q = queries(2, 2, 4, 128)
    out, lse = binding.shared_prefix_attention(q, s.k, s.v, s.prefix, s.table[:, :0], s.lengths, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all() and binding.device_status() == 0


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 4.0])
def test_scales(scale):
    s = Shared(20, [12, 50], 2, 128, 16, seed=5)
    check(queries(2, 3, 4, 128), s, scale=scale)


def test_peaked_and_large_scores():
    """One token holds nearly all the weight, in the prefix for some rows and among the own for others; scores beyond
    32-bit exponentials' range."""
    s = Shared(40, [30, 30], 1, 128, 16, seed=6)
    q = queries(2, 2, 4, 128)
    for scale in (1.0, 20.0):
        check(q, s, scale=scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
def test_equals_attention_over_whole_tables(dtype):
    """The same sequences with the prefix in every table, by paged_attention: within both bounds."""
    s = Shared(30, [20, 5, 64], 2, 128, 16, dtype, seed=7)
    q = queries(3, 4, 8, 128)
    a, la = check(q, s)
    table = torch.cat((s.prefix[None].expand(3, -1), s.table), 1).contiguous()
    b, lb = binding.paged_attention(q, s.k, s.v, table, s.lengths, return_lse=True)
    assert (a.float() - b.float()).abs().max() <= 2.0**-6 and (la - lb).abs().max() <= 2.0**-15
    # and from a table that names the prefix too
    c, _ = binding.shared_prefix_attention(q, s.k, s.v, s.prefix, table[:, 30:], s.lengths, return_lse=True)
    assert torch.equal(a, c)


def test_values_that_are_not_finite():
    """Seen ones reach their column, unseen ones (later draft rows', past the lengths: NaN in these caches) nothing."""
    s = Shared(20, [12, 50], 1, 128, 16, seed=8)
    q = queries(2, 3, 4, 128)
    want, _ = check(q, s)
    at = 37
    s.v[int(s.prefix[at // 16]), at % 16, 0, 5] = math.inf
    out = binding.shared_prefix_attention(q, *s.args())
    assert (out[..., 5] == math.inf).all()
    others = [d for d in range(128) if d != 5]
    assert torch.equal(out[..., others], want[..., others])
    s.v[int(s.table[0, 0]), 11, 0, 9] = math.nan  # the last new row of sequence 0
    out = binding.shared_prefix_attention(q, *s.args())
    assert torch.isnan(out[0, 2, :, 9]).all() and torch.equal(out[0, :2, :, 9], want[0, :2, :, 9]) and torch.equal(out[1, ..., 9], want[1, ..., 9])


@pytest.mark.parametrize("order", [(0, 2, 1, 3), (2, 0, 1, 3), (1, 0, 2, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
def test_orders_of_the_cache(order, dtype):
    s = Shared(12, [12, 50], 2, 64, 16, dtype, seed=9, order=order)
    check(queries(2, 3, 4, 64), s)


def test_strided_queries():
    s = Shared(12, [12, 50], 2, 64, 16, seed=10)
    wide = queries(2, 3, 8, 64)
    check(wide[:, :, 2:6], s)


def test_results_repeat():
    s = Shared(300, [9 + b for b in range(12)], 2, 128, 16, seed=11)
    q = queries(12, 4, 16, 128)
    first = binding.shared_prefix_attention(q, *s.args(), return_lse=True)
    ws = torch.empty(binding.shared_prefix_attention_workspace(12, 4, 16, 2, 128), dtype=torch.uint8, device="cuda")
    for fill in (0, 255):
        ws.fill_(fill)  # NaN patterns
        again = binding.shared_prefix_attention(q, *s.args(), return_lse=True, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_bad_pages_and_lengths():
    """Bad numbers set the status bit; a page outside the cache reads as zeros."""
    s = Shared(20, [12, 50], 1, 128, 16, seed=12)
    q = queries(2, 3, 4, 128)
    want, _ = check(q, s)
    s.prefix[3] = 10**6
    for cache in s.c.dense[0]:
        cache[48:64] = 0
    out = binding.shared_prefix_attention(q, *s.args())
    torch.cuda.synchronize()
    assert binding.device_status() == 32
    o, _, bo, _ = reference(q, s, [3, 3], 1 / math.sqrt(128))
    assert ((out.double() - o).abs() <= bo).all()
    s = Shared(20, [12, 50], 1, 128, 16, seed=12)
    for bad in (s.P + 2, s.P - 5, 1, -1, 10**6):  # new rows inside the prefix, or no such length
        s.lengths[0] = bad
        out, lse = binding.shared_prefix_attention(q, *s.args(), return_lse=True)
        torch.cuda.synchronize()
        assert binding.device_status() == 32
        assert (out[0] == 0).all() and (lse[0] == -math.inf).all() and torch.equal(out[1], want[1])


def test_refusals():
    s = Shared(4, [12, 50], 2, 128, 16)
    q = queries(2, 3, 4, 128)
    bad = [(dict(scale=math.nan), binding.QmmError), (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), binding.QmmError),
           (dict(out=torch.empty(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")), ValueError),
           (dict(q_lens=torch.ones(3, dtype=torch.int32, device="cuda")), ValueError)]
    for more, kind in bad:
        with pytest.raises(kind):
            binding.shared_prefix_attention(q, *s.args(), **more)
    for q2 in (queries(2, 17, 4, 128), queries(2, 3, 3, 128)):
        with pytest.raises(binding.QmmError):
            binding.shared_prefix_attention(q2, *s.args())
    with pytest.raises(ValueError):
        binding.shared_prefix_attention(q, s.k, s.v, s.prefix.long(), s.table, s.lengths)
    with pytest.raises(ValueError):
        binding.shared_prefix_attention(q, s.k, s.v, s.prefix.cpu(), s.table, s.lengths)
    with pytest.raises(ValueError):
        binding.shared_prefix_attention(queries(2, 3, 4, 64), *s.args())
    with pytest.raises(TypeError):
        binding.shared_prefix_attention(q.float(), *s.args())


def test_nothing_to_do():
    s = Shared(4, [12, 50], 2, 128, 16)
    out = binding.shared_prefix_attention(queries(2, 3, 4, 128)[:, :0], *s.args())
    assert out.shape == (2, 0, 4, 128)
    out = binding.shared_prefix_attention(queries(2, 3, 4, 128)[:0], s.k, s.v, s.prefix, s.table[:0], s.lengths[:0])
    assert out.shape == (0, 3, 4, 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [1, 3, 5, 7, 20, 100, 129])
def test_pages_that_no_box_divides(page, D, dtype):
    """Rows copied one by one, keys and values in orders of their own."""
    s = Shared(-(-700 // page), [5, 17], 2, D, page, dtype, seed=page + D)
    q = queries(2, 3, 6, D)
    out, lse = check(q, s)
    s.v = s.v.view(torch.uint8).permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3).view(dtype) if dtype == E4M3 else \
        s.v.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    assert s.v.stride() != s.k.stride()
    again, lse2 = check(q, s)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (1, 128), (1, 256), (3, 128)])
def test_a_row_in_parts_of_every_sm(Hkv, D, dtype):
    """Few rows behind a long prefix, which lie in a part of each SM, and rows enough that many CTAs join them."""
    s = Shared(170, [3, 9], Hkv, D, 128, dtype, seed=21)
    check(queries(2, 2, 4 * Hkv, D), s)
    s = Shared(170, [16] * 40, Hkv, D, 128, dtype, seed=22)
    check(queries(40, 4, 2 * Hkv, D), s)
