"""What paged attention's outputs hold beyond the general bounds: the weights' bits, infinite values that a row sees,
and scales at the ends of their range.

A bf16 cache's weights enter the second product with 16 bits: beside what test_gpu_paged derives for the scores, an output
may be off by (2^-15 + n 2^-24) P + 2^-9 |o|, with P = sum_j p_j |v_j| and n the tokens, for the fp32 sums over them.  An
E4M3 cache's are fp16: 2^-11 in the place of 2^-15."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding
from test_gpu_paged import Cache, check, queries, reference

pytestmark = pytest.mark.gpu


def bf16(x):
    return torch.tensor(x, dtype=torch.float64).to(torch.bfloat16).double().numpy()


def badly_rounded():
    """A bf16 score below 0 whose weight e^x lies as far from bf16's values as any (relatively)."""
    x = np.unique(bf16(-np.linspace(0.05, 0.69, 2000)))
    w = np.exp(x)
    return float(x[np.argmax(np.abs(bf16(w) - w) / w)])


@pytest.mark.parametrize("D,M,Hq", [(64, 1, 4), (64, 8, 4), (128, 1, 4), (128, 8, 4), (256, 2, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_weights_that_cancel(dtype, D, M, Hq):
    """Half of the tokens weigh 1, half e^x; their values are of opposite signs, so that the weights' last bits stay."""
    n = 2000
    c = Cache([n], 1, D, 16, dtype)
    x = badly_rounded()
    if dtype != torch.bfloat16:
        x = -0.46875  # of E4M3's values the one whose weight fp16 rounds worst, by 0.63 2^-11
    q = torch.zeros(1, M, Hq, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 1.0
    light = torch.arange(n, device="cuda") % 2 == 1
    for kv, a, b in ((0, 0.0, x), (1, 1.0, -1.0 / math.exp(x))):
        row = torch.zeros(n, 1, D, device="cuda")
        row[light] = b if kv else 0.0
        row[light, :, 0] = b
        row[~light] = a if kv else 0.0
        row[~light, :, 0] = a
        row = row.to(dtype)
        cache = (c.k, c.v)[kv]
        raw = cache if dtype == torch.bfloat16 else cache.view(torch.uint8)
        j = torch.arange(n, device="cuda")
        raw[c.table[0].long()[j // 16], j % 16] = row if dtype == torch.bfloat16 else row.view(torch.uint8)
        c.dense[0][kv] = row.double()
    out, _ = binding.paged_attention(q, *c.args(), scale=1.0, return_lse=True)
    o, _, bo, _ = reference(q, c, [M], 1.0, 0, 0)
    P = 2.0 / (1 + math.exp(x))
    bits = 2.0**-15 if dtype == torch.bfloat16 else 2.0**-11
    bound = (bits + n * 2.0**-24) * P + 2.0**-9 * o.abs()
    assert ((out.double() - o).abs() <= bound).all(), float(((out.double() - o).abs() / bound).max())


@pytest.mark.parametrize("D,M,Hq", [(64, 1, 4), (128, 1, 4), (128, 8, 8), (256, 4, 4)])
@pytest.mark.parametrize("token", [0, 5, 299])
def test_infinite_values_that_a_row_sees(D, M, Hq, token):
    """A value of +inf at a token that rows see gives them +inf in that column, and the other columns do not change."""
    c = Cache([300], 1, D, 16, seed=D + token)
    q = queries(1, M, Hq, D)
    for std in (0.05, 1.0, 3.0):  # from flat weights to ones that a single token leads
        o0, l0 = binding.paged_attention(q * std, *c.args(), return_lse=True)
        at = int(c.table[0, token // 16]), token % 16
        was = c.v[at][0, 3].clone()
        c.v[at][0, 3] = float("inf")
        o1, l1 = binding.paged_attention(q * std, *c.args(), return_lse=True)
        c.v[at][0, 3] = was
        sees = torch.tensor([300 - M + i >= token for i in range(M)], device="cuda")
        assert torch.equal(l0, l1)
        assert (o1[0, sees][..., 3] == math.inf).all()
        assert torch.equal(o1[0, ~sees], o0[0, ~sees])
        rest = torch.arange(D, device="cuda") != 3
        assert torch.equal(o1[..., rest], o0[..., rest])


@pytest.mark.parametrize("D,M,Hq", [(64, 1, 4), (64, 4, 8), (128, 1, 1), (256, 1, 2)])
@pytest.mark.parametrize("n,where", [(3000, 0), (3000, 2999), (40000, 17)])
def test_light_tokens_of_an_e4m3_cache(D, M, Hq, n, where):
    """One token leads a row and has value 0; the others, e^-18 (2^-26) of it, are all that the output is made of."""
    c = Cache([n], 1, D, 16, torch.float8_e4m3fn)
    q = torch.zeros(1, M, Hq, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 1.0
    j = torch.arange(n, device="cuda")
    k, v = torch.zeros(n, 1, D, device="cuda"), torch.ones(n, 1, D, device="cuda")
    k[:, :, 0] = -18.0
    k[where, :, 0], v[where] = 0.0, 0.0
    for cache, kv, x in ((c.k, 0, k), (c.v, 1, v)):
        cache.view(torch.uint8)[c.table[0].long()[j // 16], j % 16] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        c.dense[0][kv] = x.double()
    out, lse = binding.paged_attention(q, *c.args(), scale=1.0, return_lse=True)
    o, l, _, bl = reference(q, c, [M], 1.0, 0, 0)
    assert ((out.double() - o).abs() <= (2.0**-11 + n * 2.0**-24 + 2.0**-9) * o).all(), (out.flatten()[0].item(), o.flatten()[0].item())
    assert ((lse.double() - l).abs() <= bl).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("scale", [0.0, 1e-38, 1e-28, -1e-28])
@pytest.mark.parametrize("size", [1e-25, 1e-20, 1.0])
def test_vanishing_scores(size, scale, dtype):
    """Queries and scales whose products are nothing beside 1: every row's mean over what it sees, and no more."""
    c = Cache([77, 3], 2, 128, 16, dtype, seed=6)
    check(c, (queries(2, 4, 8, 128).float() * size).bfloat16(), scale=scale)
