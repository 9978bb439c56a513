"""Attention behind a prefix of which one token holds nearly all the weight, and the rest in equal shares of 2^-24.5 of it:
the log-sum-exp has to hold them all, however many of them one CTA adds up.

All scores are exact (17 and 0), so that of the bounds in test_gpu_prefix.py d is 17 2^-22 (the scale and log2(e), each
rounded, and the lse's way back), with the output off by at most (2^-14 + 2 d) P + 2^-8 |o| (2^-11 more for E4M3), P = sum p |v|,
and the log-sum-exp by d + 2^-16 + 2^-20 |lse|."""
import math

import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("tokens,B,M,G,D", [(32768, 1, 1, 1, 64), (32768, 2, 16, 8, 64), (32768, 2, 16, 8, 128),
                                            (32768, 1, 1, 4, 128), (32768, 4, 8, 4, 256), (4096, 2, 16, 8, 64)])
def test_a_leading_token_and_a_long_flat_tail(tokens, B, M, G, D, dtype):
    heads, page = torch.cuda.get_device_properties(0).multi_processor_count, 128  # a head a CTA: its share is the whole prefix
    own = M
    k = torch.zeros(2 + B, page, heads, D, device="cuda")
    v = torch.zeros(2 + B, page, heads, D, device="cuda")
    k[0, 0, :, 0], k[0, 0, :, 1] = 4.0, 0.25
    v[..., 0] = v[..., 1] = v[..., 3] = 1.0
    v[..., 2] = -1.0
    v[0, 0, :, 1], v[0, 0, :, 2], v[0, 0, :, 3] = 0.0, 1.0, -1.0
    k, v = k.to(dtype), v.to(dtype)
    q = torch.zeros(B, M, heads * G, D, device="cuda")
    q[..., :2] = 4.0
    q = q.to(torch.bfloat16)
    prefix = torch.ones(tokens // page, dtype=torch.int32, device="cuda")  # the tail's page, again and again
    prefix[0] = 0
    table = torch.arange(2, 2 + B, dtype=torch.int32, device="cuda")[:, None]
    lengths = torch.full((B,), tokens + own, dtype=torch.int32, device="cuda")
    out, lse = binding.shared_prefix_attention(q, k, v, prefix, table, lengths, scale=1.0, return_lse=True)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    d = 17 * 2.0**-22
    weight = 2.0**-14 + (2.0**-11 if dtype == E4M3 else 0.0) + 2 * d
    for i in range(M):
        tail = (tokens + i) * math.exp(-17.0)  # tokens - 1 of the prefix and 1 + i own ones
        want = 17 + math.log1p(tail)
        assert float((lse[:, i].double() - want).abs().max()) <= d + 2.0**-16 + 2.0**-20 * want
        for column, (lead, rest) in enumerate(((1, 1), (0, 1), (1, -1), (-1, 1))):
            o, P = (lead + rest * tail) / (1 + tail), (abs(lead) + abs(rest) * tail) / (1 + tail)
            assert float((out[:, i, :, column].double() - o).abs().max()) <= weight * P + 2.0**-8 * abs(o)
