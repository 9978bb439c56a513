"""The operators together: the example generates, and a forward pass of it agrees with the network in fp64."""
import sys
from pathlib import Path

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, str(Path(__file__).resolve().parents[1] / "examples"))

pytestmark = pytest.mark.gpu


def decode(w, fmt):
    """fp64 values of quantised weights."""
    codes, scales = w
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    table = torch.cat([table, -table])
    c = ((codes[..., None] >> (4 * torch.arange(8, device="cuda", dtype=torch.int32))) & 15).long()
    v = table[c.reshape(codes.shape[0], scales.shape[1], -1)]
    s = scales.view(torch.float8_e4m3fn).double() if fmt == "nvfp4" else torch.exp2(scales.double() - 127)
    return (v * s[..., None]).reshape(codes.shape[0], -1)


@pytest.mark.parametrize("fmt,cache,window", [("nvfp4", torch.bfloat16, 0), ("mxfp4", torch.float8_e4m3fn, 0),
                                              ("nvfp4", torch.bfloat16, 24)])
@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_generation_runs(fmt, cache, window, temperature):
    """Prompts stay, every sequence grows by what was asked for, refused and accepted drafts both occur.  (Tokens of
    runs with and without drafts are not compared: a last bit that another row count's order of sums turns can become
    a whole step of a 4-bit activation code.)"""
    import batched_verify as ex
    from quantized_matmul_speculative_gb300 import binding

    cfg = ex.Config(fmt=fmt, cache=cache, window=window, sinks=2 if window else 0, vocab=300, mlp=1024)
    prompts = [[5, 6, 7], [1], list(range(20, 57)), [9] * 18, [3, 3], [250, 4]]
    out, offered, taken = ex.generate(ex.Decoder(cfg, 6, 360), prompts, steps=40, k=6, temperature=temperature)
    assert binding.device_status() == 0
    assert 0 <= taken <= offered and offered > 0
    for h, p in zip(out, prompts):
        assert h[:len(p)] == p and len(h) >= len(p) + 40 and all(0 <= t < 300 for t in h)


def test_forward_against_fp64():
    """One forward pass of prompts of different lengths against the same network in fp64 on the dequantised weights.
    What is rounded on the way (activations to 4 bits, bf16 between the operators) is rounded there too, so logits
    differ by single steps of those roundings only: a tenth of their spread at most."""
    import batched_verify as ex
    from quantized_matmul_speculative_gb300 import binding

    cfg = ex.Config(vocab=500)
    model = ex.Decoder(cfg, 3, 64)
    rows = [[7, 8, 9, 10, 11, 12, 13], [3, 4], [400]]
    M = 7
    tokens = torch.tensor([r + [0] * (M - len(r)) for r in rows], device="cuda")
    n = torch.tensor([len(r) for r in rows], dtype=torch.int32, device="cuda")
    got = model.forward(tokens, n, n).double()

    def project(x, w):
        v = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        binding.quantize_mx(x.to(torch.bfloat16), cfg.fmt, values=v)
        return v.double() @ decode(w, cfg.fmt).t()

    def bf(x):
        return x.to(torch.bfloat16).double()

    def norm(x):
        return torch.nn.functional.rms_norm(x.to(torch.bfloat16), (cfg.hidden,)).double()

    for b, r in enumerate(rows):
        x = model.embedding[torch.tensor(r, device="cuda")].double()
        L, G = len(r), cfg.q_heads // cfg.kv_heads
        for block in model.blocks:
            q, k, v = bf(project(norm(x), block["qkv"])).view(L, -1, cfg.head_dim).split([cfg.q_heads, cfg.kv_heads, cfg.kv_heads], 1)
            s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(G, 1)) / cfg.head_dim ** 0.5
            s = s.masked_fill(torch.ones(L, L, device="cuda", dtype=torch.bool).triu(1), float("-inf"))
            a = bf(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v.repeat_interleave(G, 1)))
            x = bf(x + bf(project(a.reshape(L, -1), block["o"])))
            gate, up = bf(project(norm(x), block["up"])).chunk(2, 1)
            x = bf(x + bf(project(bf(bf(torch.nn.functional.silu(gate)) * up), block["down"])))
        want = project(norm(x), model.head)
        err = (got[b, :L] - want).pow(2).mean().sqrt() / want.std()
        assert err < 0.1, float(err)
