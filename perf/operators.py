"""Operators of a batched speculative-decoding verify step: their cases, plain forms and 64-bit definitions.

quantize   rows -> microscaled codes and scale bytes (mxfp4, nvfp4, mxfp8)
matmul     product of two microscaled 4-bit matrices, any number of rows
append     new key / value rows into a paged cache (bf16 or FP8 E4M3)
attention  1..16 new rows of each sequence over its paged cache, with window and sinks
verify     drafted tokens against the target's logits, from given random numbers

With ``own`` false, ``run`` computes the plain form (elementary torch
operations in 32 bits); with ``own`` true it calls the framework.
"""
import math

import torch

own = False

FORMATS = {"mxfp4": (4, 32), "nvfp4": (4, 16), "mxfp8": (8, 32)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one verify step's activations before a projection: 16 rows, latency counts
        dict(name="quantize 16x5120 mxfp4", op="quantize", rows=16, K=5120, fmt="mxfp4", dtype="bf16"),
        # a 27B-class gate+up weight matrix, converted once when a model is loaded
        dict(name="quantize 34816x5120 nvfp4", op="quantize", rows=34816, K=5120, fmt="nvfp4", dtype="bf16"),
        # one sequence's draft rows through one square layer: the smallest product, fp32 result
        dict(name="matmul 8x5120x5120 mxfp4", op="matmul", M=8, N=5120, K=5120, fmt="mxfp4", out="f32"),
        # about 125 sequences x 8 draft rows through gate+up: tensor-core bound
        dict(name="matmul 1000x34816x5120 nvfp4", op="matmul", M=1000, N=34816, K=5120, fmt="nvfp4", out="bf16"),
        # the new rows of four sequences into a bf16 cache: latency
        dict(name="append 4x5 bf16", op="append", B=4, M=5, Hkv=8, D=128, page=16, lmin=90, lmax=700, ragged=True,
             cache="bf16"),
        # a full batch of draft rows into an FP8 cache
        dict(name="append 128x16 e4m3", op="append", B=128, M=16, Hkv=8, D=128, page=64, lmin=16, lmax=257, ragged=False,
             cache="e4m3"),
        # plain decoding of a few short sequences: latency
        dict(name="attention 4x1 short", op="attention", B=4, M=1, Hq=32, Hkv=8, D=128, page=16, lmin=1, lmax=1000,
             ragged=False, window=0, sinks=0, cache="bf16"),
        # one long document, one new token: the length is all there is to split
        dict(name="attention 1x1 long", op="attention", B=1, M=1, Hq=32, Hkv=8, D=128, page=16, lmin=65001, lmax=65001,
             ragged=False, window=0, sinks=0, cache="bf16"),
        # a batched verify step, 8 draft rows for each of 32 sequences of very different lengths
        dict(name="attention 32x8 ragged", op="attention", B=32, M=8, Hq=32, Hkv=8, D=128, page=64, lmin=8, lmax=8200,
             ragged=True, window=0, sinks=0, cache="bf16"),
        # sliding-window layer with sinks on an FP8 cache, long sequences
        dict(name="attention 16x4 window e4m3", op="attention", B=16, M=4, Hq=64, Hkv=8, D=64, page=32, lmin=500,
             lmax=30000, ragged=False, window=4096, sinks=4, cache="e4m3"),
        # one sequence's seven drafts, bf16 logits: latency
        dict(name="verify 1x7x32000", op="verify", B=1, k=7, V=32000, dtype="bf16", q=True, greedy=0.0),
        # a batch of 64 sequences, fp32 logits over a large vocabulary, a quarter of them greedy
        dict(name="verify 64x5x128000", op="verify", B=64, k=5, V=128000, dtype="f32", q=True, greedy=0.25),
    ]


def _log_int(rng, lo, hi, step=1):
    """An integer of [lo, hi], spread over its logarithm, a multiple of `step`."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi and v != 3 * 1024:
            return v


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "append", "attention", "attention", "attention", "verify"])
    if op == "quantize":
        K = _log_int(rng, 32, 34816, 32)
        rows = _log_int(rng, 1, max(2, min(34816, 34816 * 5120 // K)))
        return dict(op=op, rows=rows, K=K, fmt=rng.choice(["mxfp4", "nvfp4", "mxfp8"]), dtype=rng.choice(["bf16", "f32"]))
    if op == "matmul":
        while True:
            M, N, K = _log_int(rng, 1, 2048), _log_int(rng, 16, 34816), _log_int(rng, 32, 17408, 32)
            if M * N * K <= 1000 * 34816 * 5120 and N * K <= 34816 * 5120:
                return dict(op=op, M=M, N=N, K=K, fmt=rng.choice(["mxfp4", "nvfp4"]), out=rng.choice(["bf16", "f32"]))
    if op == "append":
        M = rng.randint(1, 16)
        return dict(op=op, B=_log_int(rng, 1, 128), M=M, Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 256]),
                    page=rng.choice([1, 16, 24, 32, 64]), lmin=M, lmax=_log_int(rng, 17, 300), ragged=rng.random() < 0.5,
                    cache=rng.choice(["bf16", "e4m3"]))
    if op == "attention":
        while True:
            B, M, lmax = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 3, 5, 8, 11, 16]), _log_int(rng, 20, 65000)
            Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([64, 128, 128, 256])
            if B * lmax * Hkv * D <= 32 * 8200 * 8 * 128 and B * lmax * Hkv * G * M * D <= 32 * 8200 * 32 * 8 * 128:
                window = _log_int(rng, 16, 8192) if rng.random() < 0.4 else 0
                return dict(op=op, B=B, M=M, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([1, 16, 24, 32, 64, 128]),
                            lmin=min(lmax, rng.choice([1, M, lmax])), lmax=lmax, ragged=rng.random() < 0.5, window=window,
                            sinks=rng.choice([0, 1, 4, 64]) if window else 0, cache=rng.choice(["bf16", "e4m3"]))
    while True:
        B, k, V = _log_int(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 7, 8, 15]), _log_int(rng, 1000, 200000)
        if B * (k + 1) * V <= 64 * 6 * 128000:
            return dict(op=op, B=B, k=k, V=V, dtype=rng.choice(["bf16", "f32"]), q=rng.random() < 0.8,
                        greedy=rng.choice([0.0, 0.5]))


def _lengths(case):
    """The cache lengths (evenly spread, new rows included) and new rows of each sequence, before they are shuffled."""
    B, M = case["B"], case["M"]
    lens = [case["lmin"] + (case["lmax"] - case["lmin"]) * i // max(1, B - 1) if B > 1 else case["lmax"] for i in range(B)]
    rows = [1 + (5 * i + M - 1) % M if case["ragged"] else M for i in range(B)]
    return lens, rows


# ------------------------------------------------------------------- the inputs
def _cache(case, g):
    """A paged cache of randomly placed pages, its block table (-1 past a sequence's pages) and lengths."""
    dev = "cuda"
    B, page, Hkv, D = case["B"], case["page"], case["Hkv"], case["D"]
    lens, rows = _lengths(case)
    order = torch.randperm(B, generator=g, device=dev).cpu().tolist()
    lens, rows = [lens[i] for i in order], [rows[i] for i in order]
    counts = [-(-n // page) for n in lens]
    total = sum(counts)
    free = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(counts)), -1, dtype=torch.int32, device=dev)
    at = torch.tensor(counts, device=dev)
    inside = torch.arange(max(counts), device=dev)[None, :] < at[:, None]
    table[inside] = free
    shape = (total, page, Hkv, D)
    scale = 1.0 if case["cache"] == "bf16" else 0.0625

    def pages():
        x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g)
        return x if case["cache"] == "bf16" else (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn)

    return {"k_cache": pages(), "v_cache": pages(), "table": table, "k_scale": scale, "v_scale": scale,
            "lengths": torch.tensor(lens, dtype=torch.int32, device=dev),
            "q_lens": torch.tensor(rows, dtype=torch.int32, device=dev)}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, op = "cuda", case["op"]
    s = {"case": case}
    if op == "quantize":
        # activations or weights with channels of different sizes
        x = torch.randn(case["rows"], case["K"], generator=g, device=dev)
        x *= torch.exp(0.7 * torch.randn(case["K"], generator=g, device=dev))
        s["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "matmul":
        bits, group = FORMATS[case["fmt"]]

        def matrix(rows):
            codes = torch.randint(-2**31, 2**31, (rows, case["K"] * bits // 32), generator=g, device=dev, dtype=torch.int64)
            lo, hi = (121, 128) if case["fmt"] == "mxfp4" else (0x28, 0x40)  # 2^-6..1; E4M3 0.25..1.875
            scales = torch.randint(lo, hi, (rows, case["K"] // group), generator=g, device=dev).to(torch.uint8)
            return codes.to(torch.int32), scales

        s["xq"], s["xs"] = matrix(case["M"])
        s["wq"], s["ws"] = matrix(case["N"])
    elif op in ("append", "attention"):
        s.update(_cache(case, g))
        new = (case["B"], case["M"], case["Hkv"], case["D"])
        if op == "append":
            s["k_new"] = torch.randn(new, generator=g, device=dev).to(torch.bfloat16)
            s["v_new"] = torch.randn(new, generator=g, device=dev).to(torch.bfloat16)
        else:
            s["q"] = torch.randn(case["B"], case["M"], case["Hq"], case["D"], generator=g, device=dev).to(torch.bfloat16)
    else:
        B, k, V = case["B"], case["k"], case["V"]
        target = 2.5 * torch.randn(B, k + 1, V, generator=g, device=dev)
        draft = target[:, :k] + 0.7 * torch.randn(B, k, V, generator=g, device=dev)
        q = torch.softmax(draft, -1)
        gumbel = torch.empty_like(q).exponential_(generator=g)
        s["draft"] = (q / gumbel).argmax(-1).to(torch.int32)
        s["q"] = q if case["q"] else None
        s["logits"] = target.to(DTYPES[case["dtype"]])
        s["u"] = torch.rand(B, k, generator=g, device=dev)
        s["noise"] = torch.empty(B, V, device=dev).exponential_(generator=g).clamp_(min=1e-20)
        greedy = torch.arange(B, device=dev) < int(case["greedy"] * B)
        s["temperature"] = torch.where(greedy, 0.0, 0.7 + 0.6 * torch.rand(B, generator=g, device=dev))
        s["draft_lens"] = torch.where(torch.rand(B, generator=g, device=dev) < 0.8, k,
                                      torch.randint(0, k + 1, (B,), generator=g, device=dev)).to(torch.int32)
    return s


# ------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from quantized_matmul_speculative_gb300 import binding

    case = s["case"]
    op = case["op"]
    if op == "quantize":
        values = torch.empty_like(s["x"], dtype=torch.bfloat16)
        codes, scales = binding.quantize_mx(s["x"], case["fmt"], values=values)
        return {"values": values, "codes": codes, "scales": scales}
    if op == "matmul":
        return binding.matmul_mx(s["xq"], s["xs"], s["wq"], s["ws"], case["fmt"], out_dtype=DTYPES[case["out"]])
    if op == "append":
        binding.kv_append(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], q_lens=s["q_lens"],
                          k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"k": s["k_cache"], "v": s["v_cache"]}
    if op == "attention":
        out, lse = binding.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], q_lens=s["q_lens"],
                                           window=case["window"], sinks=case["sinks"], k_scale=s["k_scale"],
                                           v_scale=s["v_scale"], return_lse=True)
        return {"out": out, "lse": lse}
    tokens, accepted = binding.verify_draft(s["logits"], s["draft"], s["q"], s["u"], s["noise"], s["temperature"],
                                            draft_lens=s["draft_lens"])
    return {"tokens": tokens, "accepted": accepted}


def _round_e2m1(a):
    """Codes 0..7 of magnitudes `a`: nearest of E2M1's values, ties to the even code, saturating."""
    return ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())


def _power(e):
    """2^e in 32 bits, for int32 tensors e in [-127, 127]: the exponent field, or the subnormal 2^-127."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantize_plain(x, fmt):
    bits, group = FORMATS[fmt]
    x = x.float().reshape(x.shape[0], -1, group)
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        scales = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        size, byte = scales.float(), scales.view(torch.uint8)
    else:
        top = 2 if fmt == "mxfp4" else 8
        e = torch.where(amax > 0, (torch.frexp(amax)[1] - 1 - top).clamp(-127, 127), -127).int()
        size, byte = _power(e), (e + 127).to(torch.uint8)
    y = torch.where(size > 0, x / size, 0.0)
    if fmt == "mxfp8":
        y8 = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        value, code = y8.float(), y8.view(torch.uint8).int()
    else:
        code = _round_e2m1(y.abs())
        value = torch.where(torch.signbit(y), -1.0, 1.0) * torch.tensor(E2M1, device=x.device)[code]
        code = code + 8 * torch.signbit(y).int()
    values = (value * size).reshape(x.shape[0], -1).to(torch.bfloat16)
    per = 32 // bits
    place = torch.arange(per, device=x.device, dtype=torch.int32) * bits
    words = (code.reshape(x.shape[0], -1, per) << place).sum(-1, dtype=torch.int32)
    return {"values": values, "codes": words, "scales": byte[..., 0]}


def _dequantize_plain(codes, scales, fmt):
    bits, group = FORMATS[fmt]
    place = torch.arange(8, device=codes.device, dtype=torch.int32) * 4
    c = ((codes[..., None] >> place) & 15).reshape(codes.shape[0], -1, group)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    size = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else _power(scales.int() - 127)
    return (table[c] * size[..., None]).reshape(codes.shape[0], -1)


def _append_plain(s):
    L, m, table = s["lengths"].long(), s["q_lens"].long(), s["table"].long()
    M, page = s["k_new"].shape[1], s["k_cache"].shape[1]
    i = torch.arange(M, device=L.device)[None, :]
    pos = L[:, None] - m[:, None] + i
    valid = (i < m[:, None]) & (pos >= 0)
    pos = pos.clamp(min=0)
    slot = torch.gather(table, 1, (pos // page).clamp(max=table.shape[1] - 1)), pos % page
    slot = slot[0][valid], slot[1][valid]
    for new, cache, scale in ((s["k_new"], s["k_cache"], s["k_scale"]), (s["v_new"], s["v_cache"], s["v_scale"])):
        rows = new[valid]
        if cache.dtype != torch.bfloat16:
            rows = (rows.float() / scale).clamp(-448.0, 448.0).to(cache.dtype).view(torch.uint8)
            cache = cache.view(torch.uint8)
        cache[slot] = rows
    return {"k": s["k_cache"], "v": s["v_cache"]}


def _attention_plain(s):
    case, q = s["case"], s["q"].float()
    B, M, Hq, D = q.shape
    Hkv, page = case["Hkv"], case["page"]
    table = s["table"].long().clamp(min=0)
    k = s["k_cache"][table].reshape(B, -1, Hkv, D).float() * s["k_scale"]
    v = s["v_cache"][table].reshape(B, -1, Hkv, D).float() * s["v_scale"]
    L, m = s["lengths"].long()[:, None, None], s["q_lens"].long()[:, None, None]
    i = torch.arange(M, device=q.device)[None, :, None]
    j = torch.arange(k.shape[1], device=q.device)[None, None, :]
    pos = L - m + i
    seen = (j <= pos) & (i < m)
    if case["window"]:
        seen &= (j > pos - case["window"]) | (j < case["sinks"])
    seen = seen[:, None, None]  # [B, 1, 1, M, tokens]
    qs = q.reshape(B, M, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    scores = torch.matmul(qs, k.permute(0, 2, 3, 1)).reshape(B, Hkv, Hq // Hkv, M, -1) * (1.0 / math.sqrt(D))
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    p = p / torch.where(total > 0, total, 1.0)
    out = torch.matmul(p.reshape(B, Hkv, -1, k.shape[1]), v.permute(0, 2, 1, 3)).reshape(B, Hkv, Hq // Hkv, M, D)
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B, M, Hq, D).to(torch.bfloat16),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, M, Hq)}


def _first(x, top):
    """The lowest index at which x equals its largest value `top`."""
    index = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == top, index, x.shape[-1]).amin(-1)


def _verify_plain(s):
    x = s["logits"].float()
    B, rows, V = x.shape
    k = rows - 1
    T = s["temperature"][:, None, None]
    greedy = s["temperature"] == 0
    best = _first(x, x.amax(-1, keepdim=True))  # [B, k + 1]
    z = x / torch.where(T > 0, T, 1.0)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    d = s["draft"].long()
    p_d = torch.gather(p[:, :k], 2, d[..., None])[..., 0]
    q_d = torch.gather(s["q"], 2, d[..., None])[..., 0] if s["q"] is not None else torch.ones_like(p_d)
    yes = torch.where(greedy[:, None], best[:, :k] == d, s["u"] * q_d < p_d)
    n_draft = s["draft_lens"].long()
    i = torch.arange(k, device=x.device)[None, :]
    n = torch.cumprod((yes & (i < n_draft[:, None])).int(), 1).sum(1)  # accepted drafts
    b = torch.arange(B, device=x.device)
    p_n = p[b, n]
    refused = n < n_draft
    at = n.clamp(max=k - 1)
    if s["q"] is not None:
        q_n = s["q"][b, at]
    else:
        q_n = (torch.arange(V, device=x.device)[None, :] == d[b, at][:, None]).float()
    rest = (p_n - q_n).clamp(min=0.0)
    if s["q"] is None:
        rest = torch.where(q_n > 0, 0.0, p_n)
    some = rest.amax(-1, keepdim=True) > 0
    weight = torch.where(refused[:, None] & some, rest, p_n)
    ratio = torch.where(weight > 0, weight / s["noise"], 0.0)
    drawn = _first(ratio, ratio.amax(-1, keepdim=True))
    last = torch.where(greedy, best[b, n], drawn)
    j = torch.arange(k + 1, device=x.device)[None, :]
    padded = torch.nn.functional.pad(d, (0, 1))
    tokens = torch.where(j < n[:, None], padded, torch.where(j == n[:, None], last[:, None], -1))
    return {"tokens": tokens.to(torch.int32), "accepted": n.to(torch.int32)}


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        return _quantize_plain(s["x"], case["fmt"])
    if op == "matmul":
        x, w = _dequantize_plain(s["xq"], s["xs"], case["fmt"]), _dequantize_plain(s["wq"], s["ws"], case["fmt"])
        return torch.matmul(x, w.t()).to(DTYPES[case["out"]])
    if op == "append":
        return _append_plain(s)
    return _attention_plain(s) if op == "attention" else _verify_plain(s)


# ------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "quantize":
        bits, group = FORMATS[case["fmt"]]
        n = case["rows"] * case["K"]
        return {"bytes": n * ((2 if case["dtype"] == "bf16" else 4) + bits / 8 + 1 / group + 2), "flops": 2 * n}
    if op == "matmul":
        M, N, K, group = case["M"], case["N"], case["K"], FORMATS[case["fmt"]][1]
        return {"bytes": (M + N) * K * (0.5 + 1 / group) + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    if op == "verify":
        B, k, V = case["B"], case["k"], case["V"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": B * V * (size * (k + 1) + 4 + (4 if case["q"] else 0)), "flops": 3 * B * V * (k + 1)}
    lens, rows = _lengths(case)
    size = 2 if case["cache"] == "bf16" else 1
    if op == "append":
        n = sum(min(r, n) for r, n in zip(rows, lens)) * case["Hkv"] * case["D"]
        return {"bytes": 2 * n * (2 + size), "flops": 2 * n}
    W, S = case["window"], case["sinks"]
    tokens = pairs = 0
    for n, r in zip(lens, rows):
        r = min(r, n)
        first = max(0, n - r - W + 1) if W else 0
        tokens += n - first + min(S, first)
        for p in range(n - r, n):
            first = max(0, p - W + 1) if W else 0
            pairs += p + 1 - first + min(S, first)
    D, Hq = case["D"], case["Hq"]
    return {"bytes": 2 * tokens * case["Hkv"] * D * size + sum(rows) * Hq * (4 * D + 4), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------- the definition, in 64 bits
def _exp2(e):
    """2^e in 64 bits, exactly: the exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e2m1(code):
    """Value of E2M1 codes from their fields: sign, two exponent bits (bias 1), one mantissa bit."""
    c = code.long()
    e, f = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * _exp2(e - 1))
    return torch.where(c >= 8, -v, v)


def _e4m3(byte):
    """Value of finite E4M3 bytes from their fields."""
    c = byte.long()
    e, f = (c >> 3) & 15, (c & 7).double() / 8
    v = torch.where(e == 0, f * 2.0**-6, (1 + f) * _exp2(e - 7))
    return torch.where(c >= 128, -v, v)


def _nearest(y, grid):
    """The nearest value of the ascending magnitudes `grid` (their index's last bit decides ties), with y's sign."""
    a = y.abs()
    hi = torch.searchsorted(grid, a).clamp(1, len(grid) - 1)
    lo = hi - 1
    mid = 0.5 * (grid[lo] + grid[hi])
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def exact(case, seed):
    s = prepare(case, seed)
    op, dev = case["op"], "cuda"
    grid8 = _e4m3(torch.arange(127, device=dev))
    if op == "quantize":
        bits, group = FORMATS[case["fmt"]]
        grid = grid8 if case["fmt"] == "mxfp8" else _e2m1(torch.arange(8, device=dev))
        parts = []
        for x in s["x"].split(2048):
            x = x.double().reshape(x.shape[0], -1, group)
            a = x.abs().amax(-1, keepdim=True)
            if case["fmt"] == "nvfp4":
                size = grid8[_nearest(a / 6, grid8)]
            else:
                top = 8 if case["fmt"] == "mxfp8" else 2
                size = _exp2((torch.frexp(a)[1] - 1 - top).clamp(-127, 127))
            y = torch.where(size > 0, x / size, 0.0)
            v = grid[_nearest(y, grid)] * size
            parts.append(torch.where(y < 0, -v, v).reshape(x.shape[0], -1))
        return {"values": torch.cat(parts), "codes": None, "scales": None}
    if op == "matmul":
        def matrix(codes, scales):
            b = codes.contiguous().view(torch.uint8)
            v = torch.stack((_e2m1(b & 15), _e2m1(b >> 4)), -1).reshape(codes.shape[0], scales.shape[1], -1)
            size = _e4m3(scales) if case["fmt"] == "nvfp4" else _exp2(scales.long() - 127)
            return (v * size[..., None]).reshape(codes.shape[0], -1)

        x = matrix(s["xq"], s["xs"])
        return torch.cat([x @ matrix(w, z).t() for w, z in zip(s["wq"].split(4096), s["ws"].split(4096))], 1)
    if op == "append":
        out = []
        for new, cache, scale in ((s["k_new"], s["k_cache"], s["k_scale"]), (s["v_new"], s["v_cache"], s["v_scale"])):
            full = cache.double()
            flat = full.view(-1, case["Hkv"], case["D"])
            for b, (n, m) in enumerate(zip(s["lengths"].tolist(), s["q_lens"].tolist())):
                keep = max(0, m - n)
                pos = torch.arange(n - m + keep, n, device=dev)
                rows = new[b, keep:m].double()
                if case["cache"] != "bf16":
                    y = rows / scale
                    rows = torch.sign(y) * grid8[_nearest(y, grid8)]
                flat[s["table"][b].long()[pos // case["page"]] * case["page"] + pos % case["page"]] = rows
            out.append(full)
        return {"k": out[0], "v": out[1]}
    if op == "attention":
        B, M, Hq, Hkv, D = case["B"], case["M"], case["Hq"], case["Hkv"], case["D"]
        o = torch.zeros(B, M, Hq, D, dtype=torch.float64, device=dev)
        lse = torch.full((B, M, Hq), -math.inf, dtype=torch.float64, device=dev)
        for b, (n, m) in enumerate(zip(s["lengths"].tolist(), s["q_lens"].tolist())):
            at = torch.arange(n, device=dev)
            at = s["table"][b].long()[at // case["page"]] * case["page"] + at % case["page"]
            k = s["k_cache"].view(-1, Hkv, D)[at].double() * s["k_scale"]
            v = s["v_cache"].view(-1, Hkv, D)[at].double() * s["v_scale"]
            for i in range(m):
                p = n - m + i
                if p < 0:
                    continue
                j = torch.arange(p + 1, device=dev)
                if case["window"]:
                    j = j[(j > p - case["window"]) | (j < case["sinks"])]
                x = torch.einsum("hgd,thd->hgt", s["q"][b, i].double().view(Hkv, Hq // Hkv, D), k[j]) / math.sqrt(D)
                lse[b, i] = torch.logsumexp(x, -1).reshape(-1)
                o[b, i] = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v[j]).reshape(Hq, D)
        return {"out": o, "lse": lse}
    k = case["k"]
    tokens, accepted = torch.full((case["B"], k + 1), -1, dtype=torch.int64), []
    for b, (T, drafts) in enumerate(zip(s["temperature"].tolist(), s["draft_lens"].tolist())):
        n = 0
        while True:
            x, d = s["logits"][b, n].double(), int(s["draft"][b, min(n, k - 1)])
            best = int(torch.nonzero(x == x.max())[0])
            p = torch.softmax(x / T, -1) if T > 0 else None
            q = s["q"][b, n].double() if s["q"] is not None and n < drafts else None
            q_d = float(q[d]) if q is not None else 1.0
            if n == drafts or not (best == d if p is None else float(s["u"][b, n]) * q_d < float(p[d])):
                break
            tokens[b, n] = d
            n += 1
        if p is None:
            tokens[b, n] = best
        else:
            weight = p
            if n < drafts:
                q = q if q is not None else torch.nn.functional.one_hot(torch.tensor(d, device=dev), case["V"]).double() * 2
                weight = (p - q).clamp(min=0) if bool((p > q).any()) else p
            tokens[b, n] = int(torch.argmax(weight / s["noise"][b].double()))
        accepted.append(n)
    return {"tokens": tokens.to(torch.int32), "accepted": torch.tensor(accepted, dtype=torch.int32)}
