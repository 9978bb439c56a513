"""Operators of a served layer beside the small-M products: their cases, plain forms and 64-bit definitions.

route    router logits -> the k experts of every token and their weights (softmax or sigmoid, bias, groups)
rope     rotation of new queries and keys by their positions, keys and values into a paged cache on the way
prefix   attention of a batch whose sequences share a long prefix and have own tokens after it, all paged
lora     low-rank adapters of many requests beside a shared projection

With ``own`` false, ``run`` computes the plain form (elementary torch
operations in 32 bits; angles of positions and expert keys, whose borders
decide, in 64); with ``own`` true it calls the framework.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one token through a layer of 128 experts: latency
        dict(name="route 1x128 softmax", op="route", T=1, E=128, k=8, score="softmax", bias=False, groups=1, top=1,
             dtype="bf16"),
        # a prompt's tokens: 256 experts with a balancing bias, 8 groups of which a token may use 4
        dict(name="route 16384x256 sigmoid groups", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top=4, dtype="f32"),
        # the new rows of four sequences into a bf16 cache: latency
        dict(name="rope 4x5 bf16", op="rope", B=4, M=5, Hq=32, Hkv=8, D=128, rot=128, page=16, lmin=90, lmax=700,
             ragged=True, cache="bf16", axes=1, pairs="halves"),
        # a full batch of draft rows into an FP8 cache, partial rotation of neighbouring elements
        dict(name="rope 128x16 e4m3", op="rope", B=128, M=16, Hq=32, Hkv=8, D=128, rot=64, page=64, lmin=16, lmax=257,
             ragged=False, cache="e4m3", axes=1, pairs="neighbours"),
        # chunks of two prompts with pictures in them: positions along time, height and width
        dict(name="rope 2x4001 axes", op="rope", B=2, M=4001, Hq=32, Hkv=8, D=128, rot=128, page=16, lmin=4001, lmax=30000,
             ragged=True, cache="bf16", axes=3, pairs="halves"),
        # plain decoding of a few sequences behind a short instruction: latency
        dict(name="prefix 4x1 2048", op="prefix", B=4, M=1, Hq=32, Hkv=8, D=128, page=16, prefix=2048, lmin=1, lmax=300,
             ragged=False, cache="bf16"),
        # 32 sequences that ask about one long document, one new token each: the document's bytes
        dict(name="prefix 32x1 32768", op="prefix", B=32, M=1, Hq=32, Hkv=8, D=128, page=64, prefix=32768, lmin=1,
             lmax=1000, ragged=False, cache="bf16"),
        # a batched verify step of 64 sequences behind one document: the tensor cores
        dict(name="prefix 64x8 16384", op="prefix", B=64, M=8, Hq=32, Hkv=8, D=128, page=64, prefix=16384, lmin=8,
             lmax=700, ragged=True, cache="bf16"),
        # the same kind on an FP8 cache, small heads, pages that divide no tile
        dict(name="prefix 48x4 20016 e4m3", op="prefix", B=48, M=4, Hq=64, Hkv=8, D=64, page=24, prefix=20016, lmin=4,
             lmax=500, ragged=True, cache="e4m3"),
        # one token each of four requests with adapters of their own, a square projection: latency
        dict(name="lora 4x1 r16 5120x5120", op="lora", requests=4, rows=1, ragged=False, L=8, R=16, K=5120, N=5120,
             none=False, out="bf16"),
        # a verify step of 64 requests on 48 adapters, gate+up of a 27B-class layer, some requests without one
        dict(name="lora 64x4 r64 34816x5120", op="lora", requests=64, rows=4, ragged=True, L=48, R=64, K=5120, N=34816,
             none=True, out="bf16"),
        # prompts of six requests, down projection: the activations' bytes
        dict(name="lora 6x700 r16 5120x17408", op="lora", requests=6, rows=700, ragged=True, L=8, R=16, K=17408, N=5120,
             none=True, out="f32"),
    ]


def _log_int(rng, lo, hi, step=1):
    """An integer of [lo, hi], spread over its logarithm, a multiple of `step`."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi:
            return v


def draw(rng):
    op = rng.choice(["route", "route", "rope", "rope", "prefix", "prefix", "prefix", "lora", "lora", "lora"])
    if op == "route":
        E = rng.choice([8, 16, 40, 60, 64, 128, 160, 256, 384, 512])
        bias = rng.random() < 0.5
        groups = rng.choice([1, 1, 2, 4, 8])
        if E // groups < 8:
            groups = 1
        top = rng.randint(1, groups)
        k = rng.choice([1, 2, 4, 6, 8])
        return dict(op=op, T=_log_int(rng, 1, 16384 * 256 // E), E=E, k=min(k, top * (E // groups)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=bias, groups=groups, top=top,
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "rope":
        while True:
            M = rng.choice([1, 1, 2, 3, 5, 8, 16, _log_int(rng, 17, 4096)])
            B = _log_int(rng, 1, 128)
            Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 256])
            if B * M * Hkv * (G + 2) * D <= 8002 * 48 * 128:
                axes = rng.choice([1, 1, 1, 3])
                return dict(op=op, B=B, M=M, Hq=Hkv * G, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, 32]),
                            page=rng.choice([1, 16, 24, 32, 64]), lmin=M, lmax=M + _log_int(rng, 1, 1000),
                            ragged=rng.random() < 0.5, cache=rng.choice(["bf16", "e4m3"]), axes=axes,
                            pairs=rng.choice(["halves", "neighbours"]))
    if op == "prefix":
        while True:
            page = rng.choice([1, 16, 24, 32, 64, 128])
            B, M = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 3, 5, 8, 11, 16])
            Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([64, 128, 128, 256])
            prefix = _log_int(rng, max(page, 100), 65000, page)
            tail = M + _log_int(rng, 1, 1000)
            if (B * M * Hkv * G * D * prefix <= 64 * 8 * 32 * 128 * 16384 and B * M * Hkv * G * prefix <= 2**29
                    and prefix * Hkv * D <= 32768 * 8 * 128 and B * tail * Hkv * D <= 64 * 1000 * 8 * 128):
                return dict(op=op, B=B, M=M, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, prefix=prefix, lmin=M, lmax=tail,
                            ragged=rng.random() < 0.5, cache=rng.choice(["bf16", "bf16", "e4m3"]))
    while True:
        R, L = rng.choice([8, 16, 16, 32, 64, 128]), _log_int(rng, 1, 64)
        K, N = _log_int(rng, 64, 34816, 8), _log_int(rng, 16, 34816)
        requests, rows = _log_int(rng, 1, 64), rng.choice([1, 1, 2, 4, 8, 16, _log_int(rng, 17, 1000)])
        out = rng.choice(["bf16", "bf16", "f32"])
        case = dict(op="lora", requests=requests, rows=rows, ragged=rng.random() < 0.5, L=L, R=R, K=K, N=N,
                    none=rng.random() < 0.5, out=out)
        if (L * R * (K + N) <= 48 * 64 * (5120 + 34816) and requests * rows * (K + 2 * N) <= 6 * 700 * 32000
                and work(case)["bytes"] <= 48 * 64 * (5120 + 34816) * 2):
            return case


def _lengths(case):
    """The own tokens (evenly spread, new rows included) and new rows of each sequence, before they are shuffled."""
    B, M = case["B"], case["M"]
    lens = [case["lmin"] + (case["lmax"] - case["lmin"]) * i // max(1, B - 1) if B > 1 else case["lmax"] for i in range(B)]
    rows = [1 + (5 * i + M - 1) % M if case["ragged"] else M for i in range(B)]
    return lens, rows


def _requests(case):
    """(rows, adapter or -1) of each request: the adapters in turn, every eighth request without one where some are."""
    M = case["rows"]
    rows = [1 + (5 * i + M - 1) % M if case["ragged"] else M for i in range(case["requests"])]
    ids = [-1 if case["none"] and i % 8 == 5 else i % case["L"] for i in range(case["requests"])]
    return rows, ids


# ------------------------------------------------------------------- the inputs
def _cache(case, g, prefix):
    """A paged cache of randomly placed pages, the sequences' tables (-1 past their pages) and lengths, and the pages of
    a shared prefix of `prefix` tokens."""
    dev = "cuda"
    B, page, Hkv, D = case["B"], case["page"], case["Hkv"], case["D"]
    lens, rows = _lengths(case)
    order = torch.randperm(B, generator=g, device=dev).cpu().tolist()
    lens, rows = [lens[i] for i in order], [rows[i] for i in order]
    counts = [-(-n // page) for n in lens]
    shared = prefix // page
    total = sum(counts) + shared
    free = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(counts)), -1, dtype=torch.int32, device=dev)
    inside = torch.arange(max(counts), device=dev)[None, :] < torch.tensor(counts, device=dev)[:, None]
    table[inside] = free[shared:]
    shape = (total, page, Hkv, D)
    scale = 1.0 if case["cache"] == "bf16" else 0.0625

    def pages():
        x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g)
        return x if case["cache"] == "bf16" else (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn)

    return {"k_cache": pages(), "v_cache": pages(), "table": table, "k_scale": scale, "v_scale": scale,
            "prefix_pages": free[:shared].contiguous(),
            "lengths": torch.tensor([n + prefix for n in lens], dtype=torch.int32, device=dev),
            "q_lens": torch.tensor(rows, dtype=torch.int32, device=dev)}


def _sections(case):
    """Pairs of each position axis: a quarter for time, the others evenly for height and width."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return None
    t = half // 4
    h = (half - t) // 2
    return (t, h, half - t - h)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, op = "cuda", case["op"]
    s = {"case": case}
    if op == "route":
        T, E = case["T"], case["E"]
        x = 1.5 * torch.randn(T, E, generator=g, device=dev) + torch.randn(E, generator=g, device=dev)
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["bias"] = 0.1 * torch.randn(E, generator=g, device=dev) if case["bias"] else None
    elif op == "rope":
        s.update(_cache(case, g, 0))
        B, M, Hkv = case["B"], case["M"], case["Hkv"]
        # the three parts of one projection's output
        qkv = torch.randn(B, M, case["Hq"] + 2 * Hkv, case["D"], generator=g, device=dev).to(torch.bfloat16)
        s["q"], s["k_new"], s["v_new"] = qkv.split([case["Hq"], Hkv, Hkv], 2)
        s["inv_freq"] = 1e6 ** (-torch.arange(0, case["rot"], 2, device=dev).float() / case["rot"])
        s["positions"] = None
        if case["axes"] > 1:
            # a picture's rows after a text: one time, a grid of 40 columns
            at = s["lengths"].long()[:, None] - s["q_lens"].long()[:, None] + torch.arange(M, device=dev)[None, :]
            s["positions"] = torch.stack((at // 400, at // 400 + at % 400 // 40, at // 400 + at % 40)).to(torch.int32)
    elif op == "prefix":
        s.update(_cache(case, g, case["prefix"]))
        s["q"] = torch.randn(case["B"], case["M"], case["Hq"], case["D"], generator=g, device=dev).to(torch.bfloat16)
    else:
        rows, ids = _requests(case)
        L, R, K, N = case["L"], case["R"], case["K"], case["N"]
        perm = torch.randperm(L, generator=g, device=dev).cpu().tolist()
        ids = [perm[i] if i >= 0 else -1 for i in ids]
        s["ids"] = torch.repeat_interleave(torch.tensor(ids), torch.tensor(rows)).to(device=dev, dtype=torch.int32)
        T = sum(rows)
        s["x"] = torch.randn(T, K, generator=g, device=dev).to(torch.bfloat16)
        s["base"] = torch.randn(T, N, generator=g, device=dev).to(DTYPES[case["out"]])
        s["a"] = torch.empty(L, R, K, dtype=torch.bfloat16, device=dev).normal_(std=K**-0.5, generator=g)
        s["b"] = torch.empty(L, N, R, dtype=torch.bfloat16, device=dev).normal_(std=0.5 * R**-0.5, generator=g)
        s["scales"] = 0.5 + torch.rand(L, generator=g, device=dev)
    return s


# ------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from quantized_matmul_speculative_gb300 import binding

    case = s["case"]
    op = case["op"]
    if op == "route":
        experts, weights = binding.route_experts(s["logits"], case["k"], case["score"], bias=s["bias"], groups=case["groups"],
                                                 top_groups=case["top"], scale=2.5)
        return {"experts": experts, "weights": weights}
    if op == "rope":
        q = binding.rope_append(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                                s["inv_freq"], q_lens=s["q_lens"], positions=s["positions"], sections=_sections(case),
                                interleaved=case["pairs"] == "neighbours", k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
    if op == "prefix":
        out, lse = binding.shared_prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["prefix_pages"], s["table"],
                                                   s["lengths"], q_lens=s["q_lens"], k_scale=s["k_scale"],
                                                   v_scale=s["v_scale"], return_lse=True)
        return {"out": out, "lse": lse}
    return binding.lora_add(s["base"], s["x"], s["a"], s["b"], s["ids"], scales=s["scales"])


def _first(x, top):
    """The lowest index at which x equals its largest value `top`."""
    index = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == top, index, x.shape[-1]).amin(-1)


def _route_plain(s):
    """Keys (scores with the bias) in 64 bits, as two that lie close together decide whole numbers."""
    case, x = s["case"], s["logits"].double()
    T, E = x.shape
    G = case["groups"]
    if case["score"] == "softmax":
        e = torch.exp(x - x.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    key = score + s["bias"].double() if s["bias"] is not None else score
    live = torch.ones_like(key, dtype=torch.bool)
    if case["top"] < G:
        parts = key.reshape(T, G, E // G)
        best = parts.amax(-1, keepdim=True)
        at = _first(parts, best)[..., None]
        second = parts.scatter(-1, at, -math.inf).amax(-1)
        worth = best[..., 0] + second
        chosen = torch.zeros_like(worth, dtype=torch.bool)
        for _ in range(case["top"]):
            left = worth.masked_fill(chosen, -math.inf)
            chosen = chosen.scatter(-1, _first(left, left.amax(-1, keepdim=True))[..., None], True)
        live = chosen[..., None].expand(T, G, E // G).reshape(T, E)
    # without a bias equal scores of different logits cannot be told apart: the logits order them
    rank = (key if s["bias"] is not None else x).masked_fill(~live, -math.inf)
    experts = []
    for _ in range(case["k"]):
        i = _first(rank, rank.amax(-1, keepdim=True))[..., None]
        rank = rank.scatter(-1, i, -math.inf)
        experts.append(i)
    experts = torch.cat(experts, -1)
    w = torch.gather(score.float(), 1, experts)
    return {"experts": experts.to(torch.int32), "weights": w / w.sum(-1, keepdim=True) * 2.5}


def _rope_plain(s):
    case, dev = s["case"], s["q"].device
    L, m, table = s["lengths"].long(), s["q_lens"].long(), s["table"].long()
    M, page = case["M"], case["page"]
    i = torch.arange(M, device=dev)[None, :]
    pos = L[:, None] - m[:, None] + i
    valid = (i < m[:, None]) & (pos >= 0)
    freq = s["inv_freq"].double()
    if s["positions"] is None:
        theta = pos[..., None].double() * freq
    else:
        sizes = torch.tensor(_sections(case), device=dev)
        axis = torch.repeat_interleave(torch.arange(len(sizes), device=dev), sizes, output_size=case["rot"] // 2)
        theta = s["positions"].permute(1, 2, 0)[..., axis].double() * freq
    cos, sin = torch.cos(theta).float()[:, :, None], torch.sin(theta).float()[:, :, None]

    def rotate(x):
        x = x.float()
        rot, half = case["rot"], case["rot"] // 2
        if case["pairs"] == "halves":
            a, b = x[..., :half], x[..., half:rot]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        return torch.cat((y, x[..., rot:]), -1)

    q = torch.where((i < m[:, None])[..., None, None], rotate(s["q"]), 0.0).to(torch.bfloat16)
    pos = pos.clamp(min=0)
    slot = torch.gather(table, 1, (pos // page).clamp(max=table.shape[1] - 1)), pos % page
    slot = slot[0][valid], slot[1][valid]
    for new, cache, scale in ((rotate(s["k_new"]), s["k_cache"], s["k_scale"]), (s["v_new"], s["v_cache"], s["v_scale"])):
        rows = new[valid]
        if cache.dtype != torch.bfloat16:
            rows = (rows.float() / scale).clamp(-448.0, 448.0).to(cache.dtype).view(torch.uint8)
            cache = cache.view(torch.uint8)
        cache[slot] = rows.to(cache.dtype)
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def _prefix_plain(s):
    """Scores against the prefix for all rows at once and against the own tokens by sequence, one softmax over both."""
    case, q = s["case"], s["q"].float()
    B, M, Hq, D = q.shape
    Hkv, P = case["Hkv"], case["prefix"]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D)

    def tokens(cache, table, scale):
        return cache[table].reshape(*table.shape[:-1], -1, Hkv, D).float() * scale

    shared, table = s["prefix_pages"].long(), s["table"].long().clamp(min=0)
    qs = q.reshape(B, M, Hkv, G, D).permute(2, 0, 3, 1, 4)  # [Hkv, B, G, M, D]
    k = tokens(s["k_cache"], shared, s["k_scale"]).permute(1, 2, 0)
    first = torch.matmul(qs.reshape(Hkv, -1, D), k).reshape(Hkv, B, G, M, P).mul_(scale)
    k = tokens(s["k_cache"], table, s["k_scale"]).permute(2, 0, 3, 1)  # [Hkv, B, D, own]
    second = torch.matmul(qs.reshape(Hkv, B, G * M, D), k).reshape(Hkv, B, G, M, -1).mul_(scale)
    L, m = s["lengths"].long()[:, None, None] - P, s["q_lens"].long()[:, None, None]
    i = torch.arange(M, device=q.device)[None, :, None]
    j = torch.arange(second.shape[-1], device=q.device)[None, None, :]
    second = second.masked_fill(~(j <= L - m + i)[None, :, None], -math.inf)
    real = (i < m)[None, :, None]  # [1, B, 1, M, 1]
    top = torch.maximum(first.amax(-1, keepdim=True), second.amax(-1, keepdim=True))
    first, second = first.sub_(top).exp_(), second.sub_(top).exp_()
    total = first.sum(-1, keepdim=True) + second.sum(-1, keepdim=True)
    lse = torch.where(real, torch.log(total) + top, -math.inf)[..., 0]
    v = tokens(s["v_cache"], shared, s["v_scale"]).permute(1, 0, 2)
    out = torch.matmul(first.reshape(Hkv, -1, P), v).reshape(Hkv, B, G, M, D)
    v = tokens(s["v_cache"], table, s["v_scale"]).permute(2, 0, 1, 3)
    out = out + torch.matmul(second.reshape(Hkv, B, G * M, -1), v).reshape(Hkv, B, G, M, D)
    out = torch.where(real, out / total, 0.0)
    return {"out": out.permute(1, 3, 0, 2, 4).reshape(B, M, Hq, D).to(torch.bfloat16),
            "lse": lse.permute(1, 3, 0, 2).reshape(B, M, Hq)}


def _lora_plain(s):
    """All adapters' inner products at once, those of other adapters than the row's masked, and one product back."""
    L, R, K = s["a"].shape
    T = s["x"].shape[0]
    hidden = torch.matmul(s["x"].float(), s["a"].float().reshape(L * R, K).t()).reshape(T, L, R)
    mine = s["ids"][:, None] == torch.arange(L, device=s["ids"].device)
    hidden = torch.where(mine[..., None], hidden * s["scales"][:, None], 0.0)
    delta = torch.matmul(hidden.reshape(T, L * R), s["b"].float().permute(0, 2, 1).reshape(L * R, -1))
    return (s["base"].float() + delta).to(s["base"].dtype)


def _run_plain(s):
    return {"route": _route_plain, "rope": _rope_plain, "prefix": _prefix_plain, "lora": _lora_plain}[s["case"]["op"]](s)


# ------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "route":
        n = case["T"] * case["E"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 8 * case["T"] * case["k"], "flops": 8 * n}
    if op == "lora":
        rows, ids = _requests(case)
        K, N, R, size = case["K"], case["N"], case["R"], 2 if case["out"] == "bf16" else 4
        T, mine = sum(rows), sum(r for r, i in zip(rows, ids) if i >= 0)
        used = len({i for i in ids if i >= 0})
        return {"bytes": mine * K * 2 + used * R * (K + N) * 2 + 2 * T * N * size, "flops": 2 * mine * R * (K + N)}
    lens, rows = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    size = 2 if case["cache"] == "bf16" else 1
    if op == "rope":
        real = sum(rows)
        new = sum(min(r, n) for r, n in zip(rows, lens))
        pad = case["B"] * case["M"]
        return {"bytes": D * (real * Hq * 2 + pad * Hq * 2 + new * Hkv * 2 * (2 + size)),
                "flops": 3 * case["rot"] * real * (Hq + Hkv)}
    P = case["prefix"]
    pairs = sum(r * P + r * (n - r) + r * (r + 1) // 2 for n, r in ((n, min(r, n)) for n, r in zip(lens, rows)))
    return {"bytes": 2 * (P + sum(lens)) * Hkv * D * size + sum(rows) * Hq * (4 * D + 4), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------- the definition, in 64 bits
def _e4m3_grid(device):
    """The finite magnitudes of E4M3, ascending."""
    c = torch.arange(127, device=device)
    e, f = c >> 3, (c & 7).double() / 8
    return torch.where(e == 0, f * 2.0**-6, (1 + f) * torch.exp2((e - 7).double()))


def _to_grid(y, grid):
    """The value of the magnitudes `grid` nearest to y (their index's last bit decides ties), with y's sign."""
    a = y.abs()
    hi = torch.searchsorted(grid, a).clamp(1, len(grid) - 1)
    mid = 0.5 * (grid[hi - 1] + grid[hi])
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    return torch.sign(y) * grid[torch.where(up, hi, hi - 1)]


def _exact_route(s):
    case = s["case"]
    T, E = s["logits"].shape
    G = case["groups"]
    x = s["logits"].double()
    score = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    key = score if s["bias"] is None else score + s["bias"].double()
    order = torch.sort(x if s["bias"] is None else key, dim=-1, descending=True, stable=True).indices
    worth = torch.sort(key.view(T, G, -1), dim=-1, descending=True).values[..., :2].sum(-1)
    groups = torch.sort(worth, dim=-1, descending=True, stable=True).indices[:, :case["top"]]
    allowed = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, groups, True)
    outside = ~torch.gather(allowed, 1, order // (E // G))
    inside_first = torch.sort(outside.to(torch.uint8), dim=-1, stable=True).indices[:, :case["k"]]
    experts = torch.gather(order, 1, inside_first)
    w = torch.gather(score, 1, experts)
    return {"experts": experts.to(torch.int32), "weights": 2.5 * w / w.sum(-1, keepdim=True)}


def _exact_rope(s):
    """Pairs as complex numbers, turned by exp(i theta), a sequence at a time."""
    case, dev = s["case"], s["q"].device
    rot, grid = case["rot"], _e4m3_grid(dev)
    q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    k_full, v_full = s["k_cache"].double(), s["v_cache"].double()
    sections = _sections(case) or (rot // 2,)

    def turn(x, z):
        x = x.double()
        pair = x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["pairs"] == "halves" else \
            x[..., :rot].unflatten(-1, (rot // 2, 2))
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z[:, None, :])
        y = y.transpose(-1, -2).flatten(-2) if case["pairs"] == "halves" else y.flatten(-2)
        return torch.cat((y, x[..., rot:]), -1)

    for b, (n, m) in enumerate(zip(s["lengths"].tolist(), s["q_lens"].tolist())):
        at = torch.arange(n - m, n, device=dev)
        angles, first = [], 0
        for axis, size in enumerate(sections):
            where = at if s["positions"] is None else s["positions"][axis, b, :m]
            angles.append(where.double()[:, None] * s["inv_freq"][first:first + size].double())
            first += size
        theta = torch.cat(angles, -1)
        z = torch.polar(torch.ones_like(theta), theta)
        q_out[b, :m] = turn(s["q"][b, :m], z)
        keep = max(0, m - n)
        at = at[keep:]
        place = s["table"][b].long()[at // case["page"]] * case["page"] + at % case["page"]
        for full, new, scale in ((k_full, turn(s["k_new"][b, :m], z), s["k_scale"]),
                                 (v_full, s["v_new"][b, :m].double(), s["v_scale"])):
            rows = new[keep:]
            full.view(-1, case["Hkv"], case["D"])[place] = rows if case["cache"] == "bf16" else _to_grid(rows / scale, grid)
    return {"q": q_out, "k": k_full, "v": v_full}


def _exact_prefix(s):
    case, dev = s["case"], s["q"].device
    B, M, Hq, Hkv, D, page = case["B"], case["M"], case["Hq"], case["Hkv"], case["D"], case["page"]
    if B * M * Hq * (case["prefix"] + case["lmax"]) * D * 4 > 1e13:
        return None
    o = torch.zeros(B, M, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, M, Hq), -math.inf, dtype=torch.float64, device=dev)

    def head(cache, scale, pages, h):
        return cache[pages.long(), :, h].reshape(-1, D).double() * scale

    for h in range(Hkv):
        mine = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
        k0, v0 = (head(s[c], s[z], s["prefix_pages"], h) for c, z in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
        for b, (n, m) in enumerate(zip(s["lengths"].tolist(), s["q_lens"].tolist())):
            own_tokens = n - case["prefix"]
            pages = s["table"][b, :-(-own_tokens // page)]
            k = torch.cat((k0, head(s["k_cache"], s["k_scale"], pages, h)[:own_tokens]))
            v = torch.cat((v0, head(s["v_cache"], s["v_scale"], pages, h)[:own_tokens]))
            x = torch.einsum("igd,td->igt", s["q"][b, :m, mine].double(), k) / math.sqrt(D)
            last = torch.arange(n - m, n, device=dev)
            x.masked_fill_(torch.arange(n, device=dev)[None, None, :] > last[:, None, None], -math.inf)
            lse[b, :m, mine] = torch.logsumexp(x, -1)
            o[b, :m, mine] = torch.softmax(x, -1) @ v
    return {"out": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "prefix":
        return _exact_prefix(s)
    y = s["base"].double()
    for adapter in range(case["L"]):
        t = torch.nonzero(s["ids"] == adapter)[:, 0]
        if len(t):
            y[t] += s["scales"][adapter].double() * (s["x"][t].double() @ s["a"][adapter].double().t()
                                                     @ s["b"][adapter].double().t())
    return y
