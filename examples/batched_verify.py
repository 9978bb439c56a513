"""Speculative decoding of a batch with the library's operators, end to end.

A small decoder (random weights, microscaled 4-bit) generates tokens for a few
sequences.  Every step drafts up to k tokens per sequence (by looking up what
followed the last token earlier in the sequence), runs one forward pass over the
drafts of all sequences and verifies them:

    quantize_mx       weights once, activations before every projection
    matmul_mx         projections of more than 16 rows (sequences x draft rows)
    small_m_mx        projections of up to 16 rows, on the same quantised values
    kv_append         the new rows' keys and values into the paged cache
    paged_attention   the new rows over their sequences' caches
    verify_draft      accepted drafts and the next token

    python examples/batched_verify.py
"""
from __future__ import annotations

import sys
from dataclasses import dataclass
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
from quantized_matmul_speculative_gb300 import binding  # noqa: E402


@dataclass
class Config:
    vocab: int = 2000
    hidden: int = 1024
    layers: int = 2
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 128
    mlp: int = 2048
    fmt: str = "nvfp4"
    page: int = 16
    window: int = 0
    sinks: int = 0
    cache: torch.dtype = torch.bfloat16


class Decoder:
    """Weights and paged cache of a batch of sequences on one GPU."""

    def __init__(self, cfg: Config, batch: int, max_tokens: int, seed: int = 0):
        self.cfg, self.batch = cfg, batch
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = (cfg.q_heads + 2 * cfg.kv_heads) * cfg.head_dim

        def weight(n, k):
            w = torch.randn(n, k, generator=g, device="cuda") / k ** 0.5
            return binding.quantize_mx(w, cfg.fmt)

        self.embedding = torch.randn(cfg.vocab, cfg.hidden, generator=g, device="cuda").to(torch.bfloat16)
        self.blocks = [{"qkv": weight(width, cfg.hidden), "o": weight(cfg.hidden, cfg.q_heads * cfg.head_dim),
                        "up": weight(2 * cfg.mlp, cfg.hidden), "down": weight(cfg.hidden, cfg.mlp)}
                       for _ in range(cfg.layers)]
        self.head = weight(cfg.vocab, cfg.hidden)
        per_seq = -(-max_tokens // cfg.page)
        # pages handed out at random, as a server's allocator would leave them
        order = torch.randperm(batch * per_seq, generator=g, device="cuda").to(torch.int32)
        self.table = order.view(batch, per_seq).contiguous()
        shape = (cfg.layers, batch * per_seq, cfg.page, cfg.kv_heads, cfg.head_dim)
        self.k = torch.zeros(shape, dtype=cfg.cache, device="cuda")
        self.v = torch.zeros(shape, dtype=cfg.cache, device="cuda")
        self.scale = 1.0 if cfg.cache == torch.bfloat16 else 0.0625

    def project(self, x, w, out_dtype=torch.bfloat16):
        """x [rows, K] times a quantised weight, x quantised to the same format."""
        values = torch.empty_like(x)
        xq = binding.quantize_mx(x, self.cfg.fmt, values=values)
        if x.shape[0] <= 16:
            return binding.small_m_mx(values, *w, self.cfg.fmt, out_dtype=out_dtype)
        return binding.matmul_mx(*xq, *w, self.cfg.fmt, out_dtype=out_dtype)

    def forward(self, tokens, lengths, new_rows):
        """Logits [B, M, V] of the new rows: ``tokens`` int [B, M] (padded),
        ``lengths`` int32 [B] the sequences' tokens with them, ``new_rows``
        int32 [B] how many of the M are real."""
        cfg = self.cfg
        B, M = tokens.shape
        x = self.embedding[tokens.clamp(min=0)].view(B * M, cfg.hidden)

        def norm(x):
            return torch.nn.functional.rms_norm(x, (cfg.hidden,))

        for i, block in enumerate(self.blocks):
            qkv = self.project(norm(x), block["qkv"]).view(B, M, cfg.q_heads + 2 * cfg.kv_heads, cfg.head_dim)
            q, k, v = qkv.split([cfg.q_heads, cfg.kv_heads, cfg.kv_heads], 2)
            at = dict(q_lens=new_rows, k_scale=self.scale, v_scale=self.scale)
            binding.kv_append(k, v, self.k[i], self.v[i], self.table, lengths, **at)
            a = binding.paged_attention(q, self.k[i], self.v[i], self.table, lengths, window=cfg.window, sinks=cfg.sinks, **at)
            x = x + self.project(a.view(B * M, -1), block["o"])
            gate, up = self.project(norm(x), block["up"]).chunk(2, 1)
            x = x + self.project(torch.nn.functional.silu(gate) * up, block["down"])
        return self.project(norm(x), self.head, torch.float32).view(B, M, cfg.vocab)


def lookup_drafts(history, k):
    """Up to k tokens that followed the last token's previous occurrence."""
    last = history[-1]
    for i in range(len(history) - 2, -1, -1):
        if history[i] == last:
            return history[i + 1:i + 1 + k]
    return []


def generate(model: Decoder, prompts, steps: int, k: int, temperature: float = 0.0, seed: int = 0):
    """Generate at least ``steps`` tokens for every prompt, drafting up to k a
    step; returns (the sequences, drafts offered, drafts accepted)."""
    B, dev = model.batch, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    history = [list(p) for p in prompts]
    cached = [0] * B  # tokens of each sequence whose keys and values are in the cache
    offered = taken = 0
    while min(len(h) - len(p) for h, p in zip(history, prompts)) < steps:
        drafts = []
        rows = []
        for b, h in enumerate(history):
            todo = h[cached[b]:]  # the prompt in pieces of up to 16 rows, then the last token and its drafts
            if len(todo) > 1:
                drafts.append([])
                rows.append(todo[:16])
            else:
                drafts.append(lookup_drafts(h, k))
                rows.append(todo + drafts[-1])
        M = max(map(len, rows))
        tokens = torch.tensor([r + [0] * (M - len(r)) for r in rows], device=dev)
        new_rows = torch.tensor([len(r) for r in rows], dtype=torch.int32, device=dev)
        lengths = torch.tensor([c + len(r) for c, r in zip(cached, rows)], dtype=torch.int32, device=dev)
        logits = model.forward(tokens, lengths, new_rows)
        # rows that verify: a sequence's last token and its drafts (of a prompt's piece, its last row)
        n = [len(d) for d in drafts]
        kk = max(n)
        first = torch.tensor([len(r) - 1 - x for r, x in zip(rows, n)], device=dev)
        pick = (first[:, None] + torch.arange(kk + 1, device=dev)).clamp(max=M - 1)
        logits = torch.gather(logits, 1, pick[..., None].expand(-1, -1, logits.shape[2]))
        out, accepted = binding.verify_draft(
            logits, torch.tensor([d + [0] * (kk - len(d)) for d in drafts], dtype=torch.int32, device=dev).view(B, kk), None,
            torch.rand(B, kk, generator=g, device=dev),
            torch.empty(B, logits.shape[2], device=dev).exponential_(generator=g).clamp_(min=1e-20),
            torch.full((B,), temperature, device=dev), draft_lens=torch.tensor(n, dtype=torch.int32, device=dev))
        out, accepted = out.tolist(), accepted.tolist()
        for b, h in enumerate(history):
            done = cached[b] + len(rows[b]) - n[b]
            cached[b] = done + accepted[b]  # keys of refused drafts are overwritten by the next step's rows
            if done == len(h):
                h += out[b][:accepted[b] + 1]
                offered += n[b]
                taken += accepted[b]
    return history, offered, taken


def main():
    cfg = Config()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, cfg.vocab, (n,), generator=g).tolist() for n in (5, 1, 40, 17, 9, 2)]
    for cache in (torch.bfloat16, torch.float8_e4m3fn):
        cfg.cache = cache
        model = Decoder(cfg, len(prompts), 256)
        history, offered, taken = generate(model, prompts, steps=48, k=4)
        new = sum(len(h) - len(p) for h, p in zip(history, prompts))
        print(f"{cache}: {new} tokens for {len(prompts)} sequences, {taken} of {offered} drafts accepted")
        assert binding.device_status() == 0


if __name__ == "__main__":
    main()
