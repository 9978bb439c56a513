"""The layer's operators together, as a server would run them: one verify step of a mixture-of-experts layer for a batch
behind a shared prompt, its projections with per-request adapters; run at once, step by step, captured into a graph and
replayed on new inputs, and with the prompt in every sequence's own table instead."""
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu

B, M, Hq, Hkv, D, PAGE, PREFIX_PAGES = 3, 2, 8, 2, 64, 16, 5
HIDDEN, EXPERTS, TOP, WIDTH = 256, 16, 4, 128


class Layer:
    """Random weights, and a cache with a shared prompt and the sequences' own first tokens in it."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(1)
        self.g = g

        def matrix(n, k, *stack):
            codes = torch.randint(-2**31, 2**31, (*stack, n, k // 8), generator=g, device="cuda").to(torch.int32)
            s = (0.2 / k**0.5 * (1 + torch.rand(*stack, n, k // 64, generator=g, device="cuda"))).half()
            return codes, s, (-7.5 * s.float()).half()

        def adapters(n, k, R, L):
            return (torch.randn(L, R, k, generator=g, device="cuda") / k**0.5).bfloat16(), \
                (torch.randn(L, n, R, generator=g, device="cuda") / R**0.5).bfloat16()

        width = (Hq + 2 * Hkv) * D
        self.qkv, self.qkv_ab = matrix(width, HIDDEN), adapters(width, HIDDEN, 16, 3)
        self.out = matrix(HIDDEN, Hq * D)
        self.router = torch.randn(HIDDEN, EXPERTS, generator=g, device="cuda").bfloat16()
        self.bias = 0.05 * torch.randn(EXPERTS, generator=g, device="cuda")
        self.up, self.down = matrix(WIDTH, HIDDEN, EXPERTS), matrix(HIDDEN, WIDTH, EXPERTS)
        pages = PREFIX_PAGES + 4 * B
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.prefix = order[:PREFIX_PAGES].contiguous()
        self.own = order[PREFIX_PAGES:].view(B, 4).contiguous()
        self.whole = torch.cat((self.prefix[None].expand(B, -1), self.own), 1).contiguous()
        self.k = torch.randn(pages, PAGE, Hkv, D, generator=g, device="cuda").bfloat16()
        self.v = torch.randn(pages, PAGE, Hkv, D, generator=g, device="cuda").bfloat16()
        self.inv_freq = 1e4 ** (-torch.arange(0, D, 2, device="cuda").float() / D)
        self.each = torch.arange(B * M * TOP, dtype=torch.int32, device="cuda")
        self.lhs = torch.arange(B * M, dtype=torch.int32, device="cuda").repeat_interleave(TOP)

    def inputs(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = torch.tensor([2, 1, 2], dtype=torch.int32, device="cuda")
        own = torch.randint(2, 60, (B,), generator=g, device="cuda", dtype=torch.int32)
        ids = torch.randint(-1, 3, (B,), generator=g, device="cuda", dtype=torch.int32).repeat_interleave(M)
        return dict(x=torch.randn(B * M, HIDDEN, generator=g, device="cuda").bfloat16(), q_lens=new,
                    lengths=own + PREFIX_PAGES * PAGE, ids=ids)

    def run(self, x, q_lens, lengths, ids, shared=True, wait=lambda: None):
        qkv = binding.small_m(x, *self.qkv, 4, 64)
        wait()
        binding.lora_add(qkv, x, *self.qkv_ab, ids, out=qkv)
        wait()
        q, k, v = qkv.view(B, M, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 2)
        q = binding.rope_append(q, k, v, self.k, self.v, self.whole, lengths, self.inv_freq, q_lens=q_lens)
        wait()
        if shared:
            a = binding.shared_prefix_attention(q, self.k, self.v, self.prefix, self.own, lengths, q_lens=q_lens)
        else:
            a = binding.paged_attention(q, self.k, self.v, self.whole, lengths, q_lens=q_lens)
        wait()
        y = binding.small_m(a.view(B * M, -1), *self.out, 4, 64, residual=x)
        wait()
        logits = y.float() @ self.router.float()
        experts, weights = binding.route_experts(logits, TOP, "sigmoid", bias=self.bias, groups=4, top_groups=2)
        wait()
        rhs = experts.view(-1)
        h = binding.gather_small_m(y, *self.up, self.lhs, rhs, 4, 64)
        wait()
        h = torch.nn.functional.silu(h)
        z = binding.gather_small_m(h, *self.down, self.each, rhs, 4, 64, out_dtype=torch.float32)
        wait()
        z = (z.view(B * M, TOP, HIDDEN) * weights[..., None]).sum(1)
        return {"y": y, "experts": experts, "weights": weights, "z": z, "q": q, "a": a}


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


def test_at_once_and_step_by_step():
    layer = Layer()
    for seed in range(3):
        inputs = layer.inputs(seed)
        want = layer.run(**inputs, wait=torch.cuda.synchronize)
        for _ in range(5):
            assert same(layer.run(**inputs), want)
    assert binding.device_status() == 0


def test_captured_and_replayed():
    layer = Layer()
    static = layer.inputs(0)
    layer.run(**static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.run(**static)
    for seed in (0, 5, 6):
        fresh = layer.inputs(seed)
        for k in static:
            static[k].copy_(fresh[k])
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        assert same(got, layer.run(**fresh))
    assert binding.device_status() == 0


def test_two_graphs_at_once():
    """Two captured layers on two streams, replayed together: nothing that they use is shared."""
    layers = [Layer(), Layer()]
    data = [layers[0].inputs(1), layers[1].inputs(2)]
    want = [layer.run(**d) for layer, d in zip(layers, data)]
    graphs, outs = [], []
    for layer, d in zip(layers, data):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer.run(**d))
        graphs.append(g)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(same(w, o) for w, o in zip(want, outs))


def test_the_prompt_in_every_table_instead():
    """Attention outputs that differ in the last bits: bf16 roundings of both, 2^-8 each of values up to the largest."""
    layer = Layer()
    inputs = layer.inputs(3)
    a, b = layer.run(**inputs), layer.run(**inputs, shared=False)
    assert torch.equal(a["q"], b["q"])
    size = b["a"].float().abs().max()
    assert (a["a"].float() - b["a"].float()).abs().max() <= 2 * 2.0**-8 * size


# ------------------------------------------------------------------- the largest
def test_offsets_beyond_32_bits():
    """Caches, adapters and logits of more than 2^31 elements, the last of them used."""
    pages, page, heads, D = 33000, 64, 8, 128  # 2.16e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros(pages, page, heads, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    last = torch.arange(pages - 12, pages, dtype=torch.int32, device="cuda")
    k[-12:] = torch.randn(12, page, heads, D, generator=g, device="cuda").bfloat16()
    v[-12:] = torch.randn(12, page, heads, D, generator=g, device="cuda").bfloat16()
    small_k, small_v = k[-12:].clone(), v[-12:].clone()
    table, lengths = last[8:].view(2, 2), torch.tensor([512 + 100, 512 + 70], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 3, 16 + 2 * heads, D, generator=g, device="cuda").bfloat16()
    q, kn, vn = x.split([16, heads, heads], 2)
    freq = 1e4 ** (-torch.arange(0, D, 2, device="cuda").float() / D)
    outs = []
    for kc, vc, first in ((k, v, 0), (small_k, small_v, pages - 12)):
        t = (table - first).contiguous()
        r = binding.rope_append(q, kn, vn, kc, vc, t, lengths - 512, freq)
        outs.append((r, *binding.shared_prefix_attention(r, kc, vc, last[:8] - first, t, lengths, return_lse=True)))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(k[-12:], small_k) and torch.equal(v[-12:], small_v)
    del k, v
    L, N, R = 1030, 16384, 128  # 2.16e9 elements of b
    b = torch.zeros(L, N, R, dtype=torch.bfloat16, device="cuda")
    b[-1] = torch.randn(N, R, generator=g, device="cuda").bfloat16()
    a = torch.randn(L, R, 64, generator=g, device="cuda").bfloat16()
    base, xx = torch.randn(2, N, generator=g, device="cuda"), torch.randn(2, 64, generator=g, device="cuda").bfloat16()
    got = binding.lora_add(base, xx, a, b, torch.tensor([L - 1, -1], dtype=torch.int32, device="cuda"))
    want = binding.lora_add(base, xx, a[-1:].contiguous(), b[-1:].contiguous(), torch.tensor([0, -1], dtype=torch.int32, device="cuda"))
    assert torch.equal(got, want)
    del b
    logits = torch.zeros(4300000, 512, dtype=torch.bfloat16, device="cuda")
    logits[-5:] = torch.randn(5, 512, generator=g, device="cuda").bfloat16()
    e, w = binding.route_experts(logits, 8)
    e1, w1 = binding.route_experts(logits[-5:].contiguous(), 8)
    assert torch.equal(e[-5:], e1) and torch.equal(w[-5:], w1)
    assert binding.device_status() == 0
