"""Calls of the layer's operators on another stream, ordered by the binding alone (as test_gpu_streams), and waits of the
prefix kernel that run out."""
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding
from test_gpu_prefix import Shared, check, queries
from test_gpu_streams import busy, randn

pytestmark = pytest.mark.gpu


class Route:
    def inputs(self, g):
        return [torch.randn(3000, 128, generator=g, device="cuda"), torch.randn(128, generator=g, device="cuda")]

    def run(self, inputs, stream):
        return binding.route_experts(inputs[0], 8, "sigmoid", bias=inputs[1], stream=stream)


class Rope:
    def __init__(self):
        self.table = torch.arange(16, dtype=torch.int32, device="cuda").view(4, 4)

    def inputs(self, g):
        return [randn(g, 4, 8, 8, 128), randn(g, 4, 8, 2, 128), randn(g, 4, 8, 2, 128),
                torch.full((4,), 50, dtype=torch.int32, device="cuda"), torch.rand(64, generator=g, device="cuda")]

    def run(self, inputs, stream):
        q, k, v, lengths, freq = inputs
        cache = [torch.zeros(16, 16, 2, 128, device="cuda").bfloat16() for _ in range(2)]
        return [binding.rope_append(q, k, v, *cache, self.table, lengths, freq, stream=stream), *cache]


class Prefix(Rope):
    def inputs(self, g):
        return [randn(g, 4, 8, 8, 128), randn(g, 24, 16, 2, 128), randn(g, 24, 16, 2, 128),
                torch.full((4,), 178, dtype=torch.int32, device="cuda"), torch.arange(16, 24, device="cuda").to(torch.int32)]

    def run(self, inputs, stream):
        q, k, v, lengths, prefix = inputs
        return binding.shared_prefix_attention(q, k, v, prefix, self.table, lengths, return_lse=True, stream=stream)


class Lora:
    def __init__(self, T):
        self.T = T

    def inputs(self, g):
        return [randn(g, self.T, 512), randn(g, self.T, 256), randn(g, 3, 16, 256), randn(g, 3, 512, 16),
                torch.randint(-1, 3, (self.T,), generator=g, device="cuda").to(torch.int32)]

    def run(self, inputs, stream):
        return [binding.lora_add(*inputs, stream=stream)]


OPS = [Route, Rope, Prefix, lambda: Lora(40), lambda: Lora(900)]


@pytest.mark.parametrize("op", OPS)
def test_inputs_still_computed_on_the_current_stream(op):
    op, side = op(), torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(1)
    true = op.inputs(g)
    want = op.run(true, None)
    inputs = [torch.zeros_like(x) for x in true]
    torch.cuda.synchronize()
    busy()
    for x, t in zip(inputs, true):
        x.copy_(t)
    got = op.run(inputs, side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("op", OPS)
def test_inputs_freed_after_the_call(op):
    op, side = op(), torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(2)
    true = op.inputs(g)
    want = op.run(true, None)
    inputs = [t.clone() for t in true]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        kept = busy()
    got = op.run(inputs, side)
    del inputs
    zeros = [torch.zeros_like(t) for t in true for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del kept, zeros


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 16), (256, 64)])
def test_a_wait_that_runs_out(monkeypatch, D, page, dtype):
    """The first CTA's first piece never completes, for 100 us; all copies land, the call returns with a status bit, and the
    next one is right."""
    s = Shared(20, [30, 9, 50], 2, D, page, dtype, seed=7)
    q = queries(3, 2, 8, D)
    want, _ = check(q, s)
    monkeypatch.setenv("QMM_TEST_INJECT", "short_wait")
    out = binding.shared_prefix_attention(q, *s.args())
    torch.cuda.synchronize()
    assert binding.device_status() & 1
    assert out.shape == want.shape
    monkeypatch.delenv("QMM_TEST_INJECT")
    again, _ = check(q, s)
    assert torch.equal(again, want)
