"""Calls of the operators around the product on another stream, ordered by the binding alone: inputs that the current
stream is still computing, and inputs whose memory is free for it again as soon as the call returns."""
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding

pytestmark = pytest.mark.gpu


def randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


class Quantize:
    def inputs(self, g):
        return [randn(g, 512, 4096)]

    def outputs(self):
        return [torch.zeros(512, 512, dtype=torch.int32, device="cuda"), torch.zeros(512, 256, dtype=torch.uint8, device="cuda")]

    def run(self, inputs, outputs, stream):
        binding.quantize_mx(*inputs, "nvfp4", out=outputs, stream=stream)


class Matmul:
    def inputs(self, g):
        m = []
        for rows in (64, 300):
            m.append(torch.randint(0, 2**31, (rows, 64), generator=g, device="cuda").to(torch.int32))
            m.append(torch.randint(0x28, 0x40, (rows, 32), generator=g, device="cuda").to(torch.uint8))
        return m

    def outputs(self):
        return [torch.zeros(64, 300, device="cuda")]

    def run(self, inputs, outputs, stream):
        binding.matmul_mx(*inputs, "nvfp4", out=outputs[0], stream=stream)


class Append:
    def __init__(self):
        self.table = torch.arange(16, dtype=torch.int32, device="cuda").view(4, 4)

    def inputs(self, g):
        return [randn(g, 4, 8, 2, 128), randn(g, 4, 8, 2, 128), torch.full((4,), 50, dtype=torch.int32, device="cuda")]

    def outputs(self):
        return [torch.zeros(16, 16, 2, 128, device="cuda").bfloat16() for _ in range(2)]

    def run(self, inputs, outputs, stream):
        k, v, lengths = inputs
        binding.kv_append(k, v, *outputs, self.table, lengths, stream=stream)


class Attention(Append):
    def __init__(self):
        super().__init__()
        self.workspace = torch.zeros(binding.paged_attention_workspace(4, 8, 8, 2, 128), dtype=torch.uint8, device="cuda")

    def inputs(self, g):
        return [randn(g, 4, 8, 8, 128), randn(g, 16, 16, 2, 128), randn(g, 16, 16, 2, 128),
                torch.full((4,), 50, dtype=torch.int32, device="cuda")]

    def outputs(self):
        return [torch.zeros(4, 8, 8, 128, device="cuda").bfloat16()]

    def run(self, inputs, outputs, stream):
        q, k, v, lengths = inputs
        binding.paged_attention(q, k, v, self.table, lengths, out=outputs[0], workspace=self.workspace, stream=stream)


def busy():
    """Some milliseconds of work on the current stream."""
    a = torch.ones(8192, 8192, device="cuda").bfloat16()
    for _ in range(20):
        a = a @ a
    return a


@pytest.mark.parametrize("op", [Quantize, Matmul, Append, Attention])
def test_inputs_still_computed_on_the_current_stream(op):
    op, side = op(), torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(1)
    true = op.inputs(g)
    want, got = op.outputs(), op.outputs()
    op.run(true, want, None)
    inputs = [torch.zeros_like(x) for x in true]
    torch.cuda.synchronize()
    busy()
    for x, t in zip(inputs, true):
        x.copy_(t)
    op.run(inputs, got, side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("op", [Quantize, Matmul, Append, Attention])
def test_inputs_freed_after_the_call(op):
    """The other stream is behind: the inputs' memory must not go to the current stream's next tensors before it reads them."""
    op, side = op(), torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(2)
    true = op.inputs(g)
    want, got = op.outputs(), op.outputs()
    op.run(true, want, None)
    inputs = [t.clone() for t in true]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        kept = busy()
    op.run(inputs, got, side)
    del inputs
    zeros = [torch.zeros_like(t) for t in true for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del kept, zeros
