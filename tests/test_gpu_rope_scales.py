"""E4M3 caches of any scale (a calibrated one is a largest value over 448, hardly ever a power of two): rotation with append
against the formula, and byte for byte against kv_append where nothing turns."""
import pytest

torch = pytest.importorskip("torch")

from quantized_matmul_speculative_gb300 import binding
from test_gpu_rope import E4M3, check, problem

pytestmark = pytest.mark.gpu

SCALES = [0.037, 3.1 / 448, 0.0625, 7.3, 1e-3, 2.0**-100, 1.5e-38]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("k_scale,v_scale", [(0.037, 0.0625), (0.0625, 0.037), (3.1 / 448, 2.9 / 448), (7.3, 0.011)])
def test_formula(k_scale, v_scale, interleaved):
    check(problem([90, 5, 3, 33], [3, 5, 1, 4], 5, 6, 2, 128, 16, E4M3), interleaved=interleaved, k_scale=k_scale, v_scale=v_scale)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("rot", [0, 64])
def test_equals_append(rot, scale):
    """What does not turn (the values, and the keys behind rot) is what kv_append writes."""
    p = problem([90, 5, 33], None, 5, 2, 2, 128, 16, E4M3, rot, seed=3)
    # every bf16 number is there, on a range of 2^9 around the scale too
    x = torch.arange(p["k_new"].numel(), device="cuda")
    bits = (x * 40503 % 65536).to(torch.int32)
    near = (scale * 2.0 ** ((x % 37).float() / 2 - 9)).to(torch.bfloat16)
    for i, name in enumerate(("k_new", "v_new")):
        new = torch.where(x % 2 == i, near, (bits - 65536 * (bits >> 15)).to(torch.int16).view(torch.bfloat16))
        p[name] = new.view(p[name].shape).contiguous()
    k, v = p["k_cache"].clone(), p["v_cache"].clone()
    binding.kv_append(p["k_new"], p["v_new"], k, v, p["block_table"], p["lengths"], k_scale=scale, v_scale=scale)
    binding.rope_append(p["q"], p["k_new"], p["v_new"], p["k_cache"], p["v_cache"], p["block_table"], p["lengths"],
                        p["inv_freq"], k_scale=scale, v_scale=scale)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    assert torch.equal(p["v_cache"].view(torch.uint8), v.view(torch.uint8))
    assert torch.equal(p["k_cache"][..., rot:].contiguous().view(torch.uint8), k[..., rot:].contiguous().view(torch.uint8))
