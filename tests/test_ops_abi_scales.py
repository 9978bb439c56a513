"""Host checks of the attention's scale, before anything touches a device."""
import ctypes

import pytest

from quantized_matmul_speculative_gb300 import binding
from test_ops_abi import OK, P, UNSUPPORTED, cache, lib  # noqa: F401

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("B", [0, 3])
def test_scale(lib, B):  # noqa: F811
    def run(c, scale):
        return lib.qmm_paged_attention(ctypes.byref(c), P, 256, B, 4, 4, None, scale, 0, 0, P, P, P, 2**40, None)

    for scale in (INF, -INF, NAN, 3e38):  # the last times log2(e) is past fp32's range
        assert run(cache(), scale) == UNSUPPORTED, scale
    f8 = cache(dtype=1, k_page=4096, v_page=4096, k_scale=1e30)
    assert run(f8, 1e10) == UNSUPPORTED
    if B == 0:
        assert run(cache(), 1e30) == run(cache(), -0.1) == run(cache(), 0.0) == run(f8, 0.1) == OK
