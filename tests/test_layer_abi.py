"""Host checks of the layer operators' C entry points: every refusal comes before anything touches a device."""
import ctypes
import math

import pytest

from quantized_matmul_speculative_gb300 import binding
from test_ops_abi import ALIGN, CACHES, NULL, OK, SHAPE, UNSUPPORTED, P, cache, call, lib  # noqa: F401


def test_route(lib):  # noqa: F811
    good = dict(logits=P, dtype=0, ld=64, bias=None, T=4, E=64, k=8, scoring=0, groups=8, top_groups=4, group_best=2,
                renormalize=1, scale=1.0, experts=P, weights=P, stream=None)
    for changes, rc in (({"T": -1}, SHAPE), ({"T": 2**31 - 1}, SHAPE), ({"E": 0}, SHAPE), ({"E": 520, "ld": 520}, SHAPE), ({"k": 0}, SHAPE), ({"k": 33}, SHAPE),
                        ({"ld": 63}, SHAPE), ({"groups": 0}, SHAPE), ({"groups": 7}, SHAPE), ({"groups": 64}, SHAPE),
                        ({"top_groups": 0}, SHAPE), ({"top_groups": 9}, SHAPE), ({"k": 9, "top_groups": 1}, SHAPE),
                        ({"dtype": 2}, UNSUPPORTED), ({"scoring": 2}, UNSUPPORTED), ({"group_best": 0}, UNSUPPORTED),
                        ({"group_best": 3}, UNSUPPORTED), ({"logits": None}, NULL), ({"experts": None}, NULL),
                        ({"weights": None}, NULL), ({"logits": P + 1}, ALIGN), ({"logits": P + 2, "dtype": 1}, ALIGN),
                        ({"bias": P + 2}, ALIGN), ({"experts": P + 1}, ALIGN), ({"weights": P + 2}, ALIGN), ({"T": 0}, OK)):
        assert call(lib.qmm_route_experts, good, changes) == rc, changes


def rope(**changes):
    good = dict(inv_freq=P, positions=None, rot=64, axes=1, sections=(ctypes.c_int32 * 4)(32, 0, 0, 0), interleaved=0, factor=1.0)
    good.update(changes)
    return binding.RopeStruct(*good.values())


def test_rope(lib):  # noqa: F811
    def run(c, r, **changes):
        good = dict(cache=ctypes.byref(c), rope=ctypes.byref(r), q=P, q_ld=256, q_heads=4, out=P, out_ld=256, k=P, k_ld=128, v=P,
                    v_ld=128, B=2, M=3, q_lens=None, stream=None)
        return call(lib.qmm_rope_append, good, changes)

    for changes, rc in CACHES:
        assert run(cache(**changes), rope()) == rc, changes
    four = ctypes.c_int32 * 4
    for changes, rc in (({"rot": -16}, SHAPE), ({"rot": 80}, SHAPE), ({"rot": 24}, SHAPE), ({"inv_freq": None}, NULL),
                        ({"inv_freq": P + 2}, ALIGN), ({"positions": P, "axes": 0}, UNSUPPORTED),
                        ({"positions": P, "axes": 5}, UNSUPPORTED), ({"positions": P + 1}, ALIGN),
                        ({"positions": P, "sections": four(31, 0, 0, 0)}, SHAPE),
                        ({"positions": P, "axes": 2, "sections": four(40, -8, 0, 0)}, SHAPE),
                        ({"factor": math.inf}, UNSUPPORTED), ({"factor": math.nan}, UNSUPPORTED)):
        assert run(cache(), rope(**changes)) == rc, changes
    for changes, rc in (({"rope": None}, NULL), ({"cache": None}, NULL), ({"q": None}, NULL), ({"out": None}, NULL), ({"k": None}, NULL),
                        ({"v": None}, NULL), ({"q_heads": 0}, SHAPE), ({"q_heads": 65536, "q_ld": 2**23, "out_ld": 2**23}, SHAPE),
                        ({"q_ld": 248}, SHAPE), ({"out_ld": 248}, SHAPE), ({"k_ld": 120}, SHAPE), ({"v_ld": 120}, SHAPE),
                        ({"B": -1}, SHAPE), ({"B": 65536}, SHAPE), ({"M": -1}, SHAPE), ({"B": 65535, "M": 65535}, SHAPE),
                        ({"q": P + 8}, ALIGN), ({"out": P + 2}, ALIGN), ({"k": P + 4}, ALIGN), ({"v": P + 4}, ALIGN),
                        ({"q_ld": 260}, ALIGN), ({"out_ld": 260}, ALIGN), ({"k_ld": 132}, ALIGN), ({"v_ld": 132}, ALIGN),
                        ({"q_lens": P + 1}, ALIGN), ({"B": 0}, OK), ({"M": 0}, OK)):
        assert run(cache(), rope(), **changes) == rc, changes


def test_shared_prefix(lib):  # noqa: F811
    def run(c, **changes):
        good = dict(cache=ctypes.byref(c), prefix=P, pages=5, q=P, q_ld=256, B=2, M=3, q_heads=4, q_lens=None, scale=0.1, out=P,
                    lse=None, ws=P, ws_bytes=2**40, stream=None)
        return call(lib.qmm_shared_prefix_attention, good, changes)

    for changes, rc in CACHES:
        assert run(cache(**changes)) == rc, changes
    need = lib.qmm_shared_prefix_attention_workspace(2, 3, 4, 2, 64)
    assert need > 0
    for changes, rc in (({"pages": -1}, SHAPE), ({"pages": 2**30}, SHAPE), ({"prefix": None}, NULL), ({"prefix": P + 2}, ALIGN),
                        ({"q": None}, NULL), ({"out": None}, NULL), ({"ws": None}, NULL), ({"q_heads": 3}, SHAPE), ({"q_heads": 0}, SHAPE),
                        ({"q_heads": 65536, "q_ld": 2**23}, SHAPE), ({"q_ld": 248}, SHAPE), ({"M": 17}, SHAPE), ({"B": 65536}, SHAPE),
                        ({"scale": math.nan}, UNSUPPORTED), ({"scale": math.inf}, UNSUPPORTED), ({"q": P + 8}, ALIGN),
                        ({"out": P + 8}, ALIGN), ({"lse": P + 2}, ALIGN), ({"ws": P + 8}, ALIGN), ({"q_ld": 260}, ALIGN),
                        ({"ws_bytes": need - 1}, SHAPE), ({"B": 0}, OK), ({"M": 0}, OK)):
        assert run(cache(), **changes) == rc, changes
    for sizes in ((0, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 17, 4, 2, 64), (1, 1, 5, 2, 64), (1, 1, 4, 0, 64), (1, 1, 0, 2, 64)):
        assert lib.qmm_shared_prefix_attention_workspace(*sizes) == 0


def test_lora(lib):  # noqa: F811
    good = dict(base=P, base_ld=100, X=P, x_ld=64, A=P, Bm=P, adapters=P, scales=None, T=5, N=100, K=64, R=16, L=3, Y=P, y_ld=100,
                dtype=0, ws=P, ws_bytes=2**30, stream=None)
    for changes, rc in (({"T": -1}, SHAPE), ({"N": -1}, SHAPE), ({"K": -8}, SHAPE), ({"L": -1}, SHAPE), ({"R": 0}, SHAPE),
                        ({"R": 12}, SHAPE), ({"R": 136}, SHAPE), ({"K": 60}, SHAPE), ({"base_ld": 99}, SHAPE), ({"y_ld": 99}, SHAPE),
                        ({"x_ld": 56}, SHAPE), ({"N": 2**30 + 1, "base_ld": 2**31, "y_ld": 2**31}, SHAPE), ({"dtype": 2}, UNSUPPORTED),
                        ({"base": None}, NULL), ({"X": None}, NULL), ({"A": None}, NULL), ({"Bm": None}, NULL),
                        ({"adapters": None}, NULL), ({"Y": None}, NULL), ({"base": P + 1}, ALIGN), ({"Y": P + 2, "dtype": 1}, ALIGN),
                        ({"X": P + 8}, ALIGN), ({"A": P + 8}, ALIGN), ({"Bm": P + 8}, ALIGN), ({"x_ld": 68}, ALIGN),
                        ({"adapters": P + 2}, ALIGN), ({"scales": P + 2}, ALIGN), ({"T": 0}, OK), ({"N": 0}, OK)):
        assert call(lib.qmm_lora_add, good, changes) == rc, changes
    need = lib.qmm_lora_workspace(5, 3, 16)
    assert need > 0 and lib.qmm_lora_workspace(100000, 3, 16) > need
    for changes, rc in (({"ws": None}, NULL), ({"ws": P + 8}, ALIGN), ({"ws_bytes": need - 1}, SHAPE),
                        ({"T": 2**23, "L": 1, "ws_bytes": 2**50}, SHAPE)):
        assert call(lib.qmm_lora_add, good, changes) == rc, changes
    for sizes in ((0, 3, 16), (5, -1, 16), (5, 3, 0), (5, 3, 136)):
        assert lib.qmm_lora_workspace(*sizes) == 0
