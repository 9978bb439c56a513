"""Host checks of the operators' C entry points: every refusal comes before anything touches a device."""
import ctypes

import pytest

from quantized_matmul_speculative_gb300 import binding, build

OK, NULL, SHAPE, UNSUPPORTED, ALIGN = range(5)
P = 0x10000  # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def call(fn, good, changes):
    args = dict(good)
    args.update(changes)
    return fn(*args.values())


def test_quantize(lib):
    good = dict(X=P, x_dtype=0, R=4, K=64, ldx=64, format=0, Wq=P, scales=P, values=P, stream=None)
    for changes, rc in (({"format": 3}, UNSUPPORTED), ({"format": -1}, UNSUPPORTED), ({"x_dtype": 2}, UNSUPPORTED),
                        ({"R": -1}, SHAPE), ({"K": -32}, SHAPE), ({"K": 48, "ldx": 48}, SHAPE), ({"ldx": 63}, SHAPE),
                        ({"R": 2**40}, SHAPE), ({"ldx": 2**50}, SHAPE), ({"X": None}, NULL), ({"Wq": None}, NULL),
                        ({"scales": None}, NULL), ({"X": P + 1}, ALIGN), ({"X": P + 2, "x_dtype": 1}, ALIGN),
                        ({"Wq": P + 2}, ALIGN), ({"values": P + 1}, ALIGN), ({"R": 0}, OK), ({"K": 0, "ldx": 0}, OK)):
        assert call(lib.qmm_quantize_mx, good, changes) == rc, changes


def test_matmul(lib):
    good = dict(Xq=P, xs=P, Wq=P, ws=P, M=4, N=8, K=64, format=0, Y=P, out=0, stream=None)
    for changes, rc in (({"M": -1}, SHAPE), ({"N": -1}, SHAPE), ({"K": 40}, SHAPE), ({"format": 1}, UNSUPPORTED),
                        ({"format": 5}, UNSUPPORTED), ({"out": 2}, UNSUPPORTED), ({"M": 2**30 + 1}, SHAPE),
                        ({"N": 2**30 + 1}, SHAPE), ({"M": 0}, OK), ({"N": 0}, OK),
                        ({"Y": None}, NULL), ({"Xq": None}, NULL), ({"Wq": None}, NULL), ({"xs": None}, NULL),
                        ({"ws": None}, NULL), ({"Xq": P + 8}, ALIGN), ({"Wq": P + 4}, ALIGN), ({"Y": P + 1}, ALIGN),
                        ({"Y": P + 2, "out": 1}, ALIGN)):
        assert call(lib.qmm_matmul_mx, good, changes) == rc, changes


def cache(**changes):
    good = dict(k=P, v=P, k_page=2048, k_token=128, k_head=64, v_page=2048, v_token=128, v_head=64, block_table=P,
                lengths=P, table_stride=4, num_pages=10, max_pages=4, page_size=16, heads=2, head_dim=64, dtype=0,
                k_scale=1.0, v_scale=1.0)
    good.update(changes)
    return binding.PagedCacheStruct(*good.values())


CACHES = (({"dtype": 2}, UNSUPPORTED), ({"head_dim": 96}, UNSUPPORTED), ({"heads": 0}, SHAPE), ({"page_size": 0}, SHAPE),
          ({"max_pages": -1}, SHAPE), ({"num_pages": -1}, SHAPE), ({"table_stride": 3}, SHAPE),
          ({"max_pages": 2**20, "table_stride": 2**20, "page_size": 2**12}, SHAPE), ({"lengths": None}, NULL),
          ({"k": None}, NULL), ({"v": None}, NULL), ({"block_table": None}, NULL), ({"k": P + 8}, ALIGN),
          ({"k_token": 4}, ALIGN), ({"v_head": 68}, ALIGN), ({"dtype": 1, "k_head": 72}, ALIGN),
          ({"dtype": 1, "k_scale": 0.0}, UNSUPPORTED), ({"dtype": 1, "v_scale": float("nan")}, UNSUPPORTED),
          ({"lengths": P + 2}, ALIGN))


def test_append(lib):
    good = dict(cache=None, k=P, k_ld=128, v=P, v_ld=128, B=3, M=4, q_lens=None, stream=None)
    run = lambda c, **kw: call(lib.qmm_kv_append, good, dict(kw, cache=ctypes.byref(c)))  # noqa: E731
    for changes, rc in CACHES:
        assert run(cache(**changes)) == rc, changes
    assert call(lib.qmm_kv_append, good, {}) == NULL
    for kw, rc in ((dict(B=-1), SHAPE), (dict(M=17), SHAPE), (dict(k_ld=64), SHAPE), (dict(v_ld=127), SHAPE),
                   (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=P + 4), ALIGN), (dict(v_ld=132), ALIGN),
                   (dict(q_lens=P + 1), ALIGN), (dict(B=0), OK), (dict(M=0), OK)):
        assert run(cache(), **kw) == rc, kw


def test_attention(lib):
    good = dict(cache=None, q=P, q_ld=256, B=3, M=4, Hq=4, q_lens=None, scale=1.0, window=0, sinks=0, out=P, lse=P, ws=P,
                ws_bytes=2**40, stream=None)
    run = lambda c, **kw: call(lib.qmm_paged_attention, good, dict(kw, cache=ctypes.byref(c)))  # noqa: E731
    for changes, rc in CACHES:
        assert run(cache(**changes)) == rc, changes
    for kw, rc in ((dict(B=-1), SHAPE), (dict(M=17), SHAPE), (dict(Hq=3), SHAPE), (dict(Hq=0), SHAPE),
                   (dict(q_ld=255), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE),
                   (dict(Hq=4096, q_ld=2**20), SHAPE), (dict(ws=None), NULL), (dict(ws=P + 8), ALIGN),
                   (dict(ws_bytes=1000), SHAPE), (dict(q=None), NULL),
                   (dict(out=None), NULL), (dict(q=P + 2), ALIGN), (dict(out=P + 8), ALIGN), (dict(q_ld=260), ALIGN),
                   (dict(lse=P + 2), ALIGN), (dict(q_lens=P + 2), ALIGN), (dict(B=0), OK), (dict(M=0), OK)):
        assert run(cache(), **kw) == rc, kw


def test_verify(lib):
    good = dict(logits=P, dtype=0, batch=400, row=100, d=P, q=P, u=P, e=P, T=P, lens=P, B=2, k=3, V=100, tokens=P,
                accepted=P, stream=None)
    for changes, rc in (({"dtype": 2}, UNSUPPORTED), ({"B": -1}, SHAPE), ({"k": -1}, SHAPE), ({"k": 32}, SHAPE),
                        ({"V": 0}, SHAPE), ({"V": 2**30 + 1, "row": 2**31, "batch": 2**34}, SHAPE), ({"row": 99}, SHAPE), ({"batch": -1}, SHAPE), ({"logits": None}, NULL),
                        ({"e": None}, NULL), ({"T": None}, NULL), ({"tokens": None}, NULL), ({"accepted": None}, NULL),
                        ({"d": None}, NULL), ({"u": None}, NULL), ({"logits": P + 1}, ALIGN),
                        ({"logits": P + 2, "dtype": 1}, ALIGN), ({"q": P + 2}, ALIGN), ({"tokens": P + 2}, ALIGN),
                        ({"B": 0}, OK)):
        assert call(lib.qmm_verify_draft, good, changes) == rc, changes


def test_injected_launch_failure(lib, monkeypatch):
    """The launch's own error comes back as QMM_ERR_CUDA; nothing is launched."""
    monkeypatch.setenv("QMM_TEST_INJECT", "launch_fail")
    assert lib.qmm_quantize_mx(P, 0, 4, 64, 64, 0, P, P, None, None) == 5
    assert lib.qmm_matmul_mx(P, P, P, P, 4, 8, 64, 0, P, 0, None) == 5
    assert lib.qmm_verify_draft(P, 0, 400, 100, P, P, P, P, P, P, 2, 3, 100, P, P, None) == 5
    c = cache()
    assert lib.qmm_kv_append(ctypes.byref(c), P, 128, P, 128, 3, 4, None, None) == 5
    assert lib.qmm_paged_attention(ctypes.byref(c), P, 256, 3, 4, 4, None, 1.0, 0, 0, P, P, P, 2**40, None) == 5
    assert lib.qmm_last_cuda_error() != 0
