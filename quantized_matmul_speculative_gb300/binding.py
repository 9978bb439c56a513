"""ctypes binding of libqmm (C ABI in ``include/qmm.h``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libqmm.so``.  PyTorch supplies device memory and the current
stream.  If the library has not been built, the first call raises
``RuntimeError``; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
from pathlib import Path

import numpy as np

LIBRARY = Path(__file__).resolve().parent / "libqmm.so"
MODULE = LIBRARY.with_name("_qmm_torch.so")

STATUS = {
    0: "QMM_OK",
    1: "QMM_ERR_NULL",
    2: "QMM_ERR_SHAPE",
    3: "QMM_ERR_UNSUPPORTED",
    4: "QMM_ERR_ALIGN",
    5: "QMM_ERR_CUDA",
    6: "QMM_ERR_TABLE",
}
OUT_BF16 = 0
OUT_F32 = 1

# Every function the header declares, with its ctypes signature.
_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
SIGNATURES = {
    "qmm_small_m": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "qmm_small_m_ex": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _i32, _i32, _i32, _vp]),
    "qmm_small_m_residual": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _i32, _i32, _i32,
                                    _vp]),
    "qmm_gather_small_m": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp,
                                  _i32, _i32, _i32, _vp]),
    "qmm_from_ggml": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "qmm_small_m_mx": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _i32, _i32, _vp]),
    "qmm_quantize_mx": (_i32, [_vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp]),
    "qmm_matmul_mx": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _vp]),
    "qmm_kv_append": (_i32, [_vp, _vp, _i64, _vp, _i64, _i32, _i32, _vp, _vp]),
    "qmm_paged_attention": (_i32, [_vp, _vp, _i64, _i32, _i32, _i32, _vp, _f32, _i32, _i32, _vp, _vp, _vp,
                                   ctypes.c_size_t, _vp]),
    "qmm_paged_attention_workspace": (ctypes.c_size_t, [_i32, _i32, _i32, _i32, _i32]),
    "qmm_verify_draft": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]),
    "qmm_packed_words": (ctypes.c_size_t, [_i64, _i64, _i32]),
    "qmm_pack": (_i32, [_vp, _i64, _i64, _i32, _vp]),
    "qmm_unpack": (_i32, [_vp, _i64, _i64, _i32, _vp]),
    "qmm_repack": (_i32, [_vp, _i64, _i64, _i32, _vp, _vp]),
    "qmm_unrepack": (_i32, [_vp, _i64, _i64, _i32, _vp, _vp]),
    "qmm_select_variant": (_i32, [_i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_i32)]),
    "qmm_num_variants": (_i32, []),
    "qmm_variant_name": (ctypes.c_char_p, [_i32]),
    "qmm_status_string": (ctypes.c_char_p, [_i32]),
    "qmm_last_cuda_error": (_i32, []),
    "qmm_device_status": (ctypes.c_uint, [_i32]),
    "qmm_version": (ctypes.c_char_p, []),
}


class PagedCacheStruct(ctypes.Structure):
    """``qmm_paged_cache`` of the header."""

    _fields_ = [("k", _vp), ("v", _vp), ("k_page", _i64), ("k_token", _i64), ("k_head", _i64), ("v_page", _i64),
                ("v_token", _i64), ("v_head", _i64), ("block_table", _vp), ("lengths", _vp), ("table_stride", _i64),
                ("num_pages", _i64), ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("k_scale", _f32),
                ("v_scale", _f32)]


class QmmError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        name = STATUS.get(status, str(status))
        super().__init__(f"{where}: {name}{(' (' + detail + ')') if detail else ''}")


_LIB = None


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        if not LIBRARY.exists():
            raise RuntimeError(f"{LIBRARY.name} is not built; run __graft_entry__.build() "
                               "or quantized_matmul_speculative_gb300/build.py")
        handle = ctypes.CDLL(str(LIBRARY))
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def _check(rc: int, where: str):
    if rc != 0:
        detail = ""
        if rc == 5:
            detail = f"cudaError {lib().qmm_last_cuda_error()}"
        raise QmmError(rc, where, detail)


# ---------------------------------------------------------------- host helpers
def packed_words(N: int, K: int, bits: int) -> int:
    return int(lib().qmm_packed_words(N, K, bits))


def pack(q: np.ndarray, bits: int) -> np.ndarray:
    """Pack uint8 codes [N, K] into uint32 words [N, K*bits/32] (host)."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    N, K = q.shape
    out = np.empty((N, K * bits // 32), dtype=np.uint32)
    _check(lib().qmm_pack(q.ctypes.data, N, K, bits, out.ctypes.data), "qmm_pack")
    return out


def unpack(wq: np.ndarray, K: int, bits: int) -> np.ndarray:
    wq = np.ascontiguousarray(wq, dtype=np.uint32)
    N = wq.shape[0]
    out = np.empty((N, K), dtype=np.uint8)
    _check(lib().qmm_unpack(wq.ctypes.data, N, K, bits, out.ctypes.data), "qmm_unpack")
    return out


def repack(wq, bits: int, out=None, inverse: bool = False, stream=None):
    """Canonical -> native packed layout on the device (inverse: native ->
    canonical).  ``wq``: CUDA int32/uint32 [N, K*bits/32]."""
    import torch

    if not wq.is_cuda or not wq.is_contiguous():
        raise ValueError("wq must be a contiguous CUDA tensor")
    N, words = wq.shape
    K = words * 32 // bits
    if out is None:
        out = torch.empty_like(wq)
    if stream is None:
        stream = torch.cuda.current_stream(wq.device)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    fn = lib().qmm_unrepack if inverse else lib().qmm_repack
    _check(fn(wq.data_ptr(), N, K, bits, out.data_ptr(), handle), "qmm_unrepack" if inverse else "qmm_repack")
    return out


GGML_TYPES = {"q4_0": (0, 18, 4), "q4_1": (1, 20, 4), "q8_0": (2, 34, 8)}
MX_FORMATS = {"mxfp4": (0, 4, 32), "mxfp8": (1, 8, 32), "nvfp4": (2, 4, 16)}


def small_m_mx(x, wq, scales, fmt: str, out=None, out_dtype=None, variant: int = -1, splits: int = -1,
               stream=None):
    """Y = X . W^T for microscaled W: ``wq`` int32 [N, K*bits/32] (E2M1 or
    E4M3 codes), ``scales`` uint8 [N, K/32] (E8M0) or [N, K/16] (nvfp4: E4M3);
    CUDA tensors."""
    import torch

    f, bits, g = MX_FORMATS[fmt]
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    M, K = x.shape
    N = wq.shape[0]
    if wq.shape[1] * 32 != K * bits or tuple(scales.shape) != (N, K // g) or scales.dtype != torch.uint8:
        raise ValueError("wq / scales do not match K and the format")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    _check(lib().qmm_small_m_mx(x.data_ptr(), wq.data_ptr(), scales.data_ptr(), M, N, K, f, out.data_ptr(),
                                OUT_F32 if out_dtype == torch.float32 else OUT_BF16, variant, splits, handle),
           "qmm_small_m_mx")
    return out


def from_ggml(kind: str, blocks, N: int, K: int, stream=None):
    """ggml blocks (CUDA uint8 tensor of N*K/32 blocks) -> (wq, scales, biases)
    in the affine layout with group size 32; returns the code width too."""
    import torch

    t, nbytes, bits = GGML_TYPES[kind]
    if not blocks.is_cuda or not blocks.is_contiguous() or blocks.numel() != N * (K // 32) * nbytes:
        raise ValueError("blocks must be a contiguous CUDA buffer of N*K/32 blocks")
    dev = blocks.device
    wq = torch.empty((N, K * bits // 32), dtype=torch.int32, device=dev)
    s = torch.empty((N, K // 32), dtype=torch.float16, device=dev)
    b = torch.empty((N, K // 32), dtype=torch.float16, device=dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    _check(lib().qmm_from_ggml(t, blocks.data_ptr(), N, K, wq.data_ptr(), s.data_ptr(), b.data_ptr(), handle),
           "qmm_from_ggml")
    return wq, s, b, bits


def select_variant(M: int, N: int, K: int, bits: int, group_size: int):
    s = ctypes.c_int(0)
    v = lib().qmm_select_variant(M, N, K, bits, group_size, ctypes.byref(s))
    return (v, s.value) if v >= 0 else (None, None)


def device_status(clear: bool = True) -> int:
    """OR of the kernels' device status words (0 = no bounded wait gave up)."""
    return int(lib().qmm_device_status(1 if clear else 0))


def variant_names():
    L = lib()
    return [L.qmm_variant_name(i).decode() for i in range(L.qmm_num_variants())]


# ---------------------------------------------------------------- device call
def small_m_ptr(x_ptr: int, wq_ptr: int, s_ptr: int, b_ptr: int, M: int, N: int, K: int, bits: int,
                group_size: int, y_ptr: int, out_dtype: int = OUT_BF16, variant: int = -1, splits: int = -1,
                stream: int = 0) -> None:
    """Raw-pointer call of qmm_small_m_ex (device pointers, cudaStream_t as int)."""
    rc = lib().qmm_small_m_ex(x_ptr, wq_ptr, s_ptr, b_ptr, M, N, K, bits, group_size, y_ptr,
                              out_dtype, variant, splits, stream)
    _check(rc, "qmm_small_m_ex")


def small_m_residual_ptr(x_ptr: int, wq_ptr: int, s_ptr: int, b_ptr: int, r_ptr: int, M: int, N: int, K: int,
                         bits: int, group_size: int, y_ptr: int, out_dtype: int = OUT_BF16, variant: int = -1,
                         splits: int = -1, stream: int = 0) -> None:
    """Raw-pointer call of qmm_small_m_residual: Y = R + X . dequant(W)^T."""
    rc = lib().qmm_small_m_residual(x_ptr, wq_ptr, s_ptr, b_ptr, r_ptr, M, N, K, bits, group_size, y_ptr,
                                    out_dtype, variant, splits, stream)
    _check(rc, "qmm_small_m_residual")


def gather_small_m_ptr(x_ptr: int, wq_ptr: int, s_ptr: int, b_ptr: int, lhs_ptr: int, rhs_ptr: int, P: int, T: int,
                       E: int, N: int, K: int, bits: int, group_size: int, y_ptr: int, out_dtype: int = OUT_BF16,
                       variant: int = -1, splits: int = -1, stream: int = 0) -> None:
    """Raw-pointer call of qmm_gather_small_m: Y[i] = X[lhs[i]] . W[rhs[i]]^T."""
    rc = lib().qmm_gather_small_m(x_ptr, wq_ptr, s_ptr, b_ptr, lhs_ptr, rhs_ptr, P, T, E, N, K, bits, group_size,
                                  y_ptr, out_dtype, variant, splits, stream)
    _check(rc, "qmm_gather_small_m")


def gather_small_m(x, wq, scales, biases, lhs, rhs, bits: int, group_size: int, out=None, out_dtype=None,
                   variant: int = -1, splits: int = -1, stream=None):
    """Y[i] = X[lhs[i]] . dequant(W[rhs[i]])^T over an expert stack.

    ``x``: bf16 [T, K]; ``wq``: int32 [E, N, K*bits/32]; ``scales``, ``biases``:
    fp16 [E, N, K/group_size]; ``lhs``, ``rhs``: int32 [P]; all contiguous CUDA
    tensors.  Returns ``out`` [P, N] (bf16 or fp32).
    """
    import torch

    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    for name, t in (("x", x), ("wq", wq), ("scales", scales), ("biases", biases), ("lhs", lhs), ("rhs", rhs)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if lhs.dtype != torch.int32 or rhs.dtype != torch.int32 or lhs.shape != rhs.shape or lhs.dim() != 1:
        raise TypeError("lhs and rhs must be int32 vectors of one length")
    T, K = x.shape
    E, N = wq.shape[0], wq.shape[1]
    if wq.shape[2] * 32 != K * bits or tuple(scales.shape) != (E, N, K // group_size):
        raise ValueError("wq / scales shapes do not match K, bits and group_size")
    P = lhs.shape[0]
    if out is None:
        out = torch.empty((P, N), dtype=out_dtype, device=x.device)
    elif tuple(out.shape) != (P, N) or out.dtype != out_dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous [P, N] tensor of out_dtype")
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    gather_small_m_ptr(x.data_ptr(), wq.data_ptr(), scales.data_ptr(), biases.data_ptr(), lhs.data_ptr(),
                       rhs.data_ptr(), P, T, E, N, K, bits, group_size, out.data_ptr(),
                       OUT_F32 if out_dtype == torch.float32 else OUT_BF16, variant, splits, handle)
    return out


def small_m(x, wq, scales, biases, bits: int, group_size: int, out=None, out_dtype=None,
            variant: int = -1, splits: int = -1, stream=None, residual=None):
    """Y = X . dequant(Wq, scales, biases)^T on the GPU (+ ``residual``).

    ``x``: bf16 [M, K]; ``wq``: int32/uint32 [N, K*bits/32]; ``scales``,
    ``biases``: fp16 [N, K/group_size]; all CUDA tensors, contiguous.  Returns
    ``out`` (bf16 or fp32 [M, N]), allocated by torch if not given.  With
    ``residual`` (a contiguous [M, N] tensor of the output dtype, which may be
    ``out`` itself) the kernels store residual + product.
    """
    import torch

    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if x.dtype != torch.bfloat16 or scales.dtype != torch.float16 or biases.dtype != torch.float16:
        raise TypeError("x must be bfloat16, scales and biases float16")
    if wq.dtype not in (torch.int32, getattr(torch, "uint32", torch.int32)):
        raise TypeError("wq must hold 32-bit words (int32 or uint32)")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out dtype must be bfloat16 or float32")
    for name, t in (("x", x), ("wq", wq), ("scales", scales), ("biases", biases)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    M, K = x.shape
    N = wq.shape[0]
    if wq.shape[1] * 32 != K * bits:
        raise ValueError("wq shape does not match K and bits")
    if tuple(scales.shape) != (N, K // group_size) or tuple(biases.shape) != (N, K // group_size):
        raise ValueError("scales/biases must be [N, K/group_size]")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    elif tuple(out.shape) != (M, N) or out.dtype != out_dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous [M, N] tensor of out_dtype")
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    od = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    if residual is None:
        small_m_ptr(x.data_ptr(), wq.data_ptr(), scales.data_ptr(), biases.data_ptr(), M, N, K, bits, group_size,
                    out.data_ptr(), od, variant, splits, handle)
        return out
    if (not residual.is_cuda or not residual.is_contiguous() or tuple(residual.shape) != (M, N)
            or residual.dtype != out_dtype):
        raise ValueError("residual must be a contiguous CUDA [M, N] tensor of the output dtype")
    small_m_residual_ptr(x.data_ptr(), wq.data_ptr(), scales.data_ptr(), biases.data_ptr(), residual.data_ptr(),
                         M, N, K, bits, group_size, out.data_ptr(), od, variant, splits, handle)
    return out


# ------------------------------------------------- the operators around the product
# A call of these takes microseconds on the GPU, so their tensors are checked and
# allocated by the native module (csrc/qmm_torch.cpp).  ``stream`` (a torch stream or
# a cudaStream_t as an integer; None: the current stream) of each: a call on another
# stream waits for the work that the current one has been given, and its tensors'
# memory is not handed out again before it is done; what reads its results on the
# current stream has to wait for it.
@functools.lru_cache(maxsize=1)
def _native():
    import torch  # noqa: F401  (loads the libraries that the module links)

    lib()
    try:
        from . import _qmm_torch
    except ImportError as e:
        what = "does not load here" if MODULE.exists() else "is not built"
        raise RuntimeError(f"{MODULE.name} {what} ({e}); run __graft_entry__.build() "
                           "or quantized_matmul_speculative_gb300/build.py") from e
    return _qmm_torch


def _handle(stream):
    """cudaStream_t of a stream (a torch stream or an integer) or None."""
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _result(r, where: str):
    if type(r) is int:
        _check(r, where)
    return r


def quantize_mx(x, fmt: str, values=None, out=None, stream=None):
    """Microscaled codes and scale bytes of ``x`` [R, K] (bf16 or fp32; rows may
    be strided), formats as :func:`small_m_mx`: returns (codes int32
    [R, K*bits/32], scales uint8 [R, K/g]), into ``out`` if given.  ``values``:
    an optional bf16 [R, K] tensor that receives what the codes stand for."""
    f, bits, g = MX_FORMATS[fmt]
    codes, scales = (None, None) if out is None else out
    return _result(_native().quantize_mx(x, f, bits, g, values, codes, scales, _handle(stream)), "qmm_quantize_mx")


def matmul_mx(xq, x_scales, wq, w_scales, fmt: str, out=None, out_dtype=None, stream=None):
    """Y = X . W^T of two microscaled 4-bit matrices (``"mxfp4"`` or ``"nvfp4"``)
    as :func:`quantize_mx` gives them, any number of rows; Y bf16 or fp32 [M, N]."""
    import torch

    f, bits, g = MX_FORMATS[fmt]
    if bits != 4:
        raise ValueError("matmul_mx takes the 4-bit formats")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    f32 = out_dtype is torch.float32
    if not (f32 or out_dtype is torch.bfloat16):
        raise TypeError("out dtype must be bfloat16 or float32")
    return _result(_native().matmul_mx(xq, x_scales, wq, w_scales, f, g, out, f32, _handle(stream)), "qmm_matmul_mx")


def kv_append(k_new, v_new, k_cache, v_cache, block_table, lengths, q_lens=None, k_scale: float = 1.0,
              v_scale: float = 1.0, stream=None):
    """Write the new rows' keys and values into a paged cache.

    ``k_new``, ``v_new``: bf16 [B, M, heads, D] (rows may be strided, e.g.
    slices of a fused projection); ``k_cache``, ``v_cache``: bf16 or
    float8_e4m3fn [pages, page_size, heads, D], any strides with D contiguous;
    ``block_table``: int32 [B, max_pages]; ``lengths``: int32 [B], tokens of
    each sequence with its new rows; ``q_lens``: int32 [B], new rows of each
    sequence (None: M).  Row i of sequence b goes to position
    lengths[b] - q_lens[b] + i.  E4M3 elements hold x / scale."""
    _result(_native().kv_append(k_new, v_new, k_cache, v_cache, block_table, lengths, q_lens, k_scale, v_scale,
                                _handle(stream)), "qmm_kv_append")


@functools.lru_cache(maxsize=256)
def paged_attention_workspace(B: int, M: int, q_heads: int, heads: int, head_dim: int) -> int:
    """Bytes of workspace that :func:`paged_attention` needs for these sizes."""
    return int(lib().qmm_paged_attention_workspace(B, M, q_heads, heads, head_dim))


def paged_attention(q, k_cache, v_cache, block_table, lengths, q_lens=None, scale: float | None = None, window: int = 0,
                    sinks: int = 0, k_scale: float = 1.0, v_scale: float = 1.0, out=None, return_lse: bool = False,
                    workspace=None, stream=None):
    """Attention of M = 1..16 new rows per sequence over a paged cache.

    ``q``: bf16 [B, M, q_heads, D] (rows may be strided); the cache as in
    :func:`kv_append`, already holding the new rows.  Row i of sequence b sees
    the tokens up to its own position; with ``window`` > 0 only the last
    ``window`` of them and the first ``sinks`` of the sequence.  ``scale``
    defaults to 1/sqrt(D).  Returns ``out`` bf16 [B, M, q_heads, D], with
    ``return_lse`` also the fp32 [B, M, q_heads] log-sum-exp of the scaled
    scores (-inf, and 0 in ``out``, for rows that see nothing).  ``workspace``:
    a uint8 tensor of :func:`paged_attention_workspace` bytes to reuse."""
    return _result(_native().paged_attention(q, k_cache, v_cache, block_table, lengths, q_lens, k_scale, v_scale, scale,
                                             window, sinks, out, return_lse, workspace, _handle(stream)),
                   "qmm_paged_attention")


def verify_draft(logits, draft_tokens, draft_probs, uniform, noise, temperature, draft_lens=None, stream=None):
    """Accept or refuse drafted tokens against the target's logits.

    ``logits``: bf16 or fp32 [B, k+1, V] (a row's elements contiguous);
    ``draft_tokens``: int32 [B, k]; ``draft_probs``: fp32 [B, k, V] the drafts
    were drawn from, or None if they were certain; ``uniform``: fp32 [B, k] in
    [0, 1); ``noise``: fp32 [B, V], exponentially distributed;
    ``temperature``: fp32 [B], 0 for greedy; ``draft_lens``: int32 [B] or None.
    Returns (tokens int32 [B, k+1]: the accepted drafts, the next token, then
    -1; accepted int32 [B])."""
    return _result(_native().verify_draft(logits, draft_tokens, draft_probs, uniform, noise, temperature, draft_lens,
                                          _handle(stream)), "qmm_verify_draft")
