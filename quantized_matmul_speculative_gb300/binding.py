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
# A call of these takes microseconds on the GPU, so the checks below are written
# for their cost: integers for devices, one comparison per property.
def _index(t, name: str) -> int:
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return i


def _same_device(index: int, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on CUDA device {index}")


def _launch_on(stream, index: int):
    """(cudaStream_t as int, the stream to record new tensors on or None) of a
    call.  Outputs and workspaces are allocated on the current stream; a call
    that runs on another one has them recorded there, so that their memory is
    not handed out again before the call is done."""
    import torch

    if torch._C._cuda_getDevice() != index:
        raise ValueError(f"the current CUDA device must be the tensors' device {index}")
    current = torch._C._cuda_getCurrentRawStream(index)
    if stream is None:
        return current, None
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle == current:
        return handle, None
    return handle, stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(handle, device=index)


def _new(like, shape, dtype, record):
    import torch

    t = torch.empty(shape, dtype=dtype, device=like.device)
    if record is not None:
        # the caching allocator may have handed out memory that the current
        # stream still works on: the call's stream waits for it
        record.wait_stream(torch.cuda.current_stream(t.device))
        t.record_stream(record)
    return t


def _is(t, dtype, shape) -> bool:
    return t.dtype is dtype and t.shape == shape and t.is_contiguous()


def quantize_mx(x, fmt: str, values=None, out=None, stream=None):
    """Microscaled codes and scale bytes of ``x`` [R, K] (bf16 or fp32; rows may
    be strided), formats as :func:`small_m_mx`: returns (codes int32
    [R, K*bits/32], scales uint8 [R, K/g]), into ``out`` if given.  ``values``:
    an optional bf16 [R, K] tensor that receives what the codes stand for."""
    import torch

    f, bits, g = MX_FORMATS[fmt]
    f32 = x.dtype is torch.float32
    if x.dim() != 2 or not (f32 or x.dtype is torch.bfloat16):
        raise TypeError("x must be a bfloat16 or float32 matrix")
    R, K = x.shape
    index = _index(x, "x")
    if K % 32 != 0:
        raise ValueError("K must be a multiple of 32")
    ld, one = x.stride()
    if R <= 1:
        ld = K
    if K > 1 and one != 1 or ld < K:
        raise ValueError("the elements of a row of x must be contiguous, and its rows apart")
    if values is not None and (not _is(values, torch.bfloat16, x.shape) or values.get_device() != index):
        raise ValueError("values must be a contiguous bfloat16 tensor of x's shape, on its device")
    handle, record = _launch_on(stream, index)
    if out is None:
        codes = _new(x, (R, K * bits // 32), torch.int32, record)
        scales = _new(x, (R, K // g), torch.uint8, record)
    else:
        codes, scales = out
        _same_device(index, codes, scales)
        if not _is(codes, torch.int32, (R, K * bits // 32)) or not _is(scales, torch.uint8, (R, K // g)):
            raise ValueError("out must be contiguous (int32 [R, K*bits/32], uint8 [R, K/g])")
    rc = lib().qmm_quantize_mx(x.data_ptr(), OUT_F32 if f32 else OUT_BF16, R, K, ld, f, codes.data_ptr(),
                               scales.data_ptr(), None if values is None else values.data_ptr(), handle)
    if rc != 0:
        _check(rc, "qmm_quantize_mx")
    return codes, scales


def matmul_mx(xq, x_scales, wq, w_scales, fmt: str, out=None, out_dtype=None, stream=None):
    """Y = X . W^T of two microscaled 4-bit matrices (``"mxfp4"`` or ``"nvfp4"``)
    as :func:`quantize_mx` gives them, any number of rows; Y bf16 or fp32 [M, N]."""
    import torch

    f, bits, g = MX_FORMATS[fmt]
    if bits != 4:
        raise ValueError("matmul_mx takes the 4-bit formats")
    if xq.dim() != 2 or wq.dim() != 2:
        raise ValueError("codes must be matrices")
    index = _index(xq, "xq")
    _same_device(index, x_scales, wq, w_scales, out)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    f32 = out_dtype is torch.float32
    if not (f32 or out_dtype is torch.bfloat16):
        raise TypeError("out dtype must be bfloat16 or float32")
    M, words = xq.shape
    N, K = wq.shape[0], words * 8
    if not (_is(xq, torch.int32, (M, words)) and _is(wq, torch.int32, (N, words))):
        raise ValueError("xq and wq must be contiguous int32 [M, K/8] and [N, K/8]")
    if not (_is(x_scales, torch.uint8, (M, K // g)) and _is(w_scales, torch.uint8, (N, K // g))):
        raise ValueError("x_scales and w_scales must be contiguous uint8 [M, K/g] and [N, K/g]")
    handle, record = _launch_on(stream, index)
    if out is None:
        out = _new(xq, (M, N), out_dtype, record)
    elif not _is(out, out_dtype, (M, N)):
        raise ValueError("out must be a contiguous [M, N] tensor of out_dtype")
    rc = lib().qmm_matmul_mx(xq.data_ptr(), x_scales.data_ptr(), wq.data_ptr(), w_scales.data_ptr(), M, N, K, f,
                             out.data_ptr(), OUT_F32 if f32 else OUT_BF16, handle)
    if rc != 0:
        _check(rc, "qmm_matmul_mx")
    return out


def _paged_cache(index, k_cache, v_cache, block_table, lengths, q_lens, k_scale, v_scale, B):
    import torch

    _same_device(index, k_cache, v_cache, block_table, lengths, q_lens)
    dtype = k_cache.dtype
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or v_cache.dtype is not dtype:
        raise ValueError("k_cache and v_cache must be [pages, page_size, heads, D] of one shape and dtype")
    if not (dtype is torch.bfloat16 or dtype is torch.float8_e4m3fn):
        raise TypeError("the cache must be bfloat16 or float8_e4m3fn")
    k_page, k_token, k_head, k_one = k_cache.stride()
    v_page, v_token, v_head, v_one = v_cache.stride()
    if k_one != 1 or v_one != 1:
        raise ValueError("the D elements of a head must be contiguous")
    rows, width = block_table.shape
    ld, one = block_table.stride()
    if rows != B or block_table.dtype is not torch.int32 or (width > 1 and one != 1):
        raise ValueError("block_table must be int32 [B, max_pages] with contiguous rows")
    if not _is(lengths, torch.int32, (B,)):
        raise ValueError("lengths must be contiguous int32 [B]")
    if q_lens is not None and not _is(q_lens, torch.int32, (B,)):
        raise ValueError("q_lens must be contiguous int32 [B]")
    pages, page_size, heads, D = k_cache.shape
    return PagedCacheStruct(k_cache.data_ptr(), v_cache.data_ptr(), k_page, k_token, k_head, v_page, v_token, v_head,
                            block_table.data_ptr(), lengths.data_ptr(), ld if B > 1 else width, pages, width, page_size,
                            heads, D, 0 if dtype is torch.bfloat16 else 1, k_scale, v_scale)


def _rows(t, B, M, heads, D, name):
    """Distance of the [B, M] rows of ``t`` [B, M, heads, D] (one distance for
    all; a row's elements are contiguous)."""
    import torch

    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    s0, s1, s2, s3 = t.stride()
    ld = s1 if M > 1 else s0 if B > 1 else heads * D
    if (D > 1 and s3 != 1) or (heads > 1 and s2 != D) or (B > 1 and M > 1 and s0 != M * ld):
        raise ValueError(f"{name}: the heads of a row must be contiguous and its rows evenly apart")
    return ld


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
    if k_new.dim() != 4 or k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new must be [B, M, heads, D] of one shape")
    B, M, heads, D = k_new.shape
    index = _index(k_new, "k_new")
    _same_device(index, v_new)
    cache = _paged_cache(index, k_cache, v_cache, block_table, lengths, q_lens, k_scale, v_scale, B)
    if heads != cache.heads or D != cache.head_dim:
        raise ValueError("k_new and the cache must have the same heads and D")
    k_ld, v_ld = _rows(k_new, B, M, heads, D, "k_new"), _rows(v_new, B, M, heads, D, "v_new")
    handle, _ = _launch_on(stream, index)
    rc = lib().qmm_kv_append(ctypes.byref(cache), k_new.data_ptr(), k_ld, v_new.data_ptr(), v_ld, B, M,
                             None if q_lens is None else q_lens.data_ptr(), handle)
    if rc != 0:
        _check(rc, "qmm_kv_append")


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
    import torch

    if q.dim() != 4:
        raise ValueError("q must be [B, M, q_heads, D]")
    B, M, Hq, D = q.shape
    index = _index(q, "q")
    _same_device(index, out, workspace)
    cache = _paged_cache(index, k_cache, v_cache, block_table, lengths, q_lens, k_scale, v_scale, B)
    if D != cache.head_dim:
        raise ValueError("q and the cache must have the same D")
    q_ld = _rows(q, B, M, Hq, D, "q")
    handle, record = _launch_on(stream, index)
    if out is None:
        out = _new(q, (B, M, Hq, D), torch.bfloat16, record)
    elif not _is(out, torch.bfloat16, (B, M, Hq, D)):
        raise ValueError("out must be a contiguous bfloat16 tensor of q's shape")
    lse = _new(q, (B, M, Hq), torch.float32, record) if return_lse else None
    if workspace is None:
        workspace = _new(q, (paged_attention_workspace(B, M, Hq, cache.heads, D),), torch.uint8, record)
    elif workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    rc = lib().qmm_paged_attention(ctypes.byref(cache), q.data_ptr(), q_ld, B, M, Hq,
                                   None if q_lens is None else q_lens.data_ptr(), D ** -0.5 if scale is None else scale,
                                   window, sinks, out.data_ptr(), None if lse is None else lse.data_ptr(),
                                   workspace.data_ptr(), workspace.numel(), handle)
    if rc != 0:
        _check(rc, "qmm_paged_attention")
    return (out, lse) if return_lse else out


def verify_draft(logits, draft_tokens, draft_probs, uniform, noise, temperature, draft_lens=None, stream=None):
    """Accept or refuse drafted tokens against the target's logits.

    ``logits``: bf16 or fp32 [B, k+1, V] (a row's elements contiguous);
    ``draft_tokens``: int32 [B, k]; ``draft_probs``: fp32 [B, k, V] the drafts
    were drawn from, or None if they were certain; ``uniform``: fp32 [B, k] in
    [0, 1); ``noise``: fp32 [B, V], exponentially distributed;
    ``temperature``: fp32 [B], 0 for greedy; ``draft_lens``: int32 [B] or None.
    Returns (tokens int32 [B, k+1]: the accepted drafts, the next token, then
    -1; accepted int32 [B])."""
    import torch

    if logits.dim() != 3 or logits.shape[1] < 1 or logits.shape[2] < 1:
        raise ValueError("logits must be [B, k+1, V]")
    f32 = logits.dtype is torch.float32
    if not (f32 or logits.dtype is torch.bfloat16):
        raise TypeError("logits must be bfloat16 or float32")
    B, rows, V = logits.shape
    k = rows - 1
    index = _index(logits, "logits")
    _same_device(index, draft_tokens, draft_probs, uniform, noise, temperature, draft_lens)
    s_batch, s_row, one = logits.stride()
    if V > 1 and one != 1:
        raise ValueError("the elements of a row of logits must be contiguous")
    if not (_is(draft_tokens, torch.int32, (B, k)) and _is(uniform, torch.float32, (B, k))):
        raise ValueError("draft_tokens and uniform must be contiguous int32 and float32 [B, k]")
    if not (_is(noise, torch.float32, (B, V)) and _is(temperature, torch.float32, (B,))):
        raise ValueError("noise and temperature must be contiguous float32 [B, V] and [B]")
    if draft_probs is not None and not _is(draft_probs, torch.float32, (B, k, V)):
        raise ValueError("draft_probs must be contiguous float32 [B, k, V]")
    if draft_lens is not None and not _is(draft_lens, torch.int32, (B,)):
        raise ValueError("draft_lens must be contiguous int32 [B]")
    handle, record = _launch_on(stream, index)
    tokens = _new(logits, (B, rows), torch.int32, record)
    accepted = _new(logits, (B,), torch.int32, record)
    rc = lib().qmm_verify_draft(logits.data_ptr(), OUT_F32 if f32 else OUT_BF16, s_batch if B > 1 else rows * V,
                                s_row if rows > 1 else V, draft_tokens.data_ptr(),
                                None if draft_probs is None else draft_probs.data_ptr(), uniform.data_ptr(),
                                noise.data_ptr(), temperature.data_ptr(),
                                None if draft_lens is None else draft_lens.data_ptr(), B, k, V, tokens.data_ptr(),
                                accepted.data_ptr(), handle)
    if rc != 0:
        _check(rc, "qmm_verify_draft")
    return tokens, accepted
