// Quantisation into the microscaling formats (qmm_quantize_mx; the arithmetic
// is defined in include/qmm.h).
#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

struct QuantArgs {
  const void* X;
  int64_t R, K, ldx;
  uint32_t* Wq;
  uint8_t* S;
  __nv_bfloat16* values;
  int wide;  // codes and values can be stored as vectors
};

// Pairs, nearest even, saturating.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float hi, float lo) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t cvt_e2m1x2(float hi, float lo) {
  uint32_t r;
  asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n cvt.u32.u8 %0, b;\n}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(0x80008000u));
  return r;
}

// Eight consecutive elements as fp32.
template <bool F32, bool VEC>
struct Eight {
  uint4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < (F32 ? 2 : 1); ++i) w[i] = ld_after_wait_v4(static_cast<const uint4*>(p) + i);
    } else {
      uint32_t u[F32 ? 8 : 4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (F32) u[i] = __float_as_uint(static_cast<const float*>(p)[i]);
        else if (i & 1) u[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16;
        else u[i / 2] = static_cast<const uint16_t*>(p)[i];
      }
#pragma unroll
      for (int i = 0; i < (F32 ? 2 : 1); ++i) w[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
    }
  }
  // The largest magnitude's bit pattern, as fp32 (magnitudes order like their patterns, NaN above infinity).
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (F32) {
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        t = max(t, max(w[i].x & 0x7FFFFFFFu, w[i].y & 0x7FFFFFFFu));
        t = max(t, max(w[i].z & 0x7FFFFFFFu, w[i].w & 0x7FFFFFFFu));
      }
      return t;
    } else {
      const uint32_t t = __vmaxu2(__vmaxu2(w[0].x & 0x7FFF7FFFu, w[0].y & 0x7FFF7FFFu),
                                  __vmaxu2(w[0].z & 0x7FFF7FFFu, w[0].w & 0x7FFF7FFFu));
      return max(t << 16, t & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (F32) x[4 * i + j] = __uint_as_float(u[j]);
        else x[2 * j] = bf16_lo(u[j]), x[2 * j + 1] = bf16_hi(u[j]);
      }
    }
  }
};

// A thread takes eight elements (a word of 4-bit codes, two of 8-bit ones) at U
// places; the threads of a group (two of nvfp4's 16, four of 32) find its
// maximum by shuffles.
//
// The rounding of x / s must be that of the exact quotient.  The mx scales are
// powers of two: the product with the reciprocal is exact.  nvfp4: fp32 inputs
// are divided; a bf16 input (8 significant bits) over an E4M3 scale (4) is
// either exactly a midpoint of two codes (a multiple of 1/4 up to 5) or 2^-10
// and more away from it, so x * (1/s), off by some 2^-22, is rounded to
// multiples of 2^-18 first (by adding 48 and subtracting it again: the quotient
// is below 16 in magnitude, or saturates), which restores exact midpoints.
//
// What bounds it: HBM.  34816 x 5120 bf16 to nvfp4 with the values written too
// took 872 us with a thread per group and scalar loads.
template <int FMT, bool F32, bool LINEAR, bool VEC, int U>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a) {
  constexpr int G = FMT == QMM_NVFP4 ? 16 : 32;
  griddep_wait();
  const int64_t total = a.R * (a.K / 8);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * U) + threadIdx.x;
  Eight<F32, VEC> in[U];
  constexpr int ES = F32 ? 4 : 2;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = first + u * 256;
    if (i < total) {
      int64_t at = i * 8;
      if constexpr (!LINEAR) {
        const int64_t row = i / (a.K / 8);
        at = row * a.ldx + (i - row * (a.K / 8)) * 8;
      }
      in[u].load(static_cast<const char*>(a.X) + at * ES);
    } else {
#pragma unroll
      for (int x = 0; x < (F32 ? 2 : 1); ++x) in[u].w[x] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = first + u * 256;
    uint32_t top = in[u].top();
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if (G == 32) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool bad = top >= 0x7F800000u;
    uint32_t byte;
    float s, r;  // the scale and its reciprocal
    if constexpr (FMT == QMM_NVFP4) {
      byte = bad ? 0x7Fu : cvt_e4m3x2(0.f, __fdiv_rn(__uint_as_float(top), 6.f)) & 0xFFu;
      s = e4m3_to_float(byte);
      r = s > 0.f ? __frcp_rn(s) : 0.f;
    } else {
      const int e = static_cast<int>(top >> 23) - (FMT == QMM_MXFP8 ? 8 : 2);
      byte = bad ? 0xFFu : static_cast<uint32_t>(max(e, 0));
      s = e8m0_to_float(byte);
      r = __uint_as_float((254u - min(byte, 253u)) << 23);
    }
    float x[8];
    in[u].get(x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (FMT == QMM_NVFP4 && F32) {
        x[j] = s > 0.f ? __fdiv_rn(x[j], s) : copysignf(0.f, x[j]);
      } else if constexpr (FMT == QMM_NVFP4) {
        const float y = __fadd_rn(__fmaf_rn(x[j], r, 48.f), -48.f);
        x[j] = __uint_as_float((__float_as_uint(y) & 0x7FFFFFFFu) | (__float_as_uint(x[j]) & 0x80000000u));
      } else {
        x[j] = x[j] * r;
      }
    }
    constexpr int W = FMT == QMM_MXFP8 ? 2 : 1;
    uint32_t code[W];
    if constexpr (FMT == QMM_MXFP8) {
#pragma unroll
      for (int j = 0; j < 2; ++j) code[j] = cvt_e4m3x2(x[4 * j + 1], x[4 * j]) | (cvt_e4m3x2(x[4 * j + 3], x[4 * j + 2]) << 16);
    } else {
      code[0] = cvt_e2m1x2(x[1], x[0]) | (cvt_e2m1x2(x[3], x[2]) << 8) | (cvt_e2m1x2(x[5], x[4]) << 16) | (cvt_e2m1x2(x[7], x[6]) << 24);
    }
    if (bad) {
#pragma unroll
      for (int j = 0; j < W; ++j) code[j] = 0;
    }
    if (i >= total) continue;
    if constexpr (W == 2) {
      if (a.wide) reinterpret_cast<uint2*>(a.Wq)[i] = make_uint2(code[0], code[1]);
      else a.Wq[2 * i] = code[0], a.Wq[2 * i + 1] = code[1];
    } else {
      a.Wq[i] = code[0];
    }
    if ((threadIdx.x & (G / 8 - 1)) == 0) a.S[i / (G / 8)] = static_cast<uint8_t>(byte);
    if (a.values != nullptr) {
      // bf16 holds the scale (a power of two, or E4M3's four bits) and the product with an E2M1 or E4M3 value
      const uint32_t sv = bad ? 0x7FC07FC0u : (__float_as_uint(s) >> 16) * 0x10001u;
      uint32_t v[4];
      if constexpr (FMT == QMM_MXFP8) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t p0 = unpack_fp8_pair(code[j], 0), p1 = unpack_fp8_pair(code[j], 1);  // (0, 2) and (1, 3)
          v[2 * j] = mul_bf16x2(prmt_lo(p0, p1), sv);
          v[2 * j + 1] = mul_bf16x2(prmt_hi(p0, p1), sv);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t p0 = unpack_fp4_pair(code[0], 2 * j), p1 = unpack_fp4_pair(code[0], 2 * j + 1);  // (2j, 2j + 4), ..
          v[j] = mul_bf16x2(prmt_lo(p0, p1), sv);
          v[j + 2] = mul_bf16x2(prmt_hi(p0, p1), sv);
        }
      }
      if (a.wide) {
        reinterpret_cast<uint4*>(a.values)[i] = make_uint4(v[0], v[1], v[2], v[3]);
      } else {
        uint16_t* const o = reinterpret_cast<uint16_t*>(a.values) + 8 * i;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[2 * j] = static_cast<uint16_t>(v[j]), o[2 * j + 1] = static_cast<uint16_t>(v[j] >> 16);
      }
    }
  }
  publish_weights();  // (what follows may be the product that reads them)
}

template <int FMT, bool F32>
cudaError_t launch_quantize(QuantArgs a, cudaStream_t st) {
  const int64_t total = a.R * (a.K / 8);
  const bool vec = reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && (a.ldx * (F32 ? 4 : 2)) % 16 == 0;
  a.wide = reinterpret_cast<uintptr_t>(a.Wq) % 8 == 0 && reinterpret_cast<uintptr_t>(a.values) % 16 == 0;
  // four places a thread (their loads in flight together) where that still fills the SMs
  const int u = total >= 4 * 256 * 4 * static_cast<int64_t>(device_sm_count()) ? 4 : 1;
  const dim3 grid(static_cast<unsigned>((total + 256 * u - 1) / (256 * u)));
  if (!vec) return launch_dependent(quantize_kernel<FMT, F32, false, false, 1>, dim3(static_cast<unsigned>((total + 255) / 256)), 256, 0, st, a);
  if (a.ldx != a.K) return u == 4 ? launch_dependent(quantize_kernel<FMT, F32, false, true, 4>, grid, 256, 0, st, a)
                                  : launch_dependent(quantize_kernel<FMT, F32, false, true, 1>, grid, 256, 0, st, a);
  return u == 4 ? launch_dependent(quantize_kernel<FMT, F32, true, true, 4>, grid, 256, 0, st, a)
                : launch_dependent(quantize_kernel<FMT, F32, true, true, 1>, grid, 256, 0, st, a);
}

}  // namespace
}  // namespace qmm

extern "C" qmm_status qmm_quantize_mx(const void* X, int x_dtype, int64_t R, int64_t K, int64_t ldx, int format,
                                      uint32_t* Wq, uint8_t* scales, void* values, void* stream) {
  using namespace qmm;
  if (format != QMM_MXFP4 && format != QMM_MXFP8 && format != QMM_NVFP4) return QMM_ERR_UNSUPPORTED;
  if (x_dtype != QMM_OUT_BF16 && x_dtype != QMM_OUT_F32) return QMM_ERR_UNSUPPORTED;
  if (R < 0 || K < 0 || K % 32 != 0 || ldx < K || R > (int64_t(1) << 38) / (K + 1)) return QMM_ERR_SHAPE;
  if (R == 0 || K == 0) return QMM_OK;
  if (ldx > (int64_t(1) << 40) / R) return QMM_ERR_SHAPE;
  if (X == nullptr || Wq == nullptr || scales == nullptr) return QMM_ERR_NULL;
  const uintptr_t esize = x_dtype == QMM_OUT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(X) % esize || reinterpret_cast<uintptr_t>(Wq) % 4 ||
      reinterpret_cast<uintptr_t>(values) % 2)
    return QMM_ERR_ALIGN;
  if (R * (K / 8) > int64_t(256) * 0x7fffffff) return QMM_ERR_SHAPE;
  const QuantArgs a{X, R, K, R == 1 ? K : ldx, Wq, scales, static_cast<__nv_bfloat16*>(values), 0};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = x_dtype == QMM_OUT_F32;
  const cudaError_t e = format == QMM_MXFP4   ? (f32 ? launch_quantize<QMM_MXFP4, true>(a, st) : launch_quantize<QMM_MXFP4, false>(a, st))
                        : format == QMM_MXFP8 ? (f32 ? launch_quantize<QMM_MXFP8, true>(a, st) : launch_quantize<QMM_MXFP8, false>(a, st))
                                              : (f32 ? launch_quantize<QMM_NVFP4, true>(a, st) : launch_quantize<QMM_NVFP4, false>(a, st));
  return static_cast<qmm_status>(finish_call(e));
}
