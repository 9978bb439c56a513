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
};

__device__ __forceinline__ uint32_t cvt_e4m3(float x) {  // nearest even, saturating
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}
__device__ __forceinline__ uint32_t cvt_e2m1(float x) {
  uint32_t r;
  asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n cvt.u32.u8 %0, b;\n}" : "=r"(r) : "f"(0.f), "f"(x));
  return r & 0xFu;
}
__device__ __forceinline__ float e2m1_to_float(uint32_t c) {
  const uint32_t v = ((c & 7u) << 22) | ((c & 8u) << 28);
  return __uint_as_float(v) * 8.507059173023461586584e37f;  // 2^126
}

// One thread per group.
template <int FMT, bool F32>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a) {
  constexpr int G = FMT == QMM_NVFP4 ? 16 : 32, BITS = FMT == QMM_MXFP8 ? 8 : 4, PER = 32 / BITS;
  griddep_wait();
  const int64_t per_row = a.K / G;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.R * per_row) return;
  const int64_t row = i / per_row, col = (i - row * per_row) * G;
  float x[G];
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    x[j] = F32 ? static_cast<const float*>(a.X)[row * a.ldx + col + j]
               : __bfloat162float(static_cast<const __nv_bfloat16*>(a.X)[row * a.ldx + col + j]);
    amax = fmaxf(amax, fabsf(x[j]));
    bad |= !(fabsf(x[j]) <= 3.4028235e38f);
  }
  uint32_t sb;
  float s;
  if (FMT == QMM_NVFP4) {
    sb = cvt_e4m3(__fdiv_rn(amax, 6.f));
    s = e4m3_to_float(sb);
  } else {
    const int e = static_cast<int>(__float_as_uint(amax) >> 23) - (FMT == QMM_MXFP8 ? 8 : 2);
    sb = static_cast<uint32_t>(e < 0 ? 0 : e);
    s = e8m0_to_float(sb);
  }
  if (bad) {
    sb = FMT == QMM_NVFP4 ? 0x7Fu : 0xFFu;
    s = __uint_as_float(0x7FC00000u);
  }
  a.S[i] = static_cast<uint8_t>(sb);
#pragma unroll
  for (int w = 0; w < G / PER; ++w) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const float v = x[w * PER + j];
      const float y = s > 0.f ? __fdiv_rn(v, s) : copysignf(0.f, v);
      const uint32_t c = bad ? 0u : FMT == QMM_MXFP8 ? cvt_e4m3(y) : cvt_e2m1(y);
      word |= c << (BITS * j);
      if (a.values != nullptr)
        a.values[row * a.K + col + w * PER + j] =
            __float2bfloat16_rn((FMT == QMM_MXFP8 ? e4m3_to_float(c) : e2m1_to_float(c)) * s);
    }
    a.Wq[i * (G / PER) + w] = word;
  }
}

template <int FMT>
cudaError_t launch_quantize(const QuantArgs& a, bool f32, cudaStream_t st) {
  const int64_t groups = a.R * (a.K / (FMT == QMM_NVFP4 ? 16 : 32));
  const dim3 grid(static_cast<unsigned>((groups + 255) / 256));
  return f32 ? launch_dependent(quantize_kernel<FMT, true>, grid, 256, 0, st, a)
             : launch_dependent(quantize_kernel<FMT, false>, grid, 256, 0, st, a);
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
  QuantArgs a{X, R, K, ldx, Wq, scales, static_cast<__nv_bfloat16*>(values)};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = x_dtype == QMM_OUT_F32;
  const cudaError_t e = format == QMM_MXFP4   ? launch_quantize<QMM_MXFP4>(a, f32, st)
                        : format == QMM_MXFP8 ? launch_quantize<QMM_MXFP8>(a, f32, st)
                                              : launch_quantize<QMM_NVFP4>(a, f32, st);
  return static_cast<qmm_status>(finish_call(e));
}
