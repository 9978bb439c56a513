// Product of two microscaled 4-bit matrices (qmm_matmul_mx, include/qmm.h).
#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

struct MxMatmulArgs {
  const uint32_t* Xq;
  const uint8_t* xs;
  const uint32_t* Wq;
  const uint8_t* ws;
  void* Y;
  int M, N, K, out_f32;
};

__device__ __forceinline__ float e2m1_to_float(uint32_t c) {
  return __uint_as_float(((c & 7u) << 22) | ((c & 8u) << 28)) * 8.507059173023461586584e37f;  // 2^126
}

// 64 x 64 output tile, 256 threads of 4 x 4 outputs, 32 codes of K at a time
// dequantised to fp32 in shared memory.
template <bool NV>
__global__ void __launch_bounds__(256) mx_matmul_kernel(const MxMatmulArgs a) {
  __shared__ float xt[32][65], wt[32][65];
  griddep_wait();
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 64, n0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 32) {
    // 128 rows of 4 words: half a word pair per thread
    for (int t = threadIdx.x; t < 512; t += 256) {
      const bool isx = t < 256;
      const int r = (t & 255) >> 2, w = t & 3;
      const int64_t row = (isx ? m0 : n0) + r;
      uint32_t word = 0;
      float s = 0.f;
      if (row < (isx ? a.M : a.N)) {
        word = (isx ? a.Xq : a.Wq)[row * (a.K / 8) + k0 / 8 + w];
        const uint8_t* sp = isx ? a.xs : a.ws;
        s = NV ? e4m3_to_float(sp[row * (a.K / 16) + k0 / 16 + w / 2]) : e8m0_to_float(sp[row * (a.K / 32) + k0 / 32]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) (isx ? xt : wt)[w * 8 + j][r] = e2m1_to_float((word >> (4 * j)) & 15u) * s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += xt[k][ty * 4 + i] * wt[k][tx + 16 * j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx + 16 * j;
      if (m < a.M && n < a.N) store_y(a.Y, nullptr, m * a.N + n, acc[i][j], a.out_f32);
    }
}

}  // namespace

unsigned int read_mx_matmul_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_qmm_status, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear && v != 0) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(g_qmm_status, &zero, sizeof(zero));
  }
  return v;
}

}  // namespace qmm

extern "C" qmm_status qmm_matmul_mx(const uint32_t* Xq, const uint8_t* x_scales, const uint32_t* Wq,
                                    const uint8_t* w_scales, int M, int N, int K, int format, void* Y, int out_dtype,
                                    void* stream) {
  using namespace qmm;
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0) return QMM_ERR_SHAPE;
  if (format != QMM_MXFP4 && format != QMM_NVFP4) return QMM_ERR_UNSUPPORTED;
  if (out_dtype != QMM_OUT_BF16 && out_dtype != QMM_OUT_F32) return QMM_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return QMM_OK;
  const size_t esize = out_dtype == QMM_OUT_F32 ? 4 : 2;
  if (Y == nullptr) return QMM_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(Y) % esize) return QMM_ERR_ALIGN;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (K == 0)
    return static_cast<qmm_status>(
        finish_call(cudaMemsetAsync(Y, 0, static_cast<size_t>(M) * static_cast<size_t>(N) * esize, st)));
  if (Xq == nullptr || Wq == nullptr || x_scales == nullptr || w_scales == nullptr) return QMM_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(Xq) | reinterpret_cast<uintptr_t>(Wq)) & 15) return QMM_ERR_ALIGN;
  const MxMatmulArgs a{Xq, x_scales, Wq, w_scales, Y, M, N, K, out_dtype == QMM_OUT_F32};
  if ((M + 63) / 64 > 65535) return QMM_ERR_SHAPE;
  const dim3 grid((N + 63) / 64, (M + 63) / 64);
  const cudaError_t e = format == QMM_NVFP4 ? launch_dependent(mx_matmul_kernel<true>, grid, 256, 0, st, a)
                                            : launch_dependent(mx_matmul_kernel<false>, grid, 256, 0, st, a);
  return static_cast<qmm_status>(finish_call(e));
}
