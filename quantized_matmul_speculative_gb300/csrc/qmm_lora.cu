// Low-rank adapters of many requests beside a shared projection (qmm_lora_add,
// include/qmm.h): Y[t] = base[t] + scale[a] B[a] (A[a] X[t]), a = adapters[t].
//
// A CTA takes a row: its warps compute the R inner products, its threads the columns.
#include <cmath>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kLoraThreads = 256;
constexpr int kMaxRank = 128;

struct LoraArgs {
  const void* base;
  const uint16_t* x;
  const uint16_t *A, *B;
  const int32_t* ids;
  const float* scales;
  void* y;
  int64_t base_ld, x_ld, y_ld;
  int T, N, K, R, L, f32;
};

__device__ __forceinline__ void eight(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

__global__ void __launch_bounds__(kLoraThreads) lora_kernel(const LoraArgs a) {
  __shared__ float h[kMaxRank];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int id = a.ids[t];
  if (id >= a.L) {
    if (threadIdx.x == 0) atomicOr(&g_qmm_status, kStatusBadGather);
    id = -1;
  }
  if (id >= 0) {
    const float scale = a.scales != nullptr ? a.scales[id] : 1.f;
    for (int r = warp; r < a.R; r += kLoraThreads / 32) {
      const uint16_t* const w = a.A + (static_cast<int64_t>(id) * a.R + r) * a.K;
      float s = 0.f;
      for (int k = lane * 8; k < a.K; k += 256) {
        float x[8], v[8];
        eight(*reinterpret_cast<const uint4*>(a.x + t * a.x_ld + k), x);
        eight(*reinterpret_cast<const uint4*>(w + k), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x[i], v[i], s);
      }
#pragma unroll
      for (int i = 16; i > 0; i /= 2) s += __shfl_xor_sync(0xffffffffu, s, i);
      if (lane == 0) h[r] = s * scale;
    }
  }
  __syncthreads();
  for (int n = threadIdx.x; n < a.N; n += kLoraThreads) {
    const float b = a.f32 ? static_cast<const float*>(a.base)[t * a.base_ld + n]
                          : __bfloat162float(static_cast<const __nv_bfloat16*>(a.base)[t * a.base_ld + n]);
    float s = 0.f;
    if (id >= 0)
      for (int r = 0; r < a.R; r += 8) {
        float v[8];
        eight(*reinterpret_cast<const uint4*>(a.B + (static_cast<int64_t>(id) * a.N + n) * a.R + r), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(v[i], h[r + i], s);
      }
    // (a row without an adapter stays as it is, bit for bit)
    if (a.f32) static_cast<float*>(a.y)[t * a.y_ld + n] = id >= 0 ? b + s : b;
    else static_cast<__nv_bfloat16*>(a.y)[t * a.y_ld + n] =
        id >= 0 ? __float2bfloat16_rn(b + s) : static_cast<const __nv_bfloat16*>(a.base)[t * a.base_ld + n];
  }
}

}  // namespace

unsigned int read_lora_status(int clear) { return read_unit_status(clear); }

}  // namespace qmm

extern "C" {

size_t qmm_lora_workspace(int T, int L) {
  if (T <= 0 || L <= 0) return 0;
  return 16;
}

qmm_status qmm_lora_add(const void* base, int64_t base_ld, const void* X, int64_t x_ld, const void* A, const void* Bm,
                        const int32_t* adapters, const float* scales, int T, int N, int K, int R, int L, void* Y, int64_t y_ld,
                        int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace qmm;
  if (T < 0 || N < 0 || K < 0 || L < 0 || R < 8 || R > kMaxRank || R % 8 != 0 || K % 8 != 0 || N > (1 << 30) || K > (1 << 30) ||
      base_ld < N || y_ld < N || x_ld < K)
    return QMM_ERR_SHAPE;
  if (out_dtype != QMM_OUT_BF16 && out_dtype != QMM_OUT_F32) return QMM_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return QMM_OK;
  if (base == nullptr || Y == nullptr || adapters == nullptr || (K > 0 && X == nullptr) ||
      (L > 0 && (Bm == nullptr || (K > 0 && A == nullptr))))
    return QMM_ERR_NULL;
  const uintptr_t es = out_dtype == QMM_OUT_F32 ? 4 : 2;
  if (((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(Y)) % es) ||
      (K > 0 && (((reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(A)) % 16) || x_ld % 8 != 0)) ||
      reinterpret_cast<uintptr_t>(Bm) % 16 || ((reinterpret_cast<uintptr_t>(adapters) | reinterpret_cast<uintptr_t>(scales)) % 4))
    return QMM_ERR_ALIGN;
  const size_t need = qmm_lora_workspace(T, L);
  if (need > 0) {
    if (workspace == nullptr) return QMM_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(workspace) % 16) return QMM_ERR_ALIGN;
    if (workspace_bytes < need) return QMM_ERR_SHAPE;
  }
  LoraArgs a = {};
  a.base = base;
  a.x = static_cast<const uint16_t*>(X);
  a.A = static_cast<const uint16_t*>(A);
  a.B = static_cast<const uint16_t*>(Bm);
  a.ids = adapters;
  a.scales = scales;
  a.y = Y;
  a.base_ld = base_ld;
  a.x_ld = x_ld;
  a.y_ld = y_ld;
  a.T = T;
  a.N = N;
  a.K = K;
  a.R = R;
  a.L = L;
  a.f32 = out_dtype == QMM_OUT_F32;
  return static_cast<qmm_status>(finish_call(
      launch_dependent(lora_kernel, dim3(static_cast<unsigned>(T)), kLoraThreads, 0, static_cast<cudaStream_t>(stream), a)));
}

}  // extern "C"
