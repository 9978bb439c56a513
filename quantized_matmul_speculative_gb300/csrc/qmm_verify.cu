// Verification of drafted tokens (qmm_verify_draft, include/qmm.h).
#include <cmath>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

struct VerifyArgs {
  const void* logits;
  int64_t batch_stride, row_stride;
  const int32_t* draft;
  const float* q;
  const float* u;
  const float* noise;
  const float* temperature;
  const int32_t* draft_lens;
  int B, k, V;
  int32_t* tokens;
  int32_t* accepted;
};

// (value, index) with the larger value, the lower index of equals.
__device__ __forceinline__ void best_of(float& v, int& i, float v2, int i2) {
  if (v2 > v || (v2 == v && i2 < i)) {
    v = v2;
    i = i2;
  }
}

constexpr int kThreads = 512;

// The CTA's best (value, index); every thread gets it.
__device__ __forceinline__ void block_best(float& v, int& i, float* sv, int* si) {
#pragma unroll
  for (int s = 16; s > 0; s /= 2)
    best_of(v, i, __shfl_xor_sync(0xffffffffu, v, s), __shfl_xor_sync(0xffffffffu, i, s));
  __syncthreads();
  if (threadIdx.x % 32 == 0) {
    sv[threadIdx.x / 32] = v;
    si[threadIdx.x / 32] = i;
  }
  __syncthreads();
  v = sv[0];
  i = si[0];
  for (int w = 1; w < kThreads / 32; ++w) best_of(v, i, sv[w], si[w]);
}

// One CTA per sequence: row by row the largest logit (with its lowest index)
// and the sum of exponentials, until a draft is refused.
template <bool F32>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
  __shared__ float sv[kThreads / 32];
  __shared__ int si[kThreads / 32];
  griddep_wait();
  const int b = blockIdx.x;
  const float T = a.temperature[b];
  const bool greedy = !(T > 0.f);
  int drafts = a.draft_lens != nullptr ? a.draft_lens[b] : a.k;
  drafts = drafts < 0 ? 0 : drafts > a.k ? a.k : drafts;
  int n = 0, token = 0;
  for (;; ++n) {
    const int64_t off = b * a.batch_stride + n * a.row_stride;
    auto logit = [&](int v) {
      const float x = F32 ? static_cast<const float*>(a.logits)[off + v]
                          : bf16_lo(static_cast<const uint16_t*>(a.logits)[off + v]);
      return x == x ? x : -INFINITY;
    };
    float top = -INFINITY;
    int at = 0x7fffffff;
    for (int v = threadIdx.x; v < a.V; v += kThreads) best_of(top, at, logit(v), v);
    block_best(top, at, sv, si);
    token = at;
    const int d = n < drafts ? a.draft[b * a.k + n] : -1;
    const bool usable = fabsf(top) <= 3.4028235e38f;
    if (greedy || !usable) {
      if (n < drafts && usable && d == at) continue;
      break;
    }
    float sum = 0.f;
    for (int v = threadIdx.x; v < a.V; v += kThreads) sum += expf((logit(v) - top) / T);
#pragma unroll
    for (int s = 16; s > 0; s /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sv[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) sum += sv[w];
    const float* q = a.q != nullptr && n < drafts ? a.q + (static_cast<int64_t>(b) * a.k + n) * a.V : nullptr;
    const bool valid = d >= 0 && d < a.V;
    if (n < drafts && valid) {
      const float qd = a.q != nullptr ? q[d] : 1.f;
      if (a.u[b * a.k + n] * qd < expf((logit(d) - top) / T) / sum) continue;
    }
    float best = -1.f, plain = -1.f;
    int besti = 0x7fffffff, plaini = 0x7fffffff;
    const float* e = a.noise + static_cast<int64_t>(b) * a.V;
    for (int v = threadIdx.x; v < a.V; v += kThreads) {
      const float p = expf((logit(v) - top) / T) / sum;
      const float w = n >= drafts ? p : q != nullptr ? p - q[v] : v == d ? 0.f : p;
      if (w > 0.f) best_of(best, besti, w / e[v], v);
      best_of(plain, plaini, p > 0.f ? p / e[v] : 0.f, v);
    }
    block_best(best, besti, sv, si);
    block_best(plain, plaini, sv, si);
    token = best > 0.f ? besti : plaini;
    break;
  }
  for (int j = threadIdx.x; j <= a.k; j += kThreads)
    a.tokens[b * (a.k + 1) + j] = j < n ? a.draft[b * a.k + j] : j == n ? token : -1;
  if (threadIdx.x == 0) a.accepted[b] = n;
}

}  // namespace
}  // namespace qmm

extern "C" qmm_status qmm_verify_draft(const void* logits, int logits_dtype, int64_t batch_stride, int64_t row_stride,
                                       const int32_t* draft_tokens, const float* draft_probs, const float* uniform,
                                       const float* noise, const float* temperature, const int32_t* draft_lens, int B,
                                       int k, int V, int32_t* tokens, int32_t* accepted, void* stream) {
  using namespace qmm;
  if (logits_dtype != QMM_OUT_BF16 && logits_dtype != QMM_OUT_F32) return QMM_ERR_UNSUPPORTED;
  if (B < 0 || k < 0 || k > 31 || V < 1 || row_stride < V || batch_stride < 0) return QMM_ERR_SHAPE;
  if (B == 0) return QMM_OK;
  if (logits == nullptr || noise == nullptr || temperature == nullptr || tokens == nullptr || accepted == nullptr)
    return QMM_ERR_NULL;
  if (k > 0 && (draft_tokens == nullptr || uniform == nullptr)) return QMM_ERR_NULL;
  const uintptr_t esize = logits_dtype == QMM_OUT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % esize ||
      ((reinterpret_cast<uintptr_t>(draft_tokens) | reinterpret_cast<uintptr_t>(draft_probs) |
        reinterpret_cast<uintptr_t>(uniform) | reinterpret_cast<uintptr_t>(noise) |
        reinterpret_cast<uintptr_t>(temperature) | reinterpret_cast<uintptr_t>(draft_lens) |
        reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(accepted)) & 3))
    return QMM_ERR_ALIGN;
  const VerifyArgs a{logits, batch_stride, row_stride, draft_tokens, draft_probs, uniform, noise, temperature, draft_lens,
                     B, k, V, tokens, accepted};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == QMM_OUT_F32 ? launch_dependent(verify_kernel<true>, dim3(B), kThreads, 0, st, a)
                                                    : launch_dependent(verify_kernel<false>, dim3(B), kThreads, 0, st, a);
  return static_cast<qmm_status>(finish_call(e));
}
