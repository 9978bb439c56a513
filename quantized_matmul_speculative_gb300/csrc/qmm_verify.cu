// Verification of drafted tokens (qmm_verify_draft, include/qmm.h).
#include <climits>
#include <cmath>
#include <type_traits>

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
  int cluster;  // CTAs of a sequence
  int round;    // rows between two exchanges
};

// (value, index) with the larger value, the lower index of equals.
__device__ __forceinline__ void best_of(float& v, int& i, float v2, int i2) {
  if (v2 > v || (v2 == v && i2 < i)) {
    v = v2;
    i = i2;
  }
}
__device__ __forceinline__ void warp_best(float& v, int& i) {
#pragma unroll
  for (int s = 16; s > 0; s /= 2) best_of(v, i, __shfl_xor_sync(0xffffffffu, v, s), __shfl_xor_sync(0xffffffffu, i, s));
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
// The whole 16-byte blocks of [p, p + bytes), or of its first MB, on their way to L2.
__device__ __forceinline__ void prefetch_l2_range(const void* p, int64_t bytes) {
  const uintptr_t from = (reinterpret_cast<uintptr_t>(p) + 15) & ~static_cast<uintptr_t>(15);
  const uintptr_t to = (reinterpret_cast<uintptr_t>(p) + bytes) & ~static_cast<uintptr_t>(15);
  if (from < to)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(static_cast<uint32_t>(to - from < (1 << 20) ? to - from : 1 << 20)) : "memory");
}
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxRows = 32, kMaxCluster = 16;

struct Partial {
  float m;  // largest logit of this CTA's part of a row
  float s;  // sum of exponentials relative to it (greedy: unused)
  int at;   // its lowest index (greedy)
};

// The lanes' partials joined, in every lane: the best of greedy ones, else the
// largest maximum and the sum relative to it.
__device__ __forceinline__ void warp_join(Partial& p, bool greedy, float c) {
  if (greedy) {
    warp_best(p.m, p.at);
    return;
  }
  float t = p.m;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
  p.s *= ex2((p.m - base_of(t)) * c);
  p.m = t;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) p.s += __shfl_xor_sync(0xffffffffu, p.s, d);
}

__device__ __forceinline__ int ld_dsmem_i32(const int* p, uint32_t rank) {
  return __float_as_int(ld_dsmem_f32(reinterpret_cast<const float*>(p), rank));
}

// One cluster per sequence; a CTA of it takes a share of the vocabulary of
// every row.  Rounds of a.round rows: each CTA's maximum and sum of
// exponentials of its share (one pass, running maximum per thread), exchanged
// through distributed shared memory; every CTA then finds the same first
// refusal.  Rows past the round of the first refusal are never read.  Then one
// pass over the refused (or last) row, its draft probabilities and the noise
// for the next token.  Sums are added in a fixed order: results do not depend
// on timing.
//
// What bounds it: the bytes of the rows read, where there are many sequences
// (rounds of two rows, several clusters an SM so that one's exchange overlaps
// another's reads); the latency of its two exchanges, where there are few (all
// rows in one round).  The noise is fetched into L2 meanwhile (fetching the next
// row too gains nothing).  Spills in its loops cost most: joining a row's partials
// by a thread, not a warp, took 6 us more, and 8 elements at a time, not 4, in the
// last pass 10 us (the bf16 kernel still spills 8 bytes, outside of them).
// 64 sequences x 5 drafts x 128000 fp32 logits: 64 us for 130 MB, of which it needs
// 108 (2.0 TB/s; two CTAs of an SM are resident at once, and the longest sequences
// end alone); 1 x 7 x 32000 bf16: 9.9 us.
template <bool F32>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs a) {
  using T = typename std::conditional<F32, float, uint16_t>::type;
  constexpr int VEC = F32 ? 4 : 8;  // logits of a 16-byte load
  __shared__ Partial warp_part[kMaxRows][kWarps];
  __shared__ Partial part[2][kMaxRows];  // this CTA's, by the round's parity
  __shared__ float s_xd[kMaxRows], s_qd[kMaxRows], s_u[kMaxRows];
  __shared__ int s_d[kMaxRows];
  __shared__ float s_top[kMaxRows], s_sum[kMaxRows];
  __shared__ int s_at[kMaxRows], s_yes[kMaxRows];
  __shared__ float best_v[2][kWarps], cta_v[2];
  __shared__ int best_i[2][kWarps], cta_i[2];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = a.cluster, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int b = blockIdx.x / C;
  const T* const rows = static_cast<const T*>(a.logits) + b * a.batch_stride;
  auto value = [](T x) { return fmaxf(F32 ? static_cast<float>(x) : bf16_lo(x), -INFINITY); };  // NaN: -inf
  const float temp = a.temperature[b];
  const bool greedy = !(temp > 0.f);
  // (finite, so that the largest logit's 0 times it is 0, and not 0, so that -inf times it is -inf)
  const float c = greedy ? 1.f : fminf(fmaxf(1.4426950408889634f / temp, 1e-30f), 3e38f);
  int drafts = a.draft_lens != nullptr ? a.draft_lens[b] : a.k;
  drafts = drafts < 0 ? 0 : drafts > a.k ? a.k : drafts;
  // draft tid's logit, draft probability and random number: used after the first round
  int my_d = -1;
  float my_u = 0.f, my_x = 0.f, my_q = 1.f;
  if (tid < drafts) {
    const int64_t at = static_cast<int64_t>(b) * a.k + tid;
    my_d = a.draft[at];
    my_u = a.u[at];
    if (my_d < 0 || my_d >= a.V) my_d = -1;
    if (my_d >= 0) my_x = value(rows[tid * a.row_stride + my_d]);
    if (my_d >= 0 && a.q != nullptr) my_q = a.q[at * a.V + my_d];
  }

  // this CTA's elements of the pass for the next token
  const int i0 = static_cast<int>(static_cast<int64_t>(a.V) * rank / C), i1 = static_cast<int>(static_cast<int64_t>(a.V) * (rank + 1) / C);
  const float* const e = a.noise + static_cast<int64_t>(b) * a.V;
  if (!greedy && tid == 0) prefetch_l2_range(e + i0, static_cast<int64_t>(i1 - i0) * 4);

  int n = 0;  // accepted drafts
  for (int r0 = 0, parity = 0;; r0 += a.round, parity ^= 1) {
    const int r1 = min(r0 + a.round, drafts + 1);
    // the warps in groups, a row each, when there are several
    int per = kWarps;  // warps of a row
    while (per > 1 && per * (r1 - r0) > kWarps) per /= 2;
    const int threads = 32 * per, t_row = tid & (threads - 1);
    for (int r = r0 + warp / per; r < r1; r += kWarps / per) {
      const T* const x = rows + r * a.row_stride;
      // elements before the first 16-byte boundary and after the last go to CTA 0
      const int head = min(a.V, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T)));
      const int vecs = (a.V - head) / VEC, tail = head + vecs * VEC;
      const int v0 = static_cast<int>(static_cast<int64_t>(vecs) * rank / C), v1 = static_cast<int>(static_cast<int64_t>(vecs) * (rank + 1) / C);
      const uint4* const xv = reinterpret_cast<const uint4*>(x + head);
      float m = -INFINITY, s = 0.f;
      int at = INT_MAX;
      auto unpack = [&](const uint4& w, float (&f)[VEC]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (F32) {
            f[i] = fmaxf(__uint_as_float(u[i]), -INFINITY);
          } else {
            f[2 * i] = fmaxf(bf16_lo(u[i]), -INFINITY);
            f[2 * i + 1] = fmaxf(bf16_hi(u[i]), -INFINITY);
          }
        }
      };
      // U vectors at a time: their maximum first, so that a thread's sum is rescaled at most once for all
      constexpr int U = 16 / VEC;
      auto take = [&](const uint4* w, int count, int first) {
        float f[U][VEC];
        float top = m;
#pragma unroll
        for (int j = 0; j < U; ++j) {
          if (j < count) unpack(w[j], f[j]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            if (j >= count) f[j][i] = -INFINITY;
            if (greedy) best_of(m, at, f[j][i], head + (first + j * threads) * VEC + i);
            else top = fmaxf(top, f[j][i]);
          }
        }
        if (greedy) return;
        const float base = base_of(top);
        s *= ex2((m - base) * c);
        m = top;
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) s += ex2((f[j][i] - base) * c);
      };
      int v = v0 + t_row;
      for (; v + 3 * threads < v1; v += 4 * threads) {
        uint4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = xv[v + j * threads];
#pragma unroll
        for (int j = 0; j < 4; j += U) take(w + j, U, v + j * threads);
      }
      if (v < v1) {
        uint4 w[4];
        int count = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (v + j * threads < v1) {
            w[j] = xv[v + j * threads];
            count = j + 1;
          }
#pragma unroll
        for (int j = 0; j < 4; j += U) take(w + j, count - j, v + j * threads);
      }
      if (rank == 0) {
        auto one = [&](int i) {
          const float f = value(x[i]);
          if (greedy) {
            best_of(m, at, f, i);
          } else {
            const float t = fmaxf(m, f), base = base_of(t);
            s = s * ex2((m - base) * c) + ex2((f - base) * c);
            m = t;
          }
        };
        if (t_row < head) one(t_row);
        if (tail + t_row < a.V && t_row < VEC) one(tail + t_row);
      }
      Partial p{m, s, at};
      warp_join(p, greedy, c);
      if (lane == 0) warp_part[r - r0][warp & (per - 1)] = p;
    }
    if (r0 == 0 && tid < drafts) s_d[tid] = my_d, s_u[tid] = my_u, s_xd[tid] = my_x, s_qd[tid] = my_q;
    __syncthreads();
    // a warp joins a row's warps
    for (int i = warp; i < r1 - r0; i += kWarps) {
      Partial p = lane < per ? warp_part[i][lane] : Partial{-INFINITY, 0.f, INT_MAX};
      warp_join(p, greedy, c);
      if (lane == 0) part[parity][i] = p;
    }
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    // and its CTAs: every CTA finds the same
    for (int i = warp; i < r1 - r0; i += kWarps) {
      const int r = r0 + i;
      Partial p = part[parity][i];
      if (C > 1) {
        const Partial* const at = &part[parity][i];
        p = Partial{-INFINITY, 0.f, INT_MAX};
        if (lane < C) p = Partial{ld_dsmem_f32(&at->m, lane), ld_dsmem_f32(&at->s, lane), ld_dsmem_i32(&at->at, lane)};
        warp_join(p, greedy, c);
      }
      if (lane != 0) continue;
      const bool usable = fabsf(p.m) <= 3.4028235e38f;
      s_top[r] = p.m;
      s_sum[r] = p.s;
      s_at[r] = p.at;
      bool yes = false;
      if (r < drafts && usable) {
        if (greedy) yes = s_d[r] == p.at;
        else if (s_d[r] >= 0) yes = s_u[r] * s_qd[r] < ex2((s_xd[r] - p.m) * c) / p.s;
      }
      s_yes[r] = yes;
    }
    __syncthreads();
    while (n < r1 && s_yes[n]) ++n;
    if (n < r1) break;  // the last row (n == drafts) never says yes
  }

  // The next token, from row n.
  const bool usable = fabsf(s_top[n]) <= 3.4028235e38f;
  int token = s_at[n];
  if (!greedy) {
    const T* const x = rows + n * a.row_stride;
    const bool refused = n < drafts;
    const float top = base_of(s_top[n]), inv = 1.f / s_sum[n];
    const float* const q = refused && a.q != nullptr && usable ? a.q + (static_cast<int64_t>(b) * a.k + n) * a.V : nullptr;
    const int d = refused && a.q == nullptr ? s_d[n] : -1;
    // largest w / noise, and largest p / noise, which stands in where w is 0 everywhere; of a row without a
    // softmax the largest logit
    float v[2] = {-INFINITY, -INFINITY};
    int at[2] = {INT_MAX, INT_MAX};
    auto look = [&](int i, float f, float qi, float ei) {
      if (!usable) {
        best_of(v[1], at[1], f, i);
        return;
      }
      const float p = ex2((f - top) * c) * inv;
      const float w = q != nullptr ? p - qi : i == d ? 0.f : p;
      // (a noise that is NaN or negative makes 0 of any weight, so that some token is always found)
      if (w > 0.f) best_of(v[0], at[0], fmaxf(__fdiv_rn(w, ei), 0.f), i);
      if (q != nullptr || d >= 0) best_of(v[1], at[1], p > 0.f ? fmaxf(__fdiv_rn(p, ei), 0.f) : 0.f, i);
    };
    for (int i = i0 + tid; i < i1; i += 4 * kThreads) {
      float f[4], qi[4], ei[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at_j = min(i + j * kThreads, i1 - 1);  // (again what the last one reads)
        f[j] = value(x[at_j]);
        qi[j] = q != nullptr ? q[at_j] : 0.f;
        ei[j] = e[at_j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) look(min(i + j * kThreads, i1 - 1), f[j], qi[j], ei[j]);
    }
    if (usable && q == nullptr && d < 0) v[1] = v[0], at[1] = at[0];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      warp_best(v[h], at[h]);
      if (lane == 0) best_v[h][warp] = v[h], best_i[h][warp] = at[h];
    }
    __syncthreads();
    if (warp < 2) {
      float bv = lane < kWarps ? best_v[warp][lane] : -INFINITY;
      int bi = lane < kWarps ? best_i[warp][lane] : INT_MAX;
      warp_best(bv, bi);
      if (lane == 0) cta_v[warp] = bv, cta_i[warp] = bi;
    }
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    if (rank == 0 && warp == 0) {
      float bv[2];
      int bi[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bv[h] = lane < C ? (C > 1 ? ld_dsmem_f32(&cta_v[h], lane) : cta_v[h]) : -INFINITY;
        bi[h] = lane < C ? (C > 1 ? ld_dsmem_i32(&cta_i[h], lane) : cta_i[h]) : INT_MAX;
        warp_best(bv[h], bi[h]);
      }
      token = usable && bv[0] > 0.f ? bi[0] : bi[1];
    }
  }
  if (rank == 0 && warp == 0) {
    for (int j = lane; j <= a.k; j += 32)
      a.tokens[static_cast<int64_t>(b) * (a.k + 1) + j] = j < n ? a.draft[static_cast<int64_t>(b) * a.k + j] : j == n ? token : -1;
    if (lane == 0) a.accepted[b] = n;
  }
  if (C > 1) cluster_sync_all();  // nobody leaves while its shared memory is read
}

template <bool F32>
cudaError_t launch_verify(VerifyArgs a, cudaStream_t stream) {
  if (injected_launch_failure()) return cudaErrorLaunchFailure;
  // CTAs of a cluster: two to four launched for an SM over all sequences, of which
  // two are resident (64 x 5 x 128000: 66.4 us; one to two 68.1, four to eight
  // 89.9), and no more than one for every 2048 logits of a row.
  const int sms = device_sm_count();
  a.cluster = 1;
  while (a.cluster < kMaxCluster && static_cast<int64_t>(a.B) * a.cluster <= 2 * sms && a.V > a.cluster * 2048) a.cluster *= 2;
  // All rows in one round while reading them takes less than the exchanges saved (about 16 MB: 2.5 us), else two:
  // 64 x 5 x 128000 takes 63.3 us, and 66.1, 66.1, 73.9 with one, three, all.
  a.round = static_cast<int64_t>(a.B) * (a.k + 1) * a.V * (F32 ? 4 : 2) <= (16 << 20) ? a.k + 1 : 2;
  auto kern = verify_kernel<F32>;
  static std::atomic<uint64_t> ready{0};
  uint64_t bit;
  if (first_on_device(ready, &bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace
}  // namespace qmm

extern "C" qmm_status qmm_verify_draft(const void* logits, int logits_dtype, int64_t batch_stride, int64_t row_stride,
                                       const int32_t* draft_tokens, const float* draft_probs, const float* uniform,
                                       const float* noise, const float* temperature, const int32_t* draft_lens, int B,
                                       int k, int V, int32_t* tokens, int32_t* accepted, void* stream) {
  using namespace qmm;
  if (logits_dtype != QMM_OUT_BF16 && logits_dtype != QMM_OUT_F32) return QMM_ERR_UNSUPPORTED;
  if (B < 0 || B > INT_MAX / 16 || k < 0 || k > 31 || V < 1 || V > (1 << 30) || row_stride < V || batch_stride < 0) return QMM_ERR_SHAPE;
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
                     B, k, V, tokens, accepted, 1, 1};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == QMM_OUT_F32 ? launch_verify<true>(a, st) : launch_verify<false>(a, st);
  return static_cast<qmm_status>(finish_call(e));
}
