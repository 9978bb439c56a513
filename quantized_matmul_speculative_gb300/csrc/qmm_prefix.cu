// Attention of a batch whose sequences share a long prefix (qmm_shared_prefix_attention,
// include/qmm.h).
//
// A CTA takes one row (sequence, new row, query head) and one share of its tokens: a
// slice of the prefix, or (the last share) the sequence's own tokens.  It leaves maximum,
// sum and unnormalised output in the workspace; a second kernel joins a row's shares.
#include <cmath>

#include "qmm_cache.cuh"

namespace qmm {
namespace {

constexpr int kShares = 9;  // of a row: eight of the prefix, one of its own tokens
constexpr int kPrefixThreads = 128, kMaxDim = 256;

struct PrefixArgs {
  qmm_paged_cache c;
  const int32_t* prefix;
  int prefix_len, pages;
  const uint16_t* q;
  int64_t q_ld;
  int B, M, Hq, G;
  const int32_t* q_lens;
  float scale;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;   // [rows][kShares][D]
  float2* part_ml;  // [rows][kShares]
};

// Tokens of sequence b with the prefix (0: it is empty), and its new rows; false where the rows are not behind the prefix.
__device__ __forceinline__ bool sequence(const PrefixArgs& a, int b, int& own, int& m) {
  const int n = a.c.lengths[b], cap = a.c.max_pages * a.c.page_size;
  m = new_rows(a.q_lens, b, a.M);
  own = n - a.prefix_len;
  if (n == 0 || m == 0) return false;
  if (own < m || own > cap) {
    bad_page();
    return false;
  }
  return true;
}

__device__ __forceinline__ float element(const qmm_paged_cache& c, const void* base, int64_t at) {
  return c.dtype == QMM_KV_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at])
                                : e4m3_to_float(static_cast<const uint8_t*>(base)[at]);
}

__global__ void __launch_bounds__(kPrefixThreads) prefix_share_kernel(const PrefixArgs a) {
  __shared__ float q[kMaxDim], s_p[4], s_m[4];
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x, share = blockIdx.y, D = a.c.head_dim;
  const int hq = row % a.Hq, bi = row / a.Hq, b = bi / a.M, i = bi - b * a.M, h = hq / a.G;
  int own, m;
  const bool real = sequence(a, b, own, m) && i < m;
  const int64_t at_part = static_cast<int64_t>(row) * kShares + share;
  int begin, end;
  if (share < kShares - 1) {
    begin = static_cast<int>(static_cast<int64_t>(a.prefix_len) * share / (kShares - 1));
    end = static_cast<int>(static_cast<int64_t>(a.prefix_len) * (share + 1) / (kShares - 1));
  } else {
    begin = 0;
    end = own - m + i + 1;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (real)
    for (int d = threadIdx.x; d < D; d += kPrefixThreads)
      q[d] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[bi * a.q_ld + static_cast<int64_t>(hq) * D + d]) * a.scale;
  __syncthreads();
  float top = -INFINITY, sum = 0.f, o[2] = {0.f, 0.f};
  if (real)
    for (int j0 = begin; j0 < end; j0 += 4) {
      const int j = j0 + warp;
      float x = -INFINITY;
      if (j < end) {
        const int64_t page = share < kShares - 1 ? a.prefix[j / a.c.page_size] : a.c.block_table[b * a.c.table_stride + j / a.c.page_size];
        const bool ok = page >= 0 && page < a.c.num_pages;
        if (!ok) bad_page();
        const int64_t at = page * a.c.k_page + j % a.c.page_size * a.c.k_token + h * a.c.k_head;
        x = 0.f;
        if (ok)
          for (int d = lane; d < D; d += 32) x = fmaf(q[d], element(a.c, a.c.k, at + d), x);
#pragma unroll
        for (int s = 16; s > 0; s /= 2) x += __shfl_xor_sync(0xffffffffu, x, s);
      }
      if (lane == 0) s_m[warp] = x;
      __syncthreads();
      float t = top;
      for (int w = 0; w < 4; ++w) t = fmaxf(t, s_m[w]);
      const float ref = t == -INFINITY ? 0.f : t, f = expf(top - ref);
      if (lane == 0) s_p[warp] = expf(x - ref);
      __syncthreads();
      top = t;
      sum *= f;
      o[0] *= f;
      o[1] *= f;
      for (int w = 0; w < 4 && j0 + w < end; ++w) {
        const int jj = j0 + w;
        sum += s_p[w];
        const int64_t page = share < kShares - 1 ? a.prefix[jj / a.c.page_size] : a.c.block_table[b * a.c.table_stride + jj / a.c.page_size];
        if (page < 0 || page >= a.c.num_pages) continue;
        const int64_t at = page * a.c.v_page + jj % a.c.page_size * a.c.v_token + h * a.c.v_head;
        for (int x2 = 0; x2 < 2; ++x2) {
          const int d = threadIdx.x + x2 * kPrefixThreads;
          if (d < D) o[x2] = fmaf(s_p[w], element(a.c, a.c.v, at + d), o[x2]);
        }
      }
    }
  for (int x2 = 0; x2 < 2; ++x2) {
    const int d = threadIdx.x + x2 * kPrefixThreads;
    if (d < D) a.part_o[at_part * D + d] = o[x2];
  }
  if (threadIdx.x == 0) a.part_ml[at_part] = make_float2(top, sum);
}

__global__ void __launch_bounds__(kPrefixThreads) prefix_join_kernel(const PrefixArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x, D = a.c.head_dim;
  float top = -INFINITY, sum = 0.f;
  for (int s = 0; s < kShares; ++s) top = fmaxf(top, a.part_ml[static_cast<int64_t>(row) * kShares + s].x);
  const float ref = top == -INFINITY ? 0.f : top;
  for (int s = 0; s < kShares; ++s) {
    const float2 ml = a.part_ml[static_cast<int64_t>(row) * kShares + s];
    sum += ml.y * expf(ml.x - ref);
  }
  const float v = a.c.dtype == QMM_KV_BF16 ? 1.f : a.c.v_scale;
  for (int d = threadIdx.x; d < D; d += kPrefixThreads) {
    float o = 0.f;
    for (int s = 0; s < kShares; ++s) {
      const float2 ml = a.part_ml[static_cast<int64_t>(row) * kShares + s];
      if (ml.y != 0.f) o += a.part_o[(static_cast<int64_t>(row) * kShares + s) * D + d] * expf(ml.x - ref);
    }
    a.out[static_cast<int64_t>(row) * D + d] = __float2bfloat16_rn(sum != 0.f ? o * v / sum : 0.f);
  }
  if (threadIdx.x == 0 && a.lse != nullptr) a.lse[row] = sum != 0.f ? ref + logf(sum) : -INFINITY;
}

}  // namespace

unsigned int read_prefix_status(int clear) { return read_unit_status(clear); }

}  // namespace qmm

extern "C" {

size_t qmm_shared_prefix_attention_workspace(int B, int M, int q_heads, int heads, int head_dim) {
  if (B <= 0 || M <= 0 || M > 16 || heads <= 0 || q_heads <= 0 || q_heads % heads != 0 || q_heads > 65535 || head_dim <= 0) return 0;
  return static_cast<size_t>(B) * M * q_heads * qmm::kShares * (head_dim * 4 + 8);
}

qmm_status qmm_shared_prefix_attention(const qmm_paged_cache* cache, const int32_t* prefix_pages, int num_prefix_pages, const void* q,
                                       int64_t q_ld, int B, int M, int q_heads, const int32_t* q_lens, float scale, void* out,
                                       float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace qmm;
  const qmm_status rc = check_cache(cache, B, M, 16);
  if (rc != QMM_OK) return rc;
  if (q_heads < 1 || q_heads > 65535 || q_heads % cache->heads != 0 || q_heads / cache->heads > 1024 || num_prefix_pages < 0 ||
      q_ld < static_cast<int64_t>(q_heads) * cache->head_dim ||
      (static_cast<int64_t>(num_prefix_pages) + cache->max_pages) * cache->page_size > 0x7fffffff ||
      static_cast<int64_t>(B) * M * q_heads > 0x7fffffff)
    return QMM_ERR_SHAPE;
  const bool e8 = cache->dtype == QMM_KV_E4M3;
  const float s = scale * (e8 ? cache->k_scale : 1.f);
  if (!std::isfinite(s)) return QMM_ERR_UNSUPPORTED;
  if (B == 0 || M == 0) return QMM_OK;
  if (q == nullptr || out == nullptr || workspace == nullptr) return QMM_ERR_NULL;
  if (num_prefix_pages > 0 && (prefix_pages == nullptr || cache->k == nullptr || cache->v == nullptr)) return QMM_ERR_NULL;
  if (misaligned(reinterpret_cast<intptr_t>(q), 16) || misaligned(reinterpret_cast<intptr_t>(out), 16) || misaligned(q_ld, 8) ||
      misaligned(reinterpret_cast<intptr_t>(lse), 4) || misaligned(reinterpret_cast<intptr_t>(q_lens), 4) ||
      misaligned(reinterpret_cast<intptr_t>(prefix_pages), 4) || misaligned(reinterpret_cast<intptr_t>(workspace), 16))
    return QMM_ERR_ALIGN;
  if (workspace_bytes < qmm_shared_prefix_attention_workspace(B, M, q_heads, cache->heads, cache->head_dim)) return QMM_ERR_SHAPE;
  PrefixArgs a = {};
  a.c = *cache;
  a.prefix = prefix_pages;
  a.pages = num_prefix_pages;
  a.prefix_len = num_prefix_pages * cache->page_size;
  a.q = static_cast<const uint16_t*>(q);
  a.q_ld = q_ld;
  a.B = B;
  a.M = M;
  a.Hq = q_heads;
  a.G = q_heads / cache->heads;
  a.q_lens = q_lens;
  a.scale = s;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  const int rows = B * M * q_heads;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<int64_t>(rows) * kShares * cache->head_dim);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_dependent(prefix_share_kernel, dim3(rows, kShares), kPrefixThreads, 0, st, a);
  if (e == cudaSuccess) e = launch_dependent(prefix_join_kernel, dim3(rows), kPrefixThreads, 0, st, a);
  return static_cast<qmm_status>(finish_call(e));
}

}  // extern "C"
