// Paged key-value cache: append of new rows and attention over it
// (qmm_kv_append, qmm_paged_attention; definitions in include/qmm.h).
#include <cmath>

#include "qmm_paged.cuh"

namespace qmm {

// Checks that append and attention share; QMM_OK if there is work to launch.
qmm_status check_cache(const qmm_paged_cache* c, int B, int M, int max_rows) {
  if (c == nullptr) return QMM_ERR_NULL;
  if (c->dtype != QMM_KV_BF16 && c->dtype != QMM_KV_E4M3) return QMM_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QMM_ERR_UNSUPPORTED;
  if (B < 0 || B > 65535 || M < 0 || M > max_rows || c->heads < 1 || c->heads > 4096 || c->page_size < 1 || c->max_pages < 0 ||
      c->num_pages < 0 || c->num_pages > 0x7fffffff || static_cast<int64_t>(c->max_pages) * c->page_size > 0x7fffffff)
    return QMM_ERR_SHAPE;
  if (c->table_stride < c->max_pages) return QMM_ERR_SHAPE;
  if (c->dtype == QMM_KV_E4M3 && !(c->k_scale > 0.f && c->v_scale > 0.f && c->k_scale < INFINITY && c->v_scale < INFINITY))
    return QMM_ERR_UNSUPPORTED;
  if (B == 0 || M == 0) return QMM_OK;
  if (c->lengths == nullptr) return QMM_ERR_NULL;
  if (c->max_pages > 0 && (c->k == nullptr || c->v == nullptr || c->block_table == nullptr)) return QMM_ERR_NULL;
  const int64_t per16 = c->dtype == QMM_KV_BF16 ? 8 : 16;
  if (misaligned(reinterpret_cast<intptr_t>(c->k), 16) || misaligned(reinterpret_cast<intptr_t>(c->v), 16) ||
      misaligned(c->k_page, per16) || misaligned(c->k_token, per16) || misaligned(c->k_head, per16) ||
      misaligned(c->v_page, per16) || misaligned(c->v_token, per16) || misaligned(c->v_head, per16) ||
      misaligned(reinterpret_cast<intptr_t>(c->lengths), 4) || misaligned(reinterpret_cast<intptr_t>(c->block_table), 4))
    return QMM_ERR_ALIGN;
  return QMM_OK;
}

namespace {

// cache[page(pos), pos mod page_size, h] = x, as E4M3 e4m3(x / scale).  A copy
// of 2 + 2 (or 2 + 1) bytes an element, bound by the chain length -> table ->
// store at small sizes: one thread per 8 elements of one row's key and value,
// both on their way before the chain starts (a thread each for key and value:
// 6.4 us for the larger case, as the index arithmetic is done twice).  4 x 5 rows
// of 8 x 128 in bf16: 1.7 us; 128 x 16 as E4M3: 4.9 us, 2.6 TB/s.
__global__ void __launch_bounds__(256)
kv_append_kernel(const qmm_paged_cache c, const uint16_t* kn, int64_t k_ld, const uint16_t* vn, int64_t v_ld, int B, int M,
                 const int32_t* q_lens) {
  griddep_wait();
  const int per_head = c.head_dim / 8, per_row = c.heads * per_head;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (t >= static_cast<int64_t>(B) * M * per_row) return;
  const int64_t row = t >> 31 ? t / per_row : static_cast<uint32_t>(t) / static_cast<uint32_t>(per_row);  // below 2^20
  const int chunk = static_cast<int>(t - row * per_row);
  const uint4 x[2] = {*reinterpret_cast<const uint4*>(kn + row * k_ld + chunk * 8),
                      *reinterpret_cast<const uint4*>(vn + row * v_ld + chunk * 8)};
  const int b = static_cast<int>(row) / M, i = static_cast<int>(row) - b * M;
  const int m = new_rows(q_lens, b, M);
  const int pos = seq_length(c, b) - m + i;
  if (i >= m || pos < 0) return;
  const int64_t page = token_page(c, b, pos);
  if (page < 0) return;
  const int h = chunk / per_head, d = (chunk - h * per_head) * 8, slot = pos % c.page_size;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const int64_t at = page * (kv ? c.v_page : c.k_page) + slot * (kv ? c.v_token : c.k_token) +
                       h * (kv ? c.v_head : c.k_head) + d;
    if (c.dtype == QMM_KV_BF16) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv ? c.v : c.k) + at) = x[kv];
    } else {
      const float s = kv ? c.v_scale : c.k_scale;
      const uint32_t w[4] = {x[kv].x, x[kv].y, x[kv].z, x[kv].w};
      uint32_t o[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j / 2] |= cvt_e4m3(__fdiv_rn(bf16_lo(w[j]), s), __fdiv_rn(bf16_hi(w[j]), s)) << (16 * (j & 1));
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(kv ? c.v : c.k) + at) = make_uint2(o[0], o[1]);
    }
  }
}

}  // namespace

extern template cudaError_t launch_attention<64, false>(AttentionArgs, bool, int, cudaStream_t);
extern template unsigned int read_attention_status<64, false>(int);
extern template cudaError_t launch_attention<64, true>(AttentionArgs, bool, int, cudaStream_t);
extern template unsigned int read_attention_status<64, true>(int);
extern template cudaError_t launch_attention<128, false>(AttentionArgs, bool, int, cudaStream_t);
extern template unsigned int read_attention_status<128, false>(int);
extern template cudaError_t launch_attention<128, true>(AttentionArgs, bool, int, cudaStream_t);
extern template unsigned int read_attention_status<128, true>(int);
extern template cudaError_t launch_attention<256, false>(AttentionArgs, bool, int, cudaStream_t);
extern template unsigned int read_attention_status<256, false>(int);
extern template cudaError_t launch_attention<256, true>(AttentionArgs, bool, int, cudaStream_t);
extern template unsigned int read_attention_status<256, true>(int);

unsigned int read_paged_status(int clear) {
  return read_unit_status(clear) | read_attention_status<64, false>(clear) | read_attention_status<128, false>(clear) |
         read_attention_status<256, false>(clear) | read_attention_status<64, true>(clear) | read_attention_status<128, true>(clear) |
         read_attention_status<256, true>(clear);
}

qmm_status run_attention(const qmm_paged_cache* cache, const void* q, int64_t q_ld, int B, int M, int q_heads,
                         const int32_t* q_lens, float scale, int window, int sinks, void* out, float* out32, float* lse, int skip,
                         void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const qmm_status rc = check_cache(cache, B, M, 16);
  if (rc != QMM_OK) return rc;
  if (q_heads < 1 || q_heads > 65535 || q_heads % cache->heads != 0 || q_heads / cache->heads > 1024 || window < 0 || sinks < 0 ||
      q_ld < static_cast<int64_t>(q_heads) * cache->head_dim)
    return QMM_ERR_SHAPE;
  const bool e8 = cache->dtype == QMM_KV_E4M3;
  const float scale_log2 = scale * 1.4426950408889634f * (e8 ? cache->k_scale : 1.f);
  if (!std::isfinite(scale_log2)) return QMM_ERR_UNSUPPORTED;
  if (B == 0 || M == 0) return QMM_OK;
  if (q == nullptr || (out == nullptr && out32 == nullptr)) return QMM_ERR_NULL;
  if (misaligned(reinterpret_cast<intptr_t>(q), 16) || misaligned(reinterpret_cast<intptr_t>(out), 16) ||
      misaligned(q_ld, 8) || misaligned(reinterpret_cast<intptr_t>(lse), 4) ||
      misaligned(reinterpret_cast<intptr_t>(q_lens), 4))
    return QMM_ERR_ALIGN;
  if (workspace == nullptr) return QMM_ERR_NULL;
  if (misaligned(reinterpret_cast<intptr_t>(workspace), 16)) return QMM_ERR_ALIGN;
  AttentionArgs a = {};
  a.inject = injected_short_wait();
  a.wait_ns = a.inject ? 100000ull : kWaitLimitNs;
  a.c = *cache;
  a.q = static_cast<const uint16_t*>(q);
  a.q_ld = q_ld;
  a.B = B;
  a.M = M;
  a.Hq = q_heads;
  a.G = q_heads / cache->heads;
  a.q_lens = q_lens;
  // at least 1e-30: a masked score of -inf stays -inf, and no finite score of use is told from 0 by less
  a.scale_log2 = std::fmax(std::fabs(scale_log2), 1e-30f);
  a.negate = scale < 0.f;
  a.v_scale = e8 ? cache->v_scale : 1.f;
  a.window = window;
  a.sinks = window != 0 ? sinks : 0;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.out32 = out32;
  a.lse = lse;
  a.skip = skip;
  a.RB = attention_row_block(M * a.G, cache->head_dim);
  a.RT = (M * a.G + a.RB - 1) / a.RB;
  a.g_magic = a.G == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + a.G - 1) / a.G);
  // (places of the list of tiles are numbered in 32 bits; a tile holds 16 tokens at least)
  if (static_cast<int64_t>(B) * cache->heads * a.RT * (static_cast<int64_t>(cache->max_pages) * cache->page_size / 16 + 1 + kLead) >
      0x7fffffff)
    return QMM_ERR_SHAPE;
  const int ctas = device_sm_count();
  const size_t workers = static_cast<size_t>(ctas) * kMaxWorkers;
  if (workspace_bytes < attention_workspace(static_cast<int>(workers), a.RB, cache->head_dim)) return QMM_ERR_SHAPE;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + workers * 2 * a.RB * cache->head_dim);
  a.part_seg = reinterpret_cast<int4*>(a.part_ml + workers * 2 * a.RB);
  const bool behind = out32 != nullptr;
  const auto launch = cache->head_dim == 64    ? (behind ? launch_attention<64, true> : launch_attention<64, false>)
                      : cache->head_dim == 128 ? (behind ? launch_attention<128, true> : launch_attention<128, false>)
                                               : (behind ? launch_attention<256, true> : launch_attention<256, false>);
  const cudaError_t e = launch(a, e8, ctas, stream);
  return static_cast<qmm_status>(finish_call(e));
}

}  // namespace qmm

extern "C" {

using namespace qmm;

qmm_status qmm_kv_append(const qmm_paged_cache* cache, const void* k_new, int64_t k_ld, const void* v_new, int64_t v_ld,
                         int B, int M, const int32_t* q_lens, void* stream) {
  const qmm_status rc = check_cache(cache, B, M, 16);
  if (rc != QMM_OK) return rc;
  const int64_t width = static_cast<int64_t>(cache->heads) * cache->head_dim;
  if (k_ld < width || v_ld < width) return QMM_ERR_SHAPE;
  if (B == 0 || M == 0) return QMM_OK;
  if (k_new == nullptr || v_new == nullptr) return QMM_ERR_NULL;
  if (misaligned(reinterpret_cast<intptr_t>(k_new), 16) || misaligned(reinterpret_cast<intptr_t>(v_new), 16) ||
      misaligned(k_ld, 8) || misaligned(v_ld, 8) || misaligned(reinterpret_cast<intptr_t>(q_lens), 4))
    return QMM_ERR_ALIGN;
  const int64_t threads = static_cast<int64_t>(B) * M * (width / 8);
  return static_cast<qmm_status>(finish_call(launch_dependent(
      kv_append_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), 256, 0, static_cast<cudaStream_t>(stream),
      *cache, static_cast<const uint16_t*>(k_new), k_ld, static_cast<const uint16_t*>(v_new), v_ld, B, M, q_lens)));
}

size_t qmm_paged_attention_workspace(int B, int M, int q_heads, int heads, int head_dim) {
  if (B <= 0 || M <= 0 || M > 16 || heads <= 0 || q_heads <= 0 || q_heads % heads != 0 || q_heads > 65535 || head_dim <= 0)
    return 0;
  return attention_workspace(kMaxWorkers * device_sm_count(), attention_row_block(M * (q_heads / heads), head_dim), head_dim);
}

qmm_status qmm_paged_attention(const qmm_paged_cache* cache, const void* q, int64_t q_ld, int B, int M, int q_heads,
                               const int32_t* q_lens, float scale, int window, int sinks, void* out, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream) {
  return run_attention(cache, q, q_ld, B, M, q_heads, q_lens, scale, window, sinks, out, nullptr, lse, 0, workspace,
                       workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
