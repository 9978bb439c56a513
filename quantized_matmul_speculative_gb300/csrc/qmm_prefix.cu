// Attention of a batch whose sequences share a long prefix: checks, workspace and
// launches (qmm_shared_prefix_attention, include/qmm.h; kernels: qmm_prefix.cuh).
#include <cmath>

#include "qmm_paged.cuh"
#include "qmm_prefix.cuh"

namespace qmm {

#define QMM_PREFIX_OF(D)                                                                  \
  extern template cudaError_t launch_prefix<D>(const PrefixArgs&, bool, cudaStream_t);      \
  extern template cudaError_t launch_prefix_join<D>(const PrefixArgs&, bool, cudaStream_t); \
  extern template unsigned int read_prefix_unit<D>(int);
QMM_PREFIX_OF(64)
QMM_PREFIX_OF(128)
QMM_PREFIX_OF(256)
#undef QMM_PREFIX_OF

unsigned int read_prefix_status(int clear) {
  return read_prefix_unit<64>(clear) | read_prefix_unit<128>(clear) | read_prefix_unit<256>(clear);
}

namespace {

// Offsets of a call's workspace.
struct PrefixSpace {
  size_t part_o, part_ml, starts, own_o, own_lse, attention, total;
  PrefixSpace(int B, int M, int Hq, int heads, int D) {
    const size_t rows = static_cast<size_t>(B) * M * Hq;
    const size_t lanes = (prefix_segments(static_cast<int64_t>(B) * M * (Hq / heads), heads, D) + device_sm_count()) * (D == 256 ? 1 : 2);
    size_t at = 0;
    auto room = [&at](size_t bytes) {
      const size_t here = at;
      at += (bytes + 255) & ~static_cast<size_t>(255);
      return here;
    };
    part_o = room(lanes * kRows * D * 4);
    part_ml = room(lanes * kRows * 8);
    starts = room((static_cast<size_t>(B) + 1) * 4);
    own_o = room(rows * D * 4);
    own_lse = room(rows * 4);
    attention = room(qmm_paged_attention_workspace(B, M, Hq, heads, D));
    total = at;
  }
};

}  // namespace
}  // namespace qmm

extern "C" {

size_t qmm_shared_prefix_attention_workspace(int B, int M, int q_heads, int heads, int head_dim) {
  if (B <= 0 || M <= 0 || M > 16 || heads <= 0 || q_heads <= 0 || q_heads % heads != 0 || q_heads > 65535 || head_dim <= 0) return 0;
  return qmm::PrefixSpace(B, M, q_heads, heads, head_dim).total;
}

qmm_status qmm_shared_prefix_attention(const qmm_paged_cache* cache, const int32_t* prefix_pages, int num_prefix_pages, const void* q,
                                       int64_t q_ld, int B, int M, int q_heads, const int32_t* q_lens, float scale, void* out,
                                       float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace qmm;
  const qmm_status rc = check_cache(cache, B, M, 16);
  if (rc != QMM_OK) return rc;
  if (q_heads < 1 || q_heads > 65535 || q_heads % cache->heads != 0 || q_heads / cache->heads > 1024 || num_prefix_pages < 0 ||
      q_ld < static_cast<int64_t>(q_heads) * cache->head_dim ||
      (static_cast<int64_t>(num_prefix_pages) + cache->max_pages) * cache->page_size > 0x7fffff00 ||
      static_cast<int64_t>(B) * M * q_heads > 0x7fffff00)
    return QMM_ERR_SHAPE;
  const bool e8 = cache->dtype == QMM_KV_E4M3;
  const float scale_log2 = scale * 1.4426950408889634f * (e8 ? cache->k_scale : 1.f);
  if (!std::isfinite(scale_log2)) return QMM_ERR_UNSUPPORTED;
  if (B == 0 || M == 0) return QMM_OK;
  if (q == nullptr || out == nullptr || workspace == nullptr) return QMM_ERR_NULL;
  if (num_prefix_pages > 0 && (prefix_pages == nullptr || cache->k == nullptr || cache->v == nullptr)) return QMM_ERR_NULL;
  if (misaligned(reinterpret_cast<intptr_t>(q), 16) || misaligned(reinterpret_cast<intptr_t>(out), 16) || misaligned(q_ld, 8) ||
      misaligned(reinterpret_cast<intptr_t>(lse), 4) || misaligned(reinterpret_cast<intptr_t>(q_lens), 4) ||
      misaligned(reinterpret_cast<intptr_t>(prefix_pages), 4) || misaligned(reinterpret_cast<intptr_t>(workspace), 16))
    return QMM_ERR_ALIGN;
  const int D = cache->head_dim;
  const PrefixSpace space(B, M, q_heads, cache->heads, D);
  if (workspace_bytes < space.total) return QMM_ERR_SHAPE;
  unsigned char* const ws = static_cast<unsigned char*>(workspace);
  PrefixArgs a = {};
  a.c = *cache;
  a.prefix = prefix_pages;
  a.tokens = num_prefix_pages * cache->page_size;
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
  a.page_log2 = (cache->page_size & (cache->page_size - 1)) == 0 ? __builtin_ctz(static_cast<unsigned>(cache->page_size)) : -1;
  const int tile = D == 256 ? 64 : 128;
  const int64_t units = prefix_segments(static_cast<int64_t>(B) * M * a.G, cache->heads, D) * ((a.tokens + tile - 1) / tile);
  if (units > 0x7fffff00) return QMM_ERR_SHAPE;  // (numbered in 32 bits)
  a.ctas = units < device_sm_count() ? static_cast<int>(units) : device_sm_count();
  a.part_o = reinterpret_cast<float4*>(ws + space.part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + space.part_ml);
  a.starts = reinterpret_cast<int*>(ws + space.starts);
  float* const own_o = reinterpret_cast<float*>(ws + space.own_o);
  float* const own_lse = reinterpret_cast<float*>(ws + space.own_lse);
  a.own_o = own_o;
  a.own_lse = own_lse;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.inject = injected_short_wait();
  a.wait_ns = a.inject ? 100000ull : kWaitLimitNs;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // (the own tokens first: they have limits of their own, beyond which nothing is launched)
  const qmm_status own = run_attention(cache, q, q_ld, B, M, q_heads, q_lens, scale, 0, 0, nullptr, own_o, own_lse, a.tokens,
                                       ws + space.attention, workspace_bytes - space.attention, st);
  if (own != QMM_OK) return own;
  if (a.tokens > 0) {
    const auto launch = D == 64 ? launch_prefix<64> : D == 128 ? launch_prefix<128> : launch_prefix<256>;
    const cudaError_t e = launch(a, e8, st);
    if (e != cudaSuccess) return static_cast<qmm_status>(finish_call(e));
  }
  const auto join = D == 64 ? launch_prefix_join<64> : D == 128 ? launch_prefix_join<128> : launch_prefix_join<256>;
  return static_cast<qmm_status>(finish_call(join(a, e8, st)));
}

}  // extern "C"
