// The attention kernels of one head size, chosen by -DQMM_HEAD_DIM, for whole sequences or (-DQMM_BEHIND=true) for tokens
// behind a shared prefix.
#include "qmm_cache_map.cuh"
#include "qmm_paged.cuh"

#if !defined(QMM_HEAD_DIM) || !defined(QMM_BEHIND)
#error "QMM_HEAD_DIM and QMM_BEHIND must be defined"
#endif

namespace qmm {

template <int D, bool E8, int RPW, bool BEHIND>
cudaError_t launch_rows(AttentionArgs a, int ctas, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
  using Cfg = AttnCfg<D, E8, RPW>;
  auto kern = attention_kernel<D, E8, RPW, BEHIND>;
  static std::atomic<uint64_t> ready{0};
  uint64_t bit;
  if (first_on_device(ready, &bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  a.tn_log2 = Cfg::TN_LOG2;
  // one CTA an SM, at most one a tile
  const int64_t cap = static_cast<int64_t>(a.c.max_pages) * a.c.page_size;
  const int64_t tiles = static_cast<int64_t>(a.B) * a.c.heads * a.RT * ((cap + Cfg::TN - 1) >> Cfg::TN_LOG2);
  if (tiles < ctas) ctas = tiles < 1 ? 1 : static_cast<int>(tiles);
  a.parts = ctas * Cfg::WORKERS;
  const cudaError_t e = launch_dependent(kern, dim3(ctas), Cfg::THREADS, Cfg::SMEM, stream, a, kmap, vmap);
  if (e != cudaSuccess) return e;
  return launch_dependent(join_kernel<D, E8, BEHIND>, dim3(2 * a.parts), kJoinThreads, 0, stream, a);
}

template <int D, bool BEHIND>
cudaError_t launch_attention(AttentionArgs a, bool e8, int ctas, cudaStream_t stream) {
  // TMA boxes where they divide a page; else, and for strides the TMA cannot
  // take, row by row.
  CUtensorMap kmap = {}, vmap = {};
  a.page_log2 = (a.c.page_size & (a.c.page_size - 1)) == 0 ? __builtin_ctz(static_cast<unsigned>(a.c.page_size)) : -1;
  a.box = a.c.page_size % 16 == 0 ? 16 : a.c.page_size % 8 == 0 ? 8 : 0;
  if (a.c.num_pages < 1) a.box = 0;
  const int rowb = D * (e8 ? 1 : 2), slices = a.box == 16 && rowb > 128 ? rowb / 128 : 1;
  if (a.box != 0 && (!cache_map(&kmap, a.c, false, a.box, slices) || !cache_map(&vmap, a.c, true, a.box, slices))) a.box = 0;
  // Two row tiles a worker share its key and value fragments (and an E4M3
  // cache's conversions); D = 256 has registers for the outputs of one only.
  if (a.RB == 16)
    return e8 ? launch_rows<D, true, 1, BEHIND>(a, ctas, kmap, vmap, stream) : launch_rows<D, false, 1, BEHIND>(a, ctas, kmap, vmap, stream);
  if constexpr (D != 256)
    return e8 ? launch_rows<D, true, 2, BEHIND>(a, ctas, kmap, vmap, stream) : launch_rows<D, false, 2, BEHIND>(a, ctas, kmap, vmap, stream);
  return cudaErrorInvalidValue;
}

template <int D, bool BEHIND>
unsigned int read_attention_status(int clear) {
  return read_unit_status(clear);
}

template cudaError_t launch_attention<QMM_HEAD_DIM, QMM_BEHIND>(AttentionArgs, bool, int, cudaStream_t);
template unsigned int read_attention_status<QMM_HEAD_DIM, QMM_BEHIND>(int);

}  // namespace qmm
