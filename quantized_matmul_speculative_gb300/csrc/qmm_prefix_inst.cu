// The kernels of attention behind a shared prefix of one head size, chosen by -DQMM_HEAD_DIM.
#include "qmm_cache_map.cuh"
#include "qmm_prefix.cuh"

#ifndef QMM_HEAD_DIM
#error "QMM_HEAD_DIM must be defined"
#endif

namespace qmm {

template <int D, bool E8, bool BOXES>
static cudaError_t launch_copies(const PrefixArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
  using Cfg = PrefixCfg<D, E8>;
  auto kern = prefix_kernel<D, E8, BOXES>;
  static std::atomic<uint64_t> ready{0};
  uint64_t bit;
  if (first_on_device(ready, &bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  return launch_dependent(kern, dim3(a.ctas), Cfg::THREADS, Cfg::SMEM, stream, a, kmap, vmap);
}
template <int D, bool E8>
static cudaError_t launch_main(PrefixArgs a, cudaStream_t stream) {
  CUtensorMap kmap = {}, vmap = {};
  a.box = 0;
  if constexpr (!E8) {
    // boxes of the largest size that divides page and tile, down to the 8 rows of the swizzle
    if (a.c.num_pages > 0)
      for (int box = PrefixCfg<D, E8>::TN; box >= 8 && a.box == 0; box /= 2)
        if (a.c.page_size % box == 0) a.box = box;
    if (a.box != 0 && cache_map(&kmap, a.c, false, a.box, 1) && cache_map(&vmap, a.c, true, a.box, 1))
      return launch_copies<D, E8, true>(a, kmap, vmap, stream);
    a.box = 0;
  }
  return launch_copies<D, E8, false>(a, kmap, vmap, stream);
}

template <int D>
cudaError_t launch_prefix(const PrefixArgs& a, bool e8, cudaStream_t stream) {
  return e8 ? launch_main<D, true>(a, stream) : launch_main<D, false>(a, stream);
}

template <int D, int SPLIT, int AHEAD>
cudaError_t launch_join(const PrefixArgs& a, bool e8, cudaStream_t stream) {
  constexpr int ROWS = kPrefixJoinThreads / (D / 4) / SPLIT;
  const int64_t ctas = a.c.heads * ((static_cast<int64_t>(a.B) * a.M * a.G + ROWS - 1) / ROWS);
  return launch_dependent(e8 ? prefix_join_kernel<D, true, SPLIT, AHEAD> : prefix_join_kernel<D, false, SPLIT, AHEAD>,
                          dim3(static_cast<unsigned>(ctas)), kPrefixJoinThreads, 0, stream, a);
}
template <int D>
cudaError_t launch_prefix_join(const PrefixArgs& a, bool e8, cudaStream_t stream) {
  constexpr int ROWS = kPrefixJoinThreads / (D / 4);
  const int64_t ctas = a.c.heads * ((static_cast<int64_t>(a.B) * a.M * a.G + ROWS - 1) / ROWS);
  return ctas <= device_sm_count()       ? launch_join<D, 4, 8>(a, e8, stream)
         : ctas <= 4 * device_sm_count() ? launch_join<D, 1, 8>(a, e8, stream)
                                         : launch_join<D, 1, 4>(a, e8, stream);
}

template <int D>
unsigned int read_prefix_unit(int clear) {
  return read_unit_status(clear);
}

template cudaError_t launch_prefix<QMM_HEAD_DIM>(const PrefixArgs&, bool, cudaStream_t);
template cudaError_t launch_prefix_join<QMM_HEAD_DIM>(const PrefixArgs&, bool, cudaStream_t);
template unsigned int read_prefix_unit<QMM_HEAD_DIM>(int);

}  // namespace qmm
