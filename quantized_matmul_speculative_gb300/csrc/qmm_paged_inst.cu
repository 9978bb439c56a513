// The attention kernels of one head size, chosen by -DQMM_HEAD_DIM.
#include <mutex>

#include "qmm_paged.cuh"

#ifndef QMM_HEAD_DIM
#error "QMM_HEAD_DIM must be defined"
#endif

namespace qmm {

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda).
static PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// The cache as (byte column of a slice, token of a page, slice, head, page),
// boxes of a.box tokens; false where the driver does not take it.
static bool cache_map(CUtensorMap* map, const AttentionArgs& a, int D, bool e8, void* base, int64_t page, int64_t token,
                      int64_t head) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (encode == nullptr) return false;
  const int es = e8 ? 1 : 2, rowb = D * es, slice = rowb < 128 ? rowb : 128, slices = rowb / slice;
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(slice), static_cast<cuuint64_t>(a.c.page_size),
                              static_cast<cuuint64_t>(slices), static_cast<cuuint64_t>(a.c.heads),
                              static_cast<cuuint64_t>(a.c.num_pages)};
  // strides of dimensions of one entry are never used: any valid value does
  auto stride = [&](int64_t elements, int64_t extent) {
    return static_cast<cuuint64_t>(extent > 1 ? elements * es : 16);
  };
  const cuuint64_t strides[4] = {stride(token, a.c.page_size), static_cast<cuuint64_t>(slice), stride(head, a.c.heads),
                                 stride(page, a.c.num_pages)};
  for (cuuint64_t s : strides)
    if (static_cast<int64_t>(s) <= 0 || s >= (1ull << 40)) return false;
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(slice), static_cast<cuuint32_t>(a.box),
                             static_cast<cuuint32_t>(a.box == 16 ? slices : 1), 1, 1};
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                slice == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E8, int RPW>
cudaError_t launch_rows(AttentionArgs a, int ctas, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
  using Cfg = AttnCfg<D, E8, RPW>;
  auto kern = attention_kernel<D, E8, RPW>;
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
  return launch_dependent(join_kernel<D, E8>, dim3(2 * a.parts), kJoinThreads, 0, stream, a);
}

template <int D>
cudaError_t launch_attention(AttentionArgs a, bool e8, int ctas, cudaStream_t stream) {
  // TMA boxes where they divide a page; else, and for strides the TMA cannot
  // take, row by row.
  CUtensorMap kmap = {}, vmap = {};
  a.page_log2 = (a.c.page_size & (a.c.page_size - 1)) == 0 ? __builtin_ctz(static_cast<unsigned>(a.c.page_size)) : -1;
  a.box = a.c.page_size % 16 == 0 ? 16 : a.c.page_size % 8 == 0 ? 8 : 0;
  if (a.c.num_pages < 1) a.box = 0;
  if (a.box != 0 && (!cache_map(&kmap, a, D, e8, a.c.k, a.c.k_page, a.c.k_token, a.c.k_head) ||
                     !cache_map(&vmap, a, D, e8, a.c.v, a.c.v_page, a.c.v_token, a.c.v_head)))
    a.box = 0;
  // Two row tiles a worker share its key and value fragments (and an E4M3
  // cache's conversions); D = 256 has registers for the outputs of one only.
  if (a.RB == 16)
    return e8 ? launch_rows<D, true, 1>(a, ctas, kmap, vmap, stream) : launch_rows<D, false, 1>(a, ctas, kmap, vmap, stream);
  if constexpr (D != 256)
    return e8 ? launch_rows<D, true, 2>(a, ctas, kmap, vmap, stream) : launch_rows<D, false, 2>(a, ctas, kmap, vmap, stream);
  return cudaErrorInvalidValue;
}

template <int D>
unsigned int read_attention_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_qmm_status, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear && v != 0) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(g_qmm_status, &zero, sizeof(zero));
  }
  return v;
}

template cudaError_t launch_attention<QMM_HEAD_DIM>(AttentionArgs, bool, int, cudaStream_t);
template unsigned int read_attention_status<QMM_HEAD_DIM>(int);

}  // namespace qmm
