// TMA descriptors of a paged cache, for the kernels that copy its pages.
#pragma once

#include <cudaTypedefs.h>

#include <mutex>

#include "../../include/qmm.h"

namespace qmm {

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda).
inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
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

// The cache as (byte column of a slice, token of a page, slice, head, page), a slice
// being 128 bytes of a head's row (64 where the row is shorter), in boxes of box_tokens
// tokens and box_slices slices; false where the driver does not take it.
inline bool cache_map(CUtensorMap* map, const qmm_paged_cache& c, bool values, int box_tokens, int box_slices) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (encode == nullptr) return false;
  void* const base = values ? c.v : c.k;
  const int64_t page = values ? c.v_page : c.k_page, token = values ? c.v_token : c.k_token, head = values ? c.v_head : c.k_head;
  const int es = c.dtype == QMM_KV_E4M3 ? 1 : 2, rowb = c.head_dim * es, slice = rowb < 128 ? rowb : 128, slices = rowb / slice;
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(slice), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(slices), static_cast<cuuint64_t>(c.heads),
                              static_cast<cuuint64_t>(c.num_pages)};
  // strides of dimensions of one entry are never used: any valid value does
  auto stride = [&](int64_t elements, int64_t extent) {
    return static_cast<cuuint64_t>(extent > 1 ? elements * es : 16);
  };
  const cuuint64_t strides[4] = {stride(token, c.page_size), static_cast<cuuint64_t>(slice), stride(head, c.heads),
                                 stride(page, c.num_pages)};
  for (cuuint64_t s : strides)
    if (static_cast<int64_t>(s) <= 0 || s >= (1ull << 40)) return false;
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(slice), static_cast<cuuint32_t>(box_tokens),
                             static_cast<cuuint32_t>(box_slices), 1, 1};
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                slice == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace qmm
