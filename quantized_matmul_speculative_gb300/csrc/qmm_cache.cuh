// A paged cache (qmm_paged_cache, include/qmm.h) as the operators on it see it:
// lengths, pages and E4M3 codes on the device, its checks on the host.
#pragma once

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {

// Tokens of sequence b, clamped to what its block table can hold.
__device__ __forceinline__ int seq_length(const qmm_paged_cache& c, int b) {
  const int cap = c.max_pages * c.page_size;
  int n = c.lengths[b];
  if (n < 0 || n > cap) {
    atomicOr(&g_qmm_status, kStatusBadPage);
    n = n < 0 ? 0 : cap;
  }
  return n;
}
__device__ __forceinline__ int new_rows(const int32_t* q_lens, int b, int M) {
  const int m = q_lens != nullptr ? q_lens[b] : M;
  return m < 0 ? 0 : m > M ? M : m;
}
__device__ __forceinline__ void bad_page() { atomicOr(&g_qmm_status, kStatusBadPage); }

// Two E4M3 codes, nearest even and saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t cvt_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Page of token j, or -1 (and the status bit) if the table names none.
__device__ __forceinline__ int64_t token_page(const qmm_paged_cache& c, int b, int64_t j) {
  const int64_t p = c.block_table[b * c.table_stride + j / c.page_size];
  if (p < 0 || p >= c.num_pages) {
    atomicOr(&g_qmm_status, kStatusBadPage);
    return -1;
  }
  return p;
}

inline bool misaligned(int64_t a, int64_t m) { return (a % m) != 0; }

// Checks of a cache and the B sequences of up to M new rows on it, M at most max_rows (qmm_paged.cu).
qmm_status check_cache(const qmm_paged_cache* c, int B, int M, int max_rows);

}  // namespace qmm
