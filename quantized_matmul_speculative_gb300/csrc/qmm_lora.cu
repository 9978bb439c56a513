// Low-rank adapters of many requests beside a shared projection (qmm_lora_add,
// include/qmm.h): Y[t] = base[t] + scale[a] B[a] (A[a] X[t]), a = adapters[t].
//
// The work.  Rows of one adapter form tiles of 16 (or 32 or 64) rows, so that its matrices are
// read once for them; the rows without an adapter form tiles too, which are copied.  Two
// kernels: H = A X, a tile's K cut into slices over warps and CTAs, whose sums lie in the
// workspace in fp32; then Y, a tile's columns cut over warps and CTAs.  Up to 256 rows the
// CTAs of both find their tiles themselves (a row's place among those of its adapter by
// comparing all pairs); more rows are sorted by adapter in a kernel before.  In which
// order the rows of a tile come changes no result.
//
// The mathematics.  Products of bf16 with fp32 sums on the warps' tensor cores (m16n8k16,
// the rows as the 16-row operand): the work is reading B and the rows (1 to 100 flop a
// byte), so that these do.  Both operands are loaded straight from memory, 16 (H) or 8 (Y)
// neighbouring elements of the inner dimension a thread, which is in any order the same
// sum.  H enters the second product as bf16 terms, two of them (16 bits) for a bf16 Y,
// three (24) for fp32.  In Y's product column g of n8 tile j stands for column
// 8 (g / 2) + 2 j + g mod 2 of 32, so that a thread ends with 8 neighbouring columns.
//
// What bounds it: HBM for many adapters (64 x 4 rows, 48 of rank 64, 34816 x 5120: 51 us,
// 4.7 TB/s), two or three launches and their loads' latency for few (4 rows of rank 16: 7 to
// 8 us) and short ones (6 x 700 rows of rank 16, 5120 x 17408, fp32: 26 us, 2.3 TB/s).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kLoraThreads = 256, kLoraWarps = kLoraThreads / 32;
constexpr int kMaxRank = 128;
constexpr int kPairRows = kLoraThreads;  // rows up to which all pairs are compared
constexpr int kTurnPitch = 36;           // floats, of 32 columns
constexpr int kMaxSlices = 8;            // of K, over CTAs
constexpr int kPlanThreads = 1024, kPlanCounts = 4096;

struct LoraArgs {
  const void* base;
  const uint16_t* x;
  const uint16_t *A, *B;
  const int32_t* ids;
  const float* scales;
  void* y;
  int64_t base_ld, x_ld, y_ld;
  int T, N, K, R, L, f32;
  int rows_log2;   // of a tile: 4, 5 or 6
  int tiles;       // at most
  int slices;      // of K at most
  int sms;
  int in_place;    // Y is base
  float* part;     // [slices][tiles][rows][R]
  // of more than kPairRows rows:
  int* plan_rows;  // [tiles][rows]: row, or -1
  int* plan_ids;   // [tiles]: adapter, or L (none)
  int* plan_total; // tiles that there are
  int* counts;     // [L + 1]: an adapter's rows, then its first tile
  int* place;      // [T]
};

// A row's adapter; L for none.
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int t) {
  const int id = __ldcg(&a.ids[t]);
  if (id >= a.L) atomicOr(&g_qmm_status, kStatusBadGather);
  return id < 0 || id >= a.L ? a.L : id;
}

// The tiles, as all threads of a CTA see them.  (Read from L2, as the second kernel does
// this before it waits for the first one.)
struct Tile {
  __align__(16) int ids[kPairRows];
  int rows[64];
  int leaders[kLoraWarps];
  int id, rank;
};
struct Tiles {
  Tile& s;
  int total;               // tiles that there are
  int id, rank, number;    // of this thread's row: its adapter, place there, and the tile that it begins (-1: none)
  __device__ __forceinline__ Tiles(const LoraArgs& a, Tile& shared) : s(shared) {
    const int t = threadIdx.x, R = 1 << a.rows_log2;
    if (a.T > kPairRows) {
      total = __ldcg(a.plan_total);
      return;
    }
    id = t < a.T ? adapter_of(a, t) : -1;
    s.ids[t] = id;
    __syncthreads();
    rank = 0;
#pragma unroll 4
    for (int i = 0; i < a.T; i += 4) {
      const int4 o = *reinterpret_cast<const int4*>(s.ids + i);
      rank += (o.x == id && i < t) + (o.y == id && i + 1 < t) + (o.z == id && i + 2 < t) + (o.w == id && i + 3 < t);
    }
    // the rows that tiles begin with, which number them
    const bool leads = t < a.T && (rank & (R - 1)) == 0;
    const unsigned who = __ballot_sync(0xffffffffu, leads);
    if ((t & 31) == 0) s.leaders[t >> 5] = __popc(who);
    __syncthreads();
    int before = __popc(who & ((1u << (t & 31)) - 1));
    total = 0;
    for (int w = 0; w < kLoraWarps; ++w) {
      if (w < t >> 5) before += s.leaders[w];
      total += s.leaders[w];
    }
    number = leads ? before : -1;
  }
  // Rows and adapter of tile q < total, in shared memory.
  __device__ __forceinline__ void select(const LoraArgs& a, int q) {
    const int t = threadIdx.x, R = 1 << a.rows_log2;
    __syncthreads();  // (the tile before has been read)
    if (a.T > kPairRows) {
      if (t == 0) s.id = __ldcg(&a.plan_ids[q]);
      if (t < R) s.rows[t] = __ldcg(&a.plan_rows[q * R + t]);
    } else {
      if (t < R) s.rows[t] = -1;
      if (number == q) {
        s.id = id;
        s.rank = rank;
      }
      __syncthreads();
      if (t < a.T && id == s.id && rank >= s.rank && rank < s.rank + R) s.rows[rank - s.rank] = t;
    }
    __syncthreads();
  }
};
// Blocks of 32 of K whose loads a warp has under way together, for so many n8 tiles of ranks.
__host__ __device__ constexpr int blocks_together(int nt) { return nt <= 2 ? 4 : nt <= 4 ? 2 : 1; }
// Slices of K that the tiles' H is computed in: up to two CTAs an SM at once (more of them than there is room for: 54.2
// us for 64 x 4 rows of rank 64 on 34816 x 5120, and 51.3), each warp with that many blocks or more.
__device__ __forceinline__ int slices_of(const LoraArgs& a, int total) {
  return max(1, min(a.slices, 2 * a.sms / max(total, 1)));
}

// Sorts the rows by adapter: one CTA.
__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(const LoraArgs a) {
  __shared__ int s_sum[kPlanThreads / 32], s_base, s_counts[kPlanCounts];
  griddep_wait();
  griddep_launch_dependents();
  const int R = 1 << a.rows_log2, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // (the adapters' numbers of rows, and then first tiles, in shared memory where there is room)
  int* const counts = a.L < kPlanCounts ? s_counts : a.counts;
  for (int i = threadIdx.x; i <= a.L; i += kPlanThreads) counts[i] = 0;
  for (int i = threadIdx.x; i < a.tiles * R; i += kPlanThreads) a.plan_rows[i] = -1;
  if (threadIdx.x == 0) s_base = 0;
  __threadfence_block();
  __syncthreads();
  for (int t = threadIdx.x; t < a.T; t += kPlanThreads) a.place[t] = atomicAdd(&counts[adapter_of(a, t)], 1);
  __threadfence_block();
  __syncthreads();
  for (int i0 = 0; i0 <= a.L; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int n = i <= a.L ? (*static_cast<volatile int*>(counts + i) + R - 1) >> a.rows_log2 : 0;
    int inc = n;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, inc, s);
      if (lane >= s) inc += o;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    int before = s_base + inc - n;
    for (int w = 0; w < warp; ++w) before += s_sum[w];
    if (i <= a.L) {
      counts[i] = before;
      for (int k = 0; k < n; ++k) a.plan_ids[before + k] = i;
    }
    __syncthreads();
    if (threadIdx.x == kPlanThreads - 1) s_base = before + n;
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.plan_total = s_base;
  __threadfence_block();
  __syncthreads();
  for (int t = threadIdx.x; t < a.T; t += kPlanThreads) {
    const int id = a.ids[t], key = id < 0 || id >= a.L ? a.L : id;
    a.plan_rows[*static_cast<volatile int*>(counts + key) * R + a.place[t]] = t;
  }
}

// H of a tile's slice of K.  A warp takes 16 rows and every KW-th block of 32 of the
// slice; the warps of the same rows add up in shared memory.  NT n8 tiles of ranks.
template <int NT, int ROWS_LOG2>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_shrink_kernel(const LoraArgs a) {
  constexpr int WR = (1 << ROWS_LOG2) / 16, KW = kLoraWarps / WR;
  __shared__ Tile tile;
  __shared__ float h[WR][16][NT * 8 + 4];
  griddep_wait();
  griddep_launch_dependents();
  Tiles tiles(a, tile);
  const int slices = slices_of(a, tiles.total);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int wr = warp % WR, kw = warp / WR, blocks = (a.K + 31) / 32;
  const uint4 none = make_uint4(0, 0, 0, 0);
  for (int unit = blockIdx.x; unit < tiles.total * slices; unit += gridDim.x) {
    const int q = unit / slices, slice = unit - q * slices;
    tiles.select(a, q);
    if (tile.id >= a.L) continue;
    const int b0 = blocks * slice / slices, b1 = blocks * (slice + 1) / slices;
    const int r0 = tile.rows[wr * 16 + g], r1 = tile.rows[wr * 16 + 8 + g];
    const uint16_t* const x0 = a.x + (r0 < 0 ? 0 : r0) * a.x_ld + 8 * c;
    const uint16_t* const x1 = a.x + (r1 < 0 ? 0 : r1) * a.x_ld + 8 * c;
    const uint16_t* const w0 = a.A + (static_cast<int64_t>(tile.id) * a.R + g) * a.K + 8 * c;
    float acc[NT][4] = {};
    constexpr int U = blocks_together(NT);
    if (tile.rows[wr * 16] >= 0)
      for (int b = b0 + kw; b < b1; b += KW * U) {
        uint4 u[U], v[U], w[U][NT];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int k = (b + i * KW) * 32;
          const bool in = b + i * KW < b1 && k + 8 * c < a.K;
          u[i] = in && r0 >= 0 ? ld_after_wait_v4(x0 + k) : none;
          v[i] = in && r1 >= 0 ? ld_after_wait_v4(x1 + k) : none;
#pragma unroll
          for (int j = 0; j < NT; ++j)
            w[i][j] = in && j * 8 < a.R ? ld_after_wait_v4(w0 + static_cast<int64_t>(j * 8) * a.K + k) : none;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const uint32_t f0[4] = {u[i].x, v[i].x, u[i].y, v[i].y}, f1[4] = {u[i].z, v[i].z, u[i].w, v[i].w};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_bf16_16816(acc[j], f0, w[i][j].x, w[i][j].y);
            mma_bf16_16816(acc[j], f1, w[i][j].z, w[i][j].w);
          }
        }
      }
    // in the order of the warps
    for (int s = 0; s < KW; ++s) {
      if (kw == s)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& to = h[wr][g + 8 * (e >> 1)][j * 8 + 2 * c + (e & 1)];
            to = s == 0 ? acc[j][e] : to + acc[j][e];
          }
      __syncthreads();
    }
    float* const out = a.part + ((static_cast<int64_t>(slice) * a.tiles + q) << ROWS_LOG2) * a.R;
    for (int i = threadIdx.x; i < (a.R << ROWS_LOG2); i += kLoraThreads) {
      const int r = i / a.R, k = i - r * a.R;
      out[i] = h[r >> 4][r & 15][k];
    }
  }
}

// A piece of base.
__device__ __forceinline__ void load_piece(uint4& v, const void* p) { v = ld_after_wait_v4(p); }
__device__ __forceinline__ void load_piece(float& v, const float* p) {
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
}
__device__ __forceinline__ void load_piece(__nv_bfloat16& v, const __nv_bfloat16* p) {
  uint16_t u;
  asm volatile("ld.global.b16 %0, [%1];" : "=h"(u) : "l"(p) : "memory");
  v = __ushort_as_bfloat16(u);
}
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store8(float* to, const float (&v)[8]) {
  reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* to, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
  *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
}
// 4 neighbouring ranks a step of one row of B: STEPS pieces of 8 bytes, in one or two
// loads where all 16 STEPS ranks exist.  CACHED: through L1, where the CTA's other row
// warps read the same; else from L2, which may be done before the wait for the kernel
// before, as B is older than that one.
template <int STEPS, bool FULL, bool CACHED>
__device__ __forceinline__ void load_ranks(uint2 (&w)[STEPS], const uint16_t* p, int valid) {
  if constexpr (!FULL) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      w[s] = make_uint2(0, 0);
      if (4 * s < valid) asm volatile("ld.global.cg.v2.b32 {%0, %1}, [%2];" : "=r"(w[s].x), "=r"(w[s].y) : "l"(p + 4 * s) : "memory");
    }
  } else if (valid <= 0) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) w[s] = make_uint2(0, 0);
  } else if constexpr (STEPS == 1) {
    if (CACHED) w[0] = ld_after_wait_v2(p);
    else asm volatile("ld.global.cg.v2.b32 {%0, %1}, [%2];" : "=r"(w[0].x), "=r"(w[0].y) : "l"(p) : "memory");
  } else {
#pragma unroll
    for (int s = 0; s < STEPS; s += 2) {
      if (CACHED)
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[s].x), "=r"(w[s].y), "=r"(w[s + 1].x), "=r"(w[s + 1].y) : "l"(p + 4 * s) : "memory");
      else
        asm volatile("ld.global.cg.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[s].x), "=r"(w[s].y), "=r"(w[s + 1].x), "=r"(w[s + 1].y) : "l"(p + 4 * s) : "memory");
    }
  }
}

// `count` columns from `first` on of rows without an adapter, bit for bit, four rows under way at a time.
template <class T, int ROWS, bool VEC>
__device__ __forceinline__ void copy_rows(const LoraArgs& a, const int* rows, int first, int count) {
  constexpr int P = VEC ? 16 / sizeof(T) : 1;
  using Piece = std::conditional_t<VEC, uint4, T>;
  const T* const base = static_cast<const T*>(a.base) + first;
  T* const y = static_cast<T*>(a.y) + first;
#pragma unroll 1
  for (int r = 0; r < ROWS && rows[r] >= 0; r += 4) {
#pragma unroll 1
    for (int i = threadIdx.x * P; i < count; i += kLoraThreads * P) {
      Piece u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (rows[r + k] >= 0) load_piece(u[k], base + rows[r + k] * a.base_ld + i);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (rows[r + k] >= 0) *reinterpret_cast<Piece*>(y + rows[r + k] * a.y_ld + i) = u[k];
    }
  }
}

// Y of a tile's share of columns, 32 at a time a warp (its 16 rows).  STEPS k16 steps of
// ranks, FULL if R is 16 STEPS; thread c of four holds ranks 4 STEPS c on.  VEC: the rows of
// base and Y are pieces of 16 bytes, and a thread adds 8 neighbouring columns of two rows;
// else the products are turned in shared memory and a thread adds a column of 16 rows, so
// that a warp's 32 elements of a row are neighbours (784 rows of 9919 columns: 42 us with
// the elements of VEC's order one by one).
template <class T, int STEPS, int ROWS_LOG2, bool FULL, bool VEC>
__global__ void __launch_bounds__(kLoraThreads, STEPS <= 2 ? 3 : 2) lora_expand_kernel(const LoraArgs a) {
  constexpr int ROWS = 1 << ROWS_LOG2, WR = ROWS / 16, NW = kLoraWarps / WR, TERMS = sizeof(T) == 4 ? 3 : 2;
  constexpr int PITCH = STEPS * 16 + 8;  // (an odd number of 16 bytes: the eight rows of a load in different banks)
  constexpr int RAW = sizeof(T) == 4 ? 2 : 1;  // 16-byte pieces of 8 columns
  __shared__ Tile tile;
  __shared__ __align__(16) __nv_bfloat16 h[TERMS][ROWS][PITCH];
  __shared__ __align__(16) float turned[VEC ? 1 : kLoraWarps][16][kTurnPitch];
  const T* const base = static_cast<const T*>(a.base);
  T* const y = static_cast<T*>(a.y);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int wr = warp % WR, nw = warp / WR;
  Tiles tiles(a, tile);
  const int slices = slices_of(a, tiles.total);
  // an equal, contiguous share of all tiles' groups of 32 columns
  const int groups = (a.N + 31) / 32;
  const int64_t units = static_cast<int64_t>(tiles.total) * groups, end = units * (blockIdx.x + 1) / gridDim.x;
  bool waited = false;
  for (int64_t u = units * blockIdx.x / gridDim.x; u < end;) {
    const int q = static_cast<int>(u / groups), n0 = static_cast<int>(u - static_cast<int64_t>(q) * groups);
    const int n1 = static_cast<int>(end - u < groups - n0 ? n0 + (end - u) : groups);
    u += n1 - n0;
    tiles.select(a, q);
    if (tile.id >= a.L) {
      if (!waited) griddep_wait();
      waited = true;
      if (!a.in_place) copy_rows<T, ROWS, VEC>(a, tile.rows, n0 * 32, min(n1 * 32, a.N) - n0 * 32);
      continue;
    }
    const int row[2] = {tile.rows[wr * 16 + g], tile.rows[wr * 16 + 8 + g]};
    const uint16_t* const w0 = a.B + static_cast<int64_t>(tile.id) * a.N * a.R + 4 * STEPS * c;
    const int valid = a.R - 4 * STEPS * c;
    uint2 w[4][STEPS];  // a thread's ranks of the group's 32 rows of B
    auto fetch = [&](int group) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = group * 32 + 8 * (g >> 1) + 2 * j + (g & 1);
        load_ranks<STEPS, FULL, (WR > 1)>(w[j], w0 + static_cast<int64_t>(n) * a.R, group < n1 && n < a.N ? valid : 0);
      }
    };
    const bool some = tile.rows[wr * 16] >= 0;  // of this warp's rows
    int group = n0 + nw;
    if (WR == 1) fetch(group);
    if (!waited) griddep_wait();
    waited = true;
    if (WR > 1 && some) fetch(group);
    // the tile's H: slices added in order, scaled, as bf16 terms
    const float scale = a.scales != nullptr ? a.scales[tile.id] : 1.f;
    for (int i = threadIdx.x; i < ROWS * STEPS * 4; i += kLoraThreads) {
      const int r = i / (STEPS * 4), k = (i - r * STEPS * 4) * 4;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (k < a.R && tile.rows[r] >= 0)
#pragma unroll 4
        for (int s = 0; s < slices; ++s) {
          const uint4 u = ld_after_wait_v4(a.part + (((static_cast<int64_t>(s) * a.tiles + q) << ROWS_LOG2) + r) * a.R + k);
          v[0] += __uint_as_float(u.x), v[1] += __uint_as_float(u.y), v[2] += __uint_as_float(u.z), v[3] += __uint_as_float(u.w);
        }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float rest = v[e] * scale;
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
          // (towards zero but for the last, so that no finite number becomes infinite)
          const __nv_bfloat16 top = term + 1 < TERMS ? __float2bfloat16_rz(rest) : __float2bfloat16_rn(rest);
          h[term][r][k + e] = top;
          // (what is not finite stays in the first term: infinity less itself would be NaN in every column)
          rest = fabsf(rest) <= 3.4028235e38f ? rest - __bfloat162float(top) : 0.f;
        }
      }
    }
    __syncthreads();
    if (some)
#pragma unroll 1
    for (; group < n1; group += NW) {
      const int n = group * 32 + 8 * c;
      uint4 b[2][RAW];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < RAW; ++i)
          if (VEC && row[r] >= 0 && n < a.N) b[r][i] = ld_after_wait_v4(base + row[r] * a.base_ld + n + i * 4);
      float acc[4][4] = {};
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int term = TERMS - 1; term >= 0; --term) {
          const int k = 4 * STEPS * c + 4 * s;
          const uint2 lo = *reinterpret_cast<const uint2*>(&h[term][wr * 16 + g][k]);
          const uint2 hi = *reinterpret_cast<const uint2*>(&h[term][wr * 16 + 8 + g][k]);
          const uint32_t f[4] = {lo.x, hi.x, lo.y, hi.y};
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_bf16_16816(acc[j], f, w[j][s].x, w[j][s].y);
        }
      fetch(group + NW);  // under way while this group is written
      if constexpr (VEC) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (row[r] < 0 || n >= a.N) continue;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = acc[i >> 1][2 * r + (i & 1)];
          if constexpr (RAW == 2) {
            const uint4 u = b[r][0], z = b[r][RAW - 1];
            const uint32_t words[8] = {u.x, u.y, u.z, u.w, z.x, z.y, z.z, z.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += __uint_as_float(words[i]);
          } else {
            const uint32_t words[4] = {b[r][0].x, b[r][0].y, b[r][0].z, b[r][0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[2 * i] += bf16_lo(words[i]);
              v[2 * i + 1] += bf16_hi(words[i]);
            }
          }
          store8(y + row[r] * a.y_ld + n, v);
        }
      } else {
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 8; i += 4)
            *reinterpret_cast<float4*>(&turned[warp][g + 8 * r][8 * c + i]) =
                make_float4(acc[i >> 1][2 * r], acc[i >> 1][2 * r + 1], acc[(i >> 1) + 1][2 * r], acc[(i >> 1) + 1][2 * r + 1]);
        __syncwarp();
        const int column = group * 32 + lane;
        const int* const rows = tile.rows + wr * 16;
        if (column < a.N)
#pragma unroll 1
          for (int i = 0; i < 16; i += 8) {
            T v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (rows[i + k] >= 0) load_piece(v[k], base + rows[i + k] * a.base_ld + column);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (rows[i + k] >= 0) y[rows[i + k] * a.y_ld + column] = static_cast<T>(widen(v[k]) + turned[warp][i + k][lane]);
          }
      }
    }
  }
  if (!waited) griddep_wait();
  griddep_launch_dependents();
}

// How T rows on up to L adapters are tiled.
struct LoraPlan {
  int rows_log2;
  int64_t tiles;
  // Tiles of 64 rows (of ranks above 64, whose terms fill the shared memory, 32) where an
  // adapter has 32 rows or more on average and its matrices are more to read than 16 rows;
  // else of 16 (700 rows of rank 16 and 17408 x 5120: 21 us in the second kernel with 64).
  LoraPlan(int T, int L, int R) {
    const int64_t most = std::min<int64_t>(T, static_cast<int64_t>(L) + 1);  // adapters, and none
    rows_log2 = T / std::max<int64_t>(most, 1) >= 32 && (R == 32 || R == 64 || R == 128) ? (R > 64 ? 5 : 6) : 4;
    tiles = (T >> rows_log2) + most;
  }
  int64_t part_floats(int R) const { return kMaxSlices * (tiles << rows_log2) * R; }
};
struct LoraSpace {
  size_t part, rows, ids, total_tiles, counts, place, total;
  LoraSpace(int T, int L, int R) {
    const LoraPlan p(T, L, R);
    size_t at = 0;
    auto room = [&at](size_t bytes) {
      const size_t here = at;
      at += (bytes + 255) & ~static_cast<size_t>(255);
      return here;
    };
    part = room(static_cast<size_t>(p.part_floats(R)) * 4);
    const bool planned = T > kPairRows;
    rows = room(planned ? static_cast<size_t>(p.tiles << p.rows_log2) * 4 : 0);
    ids = room(planned ? static_cast<size_t>(p.tiles) * 4 : 0);
    total_tiles = room(planned ? 4 : 0);
    counts = room(planned ? (static_cast<size_t>(L) + 1) * 4 : 0);
    place = room(planned ? static_cast<size_t>(T) * 4 : 0);
    total = at;
  }
};

cudaError_t launch_shrink(const LoraArgs& a, cudaStream_t stream) {
  const int nt = a.R / 8;
  auto kern = a.rows_log2 == 6   ? (nt <= 4 ? lora_shrink_kernel<4, 6> : lora_shrink_kernel<8, 6>)
              : a.rows_log2 == 5 ? lora_shrink_kernel<16, 5>
              : nt <= 1          ? lora_shrink_kernel<1, 4>
              : nt <= 2          ? lora_shrink_kernel<2, 4>
              : nt <= 4          ? lora_shrink_kernel<4, 4>
              : nt <= 8          ? lora_shrink_kernel<8, 4>
                                 : lora_shrink_kernel<16, 4>;
  const int64_t units = static_cast<int64_t>(a.slices) * a.tiles;
  return launch_dependent(kern, dim3(static_cast<unsigned>(std::min<int64_t>(units, 2 * a.sms))), kLoraThreads, 0, stream, a);
}
template <class T, bool VEC>
cudaError_t launch_expand(const LoraArgs& a, cudaStream_t stream) {
  const int R = a.R;
  auto kern = a.rows_log2 == 6   ? (R == 32 ? lora_expand_kernel<T, 2, 6, true, VEC> : lora_expand_kernel<T, 4, 6, true, VEC>)
              : a.rows_log2 == 5 ? lora_expand_kernel<T, 8, 5, true, VEC>
              : R == 16          ? lora_expand_kernel<T, 1, 4, true, VEC>
              : R < 16           ? lora_expand_kernel<T, 1, 4, false, VEC>
              : R == 32          ? lora_expand_kernel<T, 2, 4, true, VEC>
              : R < 32           ? lora_expand_kernel<T, 2, 4, false, VEC>
              : R == 64          ? lora_expand_kernel<T, 4, 4, true, VEC>
              : R < 64           ? lora_expand_kernel<T, 4, 4, false, VEC>
              : R == 128         ? lora_expand_kernel<T, 8, 4, true, VEC>
                                 : lora_expand_kernel<T, 8, 4, false, VEC>;
  // as many CTAs as the SMs hold, each warp with 32 columns or more, but tiles apart (8 tiles of 21 columns: 15.7 us in one CTA)
  const int64_t warps = kLoraWarps >> (a.rows_log2 - 4), groups = (a.N + 31) / 32;
  const int64_t ctas = std::min<int64_t>(a.tiles * ((groups + warps - 1) / warps), (a.R <= 32 ? 3 : 2) * a.sms);
  return launch_dependent(kern, dim3(static_cast<unsigned>(ctas)), kLoraThreads, 0, stream, a);
}

}  // namespace

unsigned int read_lora_status(int clear) { return read_unit_status(clear); }

}  // namespace qmm

extern "C" {

size_t qmm_lora_workspace(int T, int L, int R) {
  if (T <= 0 || L < 0 || R < 8 || R > qmm::kMaxRank) return 0;
  return qmm::LoraSpace(T, L, R).total;
}

qmm_status qmm_lora_add(const void* base, int64_t base_ld, const void* X, int64_t x_ld, const void* A, const void* Bm,
                        const int32_t* adapters, const float* scales, int T, int N, int K, int R, int L, void* Y, int64_t y_ld,
                        int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace qmm;
  if (T < 0 || N < 0 || K < 0 || L < 0 || R < 8 || R > kMaxRank || R % 8 != 0 || K % 8 != 0 || N > (1 << 30) || K > (1 << 30) ||
      L > (1 << 30) || base_ld < N || y_ld < N || x_ld < K)
    return QMM_ERR_SHAPE;
  const LoraPlan plan(T, L, R);
  if (plan.tiles > 65535) return QMM_ERR_SHAPE;
  if (out_dtype != QMM_OUT_BF16 && out_dtype != QMM_OUT_F32) return QMM_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return QMM_OK;
  if (base == nullptr || Y == nullptr || adapters == nullptr || (K > 0 && X == nullptr) ||
      (L > 0 && (Bm == nullptr || (K > 0 && A == nullptr))))
    return QMM_ERR_NULL;
  const uintptr_t es = out_dtype == QMM_OUT_F32 ? 4 : 2;
  if (((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(Y)) % es) ||
      (K > 0 && (((reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(A)) % 16) || x_ld % 8 != 0)) ||
      reinterpret_cast<uintptr_t>(Bm) % 16 || ((reinterpret_cast<uintptr_t>(adapters) | reinterpret_cast<uintptr_t>(scales)) % 4))
    return QMM_ERR_ALIGN;
  const LoraSpace space(T, L, R);
  if (workspace == nullptr) return QMM_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(workspace) % 16) return QMM_ERR_ALIGN;
  if (workspace_bytes < space.total) return QMM_ERR_SHAPE;
  unsigned char* const ws = static_cast<unsigned char*>(workspace);
  LoraArgs a = {};
  a.base = base;
  a.x = static_cast<const uint16_t*>(X);
  a.A = static_cast<const uint16_t*>(A);
  a.B = static_cast<const uint16_t*>(Bm);
  a.ids = adapters;
  a.scales = scales;
  a.y = Y;
  a.base_ld = base_ld;
  a.x_ld = x_ld;
  a.y_ld = y_ld;
  a.T = T;
  a.N = N;
  a.K = K;
  a.R = R;
  a.L = L;
  a.f32 = out_dtype == QMM_OUT_F32;
  a.rows_log2 = plan.rows_log2;
  a.tiles = static_cast<int>(plan.tiles);
  a.in_place = base == Y && base_ld == y_ld;
  const bool vector = N % 8 == 0 && ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(Y)) % 16) == 0 &&
                      base_ld * es % 16 == 0 && y_ld * es % 16 == 0;
  a.sms = device_sm_count();
  a.slices = std::max(1, std::min(kMaxSlices, (K + 31) / 32 / (blocks_together(R / 8) * (kLoraWarps >> (a.rows_log2 - 4)))));
  a.part = reinterpret_cast<float*>(ws + space.part);
  a.plan_rows = reinterpret_cast<int*>(ws + space.rows);
  a.plan_ids = reinterpret_cast<int*>(ws + space.ids);
  a.plan_total = reinterpret_cast<int*>(ws + space.total_tiles);
  a.counts = reinterpret_cast<int*>(ws + space.counts);
  a.place = reinterpret_cast<int*>(ws + space.place);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (T > kPairRows) e = launch_dependent(lora_plan_kernel, dim3(1), kPlanThreads, 0, st, a);
  if (e == cudaSuccess) e = launch_shrink(a, st);
  if (e == cudaSuccess)
    e = a.f32 ? (vector ? launch_expand<float, true>(a, st) : launch_expand<float, false>(a, st))
              : (vector ? launch_expand<__nv_bfloat16, true>(a, st) : launch_expand<__nv_bfloat16, false>(a, st));
  return static_cast<qmm_status>(finish_call(e));
}

}  // extern "C"
