// Product of two microscaled 4-bit matrices (qmm_matmul_mx, include/qmm.h) on
// the block-scaled tensor cores.
//
// The weights are the 128-row operand and the activations the narrow one, so a
// call of a few rows pads the activations to 16 only, and a thread of the
// epilogue, which owns one of the 128 accumulator lanes, writes one output
// column: a warp's store covers 32 consecutive columns of a row of Y.
//
// A CTA computes tiles of 128 columns x BN rows over K, one after the other, the
// next one's copies and scales under way while it writes; or, where there are
// few tiles, a cluster of C CTAs one tile, a share of K each, added in rank order
// through distributed shared memory.  Warp 0 copies code tiles (256 codes = 128 bytes a
// row, TMA with the 128-byte swizzle), one thread of warp 1 issues four MMAs of
// 64 codes a stage, and warps 2..9 move the scale bytes from the canonical
// [rows, K/g] layout into tensor memory, where an MMA wants, for 4 bytes of K
// (64 codes of nvfp4, 128 of mxfp4) and rows 32 c + l, lane l of each of the
// four lane quarters, column c: a thread loads its own rows' bytes, they pass
// through shared memory, and every warp stores the words of all rows to its
// quarter.  (With the tensor core's own copies from shared memory instead, 12
// of 50 ns a stage at BN = 256 beside 260 ns of MMAs, the 1000 x 34816 x 5120
// product took 201 us.)
//
// What bounds it: the scales' way at BN = 256, a stage's taking longer than its
// 0.26 us of MMAs (without their loads the call took 24 us less, without their
// stores 12; half the activations' codes changed nothing); a tile of 20 stages has
// 1.4 us more to its first and 1.5 us to write.  1000 x 34816 x 5120 nvfp4: 94 us,
// 3.8 PFLOP/s (at 97, with the scales of single stages loaded 111, with a tile a CTA
// too 131; the activations multicast to the 2 or 4 CTAs of a cluster: 110 and 194 for
// 111, so not done).  8 x 5120 x 5120 mxfp4: 5.9 us, 2.4 TB/s,
// its latency from first copy to the sum over the cluster.
//
// Arithmetic: codes and scales are exact, their products too; the accumulator
// is fp32.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <mutex>
#include <type_traits>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kTileN = 128;   // columns of Y (rows of W) of a tile: the MMA's M
constexpr int kTileK = 256;   // codes of a stage: 128 bytes a row
constexpr int kScaleGroups = 2;  // of four warps, each with every second stage's scales
constexpr int kGemmThreads = 64 + 128 * kScaleGroups;
constexpr int kCodesW = kTileN * kTileK / 2;  // bytes of a stage's weight codes

struct MxMatmulArgs {
  const uint8_t* xs;
  const uint8_t* ws;
  void* Y;
  int M, N, K, out_f32;
  int BN;       // rows of Y of a tile: the MMA's N, a multiple of 16, at most 256
  int tiles;    // of Y
  int tiles_m;  // along M
  int ktiles;   // stages of K
  int split;    // CTAs of a cluster
  int stages;
  int pitch;    // scale bytes of a row
  int aligned;  // rows of scales are whole, aligned stages (1), or pairs of them (2)
  uint32_t tmem_cols;
  unsigned long long wait_ns;  // limit of the waits for a stage
  int inject;                  // CTA 0's first stage never completes (tests)
};

// Shared-memory layout (offsets from a 1024-byte aligned start).
struct GemmSmem {
  int x, stage;  // a stage: weight codes, activation codes
  int scales;    // [groups][2][blocks of 128 rows][128] rows' words on their way
  int bars, total;
  __host__ __device__ GemmSmem(int BN, int stages, int sf_words) {
    x = kCodesW;
    stage = x + ((BN * (kTileK / 2) + 1023) & ~1023);
    scales = stages * stage;
    bars = scales + kScaleGroups * 2 * (1 + (BN + 127) / 128) * 128 * 4 * sf_words;
    total = bars + (2 * stages + 2) * 8 + 16;
  }
};

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t stride_bytes, uint32_t layout) {
  // start address, leading offset (unused: one swizzle atom / one core matrix
  // wide), stride between 8-row groups, version 1, swizzle mode
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (1ull << 16) | (static_cast<uint64_t>(stride_bytes >> 4) << 32) |
         (1ull << 46) | (static_cast<uint64_t>(layout) << 61);
}
constexpr uint32_t kSwizzle128 = 2;

// N columns of this warp's lane quarter.
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t* v) {
  if constexpr (N == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
  } else {
    static_assert(N == 8, "8 or 16 columns");
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
  }
}
template <bool NV>
__device__ __forceinline__ void mma_block_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                                 bool accumulate) {
  if constexpr (NV) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(static_cast<uint32_t>(accumulate)) : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(static_cast<uint32_t>(accumulate)) : "memory");
  }
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]) : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// The scale bytes of one row, every second stage's (4 SFW bytes each), loaded
// kAhead of them ahead into a ring whose places are compile-time numbers (u).
// ALIGNED: every row starts on a multiple of a stage's bytes and holds whole
// stages.  Else a stage's bytes lie in two aligned chunks and are shifted
// together; chunks that reach out of the matrix are loaded byte by byte, and
// bytes past the row's end are 0 (the codes there are 0, and 0 times a foreign
// NaN would not be).  Rows past the matrix read its last row: their codes are
// 0 and their outputs not stored.
template <int SFW, bool ALIGNED>
struct ScaleRow {
  static constexpr int kAhead = 2, kChunks = ALIGNED ? 1 : 2;
  const uint8_t* next;  // the chunk to load next
  const uint8_t* begin;
  const uint8_t* end;   // of the matrix
  uint32_t c[kAhead][kChunks * SFW];
  int shift;            // the stage's first byte in its first chunk

  __device__ __forceinline__ void load(uint32_t (&w)[kChunks * SFW], bool wanted) {
    if (wanted) {
#pragma unroll
      for (int h = 0; h < kChunks; ++h) {
        const uint8_t* const p = next + h * 4 * SFW;
        if (ALIGNED || (p >= begin && p + 4 * SFW <= end)) {
          if constexpr (SFW == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[4 * h] = v.x, w[4 * h + 1] = v.y, w[4 * h + 2] = v.z, w[4 * h + 3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[2 * h] = v.x, w[2 * h + 1] = v.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < SFW; ++i) w[h * SFW + i] = 0;
#pragma unroll 1
          for (int i = 0; i < 4 * SFW; ++i)
            if (p + i >= begin && p + i < end) {
              const uint32_t byte = static_cast<uint32_t>(p[i]) << (8 * (i & 3));
#pragma unroll
              for (int x = 0; x < SFW; ++x)
                if (x == i >> 2) w[h * SFW + x] |= byte;
            }
        }
      }
    }
    next += kScaleGroups * 4 * SFW;
  }
  // Row `row` (the last one if there is none), stages `stage`, stage + 2, .. before stage_end.
  __device__ __forceinline__ void start(const uint8_t* s, int row, int rows, int pitch, int stage, int stage_end) {
    const uint8_t* at = s + static_cast<int64_t>(min(row, rows - 1)) * pitch + stage * (4 * SFW);
    shift = ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(at) & (4 * SFW - 1));
    next = at - shift;
    begin = s;
    end = s + static_cast<int64_t>(rows) * pitch;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(c[i], stage + kScaleGroups * i < stage_end);
  }
  // The stage's words, of which `valid` bytes are the row's; place u is then
  // refilled, if that stage is wanted.
  template <int U>
  __device__ __forceinline__ void take(uint32_t (&w)[SFW], int valid, bool wanted) {
    if constexpr (ALIGNED) {
#pragma unroll
      for (int i = 0; i < SFW; ++i) w[i] = c[U][i];
    } else {
      uint32_t x[2 * SFW];
#pragma unroll
      for (int i = 0; i < 2 * SFW; ++i) x[i] = c[U][i];
      if (SFW == 4 && (shift & 8)) {
#pragma unroll
        for (int i = 0; i < 2 * SFW - 2; ++i) x[i] = x[i + 2];
      }
      if (shift & 4) {
#pragma unroll
        for (int i = 0; i < 2 * SFW - 1; ++i) x[i] = x[i + 1];
      }
#pragma unroll
      for (int i = 0; i < SFW; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], 8 * (shift & 3));
      if (valid < 4 * SFW) {
#pragma unroll
        for (int i = 0; i < SFW; ++i) {
          const int left = valid - 4 * i;
          w[i] = left >= 4 ? w[i] : left <= 0 ? 0u : w[i] & ((1u << (8 * left)) - 1u);
        }
      }
    }
    load(c[U], wanted);
  }
};

// The scale warps, in two groups.  Measured at 1000 x 34816 x 5120: with the
// loads' bounds and shifts decided per stage (580 instructions a stage and warp)
// this alone was the bound, 250 us; with one group, whose chain of load, pass,
// store and wait takes longer than a stage's MMAs, 149 us.
template <int SFW, int XB>
struct ScaleStage {
  using Words = typename std::conditional<SFW == 4, uint4, uint2>::type;
  int flip = 0;  // place of the next stage's words
  bool ok = true;
  static __device__ __forceinline__ int half() { return (threadIdx.x - 64) >> 7; }

  // The words w of this thread's rows (a weight row, activation rows), of the CTA's it-th stage, into tensor memory.
  __device__ __forceinline__ void put(const MxMatmulArgs& a, unsigned char* pass_all, uint32_t full, uint32_t empty,
                                      uint32_t columns, const uint32_t (&w)[1 + XB][SFW], int it) {
    const int r = threadIdx.x & 127, lane = r & 31, s = it % a.stages;
    // (two places in turn: a thread that passed the barrier of its next stage has read this one's)
    Words* const pass = reinterpret_cast<Words*>(pass_all) + (half() * 2 + flip) * (1 + XB) * 128;
    flip ^= 1;
#pragma unroll
    for (int b = 0; b <= XB; ++b) {
      if constexpr (SFW == 4) pass[b * 128 + r] = make_uint4(w[b][0], w[b][1], w[b][2], w[b][3]);
      else pass[b * 128 + r] = make_uint2(w[b][0], w[b][1]);
    }
    asm volatile("barrier.sync %0, 128;" ::"r"(1 + half()) : "memory");
    // columns: word w of the weights' rows (4), then word w of the activations' (4 XB)
    uint32_t v[(1 + XB) * 4 * SFW];
#pragma unroll
    for (int b = 0; b <= XB; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const Words x = pass[b * 128 + c * 32 + lane];
        uint32_t w[4] = {x.x, x.y, 0, 0};
        if constexpr (SFW == 4) w[2] = x.z, w[3] = x.w;
#pragma unroll
        for (int i = 0; i < SFW; ++i)
          v[b == 0 ? i * 4 + c : SFW * 4 + i * XB * 4 + (b - 1) * 4 + c] = w[i];
      }
    // after a wait that ran out the rest is left out (a status bit); the warps still meet at every barrier above
    if (ok && it >= a.stages)
      ok = !__any_sync(0xffffffffu, !mbar_wait(empty + s * 8, ((it / a.stages) & 1) ^ 1, kStatusTimeoutEmpty));
    if (!ok) return;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    constexpr int kCols = (1 + XB) * 4 * SFW;  // 16, 24, 32 or 48
    const uint32_t at = columns + s * kCols;
#pragma unroll
    for (int c = 0; c + 16 <= kCols; c += 16) tmem_store<16>(at + c, v + c);
    if constexpr (kCols % 16 != 0) tmem_store<8>(at + kCols - 8, v + kCols - 8);
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    mbar_arrive(full + s * 8);
  }
};

template <int SFW, bool ALIGNED, int XB>
struct ScaleFeed : ScaleStage<SFW, XB> {
  using ScaleStage<SFW, XB>::half;
  using Row = ScaleRow<SFW, ALIGNED>;
  Row rows[1 + XB];  // a weight row, activation rows

  // Load ahead for the tile at (m0, n0), whose first stage is the CTA's it0-th.
  __device__ __forceinline__ void start(const MxMatmulArgs& a, int m0, int n0, int k_begin, int k_end, int it0) {
    const int r = threadIdx.x & 127, first = k_begin + (half() ^ (it0 & 1));
    rows[0].start(a.ws, n0 + r, a.N, a.pitch, first, k_end);
#pragma unroll
    for (int b = 0; b < XB; ++b) rows[1 + b].start(a.xs, m0 + b * 128 + r, a.M, a.pitch, first, k_end);
  }

  template <int U>
  __device__ __forceinline__ void stage(const MxMatmulArgs& a, unsigned char* pass_all, uint32_t full, uint32_t empty,
                                        uint32_t columns, int k, int k_end, int it) {
    if (k >= k_end) return;
    const int valid = a.pitch - k * (4 * SFW);
    const bool wanted = k + kScaleGroups * Row::kAhead < k_end;
    uint32_t w[1 + XB][SFW];
#pragma unroll
    for (int b = 0; b <= XB; ++b) rows[b].template take<U>(w[b], valid, wanted);
    this->put(a, pass_all, full, empty, columns, w, it);
  }
  // The tile's stages k_begin .. k_end - 1; the first is the CTA's it0-th.
  __device__ __forceinline__ void run(const MxMatmulArgs& a, unsigned char* pass, uint32_t full, uint32_t empty, uint32_t columns,
                                      int k_begin, int k_end, int it0) {
    const int group = half() ^ (it0 & 1);
    int it = it0 + group;
    for (int k = k_begin + group; k < k_end; k += kScaleGroups * Row::kAhead, it += kScaleGroups * Row::kAhead) {
      stage<0>(a, pass, full, empty, columns, k, k_end, it);
      stage<1>(a, pass, full, empty, columns, k + kScaleGroups, k_end, it + kScaleGroups);
    }
  }
};

// The same where a row's stages come in aligned pairs: a thread loads a pair at
// once (32 bytes for nvfp4, a whole sector of L2), the groups take pairs in turn.
// Every lane's load is a line of its own, so that half as many of them count:
// 97 us at 1000 x 34816 x 5120 for 111 (104 with the next pair asked for after
// the second stage, not the first).
template <int SFW, int XB>
struct PairFeed : ScaleStage<SFW, XB> {
  using ScaleStage<SFW, XB>::half;
  const uint8_t* next[1 + XB];  // the pair to load next
  uint32_t c[1 + XB][2 * SFW];

  __device__ __forceinline__ void load() {
#pragma unroll
    for (int b = 0; b <= XB; ++b) {
      if constexpr (SFW == 4)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(c[b][0]), "=r"(c[b][1]), "=r"(c[b][2]), "=r"(c[b][3]), "=r"(c[b][4]), "=r"(c[b][5]),
                       "=r"(c[b][6]), "=r"(c[b][7]) : "l"(next[b]) : "memory");
      else
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(c[b][0]), "=r"(c[b][1]), "=r"(c[b][2]), "=r"(c[b][3]) : "l"(next[b]) : "memory");
      next[b] += kScaleGroups * 8 * SFW;
    }
  }
  __device__ __forceinline__ void start(const MxMatmulArgs& a, int m0, int n0, int k_begin, int k_end, int it0) {
    const int r = threadIdx.x & 127, first = k_begin + 2 * (half() ^ ((it0 >> 1) & 1));
    next[0] = a.ws + static_cast<int64_t>(min(n0 + r, a.N - 1)) * a.pitch + first * (4 * SFW);
#pragma unroll
    for (int b = 0; b < XB; ++b)
      next[1 + b] = a.xs + static_cast<int64_t>(min(m0 + b * 128 + r, a.M - 1)) * a.pitch + first * (4 * SFW);
    if (first < k_end) load();
  }
  // (k_begin, k_end and it0 are even)
  __device__ __forceinline__ void run(const MxMatmulArgs& a, unsigned char* pass, uint32_t full, uint32_t empty, uint32_t columns,
                                      int k_begin, int k_end, int it0) {
    for (int k = k_begin + 2 * (half() ^ ((it0 >> 1) & 1)); k < k_end; k += 2 * kScaleGroups) {
      uint32_t w[2][1 + XB][SFW];
#pragma unroll
      for (int b = 0; b <= XB; ++b)
#pragma unroll
        for (int i = 0; i < 2 * SFW; ++i) w[i / SFW][b][i % SFW] = c[b][i];
      this->put(a, pass, full, empty, columns, w[0], it0 + k - k_begin);
      if (k + 2 * kScaleGroups < k_end) load();
      this->put(a, pass, full, empty, columns, w[1], it0 + k - k_begin + 1);
    }
  }
};

// A warp's 32 accumulator lanes (columns of Y) to the rows `first` .. rows - 1
// of Y, every second 16 of them; `y` is its lane's element of row 0.  Whole
// groups of 16 rows need no test.
template <class T>
__device__ __forceinline__ void store_tile(uint32_t acc, T* y, int64_t ld, int first, int rows, bool inside) {
  y += first * ld;
  for (int c = first; c < rows; c += 16 * kScaleGroups, y += 16 * kScaleGroups * ld) {
    uint32_t v[16];
    tmem_load16(v, acc + c);
    tmem_wait_load();
    if (!inside) continue;
    if (c + 16 <= rows) {
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i * ld] = static_cast<T>(__uint_as_float(v[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c + i < rows) y[i * ld] = static_cast<T>(__uint_as_float(v[i]));
    }
  }
}

template <bool NV, int XB>  // XB blocks of 128 activation rows
__global__ void __launch_bounds__(kGemmThreads, 3 - XB)
mx_matmul_kernel(const MxMatmulArgs a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap) {
  constexpr int SFW = NV ? 4 : 2;  // 4-byte scale words of a row in a stage
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const GemmSmem L(a.BN, a.stages, SFW);
  // barriers: a stage is full, is empty; a tile's accumulators are done, are free
  const uint32_t full = sbase + L.bars, empty = full + a.stages * 8, done = empty + a.stages * 8, free = done + 8;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L.bars + (2 * a.stages + 2) * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile0 = blockIdx.x / a.split, tile_step = gridDim.x / a.split;
  const int k_begin = a.ktiles * rank / a.split, k_end = a.ktiles * (rank + 1) / a.split, per_tile = k_end - k_begin;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&wmap);
    prefetch_tmap(&xmap);
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full + s * 8, 1 + 128);
      mbar_init(empty + s * 8, 1);
    }
    mbar_init(done, 1);
    mbar_init(free, 128 * kScaleGroups);
    fence_mbar_init();
    if (a.inject && blockIdx.x == 0) mbar_expect_tx(full, 16);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(a.tmem_cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  // Every role walks the CTA's tiles with a running count of stages, so that the
  // copies for the next tile go on while the last one's outputs are written.  A
  // wait that gave up (a status bit) skips the later ones: wrong results, no hang.
  // Its role does nothing more to the stages, so that the others give up too, and the
  // copies under way are waited for (with the limit again) before the CTA ends.
  if (warp == 0) {
    if (lane == 0) {
      bool lost = false;
      const uint32_t bytes = kCodesW + a.BN * (kTileK / 2);
      int it = 0;
      for (int tile = tile0; tile < a.tiles && !lost; tile += tile_step) {
        const int m0 = (tile % a.tiles_m) * a.BN, n0 = (tile / a.tiles_m) * kTileN;
        for (int k = k_begin; k < k_end; ++k, ++it) {
          const int s = it % a.stages;
          if (it >= a.stages) lost = !mbar_wait(empty + s * 8, ((it / a.stages) & 1) ^ 1, kStatusTimeoutEmpty);
          if (lost) break;
          mbar_arrive_expect_tx(full + s * 8, bytes);
          tma_load_2d(sbase + s * L.stage, &wmap, k * (kTileK / 2), n0, full + s * 8);
          tma_load_2d(sbase + s * L.stage + L.x, &xmap, k * (kTileK / 2), m0, full + s * 8);
        }
      }
      // (the MMAs wait for the same; where one is given up, the limit was time enough for the others)
      for (int i = max(it - a.stages, 0); i < it; ++i)
        if (!mbar_wait(full + i % a.stages * 8, (i / a.stages) & 1, kStatusTimeoutDrain, a.wait_ns)) break;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool lost = false;
      const uint32_t idesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(a.BN >> 3) << 17) | (NV ? 0u : 1u << 23) |
                             (static_cast<uint32_t>(kTileN >> 4) << 24);
      int it = 0, turn = 0;
      for (int tile = tile0; tile < a.tiles; tile += tile_step, ++turn) {
        if (turn > 0 && !lost) lost = !mbar_wait(free, (turn - 1) & 1, kStatusTimeoutEmpty);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        for (int k = k_begin; k < k_end; ++k, ++it) {
          const int s = it % a.stages;
          if (!lost) lost = !mbar_wait(full + s * 8, (it / a.stages) & 1, kStatusTimeoutFull, a.wait_ns);
          if (lost) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t base = sbase + s * L.stage;
          const uint32_t sfw = tmem + a.BN + s * (SFW * 4 * (1 + XB)), sfx = sfw + SFW * 4;
          const uint64_t da = smem_desc(base, 1024, kSwizzle128), db = smem_desc(base + L.x, 1024, kSwizzle128);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // nvfp4: a word of scales for 64 codes; mxfp4: its lower, then its upper half
            const int w = NV ? j : j >> 1;
            const uint32_t id = NV ? 0u : (j & 1) * 2u;
            mma_block_scaled<NV>(tmem, da + j * 2, db + j * 2, idesc | (id << 4) | (id << 29), sfw + w * 4, sfx + w * XB * 4,
                                 k > k_begin || j > 0);
          }
          mma_commit(empty + s * 8);
        }
        mma_commit(done);
      }
    }
  } else {
    // scales of a tile, the first ones of the next already asked for, then the tile's outputs
    auto feed = [&](auto scales) {
      const uint32_t quarter = static_cast<uint32_t>(warp & 3) << 21;
      unsigned char* const pass = smem + L.scales;
      int it = 0, turn = 0;
      bool lost = false;
      scales.start(a, (tile0 % a.tiles_m) * a.BN, (tile0 / a.tiles_m) * kTileN, k_begin, k_end, it);
      for (int tile = tile0; tile < a.tiles; tile += tile_step, ++turn) {
        const int m0 = (tile % a.tiles_m) * a.BN, n = (tile / a.tiles_m) * kTileN + (warp & 3) * 32 + lane;
        scales.run(a, pass, full, empty, tmem + a.BN + quarter, k_begin, k_end, it);
        it += per_tile;
        const int after = tile + tile_step;
        if (after < a.tiles) scales.start(a, (after % a.tiles_m) * a.BN, (after / a.tiles_m) * kTileN, k_begin, k_end, it);
        if (!lost) lost = __any_sync(0xffffffffu, !mbar_wait(done, turn & 1, kStatusTimeoutDrain));
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t acc = tmem + quarter;
        const int first = 16 * scales.half(), rows = min(a.BN, a.M - m0);  // the groups take 16 rows in turn
        const int64_t at = static_cast<int64_t>(m0) * a.N + n;
        if (a.split > 1) {  // (one tile a CTA)
          float* part = reinterpret_cast<float*>(smem) + first * kTileN + (warp & 3) * 32 + lane;  // [BN][128], over the stages
          for (int c = first; c < a.BN; c += 16 * kScaleGroups, part += 16 * kScaleGroups * kTileN) {
            uint32_t v[16];
            tmem_load16(v, acc + c);
            tmem_wait_load();
#pragma unroll
            for (int i = 0; i < 16; ++i) part[i * kTileN] = __uint_as_float(v[i]);
          }
        } else if (a.out_f32) {
          store_tile<float>(acc, static_cast<float*>(a.Y) + at, a.N, first, rows, n < a.N);
        } else {
          store_tile<__nv_bfloat16>(acc, static_cast<__nv_bfloat16*>(a.Y) + at, a.N, first, rows, n < a.N);
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        mbar_arrive(free);
      }
    };
    if (XB == 2 && a.aligned == 2) feed(PairFeed<SFW, XB>{});
    else if (a.aligned) feed(ScaleFeed<SFW, true, XB>{});
    else feed(ScaleFeed<SFW, false, XB>{});
  }
  __syncwarp();
  __syncthreads();
  __syncwarp();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(a.tmem_cols));
  if (a.split > 1) {
    // the cluster's partial tiles, added in rank order; each CTA writes its share of the rows
    cluster_sync_all();
    const int m0 = (tile0 % a.tiles_m) * a.BN, n0 = (tile0 / a.tiles_m) * kTileN;
    const int rows = min(a.BN, a.M - m0);
    const int r0 = rows * rank / a.split, r1 = rows * (rank + 1) / a.split;
    for (int x = threadIdx.x; x < (r1 - r0) * kTileN; x += kGemmThreads) {
      const int row = r0 + x / kTileN, col = x % kTileN;
      if (n0 + col >= a.N) continue;
      const float* at = reinterpret_cast<const float*>(smem) + row * kTileN + col;
      float v = 0.f;
      for (int c = 0; c < a.split; ++c) v += ld_dsmem_f32(at, c);
      store_y(a.Y, nullptr, static_cast<int64_t>(m0 + row) * a.N + n0 + col, v, a.out_f32);
    }
    cluster_sync_all();  // nobody leaves while its partial tile is read
  }
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
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

// Code rows as bytes [rows, K/2], boxes of 128 bytes x `box` rows; what lies
// outside reads as zeros.
bool codes_map(CUtensorMap* map, const void* codes, int rows, int K, int box) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t extent[2] = {kTileK / 2, static_cast<cuuint32_t>(box)};
  const cuuint32_t step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, extent, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tile height and cluster size: the cheapest by an estimate in SM cycles.  A
// stage costs its MMAs (four of 128 x BN x 64) or, from HBM, the bytes that the
// SMs' tiles of one wave need; a tile costs a fixed start and end and its
// outputs.
void plan(MxMatmulArgs& a, int sms) {
  double best = 1e300;
  for (int bn : {16, 32, 64, 128, 256}) {
    if (bn > 16 && bn >= 2 * a.M) break;
    const int64_t tiles = static_cast<int64_t>((a.N + kTileN - 1) / kTileN) * ((a.M + bn - 1) / bn);
    for (int c : {1, 2, 4, 8}) {
      if (c > 1 && (c > a.ktiles / 2 || tiles * c > 2 * sms || bn > 128)) break;
      const int per_sm = bn <= 32 ? 2 : 1;
      const double waves = static_cast<double>((tiles * c + sms * per_sm - 1) / (sms * per_sm));
      const double stage = per_sm * std::max(bn * 1.5, 790.0 / ((a.M + bn - 1) / bn));
      const double cost = waves * ((a.ktiles + c - 1) / c * stage + 2500.0 + bn * 8.0 + (c > 1 ? 1500.0 : 0.0));
      if (cost < best) {
        best = cost;
        a.BN = bn;
        a.split = c;
      }
    }
  }
}

template <bool NV>
cudaError_t launch_mx_matmul(MxMatmulArgs a, const void* Xq, const void* Wq, cudaStream_t stream) {
  if (injected_launch_failure()) return cudaErrorLaunchFailure;
  a.inject = injected_short_wait();
  a.wait_ns = a.inject ? 100000ull : kWaitLimitNs;
  constexpr int SFW = NV ? 4 : 2;
  a.ktiles = (a.K + kTileK - 1) / kTileK;
  a.pitch = a.K / (NV ? 16 : 32);
  a.aligned = a.pitch % (4 * SFW) == 0 &&
              ((reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.ws)) & (4 * SFW - 1)) == 0;
  plan(a, device_sm_count());
  a.tiles_m = (a.M + a.BN - 1) / a.BN;
  const int64_t tiles = static_cast<int64_t>((a.N + kTileN - 1) / kTileN) * a.tiles_m;
  if (tiles > INT_MAX / 8) return cudaErrorInvalidValue;
  a.tiles = static_cast<int>(tiles);
  // as many CTAs as the SMs hold, each with every so manieth tile; a cluster that shares K has one
  const int per_sm = a.BN <= 32 ? 2 : 1;
  const int64_t ctas = a.split > 1 ? tiles * a.split : std::min<int64_t>(tiles, static_cast<int64_t>(per_sm) * device_sm_count());
  // Two CTAs an SM up to 32 rows, else one; stages as shared memory and the
  // tensor memory's columns (accumulators, then each stage's scales) allow.
  const int budget = a.BN <= 32 ? 113 * 1024 : 227 * 1024, cols = a.BN <= 32 ? 256 : 512;
  const int sf_cols = SFW * 4 * (1 + (a.BN + 127) / 128);
  // (an even number, and of pairs too: a stage's scales always come from one group)
  a.stages = 2;
  while (a.stages < 8 && GemmSmem(a.BN, a.stages + 2, SFW).total + 1024 <= budget && a.BN + (a.stages + 2) * sf_cols <= cols)
    a.stages += 2;
  const int pair = 8 * SFW;
  if (a.BN > 128 && a.split == 1 && a.stages % 4 == 0 && a.K % (2 * kTileK) == 0 && a.pitch % pair == 0 &&
      ((reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.ws)) & (pair - 1)) == 0)
    a.aligned = 2;
  a.tmem_cols = cols;
  const int smem = GemmSmem(a.BN, a.stages, SFW).total + 1024;
  CUtensorMap wmap, xmap;
  if (!codes_map(&wmap, Wq, a.N, a.K, kTileN) || !codes_map(&xmap, Xq, a.M, a.K, a.BN)) return cudaErrorNotSupported;
  auto kern = a.BN > 128 ? mx_matmul_kernel<NV, 2> : mx_matmul_kernel<NV, 1>;
  static std::atomic<uint64_t> ready[2] = {};
  uint64_t bit;
  if (first_on_device(ready[a.BN > 128], &bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    ready[a.BN > 128].fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, wmap, xmap);
}

}  // namespace

unsigned int read_mx_matmul_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_qmm_status, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear && v != 0) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(g_qmm_status, &zero, sizeof(zero));
  }
  return v;
}

}  // namespace qmm

extern "C" qmm_status qmm_matmul_mx(const uint32_t* Xq, const uint8_t* x_scales, const uint32_t* Wq,
                                    const uint8_t* w_scales, int M, int N, int K, int format, void* Y, int out_dtype,
                                    void* stream) {
  using namespace qmm;
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0 || M > (1 << 30) || N > (1 << 30)) return QMM_ERR_SHAPE;
  if (format != QMM_MXFP4 && format != QMM_NVFP4) return QMM_ERR_UNSUPPORTED;
  if (out_dtype != QMM_OUT_BF16 && out_dtype != QMM_OUT_F32) return QMM_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return QMM_OK;
  const size_t esize = out_dtype == QMM_OUT_F32 ? 4 : 2;
  if (Y == nullptr) return QMM_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(Y) % esize) return QMM_ERR_ALIGN;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (K == 0)
    return static_cast<qmm_status>(
        finish_call(cudaMemsetAsync(Y, 0, static_cast<size_t>(M) * static_cast<size_t>(N) * esize, st)));
  if (Xq == nullptr || Wq == nullptr || x_scales == nullptr || w_scales == nullptr) return QMM_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(Xq) | reinterpret_cast<uintptr_t>(Wq)) & 15) return QMM_ERR_ALIGN;
  MxMatmulArgs a = {};
  a.xs = x_scales;
  a.ws = w_scales;
  a.Y = Y;
  a.M = M;
  a.N = N;
  a.K = K;
  a.out_f32 = out_dtype == QMM_OUT_F32;
  const cudaError_t e = format == QMM_NVFP4 ? launch_mx_matmul<true>(a, Xq, Wq, st) : launch_mx_matmul<false>(a, Xq, Wq, st);
  return static_cast<qmm_status>(finish_call(e));
}
