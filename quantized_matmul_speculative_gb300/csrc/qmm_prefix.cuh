// Attention of a batch of sequences over a prefix that they share, on the tensor cores
// (qmm_shared_prefix_attention, include/qmm.h).
//
// The work.  For one key-value head the rows of all sequences (new rows x the G query
// heads of the head, without those that do not exist) meet the same keys, so they form
// tiles of 128 rows, and one copy of a key and value tile serves 256 of them.  A segment
// is a pair of row tiles of one head; its prefix is cut into tiles of TN tokens; the
// tiles of all segments form one list, of which every CTA takes an equal, contiguous
// share.  What a CTA leaves of a segment (maximum, sum, unnormalised output of its share)
// is a part; a second kernel adds a row's parts to the sequence's own tokens' attention,
// which the paged kernel (qmm_paged.cuh) has left unrounded.
//
// A CTA.  Two lanes, each a warpgroup with a thread a row, and a row tile of scores and
// of outputs in tensor memory.  In a pair both lanes take every token tile, each with
// rows of its own; a row tile without a partner is both lanes', which take the token
// tiles in turn, so that one lane's exponentials run beside the other's products either
// way.  One thread issues the products, in the order
//   S(0) S(1) | PV(0) S(2) | PV(1) S(3) | ..   of jobs (token tile, lane)
// where job j's scores go to buffer j mod 2, whose probabilities PV(j - 2) has read (the
// tensor cores work in order).  Warps of their own copy keys and values, a ring of pieces:
// by TMA where boxes of 8 tokens divide a page and the cache is bf16, else by 16-byte
// asynchronous copies, which of E4M3 go to a ring of their own and are turned into fp16 by
// further warps.
// D = 256: the outputs of one row tile fill half the tensor memory, so there is one lane,
// with two buffers of scores.
//
// The mathematics.  As in qmm_paged.cuh: s = q.k scale log2(e), p = 2^(s - m), sums and
// outputs in fp32.  m is not the running maximum but follows it where that has grown by
// more than kSlack (a factor 2^kSlack that fp32 has room for), so that the outputs in
// tensor memory are seldom scaled.  Sums are taken a tile at a time, and the tiles' with
// what each addition rounds off; the outputs round in tensor memory after every 16 tokens,
// together less than bf16 does for shares of up to 2^17 tokens.  bf16: p enters the second product as two operands of
// 16 bits together; the probabilities of a chunk of 32 tokens replace its scores, upper
// halves in 16 columns, lower ones in the next 16.  E4M3: as one fp16 operand relative to
// the maximum less kLiftE8 in base 2, so that weights from 2^-25 of the largest on keep 11
// bits and none below 2^-36 remain.
//
// What bounds it.  The products' warp: bf16, 64 x 8 rows of 8 x 4 heads x 128 behind 16384
// tokens take 85 of 148 us with own tokens and joins, a pair of row tiles times 128 tokens
// 4260 cycles, in which it is busy throughout.  A product of scores reads 8 KB of shared
// memory, 64 cycles for 32 of mathematics; one of outputs, whose weights are in tensor memory,
// 4 KB.  E4M3, 48 x 4 rows of 8 x 8 heads x 64 behind 20016: 67 of 104 us, the chain of steps
// between that warp and the lanes; without the exponentials, three quarters of the conversions
// or most copies 103 to 104, with half of the weights 96, with a third buffer of scores or
// with the queries in tensor memory 103.  32 x 1 rows behind 32768: 37 of 73 us, a tile's chain from scores to weights
// to products, 3.6 TB/s.  4 x 1 behind 2048: 9 of 25 us, pages, copies and products in turn.
#pragma once

#include <climits>
#include <type_traits>

#include "qmm_cache.cuh"

namespace qmm {

constexpr int kRows = 128;        // of a tile
constexpr int kLoadWarps = 3;     // (12 warps in all: a thread may have 168 registers, of 13 and more 128)
constexpr int kConvertWarps = 4;  // more for an E4M3 cache
constexpr int kMaxStarts = 400;   // sequences whose first rows a CTA lists; of more, rows that do not exist are computed too
constexpr float kSlack = 8.f, kSlackE8 = 4.f, kLiftE8 = 11.f;

struct PrefixArgs {
  qmm_paged_cache c;
  const int32_t* prefix;  // pages
  int tokens;             // of the prefix
  const uint16_t* q;
  int64_t q_ld;
  int B, M, Hq, G;
  const int32_t* q_lens;
  float scale_log2;       // |scale| log2(e), times k_scale for an E4M3 cache; > 0
  int negate;
  float v_scale;
  int box;                // tokens of a TMA box
  int page_log2;          // of the page size, or -1
  int ctas;
  float4* part_o;         // [parts][lanes][D / 4][128 rows], part: segment + CTA
  float2* part_ml;        // [parts][lanes][128]: (m, sum)
  int* starts;            // [B + 1]: first token row of every sequence
  const float* own_o;     // [B][M][Hq][D], the own tokens' outputs
  const float* own_lse;   // [B][M][Hq]
  __nv_bfloat16* out;
  float* lse;
  unsigned long long wait_ns;
  int inject;
};

template <int D, bool E8>
struct PrefixCfg {
  static constexpr int TN = D == 256 ? 64 : 128;   // tokens of a tile
  static constexpr int LANES = D == 256 ? 1 : 2;
  static constexpr int SLICES = D / 64;            // of 128 bytes of a row
  static constexpr int PIECE = TN * D * 2, QB = kRows * D * 2;
  static constexpr int BARS = 384, MISC = BARS + (kMaxStarts + 1) * 4 + 1024;  // barriers; and starts, alignment
  // an E4M3 cache's pieces as they lie there, on their way to fp16
  static constexpr int RAW = TN * D, RAWS = !E8 ? 0 : D == 64 ? 8 : 4;
  static constexpr int FIT = (232448 - MISC - LANES * QB - RAWS * RAW) / PIECE, SLOTS = FIT > 8 ? 8 : FIT;
  static constexpr int OFF_RAW = SLOTS * PIECE, OFF_Q = OFF_RAW + RAWS * RAW, OFF_BAR = OFF_Q + LANES * QB, OFF_STARTS = OFF_BAR + BARS;
  static constexpr int SMEM = OFF_STARTS + (kMaxStarts + 1) * 4 + 1024;
  static constexpr int WG = 128 * LANES, THREADS = WG + 32 + 32 * kLoadWarps + (E8 ? 32 * kConvertWarps : 0);
  // E4M3, two lanes: of the launch's 512 x 128 registers, 256 x 168 for the threads with rows and 256 x 88 for the others
  static constexpr bool MOVE_REGS = E8 && LANES == 2;
  static constexpr int ROW_REGS = 168, OTHER_REGS = 88;
  static constexpr int O_COL = 256;                // scores in columns 0 .. 2 TN - 1, outputs from 256 on
  static_assert(SLOTS >= 3 && SMEM <= 232448 && O_COL + LANES * D <= 512 && 2 * TN <= O_COL, "room of an SM");
};

// New rows of sequence b that exist (0 where they do not come behind the prefix).
__device__ __forceinline__ int rows_of(const PrefixArgs& a, int b) {
  const int m = new_rows(a.q_lens, b, a.M), n = a.c.lengths[b], own = n - a.tokens;
  return n <= 0 || own < m || own > a.c.max_pages * a.c.page_size ? 0 : m;
}

// How a CTA sees the list.
struct PrefixList {
  int rows, tiles, pairs, tiles_n;  // rows of a head, row tiles, segments of a head, token tiles
  int ctas;                         // with a share: no more than there are units, so that every share holds one
  int units, each, more;            // units of a share; how many of the first shares hold one more
  template <class Cfg>
  static __device__ __forceinline__ PrefixList make(const PrefixArgs& a, int token_rows) {
    PrefixList l;
    l.rows = token_rows * a.G;
    l.tiles = (l.rows + kRows - 1) / kRows;
    l.pairs = (l.tiles + Cfg::LANES - 1) / Cfg::LANES;
    l.tiles_n = (a.tokens + Cfg::TN - 1) / Cfg::TN;
    l.units = a.c.heads * l.pairs * l.tiles_n;
    l.ctas = min(l.units, a.ctas);
    l.each = l.ctas > 0 ? l.units / l.ctas : 0;
    l.more = l.units - l.each * l.ctas;
    return l;
  }
  __device__ __forceinline__ int begin(int cta) const { return cta < ctas ? cta * each + min(cta, more) : units; }
  // the CTA whose share holds unit u
  __device__ __forceinline__ int holder(int u) const {
    const int long_ones = more * (each + 1);
    return u < long_ones ? u / (each + 1) : more + (u - long_ones) / each;
  }
};

// One segment of a CTA's share.
struct PrefixSegment {
  int s, h, pair, kb, ke;  // segment, head, pair of row tiles, token tiles
  bool split;              // one row tile, the token tiles taken in turn (two lanes only)
  __device__ __forceinline__ PrefixSegment(const PrefixList& l, int u, int end, int lanes) {
    s = u / l.tiles_n;
    h = s / l.pairs;
    pair = s - h * l.pairs;
    kb = u - s * l.tiles_n;
    ke = min(l.tiles_n, kb + end - u);
    split = lanes == 2 && 2 * pair + 1 >= l.tiles;
  }
  __device__ __forceinline__ int jobs(int lanes) const { return (ke - kb) * (lanes == 2 && !split ? 2 : 1); }
  // of one lane of two
  __device__ __forceinline__ int lane_jobs(int lane) const { return split ? (ke - kb + 1 - lane) / 2 : ke - kb; }
};

// Sequence of token row tr: the last one that starts at or before it.
__device__ __forceinline__ int sequence_of(const int* starts, int B, int tr) {
  int lo = 0, hi = B;  // starts[lo] <= tr < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= tr) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---- tensor memory and products ----
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lead_bytes, uint32_t stride_bytes) {
  // 128-byte swizzle; leading offset: between slices (read for outputs wider than one), stride: between groups of 8 rows
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>(lead_bytes >> 4) << 16) |
         (static_cast<uint64_t>(stride_bytes >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void mma_commit_to(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld32(float (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]),
        "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]),
        "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float (&v)[32]) {
  uint32_t u[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(v[16 * h + i]);
    tmem_st16(addr + 16 * h, u);
  }
}
__device__ __forceinline__ float exp2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_of3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(v));
  return r;
}
// (x0, x1) = x - (1 - 2^-20) (x's upper 16 bits), as a packed pair.
__device__ __forceinline__ void rest_of(float& x0, float& x1) {
  const uint32_t h0 = __float_as_uint(x0) & 0xFFFF0000u, h1 = __float_as_uint(x1) & 0xFFFF0000u;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n mov.b64 d, {%4, %4};\n"
      " fma.rn.f32x2 a, b, d, a;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x0), "+f"(x1) : "f"(__uint_as_float(h0)), "f"(__uint_as_float(h1)), "f"(-(1.f - 1.f / 1048576.f)));
}
// (x0, x1) = (x0, x1) * f - c as a packed pair.
__device__ __forceinline__ void scale_less(float& x0, float& x1, float f, float c) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %2};\n mov.b64 d, {%3, %3};\n"
      " fma.rn.f32x2 a, a, b, d;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x0), "+f"(x1) : "f"(f), "f"(-c));
}
__device__ __forceinline__ void add_pair(float& s0, float& s1, float x0, float x1) {
  asm("{\n .reg .b64 a, c;\n mov.b64 a, {%0, %1};\n mov.b64 c, {%2, %3};\n add.rn.f32x2 a, a, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(s0), "+f"(s1) : "f"(x0), "f"(x1));
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tma_box(uint32_t dst, const void* tmap, int token, int slice, int head, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      ::"r"(dst), "l"(tmap), "r"(0), "r"(token), "r"(slice), "r"(head), "r"(page), "r"(bar) : "memory");
}
__device__ __forceinline__ void copy_16(uint32_t dst, unsigned long long src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}

// Byte of 16-byte chunk c (of D / 8) of row r in a tile of `rows` rows: slices of 128
// bytes of the rows, chunks permuted as the 128-byte swizzle wants them.
__device__ __forceinline__ uint32_t swizzled(int r, int c, int rows) {
  return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// ---- the roles of a CTA's warps ----
template <int D, bool E8>
struct PrefixRoles {
  using Cfg = PrefixCfg<D, E8>;
  static constexpr int TN = Cfg::TN, LANES = Cfg::LANES, SLOTS = Cfg::SLOTS;
  static constexpr int HALVES = TN / 64;  // of a tile's probabilities, handed over one after the other
  const PrefixArgs& a;
  const PrefixList l;
  unsigned char* smem;
  uint32_t sbase, full, empty, s_full, p_full, q_full, o_full, pv_done, fin, raw_full, raw_empty, tmem;
  const int* starts;
  int begin, end;

  // --- copies ---
  // A tile's boxes along its tokens, 16 at most, one a lane: the entry of the prefix's table and the place in that page.  The
  // entry is looked at when its turn comes, so that it may be on its way until then.
  __device__ __forceinline__ void find_boxes(int t, int& entry, int& place) const {
    const int lane = threadIdx.x & 31, j = t * TN + lane * a.box;
    entry = INT_MIN;  // outside the prefix
    place = 0;
    if (lane * a.box < TN && j < a.tokens) {
      const int block = a.page_log2 >= 0 ? j >> a.page_log2 : j / a.c.page_size;
      place = j - block * a.c.page_size;
      entry = a.prefix[block];
    }
  }
  __device__ __forceinline__ void load_tma(const CUtensorMap* kmap, const CUtensorMap* vmap) {
    // (a warp asks for one box after another, 110 cycles each: the copying warps share them)
    const int lane = threadIdx.x & 31, loader = (threadIdx.x - Cfg::WG - 32) >> 5;
    bool lost = false;
    int it = 0;
    const int groups = TN / a.box, boxes = groups * Cfg::SLICES, groups_log2 = 31 - __clz(groups);  // (box is a power of two)
    int entry = 0, place = 0;
    if (begin < end) find_boxes(PrefixSegment(l, begin, end, LANES).kb, entry, place);
    for (int u = begin; u < end && !lost;) {
      const PrefixSegment g(l, u, end, LANES);
      u += g.ke - g.kb;
      for (int t = g.kb; t < g.ke && !lost; ++t) {
        // the next tile's page numbers are on their way while this one's copies are issued
        int entry2 = 0, place2 = 0;
        if (t + 1 < g.ke || u < end) find_boxes(t + 1 < g.ke ? t + 1 : 0, entry2, place2);
        // (what lies outside the prefix and the cache is outside the tensor and reads as zeros)
        const bool none = entry < 0 || entry >= a.c.num_pages;
        if (none && entry != INT_MIN) bad_page();
        const int page = none ? static_cast<int>(a.c.num_pages) : entry;
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int slot = it % SLOTS;
          if (it >= SLOTS) lost = !mbar_wait(empty + slot * 8, ((it / SLOTS) & 1) ^ 1, kStatusTimeoutEmpty, a.wait_ns);
          lost = __any_sync(0xffffffffu, lost);
          if (lost) break;
          if (loader == 0 && lane == 0) mbar_arrive_expect_tx(full + slot * 8, Cfg::PIECE);
          __syncwarp();
          for (int x0 = 0; x0 < boxes; x0 += 32 * kLoadWarps) {
            const int x = x0 + lane * kLoadWarps + loader, slice = x >> groups_log2, box = x & (groups - 1);
            const int pg = __shfl_sync(0xffffffffu, page, box), pl = __shfl_sync(0xffffffffu, place, box);
            if (x < boxes)
              tma_box(sbase + slot * Cfg::PIECE + slice * TN * 128 + box * a.box * 128, kv ? vmap : kmap, pl, slice, g.h, pg,
                      full + slot * 8);
          }
        }
        entry = entry2;
        place = place2;
      }
    }
    // (the products wait for the same; where one is given up, the limit was time enough for the others)
    for (int i = max(it - SLOTS, 0); i < it; ++i)
      if (__any_sync(0xffffffffu, !mbar_wait(full + i % SLOTS * 8, (i / SLOTS) & 1, kStatusTimeoutDrain, a.wait_ns))) break;
  }

  // A thread's rows of a tile, each STEP-th from r0 on: the prefix's entries (INT_MIN: no token), and the places in their pages.
  template <int N, int STEP>
  struct Rows {
    int page[N], place[N];
    __device__ __forceinline__ void find(const PrefixArgs& a, int t, int r0) {
      const int size = a.c.page_size, j0 = t * TN + r0;
      int block = a.page_log2 >= 0 ? j0 >> a.page_log2 : j0 / size, at = j0 - block * size;
      const int step = a.page_log2 >= 0 ? STEP >> a.page_log2 : STEP / size, rest = STEP - step * size;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        page[i] = r0 + i * STEP < TN && j0 + i * STEP < a.tokens ? a.prefix[block] : INT_MIN;
        place[i] = at;
        block += step;
        at += rest;
        if (at >= size) {
          at -= size;
          ++block;
        }
      }
    }
    __device__ __forceinline__ void offsets(int64_t (&from)[N], int64_t s_page, int64_t s_token) const {
#pragma unroll
      for (int i = 0; i < N; ++i) from[i] = page[i] < 0 ? 0 : page[i] * s_page + place[i] * s_token;
    }
    // Entries that are no pages become -1.
    __device__ __forceinline__ void check(const PrefixArgs& a) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (page[i] < 0 || page[i] >= a.c.num_pages) {
          if (page[i] != INT_MIN) bad_page();
          page[i] = -1;
        }
    }
  };

  // bf16 pages that no box divides: rows by 16-byte asynchronous copies, kLag pieces under way.  The next tile's entries are on
  // their way while this one's copies are issued (looked up one by one: 239 us for 32 x 1 rows behind 32768 pages of a token).
  __device__ __forceinline__ void load_rows() {
    constexpr int CPR = D / 8, STEP = 32 * kLoadWarps / CPR, N = (TN + STEP - 1) / STEP, kLag = 2;  // chunks of a row; rows between a thread's
    const int x = threadIdx.x - Cfg::WG - 32, ch = x % CPR, r0 = x / CPR;
    const bool alike = a.c.k_page == a.c.v_page && a.c.k_token == a.c.v_token && a.c.k_head == a.c.v_head;
    Rows<N, STEP> next;
    uint32_t to[N];  // in a piece
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = swizzled(r0 + i * STEP, ch, TN);
    bool lost = false;
    int it = 0;
    if (begin < end) next.find(a, PrefixSegment(l, begin, end, LANES).kb, r0);
    for (int u = begin; u < end && !lost;) {
      const PrefixSegment g(l, u, end, LANES);
      u += g.ke - g.kb;
      for (int t = g.kb; t < g.ke && !lost; ++t) {
        Rows<N, STEP> rows = next;
        rows.check(a);
        if (t + 1 < g.ke || u < end) next.find(a, t + 1 < g.ke ? t + 1 : 0, r0);
        int64_t from[N];
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int slot = it % SLOTS;
          if (it >= SLOTS) lost = !mbar_wait(empty + slot * 8, ((it / SLOTS) & 1) ^ 1, kStatusTimeoutEmpty, a.wait_ns);
          if (lost) break;
          if (kv == 0 || !alike) rows.offsets(from, (kv ? a.c.v_page : a.c.k_page) * 2, (kv ? a.c.v_token : a.c.k_token) * 2);
          const unsigned long long cache =
              reinterpret_cast<unsigned long long>(kv ? a.c.v : a.c.k) + (g.h * (kv ? a.c.v_head : a.c.k_head) + ch * 8) * 2;
          const uint32_t piece = sbase + slot * Cfg::PIECE;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (r0 + i * STEP < TN) copy_16(piece + to[i], cache + from[i], rows.page[i] >= 0);
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (it >= kLag) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
            fence_async_shared();
            mbar_arrive(full + (it - kLag) % SLOTS * 8);
          }
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    fence_async_shared();
    if (!lost)
      for (int i = max(it - kLag, 0); i < it; ++i) mbar_arrive(full + i % SLOTS * 8);
  }

  // E4M3: rows by 16-byte asynchronous copies to the ring of raw pieces, whatever the page size (boxes of 8 tokens took a warp
  // 110 cycles each to ask for).
  static __device__ __forceinline__ uint32_t raw_at(int r, int ch) {
    return D == 64 ? r * 64 + ((ch ^ ((r >> 1) & 3)) << 4) : (ch >> 3) * TN * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
  }
  __device__ __forceinline__ void copy_raw() {
    constexpr int CPR = D / 16, STEP = 32 * kLoadWarps / CPR, N = (TN + STEP - 1) / STEP;
    const int x = threadIdx.x - Cfg::WG - 32, ch = x % CPR, r0 = x / CPR;
    Rows<N, STEP> next;
    bool lost = false;
    int it = 0;
    if (begin < end) next.find(a, PrefixSegment(l, begin, end, LANES).kb, r0);
    for (int u = begin; u < end && !lost;) {
      const PrefixSegment g(l, u, end, LANES);
      u += g.ke - g.kb;
      for (int t = g.kb; t < g.ke && !lost; ++t) {
        Rows<N, STEP> rows = next;
        rows.check(a);
        // (the next tile's entries are on their way while this one's copies are issued)
        if (t + 1 < g.ke || u < end) next.find(a, t + 1 < g.ke ? t + 1 : 0, r0);
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int slot = it % Cfg::RAWS;
          if (it >= Cfg::RAWS) lost = !mbar_wait(raw_empty + slot * 8, ((it / Cfg::RAWS) & 1) ^ 1, kStatusTimeoutEmpty, a.wait_ns);
          if (lost) break;
          const unsigned long long cache = reinterpret_cast<unsigned long long>(kv ? a.c.v : a.c.k) + ch * 16;
          const int64_t s_page = kv ? a.c.v_page : a.c.k_page, s_token = kv ? a.c.v_token : a.c.k_token,
                        head = g.h * (kv ? a.c.v_head : a.c.k_head);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int r = r0 + i * STEP;
            if (r < TN)
              copy_16(sbase + Cfg::OFF_RAW + slot * Cfg::RAW + raw_at(r, ch),
                      cache + (rows.page[i] >= 0 ? rows.page[i] * s_page + rows.place[i] * s_token + head : 0), rows.page[i] >= 0);
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(raw_full + slot * 8) : "memory");
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  // Raw pieces to fp16, by warps of their own.
  __device__ __forceinline__ void convert() {
    constexpr int CPR = D / 16, STEP = 32 * kConvertWarps / CPR;
    const int x = threadIdx.x - Cfg::WG - 32 - 32 * kLoadWarps, ch = x % CPR, r0 = x / CPR, lane = threadIdx.x & 31;
    const int pieces = 2 * (end - begin);
    for (int it = 0; it < pieces; ++it) {
      const int from = it % Cfg::RAWS, to = it % SLOTS;
      bool lost = !mbar_wait(raw_full + from * 8, (it / Cfg::RAWS) & 1, kStatusTimeoutFull, a.wait_ns);
      if (it >= SLOTS) lost = lost || !mbar_wait(empty + to * 8, ((it / SLOTS) & 1) ^ 1, kStatusTimeoutEmpty, a.wait_ns);
      if (__any_sync(0xffffffffu, lost)) return;
      const unsigned char* const raw = smem + Cfg::OFF_RAW + from * Cfg::RAW;
      unsigned char* const piece = smem + to * Cfg::PIECE;
#pragma unroll
      for (int r = r0; r < TN; r += STEP) {
        const uint4 u = *reinterpret_cast<const uint4*>(raw + raw_at(r, ch));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint4 o[2];
        o[0] = make_uint4(e4m3x2_f16x2(w[0]), e4m3x2_f16x2(w[0] >> 16), e4m3x2_f16x2(w[1]), e4m3x2_f16x2(w[1] >> 16));
        o[1] = make_uint4(e4m3x2_f16x2(w[2]), e4m3x2_f16x2(w[2] >> 16), e4m3x2_f16x2(w[3]), e4m3x2_f16x2(w[3] >> 16));
        // (of a row's two slices, which lie in the same banks, one half's chunks are stored in the other order)
        const int odd = (ch >> 2) & 1;
        *reinterpret_cast<uint4*>(piece + swizzled(r, 2 * ch + odd, TN)) = odd ? o[1] : o[0];
        *reinterpret_cast<uint4*>(piece + swizzled(r, 2 * ch + 1 - odd, TN)) = odd ? o[0] : o[1];
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(raw_empty + from * 8);
        mbar_arrive(full + to * 8);
      }
    }
  }

  // --- products: one warp, whose loop is uniform (the products' descriptors are made in uniform registers) and of which
  // one thread issues them (with all of it in that thread's branch a product took 112 cycles to issue, and 64 to do).  A
  // job's way through this warp is on both lanes' path, so that it is kept short: slots and phases are counted, not
  // computed, and a wait that is over costs one test. ---
  struct Place {  // of the next key (or value) piece
    int slot;
    uint32_t phase;
    __device__ __forceinline__ void next() {  // they take turns
      slot += 2;
      if (slot >= SLOTS) {
        slot -= SLOTS;
        phase ^= 1;
      }
    }
  };
  static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t phase, unsigned long long wait_ns) {
    return mbar_wait(bar, phase, kStatusTimeoutFull, wait_ns);
  }
  __device__ __forceinline__ void multiply() {
    constexpr uint32_t kType = E8 ? 0u : 1u;  // fp16 or bf16 operands, fp32 sums
    constexpr uint32_t kS = (1u << 4) | (kType << 7) | (kType << 10) | ((TN >> 3) << 17) | ((kRows >> 4) << 24);
    constexpr uint32_t kPV = (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) | ((D >> 3) << 17) | ((kRows >> 4) << 24);
    const bool leader = elect_one();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t q_desc = tile_desc(sbase + Cfg::OFF_Q, 16, 1024), k_desc = tile_desc(sbase, 16, 1024),
                   v_desc = tile_desc(sbase, TN * 128, 1024);
    bool lost = false;  // after a wait that gave up nothing more is issued or waited for
    Place key = {0, 0}, value = {1, 0};
    uint32_t p_phase = 0;     // of the buffers' next probabilities, a bit each
    uint32_t q_phase = 0;     // of the lanes' next query tiles
    auto wait = [&](uint32_t bar, uint32_t phase) {
      if (!lost && !mbar_try_wait(bar, phase & 1, 20000u)) lost = !wait_long(bar, phase & 1, a.wait_ns);
    };
    auto commit = [&](uint32_t bar) {
      if (leader && !lost) mma_commit_to(bar);
    };
    // PV(i) of a segment of J jobs; jobs of buffer BUF.  In a pair both lanes use a piece, else one job.
    auto second = [&](auto buf_of, bool pair, int i, int J) {
      constexpr int BUF = decltype(buf_of)::value, O = LANES == 2 ? BUF : 0;
      const bool first_use = !pair || BUF == 0, last_use = !pair || BUF == 1;
      if (first_use) wait(full + value.slot * 8, value.phase);
      const uint64_t v = v_desc + value.slot * (Cfg::PIECE >> 4);
      const uint32_t p = tm + BUF * TN, d = tm + Cfg::O_COL + O * D;
      const bool more = i >= LANES;
#pragma unroll
      for (int half = 0; half < HALVES; ++half) {
        wait(p_full + (BUF * 2 + half) * 8, p_phase >> BUF);
        tmem_after();
        if (leader && !lost) {
#pragma unroll
          for (int x = half * 4; x < half * 4 + 4; ++x) {
            mma_ts(d, p + (x >> 1) * 32 + (x & 1) * 8, v + x * (2048 >> 4), kPV, x > 0 || more);
            if constexpr (!E8) mma_ts(d, p + (x >> 1) * 32 + (x & 1) * 8 + 16, v + x * (2048 >> 4), kPV, true);
          }
        }
      }
      p_phase ^= 1u << BUF;
      if (last_use) {
        commit(empty + value.slot * 8);
        value.next();
      }
      if (LANES == 1) commit(pv_done);
      if (i + LANES >= J) commit(o_full + O * 8);
    };
    // S(j)
    auto first = [&](auto buf_of, bool pair, int j) {
      constexpr int BUF = decltype(buf_of)::value, O = LANES == 2 ? BUF : 0;
      const bool first_use = !pair || BUF == 0, last_use = !pair || BUF == 1;
      if (first_use) wait(full + key.slot * 8, key.phase);
      if (j < LANES) {
        wait(q_full + O * 8, q_phase >> O);
        q_phase ^= 1u << O;
      }
      // (no fence: the operands are in shared memory, and PV(j - 2), issued after one, has read what lies in the buffer)
      const uint64_t k = k_desc + key.slot * (Cfg::PIECE >> 4), q = q_desc + O * (Cfg::QB >> 4);
      if (leader && !lost) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          mma_ss(tm + BUF * TN, q + (((x >> 2) * kRows * 128 + (x & 3) * 32) >> 4), k + (((x >> 2) * TN * 128 + (x & 3) * 32) >> 4),
                 kS, x > 0);
      }
      if (last_use) {
        commit(empty + key.slot * 8);
        key.next();
      }
      commit(s_full + BUF * 8);
    };
    for (int u = begin; u < end;) {
      const PrefixSegment g(l, u, end, LANES);
      u += g.ke - g.kb;
      const int J = g.jobs(LANES);
      const bool pair = LANES == 2 && !g.split;
      // S(j) for j < J, after PV(j - 2); then the last two
#pragma unroll 1
      for (int j = 0; j < J + 2; j += 2) {
        if (j >= 2) second(std::integral_constant<int, 0>{}, pair, j - 2, J);
        if (j < J) first(std::integral_constant<int, 0>{}, pair, j);
        if (j >= 2 && j - 1 < J) second(std::integral_constant<int, 1>{}, pair, j - 1, J);
        if (j + 1 < J) first(std::integral_constant<int, 1>{}, pair, j + 1);
      }
    }
    // all products are done before the tensor memory is given back
    if (leader) mma_commit_to(fin);
    mbar_wait(fin, 0, kStatusTimeoutDrain, a.wait_ns);
  }

  // --- rows: queries, probabilities, outputs; a thread a row ---
  __device__ __forceinline__ float load_query(const PrefixSegment& g, int lane, int row) {
    const int r = (LANES == 2 ? (g.split ? 2 * g.pair : 2 * g.pair + lane) : g.pair) * kRows + row;
    const uint16_t* src = nullptr;
    if (r < l.rows) {
      const int tr = r / a.G;
      int at = tr;  // of the B x M rows
      if (a.B <= kMaxStarts) {
        const int b = sequence_of(starts, a.B, tr);
        at = b * a.M + tr - starts[b];
      }
      src = a.q + at * a.q_ld + static_cast<int64_t>(g.h * a.G + r - tr * a.G) * D;
    }
    unsigned char* const tile = smem + Cfg::OFF_Q + lane * Cfg::QB;
    const uint32_t flip = a.negate ? 0x80008000u : 0u;
    float scale = a.scale_log2, f = 1.f;
    if constexpr (E8) {
      // fp16, scaled by a power of two so that the row's largest element lies in [2^14, 2^15); 0, tiny and infinite rows stay
      float top = 0.f;
      if (src != nullptr)
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = ld_after_wait_v4(src + c * 8);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
        }
      const int e = static_cast<int>(__float_as_uint(top) >> 23), up = (e < 30 || e == 255) ? 0 : 14 + 127 - e;
      f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
      scale = fmaxf(scale * __uint_as_float(static_cast<uint32_t>(127 - up) << 23), 1e-30f);
    }
#pragma unroll 8
    for (int c = 0; c < D / 8; ++c) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (src != nullptr) {
        x = ld_after_wait_v4(src + c * 8);
        x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
        if constexpr (E8)
          x = make_uint4(f16x2_of(bf16_lo(x.x) * f, bf16_hi(x.x) * f), f16x2_of(bf16_lo(x.y) * f, bf16_hi(x.y) * f),
                         f16x2_of(bf16_lo(x.z) * f, bf16_hi(x.z) * f), f16x2_of(bf16_lo(x.w) * f, bf16_hi(x.w) * f));
      }
      *reinterpret_cast<uint4*>(tile + swizzled(row, c, kRows)) = x;
    }
    fence_async_shared();
    mbar_arrive(q_full + lane * 8);
    return scale;
  }

  // The scores of the 32 columns from c on that are tokens, the others -inf.
  __device__ __forceinline__ static void cut(float (&x)[32], int c, int valid) {
    if (valid < c + 32)
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i >= valid) x[i] = -INFINITY;
  }
  // 32 scores to probabilities, to the columns that held the scores; their sums.
  __device__ __forceinline__ static void weigh(float (&x)[32], uint32_t at, float scale, float base, float& sum0, float& sum1) {
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      scale_less(x[2 * i], x[2 * i + 1], scale, base);
      x[2 * i] = exp2_of(x[2 * i]);
      x[2 * i + 1] = exp2_of(x[2 * i + 1]);
      add_pair(sum0, sum1, x[2 * i], x[2 * i + 1]);
      if constexpr (E8) p[i] = f16x2_of(x[2 * i], x[2 * i + 1]);
      else p[i] = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
    }
    tmem_st16(at, p);
    if constexpr (!E8) {
      // The upper half of a probability goes in as it is, the rest as a second operand: x - hi (1 - 2^-20), which is 0 for x = 0
      // alone, so that an infinite value times it is that infinity and not NaN; the 2^-20 of x is below the 16 bits' own rounding.
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        rest_of(x[2 * i], x[2 * i + 1]);
        p[i] = bf16x2_of(x[2 * i], x[2 * i + 1]);
      }
      tmem_st16(at + 16, p);
    }
  }

  __device__ __forceinline__ void rows() {
    const int lane = threadIdx.x >> 7, row = threadIdx.x & 127;
    const uint32_t mine = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;  // this warp's quarter of the tensor memory's lanes
    const uint32_t o_at = tmem + Cfg::O_COL + lane * D + mine;
    bool lost = false;
    int n_jobs = 0;            // of this lane so far
    int n_o = 0, n_other = 0;  // segments with jobs of this lane, and of the other one
    uint32_t phases = 0;       // one lane's buffers of scores
    auto wait = [&](uint32_t bar, int phase) {
      if (!lost) lost = __any_sync(0xffffffffu, !mbar_wait(bar, phase & 1, kStatusTimeoutFull, a.wait_ns));
      tmem_after();
    };
    auto jobs_of = [&](const PrefixSegment& g, int x) { return LANES == 2 ? g.lane_jobs(x) : g.ke - g.kb; };
    float scale = 0.f;
    if (begin < end) {
      const PrefixSegment g(l, begin, end, LANES);
      if (jobs_of(g, lane) > 0) scale = load_query(g, lane, row);
    }
    for (int u = begin; u < end;) {
      const PrefixSegment g(l, u, end, LANES);
      u += g.ke - g.kb;
      const int jobs = jobs_of(g, lane);
      float m = -INFINITY, sum = 0.f, rest = 0.f;  // what the sum was rounded by
#pragma unroll 1
      for (int j = 0; j < jobs; ++j) {
        const int buf = LANES == 2 ? lane : j & 1;
        const int t = LANES == 2 && g.split ? g.kb + 2 * j + lane : g.kb + j;
        const int valid = a.tokens - t * TN;  // of the tile's columns, if fewer than TN
        const uint32_t s_at = tmem + buf * TN + mine;
        wait(s_full + buf * 8, LANES == 2 ? n_jobs : phases >> buf);
        phases ^= 1u << buf;
        if (lost) break;
        // The row's largest score, then its probabilities, 64 columns at a time, which are read twice (with all 128 in registers,
        // or with half of them kept, some of those were spilled).
        float x0[32], x1[32];
        float top = -INFINITY, top1 = -INFINITY;
        auto scores = [&](int c) {
          tmem_ld32(x0, s_at + c);
          tmem_ld32(x1, s_at + c + 32);
          tmem_loaded();
          if (valid < TN) {
            cut(x0, c, valid);
            cut(x1, c + 32, valid);
          }
        };
#pragma unroll 1
        for (int c = 0; c < TN; c += 64) {
          scores(c);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            top = max_of3(top, x0[i], x0[i + 1]);
            top1 = max_of3(top1, x1[i], x1[i + 1]);
          }
        }
        top = fmaxf(top, top1) * scale;
        const float want = E8 ? top - kLiftE8 : top;
        const bool grown = want > m + (E8 ? kSlackE8 : kSlack) || m == -INFINITY;
        float f = 1.f;
        if (grown) {
          f = exp2_of(m - (want == -INFINITY ? 0.f : want));
          m = want;
        }
        const float base = m == -INFINITY ? 0.f : m;
        const bool again = j > 0 && __any_sync(0xffffffffu, f != 1.f);
        if (again) {
          sum *= f;
          rest *= f;
          if (LANES == 1) wait(pv_done, n_jobs - 1);  // (of two lanes, the one's products end before its next scores)
          float y[32];
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            tmem_ld32(y, o_at + c);
            tmem_loaded();
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] *= f;
            tmem_st32(o_at + c, y);
          }
        }
        // 64 columns' probabilities at a time, so that the products with the first begin beside the second
        float sum0 = 0.f, sum1 = 0.f;  // of the tile
#pragma unroll 1
        for (int half = 0; half < HALVES; ++half) {
          const int c = half * 64;
          scores(c);
          weigh(x0, s_at + c, scale, base, sum0, sum1);
          weigh(x1, s_at + c + 32, scale, base, sum0, sum1);
          tmem_stored();
          tmem_before();
          __syncwarp();
          if ((threadIdx.x & 31) == 0) mbar_arrive(p_full + (buf * 2 + half) * 8);
        }
        ++n_jobs;
        // (A share may be tens of thousands of tokens.  In one chain of sums those below 2^-24 of a leading one were lost: the
        // log-sum-exp was 6.8e-4 off behind 32768 of e^-17 each, and is 3.4e-6, at the same time a tile.)
        const float tile = sum0 + sum1 + rest, all = sum + tile;
        rest = tile - (all - sum);
        sum = all;
      }
      // the next segment's queries, whose scores may begin beside this one's end
      if (u < end) {
        const PrefixSegment next(l, u, end, LANES);
        if (jobs_of(next, lane) > 0 && !lost) scale = load_query(next, lane, row);
      }
      const bool both = LANES == 2 && g.split;
      if (!both) {
        const int64_t part = (static_cast<int64_t>(g.s) + blockIdx.x) * LANES + lane;
        wait(o_full + lane * 8, n_o);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float x[32];
          tmem_ld32(x, o_at + c);
          tmem_loaded();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            a.part_o[(part * (D / 4) + c / 4 + i) * kRows + row] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
        a.part_ml[part * kRows + row] = make_float2(m, sum);
      } else {
        // one part of both lanes' outputs, which lie in the same lanes of tensor memory: a lane adds half of the columns
        const int64_t part = (static_cast<int64_t>(g.s) + blockIdx.x) * LANES;
        a.part_ml[(part + lane) * kRows + row] = make_float2(m, sum);  // (shared memory is full)
        __threadfence_block();
        asm volatile("barrier.sync 1, 256;" ::: "memory");
        const float2 other = __ldcg(&a.part_ml[(part + (lane ^ 1)) * kRows + row]);
        const bool second = g.lane_jobs(1) > 0;
        wait(o_full, lane == 0 ? n_o : n_other);
        if (second) wait(o_full + 8, lane == 0 ? n_other : n_o);
        const float top = fmaxf(m, other.x), ref = top == -INFINITY ? 0.f : top;
        const float f_mine = exp2_of(m - ref), f_other = exp2_of(other.x - ref);
        const float f0 = lane == 0 ? f_mine : f_other, f1 = lane == 0 ? f_other : f_mine;
        const uint32_t at = tmem + Cfg::O_COL + mine + lane * (D / 2);
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
          float x[32], y[32];
          tmem_ld32(x, at + c);
          if (second) tmem_ld32(y, at + D + c);
          tmem_loaded();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            x[i] *= f0;
            if (second) x[i] = fmaf(y[i], f1, x[i]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            a.part_o[(part * (D / 4) + lane * (D / 8) + c / 4 + i) * kRows + row] =
                make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
        asm volatile("barrier.sync 1, 256;" ::: "memory");  // both have read both
        if (lane == 0) a.part_ml[part * kRows + row] = make_float2(top, fmaf(sum, f_mine, other.y * f_other));
      }
      n_o += jobs > 0;
      if (LANES == 2) n_other += g.lane_jobs(lane ^ 1) > 0;
      tmem_before();
    }
  }
};

// BOXES: bf16 pages that TMA boxes divide.
template <int D, bool E8, bool BOXES>
__global__ void __launch_bounds__(PrefixCfg<D, E8>::THREADS, 1)
prefix_kernel(const PrefixArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using Cfg = PrefixCfg<D, E8>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const uint32_t full = sbase + Cfg::OFF_BAR, empty = full + Cfg::SLOTS * 8, s_full = empty + Cfg::SLOTS * 8, p_full = s_full + 16,
                 q_full = p_full + 32, o_full = q_full + 16, pv_done = o_full + 16, fin = pv_done + 8;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_BAR + Cfg::SLOTS * 16 + 96);
  const uint32_t raw_full = sbase + Cfg::OFF_BAR + Cfg::SLOTS * 16 + 112, raw_empty = raw_full + Cfg::RAWS * 8;
  int* const starts = reinterpret_cast<int*>(smem + Cfg::OFF_STARTS);
  int* const s_sum = reinterpret_cast<int*>(smem + Cfg::OFF_Q);  // (before the queries)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::SLOTS; ++s) {
      mbar_init(full + s * 8, E8 ? kConvertWarps : BOXES ? 1 : 32 * kLoadWarps);
      mbar_init(empty + s * 8, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i * 8, 1);
      mbar_init(p_full + i * 16, 4);
      mbar_init(p_full + i * 16 + 8, 4);
      mbar_init(q_full + i * 8, 128);
      mbar_init(o_full + i * 8, 1);
    }
    mbar_init(pv_done, 1);
    mbar_init(fin, 1);
    for (int s = 0; s < Cfg::RAWS; ++s) {
      mbar_init(raw_full + s * 8, 32 * kLoadWarps);
      mbar_init(raw_empty + s * 8, kConvertWarps);
    }
    fence_mbar_init();
    if (a.inject && blockIdx.x == 0) mbar_expect_tx(E8 ? raw_full : full, 16);
  }
  if (warp == Cfg::WG / 32) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  griddep_wait();
  griddep_launch_dependents();
  // the sequences' first token rows
  int token_rows = a.B * a.M;
  if (a.B <= kMaxStarts) {
    // (a thread takes neighbouring sequences, at most two)
    constexpr int kPer = (kMaxStarts + Cfg::THREADS - 1) / Cfg::THREADS;
    int m[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = threadIdx.x * kPer + i;
      m[i] = b < a.B ? rows_of(a, b) : 0;
      mine += m[i];
    }
    int inc = mine;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, inc, s);
      if (lane >= s) inc += o;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    int before = inc - mine;
    for (int w = 0; w < warp; ++w) before += s_sum[w];
    token_rows = 0;
    for (int w = 0; w < Cfg::THREADS / 32; ++w) token_rows += s_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = threadIdx.x * kPer + i;
      if (b < a.B) {
        starts[b] = before;
        if (blockIdx.x == 0) a.starts[b] = before;
      }
      before += m[i];
    }
    if (threadIdx.x == 0) {
      starts[a.B] = token_rows;
      if (blockIdx.x == 0) a.starts[a.B] = token_rows;
    }
  } else if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b <= a.B; b += Cfg::THREADS) a.starts[b] = b * a.M;
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = *tmem_slot;
  const PrefixList l = PrefixList::make<Cfg>(a, token_rows);
  PrefixRoles<D, E8> r{a, l, smem, sbase, full, empty, s_full, p_full, q_full, o_full, pv_done, fin, raw_full, raw_empty, tmem, starts,
                       l.begin(blockIdx.x), l.begin(blockIdx.x + 1)};
  if constexpr (Cfg::MOVE_REGS) {
    static_assert(256 * Cfg::ROW_REGS + 256 * Cfg::OTHER_REGS <= 512 * 128 && Cfg::THREADS == 512, "registers of the launch");
    if (warp < Cfg::WG / 32) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::ROW_REGS));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::OTHER_REGS));
  }
  if (warp < Cfg::WG / 32) {
    r.rows();
  } else if (warp == Cfg::WG / 32) {
    r.multiply();
  } else if constexpr (E8) {
    if (warp <= Cfg::WG / 32 + kLoadWarps) r.copy_raw();
    else r.convert();
  } else if constexpr (BOXES) {
    r.load_tma(&kmap, &vmap);
  } else {
    r.load_rows();
  }
  __syncwarp();
  tmem_before();
  __syncthreads();
  tmem_after();
  if (warp == Cfg::WG / 32) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// Adds a row's parts and its own tokens' share, in the order of the list.  A CTA takes a
// head and a few neighbouring rows of the B x M x G of it, a thread four of their columns.
constexpr int kPrefixJoinThreads = 256;
// AHEAD parts are under way at a time: 4 where many CTAs cover for each other, 8 where the
// CTAs are few (64 x 8 rows, 5 parts: 11.8 us with 4, 14.4 with 8; 32 x 1 rows, 20 parts:
// 11.7 and 8.4).  Where they are fewer than the SMs, SPLIT threads share a row's parts, which
// are then added in order (32 x 1: 6.5 us, 2 x 16 of 5 heads, 76 parts: 8 us, and 13.2
// without; but 9 x 16 of 7 heads, a part each: 8.8 and 5.2).
template <int D, bool E8, int SPLIT, int AHEAD>
__global__ void __launch_bounds__(kPrefixJoinThreads) prefix_join_kernel(const PrefixArgs a) {
  using Cfg = PrefixCfg<D, E8>;
  constexpr int COLS = D / 4, ROWS = kPrefixJoinThreads / COLS / SPLIT;
  // where the CTA's rows are: place among the B x M x q_heads (-1: none), their first part (that lane's), how many, row there
  __shared__ int64_t s_at[ROWS], s_part[ROWS];
  __shared__ int s_parts[ROWS], s_row[ROWS];
  __shared__ bool s_real[ROWS];
  __shared__ float4 s_acc[SPLIT][SPLIT > 1 ? ROWS * COLS : 1];
  __shared__ float2 s_sum[SPLIT][SPLIT > 1 ? ROWS * COLS : 1];
  griddep_wait();
  griddep_launch_dependents();
  if (threadIdx.x < ROWS) {
    const int all = a.B * a.M * a.G, blocks = (all + ROWS - 1) / ROWS;
    const int h = blockIdx.x / blocks, x = (blockIdx.x - h * blocks) * ROWS + threadIdx.x;
    const int tr = x / a.G, b = tr / a.M, i = tr - b * a.M;
    s_at[threadIdx.x] = x < all ? static_cast<int64_t>(tr) * a.Hq + h * a.G + x - tr * a.G : -1;
    s_parts[threadIdx.x] = 0;
    const bool real = x < all && i < rows_of(a, b);
    s_real[threadIdx.x] = real;
    if (real && a.tokens > 0) {
      const PrefixList l = PrefixList::make<Cfg>(a, a.starts[a.B]);
      const int r = (a.starts[b] + i) * a.G + x - tr * a.G;
      const int tile = r / kRows, pair = tile / Cfg::LANES, s = h * l.pairs + pair, u0 = s * l.tiles_n;
      const int first = l.holder(u0);
      const bool split = Cfg::LANES == 2 && 2 * pair + 1 >= l.tiles;
      s_part[threadIdx.x] = (static_cast<int64_t>(s) + first) * Cfg::LANES + (Cfg::LANES == 2 && !split ? tile & 1 : 0);
      s_parts[threadIdx.x] = l.holder(u0 + l.tiles_n - 1) - first + 1;
      s_row[threadIdx.x] = r - tile * kRows;
    }
  }
  __syncthreads();
  const int place = threadIdx.x % (ROWS * COLS), turn = threadIdx.x / (ROWS * COLS);
  const int mine = place % ROWS, col = place / ROWS;
  const int64_t at = s_at[mine];
  const bool real = at >= 0 && s_real[mine];
  // running maximum, sum and output over the row's parts, some under way at a time
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float top = -INFINITY, sum = 0.f;
  if (real) {
    if (turn == 0) {
      const float own_lse = a.own_lse[at];
      const float4 own = reinterpret_cast<const float4*>(a.own_o)[at * COLS + col];
      top = own_lse * 1.4426950408889634f;
      sum = own_lse == -INFINITY ? 0.f : 1.f;
      if (sum != 0.f) acc = own;
    }
    const int parts = s_parts[mine], r = s_row[mine];
    const int64_t p0 = s_part[mine];
    for (int p = turn * AHEAD; p < parts; p += SPLIT * AHEAD) {
      float2 ml[AHEAD];
      float4 v[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p + k < parts) {
          const int64_t at_part = p0 + (p + k) * Cfg::LANES;
          ml[k] = a.part_ml[at_part * kRows + r];
          v[k] = a.part_o[(at_part * COLS + col) * kRows + r];
        }
      }
      float t = top;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) t = fmaxf(t, ml[k].x);
      const float ref = t == -INFINITY ? 0.f : t, f = exp2_of(top - ref);
      top = t;
      sum *= f;
      acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (p + k >= parts) break;
        const float g = exp2_of(ml[k].x - ref), gv = g * a.v_scale;  // (what the own tokens' outputs have been scaled by already)
        sum += g * ml[k].y;
        acc.x += gv * v[k].x, acc.y += gv * v[k].y, acc.z += gv * v[k].z, acc.w += gv * v[k].w;
      }
    }
  }
  if constexpr (SPLIT > 1) {
    s_acc[turn][place] = acc;
    s_sum[turn][place] = make_float2(top, sum);
    __syncthreads();
    if (turn != 0) return;
    float2 ml[SPLIT];
#pragma unroll
    for (int k = 0; k < SPLIT; ++k) {
      ml[k] = s_sum[k][place];
      top = fmaxf(top, ml[k].x);
    }
    const float ref = top == -INFINITY ? 0.f : top;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < SPLIT; ++k) {
      const float g = exp2_of(ml[k].x - ref);
      const float4 v = s_acc[k][place];
      if (ml[k].y == 0.f) continue;
      sum += g * ml[k].y;
      acc.x += g * v.x, acc.y += g * v.y, acc.z += g * v.z, acc.w += g * v.w;
    }
  }
  if (at < 0) return;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float lse = -INFINITY;
  if (sum != 0.f) {
    const float f = 1.f / sum;
    o = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    lse = (top + log2f(sum)) * 0.6931471805599453f;
  }
  *reinterpret_cast<uint2*>(a.out + at * D + col * 4) = make_uint2(bf16x2_of(o.x, o.y), bf16x2_of(o.z, o.w));
  if (col == 0 && a.lse != nullptr) a.lse[at] = lse;
}

// Segments of a call at most, whatever exists of its rows.
inline int64_t prefix_segments(int64_t rows, int heads, int D) {
  const int64_t tiles = (rows + kRows - 1) / kRows;
  return heads * (D == 256 ? tiles : (tiles + 1) / 2);
}

// Launchers of one head size (qmm_prefix_inst.cu).
template <int D>
cudaError_t launch_prefix(const PrefixArgs& a, bool e8, cudaStream_t stream);
template <int D>
cudaError_t launch_prefix_join(const PrefixArgs& a, bool e8, cudaStream_t stream);
template <int D>
unsigned int read_prefix_unit(int clear);

}  // namespace qmm
