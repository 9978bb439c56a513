// Paged attention over a split list of key-value tiles, and the join of the
// parts (definition in include/qmm.h, qmm_paged_attention).
//
// The work.  A segment is one (sequence, key-value head, block of query rows):
// its rows are the new rows x the G query heads of the key-value head, so one
// pass over the keys and values serves 16 or 32 of them.  A segment's visible
// tokens are cut into tiles; the tiles of all segments form one list (sequence,
// head, row block, tile order), and every warp of the grid is a worker with an
// equal, contiguous share of it, whatever the lengths: a single long sequence
// is split over all SMs, a batch of ragged ones is balanced, and no warp waits
// for another.  A segment that one worker finishes is written directly; the
// others leave (maximum, sum, unnormalised output) of their share in the
// workspace, which join_kernel combines in list order.
//
// A worker streams its own tiles: a ring of SLOTS pieces (the keys of a tile,
// its values, the next tile's keys, ..), each refilled by TMA as soon as the
// warp has read it.
//
// The mathematics.  One pass with running maximum m and sum l per row, in
// base-2 exponents: s = q.k scale log2(e), p = 2^(s - m'), o = o 2^(m - m') +
// p v, l likewise; o / l and (m + log2 l) ln 2 at the end.  An E4M3 cache's m is
// the maximum less kLift: weights go up to 2^15 then, the upper end of the fp16
// that they enter the second product in, so that those down to 2^-29 of the
// row's largest keep 11 bits and only those below 2^-40 vanish (2^-14 and 2^-25
// without: many tokens far below one vanished from o and not from l).
//
// What bounds it: a worker's chain load -> scores -> maximum -> weights ->
// output products, a tile at a time, with two or three warps a scheduler to
// cover it; then the start (lengths, table, first pieces: about 5 us) and the
// join.  One row over 65001 tokens, 8 heads x 128 in bf16: 66 us, 4.0 TB/s;
// 32 ragged sequences x 8 rows: 154 us, 3.5 TB/s; 16 x 4 rows, a window of
// 4096 tokens, 8 x 64 in E4M3: 57 us; 4 short sequences: 13.6 us.
#pragma once

#include <cudaTypedefs.h>

#include <climits>
#include <type_traits>

#include "../../include/qmm.h"
#include "qmm_cache.cuh"

namespace qmm {

constexpr int kJoinThreads = 128;
constexpr int kMaxWorkers = 12;  // of a CTA, at most
constexpr float kLift = 15.f;

struct AttentionArgs {
  qmm_paged_cache c;
  const uint16_t* q;
  int64_t q_ld;
  int B, M, Hq, G;  // G = Hq / c.heads
  const int32_t* q_lens;
  float scale_log2;  // |scale| log2(e), times k_scale for an E4M3 cache; > 0
  int negate;        // the queries' signs are flipped (a negative scale)
  float v_scale;
  int window, sinks;
  __nv_bfloat16* out;
  float* out32;      // behind a prefix the outputs go there, unrounded
  float* lse;
  int skip;          // tokens of that prefix, which the lengths count
  int box;        // tokens of a TMA box (8 or 16); 0: copied row by row
  int page_log2;  // of the page size, or -1
  int RB, RT;     // rows of a row block (16 or 32), row blocks of a segment's M * G rows
  int tn_log2;    // of a tile's tokens
  uint32_t g_magic;          // ceil(2^32 / G); 0 for G = 1
  int parts;      // workers
  float* part_o;  // [parts][2][RB / 16][D / 8][32 lanes][4], as the MMA leaves them
  float2* part_ml;  // [parts][2][RB]
  unsigned long long wait_ns;  // limit of a wait for copies
  int inject;                  // the list's first piece never completes (tests)
  int4* part_seg;   // [parts][2][2] of a part: (b, h, rt, workers that hold the segment; 0: no such part), (the first of them, -, -, -)
};

// Bytes of the parts that `workers` can leave.
inline size_t attention_workspace(int workers, int RB, int D) {
  return static_cast<size_t>(workers) * (2 * RB * (static_cast<size_t>(D) * 4 + 8) + 64);
}
// Rows of a block: what one warp holds the outputs of.
inline int attention_row_block(int rows, int D) { return rows <= 16 || D == 256 ? 16 : 32; }


// Tokens of sequence b that its table holds; behind a prefix 0 (and, unless it is empty or has no new rows, the
// status bit) where its new rows do not come after the prefix.
template <bool BEHIND>
__device__ __forceinline__ int own_length(const AttentionArgs& a, int b) {
  if constexpr (!BEHIND) return seq_length(a.c, b);
  const int m = new_rows(a.q_lens, b, a.M), n = a.c.lengths[b], own = n - a.skip;
  if (n == 0 || m == 0) return 0;
  if (n < 0 || own < m || own > a.c.max_pages * a.c.page_size) {
    bad_page();
    return 0;
  }
  return own;
}

// The new row that row gr of a segment belongs to: gr / G (exact for gr * G < 2^32).
__device__ __forceinline__ int row_of(const AttentionArgs& a, int gr) {
  return a.G == 1 ? gr : static_cast<int>(__umulhi(static_cast<uint32_t>(gr), a.g_magic));
}

// What the rows of row block rt of a sequence (L tokens, m new rows) see.
struct Visible {
  int pos_lo, pos_hi;  // positions of its first and last valid row
  int hi;              // tokens j < hi are seen by some row, if also
  int first;           // j >= first, or j < sinks
  int sink_tiles, win_tile;  // tile k is k, from k = sink_tiles on k - sink_tiles + win_tile
  int tiles;
};
__device__ __forceinline__ Visible visible(const AttentionArgs& a, int L, int m, int rt) {
  Visible v;
  const int i0 = row_of(a, rt * a.RB);
  const int i1 = min(row_of(a, min((rt + 1) * a.RB, a.M * a.G) - 1), m - 1);
  v.pos_lo = L - m + i0;
  v.pos_hi = L - m + i1;
  v.hi = v.pos_hi + 1;
  v.first = a.window ? max(0, max(v.pos_lo, 0) - a.window + 1) : 0;
  v.sink_tiles = 0;
  v.win_tile = 0;
  v.tiles = 0;
  if (i0 > i1 || v.hi <= 0) return v;
  const int up = (1 << a.tn_log2) - 1;
  const int all = (v.hi + up) >> a.tn_log2;
  const int ns = a.window ? (min(a.sinks, v.hi) + up) >> a.tn_log2 : 0;
  const int w0 = v.first >> a.tn_log2;
  if (ns >= w0) {
    v.tiles = all;
  } else {
    v.sink_tiles = ns;
    v.win_tile = w0;
    v.tiles = ns + all - w0;
  }
  return v;
}

// The list counts kLead places before a segment's tiles: what its start and end
// cost (queries, outputs), in tiles, so that shares of many short segments are
// not longer than the others.  32 ragged sequences x 8 rows took 186, 149 and
// 143 us with 0, 2 and 4; a single long sequence is indifferent.
constexpr int kLead = 4;
__device__ __forceinline__ int places(const Visible& v) { return v.tiles > 0 ? v.tiles + kLead : 0; }

// Places of one head of sequence b, over its row blocks.
template <bool BEHIND>
__device__ __forceinline__ int head_places(const AttentionArgs& a, int b) {
  const int L = own_length<BEHIND>(a, b), m = new_rows(a.q_lens, b, a.M);
  int n = 0;
  for (int rt = 0; rt < a.RT; ++rt) n += places(visible(a, L, m, rt));
  return n;
}

// Inclusive prefix of v over the warp.
__device__ __forceinline__ int warp_scan(int v) {
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const int o = __shfl_up_sync(0xffffffffu, v, s);
    if ((threadIdx.x & 31) >= s) v += o;
  }
  return v;
}

// How the list of T places is shared: workers with a share (no more than there are
// places, so that every share holds one), places of each, and how many of the
// first ones hold one more.
struct Shares {
  int parts, each, more;
  __device__ __forceinline__ Shares(const AttentionArgs& a, int T) {
    parts = min(T, a.parts);
    each = parts > 0 ? T / parts : 0;
    more = T - each * parts;
  }
  __device__ __forceinline__ int begin(int c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int holder(int t) const {  // the worker whose share holds place t
    const int long_ones = more * (each + 1);
    return t < long_ones ? t / (each + 1) : more + (t - long_ones) / each;
  }
};

// A worker's share of the list, segment by segment.
template <bool BEHIND>
struct Cursor {
  int u, end;  // place of the list that this segment begins at; end of the share
  int b, h, rt;
  int kb, ke;  // tiles of the segment in this share
  int L, m;
  Visible v;

  __device__ __forceinline__ void load(const AttentionArgs& a) {
    L = own_length<BEHIND>(a, b);
    m = new_rows(a.q_lens, b, a.M);
  }
  // Places of sequence s over all heads.
  static __device__ __forceinline__ int seq_places(const AttentionArgs& a, int s) {
    return s < a.B ? head_places<BEHIND>(a, s) * a.c.heads : 0;
  }
  // The first segment with tiles in this worker's share (every lane of the warp
  // calls); false: none.  T: the list's places.
  __device__ __forceinline__ bool begin(const AttentionArgs& a, int worker, int& T) {
    const int lane = threadIdx.x & 31;
    T = 0;
    int n = 0;  // places of sequence (last base) + lane
#pragma unroll 1
    for (int base = 0; base < a.B; base += 32) {
      n = seq_places(a, base + lane);
      T += __reduce_add_sync(0xffffffffu, n);
    }
    const Shares sh(a, T);
    if (worker >= sh.parts) return false;
    const int start = sh.begin(worker);
    end = sh.begin(worker + 1);
    int before = 0;
    b = 0;
#pragma unroll 1
    for (int base = 0; base < a.B; base += 32) {
      if (a.B > 32) n = seq_places(a, base + lane);
      const int inc = warp_scan(n);
      const unsigned who = __ballot_sync(0xffffffffu, before + inc > start);
      if (who != 0) {
        const int l = __ffs(who) - 1;
        b = base + l;
        before += __shfl_sync(0xffffffffu, inc - n, l);
        break;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    load(a);
    const int per_head = max(head_places<BEHIND>(a, b), 1);
    h = (start - before) / per_head;
    u = before + h * per_head;
    for (rt = 0; rt < a.RT - 1; ++rt) {
      v = visible(a, L, m, rt);
      if (start < u + places(v)) break;
      u += places(v);
    }
    v = visible(a, L, m, rt);
    kb = max(0, start - u - kLead);
    ke = min(v.tiles, end - u - kLead);
    return kb < ke || next(a);
  }
  // The next segment with tiles in the share; false: none.
  __device__ __forceinline__ bool next(const AttentionArgs& a) {
    u += places(v);
    if (u + kLead >= end) return false;
    do {
      if (++rt == a.RT) {
        rt = 0;
        if (++h == a.c.heads) {
          h = 0;
          if (++b >= a.B) return false;
          load(a);
        }
      }
      v = visible(a, L, m, rt);
    } while (v.tiles == 0);
    kb = 0;
    ke = min(v.tiles, end - u - kLead);
    return true;
  }
  __device__ __forceinline__ int tile(int k) const { return k < v.sink_tiles ? k : k - v.sink_tiles + v.win_tile; }
};

// ---------------------------------------------------------------------------
// Shared-memory tiles: groups of 16 tokens, each as slices of 128 bytes of the
// tokens' rows ([slice][16 tokens][128 bytes]; rows of 64 bytes: [16][64]), the
// 16-byte chunks permuted as the TMA's 128-byte (64-byte) swizzle leaves them:
// the eight rows of one ldmatrix phase lie in different banks.
// ---------------------------------------------------------------------------
template <int ROWB>
__device__ __forceinline__ uint32_t tile_at(int token, int chunk) {
  const int r = token & 15, g = (token >> 4) * 16 * ROWB;
  if constexpr (ROWB >= 128) return g + (chunk >> 3) * 2048 + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
  else return g + r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, unsigned long long src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* tmap, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      ::"r"(dst), "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b with a zero accumulator input.
__device__ __forceinline__ void mma_f16_16816_z(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// (x0, x1) = (x0, x1) * f, and s += (x0, x1), as packed pairs.
__device__ __forceinline__ void fmul2(float& x0, float& x1, float f) {
  asm("{\n .reg .b64 a, c;\n mov.b64 a, {%0, %1};\n mov.b64 c, {%2, %2};\n mul.rn.f32x2 a, a, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x0), "+f"(x1) : "f"(f));
}
__device__ __forceinline__ void fadd2(float& s0, float& s1, float x0, float x1) {
  asm("{\n .reg .b64 a, c;\n mov.b64 a, {%0, %1};\n mov.b64 c, {%2, %3};\n add.rn.f32x2 a, a, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(s0), "+f"(s1) : "f"(x0), "f"(x1));
}
// (x0, x1) = (x0, x1) * f - c.
__device__ __forceinline__ void fms2(float& x0, float& x1, float f, float c) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %2};\n mov.b64 d, {%3, %3};\n"
      " fma.rn.f32x2 a, a, b, d;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x0), "+f"(x1) : "f"(f), "f"(-c));
}
// Two E4M3 codes (low 16 bits) to two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The elements of a word that are NaN or infinite, all their bits set.
template <bool E8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return E8 ? (((((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu)
            : (((((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u) >> 15) * 0xFFFFu);
}

// RPW 16-row tiles a worker.
template <int D, bool E8, int RPW>
struct AttnCfg {
  // Workers of an SM: as many as their registers allow (spilled ones would go to L2: shared memory takes the
  // L1's room; only D = 64 with two row tiles spills, 28 bytes a thread in bf16 and 64 in E4M3); seven where eight
  // would have room for two pieces only.
  static constexpr int WORKERS = D == 256 ? (E8 ? 8 : 7) : D == 64 ? 12 : RPW == 1 ? 10 : 8;
  // Tokens of a tile.  Small ones share a few tokens among more workers and need fewer registers for scores, large
  // ones have less to do beside their products.  D = 64, one row tile, 4 x 1000 tokens and 1 x 65001: 12.4 and 51 us
  // with 16, 15.8 and 46 with 32, 19.7 and 41 with 64 (8 workers); D = 128: 13.6 and 63.9 with 16, 18.2 and 62.9
  // with 32 (8 workers).  Two row tiles, window of 4096, D = 64: 56.7 with 16, 58.6 with 32 (8 workers).
  static constexpr int TN = D == 64 && RPW == 1 ? 32 : 16;
  static constexpr int TN_LOG2 = TN == 32 ? 5 : 4;
  static constexpr int ROWB = D * (E8 ? 1 : 2);
  static constexpr int TILEB = TN * ROWB;  // bytes of a key (or value) tile
  static constexpr bool QREG = D * RPW <= 64;  // query fragments stay in registers (D = 128: they spill, 77 us for 63.9)
  static constexpr int QB = QREG ? 0 : RPW * 16 * D * 2;  // [D / 16][RPW][32] query fragments, if not
  static constexpr int ROOM = (232448 - 1024) / WORKERS - QB;
  static constexpr int SLOTS = ROOM / (TILEB + 8) > 6 ? 6 : ROOM / (TILEB + 8);
  static constexpr int OFF_Q = WORKERS * SLOTS * TILEB;
  static constexpr int OFF_BAR = OFF_Q + WORKERS * QB;
  static constexpr int SMEM = OFF_BAR + WORKERS * SLOTS * 8 + 1024;  // and the alignment of its start
  static constexpr int THREADS = 32 * WORKERS;
  static_assert(TILEB % 1024 == 0 && SMEM <= 232448 && SLOTS >= 3, "shared memory of an SM");
};

// Query fragments of one warp: rows r0 = lane / 4 and r0 + 8 of its row group.
// bf16: as the MMA lays them out.  E4M3 cache: fp16, each row scaled by a power
// of two so that its largest element is just inside fp16 (elements 2^-38 below
// it vanish; the factor is undone in the score's scale), and with the columns
// of a k16 step in the order in which a key fragment's bytes come: slot pairs
// (2c, 2c+1) and (2c+8, 2c+9) hold columns 4c, 4c+1 and 4c+2, 4c+3.
template <int D, bool E8>
struct Query {
  uint32_t a[D / 16][4];
  float scale[2];  // score scale of the two rows
};

template <int D, int N, bool E8>
__device__ __forceinline__ void load_query(const AttentionArgs& a, Query<N, E8>& f, const uint16_t* const (&row)[2]) {
  const int c = threadIdx.x & 3;
  const uint32_t flip = a.negate ? 0x80008000u : 0u;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    f.scale[r] = a.scale_log2;
    if constexpr (!E8) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        f.a[kk][r] = row[r] ? *reinterpret_cast<const uint32_t*>(row[r] + kk * 16 + 2 * c) ^ flip : 0u;
        f.a[kk][r + 2] = row[r] ? *reinterpret_cast<const uint32_t*>(row[r] + kk * 16 + 8 + 2 * c) ^ flip : 0u;
      }
    } else {
      uint2 x[D / 16];
      float top = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        x[kk] = row[r] ? *reinterpret_cast<const uint2*>(row[r] + kk * 16 + 4 * c) : make_uint2(0, 0);
        x[kk].x ^= flip;
        x[kk].y ^= flip;
        top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(x[kk].x)), fabsf(bf16_hi(x[kk].x))),
                               fmaxf(fabsf(bf16_lo(x[kk].y)), fabsf(bf16_hi(x[kk].y)))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // top in [2^e, 2^(e+1)) goes to [2^14, 2^15); 0, tiny and infinite rows stay
      const int e = static_cast<int>(__float_as_uint(top) >> 23);
      const int up = (e < 30 || e == 255) ? 0 : 14 + 127 - e;  // exponent of the factor
      const float f1 = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
      // (not 0 either: a masked score of -inf stays -inf)
      f.scale[r] = fmaxf(a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23), 1e-30f);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        f.a[kk][r] = pack_f16(bf16_lo(x[kk].x) * f1, bf16_hi(x[kk].x) * f1);
        f.a[kk][r + 2] = pack_f16(bf16_lo(x[kk].y) * f1, bf16_hi(x[kk].y) * f1);
      }
    }
  }
}

// The natural logarithm of a row's sum l relative to its m (see above; the lift is taken back first, exactly).
template <bool E8>
__device__ __forceinline__ float log_sum(float m, float l) {
  if constexpr (E8) return (m + kLift + log2f(l * (1.f / (1 << static_cast<int>(kLift))))) * 0.6931471805599453f;
  else return (m + log2f(l)) * 0.6931471805599453f;
}

// Output column of element e (0, 1) of accumulator tile ot.
template <bool E8>
__device__ __forceinline__ int out_col(int ot, int e) {
  const int c = threadIdx.x & 3;
  return E8 ? (ot >> 1) * 16 + 4 * c + 2 * e + (ot & 1) : ot * 8 + 2 * c + e;
}

// Unrounded outputs: two neighbouring columns of one tile (E4M3: four, of two tiles in turn), times f, or 0.
template <bool E8>
__device__ __forceinline__ void store_f32(float* to, float x0, float x1, float y0, float y1, float f, bool some) {
  if constexpr (E8) {
    *reinterpret_cast<float4*>(to) = some ? make_float4(x0 * f, y0 * f, x1 * f, y1 * f) : make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    *reinterpret_cast<float2*>(to) = some ? make_float2(x0 * f, x1 * f) : make_float2(0.f, 0.f);
  }
}

// Whether some row of queries sees one of the tokens j .. j + count - 1.
template <class C>
__device__ __forceinline__ bool seen(const AttentionArgs& a, const C& p, int j, int count) {
  return j < p.v.hi && (j + count > p.v.first || j < a.sinks);
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A worker's stream of pieces.
//
// Where pages divide into boxes of 8 or 16 tokens (a.box), TMA copies boxes of
// [tokens][128 bytes] (16 tokens: all slices at once); coordinates are (byte
// column, token of the page, slice, head, page).  A page outside the cache is
// outside the tensor too and reads as zeros; boxes that nobody sees are left
// out, and what tokens past the length hold is dealt with where the values are
// used.  Any other page size: 16-byte asynchronous copies of the tokens' rows;
// tokens that nobody sees and those of pages outside the cache become zeros.
template <class Cfg, bool E8, bool BEHIND>
struct Stream {
  static constexpr int SL = Cfg::ROWB >= 128 ? Cfg::ROWB / 128 : 1, ROW = Cfg::ROWB >= 128 ? 128 : 64;
  static constexpr int CPR = Cfg::ROWB / 16, ES = E8 ? 1 : 2, RPI = 32 / CPR;
  static_assert(Cfg::TN <= 32, "a lane finds the page of one token or box of a tile");
  uint32_t ring, bars;  // shared-memory addresses
  Cursor<BEHIND> c;     // the segment of the next tile
  int k;
  bool more;            // there is such a tile
  int slot;             // of the next piece
  bool values;          // the next piece is a tile's values
  int page, place, head;  // of the tile that is copied: this lane's token (row copies) or box
  // Page numbers of the blocks first .. first + 31 of the sequence, a lane each,
  // and of the 32 after them, loaded when the ones before come into use.
  int pages, pages2, first, seq;

  static __device__ __forceinline__ int block_of(const AttentionArgs& a, int j) {
    return a.page_log2 >= 0 ? j >> a.page_log2 : j / a.c.page_size;
  }
  __device__ __forceinline__ int load_pages(const AttentionArgs& a, int block) const {
    const int i = block + (threadIdx.x & 31);
    return i < a.c.max_pages ? a.c.block_table[seq * a.c.table_stride + i] : -1;
  }
  // Page numbers and places in their pages of the next tile's tokens or boxes;
  // place -1: nobody sees it, page -1: outside the cache.
  __device__ __forceinline__ void find(const AttentionArgs& a) {
    const int lane = threadIdx.x & 31;
    const int step = a.box ? a.box : 1;                       // tokens a lane finds the page of
    const int finders = a.box ? Cfg::TN / a.box : Cfg::TN;    // lanes that do
    head = c.h;
    const int t0 = c.tile(k) * Cfg::TN;
    const int j = t0 + lane * step;
    int block = block_of(a, j);
    place = lane < finders && seen(a, c, j, step) ? j - block * a.c.page_size : -1;
    if (place < 0) block = INT_MAX;
    page = -1;
    if (c.b == seq && block_of(a, t0) >= first && block_of(a, t0 + Cfg::TN - 1) < first + 32) {
      const int got = __shfl_sync(0xffffffffu, pages, (block - first) & 31);
      if (block != INT_MAX) page = got;
    } else {
      // the lanes' blocks ascend: a window after another until all have been met
      for (;;) {
        const int low = __reduce_min_sync(0xffffffffu, block);
        if (low == INT_MAX) break;
        if (c.b != seq || low < first || low >= first + 32) {
          const bool follows = c.b == seq && low >= first + 32 && low < first + 64;
          seq = c.b;
          first = follows ? first + 32 : low;
          pages = follows ? pages2 : load_pages(a, first);
          pages2 = load_pages(a, first + 32);
        }
        const int got = __shfl_sync(0xffffffffu, pages, (block - first) & 31);
        if (block < first + 32) {
          page = got;
          block = INT_MAX;
        }
      }
    }
    if (place >= 0 && (page < 0 || page >= a.c.num_pages)) {
      bad_page();
      page = -1;
    }
    if (++k >= c.ke) {
      more = c.next(a);
      k = c.kb;
    }
  }
  __device__ __forceinline__ void begin(const AttentionArgs& a, const Cursor<BEHIND>& at, uint32_t ring_addr, uint32_t bar_addr) {
    ring = ring_addr;
    bars = bar_addr;
    c = at;
    k = c.kb;
    more = true;
    slot = 0;
    values = false;
    seq = -1;
    first = 0;
    pages = pages2 = -1;
  }
  // Copy the next piece into its slot (which the warp is done with).
  __device__ __forceinline__ void issue(const AttentionArgs& a, const void* kmap, const void* vmap) {
    const int lane = threadIdx.x & 31;
    bool any = true;
    if (!values) {
      any = more;
      if (any) find(a);
    }
    if (any) {
      const uint32_t base = ring + slot * Cfg::TILEB;
      if (a.box) {
        const uint32_t full = bars + slot * 8;
        const int per = a.box == 16 ? 1 : SL;  // copies of a box
        const uint32_t loaded = __ballot_sync(0xffffffffu, place >= 0);
        if (lane == 0) mbar_arrive_expect_tx(full, __popc(loaded) * a.box * Cfg::ROWB);
        __syncwarp();
        const int box = lane / per, sl = lane - box * per;  // at most 16 boxes x slices
        const int p = __shfl_sync(0xffffffffu, page, box & 31), s = __shfl_sync(0xffffffffu, place, box & 31);
        if (box * a.box < Cfg::TN && s >= 0) {
          const int token = box * a.box;
          tma_load_5d(base + (token >> 4) * 16 * Cfg::ROWB + sl * 2048 + (token & 15) * ROW, values ? vmap : kmap, 0, s, sl, head,
                      p, full);
        }
      } else {
        // byte offset of this lane's token from the cache's start, -1: zeros; it
        // reaches the lanes that copy the row by shuffles
        const unsigned long long cache = reinterpret_cast<unsigned long long>(values ? a.c.v : a.c.k);
        const int64_t s_page = values ? a.c.v_page : a.c.k_page, s_token = values ? a.c.v_token : a.c.k_token,
                      s_head = values ? a.c.v_head : a.c.k_head;
        const long long at = place >= 0 && page >= 0 ? (page * s_page + place * s_token + head * s_head) * ES : -1;
        const int ch = lane % CPR;
#pragma unroll 4
        for (int g = 0; g < Cfg::TN / RPI; ++g) {
          const int row = g * RPI + lane / CPR;
          const long long r = __shfl_sync(0xffffffffu, at, row);
          // nothing is read where zeros are filled in
          cp_async_16(base + tile_at<Cfg::ROWB>(row, ch), cache + (r < 0 ? 0 : r) + ch * 16, r >= 0);
        }
      }
      slot = slot + 1 == Cfg::SLOTS ? 0 : slot + 1;
      values = !values;
    }
    if (!a.box) cp_async_commit();  // a group for every call, so that counting them back finds a piece's
  }
};

// Waits for the pieces after `slot` and before `next` of a ring, on their way while the one in `slot` is given up.
// (Not inlined: what it needs would be spilled in the loop that never calls it.)
static __device__ __noinline__ void drain(uint32_t bars, int slot, int next, int slots, uint32_t phase, unsigned long long wait_ns) {
  for (int s = slot;;) {
    s = s + 1 == slots ? 0 : s + 1;
    if (s == next) return;
    mbar_wait(bars + s * 8, phase ^ (s < slot), kStatusTimeoutDrain, wait_ns);
  }
}

// Rows of segments without tiles: the worker of the sequence's number writes them.
template <int D>
__device__ __forceinline__ void empty_rows(const AttentionArgs& a, int worker) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int b = worker; b < a.B; b += a.parts) {
    const int L = seq_length(a.c, b), m = new_rows(a.q_lens, b, a.M);
#pragma unroll 1
    for (int rt = 0; rt < a.RT; ++rt) {
      if (visible(a, L, m, rt).tiles != 0) continue;
      const int r0 = rt * a.RB, rows = min(a.RB, a.M * a.G - r0), per_head = rows * (D / 8);
#pragma unroll 1
      for (int x = lane; x < per_head * a.c.heads; x += 32) {
        const int h = x / per_head, gr = r0 + (x - h * per_head) / (D / 8), col = (x % (D / 8)) * 8, i = row_of(a, gr);
        const int64_t at = (static_cast<int64_t>(b) * a.M + i) * a.Hq + h * a.G + gr - i * a.G;
        *reinterpret_cast<uint4*>(a.out + at * D + col) = make_uint4(0, 0, 0, 0);
        if (col == 0 && a.lse != nullptr) a.lse[at] = -INFINITY;
      }
    }
  }
}

// BEHIND: behind a prefix, with unrounded outputs (see AttentionArgs).  Nothing is written there for rows that do not
// exist, which the last kernel knows (9 sequences x 112 rows: 26.7 us with a warp a sequence writing them, 10.6 without).
template <int D, bool E8, int RPW, bool BEHIND>
__global__ void __launch_bounds__(AttnCfg<D, E8, RPW>::THREADS, 1)
attention_kernel(const AttentionArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using Cfg = AttnCfg<D, E8, RPW>;
  constexpr int SLOTS = Cfg::SLOTS, NT = Cfg::TN, ROWB = Cfg::ROWB, CPR = ROWB / 16;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int worker = warp * gridDim.x + blockIdx.x;  // the first shares go to different SMs

  if (tid == 0) {
    for (int s = 0; s < Cfg::WORKERS * SLOTS; ++s) mbar_init(sbase + Cfg::OFF_BAR + s * 8, 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  Cursor<BEHIND> cc;
  int T;
  if (lane < 2) a.part_seg[(worker * 2 + lane) * 2] = make_int4(0, 0, 0, 0);
  __syncwarp();
  if (!cc.begin(a, worker, T)) {
    if constexpr (!BEHIND) empty_rows<D>(a, worker);
    return;
  }
  {
    // the first segment's queries, on their way while the first pieces are asked for
    const int gr = cc.rt * a.RB + lane, i = row_of(a, gr);
    if (lane < a.RB && gr < a.M * a.G)
      for (int x = 0; x < D; x += 64)
        prefetch_l2(a.q + (static_cast<int64_t>(cc.b) * a.M + i) * a.q_ld + static_cast<int64_t>(cc.h * a.G + gr - i * a.G) * D + x);
  }
  const int ring_off = warp * SLOTS * Cfg::TILEB;
  const uint32_t bars = sbase + Cfg::OFF_BAR + warp * SLOTS * 8;
  Stream<Cfg, E8, BEHIND> in;
  in.begin(a, cc, sbase + ring_off, bars);
  if (a.inject && (cc.b | cc.h | cc.rt | cc.kb) == 0 && lane == 0) mbar_expect_tx(bars, 16);
#pragma unroll 1
  for (int s = 0; s < SLOTS; ++s) in.issue(a, &kmap, &vmap);

  float o[RPW][D / 8][4];
  float mx[RPW][2], sum[RPW][2][2];  // running maximum; sum of the even and of the odd columns
  Query<Cfg::QREG ? D : 16, E8> qf[RPW];  // the query fragments, or where they are
  uint4* const q_frag = reinterpret_cast<uint4*>(smem + Cfg::OFF_Q + warp * Cfg::QB) + lane;
  int pos[RPW][2];  // positions of this thread's rows; INT_MIN / 2 for rows that do not exist
  bool lost = false;
  int slot = 0;        // of the next piece to use
  uint32_t phase = 0;  // of its barrier
  // A wait that gave up (status bit 0) leaves wrong results, never a hang: the pieces that are still on their way
  // are waited for (status bit 2 where that gives up too), then no more are asked for and later waits are skipped.
  auto wait = [&]() {
    if (a.box) {
      if (!lost && __any_sync(0xffffffffu, !mbar_wait(bars + slot * 8, phase, kStatusTimeoutFull, a.wait_ns))) {
        lost = true;
        drain(bars, slot, in.slot, SLOTS, phase, a.wait_ns);
      }
    } else {
      cp_async_wait<SLOTS - 1>();
      __syncwarp();
    }
  };
  auto used = [&]() {
    __syncwarp();
    if (!lost) in.issue(a, &kmap, &vmap);
    if (++slot == SLOTS) {
      slot = 0;
      phase ^= 1;
    }
  };

  do {  // segment by segment
#pragma unroll
    for (int w = 0; w < RPW; ++w) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[w][i][0] = o[w][i][1] = o[w][i][2] = o[w][i][3] = 0.f;
      const uint16_t* row[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[w][r] = -INFINITY;
        sum[w][r][0] = sum[w][r][1] = 0.f;
        const int gr = cc.rt * a.RB + w * 16 + (lane >> 2) + 8 * r;
        const int i = row_of(a, gr);
        const bool ok = gr < a.M * a.G && i < cc.m;
        pos[w][r] = ok ? cc.L - cc.m + i : INT_MIN / 2;
        row[r] = ok ? a.q + (static_cast<int64_t>(cc.b) * a.M + i) * a.q_ld +
                          static_cast<int64_t>(cc.h * a.G + gr - i * a.G) * D
                    : nullptr;
      }
      if constexpr (Cfg::QREG) {
        load_query<Cfg::QREG ? D : 16>(a, qf[w], row);
      } else {
        Query<D, E8> f;
        load_query<D>(a, f, row);
        qf[w].scale[0] = f.scale[0];
        qf[w].scale[1] = f.scale[1];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          q_frag[(kk * RPW + w) * 32] = make_uint4(f.a[kk][0], f.a[kk][1], f.a[kk][2], f.a[kk][3]);
      }
    }
#pragma unroll 1
    for (int k = cc.kb; k < cc.ke; ++k) {
      const int j0 = cc.tile(k) * NT;
      const bool full = j0 + NT - 1 <= cc.v.pos_lo &&
                        (a.window == 0 || j0 > cc.v.pos_hi - a.window || j0 + NT <= a.sinks);
      float s[RPW][NT / 8][4];
      // the tile's keys, then its values (a loop, so that the refill's code is there once)
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        wait();
        const int off = ring_off + slot * Cfg::TILEB;
        const uint32_t kt = sbase + off, vt = kt;
        if (half == 0) {
          // scores
          auto query = [&](int kk, int w, uint32_t (&f)[4]) {
            if constexpr (Cfg::QREG) {
#pragma unroll
              for (int x = 0; x < 4; ++x) f[x] = qf[w].a[kk][x];
            } else {
              const uint4 u = q_frag[(kk * RPW + w) * 32];
              f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
            }
          };
          if constexpr (!E8) {
            const int kr = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              uint32_t f[RPW][4];
#pragma unroll
              for (int w = 0; w < RPW; ++w) query(kk, w, f[w]);
#pragma unroll
              for (int t = 0; t < NT / 16; ++t) {
                uint32_t b[4];
                ldsm_x4(b, kt + tile_at<ROWB>(t * 16 + kr, kk * 2 + ((lane >> 3) & 1)));
#pragma unroll
                for (int w = 0; w < RPW; ++w) {
                  if (kk == 0) {
                    mma_bf16_16816_z(s[w][2 * t], f[w], b[0], b[1]);
                    mma_bf16_16816_z(s[w][2 * t + 1], f[w], b[2], b[3]);
                  } else {
                    mma_bf16_16816(s[w][2 * t], f[w], b[0], b[1]);
                    mma_bf16_16816(s[w][2 * t + 1], f[w], b[2], b[3]);
                  }
                }
              }
            }
          } else {
            const int kr = lane & 15;
#pragma unroll
            for (int kk = 0; kk < D / 16; kk += 2) {
              uint32_t f[RPW][2][4];
#pragma unroll
              for (int w = 0; w < RPW; ++w) {
                query(kk, w, f[w][0]);
                query(kk + 1, w, f[w][1]);
              }
#pragma unroll
              for (int t = 0; t < NT / 16; ++t) {
                uint32_t b[4];
                ldsm_x4(b, kt + tile_at<ROWB>(t * 16 + kr, kk + (lane >> 4)));
#pragma unroll
                for (int x = 0; x < 4; ++x) {  // (token octet, k16 step) = (x & 1, x >> 1)
                  const uint32_t b0 = e4m3x2_to_f16x2(b[x]), b1 = e4m3x2_to_f16x2(b[x] >> 16);
#pragma unroll
                  for (int w = 0; w < RPW; ++w) {
                    if (kk + (x >> 1) == 0) mma_f16_16816_z(s[w][2 * t + (x & 1)], f[w][x >> 1], b0, b1);
                    else mma_f16_16816(s[w][2 * t + (x & 1)], f[w][x >> 1], b0, b1);
                  }
                }
              }
            }
          }
        } else {
#pragma unroll
          for (int w = 0; w < RPW; ++w) {
            // mask, running maximum, weights 2^(s scale - m)
            if (!full) {
#pragma unroll
              for (int i = 0; i < NT / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int j = j0 + i * 8 + 2 * (lane & 3) + (e & 1), p = pos[w][e >> 1];
                  const bool see = j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
                  s[w][i][e] = see ? s[w][i][e] : -INFINITY;
                }
            }
            float corr[2], base[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float top = fmaxf(s[w][0][2 * r], s[w][0][2 * r + 1]);
#pragma unroll
              for (int i = 1; i < NT / 8; ++i) top = max3(top, s[w][i][2 * r], s[w][i][2 * r + 1]);
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
              top = fmaxf(E8 ? fmaf(top, qf[w].scale[r], -kLift) : top * qf[w].scale[r], mx[w][r]);
              base[r] = top == -INFINITY ? 0.f : top;
              corr[r] = ex2(mx[w][r] - base[r]);
              mx[w][r] = top;
              sum[w][r][0] *= corr[r];
              sum[w][r][1] *= corr[r];
            }
            if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
              for (int i = 0; i < D / 8; ++i) {
                fmul2(o[w][i][0], o[w][i][1], corr[0]);
                fmul2(o[w][i][2], o[w][i][3], corr[1]);
              }
            }
#pragma unroll
            for (int i = 0; i < NT / 8; ++i)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                fms2(s[w][i][2 * r], s[w][i][2 * r + 1], qf[w].scale[r], base[r]);
                s[w][i][2 * r] = ex2(s[w][i][2 * r]);
                s[w][i][2 * r + 1] = ex2(s[w][i][2 * r + 1]);
                fadd2(sum[w][r][0], sum[w][r][1], s[w][i][2 * r], s[w][i][2 * r + 1]);
              }
          }

          // A token that a row does not see meets it with weight 0, and 0 times its
          // value must be 0.  Where such a value is not finite (a later draft row's, or
          // what lies past the length), the product is taken with 0 in the place of
          // every value that is not, and those are added element by element to the
          // rows that see them.
          constexpr int RPI = 32 / CPR;  // rows a warp looks at at once, a chunk a lane
          auto row_bad = [&](int t) {    // some element of this lane's chunk of row t + lane / CPR is not finite
            const uint4 u = *reinterpret_cast<const uint4*>(smem + off + tile_at<ROWB>(t + lane / CPR, lane % CPR));
            return (not_finite<E8>(u.x) | not_finite<E8>(u.y) | not_finite<E8>(u.z) | not_finite<E8>(u.w)) != 0;
          };
          bool bad = false;
          if (!full) {
#pragma unroll 1
            for (int t = 0; t < NT; t += RPI) {
              const int j = j0 + t + lane / CPR;
              const bool unseen = j > cc.v.pos_lo || (a.window != 0 && j >= a.sinks && j <= cc.v.pos_hi - a.window);
              if (unseen) bad |= row_bad(t);
            }
          }
          bad = __any_sync(0xffffffffu, bad);
          auto values = [&](auto clean) {
            constexpr bool kClean = decltype(clean)::value;
#pragma unroll
            for (int t = 0; t < NT / 16; ++t) {
              // fp16 holds a weight (up to 2^kLift) to 11 bits, which an E4M3 value's 4 leave unseen.  bf16 holds 8, no more than the
              // output: the weight's upper half goes in as it is and the rest as a second operand, 16 bits together
              // (66 for 64 us and 152 for 143 us in the two bf16 cases above).
              // The rest of a weight that is not 0 is not 0 either (its last bit is set first), so that an
              // infinite value times it is that infinity and not NaN.
              uint32_t p[RPW][4];
              [[maybe_unused]] uint32_t rest[RPW][E8 ? 1 : 4];
#pragma unroll
              for (int w = 0; w < RPW; ++w)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const float lo = s[w][2 * t + (x >> 1)][2 * (x & 1)], hi = s[w][2 * t + (x >> 1)][2 * (x & 1) + 1];
                  if constexpr (E8) {
                    p[w][x] = pack_f16(lo, hi);
                  } else {
                    const uint32_t l = __float_as_uint(lo), h = __float_as_uint(hi);
                    p[w][x] = __byte_perm(l, h, 0x7632);
                    rest[w][x] = pack_bf16(__uint_as_float(l | 1u) - __uint_as_float(l & 0xFFFF0000u),
                                           __uint_as_float(h | 1u) - __uint_as_float(h & 0xFFFF0000u));
                  }
                }
#pragma unroll
              for (int d = 0; d < D / 16; d += E8 ? 2 : 1) {
                uint32_t b[4];
                ldsm_x4_t(b, vt + tile_at<ROWB>(t * 16 + (lane & 15), (E8 ? d : 2 * d) + (lane >> 4)));
                if constexpr (kClean)
#pragma unroll
                  for (int x = 0; x < 4; ++x) b[x] &= ~not_finite<E8>(b[x]);
                if constexpr (!E8) {
#pragma unroll
                  for (int w = 0; w < RPW; ++w) {
                    mma_bf16_16816(o[w][2 * d], p[w], b[0], b[1]);
                    mma_bf16_16816(o[w][2 * d + 1], p[w], b[2], b[3]);
                    mma_bf16_16816(o[w][2 * d], rest[w], b[0], b[1]);
                    mma_bf16_16816(o[w][2 * d + 1], rest[w], b[2], b[3]);
                  }
                } else {
                  // a chunk's 16 dims come in pairs: even and odd dims become one tile each
#pragma unroll
                  for (int x = 0; x < 2; ++x) {  // chunk d + x
                    const uint32_t e0 = e4m3x2_to_f16x2(__byte_perm(b[2 * x], 0, 0x4420));
                    const uint32_t e1 = e4m3x2_to_f16x2(__byte_perm(b[2 * x + 1], 0, 0x4420));
                    const uint32_t f0 = e4m3x2_to_f16x2(__byte_perm(b[2 * x], 0, 0x4431));
                    const uint32_t f1 = e4m3x2_to_f16x2(__byte_perm(b[2 * x + 1], 0, 0x4431));
#pragma unroll
                    for (int w = 0; w < RPW; ++w) {
                      mma_f16_16816(o[w][2 * (d + x)], p[w], e0, e1);
                      mma_f16_16816(o[w][2 * (d + x) + 1], p[w], f0, f1);
                    }
                  }
                }
              }
            }
          };
          if (!bad) {
            values(std::false_type{});
          } else {
            values(std::true_type{});
#pragma unroll 1
            for (int t = 0; t < NT; ++t) {
              if (t % RPI == 0) bad = row_bad(t);
              if (((__ballot_sync(0xffffffffu, bad) >> (t % RPI * CPR)) & (CPR == 32 ? 0xffffffffu : (1u << (CPR & 31)) - 1u)) == 0)
                continue;
              const int src = (lane & 28) | ((t & 7) >> 1), j = j0 + t;
              float p[RPW][2];  // the token's weight for this thread's rows; 0 and not added where it is not seen
              bool see[RPW][2];
#pragma unroll
              for (int w = 0; w < RPW; ++w)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  float x = 0.f;
#pragma unroll
                  for (int i = 0; i < NT / 8; ++i)
                    if (i == t >> 3) x = (t & 1) ? s[w][i][2 * r + 1] : s[w][i][2 * r];
                  p[w][r] = __shfl_sync(0xffffffffu, x, src);
                  see[w][r] = j <= pos[w][r] && (a.window == 0 || j > pos[w][r] - a.window || j < a.sinks);
                }
              // four bytes at a time: two columns of one output tile, or (E4M3) two each of two
#pragma unroll
              for (int i = 0; i < D / 8; i += E8 ? 2 : 1) {
                const int at = out_col<E8>(i, 0) * (E8 ? 1 : 2);
                const uint32_t u = *reinterpret_cast<const uint32_t*>(smem + off + tile_at<ROWB>(t, at / 16) + at % 16);
                if (not_finite<E8>(u) == 0) continue;
#pragma unroll
                for (int x = 0; x < (E8 ? 4 : 2); ++x) {
                  const float f = E8 ? e4m3_to_float((u >> (8 * x)) & 0xFFu) : x ? bf16_hi(u) : bf16_lo(u);
                  if (fabsf(f) <= 3.4028235e38f) continue;
                  const int ot = E8 ? i + (x & 1) : i, e = E8 ? x >> 1 : x;
#pragma unroll
                  for (int w = 0; w < RPW; ++w) {
                    if (see[w][0]) o[w][ot][e] += p[w][0] * f;
                    if (see[w][1]) o[w][ot][2 + e] += p[w][1] * f;
                  }
                }
              }
            }
          }
        }
        used();
      }
    }

    // the end of the segment, or of this worker's share of it
    const bool whole = cc.kb == 0 && cc.ke == cc.v.tiles;
    const int64_t part = static_cast<int64_t>(worker) * 2 + (cc.kb == 0 ? 1 : 0);
    if (!whole && lane == 0) {
      const Shares sh(a, T);
      const int begin = cc.u + kLead, first = sh.holder(begin);  // the segment's first tile, and its holder
      a.part_seg[part * 2] = make_int4(cc.b, cc.h, cc.rt, sh.holder(begin + cc.v.tiles - 1) - first + 1);
      a.part_seg[part * 2 + 1] = make_int4(first, 0, 0, 0);
    }
#pragma unroll
    for (int w = 0; w < RPW; ++w) {
      float f[2];
      typename std::conditional<BEHIND, float, __nv_bfloat16>::type* to[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float l = sum[w][r][0] + sum[w][r][1];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int row = w * 16 + (lane >> 2) + 8 * r, gr = cc.rt * a.RB + row;
        to[r] = nullptr;
        if (!whole) {
          if ((lane & 3) == 0) a.part_ml[part * a.RB + row] = make_float2(mx[w][r], l);
        } else if (gr < a.M * a.G) {
          const int i = row_of(a, gr);
          const bool some = i < cc.m && l != 0.f;  // NaN sums count
          f[r] = some ? a.v_scale / l : 0.f;
          const int64_t at = (static_cast<int64_t>(cc.b) * a.M + i) * a.Hq + cc.h * a.G + gr - i * a.G;
          if constexpr (BEHIND) to[r] = a.out32 + at * D;
          else to[r] = a.out + at * D;
          if (a.lse != nullptr && (lane & 3) == 0) a.lse[at] = some ? log_sum<E8>(mx[w][r], l) : -INFINITY;
        }
      }
      if (!whole) {
        float4* const dst = reinterpret_cast<float4*>(a.part_o) + (part * RPW + w) * (D / 8) * 32 + lane;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) dst[i * 32] = make_float4(o[w][i][0], o[w][i][1], o[w][i][2], o[w][i][3]);
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (to[r] == nullptr) continue;
#pragma unroll
          for (int i = 0; i < D / 8; i += E8 ? 2 : 1) {
            // (a row without weight: 0 whatever the accumulators hold)
            const bool some = f[r] != 0.f;
            if constexpr (BEHIND) {
              store_f32<E8>(to[r] + out_col<E8>(i, 0), o[w][i][2 * r], o[w][i][2 * r + 1],
                            E8 ? o[w][i + E8][2 * r] : 0.f, E8 ? o[w][i + E8][2 * r + 1] : 0.f, f[r], some);
            } else if constexpr (E8) {
              uint2 u = make_uint2(0u, 0u);
              if (some) u = make_uint2(pack_bf16(o[w][i][2 * r] * f[r], o[w][i + 1][2 * r] * f[r]),
                                       pack_bf16(o[w][i][2 * r + 1] * f[r], o[w][i + 1][2 * r + 1] * f[r]));
              *reinterpret_cast<uint2*>(to[r] + out_col<true>(i, 0)) = u;
            } else {
              *reinterpret_cast<uint32_t*>(to[r] + out_col<false>(i, 0)) =
                  some ? pack_bf16(o[w][i][2 * r] * f[r], o[w][i][2 * r + 1] * f[r]) : 0u;
            }
          }
        }
      }
    }
  } while (cc.next(a));
  if (!a.box) cp_async_wait<0>();
  if constexpr (!BEHIND) empty_rows<D>(a, worker);
}

// Combines the parts of segments that several workers share.  A segment's
// output is cut into items of 16 rows and two output tiles (of 8 columns, in
// the layout the parts are in); the CTA of a part, the j-th of its segment's n,
// takes the items j, j + n, ..  Up to eight parts are added by one warp, which
// has an item of its own; of more, the warps share the parts of an item and are
// added in order through shared memory.  (One warp an item for any number: 25 us
// of the 72 us that one 65001-token row took, in 152 parts a head.)
template <int D, bool E8, bool BEHIND>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttentionArgs a) {
  constexpr int IW = 2, PER = D / 8 / IW, WARPS = kJoinThreads / 32;
  __shared__ float4 s_v[WARPS][IW][32];
  __shared__ float4 s_ml[WARPS][32];  // (max, sum) of the lane's two rows
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t mine = blockIdx.x;  // a part: worker * 2 + slot
  const int4 seg = a.part_seg[mine * 2];
  if (seg.w < 2) return;
  const int first = a.part_seg[mine * 2 + 1].x, nth = static_cast<int>(mine >> 1) - first;
  const int RPW = a.RB / 16, m = new_rows(a.q_lens, seg.x, a.M);
  // the first part is its worker's second slot, the others the first
  auto part = [&](int c) { return static_cast<int64_t>(first + c) * 2 + (c == 0); };
  const bool solo = seg.w <= 8;
  for (int item = solo ? nth * WARPS + warp : nth; item < RPW * PER; item += solo ? seg.w * WARPS : seg.w) {
    const int w = item / PER, i0 = (item - w * PER) * IW;
    const int base_row = seg.z * a.RB + w * 16;
    if (base_row >= a.M * a.G) continue;
    float v[IW][4] = {};
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    const int r0 = w * 16 + (lane >> 2);
    const int c0 = solo ? 0 : seg.w * warp / WARPS, c1 = solo ? seg.w : seg.w * (warp + 1) / WARPS;
#pragma unroll 1
    for (int base = c0; base < c1; base += 4) {
      float2 ml[4][2];
      float4 u[4][IW];
      const int n = min(4, c1 - base);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c >= n) break;
        const int64_t p = part(base + c);
        ml[c][0] = a.part_ml[p * a.RB + r0];
        ml[c][1] = a.part_ml[p * a.RB + r0 + 8];
#pragma unroll
        for (int i = 0; i < IW; ++i)
          u[c][i] = reinterpret_cast<const float4*>(a.part_o)[((p * RPW + w) * (D / 8) + i0 + i) * 32 + lane];
      }
      float ref[2], old[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float t = top[r];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < n) t = fmaxf(t, ml[c][r].x);
        ref[r] = t == -INFINITY ? 0.f : t;
        old[r] = ex2(top[r] - ref[r]);
        top[r] = t;
        sum[r] *= old[r];
      }
#pragma unroll
      for (int i = 0; i < IW; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] *= old[e >> 1];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c >= n) break;
        const float f0 = ex2(ml[c][0].x - ref[0]), f1 = ex2(ml[c][1].x - ref[1]);
        sum[0] += f0 * ml[c][0].y;
        sum[1] += f1 * ml[c][1].y;
#pragma unroll
        for (int i = 0; i < IW; ++i) {
          v[i][0] += f0 * u[c][i].x;
          v[i][1] += f0 * u[c][i].y;
          v[i][2] += f1 * u[c][i].z;
          v[i][3] += f1 * u[c][i].w;
        }
      }
    }
    float t[2] = {top[0], top[1]}, l[2] = {sum[0], sum[1]}, o[IW][4];
#pragma unroll
    for (int i = 0; i < IW; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = v[i][e];
    if (!solo) {
      __syncthreads();  // (of the item before: read)
#pragma unroll
      for (int i = 0; i < IW; ++i) s_v[warp][i][lane] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
      s_ml[warp][lane] = make_float4(top[0], sum[0], top[1], sum[1]);
      __syncthreads();
      if (warp != 0) continue;
      t[0] = t[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int i = 0; i < IW; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      float4 q[WARPS];
#pragma unroll
      for (int x = 0; x < WARPS; ++x) {
        q[x] = s_ml[x][lane];
        t[0] = fmaxf(t[0], q[x].x);
        t[1] = fmaxf(t[1], q[x].z);
      }
      const float b0 = t[0] == -INFINITY ? 0.f : t[0], b1 = t[1] == -INFINITY ? 0.f : t[1];
#pragma unroll
      for (int x = 0; x < WARPS; ++x) {
        const float f0 = ex2(q[x].x - b0), f1 = ex2(q[x].z - b1);
        l[0] += f0 * q[x].y;
        l[1] += f1 * q[x].w;
#pragma unroll
        for (int i = 0; i < IW; ++i) {
          const float4 u = s_v[x][i][lane];
          o[i][0] += f0 * u.x;
          o[i][1] += f0 * u.y;
          o[i][2] += f1 * u.z;
          o[i][3] += f1 * u.w;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int gr = base_row + (lane >> 2) + 8 * r;
      if (gr >= a.M * a.G) continue;
      const int i = row_of(a, gr);
      const bool some = i < m && l[r] != 0.f;
      const float f = some ? a.v_scale / l[r] : 0.f;
      const int64_t at = (static_cast<int64_t>(seg.x) * a.M + i) * a.Hq + seg.y * a.G + gr - i * a.G;
      __nv_bfloat16* const to = a.out + at * D;
      if constexpr (BEHIND) {
        float* const to32 = a.out32 + at * D;
        if constexpr (E8) {
          store_f32<true>(to32 + out_col<true>(i0, 0), o[0][2 * r], o[0][2 * r + 1], o[1][2 * r], o[1][2 * r + 1], f, some);
        } else {
#pragma unroll
          for (int j = 0; j < IW; ++j)
            store_f32<false>(to32 + out_col<false>(i0 + j, 0), o[j][2 * r], o[j][2 * r + 1], 0.f, 0.f, f, some);
        }
      } else if constexpr (E8) {
        static_assert(IW == 2, "an E4M3 cache's output tiles come in pairs");
        uint2 p = make_uint2(0u, 0u);
        if (some) p = make_uint2(pack_bf16(o[0][2 * r] * f, o[1][2 * r] * f), pack_bf16(o[0][2 * r + 1] * f, o[1][2 * r + 1] * f));
        *reinterpret_cast<uint2*>(to + out_col<true>(i0, 0)) = p;
      } else {
#pragma unroll
        for (int j = 0; j < IW; ++j)
          *reinterpret_cast<uint32_t*>(to + out_col<false>(i0 + j, 0)) = some ? pack_bf16(o[j][2 * r] * f, o[j][2 * r + 1] * f) : 0u;
      }
      if (a.lse != nullptr && i0 == 0 && (lane & 3) == 0) a.lse[at] = some ? log_sum<E8>(t[r], l[r]) : -INFINITY;
    }
  }
}

// Checks and launches of qmm_paged_attention (qmm_paged.cu).  With out32 the tokens come
// behind a prefix of `skip` (see AttentionArgs).
qmm_status run_attention(const qmm_paged_cache* cache, const void* q, int64_t q_ld, int B, int M, int q_heads,
                         const int32_t* q_lens, float scale, int window, int sinks, void* out, float* out32, float* lse, int skip,
                         void* workspace, size_t workspace_bytes, cudaStream_t stream);

// Launcher of one head size (qmm_paged_inst.cu): the attention kernel, of at most
// `ctas` CTAs, then the join.
template <int D, bool BEHIND>
cudaError_t launch_attention(AttentionArgs a, bool e8, int ctas, cudaStream_t stream);
template <int D, bool BEHIND>
unsigned int read_attention_status(int clear);

}  // namespace qmm
