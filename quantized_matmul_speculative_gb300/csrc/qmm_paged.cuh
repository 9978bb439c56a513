// Paged attention over a split list of key-value tiles, and the join of the
// parts (definition in include/qmm.h, qmm_paged_attention).
//
// The work.  A segment is one (sequence, key-value head, block of query rows):
// its rows are the new rows x the G query heads of the key-value head, so one
// pass over the keys and values serves them all.  A segment's visible tokens
// are cut into tiles of 64; the tiles of all segments form one list (sequence,
// head, row block, tile order), and CTA c of the grid takes the c-th equal
// share of it, whatever the lengths: a single long sequence is split over all
// SMs, a batch of ragged ones is balanced.  A segment that one CTA finishes is
// written directly; the others leave (max, sum, unnormalised output) of their
// share in the workspace, which join_kernel combines in list order.
//
// The mathematics.  One pass with running maximum m and sum l per row, in
// base-2 exponents: s = q.k scale log2(e), p = 2^(s - m'), o = o 2^(m - m') +
// p v, l likewise; o / l and (m + log2 l) ln 2 at the end.
#pragma once

#include <climits>
#include <type_traits>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {

constexpr int kKvTile = 64;       // tokens of a tile
constexpr int kAttnThreads = 128;

struct AttentionArgs {
  qmm_paged_cache c;
  const uint16_t* q;
  int64_t q_ld;
  int B, M, Hq, G;  // G = Hq / c.heads
  const int32_t* q_lens;
  float scale_log2;  // scale * log2(e), times k_scale for an E4M3 cache
  float v_scale;
  int window, sinks;
  __nv_bfloat16* out;
  float* lse;
  int RB, RT;     // rows of a row block, row blocks of a segment's M * G rows
  int parts;      // CTAs of the attention kernel
  float* part_o;  // [parts][2][RB][D]
  float2* part_ml;  // [parts][2][RB]
};

// Bytes of the parts that `ctas` CTAs can leave.
inline size_t attention_workspace(int ctas, int RB, int D) {
  return static_cast<size_t>(ctas) * 2 * RB * (static_cast<size_t>(D) * 4 + 8);
}
inline int attention_row_block(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

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
  const int rows = a.M * a.G;
  const int i0 = rt * a.RB / a.G;
  const int last = min((rt + 1) * a.RB, rows) - 1;
  const int i1 = min(last / a.G, m - 1);
  v.pos_lo = L - m + i0;
  v.pos_hi = L - m + i1;
  v.hi = v.pos_hi + 1;
  v.first = a.window ? max(0, max(v.pos_lo, 0) - a.window + 1) : 0;
  v.sink_tiles = 0;
  v.win_tile = 0;
  v.tiles = 0;
  if (i0 > i1 || v.hi <= 0) return v;
  const int all = (v.hi + kKvTile - 1) / kKvTile;
  const int ns = a.window ? (min(a.sinks, v.hi) + kKvTile - 1) / kKvTile : 0;
  const int w0 = v.first / kKvTile;
  if (ns >= w0) {
    v.tiles = all;
  } else {
    v.sink_tiles = ns;
    v.win_tile = w0;
    v.tiles = ns + all - w0;
  }
  return v;
}

// Tiles of one head of sequence b, over its row blocks.
__device__ __forceinline__ int head_tiles(const AttentionArgs& a, int b) {
  const int L = seq_length(a.c, b), m = new_rows(a.q_lens, b, a.M);
  int n = 0;
  for (int rt = 0; rt < a.RT; ++rt) n += visible(a, L, m, rt).tiles;
  return n;
}

// Total of `v` over the warp; inclusive prefix in `inc`.
__device__ __forceinline__ long long warp_scan(long long v, long long& inc) {
  inc = v;
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, s);
    if ((threadIdx.x & 31) >= s) inc += o;
  }
  return __shfl_sync(0xffffffffu, inc, 31);
}

// Tiles of all sequences, and of those before sequence `b` (every lane calls).
__device__ __forceinline__ long long total_tiles(const AttentionArgs& a, int b, long long* before) {
  long long total = 0, pre = 0;
  for (int base = 0; base < a.B; base += 32) {
    const int s = base + (threadIdx.x & 31);
    const long long n = s < a.B ? static_cast<long long>(head_tiles(a, s)) * a.c.heads : 0;
    long long inc;
    total += warp_scan(n, inc);
    long long mine = s < b ? n : 0;
#pragma unroll
    for (int x = 16; x > 0; x /= 2) mine += __shfl_xor_sync(0xffffffffu, mine, x);
    pre += mine;
  }
  if (before != nullptr) *before = pre;
  return total;
}

// CTAs that work: no more than there are tiles, so that every share holds one.
__device__ __forceinline__ int working(const AttentionArgs& a, long long T) {
  return T < a.parts ? static_cast<int>(T) : a.parts;
}
// First tile of CTA c's share of T tiles over P working CTAs.
__device__ __forceinline__ long long share_begin(long long T, int P, int c) { return T * c / P; }
// The CTA whose share holds tile t.
__device__ __forceinline__ int share_of(long long T, int P, long long t) {
  int c = static_cast<int>((t * P) / T);
  while (c + 1 < P && share_begin(T, P, c + 1) <= t) ++c;
  while (c > 0 && share_begin(T, P, c) > t) --c;
  return c;
}

// A place in the list of tiles.
struct Cursor {
  int b, h, rt, k;
  int L, m;
  Visible v;

  __device__ __forceinline__ void load(const AttentionArgs& a) {
    L = seq_length(a.c, b);
    m = new_rows(a.q_lens, b, a.M);
  }
  // The place of tile t < T (every lane of the warp calls).
  __device__ __forceinline__ void seek(const AttentionArgs& a, long long t) {
    long long before = 0;
    b = 0;
    for (int base = 0; base < a.B; base += 32) {
      const int s = base + (threadIdx.x & 31);
      const long long n = s < a.B ? static_cast<long long>(head_tiles(a, s)) * a.c.heads : 0;
      long long inc;
      const long long sum = warp_scan(n, inc);
      if (before + sum > t) {
        const unsigned who = __ballot_sync(0xffffffffu, before + inc > t);
        const int lane = __ffs(who) - 1;
        b = base + lane;
        before += __shfl_sync(0xffffffffu, inc - n, lane);
        break;
      }
      before += sum;
    }
    load(a);
    const int per_head = max(head_tiles(a, b), 1);
    h = static_cast<int>((t - before) / per_head);
    int r = static_cast<int>(t - before - static_cast<long long>(h) * per_head);
    for (rt = 0; rt < a.RT; ++rt) {
      v = visible(a, L, m, rt);
      if (r < v.tiles) break;
      r -= v.tiles;
    }
    k = r;
  }
  // The next tile; past the last one nothing is valid.
  __device__ __forceinline__ void next(const AttentionArgs& a) {
    if (++k < v.tiles) return;
    k = 0;
    do {
      if (++rt == a.RT) {
        rt = 0;
        if (++h == a.c.heads) {
          h = 0;
          if (++b >= a.B) return;
          load(a);
        }
      }
      v = visible(a, L, m, rt);
    } while (v.tiles == 0);
  }
  __device__ __forceinline__ int token0() const {
    return (k < v.sink_tiles ? k : k - v.sink_tiles + v.win_tile) * kKvTile;
  }
};

// ---------------------------------------------------------------------------
// Shared-memory tiles: rows of RB bytes (64, 128, 256 or 512), 16-byte chunks
// permuted so that the eight rows one ldmatrix phase reads lie in different
// banks.  Rows of 64 bytes share a 128-byte line in pairs.
// ---------------------------------------------------------------------------
template <int ROWB>
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  if constexpr (ROWB >= 128) {
    return row * ROWB + ((chunk ^ (row & 7)) << 4);
  } else {
    return (row >> 1) * 128 + (((((row & 1) << 2) | chunk) ^ ((row >> 1) & 7)) << 4);
  }
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
// Two E4M3 codes (low 16 bits) to two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(v));
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

template <int D, bool E8, int RG>
struct AttnCfg {
  static constexpr int ROWB = D * (E8 ? 1 : 2);
  static constexpr int TILEB = kKvTile * ROWB;  // bytes of a key (or value) tile
  // two CTAs an SM (113 KB each); one for D = 256, whose accumulators and stages fill it
  static constexpr int CTAS = D == 256 ? 1 : 2;
  static constexpr int STAGES = D == 256 ? (E8 ? 5 : 3) : TILEB >= 16384 ? 3 : TILEB >= 8192 ? 6 : 8;
  static constexpr int WT = 4 / RG;     // warps that share a row group, each with its tokens of the tile
  static constexpr int NT = kKvTile / WT;  // tokens of a warp
  static constexpr int DS = 32;         // output columns joined at a time
  static constexpr bool QREG = D <= 128;  // query fragments stay in registers
  static constexpr int OFF_ADDR = STAGES * 2 * TILEB;            // [STAGES][64] key and value addresses
  static constexpr int OFF_JOIN = OFF_ADDR + STAGES * kKvTile * 16;  // [4][16][DS + 4] floats
  static constexpr int OFF_ML = OFF_JOIN + (WT > 1 ? 4 * 16 * (DS + 4) * 4 : 0);  // [4][16] (m, l)
  static constexpr int OFF_Q = OFF_ML + (WT > 1 ? 4 * 16 * 8 : 0);  // [RG][D / 16][32] query fragments, if not in registers
  static constexpr int SMEM = OFF_Q + (QREG ? 0 : RG * 16 * D * 2);
  static_assert(CTAS * (SMEM + 1024) <= 233472 && SMEM <= 232448, "shared memory of an SM");
};

// CTAs an SM holds (AttnCfg::CTAS).
inline int attention_ctas_per_sm(int D) { return D == 256 ? 1 : 2; }

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
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    f.scale[r] = a.scale_log2;
    if constexpr (!E8) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        f.a[kk][r] = row[r] ? *reinterpret_cast<const uint32_t*>(row[r] + kk * 16 + 2 * c) : 0u;
        f.a[kk][r + 2] = row[r] ? *reinterpret_cast<const uint32_t*>(row[r] + kk * 16 + 8 + 2 * c) : 0u;
      }
    } else {
      uint2 x[D / 16];
      float top = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        x[kk] = row[r] ? *reinterpret_cast<const uint2*>(row[r] + kk * 16 + 4 * c) : make_uint2(0, 0);
        top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(x[kk].x)), fabsf(bf16_hi(x[kk].x))),
                               fmaxf(fabsf(bf16_lo(x[kk].y)), fabsf(bf16_hi(x[kk].y)))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // top in [2^e, 2^(e+1)) goes to [2^14, 2^15); 0, tiny and infinite rows stay
      const int e = static_cast<int>(__float_as_uint(top) >> 23);
      const int up = (e < 30 || e == 255) ? 0 : 14 + 127 - e;  // exponent of the factor
      const float f1 = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
      f.scale[r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        f.a[kk][r] = pack_f16(bf16_lo(x[kk].x) * f1, bf16_hi(x[kk].x) * f1);
        f.a[kk][r + 2] = pack_f16(bf16_lo(x[kk].y) * f1, bf16_hi(x[kk].y) * f1);
      }
    }
  }
}

// Output column of element e (0, 1) of accumulator tile ot.
template <bool E8>
__device__ __forceinline__ int out_col(int ot, int e) {
  const int c = threadIdx.x & 3;
  return E8 ? (ot >> 1) * 16 + 4 * c + 2 * e + (ot & 1) : ot * 8 + 2 * c + e;
}

template <int D, bool E8, int RG>
__global__ void __launch_bounds__(kAttnThreads, AttnCfg<D, E8, RG>::CTAS) attention_kernel(const AttentionArgs a) {
  using Cfg = AttnCfg<D, E8, RG>;
  constexpr int ST = Cfg::STAGES, NT = Cfg::NT, ROWB = Cfg::ROWB, CPR = ROWB / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t sbase = smem_addr(smem);
  ulonglong2* const addr = reinterpret_cast<ulonglong2*>(smem + Cfg::OFF_ADDR);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rg = warp / Cfg::WT, wt = warp % Cfg::WT;  // row group, token part

  griddep_wait();
  griddep_launch_dependents();
  const long long T = total_tiles(a, 0, nullptr);
  const int P = working(a, T);
  if (static_cast<int>(blockIdx.x) >= P) return;
  const long long t0 = share_begin(T, P, blockIdx.x);
  const int n = static_cast<int>(share_begin(T, P, blockIdx.x + 1) - t0);

  Cursor pc;  // runs ahead: the tile whose addresses are made next
  pc.seek(a, t0);
  Cursor cc = pc;  // the tile that is computed

  // Key and value address of token `r` of the cursor's tile: its page (loaded
  // here), then the sums in finish.  -1: not seen by any row.
  struct Place {
    int page, slot;
  };
  auto find = [&](int r) {
    Place p{-1, 0};
    const int j = pc.token0() + r;
    if (pc.b < a.B && j < pc.v.hi && (j >= pc.v.first || j < a.sinks)) {
      const int block = j / a.c.page_size;
      p.slot = j - block * a.c.page_size;
      p.page = a.c.block_table[pc.b * a.c.table_stride + block];
      if (p.page < 0 || p.page >= a.c.num_pages) {
        bad_page();
        p.page = -1;
      }
    }
    return p;
  };
  auto finish = [&](const Place& p, int h, int stage, int r) {
    ulonglong2 o = make_ulonglong2(0, 0);
    if (p.page >= 0) {
      constexpr int ES = E8 ? 1 : 2;
      o.x = reinterpret_cast<unsigned long long>(a.c.k) +
            (p.page * a.c.k_page + p.slot * a.c.k_token + h * a.c.k_head) * ES;
      o.y = reinterpret_cast<unsigned long long>(a.c.v) +
            (p.page * a.c.v_page + p.slot * a.c.v_token + h * a.c.v_head) * ES;
    }
    addr[stage * kKvTile + r] = o;
  };
  auto issue = [&](int stage) {
    const int ch = tid % CPR;
#pragma unroll
    for (int p = 0; p < CPR / 2; ++p) {
      const int row = p * (kAttnThreads / CPR) + tid / CPR;
      const ulonglong2 o = addr[stage * kKvTile + row];
      const uint32_t d = sbase + stage * 2 * Cfg::TILEB + tile_at<ROWB>(row, ch);
      // nothing is read where the size is 0; the address is the cache's own start
      cp_async_16(d, reinterpret_cast<const char*>(o.x ? o.x : reinterpret_cast<unsigned long long>(a.c.k)) + ch * 16,
                  o.x != 0);
      cp_async_16(d + Cfg::TILEB,
                  reinterpret_cast<const char*>(o.y ? o.y : reinterpret_cast<unsigned long long>(a.c.v)) + ch * 16,
                  o.y != 0);
    }
  };

  {
    // Addresses of the first ST tiles: all page numbers are loaded before the first is used.
    Place pl[(ST + 1) / 2];
    int ph[(ST + 1) / 2];
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      if ((tid >> 6) == (s & 1)) {
        pl[s / 2] = s < n ? find(tid & 63) : Place{-1, 0};
        ph[s / 2] = pc.h;
      }
      if (s < n) pc.next(a);
    }
#pragma unroll
    for (int s = 0; s < ST; ++s)
      if ((tid >> 6) == (s & 1)) finish(pl[s / 2], ph[s / 2], s, tid & 63);
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) {
    if (s < n) issue(s);
    cp_async_commit();
  }

  float o[D / 8][4];
  float mx[2], sum[2];
  Query<Cfg::QREG ? D : 16, E8> qf;  // the query fragments, or
  uint4* const q_frag = reinterpret_cast<uint4*>(smem + Cfg::OFF_Q) + rg * (D / 16) * 32 + lane;  // where they are
  float (&q_scale)[2] = qf.scale;
  int pos[2];       // positions of this thread's two rows; INT_MIN / 2 for rows that do not exist
  bool fresh = true;
  int k_first = 0;  // first tile of the current segment in this CTA

  for (int it = 0; it < n; ++it) {
    const int stage = it % ST;
    cp_async_wait<ST - 2>();
    __syncthreads();
    if (it + ST - 1 < n) issue((it + ST - 1) % ST);
    cp_async_commit();
    const bool more = it + ST < n;
    Place np{-1, 0};
    int nh = 0;
    if (more) {
      nh = pc.h;
      if (tid < kKvTile) np = find(tid);
    }

    if (fresh) {
      fresh = false;
      k_first = cc.k;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      const uint16_t* row[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = -INFINITY;
        sum[r] = 0.f;
        const int gr = cc.rt * a.RB + rg * 16 + (lane >> 2) + 8 * r;
        const int i = gr / a.G;
        const bool ok = gr < a.M * a.G && i < cc.m;
        pos[r] = ok ? cc.L - cc.m + i : INT_MIN / 2;
        row[r] = ok ? a.q + (static_cast<int64_t>(cc.b) * a.M + i) * a.q_ld +
                          static_cast<int64_t>(cc.h * a.G + gr - i * a.G) * D
                    : nullptr;
      }
      if constexpr (Cfg::QREG) {
        load_query<Cfg::QREG ? D : 16>(a, qf, row);
      } else {
        Query<D, E8> f;
        load_query<D>(a, f, row);
        q_scale[0] = f.scale[0];
        q_scale[1] = f.scale[1];
        if (wt == 0)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) q_frag[kk * 32] = make_uint4(f.a[kk][0], f.a[kk][1], f.a[kk][2], f.a[kk][3]);
        if (Cfg::WT > 1) __syncthreads();
        else __syncwarp();
      }
    }

    const int j0 = cc.token0() + wt * NT;  // this warp's first token
    const bool full = cc.token0() + kKvTile - 1 <= cc.v.pos_lo &&
                      (a.window == 0 || cc.token0() > cc.v.pos_hi - a.window || cc.token0() + kKvTile <= a.sinks);
    const uint32_t kt = sbase + stage * 2 * Cfg::TILEB, vt = kt + Cfg::TILEB;

    // scores
    float s[NT / 8][4];
#pragma unroll
    for (int i = 0; i < NT / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
    auto query = [&](int kk, uint32_t (&f)[4]) {
      if constexpr (Cfg::QREG) {
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] = qf.a[kk][x];
      } else {
        const uint4 w = q_frag[kk * 32];
        f[0] = w.x, f[1] = w.y, f[2] = w.z, f[3] = w.w;
      }
    };
    if constexpr (!E8) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t f[4];
        query(kk, f);
#pragma unroll
        for (int t = 0; t < NT / 16; ++t) {
          uint32_t b[4];
          ldsm_x4(b, kt + tile_at<ROWB>(wt * NT + t * 16 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
          mma_bf16_16816(s[2 * t], f, b[0], b[1]);
          mma_bf16_16816(s[2 * t + 1], f, b[2], b[3]);
        }
      }
    } else {
#pragma unroll
      for (int kk = 0; kk < D / 16; kk += 2) {
        uint32_t f[2][4];
        query(kk, f[0]);
        query(kk + 1, f[1]);
#pragma unroll
        for (int t = 0; t < NT / 16; ++t) {
          uint32_t b[4];
          ldsm_x4(b, kt + tile_at<ROWB>(wt * NT + t * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), kk + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < 4; ++x)  // (token octet, k16 step) = (x & 1, x >> 1)
            mma_f16_16816(s[2 * t + (x & 1)], f[x >> 1], e4m3x2_to_f16x2(b[x]), e4m3x2_to_f16x2(b[x] >> 16));
        }
      }
    }

    // scale, mask, running maximum
    float top[2] = {mx[0], mx[1]};
#pragma unroll
    for (int i = 0; i < NT / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = s[i][e] * q_scale[e >> 1];
        if (!full) {
          const int j = j0 + i * 8 + 2 * (lane & 3) + (e & 1), p = pos[e >> 1];
          const bool see = j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
          x = see ? x : -INFINITY;
        }
        s[i][e] = x;
        top[e >> 1] = fmaxf(top[e >> 1], x);
      }
    float corr[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      const float base = top[r] == -INFINITY ? 0.f : top[r];
      corr[r] = ex2(mx[r] - base);
      mx[r] = top[r];
      top[r] = base;
      sum[r] *= corr[r];
    }
    if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= corr[0];
        o[i][1] *= corr[0];
        o[i][2] *= corr[1];
        o[i][3] *= corr[1];
      }
    }
#pragma unroll
    for (int i = 0; i < NT / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = ex2(s[i][e] - top[e >> 1]);
        sum[e >> 1] += s[i][e];
      }

    // A token that only some rows see meets the others with weight 0, and 0
    // times its value must be 0.  Where such a value is not finite, the product
    // is taken with 0 in the place of every value that is not, and those are
    // added element by element to the rows that see them.
    bool bad = false;
    if (!full && cc.v.pos_lo != cc.v.pos_hi) {
      for (int t = 0; t < NT; ++t) {
        const int j = j0 + t;
        if (j >= cc.v.hi) break;
        if (j > cc.v.pos_lo || (a.window != 0 && j <= cc.v.pos_hi - a.window && j >= a.sinks)) {
          for (int ch = lane; ch < CPR; ch += 32) {
            const uint4 w = *reinterpret_cast<const uint4*>(smem + (vt - sbase) + tile_at<ROWB>(wt * NT + t, ch));
            bad |= (not_finite<E8>(w.x) | not_finite<E8>(w.y) | not_finite<E8>(w.z) | not_finite<E8>(w.w)) != 0;
          }
        }
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    auto values = [&](auto clean) {
      constexpr bool kClean = decltype(clean)::value;
#pragma unroll
      for (int t = 0; t < NT / 16; ++t) {
        // fp16 holds a probability to 11 bits; bf16 to 8 only, so its rest goes in as a second operand
        uint32_t p[4], rest[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float lo = s[2 * t + (x >> 1)][2 * (x & 1)], hi = s[2 * t + (x >> 1)][2 * (x & 1) + 1];
          p[x] = E8 ? pack_f16(lo, hi) : pack_bf16(lo, hi);
          rest[x] = E8 ? 0u : pack_bf16(lo - bf16_lo(p[x]), hi - bf16_hi(p[x]));
        }
#pragma unroll
        for (int d = 0; d < D / 16; d += E8 ? 2 : 1) {
          uint32_t b[4];
          ldsm_x4_t(b, vt + tile_at<ROWB>(wt * NT + t * 16 + (lane & 15), (E8 ? d : d * 2) + (lane >> 4)));
          if constexpr (kClean)
#pragma unroll
            for (int x = 0; x < 4; ++x) b[x] &= ~not_finite<E8>(b[x]);
          if constexpr (!E8) {
            mma_bf16_16816(o[2 * d], p, b[0], b[1]);
            mma_bf16_16816(o[2 * d + 1], p, b[2], b[3]);
            mma_bf16_16816(o[2 * d], rest, b[0], b[1]);
            mma_bf16_16816(o[2 * d + 1], rest, b[2], b[3]);
          } else {
            // a chunk's 16 dims come in pairs: even and odd dims become one tile each
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // chunk d + x
              mma_f16_16816(o[2 * (d + x)], p, e4m3x2_to_f16x2(__byte_perm(b[2 * x], 0, 0x4420)),
                            e4m3x2_to_f16x2(__byte_perm(b[2 * x + 1], 0, 0x4420)));
              mma_f16_16816(o[2 * (d + x) + 1], p, e4m3x2_to_f16x2(__byte_perm(b[2 * x], 0, 0x4431)),
                            e4m3x2_to_f16x2(__byte_perm(b[2 * x + 1], 0, 0x4431)));
            }
          }
        }
      }
    };
    if (!bad) {
      values(std::false_type{});
    } else {
      values(std::true_type{});
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int src = (lane & 28) | ((t & 7) >> 1);
        const float p0 = __shfl_sync(0xffffffffu, s[t / 8][t & 1], src);
        const float p1 = __shfl_sync(0xffffffffu, s[t / 8][2 + (t & 1)], src);
        const int j = j0 + t;
        const bool see0 = j <= pos[0] && (a.window == 0 || j > pos[0] - a.window || j < a.sinks);
        const bool see1 = j <= pos[1] && (a.window == 0 || j > pos[1] - a.window || j < a.sinks);
        bool some = false;
        for (int ch = lane; ch < CPR; ch += 32) {
          const uint4 w = *reinterpret_cast<const uint4*>(smem + (vt - sbase) + tile_at<ROWB>(wt * NT + t, ch));
          some |= (not_finite<E8>(w.x) | not_finite<E8>(w.y) | not_finite<E8>(w.z) | not_finite<E8>(w.w)) != 0;
        }
        if (!__any_sync(0xffffffffu, some)) continue;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = out_col<E8>(i, e) * (E8 ? 1 : 2);
            const unsigned char* w = smem + (vt - sbase) + tile_at<ROWB>(wt * NT + t, col / 16) + col % 16;
            const float v = E8 ? e4m3_to_float(*w) : bf16_lo(*reinterpret_cast<const uint16_t*>(w));
            if (fabsf(v) <= 3.4028235e38f) continue;
            if (see0) o[i][e] += p0 * v;
            if (see1) o[i][2 + e] += p1 * v;
          }
      }
    }

    // the end of a segment, or of this CTA's share of it
    if (cc.k + 1 == cc.v.tiles || it + 1 == n) {
      const bool whole = k_first == 0 && cc.k + 1 == cc.v.tiles;
      const int slot = blockIdx.x * 2 + (k_first == 0 ? 1 : 0);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
      }
      float2* const ml = reinterpret_cast<float2*>(smem + Cfg::OFF_ML);
      float* const join = reinterpret_cast<float*>(smem + Cfg::OFF_JOIN);
      if (Cfg::WT > 1 && (lane & 3) == 0) {
        ml[warp * 16 + (lane >> 2)] = make_float2(mx[0], sum[0]);
        ml[warp * 16 + (lane >> 2) + 8] = make_float2(mx[1], sum[1]);
      }
      // Rows in slices of DS columns through shared memory: the warps of a row
      // group are added, and a thread then holds four columns of a row.
      constexpr int DS = Cfg::DS;
      const int rows = a.M * a.G - cc.rt * a.RB;  // rows of this block that exist
      auto put = [&](int row, int col, float4 v, float m_all, float l_all) {
        if (row >= rows) return;
        if (whole) {
          const int gr = cc.rt * a.RB + row, i = gr / a.G;
          const bool some = i < cc.m && l_all != 0.f;  // NaN sums count
          const float f = some ? a.v_scale / l_all : 0.f;
          const int64_t at = (static_cast<int64_t>(cc.b) * a.M + i) * a.Hq + cc.h * a.G + gr - i * a.G;
          uint2 w = make_uint2(0u, 0u);
          if (some) w = make_uint2(pack_bf16(v.x * f, v.y * f), pack_bf16(v.z * f, v.w * f));
          *reinterpret_cast<uint2*>(a.out + at * D + col) = w;
          if (col == 0 && a.lse != nullptr) a.lse[at] = some ? (m_all + log2f(l_all)) * 0.6931471805599453f : -INFINITY;
        } else {
          *reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(slot) * a.RB + row) * D + col) = v;
          if (col == 0) a.part_ml[static_cast<int64_t>(slot) * a.RB + row] = make_float2(m_all, l_all);
        }
      };
      if constexpr (Cfg::WT > 1) {
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += DS) {
          __syncthreads();
#pragma unroll
          for (int i = d0 / 8; i < (d0 + DS) / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              join[(warp * 16 + (lane >> 2) + 8 * (e >> 1)) * (DS + 4) + out_col<E8>(i, e & 1) - d0] = o[i][e];
          __syncthreads();
#pragma unroll
          for (int x = tid; x < RG * 16 * (DS / 4); x += kAttnThreads) {
            const int row = x / (DS / 4), col = (x % (DS / 4)) * 4, w0 = (row / 16) * Cfg::WT;
            float m_all = -INFINITY, l_all = 0.f;
#pragma unroll
            for (int w = 0; w < Cfg::WT; ++w) m_all = fmaxf(m_all, ml[(w0 + w) * 16 + row % 16].x);
            const float base = m_all == -INFINITY ? 0.f : m_all;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < Cfg::WT; ++w) {
              const float2 p = ml[(w0 + w) * 16 + row % 16];
              const float f = ex2(p.x - base);
              const float4 u = *reinterpret_cast<const float4*>(join + ((w0 + w) * 16 + row % 16) * (DS + 4) + col);
              l_all += f * p.y;
              v.x += f * u.x;
              v.y += f * u.y;
              v.z += f * u.z;
              v.w += f * u.w;
            }
            put(row, d0 + col, v, m_all, l_all);
          }
        }
        __syncthreads();
      } else {
        // four columns of a row from two lanes: even lanes take the upper row, odd ones the lower
#pragma unroll
        for (int i = 0; i < D / 8; i += E8 ? 2 : 1) {
          const int odd = lane & 1;
          if constexpr (E8) {
            put(rg * 16 + (lane >> 2), out_col<true>(i, 0), make_float4(o[i][0], o[i + 1][0], o[i][1], o[i + 1][1]), mx[0], sum[0]);
            put(rg * 16 + (lane >> 2) + 8, out_col<true>(i, 0), make_float4(o[i][2], o[i + 1][2], o[i][3], o[i + 1][3]), mx[1], sum[1]);
          } else {
            const float x0 = __shfl_xor_sync(0xffffffffu, odd ? o[i][0] : o[i][2], 1);
            const float x1 = __shfl_xor_sync(0xffffffffu, odd ? o[i][1] : o[i][3], 1);
            const int col = i * 8 + ((lane & 2) << 1);
            if (!odd) put(rg * 16 + (lane >> 2), col, make_float4(o[i][0], o[i][1], x0, x1), mx[0], sum[0]);
            else put(rg * 16 + (lane >> 2) + 8, col, make_float4(x0, x1, o[i][2], o[i][3]), mx[1], sum[1]);
          }
        }
      }
      fresh = true;
    }
    if (it + 1 < n) cc.next(a);
    if (more) {
      if (tid < kKvTile) finish(np, nh, stage, tid);
      pc.next(a);
    }
  }
}

// Combines the parts of segments that several CTAs share, and writes the rows
// of segments without tiles.  One warp per row, D / 32 columns a lane.
template <int D>
__global__ void __launch_bounds__(kAttnThreads) join_kernel(const AttentionArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int per_seg = a.RB / 4;
  const int seg = blockIdx.x / per_seg;
  const int row = (blockIdx.x % per_seg) * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rt = seg % a.RT, h = (seg / a.RT) % a.c.heads, b = seg / a.RT / a.c.heads;
  const int gr = rt * a.RB + row;
  if (gr >= a.M * a.G) return;
  long long begin;
  const long long T = total_tiles(a, b, &begin);
  const int L = seq_length(a.c, b), m = new_rows(a.q_lens, b, a.M);
  begin += static_cast<long long>(head_tiles(a, b)) * h;
  for (int r = 0; r < rt; ++r) begin += visible(a, L, m, r).tiles;
  const int n = visible(a, L, m, rt).tiles;
  const int i = gr / a.G;
  const int64_t at = (static_cast<int64_t>(b) * a.M + i) * a.Hq + h * a.G + gr - i * a.G;
  constexpr int E = D / 32;  // 2, 4 or 8 columns
  float v[E] = {};
  float top = -INFINITY, sum = 0.f;
  if (n > 0) {
    const int P = working(a, T), c0 = share_of(T, P, begin), c1 = share_of(T, P, begin + n - 1);
    if (c0 == c1) return;
    for (int c = c0; c <= c1; ++c) top = fmaxf(top, a.part_ml[static_cast<int64_t>(c * 2 + (c == c0)) * a.RB + row].x);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const int64_t p = static_cast<int64_t>(c * 2 + (c == c0)) * a.RB + row;
      const float2 ml = a.part_ml[p];
      const float f = ex2(ml.x - base);
      sum += f * ml.y;
      const float2* src = reinterpret_cast<const float2*>(a.part_o + p * D + lane * E);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const float2 u = src[e];
        v[2 * e] += f * u.x;
        v[2 * e + 1] += f * u.y;
      }
    }
  }
  const bool some = i < m && n > 0 && sum != 0.f;
  const float f = some ? a.v_scale / sum : 0.f;
#pragma unroll
  for (int e = 0; e < E / 2; ++e)
    reinterpret_cast<uint32_t*>(a.out + at * D + lane * E)[e] = some ? pack_bf16(v[2 * e] * f, v[2 * e + 1] * f) : 0u;
  if (a.lse != nullptr && lane == 0) a.lse[at] = some ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// Launcher of one head size (qmm_paged_inst.cu): a.parts CTAs, then the join.
template <int D>
cudaError_t launch_attention(AttentionArgs a, bool e8, cudaStream_t stream);
template <int D>
unsigned int read_attention_status(int clear);

}  // namespace qmm
