// Rotation of new queries and keys by their positions, and their keys and values
// into the paged cache on the way (qmm_rope_append, include/qmm.h).
//
// The mathematics.  A pair of elements (x1, x2) of a head turns by the angle p f, with
// p the row's position and f the pair's frequency: (x1 c - x2 s, x2 c + x1 s).  p f is
// thousands of turns at far positions, of which 32 bits would keep few digits; so f is
// taken as f / 2 pi = turns a position, in 64 bits after the point, whole turns dropped,
// and times p by a product of integers, which drops whole turns by itself: its upper 32
// bits, off by less than p 2^-64 turns, are the angle.
//
// A row's angles are computed once for all its heads, while its elements are on their way.
//
// What bounds it: the copies, whose places depend on lengths and table: 2 x 4001 rows of
// 32 + 16 heads x 128, 26 us, 5.0 TB/s; 128 x 16 rows into E4M3 13.3 us, 3.5 TB/s (1.4
// us more with scales that are no powers of two); 4 x 5 rows 4.6 us, a launch and that chain.
#include <algorithm>
#include <cmath>

#include "qmm_cache.cuh"

namespace qmm {
namespace {

constexpr int kRopeThreads = 128;  // that turn
constexpr int kRopeRing = 30720, kRopePiece = 15360, kRopeStages = 4;  // bytes of a CTA's ring, of a piece at most; pieces at most

struct RopeArgs {
  qmm_paged_cache c;
  qmm_rope r;
  const uint16_t *q, *kn, *vn;
  uint16_t* out;
  int64_t q_ld, out_ld, k_ld, v_ld;
  int B, M, Hq, per_head_log2;  // items of a head
  int heads, pieces, stages, stage_bytes;  // heads of a piece, pieces of a row; of the ring
  float k_inverse, v_inverse;   // of the scales that are powers of two, else 0
  const int32_t* q_lens;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// f / 2 pi in units of 2^-64 turns, modulo a turn.
__device__ __forceinline__ unsigned long long turns_of(float f) {
  // 1 / 2 pi = 0x0.28BE60DB 9391054A 7F09D5F4 ..
  const uint32_t u = __float_as_uint(f), e = (u >> 23) & 255u;
  const uint32_t m = e != 0 ? (u & 0x7FFFFFu) | 0x800000u : (u & 0x7FFFFFu) << 1;
  // m * 96 bits: 120 bits of |f| / 2 pi, times 2^(246 - e)
  const unsigned long long p0 = static_cast<unsigned long long>(m) * 0x7F09D5F4u;
  const unsigned long long p1 = static_cast<unsigned long long>(m) * 0x9391054Au + (p0 >> 32);
  const unsigned long long p2 = static_cast<unsigned long long>(m) * 0x28BE60DBu + (p1 >> 32);
  const unsigned long long lo = (p1 << 32) | (p0 & 0xFFFFFFFFu);
  const int down = 182 - static_cast<int>(e);  // to 2^64
  unsigned long long t;
  if (down >= 128 || down <= -64) t = 0;
  else if (down >= 64) t = p2 >> (down - 64);
  else if (down > 0) t = (lo >> down) | (p2 << (64 - down));
  else t = lo << -down;
  return u >> 31 ? 0ull - t : t;
}

// Eight elements of a row, and back.
struct Eight {
  float v[8];
  __device__ __forceinline__ void set(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  __device__ __forceinline__ uint4 bf16() const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // Quotients by s: products with its inverse r where s is a power of two, which are the same (r = 0: it is not).  128 x 16
  // rows into E4M3, one call after another on the device: 11.7 us with products, 13.1 with quotients.
  __device__ __forceinline__ uint2 e4m3(float s, float r) const {
    uint32_t w[4];
    if (r != 0.f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = cvt_e4m3(v[2 * i] * r, v[2 * i + 1] * r);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = cvt_e4m3(__fdiv_rn(v[2 * i], s), __fdiv_rn(v[2 * i + 1], s));
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  }
};

// Item x of a piece, which begins at head `first` of queries, keys and values in a row: two chunks of 8 elements of a head that
// turn together, or neighbours.
struct Item {
  int h, c0, c1;     // head; first elements of the chunks
  bool is_q, is_v, turned;
  __device__ __forceinline__ Item(const RopeArgs& a, int first, int x) {
    const int in = x >> a.per_head_log2, head = first + in, j = x - (in << a.per_head_log2), half = a.r.rot / 2;
    is_q = head < a.Hq;
    is_v = head >= a.Hq + a.c.heads;
    h = is_q ? head : is_v ? head - a.Hq - a.c.heads : head - a.Hq;
    turned = !is_v && j < half / 8;
    const bool halves = turned && !a.r.interleaved;
    c0 = halves ? j * 8 : j * 16;
    c1 = halves ? half + j * 8 : j * 16 + 8;
  }
  __device__ __forceinline__ void finish(const RopeArgs& a, const float2* turn, int64_t row, int64_t page, int slot, const uint4& u,
                                         const uint4& w) const {
    const int64_t at = is_q ? row * a.out_ld + static_cast<int64_t>(h) * a.c.head_dim
                     : is_v ? page * a.c.v_page + slot * a.c.v_token + h * a.c.v_head
                            : page * a.c.k_page + slot * a.c.k_token + h * a.c.k_head;
    void* const to = is_q ? static_cast<void*>(a.out) : is_v ? a.c.v : a.c.k;
    const bool codes = !is_q && a.c.dtype != QMM_KV_BF16;
    if (!turned && !codes) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(to) + at + c0) = u;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(to) + at + c1) = w;
      return;
    }
    Eight x0, x1;
    x0.set(u);
    x1.set(w);
    if (turned) {
      // (the pair's first elements are c0 on with halves, and c0 / 2 on of the pairs with neighbours)
      const float4* const t = reinterpret_cast<const float4*>(turn + (a.r.interleaved ? c0 / 2 : c0));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 z = t[e];  // two pairs' (cos, sin)
        if (a.r.interleaved) {
          float* const p = e < 2 ? x0.v + 4 * e : x1.v + 4 * e - 8;
          rotate(p[0], p[1], z.x, z.y);
          rotate(p[2], p[3], z.z, z.w);
        } else {
          rotate(x0.v[2 * e], x1.v[2 * e], z.x, z.y);
          rotate(x0.v[2 * e + 1], x1.v[2 * e + 1], z.z, z.w);
        }
      }
    }
    if (codes) {
      const float s = is_v ? a.c.v_scale : a.c.k_scale, r = is_v ? a.v_inverse : a.k_inverse;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(to) + at + c0) = x0.e4m3(s, r);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(to) + at + c1) = x1.e4m3(s, r);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(to) + at + c0) = x0.bf16();
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(to) + at + c1) = x1.bf16();
    }
  }
  static __device__ __forceinline__ void rotate(float& x, float& y, float c, float s) {
    const float u = x;
    x = u * c - y * s;
    y = y * c + u * s;
  }
};

// What the turning warps have to know of a piece.
struct Piece {
  int row, first;   // its first head
  int page, slot;   // page -1: its keys and values are dropped
  int real;         // 0: a row that does not exist
};

// A row, or its next `a.heads` heads of queries, keys and values where it has more, is a
// piece.  CTAs take pieces in turn.  One warp of a CTA prepares them, as many ahead as its
// ring in shared memory holds: where the row is and goes to (a lane a piece, 32 of them at
// once), its angles, the bulk copies of its elements; the others turn and store them.
// (Every thread finding the rows by itself, with 600 integer instructions a warp and row and
// two barriers: 15.7 us for 128 x 16 rows into E4M3, 34 us for 2 x 4001.)
__global__ void __launch_bounds__(kRopeThreads + 32, 6) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ __align__(16) float2 turn[kRopeStages][128];  // (cos, sin) of the pieces' pairs
  __shared__ Piece s_piece[kRopeStages];
  __shared__ __align__(8) unsigned long long s_bar[2 * kRopeStages];
  const int half = a.r.rot / 2, rows = a.B * a.M, step = gridDim.x, total = rows * a.pieces;
  const int all = a.Hq + 2 * a.c.heads, head_bytes = a.c.head_dim * 2;
  const uint32_t full = smem_addr(s_bar), empty = full + kRopeStages * 8, ring_at = smem_addr(ring);
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(full + i * 8, 1);
      mbar_init(empty + i * 8, kRopeThreads / 32);
    }
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kRopeThreads / 32) {
    // this lane's pairs: turns a position, and the axis they go by
    unsigned long long turns[4];
    int axis[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = lane + 32 * k;
      turns[k] = j < half ? turns_of(a.r.inv_freq[j]) : 0;
      axis[k] = 0;
      if (a.r.positions != nullptr) {
        int end = a.r.sections[0];
#pragma unroll
        for (int x = 1; x < 4; ++x)
          if (x < a.r.axes && j >= end) {
            axis[k] = x;
            end += a.r.sections[x];
          }
      }
    }
    bool lost = false;
    int n = 0;
    for (int base = blockIdx.x; base < total && !lost; base += 32 * step) {
      // 32 pieces' rows
      const int mine = base + lane * step;
      Piece q = {0, 0, -1, 0, 0};
      int at[4] = {0, 0, 0, 0};
      if (mine < total) {
        q.row = a.pieces == 1 ? mine : mine / a.pieces;
        q.first = (mine - q.row * a.pieces) * a.heads;
        const int b = q.row / a.M, i = q.row - b * a.M, m = new_rows(a.q_lens, b, a.M), length = seq_length(a.c, b);
        q.real = i < m;
        const int pos = length - m + i;
        if (q.real) {
          if (a.r.positions == nullptr) at[0] = pos;
          else
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (x < a.r.axes) at[x] = a.r.positions[static_cast<int64_t>(x) * rows + q.row];
          if (pos >= 0) {
            q.page = static_cast<int>(token_page(a.c, b, pos));
            q.slot = pos % a.c.page_size;
          }
        }
      }
      for (int k = 0; k < 32 && base + k * step < total && !lost; ++k, ++n) {
        const int stage = n % a.stages;
        if (n >= a.stages)
          lost = __any_sync(0xffffffffu, !mbar_wait(empty + stage * 8, ((n / a.stages) & 1) ^ 1, kStatusTimeoutEmpty));
        if (lost) break;
        const int row = __shfl_sync(0xffffffffu, q.row, k), first = __shfl_sync(0xffffffffu, q.first, k),
                  real = __shfl_sync(0xffffffffu, q.real, k);
        if (lane == k) s_piece[stage] = q;
        if (real) {
          int p[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) p[x] = __shfl_sync(0xffffffffu, at[x], k);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (lane + 32 * x >= half) break;
            const int where = axis[x] == 0 ? p[0] : axis[x] == 1 ? p[1] : axis[x] == 2 ? p[2] : p[3];
            const unsigned long long t = turns[x] * static_cast<unsigned long long>(static_cast<long long>(where));
            const int top = static_cast<int>((t + 0x80000000ull) >> 32);
            float s, c;
            sincospif(static_cast<float>(top) * (1.f / 2147483648.f), &s, &c);
            turn[stage][lane + 32 * x] = make_float2(c * a.r.factor, s * a.r.factor);
          }
        }
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = full + stage * 8;
          if (!real) {
            mbar_arrive(bar);
          } else {
            const int end = min(first + a.heads, all);
            mbar_arrive_expect_tx(bar, (end - first) * head_bytes);
            auto part = [&](const uint16_t* from, int begin, int count) {  // heads begin .. begin + count - 1 of the row's list
              const int lo = max(first, begin), hi = min(end, begin + count);
              if (lo < hi)
                bulk_load(ring_at + stage * a.stage_bytes + (lo - first) * head_bytes,
                          from + static_cast<int64_t>(lo - begin) * a.c.head_dim, (hi - lo) * head_bytes, bar);
            };
            part(a.q + row * a.q_ld, 0, a.Hq);
            part(a.kn + row * a.k_ld, a.Hq, a.c.heads);
            part(a.vn + row * a.v_ld, a.Hq + a.c.heads, a.c.heads);
          }
        }
        __syncwarp();
      }
    }
    if (lost)  // copies that are still under way
      for (int i = max(n - a.stages, 0); i < n; ++i)
        if (__any_sync(0xffffffffu, !mbar_wait(full + i % a.stages * 8, (i / a.stages) & 1, kStatusTimeoutDrain))) break;
    return;
  }
  int n = 0;
  for (int piece = blockIdx.x; piece < total; piece += step, ++n) {
    const int stage = n % a.stages;
    if (__any_sync(0xffffffffu, !mbar_wait(full + stage * 8, (n / a.stages) & 1, kStatusTimeoutFull))) return;
    const Piece q = s_piece[stage];
    const int64_t row = q.row;
    if (q.real) {
      const unsigned char* const data = ring + stage * a.stage_bytes;
      const int items = min(a.heads, all - q.first) << a.per_head_log2;
      for (int x = threadIdx.x; x < items; x += kRopeThreads) {
        const Item item(a, q.first, x);
        if (!item.is_q && q.page < 0) continue;
        const unsigned char* const from = data + (x >> a.per_head_log2) * head_bytes;
        item.finish(a, turn[stage], row, q.page, q.slot, *reinterpret_cast<const uint4*>(from + item.c0 * 2),
                    *reinterpret_cast<const uint4*>(from + item.c1 * 2));
      }
    } else {
      const int chunks = min(a.heads, a.Hq - q.first) * (a.c.head_dim / 8);
      for (int x = threadIdx.x; x < chunks; x += kRopeThreads)
        *reinterpret_cast<uint4*>(a.out + row * a.out_ld + static_cast<int64_t>(q.first) * a.c.head_dim + x * 8) = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + stage * 8);
  }
}

}  // namespace

unsigned int read_rope_status(int clear) { return read_unit_status(clear); }

}  // namespace qmm

extern "C" qmm_status qmm_rope_append(const qmm_paged_cache* cache, const qmm_rope* rope, const void* q, int64_t q_ld, int q_heads,
                                      void* q_out, int64_t q_out_ld, const void* k_new, int64_t k_ld, const void* v_new,
                                      int64_t v_ld, int B, int M, const int32_t* q_lens, void* stream) {
  using namespace qmm;
  if (rope == nullptr) return QMM_ERR_NULL;
  const qmm_status rc = check_cache(cache, B, M, 0x7fffffff);
  if (rc != QMM_OK) return rc;
  const int64_t width = static_cast<int64_t>(cache->heads) * cache->head_dim, q_width = static_cast<int64_t>(q_heads) * cache->head_dim;
  if (q_heads < 1 || q_heads > 65535 || k_ld < width || v_ld < width || q_ld < q_width || q_out_ld < q_width ||
      static_cast<int64_t>(B) * M > 0x7fff0000 || rope->rot < 0 || rope->rot > cache->head_dim || rope->rot % 16 != 0)
    return QMM_ERR_SHAPE;
  if (rope->positions != nullptr) {
    if (rope->axes < 1 || rope->axes > 4) return QMM_ERR_UNSUPPORTED;
    int64_t pairs = 0;
    for (int i = 0; i < rope->axes; ++i) {
      if (rope->sections[i] < 0) return QMM_ERR_SHAPE;
      pairs += rope->sections[i];
    }
    if (pairs != rope->rot / 2) return QMM_ERR_SHAPE;
  }
  if (!std::isfinite(rope->factor)) return QMM_ERR_UNSUPPORTED;
  if (B == 0 || M == 0) return QMM_OK;
  if (q == nullptr || q_out == nullptr || k_new == nullptr || v_new == nullptr || (rope->inv_freq == nullptr && rope->rot > 0))
    return QMM_ERR_NULL;
  if (misaligned(reinterpret_cast<intptr_t>(q), 16) || misaligned(reinterpret_cast<intptr_t>(q_out), 16) ||
      misaligned(reinterpret_cast<intptr_t>(k_new), 16) || misaligned(reinterpret_cast<intptr_t>(v_new), 16) ||
      misaligned(q_ld, 8) || misaligned(q_out_ld, 8) || misaligned(k_ld, 8) || misaligned(v_ld, 8) ||
      misaligned(reinterpret_cast<intptr_t>(rope->inv_freq), 4) || misaligned(reinterpret_cast<intptr_t>(rope->positions), 4) ||
      misaligned(reinterpret_cast<intptr_t>(q_lens), 4))
    return QMM_ERR_ALIGN;
  RopeArgs a = {};
  a.c = *cache;
  a.r = *rope;
  a.q = static_cast<const uint16_t*>(q);
  a.kn = static_cast<const uint16_t*>(k_new);
  a.vn = static_cast<const uint16_t*>(v_new);
  a.out = static_cast<uint16_t*>(q_out);
  a.q_ld = q_ld;
  a.out_ld = q_out_ld;
  a.k_ld = k_ld;
  a.v_ld = v_ld;
  a.B = B;
  a.M = M;
  a.Hq = q_heads;
  a.q_lens = q_lens;
  a.per_head_log2 = __builtin_ctz(static_cast<unsigned>(cache->head_dim / 16));
  const auto inverse = [](float s) {
    int e;
    return s > 0x1p-100f && s < 0x1p100f && std::frexp(s, &e) == 0.5f ? 1.f / s : 0.f;
  };
  a.k_inverse = inverse(cache->k_scale);
  a.v_inverse = inverse(cache->v_scale);
  const int64_t all = q_heads + 2 * static_cast<int64_t>(cache->heads), head_bytes = cache->head_dim * 2;
  a.heads = static_cast<int>(std::min<int64_t>(all, kRopePiece / head_bytes));
  a.pieces = static_cast<int>((all + a.heads - 1) / a.heads);
  a.stage_bytes = static_cast<int>(a.heads * head_bytes);
  a.stages = std::min(kRopeStages, kRopeRing / a.stage_bytes);
  const int64_t total = static_cast<int64_t>(B) * M * a.pieces;
  const int64_t ctas = std::min<int64_t>(total, 6 * device_sm_count());  // as many as the SMs hold
  if (total > 0x7fffffff - 64 * ctas) return QMM_ERR_SHAPE;  // (pieces are numbered in 32 bits, some ahead of the last)
  return static_cast<qmm_status>(finish_call(launch_dependent(rope_append_kernel, dim3(static_cast<unsigned>(ctas)), kRopeThreads + 32,
                                                              static_cast<size_t>(a.stages) * a.stage_bytes,
                                                              static_cast<cudaStream_t>(stream), a)));
}
