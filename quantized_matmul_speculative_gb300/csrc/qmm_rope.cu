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
// A CTA takes rows, one after another: its threads compute the row's angles once for all
// heads, while the row's elements are on their way.
#include <cmath>

#include "qmm_cache.cuh"

namespace qmm {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  qmm_paged_cache c;
  qmm_rope r;
  const uint16_t *q, *kn, *vn;
  uint16_t* out;
  int64_t q_ld, out_ld, k_ld, v_ld;
  int B, M, Hq, per_head_log2;  // items of a head
  float k_inverse, v_inverse;   // of the scales that are powers of two, else 0
  const int32_t* q_lens;
};

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
  // Quotients by s: products with its inverse r where s is a power of two, which are the same (r = 0: it is not).
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

// Item x of a row: two chunks of 8 elements of a head that turn together, or neighbours.
struct Item {
  int h, c0, c1;     // head; first elements of the chunks
  bool is_q, is_v, turned;
  __device__ __forceinline__ Item(const RopeArgs& a, int x) {
    const int head = x >> a.per_head_log2, j = x - (head << a.per_head_log2), half = a.r.rot / 2;
    is_q = head < a.Hq;
    is_v = head >= a.Hq + a.c.heads;
    h = is_q ? head : is_v ? head - a.Hq - a.c.heads : head - a.Hq;
    turned = !is_v && j < half / 8;
    const bool halves = turned && !a.r.interleaved;
    c0 = halves ? j * 8 : j * 16;
    c1 = halves ? half + j * 8 : j * 16 + 8;
  }
  __device__ __forceinline__ void load(const RopeArgs& a, int64_t row, uint4& u, uint4& w) const {
    const uint16_t* const src =
        (is_q ? a.q + row * a.q_ld : is_v ? a.vn + row * a.v_ld : a.kn + row * a.k_ld) + static_cast<int64_t>(h) * a.c.head_dim;
    u = ld_after_wait_v4(src + c0);
    w = ld_after_wait_v4(src + c1);
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

// What a CTA knows of a row ahead of its turn.
struct RowAhead {
  int row, m, length, i, b;  // m and the length are asked for first, ..
  int pos, slot, entry;      // .. then the table's entry
  __device__ __forceinline__ void ask(const RopeArgs& a, int r, int rows) {
    row = r;
    if (r >= rows) return;
    b = r / a.M;
    i = r - b * a.M;
    m = a.q_lens != nullptr ? a.q_lens[b] : a.M;
    length = a.c.lengths[b];
  }
  __device__ __forceinline__ bool real(int rows) const { return row < rows && i < m; }
  // (as seq_length and new_rows; bad lengths set the status bit)
  __device__ __forceinline__ void place(const RopeArgs& a, int rows) {
    entry = -1;
    slot = 0;
    if (row >= rows) return;
    m = max(0, min(m, a.M));
    const int cap = a.c.max_pages * a.c.page_size;
    if (length < 0 || length > cap) {
      bad_page();
      length = length < 0 ? 0 : cap;
    }
    pos = length - m + i;
    if (i >= m || pos < 0) return;
    const int block = pos / a.c.page_size;
    slot = pos - block * a.c.page_size;
    entry = a.c.block_table[b * a.c.table_stride + block];
  }
  __device__ __forceinline__ int64_t page(const RopeArgs& a) const {
    if (pos < 0) return -1;
    if (entry < 0 || entry >= a.c.num_pages) {
      bad_page();
      return -1;
    }
    return entry;
  }
};

// While a row is turned, the next one's first 512 items and table entry are under way,
// and the lengths of the one after it.
__global__ void __launch_bounds__(kRopeThreads, 3) rope_append_kernel(const RopeArgs a) {
  constexpr int AHEAD = 2;
  __shared__ __align__(16) float2 turn[2][128];  // (cos, sin) of a row's pairs, two rows in turn
  griddep_wait();
  griddep_launch_dependents();
  const int half = a.r.rot / 2, items = (a.Hq + 2 * a.c.heads) << a.per_head_log2;
  const int rows = a.B * a.M, step = gridDim.x;
  uint4 u[AHEAD], w[AHEAD], u2[AHEAD], w2[AHEAD];
  auto load = [&](uint4 (&p)[AHEAD], uint4 (&q)[AHEAD], const RowAhead& r) {
    if (!r.real(rows)) return;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int x = threadIdx.x + k * kRopeThreads;
      if (x < items) Item(a, x).load(a, r.row, p[k], q[k]);
    }
  };
  int flip = 0;
  auto turn_row = [&](const RowAhead& r, const uint4 (&p)[AHEAD], const uint4 (&q)[AHEAD]) {
    const int64_t row = r.row;
    if (r.i >= r.m) {
      for (int x = threadIdx.x; x < a.Hq * a.c.head_dim / 8; x += kRopeThreads)
        *reinterpret_cast<uint4*>(a.out + row * a.out_ld + x * 8) = make_uint4(0, 0, 0, 0);
      return;
    }
    flip ^= 1;  // (who passes the barrier of a row has read the angles of the one before the last)
    for (int j = threadIdx.x; j < half; j += kRopeThreads) {
      int at = r.pos;
      if (a.r.positions != nullptr) {
        int axis = 0, end = a.r.sections[0];
        while (axis + 1 < a.r.axes && j >= end) end += a.r.sections[++axis];
        at = a.r.positions[static_cast<int64_t>(axis) * rows + row];
      }
      const unsigned long long t = turns_of(a.r.inv_freq[j]) * static_cast<unsigned long long>(static_cast<long long>(at));
      const int top = static_cast<int>((t + 0x80000000ull) >> 32);
      float s, c;
      sincospif(static_cast<float>(top) * (1.f / 2147483648.f), &s, &c);
      turn[flip][j] = make_float2(c * a.r.factor, s * a.r.factor);
    }
    __syncthreads();
    const int64_t page = r.page(a);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int x = threadIdx.x + k * kRopeThreads;
      if (x >= items) break;
      const Item item(a, x);
      if (item.is_q || page >= 0) item.finish(a, turn[flip], row, page, r.slot, p[k], q[k]);
    }
    for (int x = threadIdx.x + AHEAD * kRopeThreads; x < items; x += kRopeThreads) {
      const Item item(a, x);
      if (!item.is_q && page < 0) continue;
      uint4 y, z;
      item.load(a, row, y, z);
      item.finish(a, turn[flip], row, page, r.slot, y, z);
    }
  };
  RowAhead now, next;
  now.ask(a, blockIdx.x, rows);
  next.ask(a, blockIdx.x + step, rows);
  load(u, w, now);
  now.place(a, rows);
  while (now.row < rows) {
    RowAhead after;
    after.ask(a, next.row + step, rows);
    load(u2, w2, next);
    next.place(a, rows);
    turn_row(now, u, w);
    now = next;
    next = after;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      u[k] = u2[k];
      w[k] = w2[k];
    }
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
  const int64_t rows = static_cast<int64_t>(B) * M;
  const int64_t ctas = rows < 3 * device_sm_count() ? rows : 3 * device_sm_count();  // as many as the SMs hold
  return static_cast<qmm_status>(finish_call(launch_dependent(rope_append_kernel, dim3(static_cast<unsigned>(ctas)), kRopeThreads, 0,
                                                              static_cast<cudaStream_t>(stream), a)));
}
