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
  int B, M, Hq;
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
  __device__ __forceinline__ uint2 e4m3(float s) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cvt_e4m3(__fdiv_rn(v[2 * i], s), __fdiv_rn(v[2 * i + 1], s));
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  }
};

__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs a) {
  __shared__ float2 turn[128];  // (cos, sin) of the row's pairs
  griddep_wait();
  griddep_launch_dependents();
  const int D = a.c.head_dim, half = a.r.rot / 2, per_head = D / 16, Hkv = a.c.heads;
  const int items = (a.Hq + 2 * Hkv) * per_head;
  const int64_t rows = static_cast<int64_t>(a.B) * a.M;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int b = static_cast<int>(row / a.M), i = static_cast<int>(row - static_cast<int64_t>(b) * a.M);
    const int m = new_rows(a.q_lens, b, a.M);
    if (i >= m) {
      for (int x = threadIdx.x; x < a.Hq * D / 8; x += kRopeThreads)
        *reinterpret_cast<uint4*>(a.out + row * a.out_ld + x * 8) = make_uint4(0, 0, 0, 0);
      continue;
    }
    const int pos = seq_length(a.c, b) - m + i;
    __syncthreads();  // (the row before: done with its angles)
    for (int j = threadIdx.x; j < half; j += kRopeThreads) {
      int p = pos;
      if (a.r.positions != nullptr) {
        int axis = 0, end = a.r.sections[0];
        while (axis + 1 < a.r.axes && j >= end) end += a.r.sections[++axis];
        p = a.r.positions[axis * rows + row];
      }
      const unsigned long long t = turns_of(a.r.inv_freq[j]) * static_cast<unsigned long long>(static_cast<long long>(p));
      const int top = static_cast<int>((t + 0x80000000ull) >> 32);
      float s, c;
      sincospif(static_cast<float>(top) * (1.f / 2147483648.f), &s, &c);
      turn[j] = make_float2(c * a.r.factor, s * a.r.factor);
    }
    __syncthreads();
    int64_t page = -1;
    int slot = 0;
    if (pos >= 0) {
      page = token_page(a.c, b, pos);
      slot = pos % a.c.page_size;
    }
    for (int x = threadIdx.x; x < items; x += kRopeThreads) {
      const int head = x / per_head, j = x - head * per_head;
      const bool is_q = head < a.Hq, is_v = head >= a.Hq + Hkv;
      const int h = is_q ? head : is_v ? head - a.Hq - Hkv : head - a.Hq;
      if (!is_q && page < 0) continue;
      // the item's two chunks of 8 elements
      const bool turned = !is_v && j < half / 8;
      const bool halves = turned && !a.r.interleaved;
      const int c0 = halves ? j * 8 : j * 16, c1 = halves ? half + j * 8 : j * 16 + 8;
      const uint16_t* const src = (is_q ? a.q + row * a.q_ld : is_v ? a.vn + row * a.v_ld : a.kn + row * a.k_ld) + h * D;
      Eight x0, x1;
      x0.set(*reinterpret_cast<const uint4*>(src + c0));
      x1.set(*reinterpret_cast<const uint4*>(src + c1));
      if (halves) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 t = turn[j * 8 + e];
          const float u = x0.v[e], w = x1.v[e];
          x0.v[e] = u * t.x - w * t.y;
          x1.v[e] = w * t.x + u * t.y;
        }
      } else if (turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 t = turn[j * 8 + e];
          float* const p = e < 4 ? x0.v + 2 * e : x1.v + 2 * e - 8;
          const float u = p[0], w = p[1];
          p[0] = u * t.x - w * t.y;
          p[1] = w * t.x + u * t.y;
        }
      }
      if (is_q) {
        uint16_t* const to = a.out + row * a.out_ld + h * D;
        *reinterpret_cast<uint4*>(to + c0) = x0.bf16();
        *reinterpret_cast<uint4*>(to + c1) = x1.bf16();
      } else {
        const int64_t at = is_v ? page * a.c.v_page + slot * a.c.v_token + h * a.c.v_head
                                : page * a.c.k_page + slot * a.c.k_token + h * a.c.k_head;
        void* const cache = is_v ? a.c.v : a.c.k;
        if (a.c.dtype == QMM_KV_BF16) {
          uint16_t* const to = static_cast<uint16_t*>(cache) + at;
          *reinterpret_cast<uint4*>(to + c0) = x0.bf16();
          *reinterpret_cast<uint4*>(to + c1) = x1.bf16();
        } else {
          const float s = is_v ? a.c.v_scale : a.c.k_scale;
          uint8_t* const to = static_cast<uint8_t*>(cache) + at;
          *reinterpret_cast<uint2*>(to + c0) = x0.e4m3(s);
          *reinterpret_cast<uint2*>(to + c1) = x1.e4m3(s);
        }
      }
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
      static_cast<int64_t>(B) * M > 0x7fffffff || rope->rot < 0 || rope->rot > cache->head_dim || rope->rot % 16 != 0)
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
  const int64_t rows = static_cast<int64_t>(B) * M;
  const int64_t ctas = rows < 64 * device_sm_count() ? rows : 64 * device_sm_count();
  return static_cast<qmm_status>(finish_call(launch_dependent(rope_append_kernel, dim3(static_cast<unsigned>(ctas)), kRopeThreads, 0,
                                                              static_cast<cudaStream_t>(stream), a)));
}
