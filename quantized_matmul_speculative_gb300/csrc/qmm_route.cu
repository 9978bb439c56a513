// Routing of tokens to experts (qmm_route_experts, include/qmm.h).
//
// A warp takes a token; its lanes hold the row, LPG neighbouring lanes a group (the
// largest power of two of which all groups fit into the warp), each up to PER
// neighbouring experts of it, so that lower lanes and places are lower experts.
//
// The mathematics.  What orders the experts (logits, or scores with the bias) is put on a
// scale of 2^23 steps between the row's greatest and its least that is not masked, with the
// expert's number, the lowest first, in the 9 bits below: one unsigned key each, no two
// alike.  Every lane sorts its own keys once; then k rounds take the largest of the lanes'
// first ones.  Keys nearer than the steps' and the scores' own errors (or than one step,
// where logits are compared) may be in the wrong order, unless they are the same logit with
// the same bias.  So the chosen ones are held against their neighbours, and the last of them
// against every key that is left that near to it, as of equals in 32 bits a better one may
// lie anywhere behind.
// Where one of those pairs is not the same logit with the same bias, in some tokens of a
// thousand, the warp does the token again in 64 bits, one maximum after another.  The errors:
// a sigmoid from the approximate exponential and reciprocal is off by 4 2^-24, a softmax by
// 24 2^-24 (exponentials 2 units in the last place each, a sum of 512 in 31 + 5 steps), a
// key's own rounding is |key| 2^-24; so two keys more than kGap (1 + |key|) apart are in their
// order, with kGap 2^-20 and 2^-18.  Groups likewise, with the sizes of both terms of a worth.
//
// What bounds it: instructions, 974 a token of 256 experts in 8 groups (62% of the issue
// slots, 57% of the integer pipe): 16384 tokens 33 to 37 us by the inputs, at a floor of 2.7.
// One token: 5 us, a launch and a chain.  As many lanes hold keys as there are experts, so that few experts
// cost much for their bytes (243398 tokens of 16: 135 us).
#include <cfloat>
#include <climits>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kRouteWarps = 4;
constexpr float kMasked = -4096.f;
constexpr float kGapSigmoid = 1.f / (1 << 20), kGapSoftmax = 1.f / (1 << 18);

struct RouteArgs {
  const void* x;
  int64_t ld;
  const float* bias;
  int32_t* experts;
  float* weights;
  int T, E, k, f32, sigmoid, groups, top_groups, group_best, renormalize;
  int size, lpg_log2, per;  // experts of a group; lanes of a group; experts of a lane
  float scale;
};

// Keys as unsigned numbers in their order; 0 is none.  NaN counts as -inf.
__device__ __forceinline__ uint32_t ordered(float v) {
  v = v == v ? v : -INFINITY;
  const uint32_t u = __float_as_uint(v + 0.f);  // (-0 is 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long ordered(double v) {
  v = v == v ? v : -static_cast<double>(INFINITY);
  const unsigned long long u = __double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ float value_of(uint32_t u) {
  return u == 0 ? -INFINITY : __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<unsigned long long>(hi) << 32 | lo;
}
__device__ __forceinline__ float warp_max(float v) { return value_of(warp_max(ordered(v))); }
template <class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int s = 16; s > 0; s /= 2) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}
// e^-by / (1 + e^-x), where by is x at least if x is negative, else 0.
__device__ __forceinline__ float sigmoid_of(float x, float by) {
  return (x < 0.f ? expf(x - by) : 1.f) / (1.f + expf(-fabsf(x)));
}
// The same within 4 2^-24, absolutely.
__device__ __forceinline__ float sigmoid_near(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
// NaN logits count as -inf, +inf as the largest number.
__device__ __forceinline__ float clean(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }
__device__ __forceinline__ float logit_of(const RouteArgs& a, int64_t t, int e) {
  return clean(a.f32 ? static_cast<const float*>(a.x)[t * a.ld + e]
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(a.x)[t * a.ld + e]));
}

// The best one or two of v[0 .. PER - 1] and of the neighbouring lanes of a group; `size`: of these terms, as numbers
// that cancel keep both their errors.
template <class F, int PER>
__device__ __forceinline__ F group_worth(const RouteArgs& a, const F (&v)[PER], F& size) {
  F best = -F(INFINITY), second = -F(INFINITY);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    second = v[i] > best ? best : v[i] > second ? v[i] : second;
    best = v[i] > best ? v[i] : best;
  }
  for (int s = 1; s < (1 << a.lpg_log2); s *= 2) {
    const F b = __shfl_xor_sync(0xffffffffu, best, s), c = __shfl_xor_sync(0xffffffffu, second, s);
    second = b > best ? (best > c ? best : c) : (b > second ? b : second);
    best = b > best ? b : best;
  }
  const bool both = a.group_best == 2 && second > -F(INFINITY);
  size = both ? fabs(best) + fabs(second) : fabs(best);
  return both ? best + second : best;
}

// Whether this lane's group is open, from its groups' worths; `last` the least that is, `left` the best that is not.
template <class Key>
__device__ __forceinline__ bool open_groups(const RouteArgs& a, Key worth, Key& last, Key& left) {
  const int lane = threadIdx.x & 31;
  bool in = false;
  for (int j = 0; j < a.top_groups; ++j) {
    last = warp_max(worth);
    const int at = __ffs(__ballot_sync(0xffffffffu, worth == last)) - 1;
    if (lane >> a.lpg_log2 == at >> a.lpg_log2) {
      in = true;
      worth = Key(0);
    }
  }
  left = warp_max(worth);
  return in;
}

// `mine` of a row's values from `first` on, others -inf.  Those of a group's neighbouring
// lanes lie behind them, so that whole 16-byte chunks serve the usual sizes.
template <int PER>
__device__ __forceinline__ void load_floats(const float* row, int mine, float (&x)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = -INFINITY;
  if (PER % 4 == 0 && mine == PER && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
#pragma unroll
    for (int i = 0; i < PER / 4; ++i) {
      const uint4 u = ld_after_wait_v4(row + 4 * i);
      x[4 * i] = __uint_as_float(u.x), x[4 * i + 1] = __uint_as_float(u.y);
      x[4 * i + 2] = __uint_as_float(u.z), x[4 * i + 3] = __uint_as_float(u.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < mine) x[i] = row[i];
  }
}
template <int PER>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t t, int first, int mine, float (&x)[PER]) {
  if (a.f32) {
    load_floats(static_cast<const float*>(a.x) + t * a.ld + first, mine, x);
    return;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = -INFINITY;
  const __nv_bfloat16* const row = static_cast<const __nv_bfloat16*>(a.x) + t * a.ld + first;
  if (PER % 4 == 0 && mine == PER && (reinterpret_cast<uintptr_t>(row) & 7) == 0) {
#pragma unroll
    for (int i = 0; i < PER / 4; ++i) {
      const uint2 u = ld_after_wait_v2(row + 4 * i);
      x[4 * i] = bf16_lo(u.x), x[4 * i + 1] = bf16_hi(u.x), x[4 * i + 2] = bf16_lo(u.y), x[4 * i + 3] = bf16_hi(u.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < mine) x[i] = __bfloat162float(row[i]);
  }
}

struct Lanes {  // this lane's experts: `mine` from `first` on
  int first, mine;
  bool real;  // of a group
  __device__ __forceinline__ explicit Lanes(const RouteArgs& a) {
    const int lane = threadIdx.x & 31, group = lane >> a.lpg_log2, inside = (lane & ((1 << a.lpg_log2) - 1)) * a.per;
    real = group < a.groups;
    first = group * a.size + inside;
    mine = real ? min(a.per, a.size - inside) : 0;
  }
};

// A token's choice in 64 bits: lane j < k gets the j-th expert.
template <int PER>
__device__ __noinline__ int choose_exactly(const RouteArgs& a, int64_t t) {
  using Key = unsigned long long;
  const int lane = threadIdx.x & 31;
  const Lanes l(a);
  const bool biased = a.bias != nullptr, grouped = a.top_groups < a.groups, by_sum = grouped && a.group_best == 2;
  float x[PER];
  load_row(a, t, l.first, l.mine, x);
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = clean(x[i]);
  Key key[PER];
  double worth[PER];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, x[i]);
  top = warp_max(top);
  double total = 1.0;
  if (!a.sigmoid && (biased || by_sum)) {
    double s = 0.0;
    for (int i = 0; i < PER; ++i)
      if (i < l.mine && x[i] != -INFINITY) s += exp(static_cast<double>(x[i]) - top);
    total = warp_sum(s);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    double v = x[i];
    worth[i] = v;
    if ((biased || by_sum) && x[i] != -INFINITY) {
      const double e = exp(a.sigmoid ? (v < 0.0 ? v : -v) : v - top);
      worth[i] = a.sigmoid ? (v < 0.0 ? e : 1.0) / (1.0 + e) : e / total;
      if (biased) worth[i] += a.bias[l.first + i];
      worth[i] = worth[i] == worth[i] ? worth[i] : -static_cast<double>(INFINITY);
      if (biased) v = worth[i];
    }
    key[i] = i < l.mine ? ordered(v) : Key(0);
  }
  if (grouped) {
    double size;
    const Key of_group = ordered(group_worth(a, worth, size));  // (every lane takes part in it)
    Key last, left;
    if (!open_groups(a, l.real ? of_group : Key(0), last, left))
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = Key(0);
  }
  int expert = 0;
  for (int j = 0; j < a.k; ++j) {
    Key m = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < PER; ++i)
      if (key[i] > m) {
        m = key[i];
        at = i;
      }
    const int src = __ffs(__ballot_sync(0xffffffffu, m == warp_max(m))) - 1;
    const int e = __shfl_sync(0xffffffffu, l.first + at, src);
    if (lane == j) expert = e;
    if (lane == src)
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i == at) key[i] = Key(0);
  }
  return expert;
}

// Descending, by merging odd and even places.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t hi = max(v[i + j], v[i + j + k]), lo = min(v[i + j], v[i + j + k]);
            v[i + j] = hi;
            v[i + j + k] = lo;
          }
}

// One token, by its warp.
template <int PER>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, int lane, const Lanes& l, const float (&bias)[PER],
                                            float (&x)[PER]) {
  const bool biased = a.bias != nullptr, grouped = a.top_groups < a.groups, by_sum = grouped && a.group_best == 2;
  const float gap = a.sigmoid ? kGapSigmoid : kGapSoftmax;
  float ref = 0.f, total = 1.f;
  if (!a.sigmoid) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) top = fmaxf(top, x[i]);
    top = warp_max(top);
    ref = top == -INFINITY ? 0.f : top;
    if (biased || by_sum || !a.renormalize) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) s += expf(x[i] - ref);  // (0 for experts that do not exist)
      total = warp_sum(s);
    }
  }
  // what orders the experts, and what they are worth in their groups
  float worth[PER];
  if (biased || by_sum) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      float v = a.sigmoid ? sigmoid_near(x[i]) : expf(x[i] - ref) / total;
      if (biased) v += bias[i];
      worth[i] = x[i] != -INFINITY && v == v ? v : -INFINITY;
      if (biased) x[i] = worth[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) worth[i] = x[i];
  }
  bool apart = true, open = l.real;
  if (grouped) {
    float size;
    const float mine = group_worth(a, worth, size);  // (every lane takes part in it)
    uint32_t last, left;
    open = open_groups(a, l.real ? ordered(mine) : 0u, last, left);
    const float hi = value_of(last), lo = value_of(left), between = 0.5f * hi + 0.5f * lo, off = gap * (1.f + size);
    // every group on its side of what lies between the open and the others (-inf is exact; with +inf nothing is told)
    if (biased || by_sum)
      apart = open ? mine - off > between || (hi == -INFINITY && mine == hi) : !l.real || mine == -INFINITY || mine + off < between;
  }
  // The scale: 3 .. 2^23 - 5 from the least that is not masked by a large negative number (-1e4 and less are in use); 2 for
  // those, among which 64 bits choose if it comes to them, and 1 for -inf.  (Where -1e9 is on the scale a step is 119 wide, and
  // every token goes to 64 bits: 16384 x 256 softmax 53 us, and 18.1; masked by their distance from the greatest, which has to
  // be known before: 19.5 for any row.)
  float hi = -INFINITY, lo = INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    hi = fmaxf(hi, x[i]);
    if (x[i] > kMasked) lo = fminf(lo, x[i]);
  }
  hi = warp_max(hi);
  lo = -warp_max(-lo);
  const float range = hi - lo;
  apart = apart && range < FLT_MAX / 2;  // (also where all are -inf)
  const float unit = range > 0.f ? 8388600.f / range : 0.f;
  apart = apart && unit < FLT_MAX;
  const uint32_t margin = biased ? static_cast<uint32_t>(fminf(gap * (1.f + fmaxf(fabsf(hi), fabsf(lo))) * unit, 8388608.f)) + 4u : 1u;
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t step = x[i] == -INFINITY ? 1u : 2u + __float2uint_rz(fmaf(x[i] - lo, unit, 1.f));  // (below 0: 0)
    key[i] = open && i < l.mine ? step << 9 | (511u - (l.first + i)) : 0u;
  }
  sort_down(key);
  uint32_t mine = 0;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t next = warp_max(key[0]);
    if (lane == j) mine = next;
    const bool taken = key[0] == next;
#pragma unroll
    for (int i = 0; i + 1 < PER; ++i) key[i] = taken ? key[i + 1] : key[i];
    if (taken) key[PER - 1] = 0u;
  }
  int expert = 511 - static_cast<int>(mine & 511u);
  float logit = lane < a.k ? logit_of(a, t, expert) : 0.f;
  {
    const float its_bias = biased && lane < a.k ? a.bias[expert] : 0.f;
    const auto same = [](float x, float b, float y, float c) { return x == y && (b == c || x == -INFINITY); };
    // neighbours among the chosen ones
    const uint32_t below = __shfl_down_sync(0xffffffffu, mine, 1);
    const float x_below = __shfl_down_sync(0xffffffffu, logit, 1), b_below = __shfl_down_sync(0xffffffffu, its_bias, 1);
    bool told = lane >= a.k - 1 || (mine >> 9) - (below >> 9) >= margin || same(logit, its_bias, x_below, b_below);
    // the last of them, and what is left
    const uint32_t last = __shfl_sync(0xffffffffu, mine, a.k - 1);
    const auto near = [&](uint32_t k) { return k != 0u && (last >> 9) - (k >> 9) < margin; };
    if (__any_sync(0xffffffffu, near(key[0]))) {
      const float x_last = __shfl_sync(0xffffffffu, logit, a.k - 1), b_last = __shfl_sync(0xffffffffu, its_bias, a.k - 1);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (near(key[i])) {
          const int e = 511 - static_cast<int>(key[i] & 511u);
          told = told && same(x_last, b_last, logit_of(a, t, e), biased ? a.bias[e] : 0.f);
        }
    }
    apart = __all_sync(0xffffffffu, told && apart);
  }
  if (!apart) {
    expert = choose_exactly<PER>(a, t);
    if (lane < a.k) logit = logit_of(a, t, expert);
  }
  // the weights, from the k logits
  const float best = warp_max(lane < a.k ? logit : -INFINITY);
  float w = 0.f;
  if (lane < a.k && logit != -INFINITY) {
    // (of sigmoids the ratios count: all are taken e^-best times where best is negative, so that none is lost below 32 bits' range)
    if (a.renormalize) w = a.sigmoid ? sigmoid_of(logit, fminf(best, 0.f)) : expf(logit - best);
    else w = a.sigmoid ? sigmoid_of(logit, 0.f) : expf(logit - ref) / total;
  }
  if (a.renormalize) {
    const float sum = warp_sum(w);
    w = sum > 0.f ? w / sum : 0.f;
  }
  if (lane < a.k) {
    a.experts[t * a.k + lane] = expert;
    a.weights[t * a.k + lane] = w * a.scale;
  }
}

template <int PER>
__global__ void __launch_bounds__(32 * kRouteWarps, PER <= 8 ? 5 : 2) route_kernel(const __grid_constant__ RouteArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, step_t = gridDim.x * kRouteWarps;
  int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const Lanes l(a);
  float bias[PER], x[PER], ahead[PER];
  if (a.bias != nullptr) load_floats(a.bias + l.first, l.mine, bias);
  load_row(a, t, l.first, l.mine, ahead);
  // a warp's tokens, the next one's logits under way
  for (; t < a.T; t += step_t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = clean(ahead[i]);
    if (t + step_t < a.T) load_row(a, t + step_t, l.first, l.mine, ahead);
    route_token(a, t, lane, l, bias, x);
  }
}

template <int PER>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  // as many CTAs as the SMs hold, each warp with every so manieth token
  const int ctas = (a.T + kRouteWarps - 1) / kRouteWarps, most = (PER <= 8 ? 5 : 2) * device_sm_count();
  return launch_dependent(route_kernel<PER>, dim3(ctas < most ? ctas : most), 32 * kRouteWarps, 0, stream, a);
}

}  // namespace
}  // namespace qmm

extern "C" qmm_status qmm_route_experts(const void* logits, int logits_dtype, int64_t ld, const float* bias, int T, int E, int k,
                                        int scoring, int groups, int top_groups, int group_best, int renormalize, float scale,
                                        int32_t* experts, float* weights, void* stream) {
  using namespace qmm;
  if (T < 0 || T > 0x7fff0000 || E < 1 || E > 512 || k < 1 || k > 32 || ld < E || groups < 1 || groups > 32 || E % groups != 0 ||
      top_groups < 1 || top_groups > groups || k > top_groups * (E / groups))
    return QMM_ERR_SHAPE;
  if ((logits_dtype != QMM_OUT_BF16 && logits_dtype != QMM_OUT_F32) || (scoring != QMM_SOFTMAX && scoring != QMM_SIGMOID) ||
      (group_best != 1 && group_best != 2))
    return QMM_ERR_UNSUPPORTED;
  if (T == 0) return QMM_OK;
  if (logits == nullptr || experts == nullptr || weights == nullptr) return QMM_ERR_NULL;
  const uintptr_t esize = logits_dtype == QMM_OUT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % esize || (reinterpret_cast<uintptr_t>(bias) | reinterpret_cast<uintptr_t>(experts) |
                                                      reinterpret_cast<uintptr_t>(weights)) % 4)
    return QMM_ERR_ALIGN;
  RouteArgs a = {};
  a.x = logits;
  a.ld = ld;
  a.bias = bias;
  a.experts = experts;
  a.weights = weights;
  a.T = T;
  a.E = E;
  a.k = k;
  a.f32 = logits_dtype == QMM_OUT_F32;
  a.sigmoid = scoring == QMM_SIGMOID;
  a.groups = groups;
  a.top_groups = top_groups;
  a.group_best = group_best;
  a.renormalize = renormalize != 0;
  a.scale = scale;
  a.size = E / groups;
  a.lpg_log2 = 0;
  while ((groups << (a.lpg_log2 + 1)) <= 32) ++a.lpg_log2;
  a.per = (a.size + (1 << a.lpg_log2) - 1) >> a.lpg_log2;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.per <= 1   ? launch_route<1>(a, st)
                        : a.per <= 2 ? launch_route<2>(a, st)
                        : a.per <= 4 ? launch_route<4>(a, st)
                        : a.per <= 8 ? launch_route<8>(a, st)
                        : a.per <= 16 ? launch_route<16>(a, st)
                                      : launch_route<32>(a, st);
  return static_cast<qmm_status>(finish_call(e));
}
