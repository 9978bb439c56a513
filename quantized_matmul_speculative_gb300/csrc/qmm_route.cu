// Routing of tokens to experts (qmm_route_experts, include/qmm.h).
//
// A warp takes a token; its lanes hold the row, LPG neighbouring lanes a group (the
// largest power of two of which all groups fit into the warp), each up to PER
// neighbouring experts of it, so that lower lanes and places are lower experts.  The k
// best are taken one after another: a maximum of ordered keys over the warp, the first
// lane that holds it, the first of its places.
//
// The mathematics.  Keys of score + bias are compared in 64 bits, where two that lie
// close together decide whole numbers.  They are computed in 32 bits first: a score is
// then off by at most a few 2^-24 (expf, a sum and a division), a key by another
// rounding of itself, so that a gap of kGap (1 + |key|) = 2^-19 (1 + |key|) between all
// neighbours down to the first expert that is left out, and between the last group taken
// and the first left, shows that 64 bits would choose the same.  Else (about one token
// in a thousand) the warp does the token again in 64 bits.  Without a bias the logits
// are the keys, exactly.
//
// What bounds it: instructions of the k rounds, and one launch for few tokens.
#include <cfloat>
#include <climits>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kRouteWarps = 8;
constexpr float kGap = 1.f / (1 << 18);

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
__device__ __forceinline__ double value_of(unsigned long long u) {
  return u == 0 ? -static_cast<double>(INFINITY) : __longlong_as_double(u >> 63 ? u & ~(1ull << 63) : ~u);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<unsigned long long>(hi) << 32 | lo;
}
__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
template <class F>
__device__ __forceinline__ F sigmoid(F x) {
  const F e = exp_of(x < F(0) ? x : -x);
  return (x < F(0) ? e : F(1)) / (F(1) + e);
}
template <class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int s = 16; s > 0; s /= 2) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}
template <class F>
struct KeyOf { using type = uint32_t; };
template <>
struct KeyOf<double> { using type = unsigned long long; };

// A token's choice, with keys in F: lane j < k gets the j-th expert and its logit.
// False: F does not tell two neighbours apart.  x: the lane's logits, in F's range
// (-inf for an expert that is out); `top` the row's largest, or 0 if that is -inf.
template <class F, int PER>
__device__ __forceinline__ bool choose(const RouteArgs& a, const float (&x)[PER], float top, const float (&bias)[PER], int first,
                                       int mine, int& expert, float& logit, F& total) {
  using Key = typename KeyOf<F>::type;
  const int lane = threadIdx.x & 31;
  const bool biased = a.bias != nullptr, grouped = a.top_groups < a.groups;
  const bool by_sum = grouped && a.group_best == 2;
  const bool scores = biased || by_sum || (!a.sigmoid && !a.renormalize);
  Key key[PER];   // order of the experts
  F worth[PER];   // of an expert in its group
  total = F(1);
  if (!a.sigmoid && scores) {
    F s = F(0);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < mine) s += exp_of(F(x[i]) - F(top));
    total = warp_sum(s);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    F v = F(x[i]);
    worth[i] = v;
    if ((biased || by_sum) && x[i] != -INFINITY) {
      worth[i] = (a.sigmoid ? sigmoid(v) : exp_of(v - F(top)) / total) + (biased ? F(bias[i]) : F(0));
      if (biased) v = worth[i];
    }
    key[i] = i < mine ? ordered(v) : Key(0);
  }
  bool apart = true;
  // whether lo is below hi in any precision (or both are -inf)
  auto told = [&](F hi, F lo) {
    return sizeof(F) == 8 || hi - lo > F(kGap) * (F(1) + fabs(hi)) || (hi == lo && hi == -F(INFINITY));
  };
  if (grouped) {
    // the group's best one or two keys, over its lanes
    F best = -F(INFINITY), second = -F(INFINITY);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const F v = i < mine && worth[i] == worth[i] ? worth[i] : -F(INFINITY);
      second = v > best ? best : v > second ? v : second;
      best = v > best ? v : best;
    }
    for (int s = 1; s < (1 << a.lpg_log2); s *= 2) {
      const F b = __shfl_xor_sync(0xffffffffu, best, s), c = __shfl_xor_sync(0xffffffffu, second, s);
      second = b > best ? (best > c ? best : c) : (b > second ? b : second);
      best = b > best ? b : best;
    }
    const F sum = a.group_best == 2 && second > -F(INFINITY) ? best + second : best;
    Key g = lane < a.groups << a.lpg_log2 ? ordered(sum) : Key(0);
    bool in = false;
    F last = F(0);
    for (int j = 0; j < a.top_groups; ++j) {
      const Key m = warp_max(g);
      const int at = __ffs(__ballot_sync(0xffffffffu, g == m)) - 1;
      if (lane >> a.lpg_log2 == at >> a.lpg_log2) {
        in = true;
        g = Key(0);
      }
      last = value_of(m);
    }
    if ((biased || by_sum) && !told(last, value_of(warp_max(g)))) apart = false;
    if (!in)
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = Key(0);
  }
  F before = F(0);
  int e_before = 0;
  float v_before = 0.f;
  const int rounds = sizeof(F) == 4 && biased ? a.k + 1 : a.k;  // with the first one that is left out
  for (int j = 0; j < rounds; ++j) {
    Key m = key[0];
    int at = 0;
    float xv = x[0];
#pragma unroll
    for (int i = 1; i < PER; ++i)
      if (key[i] > m) {
        m = key[i];
        at = i;
        xv = x[i];
      }
    const Key top_key = warp_max(m);
    const int src = __ffs(__ballot_sync(0xffffffffu, m == top_key)) - 1;
    const int e = __shfl_sync(0xffffffffu, first + at, src);
    const float v = __shfl_sync(0xffffffffu, xv, src);
    if (biased && sizeof(F) == 4) {
      if (j > 0 && top_key != 0 && !told(before, value_of(top_key)) && !(v == v_before && a.bias[e] == a.bias[e_before]))
        apart = false;
      before = value_of(top_key);
      e_before = e;
      v_before = v;
    }
    if (lane == j && j < a.k) {
      expert = e;
      logit = v;
    }
    if (lane == src)
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i == at) key[i] = Key(0);
  }
  return apart;
}

// A lane's `mine` logits from `first` on; those of a group's neighbouring lanes lie
// behind them, so that whole 16-byte chunks serve the usual sizes.
template <int PER>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t t, int first, int mine, float (&x)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = -INFINITY;
  if (mine <= 0) return;
  if (a.f32) {
    const float* const row = static_cast<const float*>(a.x) + t * a.ld + first;
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
  } else {
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
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = x[i] == x[i] ? fminf(x[i], FLT_MAX) : -INFINITY;
}

template <int PER>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int group = lane >> a.lpg_log2, sub = lane & ((1 << a.lpg_log2) - 1);
  const int inside = sub * a.per, first = group * a.size + inside;
  const int mine = group < a.groups ? min(a.per, a.size - inside) : 0;
  float x[PER], bias[PER];
  load_row(a, t, first, mine, x);
#pragma unroll
  for (int i = 0; i < PER; ++i) bias[i] = a.bias != nullptr && i < mine ? a.bias[first + i] : 0.f;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, x[i]);
  top = value_of(warp_max(ordered(top)));
  if (top == -INFINITY) top = 0.f;

  int expert = 0;
  float logit = -INFINITY, total;
  if (!choose<float>(a, x, top, bias, first, mine, expert, logit, total)) {
    double exact_total;
    choose<double>(a, x, top, bias, first, mine, expert, logit, exact_total);
  }
  // the weights, from the k logits
  const float best = value_of(warp_max(ordered(lane < a.k ? logit : -INFINITY)));
  float w = 0.f;
  if (lane < a.k && logit != -INFINITY) {
    // (sigmoids below 2^-43 are exponentials, whose ratios do not depend on the largest)
    if (a.renormalize && (!a.sigmoid || best < -30.f)) w = expf(logit - best);
    else w = a.sigmoid ? sigmoid(logit) : expf(logit - top) / total;
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
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  return launch_dependent(route_kernel<PER>, dim3(static_cast<unsigned>((a.T + kRouteWarps - 1) / kRouteWarps)),
                          32 * kRouteWarps, 0, stream, a);
}

}  // namespace
}  // namespace qmm

extern "C" qmm_status qmm_route_experts(const void* logits, int logits_dtype, int64_t ld, const float* bias, int T, int E, int k,
                                        int scoring, int groups, int top_groups, int group_best, int renormalize, float scale,
                                        int32_t* experts, float* weights, void* stream) {
  using namespace qmm;
  if (T < 0 || E < 1 || E > 512 || k < 1 || k > 32 || ld < E || groups < 1 || groups > 32 || E % groups != 0 ||
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
