// Routing: scores of a router -> the k experts of each token and their weights.
//
// One wavefront per token.  A group of experts lies on 2^gl neighbouring
// lanes (one group: all 64), VPL consecutive experts to a lane, so a group's
// best values come from a butterfly over its lanes, and the lowest lane that
// holds a value is the lowest expert that does, which is how ties are
// decided.  Each of the k rounds takes the wavefront's maximum and strikes it
// out.
//
// Which experts are chosen is decided so that a rounding cannot swap two of
// them: by the logits themselves where the scores enter as they are (both
// score functions increase with the logit), by scores in 64 bits where a bias
// or a sum of scores decides.  The weights are the 32-bit scores.
#include <cfloat>
#include <type_traits>

#include "experts.h"
#include "route.h"

namespace w4a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 64;

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float lane_of(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Keys: integers in the order of the values (a zero's sign aside), which the
// scalar unit compares as well and whose maximum needs no NaN rule.
template <typename S>
using Key = typename std::conditional<sizeof(S) == 4, int32_t, int64_t>::type;
__device__ __forceinline__ int32_t key_of(float v) {
  const int32_t b = __builtin_bit_cast(int32_t, v + 0.0f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ int64_t key_of(double v) {
  const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);
  return b ^ ((b >> 63) & 0x7FFFFFFFFFFFFFFF);
}
__device__ __forceinline__ float value_of(int32_t k) {
  return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7FFFFFFF));
}
template <int CTRL>
__device__ __forceinline__ int32_t key_max_step(int32_t v) {
  const int32_t o = __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
  return v > o ? v : o;
}
template <int CTRL>
__device__ __forceinline__ int64_t key_max_step(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, 0xF, 0xF, true);
  const int64_t o = (int64_t)((uint64_t)hi << 32 | lo);
  return v > o ? v : o;
}
__device__ __forceinline__ int32_t key_lane(int32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ int64_t key_lane(int64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}
// The largest key of the wavefront (the lane maps of wave_max64).
template <typename K>
__device__ __forceinline__ K key_top(K v) {
  v = key_max_step<0xB1>(v);
  v = key_max_step<0x4E>(v);
  v = key_max_step<0x141>(v);
  v = key_max_step<0x140>(v);
  const K a = key_lane(v, 0), b = key_lane(v, 16), c = key_lane(v, 32), d = key_lane(v, 48);
  const K ab = a > b ? a : b, cd = c > d ? c : d;
  return ab > cd ? ab : cd;
}

// The choice by sel (minus infinity: not to be chosen), with the limit to
// groups where there are any; first: the lane's first expert; id: of rank
// `lane`.  A round's winner is found and struck out by lane masks, which the
// scalar unit works on beside the vector unit (16384 tokens, 256 experts in 8
// groups, top 8: 27 us against 30 with the lane's slot and score searched and
// carried along in vector registers; bound by vector issue, 700 per token).
// CHECKED: sel is rounded; false where two values that decide lie within
// `tol` of each other (2 tol for sums of two), so that the rounding could
// have swapped them.
template <int VPL, bool CHECKED, typename S>
__device__ __forceinline__ bool choose(const RouteArgs& a, S (&sel)[VPL], int first, S tol, int& id) {
  const S kNone = -__builtin_inf();
  const int lane = threadIdx.x & 63;
  if (a.n_groups > 1) {
    // a group's best one or two values; the groups' values ranked
    S t1 = sel[0], t2 = kNone;
#pragma unroll
    for (int i = 1; i < VPL; ++i) {
      t2 = fmax(t2, fmin(t1, sel[i]));
      t1 = fmax(t1, sel[i]);
    }
    for (int d = 1; d < 1 << a.gl; d *= 2) {
      const S o1 = __shfl_xor(t1, d), o2 = __shfl_xor(t2, d);
      t2 = fmax(fmin(t1, o1), fmax(t2, o2));
      t1 = fmax(t1, o1);
    }
    const S value = a.group_top > 1 && t2 > kNone ? t1 + t2 : t1;
    const int mine = lane >> a.gl;
    int rank = 0;
    for (int g = 0; g < a.n_groups; ++g) {
      const S o = lane_of(value, g << a.gl);
      rank += o > value || (o == value && g < mine);
    }
    const bool keep = mine < a.n_groups && rank < a.topk_groups;
    if constexpr (CHECKED) {
      static_assert(sizeof(S) == 4, "rounded scores are floats");
      const S most = wave_max64(keep ? kNone : value);  // of the groups left out
      if (__ballot(keep && !(value - most > 2 * tol))) return false;
    }
    if (!keep) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) sel[i] = kNone;
    }
  }

  // the k rounds, on keys in which an order of integers is the order of values
  Key<S> key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = key_of(sel[i]);
  const Key<S> none = key_of(kNone);
  S before = __builtin_inf();
  for (int r = 0; r < a.k + (CHECKED ? 1 : 0); ++r) {
    Key<S> top = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = top > key[i] ? top : key[i];
    const Key<S> best = key_top(top);  // (scalar)
    if (!(best > none)) break;
    if constexpr (CHECKED) {
      const S value = value_of(best);
      if (!(before - value > tol)) return false;
      before = value;
    }
    // the first of equals: of the lanes, then of the lane's values
    uint64_t eq[VPL], any = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      eq[i] = __ballot(key[i] == best);
      any |= eq[i];
    }
    uint64_t left = any & (0 - any);  // the winning lane, until its value is found
    int slot = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint64_t hit = eq[i] & left;
      left &= ~hit;
      slot = hit ? i : slot;
      key[i] = __builtin_amdgcn_inverse_ballot_w64(hit) ? none : key[i];
    }
    const int e = __builtin_amdgcn_readlane(first, __builtin_ctzll(any)) + slot;
    if (lane == r && r < a.k) id = e;
  }
  return true;
}

// WIDE: a bias or a sum of scores decides.  The choice is then made on the
// float scores first.  A float score is within 2^-18 of the largest score of
// the exact one (an exp, a sum of at most 38 steps and a product, or an
// exponential and a reciprocal of one ulp each), and the bias adds 2^-24 of
// the largest sum; where no two deciding values lie closer
// than twice that, the exact scores decide the same.  Else (1 % of tokens of
// 256 experts with a bias of 0.1) the scores are taken in 64 bits.
// The weights are taken for the chosen experts alone.
template <int VPL, bool WIDE>
__global__ void __launch_bounds__(kThreads)
route_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = (int64_t)blockIdx.x * kTokens + wave;
  if (m >= a.M) return;
  // this lane's experts: `count` of them from `first`
  const int per = a.E / a.n_groups, mine = lane >> a.gl, inner = (lane & ((1 << a.gl) - 1)) * VPL;
  const int first = mine * per + inner;
  const int count = mine < a.n_groups ? min(max(per - inner, 0), VPL) : 0;

  // logits: minus infinity and NaN switch an expert off, plus infinity counts
  // as the largest finite value
  auto logit = [&](int e) __attribute__((always_inline)) {
    return a.dtype == 0 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[m * a.E + e] << 16)
                        : static_cast<const float*>(a.logits)[m * a.E + e];
  };
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float v = i < count ? logit(first + i) : -__builtin_inff();
    l[i] = v >= -FLT_MAX ? fminf(v, FLT_MAX) : -__builtin_inff();
  }
  float mx = 0.0f, sum = 1.0f, p[VPL];  // p: softmax numerators
  if (a.softmax) {
    mx = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) mx = fmaxf(mx, l[i]);
    mx = fmaxf(wave_max64(mx), -FLT_MAX);  // (no expert alive: every score is 0)
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = expf(l[i] - mx);
      sum += p[i];
    }
    sum = wave_sum(sum);
  }

  int id = -1;
  if constexpr (!WIDE) {
    float sel[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) sel[i] = l[i];
    choose<VPL, false, float>(a, sel, first, 0.0f, id);
  } else {
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    float b[VPL], sel[VPL], cm = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      b[i] = a.bias && i < count ? a.bias[first + i] : 0.0f;
      const float q = a.softmax ? p[i] * inv
                                : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * l[i]));
      sel[i] = q + b[i];
      if (!(l[i] >= -FLT_MAX) || !(sel[i] > -__builtin_inff()))
        sel[i] = -__builtin_inff();  // off (a NaN bias too)
      else
        cm = fmaxf(cm, fabsf(sel[i]));
    }
    // (inv: the largest score, or 1)
    const float tol = __int_as_float(
        __builtin_amdgcn_readfirstlane(__float_as_int(0x1p-17f * inv + 0x1p-22f * wave_max64(cm))));
    if (!choose<VPL, true, float>(a, sel, first, tol, id)) {
      id = -1;
      double wide[VPL], t = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        wide[i] = a.softmax ? exp((double)l[i] - (double)mx) : 1.0 / (1.0 + exp(-(double)l[i]));
        t += wide[i];
      }
      t = wave_sum(t);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (a.softmax) wide[i] = t > 0.0 ? wide[i] / t : 0.0;
        wide[i] += (double)b[i];
        if (!(l[i] >= -FLT_MAX) || !(wide[i] > -__builtin_inf())) wide[i] = -__builtin_inf();
      }
      choose<VPL, false, double>(a, wide, first, 0.0, id);
    }
  }
  float score = 0.0f;
  if (id >= 0) {
    const float v = fminf(logit(id), FLT_MAX);
    score = a.softmax ? expf(v - mx) / sum : 1.0f / (1.0f + expf(-v));
  }
  if (a.renormalize) {
    const float total = wave_sum(score);
    score = total > 0.0f ? score / total : 0.0f;
  }
  if (lane < a.k) {
    a.ids[m * a.k + lane] = id;
    a.weights[m * a.k + lane] = score * a.scale;
  }
}

template <bool WIDE>
void launch_w(RouteArgs a, hipStream_t st) {
  const dim3 grid((unsigned)((a.M + kTokens - 1) / kTokens)), block(kThreads);
  // the fewest experts per lane with which the groups' lanes, a power of two
  // each, fit the wavefront
  const int per = a.E / a.n_groups;
  a.gl = 6;
  while ((a.n_groups << a.gl) > 64) --a.gl;
  int vpl = 1;
  while ((vpl << a.gl) < per) vpl *= 2;
  switch (vpl) {
    case 1: hipLaunchKernelGGL((route_kernel<1, WIDE>), grid, block, 0, st, a); break;
    case 2: hipLaunchKernelGGL((route_kernel<2, WIDE>), grid, block, 0, st, a); break;
    case 4: hipLaunchKernelGGL((route_kernel<4, WIDE>), grid, block, 0, st, a); break;
    case 8: hipLaunchKernelGGL((route_kernel<8, WIDE>), grid, block, 0, st, a); break;
    case 16: hipLaunchKernelGGL((route_kernel<16, WIDE>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((route_kernel<32, WIDE>), grid, block, 0, st, a); break;
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
  if (a.bias || (a.n_groups > 1 && a.group_top > 1))
    launch_w<true>(a, st);
  else
    launch_w<false>(a, st);
  return hipGetLastError();
}

}  // namespace w4a8
