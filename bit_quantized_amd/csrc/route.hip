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

#include "experts.h"
#include "route.h"

namespace w4a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kThreads / 64;

template <int CTRL>
__device__ __forceinline__ double dpp_max_step(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xF, 0xF, true);
  return fmax(v, __builtin_bit_cast(double, (uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Maximum over the wavefront, as wave_max64 for floats.
__device__ __forceinline__ double wave_top(double v) {
  v = dpp_max_step<0xB1>(v);
  v = dpp_max_step<0x4E>(v);
  v = dpp_max_step<0x141>(v);
  v = dpp_max_step<0x140>(v);
  return fmax(fmax(lane_value(v, 0), lane_value(v, 16)), fmax(lane_value(v, 32), lane_value(v, 48)));
}
__device__ __forceinline__ float wave_top(float v) { return wave_max64(v); }

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// What a token's choice left in a lane: expert and score of rank `lane`.
struct Choice {
  int id;
  float score;
};

__device__ __forceinline__ double lane_of(double v, int lane) { return lane_value(v, lane); }
__device__ __forceinline__ float lane_of(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// The choice by sel (minus infinity: not to be chosen), with the limit to
// groups where there are any; first: the lane's first expert.
// CHECKED: sel is rounded; false where two values that decide lie within
// `tol` of each other (2 tol for sums of two), so that the rounding could
// have swapped them.
template <int VPL, bool CHECKED, typename S>
__device__ __forceinline__ bool choose(const RouteArgs& a, S (&sel)[VPL], const float (&p)[VPL], int first,
                                       S tol, Choice& out) {
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
      const S most = wave_top(keep ? kNone : value);  // of the groups left out
      if (__ballot(keep && !(value - most > 2 * tol))) return false;
    }
    if (!keep) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) sel[i] = kNone;
    }
  }

  S before = __builtin_inf();
  for (int r = 0; r < a.k + (CHECKED ? 1 : 0); ++r) {
    S top = sel[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = fmax(top, sel[i]);
    const S best = wave_top(top);
    if (!(best > kNone)) break;
    if constexpr (CHECKED) {
      if (!(before - best > tol)) return false;
      before = best;
    }
    // the first of equals: of the lane's values, then of the lanes
    int at = VPL;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i) at = sel[i] == best ? i : at;
    const int win = __builtin_ctzll(__ballot(at < VPL));
    const int e = __builtin_amdgcn_readlane(first + at, win);
    float pw = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool hit = first + i == e;
      pw = hit ? p[i] : pw;
      sel[i] = hit ? kNone : sel[i];
    }
    pw = lane_of(pw, win);
    if (lane == r && r < a.k) out = Choice{e, pw};
  }
  return true;
}

// WIDE: a bias or a sum of scores decides.  The choice is then made on the
// float scores first.  A float score is within 2^-18 of the largest score of
// the exact one (an exp, a sum of at most 22 steps and a quotient), and the
// bias adds 2^-24 of the largest sum; where no two deciding values lie closer
// than twice that, the exact scores decide the same.  Else (1 % of tokens of
// 256 experts with a bias of 0.1) the scores are taken in 64 bits.
// 16384 tokens, 256 experts in 8 groups, top 8: 30 us, against 38 with 64-bit
// scores throughout; bound by instruction issue, about 950 per token.
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
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    float v = -__builtin_inff();
    if (i < count)
      v = a.dtype == 0
              ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[m * a.E + first + i] << 16)
              : static_cast<const float*>(a.logits)[m * a.E + first + i];
    l[i] = v >= -FLT_MAX ? fminf(v, FLT_MAX) : -__builtin_inff();
  }
  float p[VPL], mx = 0.0f, pm = 1.0f;  // pm: at least the largest score
  if (a.softmax) {
    mx = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) mx = fmaxf(mx, l[i]);
    mx = fmaxf(wave_max64(mx), -FLT_MAX);  // (no expert alive: every score is 0)
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = expf(l[i] - mx);
      sum += p[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] = sum > 0.0f ? p[i] / sum : 0.0f;
    pm = sum > 0.0f ? 1.0f / sum : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] = 1.0f / (1.0f + expf(-l[i]));
  }

  Choice c{-1, 0.0f};
  if constexpr (!WIDE) {
    float sel[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) sel[i] = l[i];
    choose<VPL, false, float>(a, sel, p, first, 0.0f, c);
  } else {
    float b[VPL], sel[VPL], cm = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      b[i] = a.bias && i < count ? a.bias[first + i] : 0.0f;
      sel[i] = p[i] + b[i];
      if (!(l[i] >= -FLT_MAX) || !(sel[i] > -__builtin_inff()))
        sel[i] = -__builtin_inff();  // off (a NaN bias too)
      else
        cm = fmaxf(cm, fabsf(sel[i]));
    }
    const float tol = 0x1p-17f * pm + 0x1p-22f * wave_max64(cm);
    if (!choose<VPL, true, float>(a, sel, p, first, tol, c)) {
      c = Choice{-1, 0.0f};
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
      choose<VPL, false, double>(a, wide, p, first, 0.0, c);
    }
  }
  if (a.renormalize) {
    const float total = wave_sum(c.score);
    c.score = total > 0.0f ? c.score / total : 0.0f;
  }
  if (lane < a.k) {
    a.ids[m * a.k + lane] = c.id;
    a.weights[m * a.k + lane] = c.score * a.scale;
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
