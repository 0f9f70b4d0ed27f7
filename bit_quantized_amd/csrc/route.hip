// Routing: scores of a router -> the k experts of each token and their weights.
//
// One wavefront per token.  Lane t holds experts VPL t .. VPL t + VPL - 1, so
// the lowest lane that holds a value is the lowest expert that does, which is
// how ties are decided.  Each of the k rounds takes the wavefront's maximum
// and strikes it out.
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

// S: the type that decides, float (logits) or double (scores).
template <int VPL, typename S>
__global__ void __launch_bounds__(kThreads)
route_kernel(RouteArgs a) {
  constexpr bool kWide = sizeof(S) == 8;
  const S kNone = -__builtin_inf();
  __shared__ double s_sel[kWide ? kTokens : 1][kWide ? 64 * VPL : 1];
  __shared__ float s_self[kWide ? 1 : kTokens][kWide ? 1 : 64 * VPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = (int64_t)blockIdx.x * kTokens + wave;
  if (m >= a.M) return;

  // logits: minus infinity and NaN switch an expert off, plus infinity counts
  // as the largest finite value
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    float v = -__builtin_inff();
    if (e < a.E)
      v = a.dtype == 0 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[m * a.E + e] << 16)
                       : static_cast<const float*>(a.logits)[m * a.E + e];
    l[i] = v >= -FLT_MAX ? fminf(v, FLT_MAX) : -__builtin_inff();
  }
  float p[VPL];
  S sel[VPL];
  if (a.softmax) {
    float mx = l[0];
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
    if constexpr (kWide) {
      double w[VPL], t = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        w[i] = exp((double)l[i] - (double)mx);
        t += w[i];
      }
      t = wave_sum(t);
#pragma unroll
      for (int i = 0; i < VPL; ++i) sel[i] = t > 0.0 ? w[i] / t : 0.0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = 1.0f / (1.0f + expf(-l[i]));
      if constexpr (kWide) sel[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane * VPL + i;
    if constexpr (kWide) {
      if (a.bias && e < a.E) sel[i] += (double)a.bias[e];
    } else {
      sel[i] = l[i];
    }
    if (!(l[i] >= -FLT_MAX) || !(sel[i] > kNone)) sel[i] = kNone;  // off (a NaN bias too)
  }

  if (a.n_groups > 1) {
    // lane g takes group g: its best one or two values, their sum ranked
    S* row;
    if constexpr (kWide)
      row = s_sel[wave];
    else
      row = s_self[wave];
#pragma unroll
    for (int i = 0; i < VPL; ++i) row[lane * VPL + i] = sel[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int per = a.E / a.n_groups;
    S value = kNone;
    if (lane < a.n_groups) {
      S t1 = kNone, t2 = kNone;
      for (int i = 0; i < per; ++i) {
        const S v = row[lane * per + i];
        t2 = fmax(t2, fmin(t1, v));
        t1 = fmax(t1, v);
      }
      value = a.group_top > 1 && t2 > kNone ? t1 + t2 : t1;
    }
    int rank = 0;
    for (int g = 0; g < a.n_groups; ++g) {
      S o;
      if constexpr (kWide)
        o = lane_value(value, g);
      else
        o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(value), g));
      rank += o > value || (o == value && g < lane);
    }
    const uint64_t kept = __ballot(lane < a.n_groups && rank < a.topk_groups);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!((kept >> min((lane * VPL + i) / per, 63)) & 1)) sel[i] = kNone;
  }

  int id = -1;
  float wt = 0.0f;
  for (int r = 0; r < a.k; ++r) {
    S top = sel[0];
    int at = 0;
    float pt = p[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) {
      const bool more = sel[i] > top;  // the first of equals stays
      at = more ? i : at;
      pt = more ? p[i] : pt;
      top = more ? sel[i] : top;
    }
    const S best = wave_top(top);
    if (!(best > kNone)) break;
    const int win = __builtin_ctzll(__ballot(top == best));
    const int e = __builtin_amdgcn_readlane(lane * VPL + at, win);
    const float pw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(pt), win));
    if (lane == r) {
      id = e;
      wt = pw;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane * VPL + i == e) sel[i] = kNone;
  }
  if (a.renormalize) {
    const float total = wave_sum(wt);
    wt = total > 0.0f ? wt / total : 0.0f;
  }
  if (lane < a.k) {
    a.ids[m * a.k + lane] = id;
    a.weights[m * a.k + lane] = wt * a.scale;
  }
}

template <typename S>
void launch_s(const RouteArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.M + kTokens - 1) / kTokens)), block(kThreads);
  if (a.E <= 64)
    hipLaunchKernelGGL((route_kernel<1, S>), grid, block, 0, st, a);
  else if (a.E <= 128)
    hipLaunchKernelGGL((route_kernel<2, S>), grid, block, 0, st, a);
  else if (a.E <= 256)
    hipLaunchKernelGGL((route_kernel<4, S>), grid, block, 0, st, a);
  else if (a.E <= 512)
    hipLaunchKernelGGL((route_kernel<8, S>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((route_kernel<16, S>), grid, block, 0, st, a);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
  if (a.bias || (a.n_groups > 1 && a.group_top > 1))
    launch_s<double>(a, st);
  else
    launch_s<float>(a, st);
  return hipGetLastError();
}

}  // namespace w4a8
