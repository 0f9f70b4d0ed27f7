// Products of many rows with a microscaled 4-bit weight: tiles of rows and
// channels, bound by the matrix cores.
//
// Both operands pass through LDS, two buffers of one stage each: 128 bytes of
// every row (256 inputs in 4 bits, 128 in 8) and the weight's code blocks of
// the same inputs, all by loads that go straight to LDS.  Code blocks are
// operands as they lie; of a row, 16-byte chunk i is kept at chunk i ^ (row %
// 8), so that the 16 rows of an operand read spread over the banks.  Scales
// come once per 512 inputs: a register of a lane then serves four products,
// which choose its byte.
//
// A wavefront holds the operands of one step of 128 inputs in registers and
// reads the next step's while it multiplies.  Before the last step of a stage
// every wavefront has all of that stage in registers: one barrier there frees
// its buffer for the stage after the next, whose loads then have a whole stage
// of products to arrive in.
#include "mx.h"

#include <type_traits>

namespace w4a8 {
namespace {

struct Spot {
  int group, first, rows, strip;
};

// Work is ordered by group, then strip, then tile: the tiles of one group that
// read the same weights run side by side on one XCD.
__device__ __forceinline__ bool locate(const MxArgs& a, Spot& s) {
  const int b = blockIdx.x;
  if (!a.offsets) {
    const int tiles = (int)((a.P + a.bm - 1) / a.bm);
    const int at = xcd_run(b, tiles * a.strips);
    const int t = at % tiles;
    s.strip = at / tiles;
    s.group = 0;
    s.first = t * a.bm;
    s.rows = (int)(a.P - s.first < a.bm ? a.P - s.first : a.bm);
    return true;
  }
  const int count = uniform(a.ntiles[0]), total = count * a.strips;
  if (b >= total) return false;
  const int at = xcd_run(b, total), t0 = at / a.strips;
  const int head = uniform(a.tiles[t0].head), n = uniform(a.tiles[t0].n);
  const int local = at - head * a.strips;
  s.strip = local / n;
  const int t = head + local % n;
  if (t >= count) return false;  // (offsets that do not ascend)
  s.group = uniform(a.tiles[t].group);
  s.first = uniform(a.tiles[t].first);
  s.rows = uniform(a.tiles[t].rows);
  return true;
}

__device__ __forceinline__ int source_row(const MxArgs& a, int p) {
  if (!a.rows) return p;
  const int r = a.rows[p];
  return r >= 0 && r < a.M ? r : -1;
}

// Every load and LDS read of this wavefront has arrived; then all wavefronts.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt 0, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// WM x WN wavefronts of 16 FM rows and 16 FN channels each.
template <int FMT, int WM, int WN, int FM, int FN>
struct Shape {
  static constexpr int kWaves = WM * WN;
  static constexpr int kRows = 16 * WM * FM, kBlocks = WN * FN;  // of the tile
  static constexpr int kSteps = FMT == kFp4 ? 2 : 1;             // steps of a stage
  static constexpr int kStages = 4 / kSteps;                     // stages of a super
  static constexpr int kRowKiB = kRows / 8, kCodeKiB = kBlocks * kSteps;
  static constexpr int kStageBytes = (kRowKiB + kCodeKiB) * 1024;
  static constexpr int kScaleKiB = (kRows + 16 * kBlocks) / 64;
  static constexpr int kLds = 2 * (kStageBytes + kScaleKiB * 1024);
};

template <int FMT, int WM, int WN, int FM, int FN, bool GATED, bool SPLIT>
__global__ void __launch_bounds__(64 * WM * WN)
mx_tile_kernel(const MxArgs a) {
  using S = Shape<FMT, WM, WN, FM, FN>;
  constexpr int kUnits = FMT == kFp4 ? 1 : 2;
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  Spot sp;
  if (!locate(a, sp)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 15, j = lane >> 4;
  const int Q0 = SPLIT ? (int)((int64_t)a.Q * blockIdx.y / gridDim.y) : 0;
  const int Q1 = SPLIT ? (int)((int64_t)a.Q * (blockIdx.y + 1) / gridDim.y) : a.Q;

  // Block i of the tile: plain: consecutive ones; gated: each wavefront has
  // FN / 2 gate blocks, then the value blocks beside them.
  auto block_of = [&](int i) __attribute__((always_inline)) {
    if constexpr (GATED) {
      const int f = i % FN, half = f / (FN / 2);
      const int at = (sp.strip * WN + i / FN) * (FN / 2) + f % (FN / 2);
      return half * (a.nb / 2) + min(at, a.nb / 2 - 1);
    } else {
      return min(sp.strip * S::kBlocks + i, a.nb - 1);  // past the end: never stored
    }
  };

  // ---- what this wavefront loads of a stage: neighbouring KiB of rows, of
  // code blocks and of scales
  const int64_t base = a.rows ? 0 : sp.first;
  const int64_t left = a.rows ? a.M : sp.rows;
  const int64_t code_bytes = (int64_t)a.nb * a.G * kBlockBytes + 1024;
  LdsSource rx = lds_source(a.qx + base * a.ldx, left * a.ldx);
  LdsSource rw = lds_source(a.codes + (int64_t)sp.group * a.nb * a.G * kBlockBytes, code_bytes);
  const LdsSource rs = lds_source(a.qs + base * a.lds, left * a.lds);
  const LdsSource rv = lds_source(a.scales + (int64_t)sp.group * a.nb * a.Q * kMxScaleBytes,
                                  (int64_t)a.nb * a.Q * kMxScaleBytes);
  auto source = [&](int r) __attribute__((always_inline)) {  // of row r of the tile, from base
    const int i = min(r, sp.rows - 1);
    return a.rows ? max(source_row(a, sp.first + i), 0) : i;
  };
  constexpr int kRowLoads = S::kRowKiB / S::kWaves;
  constexpr int kCodeLoads = S::kCodeKiB / S::kWaves;
  constexpr int kScaleLoads = (S::kScaleKiB + S::kWaves - 1) / S::kWaves;
  static_assert(S::kRowKiB % S::kWaves == 0 && S::kCodeKiB % S::kWaves == 0, "whole loads");
  uint32_t ox[kRowLoads], ow[kCodeLoads], os[kScaleLoads];
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    const int r = (wave * kRowLoads + i) * 8 + (lane >> 3);
    ox[i] = (uint32_t)source(r) * a.ldx + 16 * ((lane & 7) ^ (r & 7));
  }
#pragma unroll
  for (int i = 0; i < kCodeLoads; ++i) {
    const int k = wave * kCodeLoads + i;
    ow[i] = ((uint32_t)block_of(k / S::kSteps) * a.G + k % S::kSteps) * kBlockBytes + lane * 16;
  }
#pragma unroll
  for (int i = 0; i < kScaleLoads; ++i) {
    const int k = i * S::kWaves + wave;
    os[i] = k < S::kRows / 64
                ? (uint32_t)source(k * 64 + lane) * a.lds
                : (uint32_t)block_of(min((k - S::kRows / 64) * 4 + (lane >> 4), S::kBlocks - 1)) * a.Q * kMxScaleBytes +
                      (lane & 15) * 16;
  }
  // Load i of the kLoads that fill a stage.
  constexpr int kLoads = kRowLoads + kCodeLoads;
  auto fill_one = [&](int i, uint8_t* at, int t) __attribute__((always_inline)) {
    if (i < kRowLoads)
      load_to_lds(rx, at + (wave * kRowLoads + i) * 1024, (int)ox[i], t * 128);
    else
      load_to_lds(rw, at + (S::kRowKiB + wave * kCodeLoads + i - kRowLoads) * 1024, (int)ow[i - kRowLoads],
                  t * S::kSteps * kBlockBytes);
  };
  auto scales_at = [&](int buf) __attribute__((always_inline)) {
    return lds + 2 * S::kStageBytes + buf * S::kScaleKiB * 1024;
  };
  auto fill_scales = [&](int buf, int q) __attribute__((always_inline)) {
    uint8_t* at = scales_at(buf);
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) {
      const int k = i * S::kWaves + wave;
      if (k < S::kRows / 64)
        load_to_lds(rs, at + k * 1024, (int)os[i], q * kMxRowScale);
      else if (k < S::kScaleKiB)
        load_to_lds(rv, at + k * 1024, (int)os[i], q * kMxScaleBytes);
    }
  };

  // ---- operands: rows in place, as soon as their products are issued; the
  // weight's in two sets
  v4i w[2][FN], x[FM][kUnits];
  int sw[FN], sw1[FN], sx[FM];
  auto read_row = [&](int m, const uint8_t* at, int step) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int chunk = (FMT == kFp4 ? 4 * (step % S::kSteps) : 4 * u) + j;
      x[m][u] = *reinterpret_cast<const v4i*>(at + ((wm * FM + m) * 16 + c) * 128 + 16 * (chunk ^ (c & 7)));
    }
  };
  auto read_block = [&](int n, int set, const uint8_t* at, int step) __attribute__((always_inline)) {
    w[set][n] = *reinterpret_cast<const v4i*>(at + S::kRowKiB * 1024 +
                                              ((wn * FN + n) * S::kSteps + step % S::kSteps) * 1024 + lane * 16);
  };
  // (half: the steps of 256 inputs, in the upper or lower half of a register)
  auto row_scale = [&](int m, const uint8_t* at, int half) __attribute__((always_inline)) {
    return (int)(*reinterpret_cast<const uint32_t*>(at + ((wm * FM + m) * 16 + c) * 16 + 4 * j) >> (16 * half));
  };
  auto block_scale = [&](int n, const uint8_t* at, int half) __attribute__((always_inline)) {
    return (int)(*reinterpret_cast<const uint32_t*>(at + S::kRows * 16 + (wn * FN + n) * 256 + lane * 4) >>
                 (16 * half));
  };

  v4f_mx acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n) acc[m][n] = v4f_mx{0.f, 0.f, 0.f, 0.f};

  // Iterations of 256 inputs (two steps); the last may end in a step past the
  // inputs, whose rows have code 0.
  const int I0 = Q0 * 2, I1 = min(Q1 * 2, (a.G + 1) / 2);
  constexpr int kPer = 2 / S::kSteps;  // stages of an iteration
  const int T1 = I1 * kPer;
  if (I0 < I1) {
    fill_scales(0, Q0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) fill_one(i, lds, I0 * kPer);
    if (I0 * kPer + 1 < T1) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) fill_one(i, lds + S::kStageBytes, I0 * kPer + 1);
    }
    stage_barrier();
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      read_row(m, lds, 0);
      sx[m] = row_scale(m, scales_at(0), 0);
    }
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      read_block(n, 0, lds, 0);
      sw[n] = block_scale(n, scales_at(0), 0);
    }
  }
  for (int it = I0; it < I1; ++it) {
    // the next iteration's scales: their super's buffer and half
    const uint8_t* next_scales = scales_at((((it + 1) >> 1) - Q0) & 1);
    const int next_half = (it + 1) & 1;
    auto step = [&](auto sc) __attribute__((always_inline)) {
      constexpr int s = decltype(sc)::value;
      constexpr bool last = s % S::kSteps == S::kSteps - 1;
      // groups of products before the barrier, which by then waits for no read
      constexpr int kBefore = last ? (FM >= 8 ? 2 : 1) : 0;
      const int t = it * kPer + (kPer == 2 ? s : 0);
      uint8_t* own = lds + (kPer == 2 ? s : (it - I0) & 1) * S::kStageBytes;
      uint8_t* other = lds + (kPer == 2 ? 1 - s : 1 - ((it - I0) & 1)) * S::kStageBytes;
      uint8_t* from = last ? other : own;
      const bool more = t + 2 < T1;
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        if (last && m == kBefore) {
          stage_barrier();
          rx.words[2] = more ? (int)(uint32_t)(left * a.ldx) : 0;  // (else without requests)
          rw.words[2] = more ? (int)(uint32_t)code_bytes : 0;
          if (more && (t + 2) % S::kStages == 0) fill_scales((((t + 2) / S::kStages) - Q0) & 1, (t + 2) / S::kStages);
        }
        v8i_mx xv;
        if constexpr (FMT == kFp4) xv = mx_wide(x[m][0]);
        else xv = mx_wide(x[m][0], x[m][kUnits - 1]);
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[m][n] = mx_mfma<FMT, s>(mx_wide(w[s][n]), xv, acc[m][n], sw[n], sx[m]);
        if (m >= kBefore) {
          // a share of the next step's reads, of the stage's loads
          constexpr int kGroups = FM - kBefore;
          const int g = m - kBefore;
#pragma unroll
          for (int i = 0; i < FN; ++i)
            if (i >= g * FN / kGroups && i < (g + 1) * FN / kGroups) {
              read_block(i, s ^ 1, from, s + 1);
              if (s == 1) sw1[i] = block_scale(i, next_scales, next_half);
            }
#pragma unroll
          for (int i = 0; i < FM; ++i)
            if (i >= g * FM / kGroups && i < (g + 1) * FM / kGroups) {
              read_row(i, from, s + 1);
              if (s == 1) sx[i] = row_scale(i, next_scales, next_half);
            }
          if (last) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
              if (i >= g * kLoads / kGroups && i < (g + 1) * kLoads / kGroups) fill_one(i, own, t + 2);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
#pragma unroll
    for (int n = 0; n < FN; ++n) sw[n] = sw1[n];
  }
  stage_barrier();  // (the last loads, none of them a request)

  // ---- out: a lane has four channels of row c of each 16
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int at = (wm * FM + m) * 16 + c;
    if (at >= sp.rows) continue;
    const int p = sp.first + at;
    const bool gone = a.rows && source_row(a, p) < 0;
    if constexpr (SPLIT) {
      float* out = a.parts + ((int64_t)blockIdx.y * a.P + p) * a.nb * 16;
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const int b = sp.strip * S::kBlocks + wn * FN + n;
        if (b < a.nb) *reinterpret_cast<v4f_mx*>(out + b * 16 + 4 * j) = acc[m][n];
      }
    } else if constexpr (GATED) {
      uint16_t* out = a.y + (int64_t)p * a.nb * 8;
#pragma unroll
      for (int n = 0; n < FN / 2; ++n) {
        const int b = (sp.strip * WN + wn) * (FN / 2) + n;
        v4f_mx v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = silu_mul(acc[m][n][i], acc[m][n + FN / 2][i]);
        uint2 bits = mx_bf16x4(v);
        if (gone) bits = uint2{0u, 0u};
        if (b < a.nb / 2) *reinterpret_cast<uint2*>(out + b * 16 + 4 * j) = bits;
      }
    } else {
      uint16_t* out = a.y + (int64_t)p * a.nb * 16;
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const int b = sp.strip * S::kBlocks + wn * FN + n;
        uint2 bits = mx_bf16x4(acc[m][n]);
        if (gone) bits = uint2{0u, 0u};
        if (b < a.nb) *reinterpret_cast<uint2*>(out + b * 16 + 4 * j) = bits;
      }
    }
  }
}

// y = bf16 of the slices' sums, in order; four channels a thread.
__global__ void __launch_bounds__(256)
mx_reduce_kernel(const float* __restrict__ parts, int64_t quads, int ksplit, uint16_t* __restrict__ y) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= quads) return;
  v4f_mx v = reinterpret_cast<const v4f_mx*>(parts)[t];
  for (int k = 1; k < ksplit; ++k) v += reinterpret_cast<const v4f_mx*>(parts)[t + k * quads];
  reinterpret_cast<uint2*>(y)[t] = mx_bf16x4(v);
}

template <int FMT, int WM, int WN, int FM, int FN, bool GATED, bool SPLIT>
hipError_t launch_one(const MxArgs& a, const MxPlan& p, unsigned blocks, hipStream_t st) {
  using S = Shape<FMT, WM, WN, FM, FN>;
  static_assert(S::kLds <= 160 * 1024, "LDS of a compute unit");
  constexpr auto kernel = mx_tile_kernel<FMT, WM, WN, FM, FN, GATED, SPLIT>;
  hipLaunchKernelGGL(kernel, dim3(blocks, (unsigned)p.ksplit), dim3(64 * S::kWaves), S::kLds, st, a);
  return hipGetLastError();
}

template <int FMT, int WM, int WN, int FM, int FN>
hipError_t launch_shape(const MxArgs& a, const MxPlan& p, bool gated, unsigned blocks, hipStream_t st) {
  if (gated) return launch_one<FMT, WM, WN, FM, FN, true, false>(a, p, blocks, st);
  if (p.ksplit > 1) return launch_one<FMT, WM, WN, FM, FN, false, true>(a, p, blocks, st);
  return launch_one<FMT, WM, WN, FM, FN, false, false>(a, p, blocks, st);
}

template <int FMT>
hipError_t launch_fmt(const MxArgs& a, const MxPlan& p, bool gated, unsigned blocks, hipStream_t st) {
  if (p.bm == 256) return launch_shape<FMT, 2, 2, 8, 8>(a, p, gated, blocks, st);
  if (p.bm == 128) return launch_shape<FMT, 2, 2, 4, 4>(a, p, gated, blocks, st);
  return launch_shape<FMT, 1, 4, 4, 2>(a, p, gated, blocks, st);
}

}  // namespace

hipError_t launch_mx_tile(const MxArgs& a, const MxPlan& p, int fmt, bool gated, hipStream_t st) {
  const int64_t tiles = a.offsets ? mx_tile_slots(a.P, a.E, a.bm) : (a.P + a.bm - 1) / a.bm;
  const int64_t blocks = tiles * a.strips;
  if (blocks * 256 >= ((int64_t)1 << 32)) return hipErrorInvalidValue;
  hipError_t e = fmt == kFp4 ? launch_fmt<kFp4>(a, p, gated, (unsigned)blocks, st)
                             : launch_fmt<kFp8>(a, p, gated, (unsigned)blocks, st);
  if (e != hipSuccess || p.ksplit == 1) return e;
  const int64_t quads = a.P * a.nb * 4;
  hipLaunchKernelGGL(mx_reduce_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, a.parts, quads,
                     p.ksplit, a.y);
  return hipGetLastError();
}

}  // namespace w4a8
