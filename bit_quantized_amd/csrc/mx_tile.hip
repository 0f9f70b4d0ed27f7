// Products of many rows with a microscaled 4-bit weight: tiles of rows and
// channels, bound by the matrix cores.
//
// Both operands pass through LDS in stages of 128 inputs, all by loads that go
// straight to LDS: of every row 64 bytes (4 bits) or 128 (8), and the weight's
// code blocks, which are operands as they lie.  16-byte chunk i of a row is
// kept at another place, i ^ (row / 4 % 4) or i ^ (row / 2 % 8), so that the
// 16 rows of a quarter of an operand read take 256 bytes of different banks.
// Scales come 512 inputs at a time, one register a lane of those of 32 rows.
//
// A wavefront multiplies half steps of 64 inputs, with the operands of one in
// registers while it reads those of the next.  At the last half step of a
// stage all of the stage is in registers: one barrier there, behind the first
// products, frees its buffer for the stage after those in flight.  Three or
// four buffers keep loads on their way behind the one that the barrier waits
// for.
//
// Measured: 4096 rows 3584 -> 18944 in 4 bits 157 to 165 us (3.4 PFLOP/s), 2048
// rows 18944 -> 3584 in 8 bits 106 to 127 (2.2 to 2.6).  The matrix cores are
// busy for 45 and 60 % of the cycles, LDS reads for 34 and 35 %, and the clock
// falls to 1.8 and 2.0 GHz: the products of random operands alone, without a
// load or an LDS read, reach 6.4 and 3.9 PFLOP/s here.
#include "mx.h"

#include <type_traits>

namespace w4a8 {
namespace {

constexpr int kBand = 8;

struct Spot {
  int group, first, rows, strip;
};

// Work is ordered by group, then strip, then tile: the tiles of one group that
// read the same weights run side by side on one XCD.
template <bool GROUPED>
__device__ __forceinline__ bool locate(const MxArgs& a, Spot& s) {
  const int b = blockIdx.x;
  if constexpr (!GROUPED) {
    // bands of kBand row tiles, strip by strip: the 32 compute units of an XCD
    // work on 8 x 4 tiles, whose rows and channels they share in its L2
    const int tiles = (int)((a.P + a.bm - 1) / a.bm);
    const int at = xcd_run(b, tiles * a.strips);
    const int band = at / (kBand * a.strips), first = band * kBand;
    const int high = min(kBand, tiles - first), local = at - first * a.strips;
    const int t = first + local % high;
    s.strip = local / high;
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

__device__ __forceinline__ int source_row(const MxArgs& a, int p) {  // (of groups)
  if (!a.rows) return p;
  const int r = a.rows[p];
  return r >= 0 && r < a.M ? r : -1;
}

// As load_to_lds (rows.h), to LDS address `at`.
__device__ __forceinline__ void load_at(const LdsSource& src, int at, uint32_t offset, int base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(uniform(at)), "v"(offset), "s"(src.words), "s"(uniform(base))
               : "memory");
}

// All but this wavefront's last N loads and every LDS read of it have arrived;
// then all wavefronts.
template <int N>
__device__ __forceinline__ void stage_barrier() {
  static_assert(N < 64, "six bits of count");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);  // lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// LDS writes of this wavefront's lanes before, reads of its other lanes after.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// What a launch computes: the linear whole or in slices of the inputs, groups,
// groups with the gated activation.
enum Kind { kWhole = 0, kSlices = 1, kGroups = 2, kGated = 3 };

// WM x WN wavefronts of 32 FM rows and 32 FN channels each.
template <int FMT, int WM, int WN, int FM, int FN, int KIND>
struct Shape {
  static constexpr int kWaves = WM * WN;
  static constexpr int kRows = 32 * WM * FM, kBlocks = 2 * WN * FN;  // of the tile
  static constexpr int kRowBytes = FMT == kFp4 ? 64 : 128;           // of a stage
  static constexpr int kRowKiB = kRows * kRowBytes / 1024, kCodeKiB = kBlocks;
  static constexpr int kStageBytes = (kRowKiB + kCodeKiB) * 1024;
  static constexpr int kScaleKiB = (kRows + 16 * kBlocks) / 64;
  // As many buffers as half of a compute unit's LDS holds (of workgroups of
  // eight wavefronts, which run alone, all of it), at most four.  Groups, whose
  // many tiles are short, take a third where that holds three buffers: 4096
  // gated rows of 128 groups, 2048 -> 1536 in 8 bits: 57 us in three buffers,
  // three workgroups to a compute unit, 59 in four and two; but 33 rows 18944
  // -> 3584 15 in four, 16.6 in three.
  static constexpr int kFixed = kScaleKiB * 1024;
  static constexpr bool kThird = KIND >= kGroups && kBlocks <= 8 && 160 * 1024 / 3 - kFixed >= 3 * kStageBytes;
  static constexpr int kRoom = (kThird ? 160 * 1024 / 3 : (kWaves > 4 ? 160 : 80) * 1024) - kFixed;
  static constexpr int kBuffers = kRoom / kStageBytes < 4 ? kRoom / kStageBytes : 4;
  static constexpr int kLds = kBuffers * kStageBytes + kFixed;
  static_assert(kBuffers >= 3, "a stage in use, one to read next, one on its way");
};

template <int FMT, int WM, int WN, int FM, int FN, int KIND>
__global__ void __launch_bounds__(64 * WM * WN, 2)
mx_tile_kernel(const MxArgs a) {
  using S = Shape<FMT, WM, WN, FM, FN, KIND>;
  constexpr bool SPLIT = KIND == kSlices, GATED = KIND == kGated;
  constexpr int kUnits = FMT == kFp4 ? 1 : 2;
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  Spot sp;
  if (!locate<(KIND >= kGroups)>(a, sp)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 31, j = lane >> 5;
  const int Q0 = SPLIT ? (int)((int64_t)a.Q * blockIdx.y / gridDim.y) : 0;
  const int Q1 = SPLIT ? (int)((int64_t)a.Q * (blockIdx.y + 1) / gridDim.y) : a.Q;

  // Block i of the tile: plain: consecutive ones; gated: each wavefront has
  // FN gate blocks, then the value blocks beside them.
  auto block_of = [&](int i) __attribute__((always_inline)) {
    if constexpr (GATED) {
      const int f = i % (2 * FN), half = f / FN;
      const int at = (sp.strip * WN + i / (2 * FN)) * FN + f % FN;
      return half * (a.nb / 2) + min(at, a.nb / 2 - 1);
    } else {
      return min(sp.strip * S::kBlocks + i, a.nb - 1);  // past the end: never stored
    }
  };

  // ---- what this wavefront loads of a stage: neighbouring KiB of rows, of
  // code blocks and of scales
  const int64_t base = a.rows ? 0 : sp.first;
  const int64_t left = a.rows ? a.M : sp.rows;
  const int64_t code_bytes = (int64_t)a.nb * a.gstride * kBlockBytes + 1024;
  LdsSource rx = lds_source(a.qx + base * a.ldx, left * a.ldx);
  LdsSource rw = lds_source(a.codes + (int64_t)sp.group * a.nb * a.gstride * kBlockBytes, code_bytes);
  auto source = [&](int r) __attribute__((always_inline)) {  // of row r of the tile, from base
    const int i = min(r, sp.rows - 1);
    return a.rows ? max(source_row(a, sp.first + i), 0) : i;
  };
  constexpr int kRowLoads = S::kRowKiB / S::kWaves;
  constexpr int kCodeLoads = S::kCodeKiB / S::kWaves;
  static_assert(S::kRowKiB % S::kWaves == 0 && S::kCodeKiB % S::kWaves == 0, "whole loads");
  uint32_t ox[kRowLoads], ow[kCodeLoads];
  constexpr int kChunks = S::kRowBytes / 16;
  auto place = [&](int r) __attribute__((always_inline)) { return FMT == kFp4 ? r >> 2 & 3 : r >> 1 & 7; };
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) {
    const int r = (wave * kRowLoads + i) * (64 / kChunks) + lane / kChunks;
    // rows past the tile's: zeros, which ask for no memory and the matrix cores for little power
    ox[i] = r < sp.rows ? (uint32_t)source(r) * a.ldx + 16 * (lane % kChunks ^ place(r)) : (uint32_t)kOob;
  }
#pragma unroll
  for (int i = 0; i < kCodeLoads; ++i)
    ow[i] = (uint32_t)block_of(wave * kCodeLoads + i) * a.gstride * kBlockBytes + lane * 16;
  // Scales of 512 inputs, rows' before blocks', a KiB at a time (wavefronts
  // past the last KiB load it as well).
  constexpr int kScaleLoads = (S::kScaleKiB + S::kWaves - 1) / S::kWaves;
  LdsSource rs[kScaleLoads];
  uint32_t os[kScaleLoads];
  int scale_at[kScaleLoads], scale_step[kScaleLoads];
  const int lds0 = uniform((int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds);
  constexpr int kScales = S::kBuffers * S::kStageBytes;
#pragma unroll
  for (int i = 0; i < kScaleLoads; ++i) {
    const int kib = min(i * S::kWaves + wave, S::kScaleKiB - 1);
    const bool rows = kib < S::kRows / 64;
    rs[i] = lds_source(rows ? a.qs + base * a.lds : a.scales + (int64_t)sp.group * a.nb * a.qstride * kMxScaleBytes,
                       rows ? left * a.lds : (int64_t)a.nb * a.qstride * kMxScaleBytes);
    os[i] = rows ? (uint32_t)source(kib * 64 + lane) * a.lds
                 : (uint32_t)block_of((kib - S::kRows / 64) * 4 + (lane >> 4)) * a.qstride * kMxScaleBytes +
                       (lane & 15) * 16;
    scale_at[i] = lds0 + kScales + kib * 1024;
    scale_step[i] = rows ? kMxRowScale : kMxScaleBytes;
  }
  // Stages of 128 inputs T0 .. T1 - 1, two to an iteration; the last one may
  // lie past the inputs, where rows have code 0.
  const int I0 = Q0 * 2, I1 = min(Q1 * 2, (a.G + 1) / 2), T0 = I0 * 2, T1 = I1 * 2;
  // Loads of stage t to the buffer at byte `at`; past the last stage without a
  // request (no records, and no scalar offset, which the bounds check may
  // subtract from them).
  constexpr int kLoads = kRowLoads + kCodeLoads;
  auto fill_one = [&](int i, int at, int t) __attribute__((always_inline)) {
    if (i == 0) {
      rx.words[2] = t < T1 ? (int)(uint32_t)(left * a.ldx) : 0;
      rw.words[2] = t < T1 ? (int)(uint32_t)code_bytes : 0;
    }
    const int from = t < T1 ? t : 0;
    if (i < kRowLoads)
      load_at(rx, lds0 + at + (wave * kRowLoads + i) * 1024, ox[i], from * S::kRowBytes);
    else
      load_at(rw, lds0 + at + (S::kRowKiB + wave * kCodeLoads + i - kRowLoads) * 1024, ow[i - kRowLoads],
              from * kBlockBytes);
  };
  // Scales of super q (or of the last), where those of the one before have
  // been read.
  auto fill_scale = [&](int i, int q) __attribute__((always_inline)) {
    load_at(rs[i], scale_at[i], os[i], min(q, (T1 - 1) >> 2) * scale_step[i]);
  };

  // ---- operands: of two half steps of 64 inputs, or (small wavefront tiles,
  // whose few products would not cover the reads) of two whole steps; scales
  // of a super, by half of a step, those of this iteration in the lower bytes
  constexpr bool kDeep = FM * FN <= 4;
  constexpr int kSets = kDeep ? 2 : 1;
  v4i w[kSets][2][FN], x[kSets][2][FM][kUnits];
  uint32_t sw[2][FN], sx[2][FM], sw1[2][FN], sx1[2][FM];
  int x_at[kChunks / 2];  // this lane's row of the first 32, chunks 2 i and 2 i + 1 of it
#pragma unroll
  for (int i = 0; i < kChunks / 2; ++i)
    x_at[i] = (wm * FM * 32 + c) * S::kRowBytes + 16 * ((2 * i + j) ^ place(c));
  const int w_at = S::kRowKiB * 1024 + (wn * FN * 2 + (c >> 4)) * 1024 + j * 256 + (c & 15) * 16;
  const int sx_at = (wm * FM * 32 + c) * 16 + 4 * j;
  const int sw_at = S::kRows * 16 + (wn * FN * 2 + (c >> 4)) * 256 + j * 64 + (c & 15) * 4;
  // read i of half h of the stage in the buffer at byte `at`
  constexpr int kReads = FM * kUnits + FN;
  auto read_one = [&](int i, int set, int h, int at) __attribute__((always_inline)) {
    if (i < FM * kUnits)
      x[set][h][i / kUnits][i % kUnits] = *reinterpret_cast<const v4i*>(
          lds + at + x_at[h * kUnits + i % kUnits] + i / kUnits * 32 * S::kRowBytes);
    else
      w[set][h][i - FM * kUnits] =
          *reinterpret_cast<const v4i*>(lds + at + w_at + (i - FM * kUnits) * 2048 + h * 512);
  };
  constexpr int kScaleReads = FM + FN;
  auto read_scale = [&](int i, int h, uint32_t (&dw)[2][FN], uint32_t (&dx)[2][FM]) __attribute__((always_inline)) {
    if (i < FM)
      dx[h][i] = *reinterpret_cast<const uint32_t*>(lds + kScales + sx_at + i * 512 + h * 8);
    else
      dw[h][i - FM] = *reinterpret_cast<const uint32_t*>(lds + kScales + sw_at + (i - FM) * 512 + h * 128);
  };

  v16f_mx acc[FM][FN];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;
  // product i of half h (step s of its iteration)
  constexpr int kProducts = FM * FN;
  auto multiply = [&](auto sc, int set, int h, int i) __attribute__((always_inline)) {
    const int m = i / FN, n = i % FN;
    v8i_mx xv;
    if constexpr (FMT == kFp4) xv = mx_wide(x[set][h][m][0]);
    else xv = mx_wide(x[set][h][m][0], x[set][h][m][kUnits - 1]);
    acc[m][n] = mx_mfma32<FMT, decltype(sc)::value>(mx_wide(w[set][h][n]), xv, acc[m][n], (int)sw[h][n], (int)sx[h][m]);
  };

  if (T0 < T1) {
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) fill_scale(i, Q0);
#pragma unroll
    for (int b = 0; b < S::kBuffers; ++b)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) fill_one(i, b * S::kStageBytes, T0 + b);
    stage_barrier<(S::kBuffers - 1) * kLoads>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < kScaleReads; ++i) read_scale(i, h, sw, sx);
    }
#pragma unroll
    for (int h = 0; h < (kDeep ? 2 : 1); ++h) {
#pragma unroll
      for (int i = 0; i < kReads; ++i) read_one(i, 0, h, 0);
    }
  }
  int own = 0;  // the buffer of the stage that is multiplied
  for (int it = I0; it < I1; ++it) {
    // Products and, between them, what they leave the issue slots for: the
    // reads of the next (half) step first, then scales, then the stage's
    // loads.  Issued in blocks of their own they add up: 622 cycles a step
    // of a 128 x 128 tile whose products take 256, 510 so.
    auto step = [&](auto sc) __attribute__((always_inline)) {
      constexpr int s = decltype(sc)::value;
      const int next = own == (S::kBuffers - 1) * S::kStageBytes ? 0 : own + S::kStageBytes;
      const int t = 2 * it + s + S::kBuffers;  // the stage that takes this one's buffer
      // Every iteration loads the scales of the next super, behind the first
      // of its barriers: all wavefronts have read this one's.  (In a super's
      // second iteration that brings the same bytes once more: a branch here
      // would let the compiler move the products of the whole iteration behind
      // it.)  Two barriers later, where an iteration's first one leaves only
      // the rows and codes of the stages behind the one that is read next,
      // they are there, and the second step reads them.
      constexpr int kBehind = S::kBuffers - 2;
      constexpr int kLeft = kBehind * kLoads + (s == 1 ? kScaleLoads : 0);
      static_assert(kBehind <= 2, "the scales come before what is left");
      constexpr int kHalves = kDeep ? 1 : 2;  // parts of a step with reads of their own
#pragma unroll
      for (int part = 0; part < kHalves; ++part) {
        const bool last = part == kHalves - 1;
        constexpr int kSlots = 2 * kProducts / kHalves;
        // this part's items, in their order
        constexpr int kOperands = kDeep ? 2 * kReads : kReads;
        const int scales = s == 1 ? 2 * kScaleReads / kHalves : 0;
        const int loads = last ? kLoads + (s == 0 ? kScaleLoads : 0) : 0;
        const int items = kOperands + scales + loads;
#pragma unroll
        for (int slot = 0; slot < kSlots; ++slot) {
          multiply(sc, kDeep ? s : 0, kDeep ? slot / kProducts : part, slot % kProducts);
          if (slot == 0 && last) stage_barrier<kLeft>();
#pragma unroll
          for (int i = slot * items / kSlots; i < (slot + 1) * items / kSlots; ++i) {
            if (i < kOperands) {
              if constexpr (kDeep) read_one(i % kReads, 1 - s, i / kReads, next);
              else read_one(i, 0, 1 - part, last ? next : own);
            } else if (i < kOperands + scales) {
              const int k = i - kOperands;
              read_scale(k % kScaleReads, kDeep ? k / kScaleReads : part, sw1, sx1);
            } else {
              const int k = i - kOperands - scales;
              if (s == 0 && k < kScaleLoads) fill_scale(k, (it >> 1) + 1);
              else fill_one(k - (s == 0 ? kScaleLoads : 0), own, t);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if constexpr (s == 1) {
        // the upper two bytes, or the next super's
        const uint32_t pick = it & 1 ? 0x07060504u : 0x0C0C0302u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int m = 0; m < FM; ++m) sx[h][m] = __builtin_amdgcn_perm(sx1[h][m], sx[h][m], pick);
#pragma unroll
          for (int n = 0; n < FN; ++n) sw[h][n] = __builtin_amdgcn_perm(sw1[h][n], sw[h][n], pick);
        }
      }
      own = next;
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
  }
  // The last loads: the stages' ask for nothing, but the scales' are requests to
  // the end, and the outputs take the LDS that they write to.
  stage_barrier<0>();

  // ---- out: a lane has row c of each 32, and of each 32 channels the four
  // from 8 i + 4 j, i = 0..3.  Each wavefront turns 32 rows of 256 bytes (or
  // what it has) around in LDS, so that stores write whole lines: written from
  // the registers, 8 bytes a row, 4096 x 16384 outputs took 100 us of their
  // own, four times as long.
  constexpr int kOut = GATED ? FN / 2 : FN;        // fragments of 32 channels
  constexpr int kSize = SPLIT ? 4 : 2;             // bytes of an output
  constexpr int kOnce = kOut * 32 * kSize > 256 ? 256 / (32 * kSize) : kOut;
  constexpr int kTurned = kOnce * 32 * kSize, kStride = kTurned + 16;
  static_assert(S::kWaves * 32 * kStride <= S::kLds, "fits the stages' LDS");
  constexpr int kLanes = kTurned / 16;             // lanes of a row
  uint8_t* mine = lds + wave * 32 * kStride;
  const int width = GATED ? a.nb * 8 : a.nb * 16;
  const int lane_row = lane / kLanes, lane_at = lane % kLanes * 16;
#pragma unroll
  for (int m = 0; m < FM; ++m) {
#pragma unroll
    for (int n0 = 0; n0 < kOut; n0 += kOnce) {
#pragma unroll
      for (int n = n0; n < n0 + kOnce; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v4f_mx v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = acc[m][n][4 * i + e];
            if constexpr (GATED) v[e] = silu_mul(v[e], acc[m][n + FN / 2][4 * i + e]);
          }
          uint8_t* to = mine + c * kStride + ((n - n0) * 32 + 8 * i + 4 * j) * kSize;
          if constexpr (SPLIT) *reinterpret_cast<v4f_mx*>(to) = v;
          else *reinterpret_cast<uint2*>(to) = mx_bf16x4(v);
        }
      wave_sync();
      const int ch = ((sp.strip * WN + wn) * kOut + n0) * 32 + lane_at / kSize;
#pragma unroll
      for (int k = 0; k < kLanes / 2; ++k) {
        const int r = k * (64 / kLanes) + lane_row, at = (wm * FM + m) * 32 + r;
        v4u_rows bits = *reinterpret_cast<const v4u_rows*>(mine + r * kStride + lane_at);
        if (at < sp.rows && ch < width) {
          const int p = sp.first + at;
          if (a.rows && source_row(a, p) < 0) bits = v4u_rows{0, 0, 0, 0};
          uint8_t* out = SPLIT ? reinterpret_cast<uint8_t*>(a.parts + (int64_t)blockIdx.y * a.P * width)
                               : reinterpret_cast<uint8_t*>(a.y);
          *reinterpret_cast<v4u_rows*>(out + ((int64_t)p * width + ch) * kSize) = bits;
        }
      }
      wave_sync();
    }
  }
}

// y = bf16 of the slices' sums, in order; four channels a thread, eight
// slices' loads at a time.
__global__ void __launch_bounds__(256)
mx_reduce_kernel(const float* __restrict__ parts, int64_t quads, int ksplit, uint16_t* __restrict__ y) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= quads) return;
  const v4f_mx* p = reinterpret_cast<const v4f_mx*>(parts) + t;
  v4f_mx v = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < ksplit; k0 += 8) {
    v4f_mx part[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) part[k] = p[min(k0 + k, ksplit - 1) * quads];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k0 + k < ksplit) v += part[k];
  }
  reinterpret_cast<uint2*>(y)[t] = mx_bf16x4(v);
}

template <int FMT, int WM, int WN, int FM, int FN, int KIND>
hipError_t launch_one(const MxArgs& a, const MxPlan& p, unsigned blocks, hipStream_t st) {
  using S = Shape<FMT, WM, WN, FM, FN, KIND>;
  static_assert(S::kLds <= 160 * 1024, "LDS of a compute unit");
  constexpr auto kernel = mx_tile_kernel<FMT, WM, WN, FM, FN, KIND>;
  hipLaunchKernelGGL(kernel, dim3(blocks, (unsigned)p.ksplit), dim3(64 * S::kWaves), S::kLds, st, a);
  return hipGetLastError();
}

template <int FMT, int WM, int WN, int FM, int FN>
hipError_t launch_shape(const MxArgs& a, const MxPlan& p, bool gated, unsigned blocks, hipStream_t st) {
  if (gated) return launch_one<FMT, WM, WN, FM, FN, kGated>(a, p, blocks, st);
  if (a.offsets) return launch_one<FMT, WM, WN, FM, FN, kGroups>(a, p, blocks, st);
  if (p.ksplit > 1) return launch_one<FMT, WM, WN, FM, FN, kSlices>(a, p, blocks, st);
  return launch_one<FMT, WM, WN, FM, FN, kWhole>(a, p, blocks, st);
}

template <int FMT>
hipError_t launch_fmt(const MxArgs& a, const MxPlan& p, bool gated, unsigned blocks, hipStream_t st) {
  if (p.bm == 256 && p.bn == 256) return launch_shape<FMT, 4, 2, 2, 4>(a, p, gated, blocks, st);
  // In 4 bits two workgroups of four wavefronts share a compute unit, one's
  // products beside the other's first loads and outputs: 24576 gated rows of 64
  // groups 195 us, 227 of one with eight.  In 8 bits LDS has no room for two.
  if (p.bm == 128 && p.bn == 256) {
    if constexpr (FMT == kFp4) return launch_shape<FMT, 2, 2, 2, 4>(a, p, gated, blocks, st);
    else return launch_shape<FMT, 2, 4, 2, 2>(a, p, gated, blocks, st);
  }
  if (p.bm == 128 && p.bn == 128) return launch_shape<FMT, 2, 2, 2, 2>(a, p, gated, blocks, st);
  if (p.bm == 64 && p.bn == 128) return launch_shape<FMT, 2, 2, 1, 2>(a, p, gated, blocks, st);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_mx_tile(const MxArgs& a, const MxPlan& p, int fmt, bool gated, hipStream_t st) {
  const int64_t tiles = a.offsets ? mx_tile_slots(a.P, a.E, a.bm) : (a.P + a.bm - 1) / a.bm;
  const int64_t blocks = tiles * a.strips;
  if (blocks * 512 >= ((int64_t)1 << 32)) return hipErrorInvalidValue;
  hipError_t e = fmt == kFp4 ? launch_fmt<kFp4>(a, p, gated, (unsigned)blocks, st)
                             : launch_fmt<kFp8>(a, p, gated, (unsigned)blocks, st);
  if (e != hipSuccess || p.ksplit == 1) return e;
  const int64_t quads = a.P * a.nb * 4;
  hipLaunchKernelGGL(mx_reduce_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, a.parts, quads,
                     p.ksplit, a.y);
  return hipGetLastError();
}

}  // namespace w4a8
