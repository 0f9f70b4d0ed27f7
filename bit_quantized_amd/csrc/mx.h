// Microscaled floating point: formats, the layout of quantised rows, and the
// interface between the kernels (mx_quant.hip, mx_stream.hip, mx_tile.hip) and
// the entry points (mx_abi.hip).
//
// The matrix core product is v_mfma_scale_f32_16x16x128 (a few rows) or
// 32x32x64 (tiles; in 4 bits it reaches 9.5 PFLOP/s where the other, bound by
// issue, reaches 6.9, and both 5.0 with 8-bit rows): c channels x c rows x 2048
// / c inputs.  Lane L = c j + i holds
//   4-bit operand: 32 values, inputs 32 j .. 32 j + 31 of row (channel) i;
//   8-bit operand: inputs 16 j .. 16 j + 15, then those 1024 / c later;
//   scale: a byte, chosen among the four of a register, for inputs 32 j ..
//   32 j + 31 of its row in both formats;
//   result: row (of the second operand) i, of each 4 * 64 / c channels the
//   four from 4 j.
// Weights are the first operand, so that four sums of a lane are neighbours in
// the output.
#pragma once

#include "rows.h"

namespace w4a8 {

enum MxFormat { kFp4 = 0, kFp8 = 1 };
enum MxRule { kFloor = 0, kCeil = 1 };
constexpr int kMxBlock = 32;             // values that share a scale
constexpr int kMxStep = 128;             // inputs of a matrix core product
constexpr int kMxSuper = 512;            // inputs whose scales share a register
constexpr int kMxScaleBytes = 256;       // of 16 channels x 512 inputs
constexpr int kMxRowScale = 16;          // bytes of a row's scales, 512 inputs
constexpr int kMxMaxGroups = 1024;
constexpr int64_t kMxMaxK = (int64_t)1 << 22;

inline int64_t mx_steps(int64_t K) { return (K + kMxStep - 1) / kMxStep; }
inline int64_t mx_supers(int64_t K) { return (K + kMxSuper - 1) / kMxSuper; }
// Strides are odd numbers of what is loaded at once (1 KiB of codes, 128 bytes
// of a row's), so that loads at the same inputs of neighbouring channels and
// rows spread over the memory channels instead of meeting in a few.
inline int64_t mx_code_stride(int64_t K) { return mx_steps(K) | 1; }
inline int64_t mx_scale_stride(int64_t K) { return mx_supers(K) | 1; }
inline int64_t mx_scales_offset(int64_t N, int64_t K) { return N / 16 * mx_code_stride(K) * kBlockBytes; }
inline int64_t mx_weight_bytes(int64_t N, int64_t K) {
  return mx_scales_offset(N, K) + N / 16 * mx_scale_stride(K) * kMxScaleBytes + 1024;
}
// Quantised rows in a workspace, in one of two layouts; in both, inputs past K
// up to whole 512 have code 0 and scale 0.
// Rows (tiles, whose loads to LDS take whole pieces of a row): codes
// [rows][mx_row_bytes], inputs in whole 256, so that no iteration of two steps
// leaves its row; scales [rows][mx_row_scale_bytes], byte 4 j + s of 16 for
// inputs 128 s + 32 j of 512.
// Interleaved (the stream, whose lanes load operands): like the weight's
// blocks.  Codes of rows 16 b + c, inputs 128 g and on, at (b G + g) blocks of 1
// KiB (4 bits) or 2, 16-byte unit 16 j + c (and 64 + 16 j + c); scales at (b Q +
// q) 256 + 4 (16 j + c).  The 16 rows of a load are at most two runs of
// consecutive bytes per j wherever they start.  Read from the other layout,
// every lane would meet a line of its own: 16 rows 18944 -> 3584 took 17.4 us.
inline int64_t mx_row_bytes(int64_t K, int fmt) {
  return ((K + 255) / 256 * (fmt == kFp4 ? 1 : 2) | 1) * 128;
}
inline int64_t mx_row_scale_bytes(int64_t K) { return mx_scale_stride(K) * kMxRowScale; }
inline int64_t mx_block_bytes(int64_t K, int fmt) {  // of 16 interleaved rows
  return mx_steps(K) * kBlockBytes * (fmt == kFp4 ? 1 : 2);
}
inline int64_t mx_block_scale_bytes(int64_t K) { return mx_supers(K) * kMxScaleBytes; }

typedef int v8i_mx __attribute__((ext_vector_type(8)));
typedef float v4f_mx __attribute__((ext_vector_type(4)));
typedef float v16f_mx __attribute__((ext_vector_type(16)));
typedef short v2s_mx __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf_mx __attribute__((ext_vector_type(2)));
typedef float v2f_mx __attribute__((ext_vector_type(2)));

// ------------------------------------------------------- quantising a block

// Eight consecutive values as loaded.
template <bool F32>
struct MxRaw {
  static constexpr int kLoads = F32 ? 2 : 1;
  v4u_rows d[kLoads];
  __device__ __forceinline__ void load(const uint8_t* row, int64_t k) {
    const v4u_rows* p = reinterpret_cast<const v4u_rows*>(row + k * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kLoads; ++i) d[i] = p[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) d[i] = v4u_rows{0, 0, 0, 0};
  }
  // The largest magnitude's bits as those of a float.  Magnitudes order as
  // integers, infinities and NaN above all numbers.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, d[i >> 2][i & 3] & 0x7FFFFFFFu);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m = max(m, d[0][i] & 0x7FFF0000u);
        m = max(m, (d[0][i] << 16) & 0x7FFF0000u);
      }
    }
    return m;
  }
  __device__ __forceinline__ v2bf_mx pair(int i) const {  // bfloat16 values 2 i and 2 i + 1
    const uint32_t bits = d[0][i];  // (a copy: the cast of a vector's element takes the first)
    return __builtin_bit_cast(v2bf_mx, bits);
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (F32) return __uint_as_float(d[i >> 2][i & 3]);
    return __uint_as_float(i & 1 ? d[0][i >> 1] & 0xFFFF0000u : d[0][i >> 1] << 16);
  }
};

__device__ __forceinline__ uint32_t dpp_umax_quad(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));  // lane ^ 1
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));  // lane ^ 2
}

// Scale byte of a block whose largest magnitude has these bits.  (An exponent
// field of 0, zero or subnormal, gives byte 0 under both rules.)
template <int FMT>
__device__ __forceinline__ int mx_scale_byte(uint32_t top, int rule) {
  const int e = (int)(top >> 23);
  const uint32_t limit = FMT == kFp4 ? 0x400000u : 0x600000u;  // mantissa of 6 and of 448
  const int over = rule == kCeil && (top & 0x7FFFFFu) > limit ? 1 : 0;
  return e == 255 ? 255 : max(e - (FMT == kFp4 ? 2 : 8) + over, 0);
}

// 2^(b - 127) for the conversions, which look at the exponent field only
// (field 0 is 2^-127, and so is the value).
__device__ __forceinline__ float mx_scale_float(int b) {
  return __uint_as_float(max((uint32_t)b << 23, 0x400000u));
}

// Codes of eight values under scale byte b: 4 bytes (FP4, in .x) or 8.  The
// conversions divide by the scale and round to nearest even; the 4-bit one
// clips at 6 by itself, the 8-bit one would make NaN of values from 464 times
// the scale, so they are clipped first.
template <int FMT, bool F32>
__device__ __forceinline__ uint2 mx_codes8(const MxRaw<F32>& r, int b) {
  const float s = mx_scale_float(b);
  uint2 out = {0u, 0u};
  if constexpr (FMT == kFp4) {
    uint32_t c = 0;
    if constexpr (F32) {
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, r.value(0), r.value(1), s, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, r.value(2), r.value(3), s, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, r.value(4), r.value(5), s, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, r.value(6), r.value(7), s, 3);
    } else {
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, r.pair(0), s, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, r.pair(1), s, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, r.pair(2), s, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, r.pair(3), s, 3);
    }
    out.x = c;
  } else {
    const float lim = 448.0f * s;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_fmed3f(r.value(i), -lim, lim);
    v2s_mx lo = {0, 0}, hi = {0, 0};
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[0], v[1], s, false);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[2], v[3], s, true);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[4], v[5], s, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[6], v[7], s, true);
    out.x = __builtin_bit_cast(uint32_t, lo);
    out.y = __builtin_bit_cast(uint32_t, hi);
  }
  if (b == 255) out = uint2{0u, 0u};
  return out;
}

// ------------------------------------------------------------ the products

// A run of at most tile_rows product rows [first, first + rows) of one group;
// it is one of the group's n tiles, which begin with tile `head`.
struct MxTile {
  int group, first, rows, head, n, pad[3];
};

struct MxArgs {
  const uint8_t* qx;      // quantised rows and their scales
  const uint8_t* qs;
  const void* x;          // raw rows (kernels that quantise them)
  int f32, rule;
  const uint8_t* codes;   // planes of the packed weight
  const uint8_t* scales;
  const int* offsets;     // [E + 1]; null: one group of all rows
  const int* rows;        // source row of a product row; null: itself
  const int* ntiles;      // tiles of the grouping step; null: found in the kernel
  const MxTile* tiles;
  int64_t M;              // source rows
  int64_t P;              // product rows
  int E, K, G, Q;         // groups, inputs, steps of 128, of 512
  int gstride, qstride;            // strides of the planes, in blocks
  int ldx, lds;           // bytes of a quantised row and of its scales
  int nb;                 // 16-channel blocks of a group
  int strips;             // column strips of a tile
  int bm;                 // rows of a tile
  uint16_t* y;            // [P][16 nb], gated: [P][8 nb]
  float* parts;           // [ksplit][P][16 nb]
};

// Where the tiles of a call are listed in its workspace.
inline int64_t mx_tile_slots(int64_t P, int E, int bm) { return (P + bm - 1) / bm + (E < P ? E : P); }

// First and one past the last product row of group e: what the caller wrote,
// bounded to [0, P] and to no fewer than zero rows.
__device__ __forceinline__ void mx_run(const int* offsets, int e, int64_t P, int& lo, int& hi) {
  lo = min(max(offsets[e], 0), (int)P);
  hi = max(min(max(offsets[e + 1], 0), (int)P), lo);
}

// Sum of v over this lane and those below it, by DPP moves: prefix sums of
// each row of 16, then the rows' totals.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add_step(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_prefix_sum(int v) {
  v = dpp_add_step<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
  v = dpp_add_step<0x112, 0xF>(v);
  v = dpp_add_step<0x114, 0xF>(v);
  v = dpp_add_step<0x118, 0xF>(v);
  v = dpp_add_step<0x142, 0xA>(v);  // row_bcast 15: lane 15 of a row to the next row (1 and 3)
  return dpp_add_step<0x143, 0xC>(v);  // row_bcast 31: lane 31 to rows 2 and 3
}

// Operand of a matrix core product from loaded registers.
__device__ __forceinline__ v8i_mx mx_wide(v4i a) {
  return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
}
__device__ __forceinline__ v8i_mx mx_wide(v4i a, v4i b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// acc += weights x rows; byte S of each scale register.
template <int FMT, int S>
__device__ __forceinline__ v4f_mx mx_mfma(v8i_mx w, v8i_mx x, v4f_mx acc, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, FMT == kFp4 ? 4 : 0, S, sw, S, sx);
}

template <int FMT, int S>
__device__ __forceinline__ v16f_mx mx_mfma32(v8i_mx w, v8i_mx x, v16f_mx acc, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc, 4, FMT == kFp4 ? 4 : 0, S, sw, S, sx);
}

__device__ __forceinline__ uint2 mx_bf16x4(v4f_mx v) {
  const v2bf_mx a = {(__bf16)v[0], (__bf16)v[1]}, b = {(__bf16)v[2], (__bf16)v[3]};
  return uint2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
}

// ---------------------------------------------------------------- launchers

struct MxQuantArgs {
  const void* x;
  int f32, fmt, rule;
  int64_t M, K;
  uint8_t *codes, *scales;
};
hipError_t launch_mx_quant(const MxQuantArgs& a, hipStream_t st);
hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t M, int64_t K,
                             void* y, int f32, hipStream_t st);
hipError_t launch_mx_pack(const uint8_t* codes, const uint8_t* scales, int64_t N, int64_t K, uint8_t* packed,
                          hipStream_t st);
hipError_t launch_mx_unpack(const uint8_t* packed, int64_t N, int64_t K, uint8_t* codes, uint8_t* scales,
                            hipStream_t st);
// Rows into a workspace layout (a.codes, a.scales), and, with offsets, the
// tiles of bm rows of each group.  Interleaved: the P product rows, with rows
// those that it names (zeros where it names none); else the a.M rows of x.
struct MxRowsArgs {
  bool interleaved;
  const int* rows;
  const int* offsets;
  int E, bm;
  int64_t P;
  int* ntiles;
  MxTile* tiles;
};
hipError_t launch_mx_rows(const MxQuantArgs& a, const MxRowsArgs& r, hipStream_t st);

enum MxPath { kMxToken = 1, kMxStream = 2, kMxTile = 3 };
struct MxPlan {
  int path = 0;
  int bm = 0, bn = 0;      // rows and channels of a tile
  int waves = 0;           // token, stream: wavefronts that share a strip's inputs
  int ksplit = 1;
  int64_t codes = 0, scales = 0, ntiles = 0, tiles = 0, parts = 0;  // offsets in the workspace
  int64_t bytes = 0;
};
// E = 0: the linear (P = M).
MxPlan mx_plan(int64_t M, int64_t P, int E, int64_t N, int64_t K, int fmt);
// Token and stream kernels: rows of fmt, raw ones with a.x set.
hipError_t launch_mx_stream(const MxArgs& a, const MxPlan& p, int fmt, bool gated, hipStream_t st);
hipError_t launch_mx_tile(const MxArgs& a, const MxPlan& p, int fmt, bool gated, hipStream_t st);

}  // namespace w4a8
