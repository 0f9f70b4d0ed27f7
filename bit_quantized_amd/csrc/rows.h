// The W4A8 product for batches whose rows use different weights, shared by the
// expert MLP (experts.hip) and the per-row adapters (lora.hip).
//
// Both products work on tiles of rows that share one weight:
//   - a tile of the expert MLP is a run of (token, slot) pairs routed to one
//     expert, from the list that the grouping step of the call wrote;
//   - the adapter linear has one weight, and its tiles are consecutive rows.
// The arithmetic is that of w4a8_gemm: exact int32 products per group of 128
// input channels, rescaled by s[n][g] in float32, groups in order.  A row's
// result depends on its own codes and on the weight only, never on which
// other rows share its tile or where in the tile it sits (every row of a
// matrix-core product is computed by itself), so the order in which rows are
// grouped does not show in the output.
#pragma once

#include "w4a8_internal.h"

namespace w4a8 {

typedef unsigned int v4u_rows __attribute__((ext_vector_type(4)));
typedef float v4f_rows __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf_rows __attribute__((ext_vector_type(8)));

// Where a workgroup's rows come from.
enum RowKind {
  kPlanned = 0,  // tiles listed by the grouping step
  kDirect = 1,   // tile t is pair t alone, its expert ids[t]
  kDense = 2,    // one weight; tile t is rows [t * BM, ...)
};
// What becomes of a row's sums.
enum RowOut {
  kSwiglu = 0,  // gate and up blocks together: silu(gate) * up as bf16
  kParts = 1,   // float, times the activation scale and the pair's weight
  kSplit = 2,   // unscaled float sums of one K slice
  kAdapt = 3,   // bf16 with the row's adapter product added
};
// The kernels that a product runs on; values of the plan queries (w4a8_rows.h).
enum RowPath {
  kTokenPath = 1,   // a single token's pairs, a single row
  kStreamPath = 2,  // rows_stream_kernel
  kRunPath = 3,     // rows_run_kernel
  kTilePath = 4,    // rows_tile_kernel
};
enum RowAct { kCodes = 0, kRawBf16 = 1, kRawF32 = 2 };

// A tile of grouped rows: pairs list[first .. first + rows) of `expert`; it is
// tile `place & 0xFFFF` of the expert's `place >> 16`.
struct RowTile {
  int expert, first, rows, place;
};

struct RowsArgs {
  const int8_t* qa;  // activation codes [source rows][K] and their scales
  const float* sa;
  const void* x;     // raw activations [source rows][K] (RowAct kRaw*)
  const uint8_t* codes;  // planes of the packed weight of all experts
  const uint8_t* zeros;
  const float* scales;
  const int* ntiles;     // kPlanned
  const RowTile* tiles;
  const int* list;       // null: the pairs (rows) as they are
  const int* ids;        // kDirect: the pairs' experts
  int n_experts;
  int kind;
  int64_t M;             // kDense: rows
  int64_t src_rows;      // rows of qa / x
  int K;                 // input channels
  int nbe;               // 16-channel blocks of one expert's weight
  int div;               // source row of pair p is p / div
  int cols;              // column units per expert: blocks, or gate/up block pairs
  int strips;            // workgroups per tile along the columns
  int halves;            // of them the last ones as two half tiles (kAdapt tiles)
  int kw;                // log2 of the wavefronts that share a column's groups
  int ncol;              // consecutive columns per wavefront
  int sg;                // groups of input channels that are staged
  const float* pw;       // weights of the pairs (kParts)
  uint16_t* h;           // kSwiglu output [pairs][16 * cols]
  float* parts;          // kParts [pairs][16 nbe]; kSplit [slices][M][16 nbe]
  uint16_t* y;           // kAdapt output [M][16 nbe]
  AdaptArgs ad;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// 16 bytes per lane from a buffer straight into LDS: lane i's go to lds + 16 i
// (lds is the same for the wavefront).  An offset past the buffer stores
// zeros without a request.  Written as an instruction because the compiler
// makes every LDS read that follows its builtin wait for the load, whatever
// buffer it reads; here nothing waits until loads_done() below, which has to
// come before the barrier that hands the bytes over.  (The compiler's own
// waits count the loads it knows of, and loads retire in order, so they only
// become stricter.)
// The compiler does not look for hazards inside: the load comes five wait
// states after whatever precedes the block, the rest that a memory request
// needs after a vector instruction wrote one of its scalar operands (src,
// base), and more than m0 needs.  m0 is reserved: the compiler sets it right
// before each use of its own, of which these kernels have none, and refuses it
// in a clobber list.  tests/test_rows_asm_cpu.py holds the built code to this.
struct LdsSource {
  v4i words;  // raw byte buffer descriptor
};
__device__ __forceinline__ LdsSource lds_source(const void* base, int64_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  return LdsSource{{uniform((int)(uint32_t)p), uniform((int)(uint32_t)(p >> 32) & 0xFFFF),
                    uniform((int)bytes), kBufferWord3}};
}
__device__ __forceinline__ void load_to_lds(const LdsSource& src, uint8_t* lds, int offset, int base) {
  const int at = uniform((int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(at), "v"(offset), "s"(src.words), "s"(uniform(base))
               : "memory");
}
// Four of them, to LDS 1 KiB apart: one rest serves all.
__device__ __forceinline__ void load4_to_lds(const LdsSource& src, uint8_t* lds, const uint32_t (&offset)[4],
                                             int base) {
  const int at = uniform((int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds);
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %5, %6 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %5, %6 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %5, %6 offen lds\n\t"
      "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 %4, %5, %6 offen lds"
      :
      : "s"(at), "v"(offset[0]), "v"(offset[1]), "v"(offset[2]), "v"(offset[3]), "s"(src.words), "s"(uniform(base))
      : "memory", "scc");
}
// Until at most N of this wavefront's memory requests are outstanding.
template <int N>
__device__ __forceinline__ void loads_done() {
  static_assert(N < 64, "six bits of count");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
  asm volatile("" ::: "memory");
}

// Workgroups are dealt to the 8 XCDs round-robin; workgroup b of T takes item
// xcd_run(b, T), so that each XCD has a contiguous run of items.
__device__ __forceinline__ int xcd_run(int b, int T) {
  const int xcd = b & 7, local = b >> 3;
  const int per = T >> 3, rem = T & 7;
  return xcd * per + (xcd < rem ? xcd : rem) + local;
}

struct Where {
  int expert, first, rows, strip;
};

// The tile and the column strip of this workgroup; false: nothing to do.
// Work is ordered by expert, then strip, then tile: the tiles of one expert
// that read the same weights run side by side on one XCD.
template <int BM>
__device__ __forceinline__ bool locate(const RowsArgs& a, Where& w) {
  const int b = blockIdx.x;
  if (a.kind == kPlanned) {
    const int total = uniform(a.ntiles[0]) * a.strips;
    if (b >= total) return false;
    const int at = xcd_run(b, total);
    const int t0 = at / a.strips;
    const int place = uniform(a.tiles[t0].place);
    const int f = t0 - (place & 0xFFFF), n = place >> 16;
    const int local = at - f * a.strips;
    w.strip = local / n;
    const RowTile t = a.tiles[f + local % n];
    w.expert = uniform(t.expert);
    w.first = uniform(t.first);
    w.rows = uniform(t.rows);
    return true;
  }
  const int tiles = (int)((a.M + BM - 1) / BM);
  const int at = xcd_run(b, tiles * (a.strips - a.halves));
  w.strip = at / tiles;
  w.first = (at % tiles) * BM;
  w.rows = (int)(a.M - w.first < BM ? a.M - w.first : BM);
  w.expert = 0;
  return true;
}

// Pair (or row) i of the tile.
__device__ __forceinline__ int pair_of(const RowsArgs& a, const Where& w, int i) {
  return a.list ? a.list[w.first + i] : w.first + i;
}

// Eight consecutive raw activations as float.
template <int ACT>
struct RawRow {
  static constexpr int kBytes = ACT == kRawF32 ? 4 : 2;
  static constexpr int kLoads = ACT == kRawF32 ? 2 : 1;
  static __device__ __forceinline__ void load(const uint8_t* row, int ch, v4u_rows* r) {
    const v4u_rows* p = reinterpret_cast<const v4u_rows*>(row + (int64_t)ch * 8 * kBytes);
#pragma unroll
    for (int l = 0; l < kLoads; ++l) r[l] = p[l];
  }
  static __device__ __forceinline__ void widen(const v4u_rows* r, float* v) {
    if constexpr (ACT == kRawF32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i >> 2][i & 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(r[0][i] << 16);
        v[2 * i + 1] = __uint_as_float(r[0][i] & 0xFFFF0000u);
      }
    }
  }
};

// One row quantised by a workgroup of kThreads (the rule of w4a8_quant_act);
// red: one float per wavefront in LDS.
constexpr int kHeld = 2;  // chunks of eight a thread keeps in registers
template <int ACT, int kThreads>
__device__ __forceinline__ void quantise_row(const uint8_t* xr, int K, int8_t* out, float* sa,
                                             float* red) {
  using RR = RawRow<ACT>;
  const int tid = threadIdx.x, nch = K / 8;
  const bool held = nch <= kHeld * kThreads;
  v4u_rows raw[kHeld][RR::kLoads];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * kThreads < nch) RR::load(xr, tid + i * kThreads, raw[i]);
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * kThreads < nch) {
      float v[8];
      RR::widen(raw[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
    }
  for (int ch = tid + kHeld * kThreads; ch < nch; ch += kThreads) {
    v4u_rows r[RR::kLoads];
    float v[8];
    RR::load(xr, ch, r);
    RR::widen(r, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
  }
  amax = wave_max64(amax);
  if ((tid & 63) == 0) red[tid >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) amax = fmaxf(amax, red[w]);
  const float scale = amax / 127.0f, inv = 1.0f / scale;
  if (tid == 0) *sa = scale;
  auto put = [&](int ch, const v4u_rows* r) __attribute__((always_inline)) {
    float v[8];
    RR::widen(r, v);
    *reinterpret_cast<uint2*>(out + 8 * (int64_t)ch) =
        quant8_codes(v, scale, inv);
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * kThreads < nch) put(tid + i * kThreads, raw[i]);
  if (!held)
    for (int ch = tid + kHeld * kThreads; ch < nch; ch += kThreads) {
      v4u_rows r[RR::kLoads];
      RR::load(xr, ch, r);
      put(ch, r);
    }
}

// Codes of one packed unit (16 channels x 128 inputs), its lane's zero point
// applied: the two int8 matrix-core operands.
__device__ __forceinline__ void unpack_unit(const v4u_rows& d, uint32_t zz, v4i& lo, v4i& hi) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    lo[t] = (int)sub_zero_bytes(d[t] & 0x0F0F0F0Fu, zz);
    hi[t] = (int)sub_zero_bytes((d[t] >> 4) & 0x0F0F0F0Fu, zz);
  }
}

// v as two bf16 parts: the rounded value and the rounded rest, 16 significant
// bits together.  The first part stops at bf16's largest value, so that a
// finite v above it stays finite (the rest is then below 2^121).
__device__ __forceinline__ void bf16_parts(float v, uint32_t& hi, uint32_t& lo) {
  constexpr float kTop = 0x1.FEp127f;
  hi = f32_to_bf16_rne(__builtin_amdgcn_fmed3f(v, -kTop, kTop));
  lo = f32_to_bf16_rne(v - __uint_as_float(hi << 16));
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// sum_r hx[r] B[n][r] over one adapter, hx already scaled (LDS), 32 ranks'
// loads at a time.  fetch() may run long before dot(): the loads of the first
// ranks then return beside whatever the wavefront waits for in between.
struct AdapterRow {
  static constexpr int kAhead = 4;  // chunks of eight ranks
  v4u_rows d[kAhead];
  __device__ __forceinline__ void fetch(const uint16_t* brow, int r0, int R) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      d[i] = *reinterpret_cast<const v4u_rows*>(brow + min(r0 + 8 * i, R - 8));
  }
  __device__ __forceinline__ float dot(const float* hx, const uint16_t* brow, int R) {
    float v = 0.0f;
    for (int r0 = 0; r0 < R; r0 += 8 * kAhead) {
      if (r0) fetch(brow, r0, R);
#pragma unroll
      for (int c = 0; c < kAhead; ++c)
        if (r0 + 8 * c < R) {
          const float* h = hx + r0 + 8 * c;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v += h[2 * i] * __uint_as_float(d[c][i] << 16);
            v += h[2 * i + 1] * __uint_as_float(d[c][i] & 0xFFFF0000u);
          }
        }
    }
    return v;
  }
};

// Row m's scaled adapter sums: scale * sum over the slices of hx[.][m][r].
// Eight slices' loads go out together.
__device__ __forceinline__ float adapter_sum(const AdaptArgs& ad, int64_t M, int64_t m, int r, float s) {
  const float* p = ad.hx + m * ad.R + r;
  const int64_t step = M * ad.R;
  float v = 0.0f;
  for (int k = 0; k < ad.slices; k += 8) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = k + i < ad.slices ? p[(k + i) * step] : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += t[i];
  }
  return s * v;
}

// Launchers (rows.hip).  act: RowAct of the input; mt: 16-row tiles per
// workgroup (1..4) of the weight-streaming kernel; one: tiles of a single row.
hipError_t launch_rows_stream(const RowsArgs& a, int mt, bool one, int act, int out, int64_t blocks,
                              int ksplit, hipStream_t st);
// mt, out (kSwiglu, kParts, kSplit) as above; codes only, eight columns of
// a.ncol each per workgroup (kw = 0); more than one column only unsplit.
hipError_t launch_rows_run(const RowsArgs& a, int mt, int out, int64_t blocks, int ksplit, hipStream_t st);
hipError_t launch_rows_tile(const RowsArgs& a, int out, int64_t blocks, int ksplit, hipStream_t st);
// Strips of an unsplit product that run as half tiles: those past the whole
// rounds of the compute units, where their halves fit one more round.
inline int half_strips(int64_t tiles, int64_t strips, int64_t cus) {
  const int64_t whole = tiles * strips / cus * cus / tiles, rest = strips - whole;
  return whole > 0 && 2 * rest * tiles <= cus ? (int)rest : 0;
}
// Rows per workgroup of launch_rows_tile, and its output channels.
constexpr int kTileRows = 256;
constexpr int kTileCols = 256;
// Groups of 16 mt rows of activations that fit 64 KiB of LDS.
constexpr int staged_groups(int mt) { return 32 / mt; }

}  // namespace w4a8
