// Row-tile kernels of the W4A8 product whose weight depends on the row.
//
// rows_stream_kernel: few rows per weight.  The call costs what streaming
// the weights costs, so the weights go straight from memory to registers
// (one 1 KiB unit of 16 channels x 128 inputs per wavefront load, D units in
// flight per wavefront), are unpacked there and multiplied on the int8 matrix
// cores with up to 64 rows of activations staged in LDS in operand order.
//
// rows_tile_kernel: many rows per weight, 256 rows x 256 channels, bound by
// the matrix cores and the per-group rescale.
#include "rows.h"

namespace w4a8 {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;

// ------------------------------------------------------------ few rows
//
// Per group: acc += s[n][g] * P, P the exact int32 product.  A workgroup of
// eight wavefronts takes one tile (up to 16 MT rows) and a strip of columns;
// 2^kw wavefronts share a column's groups (summed in order through LDS), the
// rest take columns of their own.  A column is a 16-channel block, or for
// kSwiglu a gate block with its up block.
//
// Staged activations: [MT][groups][2 halves][64 lanes][16 B], lane 16 j + r
// holding row r, input channels 128 g + 64 h + 16 j .. + 15, so a fragment is
// one conflict-free 16-byte read per lane.  Rows past the tile are never
// written: an int8 product of any bytes is finite and belongs to no output.
// ONE: the tile is a single raw row, kept as [groups][2][4][16 B] and read by
// all rows of the operand.
// Memory order: the activations' loads go first, then the first D weight
// units, then whatever else the tile needs, so that the activations (waited
// for first) do not queue behind the weights, and the weights stay in flight
// across the barriers, which wait for LDS only.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
// Groups whose activations fit the 64 KiB that rows_stream_kernel stages at
// once; past them rows_run_kernel, whose buffers hold run_groups() each.
constexpr int run_groups(int mt, int out) { return mt <= 2 && out != kSwiglu ? 8 : 4; }
constexpr int kStageChunks = 8;  // 16-byte pieces of activations a thread stages

template <int MT, bool ONE, int ACT, int OUT>
__global__ void __launch_bounds__(kThreads, MT > 2 || OUT == kAdapt ? 2 : 4)
rows_stream_kernel(RowsArgs a) {
  static_assert(!ONE || ACT != kCodes, "a lone row is quantised here");
  constexpr int BM = ONE ? 1 : 16 * MT;
  constexpr int NBK = OUT == kSwiglu ? 2 : 1;  // blocks per column
  constexpr int D = NBK == 2 ? 4 : 8;          // columns' units in flight
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int s_pair[BM];
  __shared__ float s_scale[BM], s_max[kWaves];
  __shared__ float s_weight[OUT == kParts ? BM : 1];  // of the pairs
  // kAdapt: scaled x A^T of the rows, and the rows' adapter products
  __shared__ float s_hx[OUT == kAdapt ? BM * kMaxRank : 1];
  __shared__ float s_dot[OUT == kAdapt ? kWaves : 1][OUT == kAdapt ? 4 : 1][64];

  Where w;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int r16 = lane & 15, j = lane >> 4;
  // raw activations: 2^rl wavefronts per row, so that a lone row is not left
  // to one of them; the first rows' chunks are held in registers
  using RR = RawRow<ACT == kCodes ? kRawBf16 : ACT>;
  constexpr int HC = ACT == kRawBf16 ? 2 : 1;
  const int nch = a.K / 8;
  v4u_rows xh[HC][RR::kLoads];
  auto raw_row = [&](int row) __attribute__((always_inline)) {
    return static_cast<const uint8_t*>(a.x) + (int64_t)(pair_of(a, w, row) / a.div) * a.K * RR::kBytes;
  };
  if constexpr (ONE) {  // (kDirect) the row's loads go out beside its expert's
    w.first = blockIdx.x / a.strips;
    w.strip = blockIdx.x % a.strips;
    w.rows = 1;
    const int e = a.ids[w.first];
    const uint8_t* xr = raw_row(0);
#pragma unroll
    for (int i = 0; i < HC; ++i)
      if (tid + i * kThreads < nch) RR::load(xr, tid + i * kThreads, xh[i]);
    __builtin_amdgcn_sched_barrier(0);
    w.expert = uniform(e);
    if (w.expert < 0 || w.expert >= a.n_experts) return;
  } else {
    if (!locate<BM>(a, w)) return;
  }
  const int rl = w.rows <= 1 ? 3 : w.rows <= 2 ? 2 : w.rows <= 4 ? 1 : 0;
  const int wpr = 1 << rl, sub = (wave & (wpr - 1)) * 64 + lane, step = 64 * wpr;
  const int G = a.K / kGroup;
  const int KW = 1 << a.kw, CW = kWaves >> a.kw;
  const int kwi = wave & (KW - 1), cw = wave >> a.kw;
  const int c0 = (w.strip * CW + cw) * a.ncol;
  const int nc = max(min(a.ncol, a.cols - c0), 0);
  const int gb = G * blockIdx.y / gridDim.y, ge = G * (blockIdx.y + 1) / gridDim.y;

  // the source rows this thread stages (kCodes: rows 16 m + r16)
  int src[MT];
  if constexpr (ACT == kCodes) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = 16 * m + r16;
      src[m] = row < w.rows ? pair_of(a, w, row) / a.div : -1;
    }
  }
  const LdsSource rqa = lds_source(a.qa, ACT == kCodes ? a.src_rows * a.K : 0);
  // kAdapt: the column's 2^kw wavefronts deal its result rows 4 j + r out, r =
  // kwi, kwi + 2^kw, ...; the first one's B row is fetched ahead
  int aid[OUT == kAdapt ? 4 : 1];
  if constexpr (OUT == kAdapt) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * j + r;
      const int id = row < w.rows ? a.ad.ids[w.first + row] : -1;
      aid[r] = nc > 0 && (r & (KW - 1)) == kwi && id >= 0 && id < a.ad.L ? id : -1;
    }
  }
  auto brow = [&](int r) __attribute__((always_inline)) {
    return a.ad.B + ((int64_t)aid[OUT == kAdapt ? r : 0] * (16 * a.nbe) + 16 * c0 + r16) * a.ad.R;
  };
  AdapterRow bh;
  if (tid < w.rows) {
    const int p = pair_of(a, w, tid);
    s_pair[tid] = p;
    if constexpr (ACT == kCodes) s_scale[tid] = a.sa[p / a.div];
    // (here, not where a column ends: a load there waits for the weights that
    // are in flight by then; expert down product of 64 tokens 24 -> 22 us)
    if constexpr (OUT == kParts) s_weight[tid] = a.pw[p];
  }

  float acc[NBK][MT][4];
#pragma unroll
  for (int b = 0; b < NBK; ++b)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[b][m][r] = 0.0f;

  // One column's sums to where they go.
  auto emit = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * m + 4 * j + r;
        if (row >= w.rows) continue;
        if constexpr (OUT == kSwiglu) {
          const float s = s_scale[row];
          a.h[(int64_t)s_pair[row] * (16 * a.cols) + 16 * c + r16] =
              f32_to_bf16_rne(silu_mul(s * acc[0][m][r], s * acc[1][m][r]));
        } else if constexpr (OUT == kParts) {
          a.parts[(int64_t)s_pair[row] * (16 * a.nbe) + 16 * c + r16] =
              s_scale[row] * s_weight[row] * acc[0][m][r];
        } else if constexpr (OUT == kSplit) {
          a.parts[((int64_t)blockIdx.y * a.M + w.first + row) * (16 * a.nbe) + 16 * c + r16] =
              acc[0][m][r];
        } else {
          a.y[(int64_t)(w.first + row) * (16 * a.nbe) + 16 * c + r16] =
              f32_to_bf16_rne(s_scale[row] * acc[0][m][r] + s_dot[cw][r][lane]);
        }
      }
  };

  const int64_t eb = (int64_t)w.expert * a.nbe;  // the expert's first block
  const int sgn = ge - gb;
  // ---- the activations' loads
  if constexpr (ACT == kCodes) {
    // straight into LDS, 1 KiB per wavefront and load (rows past the tile:
    // zeros, no request)
#pragma unroll
    for (int i = 0; i < kStageChunks; ++i) {
      const int c = tid + i * kThreads;
      const int q = c >> 7, h = (c >> 6) & 1;
      int off = kOob, m = 0, sr = src[0];
#pragma unroll
      for (int t = 1; t < MT; ++t) {
        m += q >= t * sgn;
        sr = m == t ? src[t] : sr;
      }
      if (sr >= 0) off = sr * a.K + (gb + q - m * sgn) * kGroup + 64 * h + 16 * j;
      if (uniform(c) < MT * sgn * 128) load_to_lds(rqa, smem + uniform(c) * 16, off, 0);
    }
  } else if constexpr (!ONE) {
    const int row = wave >> rl;
    if (row < w.rows) {
      const uint8_t* xr = raw_row(row);
#pragma unroll
      for (int i = 0; i < HC; ++i)
        if (sub + i * step < nch) RR::load(xr, sub + i * step, xh[i]);
    }
  }
  __builtin_amdgcn_sched_barrier(0);

  // ---- the first weight units.  This wavefront's groups, and its run of
  // units: nc columns of them (several columns only when they cover all
  // groups, so the run is contiguous in the packed planes)
  const int k0 = sgn * kwi / KW, kn = sgn * (kwi + 1) / KW - k0;
  const int T = kn * nc;
  __amdgpu_buffer_rsrc_t rc[NBK], rs[NBK], rz[NBK];
#pragma unroll
  for (int b = 0; b < NBK; ++b) {
    const int64_t b0 = (eb + b * a.cols + (nc > 0 ? c0 : 0)) * G + gb + k0;
    rc[b] = rsrc_of(a.codes + b0 * kBlockBytes, (int64_t)T * kBlockBytes);
    rs[b] = rsrc_of(a.scales + b0 * 16, (int64_t)T * 64);
    rz[b] = rsrc_of(a.zeros + b0 * kZeroBlockBytes, (int64_t)T * kZeroBlockBytes);
  }
  v4u_rows d[D][NBK];
  float s[D][NBK];
  uint32_t z[D][NBK];
  // past the run (the descriptors' end): no memory request, zeros
  auto load = [&](int i, int t) __attribute__((always_inline)) {
    t = min(t, T);
#pragma unroll
    for (int b = 0; b < NBK; ++b) {
      d[i][b] = __builtin_amdgcn_raw_buffer_load_b128(rc[b], 16 * lane, (unsigned)uniform(t * kBlockBytes),
                                                      kNontemporal);
      s[i][b] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(rs[b], 4 * r16, (unsigned)uniform(t * 64), 0));
      z[i][b] = __builtin_amdgcn_raw_buffer_load_b8(rz[b], r16 >> 1, (unsigned)uniform(t * kZeroBlockBytes), 0);
    }
  };
#pragma unroll
  for (int i = 0; i < D; ++i) {
    load(i, i);
    __builtin_amdgcn_sched_barrier(0);
  }

  // ---- activations -> LDS
  if constexpr (ACT == kCodes) {
    loads_done<3 * NBK * D>();
  } else {
    // quantised here (the rule of w4a8_quant_act)
    for (int row0 = 0; row0 < w.rows; row0 += kWaves >> rl) {
      const int row = row0 + (wave >> rl);
      const bool live = row < w.rows, held = row0 == 0;
      const uint8_t* xr = raw_row(live ? row : 0);
      float amax = 0.0f;
      auto most = [&](const v4u_rows* r) __attribute__((always_inline)) {
        float v[8];
        RR::widen(r, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
      };
      if (live) {
        if (held) {
#pragma unroll
          for (int i = 0; i < HC; ++i)
            if (sub + i * step < nch) most(xh[i]);
        }
        for (int ch = sub + (held ? HC * step : 0); ch < nch; ch += step) {
          v4u_rows r[RR::kLoads];
          RR::load(xr, ch, r);
          most(r);
        }
      }
      amax = wave_max64(amax);
      if (wpr > 1) {  // (the only pass of the row loop: at most 8 / wpr rows)
        if (lane == 0) s_max[wave] = amax;
        lds_barrier();
        for (int i = 0; i < wpr; ++i) amax = fmaxf(amax, s_max[(wave & ~(wpr - 1)) + i]);
      }
      if (live) {
        const float scale = amax / 127.0f, inv = 1.0f / scale;
        if (sub == 0) s_scale[row] = scale;
        auto put = [&](int ch, const v4u_rows* r) __attribute__((always_inline)) {
          float v[8];
          RR::widen(r, v);
          const uint2 codes = quant8_codes(v, scale, inv);
          const int g = ch >> 4, h = (ch >> 3) & 1, jj = (ch >> 1) & 3;
          const int at = ONE ? ((g * 2 + h) * 4 + jj) * 16
                             : (((row >> 4) * sgn + g) * 2 + h) * 1024 + (16 * jj + (row & 15)) * 16;
          *reinterpret_cast<uint2*>(smem + at + 8 * (ch & 1)) = codes;
        };
        if (held) {
#pragma unroll
          for (int i = 0; i < HC; ++i)
            if (sub + i * step < nch) put(sub + i * step, xh[i]);
        }
        for (int ch = sub + (held ? HC * step : 0); ch < nch; ch += step) {
          v4u_rows r[RR::kLoads];
          RR::load(xr, ch, r);
          put(ch, r);
        }
      }
    }
  }
  if constexpr (OUT == kAdapt) {
    if (kwi < 4) {
      const int f = kwi == 0 ? aid[0] : kwi == 1 ? aid[1] : kwi == 2 ? aid[2] : aid[3];
      if (f >= 0)
        bh.fetch(a.ad.B + ((int64_t)f * (16 * a.nbe) + 16 * c0 + r16) * a.ad.R, 0, a.ad.R);
    }
    for (int i = tid; i < w.rows * a.ad.R; i += kThreads) {
      const int row = i / a.ad.R, id = a.ad.ids[w.first + row];
      if (id >= 0 && id < a.ad.L)
        s_hx[i] = adapter_sum(a.ad, a.M, w.first + row, i - row * a.ad.R, a.ad.scale[id]);
    }
  }
  lds_barrier();
  if constexpr (OUT == kAdapt) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if ((r & (KW - 1)) == kwi) {
        float v = 0.0f;
        if (aid[r] >= 0) {
          if (r != kwi) bh.fetch(brow(r), 0, a.ad.R);
          v = bh.dot(s_hx + (4 * j + r) * a.ad.R, brow(r), a.ad.R);
        }
        s_dot[cw][r][lane] = v;
      }
  }

  // ---- stream the run
  int g = 0, c = c0;
  for (int tb = 0; tb < T; tb += D) {
#pragma unroll
    for (int i = 0; i < D; ++i) {
      if (tb + i < T) {
        v4i lo[NBK], hi[NBK];
        float sc[NBK];
#pragma unroll
        for (int b = 0; b < NBK; ++b) {
          const uint32_t zz = ((z[i][b] >> (4 * (r16 & 1))) & 0xFu) * 0x01010101u;
          unpack_unit(d[i][b], zz, lo[b], hi[b]);
          sc[b] = s[i][b];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint8_t* frag = ONE ? smem + (k0 + g) * 128 + 16 * j
                                    : smem + (m * sgn + k0 + g) * 2048 + 16 * lane;
          const v4i a0 = *reinterpret_cast<const v4i*>(frag);
          const v4i a1 = *reinterpret_cast<const v4i*>(frag + (ONE ? 64 : 1024));
#pragma unroll
          for (int b = 0; b < NBK; ++b) {
            v4i p = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, lo[b], kBiasSeed, 0, 0, 0);
            p = __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, hi[b], p, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[b][m][r] += sc[b] * unbias(p[r]);
          }
        }
        if (++g == kn) {
          g = 0;
          if (a.kw == 0) {
            emit(c);
            ++c;
#pragma unroll
            for (int b = 0; b < NBK; ++b)
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[b][m][r] = 0.0f;
          }
        }
      }
      load(i, tb + i + D);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (a.kw == 0) return;

  // the wavefronts of a column, summed in group order
  lds_barrier();
  float* red = reinterpret_cast<float*>(smem) + cw * KW * (NBK * MT * 256);
#pragma unroll
  for (int b = 0; b < NBK; ++b)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[kwi * (NBK * MT * 256) + ((b * MT + m) * 4 + r) * 64 + lane] = acc[b][m][r];
  lds_barrier();
  if (kwi != 0 || nc == 0) return;
#pragma unroll
  for (int b = 0; b < NBK; ++b)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        for (int k = 1; k < KW; ++k)
          acc[b][m][r] += red[k * (NBK * MT * 256) + ((b * MT + m) * 4 + r) * 64 + lane];
  emit(c0);
}

// ------------------------------------------- few rows, many groups
//
// The same product where a tile's activations exceed 64 KiB of LDS: they pass
// through two LDS buffers of SG groups each, the next slice's loads going out
// when the current slice begins.  A wavefront's weights (ncol columns, all
// their groups: one run of the packed planes) flow through a ring of SG units
// that the slices do not interrupt: slot i holds unit i of a slice and is
// refilled with unit i of the next one.  Slices have L <= SG units each (the
// last of a column may have fewer); a slot without a unit loads nothing.
// (517 tokens, 32 experts, 3584 -> 2 x 1280: 53 us, against 73 when every
// slice drained the ring and waited for its activations.)
// ML: the 16-row fragments that the tile's rows reach (a tile of at most 16
// MT rows often has fewer).
template <int ML, int MT, int OUT>
__device__ __forceinline__ void run_tile(const RowsArgs& a, const Where& w, uint8_t* smem, int* s_pair,
                                         uint32_t* s_off, float* s_scale) {
  constexpr int BM = 16 * ML;
  constexpr int NBK = OUT == kSwiglu ? 2 : 1;
  constexpr int SG = run_groups(MT, OUT);
  constexpr int kSlice = SG * MT * 2048;  // bytes of a buffer
  static_assert(SG % 4 == 0, "a whole number of loads per wavefront");
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int r16 = lane & 15, j = lane >> 4;
  const int G = a.K / kGroup;
  const int gb = G * blockIdx.y / gridDim.y, Gs = G * (blockIdx.y + 1) / gridDim.y - gb;
  const int c0 = (w.strip * kWaves + wave) * a.ncol;
  const int nc = max(min(a.ncol, a.cols - c0), 0);
  const int columns = min(a.ncol, a.cols - w.strip * kWaves * a.ncol);  // of the first wavefront
  const int S = (Gs + SG - 1) / SG, L = (Gs + S - 1) / S;

  // slice s of the activations into a buffer, [MT][SG][2 halves][64 lanes]
  // [16 B]: of the 2 SG KiB of 16 rows this wavefront loads KiB wave, wave + 8
  // (the rows' offsets wait in LDS: kept in registers they were spilled, and
  // a reload from memory queues behind the weights in flight)
  constexpr int kPer = SG / 4;
  const LdsSource rqa = lds_source(a.qa, a.src_rows * a.K);
  if (tid < BM) {
    int off = kOob;
    if (tid < w.rows) {
      const int p = pair_of(a, w, tid), src = p / a.div;
      off = src * a.K + gb * kGroup;
      s_pair[tid] = p;
      s_scale[tid] = OUT == kParts ? a.sa[src] * a.pw[p] : a.sa[src];
    }
    s_off[tid] = off;
  }
  auto stage = [&](uint8_t* buf, int s) __attribute__((always_inline)) {
    const int live = 2 * min(L, Gs - s * L);
    uint32_t off[ML];
#pragma unroll
    for (int m = 0; m < ML; ++m) off[m] = s_off[16 * m + r16] + 64 * wave + 16 * j;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = wave + i * kWaves;
      if (c >= live) break;
#pragma unroll
      for (int m = 0; m < ML; ++m)
        load_to_lds(rqa, buf + (m * 2 * SG + c) * 1024, (int)off[m], s * L * kGroup + i * kWaves * 64);
    }
  };

  // the run's planes; unit t of the run is group t % G of column t / G (one
  // column where K is split)
  __amdgpu_buffer_rsrc_t rc[NBK], rs[NBK], rz[NBK];
  const int T = nc > 1 ? nc * G : nc * Gs;
#pragma unroll
  for (int b = 0; b < NBK; ++b) {
    const int64_t b0 = ((int64_t)w.expert * a.nbe + b * a.cols + (nc > 0 ? c0 : 0)) * G + gb;
    rc[b] = rsrc_of(a.codes + b0 * kBlockBytes, (int64_t)T * kBlockBytes);
    rs[b] = rsrc_of(a.scales + b0 * 16, (int64_t)T * 64);
    rz[b] = rsrc_of(a.zeros + b0 * kZeroBlockBytes, (int64_t)T * kZeroBlockBytes);
  }
  v4u_rows d[SG][NBK];
  float s[SG][NBK];
  uint32_t z[SG][NBK];
  auto load = [&](int i, int t) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < NBK; ++b) {
      d[i][b] = __builtin_amdgcn_raw_buffer_load_b128(rc[b], 16 * lane, (unsigned)uniform(t * kBlockBytes),
                                                      kNontemporal);
      s[i][b] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(rs[b], 4 * r16, (unsigned)uniform(t * 64), 0));
      z[i][b] = __builtin_amdgcn_raw_buffer_load_b8(rz[b], r16 >> 1, (unsigned)uniform(t * kZeroBlockBytes), 0);
    }
  };

  float acc[NBK][ML][4];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < NBK; ++b)
#pragma unroll
      for (int m = 0; m < ML; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[b][m][r] = 0.0f;
  };
  clear();
  lds_barrier();
  stage(smem, 0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < SG; ++i) {
    load(i, i < min(L, Gs) ? i : T);
    __builtin_amdgcn_sched_barrier(0);
  }

  int col = 0, sl = 0;
  for (int q = 0; q < columns * S; ++q) {
    // the slice after this one
    const bool wrap = sl + 1 == S;
    const int nsl = wrap ? 0 : sl + 1, ncol = wrap ? col + 1 : col;
    const int live = min(L, Gs - sl * L), nlive = ncol < nc ? min(L, Gs - nsl * L) : 0;
    const int nt = ncol * G + nsl * L;
    uint8_t* buf = smem + (q & 1) * kSlice;
    loads_done<3 * NBK * SG>();  // this slice's activations
    lds_barrier();
    if (q + 1 < columns * S) stage(smem + ((q + 1) & 1) * kSlice, nsl);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      if (i < live && col < nc) {
        v4i lo[NBK], hi[NBK];
        float sc[NBK];
#pragma unroll
        for (int b = 0; b < NBK; ++b) {
          const uint32_t zz = ((z[i][b] >> (4 * (r16 & 1))) & 0xFu) * 0x01010101u;
          unpack_unit(d[i][b], zz, lo[b], hi[b]);
          sc[b] = s[i][b];
        }
#pragma unroll
        for (int m = 0; m < ML; ++m) {
          const uint8_t* frag = buf + (m * SG + i) * 2048 + 16 * lane;
          const v4i a0 = *reinterpret_cast<const v4i*>(frag);
          const v4i a1 = *reinterpret_cast<const v4i*>(frag + 1024);
#pragma unroll
          for (int b = 0; b < NBK; ++b) {
            v4i p = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, lo[b], kBiasSeed, 0, 0, 0);
            p = __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, hi[b], p, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[b][m][r] += sc[b] * unbias(p[r]);
          }
        }
      }
      load(i, i < nlive ? nt + i : T);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (wrap) {
      if (col < nc) {
        const int c = c0 + col;
        int first = 4 * j;
        asm volatile("" : "+v"(first));  // nothing of the rows' addresses is kept over the loop
#pragma unroll
        for (int m = 0; m < ML; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 16 * m + first + r;
            if (row >= w.rows) continue;
            if constexpr (OUT == kSwiglu)
              a.h[(int64_t)s_pair[row] * (16 * a.cols) + 16 * c + r16] = f32_to_bf16_rne(
                  silu_mul(s_scale[row] * acc[0][m][r], s_scale[row] * acc[1][m][r]));
            else if constexpr (OUT == kParts)
              a.parts[(int64_t)s_pair[row] * (16 * a.nbe) + 16 * c + r16] = s_scale[row] * acc[0][m][r];
            else
              a.parts[((int64_t)blockIdx.y * a.M + w.first + row) * (16 * a.nbe) + 16 * c + r16] =
                  acc[0][m][r];
          }
        clear();
      }
    }
    sl = nsl;
    col = ncol;
  }
}

template <int MT, int OUT>
__global__ void __launch_bounds__(kThreads, 4)
rows_run_kernel(RowsArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int s_pair[16 * MT];
  __shared__ uint32_t s_off[16 * MT];
  __shared__ float s_scale[16 * MT];
  Where w;
  if (!locate<16 * MT>(a, w)) return;
  if (MT == 1 || w.rows <= 16)
    run_tile<1, MT, OUT>(a, w, smem, s_pair, s_off, s_scale);
  else if (MT == 2 || w.rows <= 32)
    run_tile<MT < 2 ? MT : 2, MT, OUT>(a, w, smem, s_pair, s_off, s_scale);
  else if (MT == 3 || w.rows <= 48)
    run_tile<MT < 3 ? MT : 3, MT, OUT>(a, w, smem, s_pair, s_off, s_scale);
  else
    run_tile<MT, MT, OUT>(a, w, smem, s_pair, s_off, s_scale);
}

// ----------------------------------------------------------- many rows
//
// 256 rows x 256 channels per workgroup of eight wavefronts (64 x 128 each).
// Per group of 128 inputs the activation tile (32 KiB) goes from memory
// straight into LDS, the 16 code blocks are unpacked once to q - z bytes in
// LDS, both double-buffered, one group ahead of the products.  The rows are
// gathered: the LDS-direct loads take a byte offset per lane.  Rows past the
// tile read as zeros without a request.
//
// The wavefronts lie 4 x 2 over the tile with rows (wave / 2) * 64, so that
// wavefronts w and w + 4, which share a SIMD, hold rows 128 apart: a tile of at most
// 128 rows leaves one working wavefront on every SIMD and takes about half
// the time, as the others skip the products.
//
// kSwiglu: the 256 channels are 128 gate channels and their 128 up channels;
// a wavefront's 8 blocks are 4 gate blocks and the matching up blocks.
constexpr int kABytes = kTileRows * kGroup;                // [256][128], chunks swizzled by row
constexpr int kBBytes = (kTileCols / 16) * 2 * kBlockBytes;  // [16][2][64 lanes][16 B]
constexpr int kBufBytes = kABytes + kBBytes + kTileCols * 4;
constexpr int kBOff = kABytes, kSOff = kABytes + kBBytes;

__device__ __forceinline__ int a_chunk(int r, int c) { return c ^ (r & 7); }

// NU = 8: a whole tile of 16 blocks from cb; 4: a half tile of 8.  s_id: the
// rows' adapters, -1 for none.
template <int OUT, int NU>
__device__ __forceinline__ void row_tile(const RowsArgs& a, const Where& w, int cb,
                                         uint8_t (&smem)[2][kBufBytes], int* s_pair, float* s_scale,
                                         int* s_id) {
  constexpr int T = 4 * NU;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int r16 = lane & 15, j = lane >> 4;
  const int wm = wave >> 1, wn = wave & 1;
  const int G = a.K / kGroup;
  const int gb = G * blockIdx.y / gridDim.y, ge = G * (blockIdx.y + 1) / gridDim.y;
  const bool works = wm * 64 < w.rows;
  const int NB = a.nbe;

  for (int i = tid; i < w.rows; i += kThreads) {
    const int p = pair_of(a, w, i);
    s_pair[i] = p;
    float sc = OUT == kSplit ? 1.0f : a.sa[p / a.div];
    if constexpr (OUT == kParts) sc *= a.pw[p];
    s_scale[i] = sc;
    if constexpr (OUT == kAdapt) {
      const int id = a.ad.ids[p];
      s_id[i] = id >= 0 && id < a.ad.L ? id : -1;
    }
  }

  // block q of the tile: wavefront column q / NU, its column u = q % NU
  auto block_of = [&](int q) __attribute__((always_inline)) {
    if constexpr (OUT == kSwiglu) {
      const int u = q & 7;
      return (u >> 2) * a.cols + w.strip * 8 + (q >> 3) * 4 + (u & 3);
    } else {
      return min(cb + q, NB - 1);  // past the end: columns that are never stored
    }
  };
  const int64_t eb = (int64_t)w.expert * NB;
  const uint8_t* codes = a.codes + eb * G * kBlockBytes;
  const uint8_t* zeros = a.zeros + eb * G * kZeroBlockBytes;
  const float* scales = a.scales + eb * G * 16;

  uint32_t oa[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * (4 * wave + i) + (lane >> 3);
    oa[i] = r < w.rows ? (uint32_t)(pair_of(a, w, r) / a.div) * a.K + 16 * a_chunk(r, lane & 7) : kOob;
  }
  const int b0 = block_of(wave), b1 = block_of(wave + 8), bs = block_of((tid >> 4) & (2 * NU - 1));
  const uint32_t ob[2] = {(uint32_t)b0 * G * kBlockBytes + lane * 16, (uint32_t)b1 * G * kBlockBytes + lane * 16};
  const uint32_t oz[2] = {(uint32_t)b0 * G * 8 + (r16 >> 1), (uint32_t)b1 * G * 8 + (r16 >> 1)};
  const uint32_t os = (uint32_t)bs * G * 16 + r16;
  const int zshift = (lane & 1) * 4;
  const LdsSource rqa = lds_source(a.qa, a.src_rows * a.K);

  v4u_rows sb[2];
  uint32_t sz[2];
  float ss;
  auto dma = [&](uint8_t* buf, int g) __attribute__((always_inline)) {
    load4_to_lds(rqa, buf + 4 * wave * 1024, oa, g * kGroup);
  };
  auto fetch = [&](int g) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < NU / 4; ++k) {
      sb[k] = *reinterpret_cast<const v4u_rows*>(codes + (int64_t)g * kBlockBytes + ob[k]);
      sz[k] = (zeros + g * kZeroBlockBytes)[oz[k]];
    }
    ss = (scales + g * 16)[os];
  };
  auto store_block = [&](uint8_t* buf, int k) __attribute__((always_inline)) {
    v4i lo, hi;
    unpack_unit(sb[k], ((sz[k] >> zshift) & 0xFu) * 0x01010101u, lo, hi);
    uint8_t* at = buf + kBOff + (wave + 8 * k) * 2 * kBlockBytes + lane * 16;
    *reinterpret_cast<v4i*>(at) = lo;
    *reinterpret_cast<v4i*>(at + kBlockBytes) = hi;
  };
  // scales as [16 channels][16 blocks]: a lane's eight are contiguous
  auto store_scale = [&](uint8_t* buf) __attribute__((always_inline)) {
    reinterpret_cast<float*>(buf + kSOff)[r16 * 16 + ((tid >> 4) & (2 * NU - 1))] = ss;
  };

  float acc[4][NU][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][u][r] = 0.0f;

  // One group: per 16 x 16 tile an MFMA pair and, two tiles later, its
  // rescale; the next group's blocks are unpacked between them.
  auto compute = [&](const uint8_t* buf, uint8_t* next) __attribute__((always_inline)) {
    v4i a0[4], a1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* arow = buf + (wm * 64 + i * 16 + r16) * kGroup;
      a0[i] = *reinterpret_cast<const v4i*>(arow + 16 * a_chunk(r16, j));
      a1[i] = *reinterpret_cast<const v4i*>(arow + 16 * a_chunk(r16, 4 + j));
    }
    float sv[NU];
    const float* srow = reinterpret_cast<const float*>(buf + kSOff) + r16 * 16 + wn * NU;
#pragma unroll
    for (int q = 0; q < NU / 4; ++q) {
      const v4i t = *reinterpret_cast<const v4i*>(srow + 4 * q);
#pragma unroll
      for (int u = 0; u < 4; ++u) sv[4 * q + u] = __int_as_float(t[u]);
    }
    v4i q0[NU], q1[NU];
    auto load_b = [&](int u) __attribute__((always_inline)) {
      const uint8_t* at = buf + kBOff + (wn * NU + u) * 2 * kBlockBytes + lane * 16;
      q0[u] = *reinterpret_cast<const v4i*>(at);
      q1[u] = *reinterpret_cast<const v4i*>(at + kBlockBytes);
    };
    load_b(0);
    v4i p[T];
#pragma unroll
    for (int t = 0; t < T + 2; ++t) {
      if (t < T) {
        const int u = t >> 2, i = t & 3;
        if (i == 0 && u + 1 < NU) load_b(u + 1);
        if (next && t == T / 2) store_block(next, 0);
        if (NU == 8 && next && t == 22) store_block(next, 1);
        if (next && t == T - 4) store_scale(next);
        p[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0[i], q0[u], kBiasSeed, 0, 0, 0);
        p[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a1[i], q1[u], p[t], 0, 0, 0);
      }
      if (t >= 2) {
        const int e = t - 2, u = e >> 2, i = e & 3;
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][u][r] += sv[u] * unbias(p[e][r]);
        if (t + 1 < T) {  // keeps pairs and rescales interleaved (no instruction)
          const int in = (t + 1) & 3;
          asm volatile("" : "+v"(a0[in]) : "v"(acc[i][u][0]), "v"(acc[i][u][1]), "v"(acc[i][u][2]),
                       "v"(acc[i][u][3]));
        }
      }
    }
  };

  dma(smem[0], gb);
  fetch(gb);
  store_block(smem[0], 0);
  if (NU == 8) store_block(smem[0], 1);
  store_scale(smem[0]);
  loads_done<0>();
  __syncthreads();
  if (!works) {  // feeds the others; the same barriers
    for (int g = gb; g < ge; ++g) {
      if (g + 1 < ge) {
        uint8_t* next = smem[(g - gb + 1) & 1];
        dma(next, g + 1);
        fetch(g + 1);
        store_block(next, 0);
        if (NU == 8) store_block(next, 1);
        store_scale(next);
      }
      loads_done<0>();
      __syncthreads();
    }
    return;
  }
  // One group from `cur` while the next one's operands go into `next`, which
  // was last read before the previous barrier.
  auto step = [&](const uint8_t* cur, uint8_t* next, int g) __attribute__((always_inline)) {
    if (g + 1 < ge) {
      dma(next, g + 1);
      fetch(g + 1);
    }
    compute(cur, g + 1 < ge ? next : nullptr);
    loads_done<0>();
    __syncthreads();
  };
  for (int g = gb; g < ge; g += 2) {
    step(smem[0], smem[1], g);
    if (g + 1 < ge) step(smem[1], smem[0], g + 1);
  }

  if constexpr (OUT == kAdapt) {
    // sums scaled, then each adapter's product added on the bf16 matrix
    // cores: per adapter present in a 16-row fragment, the scaled x A^T of its
    // rows as two bf16 parts (16 significant bits) against B.  The product is
    // made apart and added to the adapter's own rows only, so what B holds
    // (an infinity, a NaN) reaches no other row.  The int8 and bf16 products
    // share one result layout.  (2048 rows, 16 adapters of rank 32, 3584 ->
    // 18944: 205 to 214 us, where the layer's own tiles take 182; 32 us more
    // with x A^T summed and split here, by every strip of channels again.)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = wm * 64 + i * 16 + 4 * j + r;
        const float s = row < w.rows ? s_scale[row] : 0.0f;
#pragma unroll
        for (int u = 0; u < NU; ++u) acc[i][u][r] *= s;
      }
    for (int r0 = 0; r0 < a.ad.R; r0 += 32) {
      const int rr = r0 + 8 * j;  // this lane's eight ranks
      int held = -1;              // the adapter whose B is in bv
      v4i bv[NU], ah[4], al[4];
      int id[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = wm * 64 + i * 16 + r16;
        id[i] = row < w.rows ? s_id[row] : -1;
        ah[i] = al[i] = v4i{0, 0, 0, 0};
        if (id[i] >= 0 && rr < a.ad.R) {
          const int64_t at = (int64_t)s_pair[row] * a.ad.R + rr;
          ah[i] = *reinterpret_cast<const v4i*>(a.ad.hi + at);
          al[i] = *reinterpret_cast<const v4i*>(a.ad.lo + at);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint64_t todo = __ballot(id[i] >= 0) & 0xFFFFull;
        while (todo) {
          const int l = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(todo));
          const uint64_t rows = __ballot(id[i] == l) & 0xFFFFull;
          todo &= ~rows;
          if (l != held) {  // (the rows come in the order of their adapters)
            held = l;
#pragma unroll
            for (int u = 0; u < NU; ++u) {
              const int nb = min(cb + wn * NU + u, NB - 1);
              bv[u] = v4i{0, 0, 0, 0};
              if (rr < a.ad.R)
                bv[u] = *reinterpret_cast<const v4i*>(
                    a.ad.B + (((int64_t)l * NB + nb) * 16 + r16) * a.ad.R + rr);
            }
          }
          const v4i zero = {0, 0, 0, 0};
          const v4i h = id[i] == l ? ah[i] : zero, lw = id[i] == l ? al[i] : zero;
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            v4f_rows c = {0.f, 0.f, 0.f, 0.f};
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_rows, h),
                                                        __builtin_bit_cast(v8bf_rows, bv[u]), c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_rows, lw),
                                                        __builtin_bit_cast(v8bf_rows, bv[u]), c, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][u][r] += (rows >> (4 * j + r)) & 1 ? c[r] : 0.0f;
          }
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = wm * 64 + i * 16 + 4 * j + r;
      if (row >= w.rows) continue;
      const float s = s_scale[row];
      const int64_t p = s_pair[row];
      if constexpr (OUT == kSwiglu) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          a.h[p * (16 * a.cols) + 16 * (w.strip * 8 + wn * 4 + u) + r16] =
              f32_to_bf16_rne(silu_mul(s * acc[i][u][r], s * acc[i][u + 4][r]));
      } else {
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const int nb = cb + wn * NU + u;
          if (nb >= NB) continue;
          const int64_t n = 16 * nb + r16;
          if constexpr (OUT == kParts)
            a.parts[p * (16 * NB) + n] = s * acc[i][u][r];
          else if constexpr (OUT == kSplit)
            a.parts[((int64_t)blockIdx.y * a.M + p) * (16 * NB) + n] = acc[i][u][r];
          else
            a.y[p * (16 * NB) + n] = f32_to_bf16_rne(acc[i][u][r]);
        }
      }
    }
}

template <int OUT>
__global__ void __launch_bounds__(kThreads)
rows_tile_kernel(RowsArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[2][kBufBytes];
  __shared__ int s_pair[kTileRows];
  __shared__ float s_scale[kTileRows];
  __shared__ int s_id[OUT == kAdapt ? kTileRows : 1];
  Where w;
  if constexpr (OUT == kAdapt) {
    // the last strips may come as half tiles: they fill a last round of the
    // compute units that whole ones would leave partly idle (half_strips)
    const int tiles = (int)((a.M + kTileRows - 1) / kTileRows), whole = tiles * (a.strips - a.halves);
    const int b = blockIdx.x;
    if (b >= whole) {
      const int at = xcd_run(b - whole, tiles * 2 * a.halves);
      w.expert = 0;
      w.strip = 0;
      w.first = at % tiles * kTileRows;
      w.rows = (int)(a.M - w.first < kTileRows ? a.M - w.first : kTileRows);
      const int cb = (a.strips - a.halves) * 16 + at / tiles * 8;
      if (cb < a.nbe) row_tile<OUT, 4>(a, w, cb, smem, s_pair, s_scale, s_id);
      return;
    }
  }
  if (!locate<kTileRows>(a, w)) return;
  row_tile<OUT, 8>(a, w, w.strip * 16, smem, s_pair, s_scale, s_id);
}

template <int MT, bool ONE, int ACT, int OUT>
hipError_t stream_launch(const RowsArgs& a, int64_t blocks, int ksplit, hipStream_t st) {
  const size_t groups = (size_t)(a.sg);
  size_t lds = ONE ? (groups * 128 + 1023) / 1024 * 1024 : groups * MT * 2048;
  const size_t red = a.kw ? (size_t)kWaves * (OUT == kSwiglu ? 2 : 1) * MT * 1024 : 0;
  if (red > lds) lds = red;
  hipLaunchKernelGGL((rows_stream_kernel<MT, ONE, ACT, OUT>), dim3((unsigned)blocks, (unsigned)ksplit),
                     dim3(kThreads), lds, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rows_stream(const RowsArgs& a, int mt, bool one, int act, int out, int64_t blocks,
                              int ksplit, hipStream_t st) {
  // what the kernel stages
  if (act == kCodes && a.sg * 128 * mt > kThreads * kStageChunks) return hipErrorInvalidValue;
#define ROWS_CASE(MTV, ONEV, ACTV, OUTV) \
  if (mt == MTV && one == ONEV && act == ACTV && out == OUTV) \
    return stream_launch<MTV, ONEV, ACTV, OUTV>(a, blocks, ksplit, st);
  ROWS_CASE(1, true, kRawBf16, kSwiglu)
  ROWS_CASE(1, true, kRawF32, kSwiglu)
  ROWS_CASE(1, false, kCodes, kSwiglu)
  ROWS_CASE(2, false, kCodes, kSwiglu)
  ROWS_CASE(4, false, kCodes, kSwiglu)
  ROWS_CASE(1, false, kRawBf16, kParts)
  ROWS_CASE(2, false, kCodes, kParts)
  ROWS_CASE(4, false, kCodes, kParts)
  ROWS_CASE(1, false, kCodes, kSplit)
  ROWS_CASE(2, false, kCodes, kSplit)
  ROWS_CASE(3, false, kCodes, kSplit)
  ROWS_CASE(4, false, kCodes, kSplit)
  ROWS_CASE(1, false, kCodes, kAdapt)
#undef ROWS_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_rows_run(const RowsArgs& a, int mt, int out, int64_t blocks, int ksplit, hipStream_t st) {
#define RUN_CASE(MTV, OUTV)                                                                      \
  if (mt == MTV && out == OUTV) {                                                                \
    hipLaunchKernelGGL((rows_run_kernel<MTV, OUTV>), dim3((unsigned)blocks, (unsigned)ksplit),   \
                       dim3(kThreads), 2 * (size_t)run_groups(MTV, OUTV) * MTV * 2048, st, a);   \
    return hipGetLastError();                                                                    \
  }
  RUN_CASE(1, kSwiglu)
  RUN_CASE(2, kSwiglu)
  RUN_CASE(4, kSwiglu)
  RUN_CASE(1, kParts)
  RUN_CASE(2, kParts)
  RUN_CASE(4, kParts)
  RUN_CASE(1, kSplit)
  RUN_CASE(2, kSplit)
  RUN_CASE(3, kSplit)
  RUN_CASE(4, kSplit)
#undef RUN_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_rows_tile(const RowsArgs& a, int out, int64_t blocks, int ksplit, hipStream_t st) {
  const dim3 grid((unsigned)blocks, (unsigned)ksplit), block(kThreads);
  if (out == kSwiglu)
    hipLaunchKernelGGL((rows_tile_kernel<kSwiglu>), grid, block, 0, st, a);
  else if (out == kParts)
    hipLaunchKernelGGL((rows_tile_kernel<kParts>), grid, block, 0, st, a);
  else if (out == kSplit)
    hipLaunchKernelGGL((rows_tile_kernel<kSplit>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((rows_tile_kernel<kAdapt>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace w4a8
