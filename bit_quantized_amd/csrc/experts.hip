// Grouping of a batch by expert, and what the expert MLP needs beside its two
// row-tile products (rows.hip): the down projection of single tokens and the
// sum over a token's experts.
#include "experts.h"

#include <algorithm>
#include <cmath>

namespace w4a8 {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;

// ------------------------------------------------ grouping + quantisation
//
// The pairs in expert order, and the tiles of at most bm pairs of one expert
// each.  Up to kOnePlace pairs a single workgroup does it: a histogram of the
// experts in LDS, prefix sums, tiles and list.  More pairs are counted by
// `counters` workgroups, a run of pairs each, and placed by as many of a second
// launch, which sum the counts before theirs (24576 pairs: 18 us with the
// quantisation beside it, against 29 with one workgroup).  The place of a
// pair inside its expert follows the order of LDS atomics and may differ
// between calls; no output depends on it (rows.h).  The other workgroups
// quantise one token each (w4a8_quant_act's rule).
constexpr int64_t kOnePlace = 4096;
constexpr int kMostCounters = 64;
int counters_of(int64_t P) {
  const int64_t n = P <= kOnePlace ? 1 : (P + 1023) / 1024;
  return (int)(n < kMostCounters ? n : kMostCounters);
}

struct GroupArgs {
  const int* ids;
  int P, E, bm, counters;
  int* ntiles;
  RowTile* tiles;
  int *list, *rank;
  int* counts;  // [counters][E]
};

// Counts of pairs [p0, p1) into s_count, and each one's place among them.
constexpr int kAtOnce = 8;
__device__ __forceinline__ void count_pairs(const GroupArgs& g, int p0, int p1, int* s_count) {
  for (int e = threadIdx.x; e < g.E; e += kThreads) s_count[e] = 0;
  __syncthreads();
  for (int p = p0 + threadIdx.x; p < p1; p += kAtOnce * kThreads) {
    int e[kAtOnce], r[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) e[i] = p + i * kThreads < p1 ? g.ids[p + i * kThreads] : -1;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) r[i] = e[i] >= 0 && e[i] < g.E ? atomicAdd(&s_count[e[i]], 1) : 0;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (p + i * kThreads < p1) g.rank[p + i * kThreads] = r[i];
  }
  __syncthreads();
}

// From the experts' counts: first places and tiles (written where `write`);
// then the list entries of pairs [p0, p1), whose run has s_before[e] pairs of
// expert e before it (null: none).
__device__ __forceinline__ void place_pairs(const GroupArgs& g, int p0, int p1, bool write, const int* s_count,
                                            const int* s_before, int* s_first, int* s_tile) {
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid < 64) {  // prefix sums of pairs and tiles, E / 64 experts per lane
    const int per = (g.E + 63) / 64, e0 = min(lane * per, g.E), e1 = min(e0 + per, g.E);
    int pairs = 0, nt = 0;
    for (int e = e0; e < e1; ++e) {
      pairs += s_count[e];
      nt += (s_count[e] + g.bm - 1) / g.bm;
    }
    int ps = pairs, ts = nt;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int a = __shfl_up(ps, d), b = __shfl_up(ts, d);
      if (lane >= d) {
        ps += a;
        ts += b;
      }
    }
    if (write && lane == 63) g.ntiles[0] = ts;
    ps -= pairs;
    ts -= nt;
    for (int e = e0; e < e1; ++e) {
      s_first[e] = ps;
      s_tile[e] = ts;
      ps += s_count[e];
      ts += (s_count[e] + g.bm - 1) / g.bm;
    }
  }
  __syncthreads();
  if (write)
    for (int e = tid >> 6; e < g.E; e += kWaves) {
      const int c = s_count[e], n = (c + g.bm - 1) / g.bm;
      for (int i = lane; i < n; i += 64)
        g.tiles[s_tile[e] + i] = RowTile{e, s_first[e] + i * g.bm, min(g.bm, c - i * g.bm), i | (n << 16)};
    }
  for (int p = p0 + tid; p < p1; p += kAtOnce * kThreads) {
    int e[kAtOnce], r[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int q = p + i * kThreads;
      e[i] = q < p1 ? g.ids[q] : -1;
      r[i] = q < p1 ? g.rank[q] : 0;
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (e[i] >= 0 && e[i] < g.E)
        g.list[s_first[e[i]] + (s_before ? s_before[e[i]] : 0) + r[i]] = p + i * kThreads;
  }
}

template <int ACT>
__global__ void __launch_bounds__(kThreads)
group_kernel(const void* __restrict__ x, int K, int8_t* __restrict__ qa, float* __restrict__ sa, GroupArgs g) {
  __shared__ float red[kWaves];
  __shared__ int s_count[kMaxExperts], s_first[kMaxExperts], s_tile[kMaxExperts];
  if ((int)blockIdx.x >= g.counters) {
    const int64_t m = blockIdx.x - g.counters;
    quantise_row<ACT, kThreads>(static_cast<const uint8_t*>(x) + m * K * RawRow<ACT>::kBytes, K, qa + m * K,
                                sa + m, red);
    return;
  }
  const int b = blockIdx.x, per = (g.P + g.counters - 1) / g.counters;
  const int p0 = min(b * per, g.P), p1 = min(p0 + per, g.P);
  count_pairs(g, p0, p1, s_count);
  if (g.counters == 1) {
    place_pairs(g, p0, p1, true, s_count, nullptr, s_first, s_tile);
  } else {
    for (int e = threadIdx.x; e < g.E; e += kThreads) g.counts[b * g.E + e] = s_count[e];
  }
}

__global__ void __launch_bounds__(kThreads) place_kernel(GroupArgs g) {
  __shared__ int s_count[kMaxExperts], s_before[kMaxExperts], s_first[kMaxExperts], s_tile[kMaxExperts];
  const int b = blockIdx.x, per = (g.P + g.counters - 1) / g.counters;
  const int p0 = min(b * per, g.P), p1 = min(p0 + per, g.P);
  for (int e = threadIdx.x; e < g.E; e += kThreads) {
    int all = 0, before = 0;
#pragma unroll 8
    for (int c = 0; c < g.counters; ++c) {
      const int v = g.counts[c * g.E + e];
      all += v;
      before += c < b ? v : 0;
    }
    s_count[e] = all;
    s_before[e] = before;
  }
  __syncthreads();
  place_pairs(g, p0, p1, b == 0, s_count, s_before, s_first, s_tile);
}

// ----------------------------------------------- quantisation of h rows
//
// One wavefront per pair, its row of at most 64 * 8 * kRowHeld values in
// registers (w4a8_quant_act's rule); slots of experts held elsewhere are
// skipped.  24576 rows of 1280: 18 us, against 36 with a workgroup per row.
constexpr int kRowHeld = 4;
__global__ void __launch_bounds__(kThreads)
quant_pairs_kernel(const uint16_t* __restrict__ h, const int* __restrict__ ids, int64_t P, int E, int I,
                   int8_t* __restrict__ hq, float* __restrict__ hs) {
  const int lane = threadIdx.x & 63, nch = I / 8;
  const int64_t p = (int64_t)blockIdx.x * kWaves + uniform(threadIdx.x >> 6);
  if (p >= P) return;
  const int e = uniform(ids[p]);
  if (e < 0 || e >= E) return;
  const uint8_t* row = reinterpret_cast<const uint8_t*>(h + p * I);
  v4u_rows raw[kRowHeld][1];
#pragma unroll
  for (int i = 0; i < kRowHeld; ++i)
    if (lane + 64 * i < nch) RawRow<kRawBf16>::load(row, lane + 64 * i, raw[i]);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kRowHeld; ++i)
    if (lane + 64 * i < nch) {
      float v[8];
      RawRow<kRawBf16>::widen(raw[i], v);
#pragma unroll
      for (int q = 0; q < 8; ++q) amax = fmaxf(amax, fabsf(v[q]));
    }
  amax = wave_max64(amax);
  const float scale = amax / 127.0f, inv = 1.0f / scale;
  if (lane == 0) hs[p] = scale;
#pragma unroll
  for (int i = 0; i < kRowHeld; ++i)
    if (lane + 64 * i < nch) {
      float v[8];
      RawRow<kRawBf16>::widen(raw[i], v);
      *reinterpret_cast<uint2*>(hq + p * I + 8 * (lane + 64 * i)) =
          quant8_codes(v, scale, inv);
    }
}

// ------------------------------------------------- down, single tokens
//
// y[m] = sum over the token's slots of weight * (h's codes x the expert's
// down weight): each wavefront takes the slots wave, wave + 8, ... of one
// 16-channel block, quantises that slot's h row itself and streams the
// block's units (all groups, D in flight); the slots are summed in slot
// order through LDS.  One launch, no partial sums in memory.
__global__ void __launch_bounds__(kThreads)
down_token_kernel(RowsArgs a, int k) {
  constexpr int D = 8;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // [wavefronts][K] codes
  __shared__ float s_part[kWaves][16];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r16 = lane & 15, j = lane >> 4;
  const int64_t m = blockIdx.y;
  const int nb = blockIdx.x, G = a.K / kGroup, nch = a.K / 8;
  uint8_t* q = smem + wave * a.K;
  float total = 0.0f;
  for (int s0 = 0; s0 < k; s0 += kWaves) {
    const int slot = s0 + wave;
    // the slot's h row goes out beside its expert's id, ahead of the weights:
    // it is quantised while they arrive
    const int64_t p = m * k + min(slot, k - 1);
    const uint8_t* hr = reinterpret_cast<const uint8_t*>(a.x) + p * a.K * 2;
    const int ev = a.ids[p];
    v4u_rows held[kRowHeld][1];
#pragma unroll
    for (int i = 0; i < kRowHeld; ++i)
      if (lane + 64 * i < nch) RawRow<kRawBf16>::load(hr, lane + 64 * i, held[i]);
    __builtin_amdgcn_sched_barrier(0);
    const int e = slot < k ? uniform(ev) : -1;
    float v = 0.0f;
    if (e >= 0 && e < a.n_experts) {
      const int64_t b0 = ((int64_t)e * a.nbe + nb) * G;
      const __amdgpu_buffer_rsrc_t rc = rsrc_of(a.codes + b0 * kBlockBytes, (int64_t)G * kBlockBytes);
      const __amdgpu_buffer_rsrc_t rs = rsrc_of(a.scales + b0 * 16, (int64_t)G * 64);
      const __amdgpu_buffer_rsrc_t rz = rsrc_of(a.zeros + b0 * kZeroBlockBytes, (int64_t)G * kZeroBlockBytes);
      v4u_rows d[D];
      float sc[D];
      uint32_t z[D];
      auto load = [&](int i, int t) __attribute__((always_inline)) {
        t = min(t, G);  // past the run: no memory request, zeros
        d[i] = __builtin_amdgcn_raw_buffer_load_b128(rc, 16 * lane, (unsigned)uniform(t * kBlockBytes),
                                                     kNontemporal);
        sc[i] = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(rs, 4 * r16, (unsigned)uniform(t * 64), 0));
        z[i] = __builtin_amdgcn_raw_buffer_load_b8(rz, r16 >> 1, (unsigned)uniform(t * kZeroBlockBytes), 0);
      };
#pragma unroll
      for (int i = 0; i < D; ++i) load(i, i);
      __builtin_amdgcn_sched_barrier(0);
      float amax = 0.0f;
      auto most = [&](const v4u_rows* raw) __attribute__((always_inline)) {
        float t[8];
        RawRow<kRawBf16>::widen(raw, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(t[i]));
      };
#pragma unroll
      for (int i = 0; i < kRowHeld; ++i)
        if (lane + 64 * i < nch) most(held[i]);
      for (int ch = lane + 64 * kRowHeld; ch < nch; ch += 64) {
        v4u_rows raw[1];
        RawRow<kRawBf16>::load(hr, ch, raw);
        most(raw);
      }
      amax = wave_max64(amax);
      const float scale = amax / 127.0f, inv = 1.0f / scale;
      auto put = [&](int ch, const v4u_rows* raw) __attribute__((always_inline)) {
        float t[8];
        RawRow<kRawBf16>::widen(raw, t);
        *reinterpret_cast<uint2*>(q + 8 * ch) =
            quant8_codes(t, scale, inv);
      };
#pragma unroll
      for (int i = 0; i < kRowHeld; ++i)
        if (lane + 64 * i < nch) put(lane + 64 * i, held[i]);
      for (int ch = lane + 64 * kRowHeld; ch < nch; ch += 64) {
        v4u_rows raw[1];
        RawRow<kRawBf16>::load(hr, ch, raw);
        put(ch, raw);
      }
      // the wavefront's own LDS writes, read by its other lanes
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      for (int tb = 0; tb < G; tb += D) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
          if (tb + i < G) {
            v4i lo, hi;
            unpack_unit(d[i], ((z[i] >> (4 * (r16 & 1))) & 0xFu) * 0x01010101u, lo, hi);
            const uint8_t* frag = q + (tb + i) * kGroup + 16 * j;  // every row the same
            v4i c = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const v4i*>(frag), lo,
                                                          kBiasSeed, 0, 0, 0);
            c = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const v4i*>(frag + 64), hi, c,
                                                      0, 0, 0);
            v += sc[i] * unbias(c[0]);
          }
          load(i, tb + i + D);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      v *= scale * a.pw[p];
    }
    if (lane < 16) s_part[wave][lane] = v;
    __syncthreads();
    if (threadIdx.x < 16) {
      const int n = min(kWaves, k - s0);
      for (int i = 0; i < n; ++i) total += s_part[i][threadIdx.x];
    }
    __syncthreads();
  }
  if (threadIdx.x < 16) a.y[m * (16 * a.nbe) + 16 * nb + threadIdx.x] = f32_to_bf16_rne(total);
}

// ------------------------------------------------------- sum over experts
//
// y[m][n] = bf16(sum_j parts[m k + j][n]) over the slots held here, in slot
// order; eight channels per thread.
__global__ void __launch_bounds__(256)
combine_kernel(const float* __restrict__ parts, const int* __restrict__ ids, int64_t M, int k, int E,
               int N, uint16_t* __restrict__ y) {
  const int per = N / 8;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= M * per) return;
  const int64_t m = t / per;
  const int n = (int)(t - m * per) * 8;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  constexpr int S = 4;  // slots whose loads go out together
  for (int s0 = 0; s0 < k; s0 += S) {
    float4 a[S], b[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int64_t q = m * k + s0 + i;
      const int e = s0 + i < k ? ids[q] : -1;
      a[i] = b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e >= 0 && e < E) {
        const float4* p = reinterpret_cast<const float4*>(parts + q * N + n);
        a[i] = p[0];
        b[i] = p[1];
      }
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      v[0] += a[i].x; v[1] += a[i].y; v[2] += a[i].z; v[3] += a[i].w;
      v[4] += b[i].x; v[5] += b[i].y; v[6] += b[i].z; v[7] += b[i].w;
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = (uint32_t)f32_to_bf16_rne(v[2 * i]) | ((uint32_t)f32_to_bf16_rne(v[2 * i + 1]) << 16);
  *reinterpret_cast<uint4*>(y + m * N + n) = make_uint4(o[0], o[1], o[2], o[3]);
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// Rows a tile of the planned kernels holds: the smallest of 16, 32, 64 and
// 256 that holds an expert's even share of the pairs with room to spare; of
// 64 and 256 past that the one that takes less time by what they measured a
// group of inputs: a round of 256-row tiles 3.0 us, 64-row ones 1.3 us where
// they lie one to a compute unit and that much more for every further one
// (768 tokens of 4, 5 experts, 3200 -> 2 x 256: 65 us against 92 on 256 rows;
// 4096 tokens, 64 experts, 3584 -> 2 x 1280 stay on 256).
static int tile_rows(int64_t P, int E, int64_t I, int64_t K) {
  const double share = (double)P / E;
  if (share <= 96) return share <= 10 ? 16 : share <= 22 ? 32 : 64;
  const double cus = device_cus(), part = E / 2.0;  // an expert's last tile is half full
  const double G = K / kGroup, GI = I / kGroup, up = I / 128.0, down = K / 256.0;
  auto rounds = [](double n) { return n <= 1 ? 1.0 : std::ceil(n); };
  const double big = P / 256.0 + part, small = P / 64.0 + part;
  const double tile = 3.0 * (G * rounds(big * up / cus) + GI * rounds(big * down / cus));
  const double run = 1.3 * (G * std::max(1.0, small * up / cus) + GI * std::max(1.0, small * down / cus));
  return run < tile ? 64 : kTileRows;
}

// Single tokens (a few pairs) skip the grouping: each pair is a tile.
static bool direct(int64_t P, int64_t I, int64_t K) {
  return P <= 16 && I <= 4096 && K <= 16384;
}

MoePlan moe_plan(int64_t M, int k, int E, int64_t I, int64_t K) {
  MoePlan p;
  // tokens of one pass: 32-bit offsets into the codes, tile counts of 16 bits
  int64_t mc = M;
  const int64_t most = (int64_t)1 << 19;
  if (mc > most / k) mc = most / k;
  const int64_t rows = kPrefillMaxBytes / (K > I * k ? K : I * k);
  if (mc > rows) mc = rows;
  p.tokens = mc;
  if (mc < 1) return p;
  const int64_t P = mc * k;
  p.direct = direct(M * k, I, K);
  p.bm = tile_rows(P, E, I, K);
  const int64_t G = K / kGroup, GI = I / kGroup;
  const int staged = p.bm < kTileRows ? staged_groups(p.bm / 16) : 0;
  p.raw = !p.direct && p.bm == 16 && GI <= 32;  // (few rows share a tile)
  p.up = p.direct ? kTokenPath : p.bm == kTileRows ? kTilePath : G <= staged ? kStreamPath : kRunPath;
  p.down = p.direct ? kTokenPath : p.bm == kTileRows ? kTilePath : p.raw || GI <= staged ? kStreamPath : kRunPath;
  if (p.direct) p.bm = 1;
  // (room for tiles of the least height, so that the workspace of a batch
  // serves every smaller one, whatever height that takes)
  const int64_t max_tiles = P / 16 + (E < P ? E : P);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += up256(bytes);
    return o;
  };
  p.h = take(P * I * 2);
  if (!p.direct) {
    p.qa = take(mc * K);
    p.sa = take(mc * 4);
    p.count = take(4);
    p.tiles = take(max_tiles * (int64_t)sizeof(RowTile));
    p.list = take(P * 4);
    p.rank = take(P * 4);
    p.counts = take((int64_t)counters_of(P) * E * 4);
    p.hq = take(P * I);
    p.hs = take(P * 4);
    p.parts = take(P * K * 4);
  }
  p.bytes = at;
  return p;
}

// Runs of about 24 units per wavefront, but columns shared out while the
// tiles that can be expected leave compute units without a workgroup (644
// tokens of 7, 15 experts, 128 -> 384: 36 us against 61).
int down_columns(const MoePlan& p, int64_t P, int E, int64_t I, int64_t K) {
  const int64_t GI = I / kGroup, cols = K / 16;
  const int64_t tiles = P / p.bm + (E < P ? E : P) / 2 + 1;
  const int64_t most = cols * tiles / (8 * (int64_t)device_cus());
  const int64_t n = (24 + GI - 1) / GI;
  return (int)(n <= most ? n : most > 1 ? most : 1);
}

static hipError_t moe_direct(const MoeArgs& m, const MoePlan& p, hipStream_t st) {
  uint16_t* h = reinterpret_cast<uint16_t*>(m.ws + p.h);
  RowsArgs a{};
  a.x = m.x;
  a.codes = m.up.codes;
  a.zeros = m.up.zeros;
  a.scales = m.up.scales;
  a.ids = m.ids;
  a.n_experts = m.E;
  a.kind = kDirect;
  a.src_rows = m.M;
  a.K = (int)m.K;
  a.nbe = (int)(2 * m.I / 16);
  a.div = m.k;
  a.cols = (int)(m.I / 16);
  a.kw = 3;
  a.ncol = 1;
  a.strips = a.cols;
  a.sg = (int)(m.K / kGroup);
  a.h = h;
  hipError_t e = launch_rows_stream(a, 1, true, m.x_dtype == 0 ? kRawBf16 : kRawF32, kSwiglu,
                                    m.M * m.k * a.strips, 1, st);
  if (e != hipSuccess) return e;
  RowsArgs d{};
  d.x = h;
  d.codes = m.down.codes;
  d.zeros = m.down.zeros;
  d.scales = m.down.scales;
  d.ids = m.ids;
  d.n_experts = m.E;
  d.K = (int)m.I;
  d.nbe = (int)(m.K / 16);
  d.pw = m.weights;
  d.y = m.y;
  hipLaunchKernelGGL(down_token_kernel, dim3((unsigned)d.nbe, (unsigned)m.M), dim3(kThreads),
                     (size_t)kWaves * m.I, st, d, m.k);
  return hipGetLastError();
}

hipError_t launch_moe(const MoeArgs& m, const MoePlan& p, hipStream_t st) {
  if (p.direct) return moe_direct(m, p, st);
  const int64_t P = m.M * m.k;
  int8_t* qa = reinterpret_cast<int8_t*>(m.ws + p.qa);
  float* sa = reinterpret_cast<float*>(m.ws + p.sa);
  int* count = reinterpret_cast<int*>(m.ws + p.count);
  RowTile* tiles = reinterpret_cast<RowTile*>(m.ws + p.tiles);
  int* list = reinterpret_cast<int*>(m.ws + p.list);
  int* rank = reinterpret_cast<int*>(m.ws + p.rank);
  uint16_t* h = reinterpret_cast<uint16_t*>(m.ws + p.h);
  int8_t* hq = reinterpret_cast<int8_t*>(m.ws + p.hq);
  float* hs = reinterpret_cast<float*>(m.ws + p.hs);
  float* parts = reinterpret_cast<float*>(m.ws + p.parts);
  const int64_t max_tiles = P / p.bm + (m.E < P ? m.E : P);

  const GroupArgs g{m.ids, (int)P, m.E, p.bm, counters_of(P), count, tiles, list, rank,
                    reinterpret_cast<int*>(m.ws + p.counts)};
  const dim3 blocks((unsigned)(g.counters + m.M));
  if (m.x_dtype == 0)
    hipLaunchKernelGGL((group_kernel<kRawBf16>), blocks, dim3(kThreads), 0, st, m.x, (int)m.K, qa, sa, g);
  else
    hipLaunchKernelGGL((group_kernel<kRawF32>), blocks, dim3(kThreads), 0, st, m.x, (int)m.K, qa, sa, g);
  if (g.counters > 1) hipLaunchKernelGGL(place_kernel, dim3(g.counters), dim3(kThreads), 0, st, g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  const int mt = p.bm / 16;
  RowsArgs a{};
  a.qa = qa;
  a.sa = sa;
  a.codes = m.up.codes;
  a.zeros = m.up.zeros;
  a.scales = m.up.scales;
  a.ntiles = count;
  a.tiles = tiles;
  a.list = list;
  a.ids = m.ids;
  a.n_experts = m.E;
  a.kind = kPlanned;
  a.src_rows = m.M;
  a.K = (int)m.K;
  a.nbe = (int)(2 * m.I / 16);
  a.div = m.k;
  a.cols = (int)(m.I / 16);
  a.h = h;
  if (p.up == kTilePath) {
    a.strips = a.cols / 8;
    e = launch_rows_tile(a, kSwiglu, max_tiles * a.strips, 1, st);
  } else {
    a.kw = 0;
    a.ncol = 1;
    a.strips = (a.cols + 7) / 8;
    a.sg = (int)(m.K / kGroup);
    e = p.up == kStreamPath
            ? launch_rows_stream(a, mt, false, kCodes, kSwiglu, max_tiles * a.strips, 1, st)
            : launch_rows_run(a, mt, kSwiglu, max_tiles * a.strips, 1, st);
  }
  if (e != hipSuccess) return e;

  if (!p.raw) {
    if (m.I <= 64 * 8 * kRowHeld) {
      hipLaunchKernelGGL(quant_pairs_kernel, dim3((unsigned)((P + kWaves - 1) / kWaves)), dim3(kThreads), 0, st,
                         h, m.ids, P, m.E, (int)m.I, hq, hs);
      e = hipGetLastError();
    } else {
      e = launch_quant(h, 0, P, m.I, hq, hs, st);
    }
    if (e != hipSuccess) return e;
  }
  RowsArgs d = a;
  d.qa = hq;
  d.sa = hs;
  d.x = h;
  d.codes = m.down.codes;
  d.zeros = m.down.zeros;
  d.scales = m.down.scales;
  d.src_rows = P;
  d.K = (int)m.I;
  d.nbe = (int)(m.K / 16);
  d.div = 1;
  d.cols = d.nbe;
  d.pw = m.weights;
  d.h = nullptr;
  d.parts = parts;
  if (p.down == kTilePath) {
    d.strips = (d.nbe + 15) / 16;
    e = launch_rows_tile(d, kParts, max_tiles * d.strips, 1, st);
  } else {
    d.sg = (int)(m.I / kGroup);
    d.kw = 0;
    d.ncol = down_columns(p, P, m.E, m.I, m.K);
    const int per = 8 * d.ncol;
    d.strips = (d.cols + per - 1) / per;
    e = p.down == kStreamPath
            ? launch_rows_stream(d, mt, false, p.raw ? kRawBf16 : kCodes, kParts, max_tiles * d.strips, 1, st)
            : launch_rows_run(d, mt, kParts, max_tiles * d.strips, 1, st);
  }
  if (e != hipSuccess) return e;
  const int64_t total = m.M * (m.K / 8);
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, parts,
                     m.ids, m.M, m.k, m.E, (int)m.K, m.y);
  return hipGetLastError();
}

}  // namespace w4a8
