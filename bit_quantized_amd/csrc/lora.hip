// A shared W4A8 projection with a low-rank adapter chosen per row:
//   y[m] = bf16( sa[m] * sum_g s P  +  scale[l] * (x[m] A[l]^T) B[l]^T ),  l = ids[m].
//
// The shared product runs on the row-tile kernels (rows.hip), a single row's
// on the GEMV (gemv.hip); this file has the adapters' first half x A^T, and
// the reduction that adds the second half where the shared product was split
// over K.  Past 64 rows everything takes the rows in the order of their
// adapters, so that 16 neighbours share one or two of them: 1024 rows of 16
// adapters of rank 128, mixed, 3584 -> 18944: 194 us, against 1005 in the
// order of the call.
#include "lora.h"

#include <algorithm>

namespace w4a8 {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;

// ------------------------------------ rows by adapter, beside quantisation
//
// Workgroup 0 writes the rows in the order of their adapters (of id mod
// kBuckets: adapters that share a bucket mix, which costs time only; rows
// without one come last), so that the 16-row fragments of the kernels that
// follow meet few adapters.  The others quantise a row each.  The place of a
// row within its bucket follows LDS atomics and may differ between calls; no
// output depends on it (rows.h).
constexpr int kBuckets = 1024;
template <int ACT>
__global__ void __launch_bounds__(kThreads)
order_kernel(LoraArgs a, int8_t* __restrict__ qa, float* __restrict__ sa, int* __restrict__ order) {
  __shared__ float s_max[kWaves];
  __shared__ int s_next[kBuckets + 1];
  const int tid = threadIdx.x, lane = tid & 63, K = (int)a.K;
  if (blockIdx.x > 0) {
    const int64_t m = blockIdx.x - 1;
    quantise_row<ACT, kThreads>(static_cast<const uint8_t*>(a.x) + m * K * RawRow<ACT>::kBytes, K, qa + m * K,
                                sa + m, s_max);
    return;
  }
  auto bucket = [&](int m) __attribute__((always_inline)) {
    const int id = a.ids[m];
    return id >= 0 && id < a.L ? id % kBuckets : kBuckets;
  };
  for (int b = tid; b <= kBuckets; b += kThreads) s_next[b] = 0;
  __syncthreads();
  for (int m = tid; m < a.M; m += kThreads) atomicAdd(&s_next[bucket(m)], 1);
  __syncthreads();
  if (tid < 64) {  // counts to first places, kBuckets / 64 per lane
    constexpr int per = kBuckets / 64;
    int sum = 0, c[per];
#pragma unroll
    for (int i = 0; i < per; ++i) {
      c[i] = s_next[lane * per + i];
      sum += c[i];
    }
    int at = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(at, d);
      if (lane >= d) at += v;
    }
    if (lane == 63) s_next[kBuckets] = at;
    at -= sum;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      s_next[lane * per + i] = at;
      at += c[i];
    }
  }
  __syncthreads();
  for (int m = tid; m < a.M; m += kThreads) order[atomicAdd(&s_next[bucket(m)], 1)] = m;
}

// Steps of 32 inputs whose loads a wavefront has in flight, by the rank.
constexpr int down_steps(int R) { return R > 64 ? 2 : 4; }

// ----------------------------------------- quantisation and x A^T together
//
// Workgroups [0, qrows) quantise one row each.  The others take a fragment of
// 16 rows (in `order`, where there is one), every `slots`-th of the distinct
// adapters among them, and a K slice, which the wavefronts share: for an adapter, v_mfma_f32_16x16x32_bf16 of the
// 16 rows (A operand) against its rows of A (B operand), float sums, and only
// the rows that use this adapter are written.  Many rows that use one adapter
// read it once; a row alone with its adapter wastes matrix-core slots, not
// memory traffic, which is what bounds this step.  bf16 activations are exact
// operands; float ones go in as two bf16 parts (16 significant bits, below
// the bf16 weights' own 8).  33 rows with 20 adapters of rank 64, 18944
// inputs: 17.6 us for 67 MB.
template <int ACT, int RT>
__global__ void __launch_bounds__(kThreads)
adapter_down_kernel(LoraArgs a, int8_t* __restrict__ qa, float* __restrict__ sa,
                    const int* __restrict__ order, float* __restrict__ hx, int qrows, int slots,
                    int slices) {
  constexpr int U = down_steps(16 * RT);
  constexpr bool F32 = ACT == kRawF32;
  __shared__ float s_red[kWaves][RT * 4][64];
  __shared__ float s_max[kWaves];
  __shared__ int s_row[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const uint8_t* x = static_cast<const uint8_t*>(a.x);
  const int K = (int)a.K;
  if ((int)blockIdx.x < qrows) {
    const int64_t m = blockIdx.x;
    quantise_row<ACT, kThreads>(x + m * K * RawRow<ACT>::kBytes, K, qa + m * K, sa + m, s_max);
    return;
  }
  const int b = (int)blockIdx.x - qrows;
  const int slice = b % slices, slot = b / slices % slots;
  const int64_t m0 = (int64_t)(b / slices / slots) * 16;
  const int r16 = lane & 15, j = lane >> 4;
  const int64_t m = m0 + r16 < a.M ? order ? order[m0 + r16] : m0 + r16 : -1;
  const int id = m >= 0 ? a.ids[m] : -1;
  if (tid < 16) s_row[tid] = (int)m;  // (read after a barrier)
  const bool has = id >= 0 && id < a.L;
  const int steps = K / 32;
  const int s0 = steps * slice / slices, s1 = steps * (slice + 1) / slices;
  const int t0 = s0 + (s1 - s0) * wave / kWaves, t1 = s0 + (s1 - s0) * (wave + 1) / kWaves;
  const uint8_t* xrow = x + (m >= 0 ? m : 0) * K * RawRow<ACT>::kBytes;
  uint64_t todo = __ballot(has) & 0xFFFFull;
  for (int at = 0; todo; ++at) {
    const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(has && id == l) & 0xFFFFull;
    todo &= ~mine;
    if (at % slots != slot) continue;
    const uint16_t* arow[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
      arow[t] = a.A + ((int64_t)l * a.R + min(16 * t + r16, a.R - 1)) * K;
    v4f_rows acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = v4f_rows{0.f, 0.f, 0.f, 0.f};
    for (int t = t0; t < t1; t += U) {
      v4u_rows xr[U][RawRow<ACT>::kLoads];
      v4i br[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u >= t1) break;
        const int k = 32 * (t + u) + 8 * j;
        RawRow<ACT>::load(xrow, k / 8, xr[u]);
#pragma unroll
        for (int q = 0; q < RT; ++q) br[u][q] = *reinterpret_cast<const v4i*>(arow[q] + k);
      }
      __builtin_amdgcn_sched_barrier(0);  // all of them in flight
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u >= t1) break;
        v4i hi, lo;
        if constexpr (F32) {
          float v[8];
          RawRow<ACT>::widen(xr[u], v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h0, h1, l0, l1;
            bf16_parts(v[2 * e], h0, l0);
            bf16_parts(v[2 * e + 1], h1, l1);
            hi[e] = (int)(h0 | (h1 << 16));
            lo[e] = (int)(l0 | (l1 << 16));
          }
        } else {
          hi = __builtin_bit_cast(v4i, xr[u][0]);
        }
#pragma unroll
        for (int q = 0; q < RT; ++q) {
          const v8bf_rows bv = __builtin_bit_cast(v8bf_rows, br[u][q]);
          acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_rows, hi), bv,
                                                           acc[q], 0, 0, 0);
          if constexpr (F32)
            acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_rows, lo), bv,
                                                             acc[q], 0, 0, 0);
        }
      }
    }
    // the wavefronts' sums, in order; one adapter after another reuses the LDS
    __syncthreads();
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int r = 0; r < 4; ++r) s_red[wave][q * 4 + r][lane] = acc[q][r];
    __syncthreads();
    for (int o = tid; o < RT * 256; o += kThreads) {
      const int q = o >> 8, r = (o >> 6) & 3, ln = o & 63;
      const int row = 4 * (ln >> 4) + r, rank = 16 * q + (ln & 15);
      if (!((mine >> row) & 1) || rank >= a.R) continue;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += s_red[w][q * 4 + r][ln];
      hx[((int64_t)slice * a.M + s_row[row]) * a.R + rank] = v;
    }
  }
}

// --------------------------------- K slices summed, adapter product added
//
// Few rows: one channel of one row per thread.  The slices' sums and the
// first ranks of B are on their way before the row's x A^T is summed, so a
// workgroup waits for memory about once.
__global__ void __launch_bounds__(256)
adapt_reduce_kernel(const float* __restrict__ parts, int ksplit, const float* __restrict__ sa,
                    int64_t M, int N, AdaptArgs ad, uint16_t* __restrict__ y) {
  __shared__ float s_hx[kMaxRank];
  const int64_t m = blockIdx.y;
  const int n = blockIdx.x * 256 + threadIdx.x;
  const int id = ad.ids[m];
  const bool has = id >= 0 && id < ad.L;
  float v = 0.0f;
  if (n < N) {
    const float* p = parts + m * N + n;
    const int64_t step = M * N;
    for (int k = 0; k < ksplit; k += 8) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = k + i < ksplit ? p[(k + i) * step] : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v += t[i];
    }
    v *= sa[m];
  }
  if (!has) {
    if (n < N) y[m * N + n] = f32_to_bf16_rne(v);
    return;
  }
  const uint16_t* brow = ad.B + ((int64_t)id * N + min(n, N - 1)) * ad.R;
  AdapterRow b;
  b.fetch(brow, 0, ad.R);
  for (int r = threadIdx.x; r < ad.R; r += 256) s_hx[r] = adapter_sum(ad, M, m, r, ad.scale[id]);
  __syncthreads();
  if (n < N) y[m * N + n] = f32_to_bf16_rne(v + b.dot(s_hx, brow, ad.R));
}

// The scaled sums x A^T of all rows as two bf16 planes [M][R], operands of the
// matrix cores: hi the rounded sums, lo the rounded rest (16 significant
// bits together).  Eight ranks per thread.
__global__ void __launch_bounds__(256)
adapter_parts_kernel(AdaptArgs ad, int64_t M, uint16_t* __restrict__ hi, uint16_t* __restrict__ lo) {
  const int per = ad.R / 8;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= M * per) return;
  const int64_t m = t / per;
  const int id = ad.ids[m];
  if (id < 0 || id >= ad.L) return;  // (never read)
  const float s = ad.scale[id];
  const v4f_rows* p = reinterpret_cast<const v4f_rows*>(ad.hx + t * 8);
  const int64_t step = M * ad.R / 4;
  v4f_rows a = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < ad.slices; ++k) {
    a += p[k * step];
    b += p[k * step + 1];
  }
  v4i h, l;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float v0 = s * (e < 2 ? a[2 * e] : b[2 * e - 4]), v1 = s * (e < 2 ? a[2 * e + 1] : b[2 * e - 3]);
    uint32_t h0, h1, l0, l1;
    bf16_parts(v0, h0, l0);
    bf16_parts(v1, h1, l1);
    h[e] = (int)(h0 | (h1 << 16));
    l[e] = (int)(l0 | (l1 << 16));
  }
  *reinterpret_cast<v4i*>(hi + t * 8) = h;
  *reinterpret_cast<v4i*>(lo + t * 8) = l;
}

// Rows in the order of their adapters: 16 rows x 64 channels per workgroup, a
// block per wavefront in the result layout of the matrix cores (lane 16 j +
// c: rows 4 j .. + 3, channel c).  Per adapter among the rows the product of
// its rows' two parts with B is added to those rows only, so an adapter's B
// is read once per 16 rows (200 rows of rank 32, three slices of 18944
// channels: 14.6 us, 60 MB).
__global__ void __launch_bounds__(256)
adapt_reduce_sorted_kernel(const float* __restrict__ parts, int ksplit, const float* __restrict__ sa,
                           const int* __restrict__ order, int64_t M, int N, AdaptArgs ad,
                           uint16_t* __restrict__ y) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r16 = lane & 15, j = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  const int NB = N / 16, nb = blockIdx.x * 4 + wave;
  if (nb >= NB) return;
  const int mrow = m0 + r16 < M ? order[m0 + r16] : -1;
  int id = mrow >= 0 ? ad.ids[mrow] : -1;
  if (id >= ad.L) id = -1;
  const float own = mrow >= 0 ? sa[mrow] : 0.0f;
  int row[4];
  float acc[4], s[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    row[r] = __shfl(mrow, 4 * j + r);
    s[r] = __shfl(own, 4 * j + r);
    acc[r] = 0.0f;
  }
  const int64_t step = M * N;
  for (int k = 0; k < ksplit; k += 4) {
    float t[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        t[i][r] = row[r] >= 0 && k + i < ksplit ? parts[(k + i) * step + (int64_t)row[r] * N + 16 * nb + r16] : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] += t[i][r];
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) acc[r] *= s[r];
  const uint64_t present = __ballot(id >= 0) & 0xFFFFull;
  for (int r0 = 0; present && r0 < ad.R; r0 += 32) {
    const int rr = r0 + 8 * j;  // this lane's eight ranks
    const v4i zero = {0, 0, 0, 0};
    v4i hi = zero, lo = zero;
    if (id >= 0 && rr < ad.R) {
      hi = *reinterpret_cast<const v4i*>(ad.hi + (int64_t)mrow * ad.R + rr);
      lo = *reinterpret_cast<const v4i*>(ad.lo + (int64_t)mrow * ad.R + rr);
    }
    uint64_t todo = present;
    while (todo) {
      const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
      const uint64_t rows = __ballot(id == l) & 0xFFFFull;
      todo &= ~rows;
      v4i bv = zero;
      if (rr < ad.R)
        bv = *reinterpret_cast<const v4i*>(ad.B + (((int64_t)l * NB + nb) * 16 + r16) * ad.R + rr);
      v4f_rows c = {0.f, 0.f, 0.f, 0.f};
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_rows, id == l ? hi : zero),
                                                  __builtin_bit_cast(v8bf_rows, bv), c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_rows, id == l ? lo : zero),
                                                  __builtin_bit_cast(v8bf_rows, bv), c, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] += (rows >> (4 * j + r)) & 1 ? c[r] : 0.0f;
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (row[r] >= 0) y[(int64_t)row[r] * N + 16 * nb + r16] = f32_to_bf16_rne(acc[r]);
}

constexpr int64_t kMaxPassRows = (int64_t)1 << 20;
constexpr int64_t kSortBytes = (int64_t)64 << 20;
constexpr int64_t kMaxSlices = 16;

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

template <int ACT, int RT>
void down_launch(const LoraArgs& l, const LoraPlan& p, int8_t* qa, float* sa, const int* order, float* hx,
                 hipStream_t st) {
  const int qrows = p.gemv || order ? 0 : (int)l.M;  // (else quantised elsewhere)
  const int64_t blocks = qrows + (l.M + 15) / 16 * p.slots * p.slices;
  hipLaunchKernelGGL((adapter_down_kernel<ACT, RT>), dim3((unsigned)blocks), dim3(kThreads), 0, st, l, qa,
                     sa, order, hx, qrows, p.slots, p.slices);
}

template <int ACT>
void down_rank(const LoraArgs& l, const LoraPlan& p, int8_t* qa, float* sa, int* order, float* hx,
               hipStream_t st) {
  if (order)
    hipLaunchKernelGGL((order_kernel<ACT>), dim3((unsigned)(l.M + 1)), dim3(kThreads), 0, st, l, qa, sa, order);
  if (l.R <= 16)
    down_launch<ACT, 1>(l, p, qa, sa, order, hx, st);
  else if (l.R <= 32)
    down_launch<ACT, 2>(l, p, qa, sa, order, hx, st);
  else if (l.R <= 64)
    down_launch<ACT, 4>(l, p, qa, sa, order, hx, st);
  else
    down_launch<ACT, 8>(l, p, qa, sa, order, hx, st);
}

}  // namespace

LoraPlan lora_plan(int64_t M, int64_t N, int64_t K, int L, int R) {
  LoraPlan p;
  const int64_t cus = device_cus(), G = K / kGroup, cols = N / kBlockCols;
  // rows of one pass: 32-bit offsets into the codes, and a grid of at most
  // 2^32 threads for the step that has a workgroup per row
  int64_t mc = kPrefillMaxBytes / K;
  if (mc > kMaxPassRows) mc = kMaxPassRows;
  if (mc >= kTileRows) mc = mc / kTileRows * kTileRows;
  if (mc > M) mc = M;
  p.rows = mc;
  if (mc < 1) return p;
  bool few = false;
  if (M == 1 && K <= kGemvMaxK) {
    const GemvShape gs = gemv_shape(N, K);
    p.gemv = gemv_shape_ok(N, K, gs);
    if (p.gemv) p.ksplit = gs.ksplit;
  }
  if (p.gemv) {
    // (no tiles)
  } else if (mc <= 64) {
    p.mt = (int)((mc + 15) / 16);
    // one launch, whole K per workgroup and eight wavefronts to a column, where
    // the columns fit one round of workgroups and the rows' groups their LDS
    p.kw = mc <= 16 && cols <= cus && cols >= cus / 2 && G <= staged_groups(1) ? 3 : -1;
    if (p.kw < 0) {  // K slices: a workgroup per compute unit, two of them of 16 rows
      // (33 rows, 18944 -> 3584: 13.1 us against 18.3 with twice the slices)
      p.kw = 0;
      const int64_t strips = (cols + 7) / 8;
      int64_t ks = (p.mt == 1 ? 2 : 1) * cus / strips;
      if (ks > G / 4) ks = G / 4;
      p.ksplit = (int)(ks > 1 ? ks : 1);
    }
  } else {
    const int64_t tiles = (mc + kTileRows - 1) / kTileRows * ((N + kTileCols - 1) / kTileCols);
    int64_t ks = cus / tiles;
    if (ks > G / 4) ks = G / 4;
    p.ksplit = (int)(ks > 1 ? ks : 1);
    few = tiles < cus / 2;
  }
  const int64_t frags = (mc + 15) / 16;
  // (few rows: sorted where reading B once per row would cost more than the
  // two small launches; 64 rows of rank 64, 3584 -> 18944: 52 us against 63
  // with 16 adapters, but 83 against 74 with 64)
  p.sorted = mc > 64 || (mc > 16 && mc * N * R * 2 > kSortBytes);
  p.slots = (int)(p.sorted ? 1 : mc < 16 ? mc : 16);  // (sorted: few adapters to a fragment)
  if (p.slots > L) p.slots = L;
  // several rounds of workgroups while every wavefront gets a step; fewer
  // where the product's tiles sum the slices again for every strip
  int64_t sl = (p.sorted ? 2 : 4) * cus / (frags * p.slots), most = (K / 32 + kWaves - 1) / kWaves;
  if (sl > most) sl = most;
  if (sl > kMaxSlices) sl = kMaxSlices;
  p.slices = (int)(sl > 1 ? sl : 1);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += up256(bytes);
    return o;
  };
  p.qa = take(mc * K);
  p.sa = take(mc * 4);
  p.hx = take((int64_t)p.slices * mc * R * 4);
  if (p.sorted) {
    p.order = take(mc * 4);
    p.hi = take(mc * R * 2);
    p.lo = take(mc * R * 2);
  }
  // (the streaming kernels go through the sums unless a column is whole, few
  // tiles so that the adapters' part runs on more compute units than they)
  p.path = p.gemv ? kTokenPath
           : !p.mt ? kTilePath
           : p.kw == 0 && (G + p.ksplit - 1) / p.ksplit > staged_groups(p.mt) ? kRunPath
                                                                              : kStreamPath;
  const bool sums = p.ksplit > 1 || (p.mt && p.kw == 0) || few;
  if (sums) p.parts = take((int64_t)p.ksplit * mc * N * 4);
  else p.parts = -1;
  p.bytes = at;
  return p;
}

// Fewer rows can need more: their K slices are more.  The buffers of lora_plan
// at their largest over 1 .. M rows, in closed form; each is at least what any
// of those plans takes.
int64_t lora_workspace(int64_t M, int64_t N, int64_t K, int L, int R) {
  const LoraPlan p = lora_plan(M, N, K, L, R);
  const int64_t cus = device_cus(), m = p.rows, nt = (N + kTileCols - 1) / kTileCols;
  if (m < 1) return 0;
  // rows of float sums: ksplit times rows.  Up to 64 rows the K split changes
  // at 1, 16 and 64; past them a split product has at most cus / 2 tiles, and
  // ksplit times its tiles is at most cus.
  int64_t sums = 0;
  for (int64_t few : {(int64_t)1, (int64_t)16, (int64_t)64}) {
    const LoraPlan q = few < m ? lora_plan(few, N, K, L, R) : p;
    if (q.parts >= 0) sums = std::max(sums, q.ksplit * q.rows);
    if (few >= m) break;
  }
  if (m > 64 && 2 * nt <= cus) {
    const int64_t ks = std::max<int64_t>(1, std::min(cus / nt, K / kGroup / 4));
    sums = std::max(sums, std::min(ks * m, kTileRows * cus / nt));
  }
  // slices of x A^T: at most kMaxSlices, and 4 cus over all 16-row fragments
  // where there is more than one
  const int64_t hx = std::max(m, std::min(kMaxSlices * m, 16 * 4 * cus));
  int64_t bytes = up256(m * K) + up256(m * 4) + up256(hx * R * 4) + up256(sums * N * 4);
  if (p.sorted) bytes += up256(m * 4) + 2 * up256(m * R * 2);
  return bytes;
}

hipError_t launch_lora(const LoraArgs& l, const LoraPlan& p, hipStream_t st) {
  int8_t* qa = reinterpret_cast<int8_t*>(l.ws + p.qa);
  float* sa = reinterpret_cast<float*>(l.ws + p.sa);
  float* hx = reinterpret_cast<float*>(l.ws + p.hx);
  float* parts = p.parts >= 0 ? reinterpret_cast<float*>(l.ws + p.parts) : nullptr;
  int* order = p.sorted ? reinterpret_cast<int*>(l.ws + p.order) : nullptr;
  if (l.x_dtype == 0)
    down_rank<kRawBf16>(l, p, qa, sa, order, hx, st);
  else
    down_rank<kRawF32>(l, p, qa, sa, order, hx, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  AdaptArgs ad{hx, nullptr, nullptr, l.B, l.scale, l.ids, p.slices, l.L, l.R};
  if (order) {
    uint16_t* hi = reinterpret_cast<uint16_t*>(l.ws + p.hi);
    uint16_t* lo = reinterpret_cast<uint16_t*>(l.ws + p.lo);
    ad.hi = hi;
    ad.lo = lo;
    const int64_t total = l.M * (l.R / 8);
    hipLaunchKernelGGL(adapter_parts_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, ad, l.M,
                       hi, lo);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  RowsArgs a{};
  a.qa = qa;
  a.sa = sa;
  a.codes = l.w.codes;
  a.zeros = l.w.zeros;
  a.scales = l.w.scales;
  a.kind = kDense;
  a.list = p.mt ? nullptr : order;
  a.M = l.M;
  a.src_rows = l.M;
  a.K = (int)l.K;
  a.nbe = (int)(l.N / 16);
  a.n_experts = 1;
  a.div = 1;
  a.cols = a.nbe;
  a.parts = parts;
  a.y = l.y;
  a.ad = ad;
  const int G = (int)(l.K / kGroup);
  if (p.gemv) {
    GemmArgs g{};
    g.x = l.x;
    g.x_dtype = l.x_dtype;
    g.w = l.w;
    g.M = 1;
    g.N = l.N;
    g.K = l.K;
    g.y = l.y;
    g.workspace = parts;
    g.sa_ws = parts ? sa : nullptr;
    const GemvShape gs = gemv_shape(l.N, l.K);
    g.cb = gs.cb;
    g.ks = gs.ks;
    g.ksplit = gs.ksplit;
    if (!parts) g.ad = a.ad;
    e = launch_gemv(g, st);
  } else if (p.mt) {
    a.kw = p.kw;
    a.ncol = 1;
    const int cw = 8 >> p.kw, per = (G + p.ksplit - 1) / p.ksplit;
    a.strips = (a.cols + cw - 1) / cw;
    if (p.path == kRunPath) {
      e = launch_rows_run(a, p.mt, kSplit, a.strips, p.ksplit, st);
    } else {
      a.sg = per;
      e = launch_rows_stream(a, p.mt, false, kCodes, parts ? kSplit : kAdapt, a.strips, p.ksplit, st);
    }
  } else {
    const int64_t tiles = (l.M + kTileRows - 1) / kTileRows;
    a.strips = (a.nbe + 15) / 16;
    if (!parts) a.halves = half_strips(tiles, a.strips, device_cus());
    e = launch_rows_tile(a, parts ? kSplit : kAdapt, tiles * (a.strips + a.halves), p.ksplit, st);
  }
  if (e != hipSuccess || !parts) return e;
  if (order)
    hipLaunchKernelGGL(adapt_reduce_sorted_kernel,
                       dim3((unsigned)((l.N + 63) / 64), (unsigned)((l.M + 15) / 16)), dim3(256), 0, st,
                       parts, p.ksplit, sa, order, l.M, (int)l.N, a.ad, l.y);
  else
    hipLaunchKernelGGL(adapt_reduce_kernel, dim3((unsigned)((l.N + 255) / 256), (unsigned)l.M), dim3(256),
                       0, st, parts, p.ksplit, sa, l.M, (int)l.N, a.ad, l.y);
  return hipGetLastError();
}

}  // namespace w4a8
