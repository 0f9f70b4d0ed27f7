// Products of a few rows with a microscaled 4-bit weight: one pass over the
// weight, bound by its stream from memory.
//
// A workgroup has one or two 16-channel blocks of one group (with the gated
// activation one of gates and one of values) and all of the inputs, dealt to
// its wavefronts in supers of 512 inputs.  A wavefront's load of a code block is 1 KiB of
// consecutive bytes and is the matrix core operand as it stands: nothing is
// unpacked, and the scales of four steps are one register.  Code blocks are
// loaded four steps ahead of their use.  The wavefronts' sums meet in LDS and
// are added in the order of the inputs.
//
// Rows (at most 16 MT of them) come quantised from the workspace, straight to
// registers four steps ahead like the weight; or raw: each wavefront quantises
// its own inputs of every row into LDS while its first code blocks are on
// their way, which saves a launch and needs no barrier.
//
// Measured: one token 3584 -> 18944 8.0 us (36 MB; the read rate of a large
// buffer, 6.9 TB/s, would take 5.2, an empty launch 1.5); 8 of 128 experts 2048
// -> 1536 gated 5.8 us (13 MB: the chain of offsets, row and first weights);
// 512 rows of 126 such experts 26 us (211 MB, some of it from the last-level
// cache).
#include "mx.h"

#include <type_traits>

namespace w4a8 {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kMaxRaw = 4;  // raw (row, super) pieces loaded ahead of the weight

struct Spot {
  int group, first, rows, strip;
};

// Tile t of bm rows, found from the offsets by every wavefront for itself, 128
// groups at a time.
__device__ __forceinline__ bool find_tile(const MxArgs& a, int t, Spot& s) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < a.E; e0 += 128) {
    int lo[2] = {0, 0}, hi[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (e0 + 64 * i + lane < a.E) mx_run(a.offsets, e0 + 64 * i + lane, a.P, lo[i], hi[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = (hi[i] - lo[i] + a.bm - 1) / a.bm;
      const int sum = wave_prefix_sum(n), head = before + sum - n;
      const uint64_t hit = __ballot(t >= head && t < head + n);
      if (hit) {
        const int l = __ffsll((unsigned long long)hit) - 1;
        const int first =
            __builtin_amdgcn_readlane(lo[i], l) + (t - __builtin_amdgcn_readlane(head, l)) * a.bm;
        s.group = e0 + 64 * i + l;
        s.first = first;
        s.rows = min(a.bm, __builtin_amdgcn_readlane(hi[i], l) - first);
        return true;
      }
      before += __builtin_amdgcn_readlane(sum, 63);
    }
  }
  return false;
}

__device__ __forceinline__ bool locate(const MxArgs& a, Spot& s) {
  const int b = blockIdx.x;
  if (!a.offsets) {  // one group: strips of a tile side by side
    const int tiles = (int)((a.P + a.bm - 1) / a.bm);
    const int at = xcd_run(b, tiles * a.strips);
    const int t = at % tiles;
    s.strip = at / tiles;
    s.group = 0;
    s.first = t * a.bm;
    s.rows = (int)(a.P - s.first < a.bm ? a.P - s.first : a.bm);
    return true;
  }
  if (!a.tiles) {
    s.strip = b % a.strips;
    return find_tile(a, b / a.strips, s);
  }
  const int total = uniform(a.ntiles[0]) * a.strips;
  if (b >= total) return false;
  const int at = xcd_run(b, total), t0 = at / a.strips;
  const int head = uniform(a.tiles[t0].head), n = uniform(a.tiles[t0].n);
  const int local = at - head * a.strips;
  s.strip = local / n;
  // (a group cut short by the number of slots names tiles that are not there)
  const int t = head + local % n;
  if (t >= uniform(a.ntiles[0])) return false;
  s.group = uniform(a.tiles[t].group);
  s.first = uniform(a.tiles[t].first);
  s.rows = uniform(a.tiles[t].rows);
  return true;
}

// Source row of product row p, or -1.
__device__ __forceinline__ int64_t source_row(const MxArgs& a, int p) {
  if (!a.rows) return p;
  const int r = a.rows[p];
  return r >= 0 && r < a.M ? r : -1;
}

template <int FMT, int MT, int RAW, int NC, bool GATED>
__global__ void __launch_bounds__(64 * (MT > 1 ? 8 : kMaxWaves))
mx_stream_kernel(const MxArgs a) {
  constexpr int kUnits = FMT == kFp4 ? 1 : 2;  // 16-byte units of a lane's row operand
  constexpr int kStepBytes = FMT == kFp4 ? 64 : 128;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  Spot sp;
  if (!locate(a, sp)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int c = lane & 15, j = lane >> 4;
  const int q0 = wave * a.Q / waves, q1 = (wave + 1) * a.Q / waves;

  int nb[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) nb[n] = GATED ? sp.strip + n * (a.nb / 2) : min(sp.strip * NC + n, a.nb - 1);
  const uint8_t* wc = a.codes + (int64_t)sp.group * a.nb * a.gstride * kBlockBytes + lane * 16;
  const uint8_t* ws = a.scales + (int64_t)sp.group * a.nb * a.qstride * kMxScaleBytes + lane * 4;

  // Where this lane's row comes from (tiles of groups have at most 16), asked
  // for here and looked at when the sums are there.
  int from = 0;
  if (a.rows) from = a.rows[sp.first + min(c, sp.rows - 1)];

  // This lane's row of each 16: past the last, the last one again.
  const uint8_t* xc[MT];
  const uint8_t* xs[MT];
  if constexpr (!RAW) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = sp.first + min(m * 16 + c, sp.rows - 1);
      xc[m] = a.qx + (int64_t)(r >> 4) * a.G * kUnits * kBlockBytes + (j * 16 + (r & 15)) * 16;
      xs[m] = a.qs + (int64_t)(r >> 4) * a.Q * kMxScaleBytes + (j * 16 + (r & 15)) * 4;
    }
  }

  v4i w[4][NC], x[4][MT][kUnits];
  int sw[NC], sx[MT], sw1[NC], sx1[MT];
  auto load_weight = [&](int s, int q) __attribute__((always_inline)) {
    const int g = min(4 * q + s, a.G - 1);
#pragma unroll
    for (int n = 0; n < NC; ++n)
      w[s][n] = __builtin_nontemporal_load(
          reinterpret_cast<const v4i*>(wc + ((int64_t)nb[n] * a.gstride + g) * kBlockBytes));
  };
  auto load_row = [&](int s, int q) __attribute__((always_inline)) {
    const int g = min(4 * q + s, a.G - 1);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        if constexpr (RAW) {
          const int r = min(c, sp.rows - 1);  // (rows of a raw tile: at most 16)
          x[s][m][u] = *reinterpret_cast<const v4i*>(lds + r * a.ldx + g * kStepBytes + u * 64 + j * 16);
        } else {
          x[s][m][u] = *reinterpret_cast<const v4i*>(xc[m] + (int64_t)(g * kUnits + u) * kBlockBytes);
        }
      }
  };
  auto load_weight_scales = [&](int q, int (&d)[NC]) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < NC; ++n)
      d[n] = *reinterpret_cast<const int*>(ws + ((int64_t)nb[n] * a.qstride + q) * kMxScaleBytes);
  };
  auto load_row_scales = [&](int q, int (&d)[MT]) __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (RAW) {
        const int r = min(c, sp.rows - 1);
        d[m] = *reinterpret_cast<const int*>(lds + sp.rows * a.ldx + r * a.lds + q * kMxRowScale + j * 4);
      } else {
        d[m] = *reinterpret_cast<const int*>(xs[m] + (int64_t)q * kMxScaleBytes);
      }
    }
  };

  if constexpr (RAW) {
    constexpr bool F32 = RAW == 2;
    const int nq = q1 - q0, pieces = sp.rows * nq;
    MxRaw<F32> raw[kMaxRaw];
    auto fetch = [&](int i, MxRaw<F32>& r) __attribute__((always_inline)) {
      const int64_t row = max(source_row(a, sp.first + i / nq), (int64_t)0);
      const int k = (q0 + i % nq) * kMxSuper + lane * 8;
      r.clear();
      if (k < a.K) r.load(static_cast<const uint8_t*>(a.x) + row * a.K * (F32 ? 4 : 2), k);
    };
    auto put = [&](int i, const MxRaw<F32>& r) __attribute__((always_inline)) {
      const int b = mx_scale_byte<FMT>(dpp_umax_quad(r.top()), a.rule);
      const uint2 code = mx_codes8<FMT, F32>(r, b);
      const int m = i / nq, q = q0 + i % nq;
      const int at = q * 4 * kStepBytes + lane * (FMT == kFp4 ? 4 : 8);
      uint8_t* to = lds + m * a.ldx + at;
      if (at < a.ldx) {
        if constexpr (FMT == kFp4)
          *reinterpret_cast<uint32_t*>(to) = code.x;
        else
          *reinterpret_cast<uint2*>(to) = code;
      }
      const int blk = lane >> 2;
      if ((lane & 3) == 0)
        lds[sp.rows * a.ldx + m * a.lds + q * kMxRowScale + 4 * (blk & 3) + (blk >> 2)] = (uint8_t)b;
    };
#pragma unroll
    for (int i = 0; i < kMaxRaw; ++i)
      if (i < pieces) fetch(i, raw[i]);
    if (nq > 0) {
      load_weight_scales(q0, sw);
#pragma unroll
      for (int s = 0; s < 4; ++s) load_weight(s, q0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kMaxRaw; ++i)
      if (i < pieces) put(i, raw[i]);
    for (int i = kMaxRaw; i < pieces; ++i) {
      MxRaw<F32> r;
      fetch(i, r);
      put(i, r);
    }
    // the lanes of a wavefront read what its other lanes wrote
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  } else if (q0 < q1) {
    load_weight_scales(q0, sw);
#pragma unroll
    for (int s = 0; s < 4; ++s) load_weight(s, q0);
  }

  v4f_mx acc[MT][NC];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NC; ++n) acc[m][n] = v4f_mx{0.f, 0.f, 0.f, 0.f};

  if (q0 < q1) {
    load_row_scales(q0, sx);
#pragma unroll
    for (int s = 0; s < 4; ++s) load_row(s, q0);
  }
  for (int q = q0; q < q1; ++q) {
    const bool more = q + 1 < q1;
    if (more) {
      load_weight_scales(q + 1, sw1);
      load_row_scales(q + 1, sx1);
    }
    auto step = [&](auto sc) __attribute__((always_inline)) {
      constexpr int s = decltype(sc)::value;
      if (4 * q + s < a.G) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          v8i_mx xv;
          if constexpr (FMT == kFp4) xv = mx_wide(x[s][m][0]);
          else xv = mx_wide(x[s][m][0], x[s][m][kUnits - 1]);
#pragma unroll
          for (int n = 0; n < NC; ++n)
            acc[m][n] = mx_mfma<FMT, s>(mx_wide(w[s][n]), xv, acc[m][n], sw[n], sx[m]);
        }
      }
      if (more) {
        load_weight(s, q + 1);
        load_row(s, q + 1);
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
#pragma unroll
    for (int n = 0; n < NC; ++n) sw[n] = sw1[n];
#pragma unroll
    for (int m = 0; m < MT; ++m) sx[m] = sx1[m];
  }

  // Sums of the wavefronts, in the order of the inputs: [wave][m][n][lane].
  // (Every wavefront is past its rows in LDS before they are overwritten.)
  v4f_mx* red = reinterpret_cast<v4f_mx*>(lds);
  constexpr int kTiles = MT * NC;
  if (waves > 1) {
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NC; ++n) red[(wave * kTiles + m * NC + n) * 64 + lane] = acc[m][n];
    __syncthreads();
  }
  constexpr int kOut = GATED ? 1 : NC;
  const int width = a.nb * (GATED ? 8 : 16);
  for (int i = wave; i < MT * kOut; i += waves) {  // (only one wavefront: all of them)
    const int m = i / kOut, n0 = i % kOut;
    auto sum = [&](int n) __attribute__((always_inline)) {
      v4f_mx v = {0.f, 0.f, 0.f, 0.f};
      if (waves > 1) {
        v = red[(m * NC + n) * 64 + lane];
        for (int k = 1; k < waves; ++k) v += red[(k * kTiles + m * NC + n) * 64 + lane];
      } else {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          if (t == m * NC + n) v = acc[t / NC][t % NC];
      }
      return v;
    };
    v4f_mx out = sum(n0);
    if constexpr (GATED) {
      const v4f_mx value = sum(1);
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = silu_mul(out[e], value[e]);
    }
    const int at = m * 16 + c, block = sp.strip * kOut + n0;
    if (at >= sp.rows || block * 16 >= width) continue;
    const int p = sp.first + at;
    uint2 bits = mx_bf16x4(out);
    if (a.rows && (from < 0 || from >= a.M)) bits = uint2{0u, 0u};  // whatever the weight holds
    *reinterpret_cast<uint2*>(a.y + (int64_t)p * width + block * 16 + 4 * j) = bits;
  }
}

template <int FMT, int MT, int RAW, int NC, bool GATED>
hipError_t launch_one(const MxArgs& a, const MxPlan& p, unsigned blocks, hipStream_t st) {
  const size_t sums = p.waves > 1 ? (size_t)p.waves * MT * NC * 1024 : 0;
  const size_t rows = RAW ? (size_t)(a.P < a.bm ? a.P : a.bm) * (a.ldx + a.lds) : 0;
  const size_t lds = sums > rows ? sums : rows;
  hipLaunchKernelGGL((mx_stream_kernel<FMT, MT, RAW, NC, GATED>), dim3(blocks), dim3(64 * p.waves), lds, st, a);
  return hipGetLastError();
}

// What plans ask for: the gated activation of groups, whose tiles have 16 rows
// at most; of raw rows one block a workgroup where nothing is gated.
template <int FMT, int MT, int RAW>
hipError_t launch_cols(const MxArgs& a, const MxPlan& p, bool gated, unsigned blocks, hipStream_t st) {
  if constexpr (MT == 1) {
    if (gated) return launch_one<FMT, MT, RAW, 2, true>(a, p, blocks, st);
  }
  if constexpr (!RAW) {
    if (p.bn == 32 && !gated) return launch_one<FMT, MT, RAW, 2, false>(a, p, blocks, st);
  }
  if (gated || p.bn != 16) return hipErrorInvalidValue;
  return launch_one<FMT, MT, RAW, 1, false>(a, p, blocks, st);
}

template <int FMT>
hipError_t launch_fmt(const MxArgs& a, const MxPlan& p, bool gated, unsigned blocks, hipStream_t st) {
  if (p.path == kMxToken)
    return a.f32 ? launch_cols<FMT, 1, 2>(a, p, gated, blocks, st) : launch_cols<FMT, 1, 1>(a, p, gated, blocks, st);
  switch (p.bm) {
    case 16: return launch_cols<FMT, 1, 0>(a, p, gated, blocks, st);
    case 32: return launch_cols<FMT, 2, 0>(a, p, gated, blocks, st);
    case 48: return launch_cols<FMT, 3, 0>(a, p, gated, blocks, st);
    default: return launch_cols<FMT, 4, 0>(a, p, gated, blocks, st);
  }
}

}  // namespace

hipError_t launch_mx_stream(const MxArgs& a, const MxPlan& p, int fmt, bool gated, hipStream_t st) {
  const int64_t tiles = a.offsets ? mx_tile_slots(a.P, a.E, a.bm) : (a.P + a.bm - 1) / a.bm;
  const int64_t blocks = tiles * a.strips;
  if (blocks * 64 * p.waves >= ((int64_t)1 << 32)) return hipErrorInvalidValue;
  return fmt == kFp4 ? launch_fmt<kFp4>(a, p, gated, (unsigned)blocks, st)
                     : launch_fmt<kFp8>(a, p, gated, (unsigned)blocks, st);
}

}  // namespace w4a8
