// Rows to microscaled codes and scales and back, and the weight layout of the
// products.  All of it streams: bound by memory (16384 x 3584 bfloat16 rows to
// 4 bits or back, 150 MB, in 22 us: 6.8 TB/s).
#include "mx.h"

#include <type_traits>

namespace w4a8 {
namespace {

constexpr int kThreads = 256;

// Chunk t (eight values) of a matrix of `per` chunks a row; four neighbouring
// lanes hold one block, so its largest magnitude takes two quad permutations.
// 16 bytes a lane in (bfloat16), 4 or 8 out.
template <int FMT, bool F32>
__global__ void __launch_bounds__(kThreads)
quant_kernel(const uint8_t* __restrict__ x, int64_t total, int rule, uint8_t* __restrict__ codes,
             uint8_t* __restrict__ scales) {
  const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (t >= total) return;  // total % 4 == 0: whole blocks leave together
  MxRaw<F32> r;
  r.load(x, t * 8);
  const int b = mx_scale_byte<FMT>(dpp_umax_quad(r.top()), rule);
  const uint2 c = mx_codes8<FMT, F32>(r, b);
  if constexpr (FMT == kFp4)
    reinterpret_cast<uint32_t*>(codes)[t] = c.x;
  else
    reinterpret_cast<uint2*>(codes)[t] = c;
  if ((t & 3) == 0) scales[t >> 2] = (uint8_t)b;
}

// Eight values a lane out: 16 or 32 bytes.
template <int FMT, bool F32>
__global__ void __launch_bounds__(kThreads)
dequant_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t total,
               uint8_t* __restrict__ y) {
  const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (t >= total) return;
  const int b = scales[t >> 2];
  const float s = mx_scale_float(b);
  uint32_t c[2] = {0u, 0u};
  if constexpr (FMT == kFp4) {
    c[0] = reinterpret_cast<const uint32_t*>(codes)[t];
  } else {
    const uint2 v = reinterpret_cast<const uint2*>(codes)[t];
    c[0] = v.x;
    c[1] = v.y;
  }
  v2f_mx v[4];
  if constexpr (FMT == kFp4) {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], s, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], s, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], s, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[0], s, 3);
  } else {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[0], s, false);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[0], s, true);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[1], s, false);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[1], s, true);
  }
  if (b == 255) {
    const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = v2f_mx{nan, nan};
  }
  if constexpr (F32) {
    float4* out = reinterpret_cast<float4*>(y) + 2 * t;
    out[0] = float4{v[0][0], v[0][1], v[1][0], v[1][1]};
    out[1] = float4{v[2][0], v[2][1], v[3][0], v[3][1]};
  } else {
    const uint2 lo = mx_bf16x4(v4f_mx{v[0][0], v[0][1], v[1][0], v[1][1]});
    const uint2 hi = mx_bf16x4(v4f_mx{v[2][0], v[2][1], v[3][0], v[3][1]});
    reinterpret_cast<uint4*>(y)[t] = uint4{lo.x, lo.y, hi.x, hi.y};
  }
}

// ------------------------------------------------- rows for the products

struct GroupTiles {
  const int* offsets;
  int E, bm, slots;
  int64_t P;
  int* ntiles;
  MxTile* tiles;
};

// The tiles of every group, by one workgroup: prefix sums of the groups' tile
// counts (four groups a thread), then a thread a tile.
struct ListLds {
  int head[kMxMaxGroups + 1], lo[kMxMaxGroups], hi[kMxMaxGroups], wave[kThreads / 64];
};
__device__ __forceinline__ void list_tiles(const GroupTiles& g, ListLds& s) {
  constexpr int kPer = kMxMaxGroups / kThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n[kPer], lo[kPer], hi[kPer], own = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    lo[i] = hi[i] = 0;
    if (tid * kPer + i < g.E) mx_run(g.offsets, tid * kPer + i, g.P, lo[i], hi[i]);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    n[i] = (hi[i] - lo[i] + g.bm - 1) / g.bm;
    own += n[i];
    if (tid * kPer + i < g.E) {
      s.lo[tid * kPer + i] = lo[i];
      s.hi[tid * kPer + i] = hi[i];
    }
  }
  const int sum = wave_prefix_sum(own);
  if (lane == 63) s.wave[wave] = sum;
  __syncthreads();
  int base = sum - own;
  for (int w = 0; w < wave; ++w) base += s.wave[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (tid * kPer + i <= g.E) s.head[tid * kPer + i] = base;
    base += n[i];
  }
  if (tid == kThreads - 1 && g.E == kMxMaxGroups) s.head[kMxMaxGroups] = base;
  __syncthreads();
  // (offsets that do not ascend can name more tiles than there are slots)
  const int total = min(s.head[g.E], g.slots);
  if (tid == 0) g.ntiles[0] = total;
  for (int t = tid; t < total; t += kThreads) {
    int a = 0, b = g.E;  // the last group whose first tile is at most t
    while (b - a > 1) {
      const int m = (a + b) / 2;
      if (s.head[m] <= t) a = m; else b = m;
    }
    const int first = s.lo[a] + (t - s.head[a]) * g.bm;
    g.tiles[t] = MxTile{a, first, min(g.bm, s.hi[a] - first), s.head[a], s.head[a + 1] - s.head[a], {0, 0, 0}};
  }
}

struct RowPlaces {
  int ldx, lds;      // rows: strides in bytes
  int G, Q;          // interleaved: steps and supers of a row
  const int* rows;   // interleaved: source rows
  int64_t M;         // of x
  int64_t first;     // row of the launch's first
  int chunks;        // of eight inputs that a row is written in
};

// Workgroup (m, i): chunks of row m, past K the zeros that the layout asks
// for.  The first workgroup lists the tiles as well.
template <int FMT, bool F32, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads)
rows_kernel(const uint8_t* __restrict__ x, int K, int rule, uint8_t* __restrict__ codes,
            uint8_t* __restrict__ scales, int wide, RowPlaces at, GroupTiles g) {
  __shared__ ListLds list;
  unsigned item = blockIdx.x;
  if (g.offsets) {
    if (item == 0) {
      list_tiles(g, list);
      return;
    }
    --item;
  }
  const int64_t m = at.first + item / (unsigned)wide;
  const int ch = (int)(item % (unsigned)wide) * kThreads + threadIdx.x;
  if (ch >= at.chunks) return;
  int64_t from = m;
  if (INTERLEAVED && at.rows) {
    const int r = at.rows[m];
    from = r >= 0 && r < at.M ? r : -1;
  }
  MxRaw<F32> r;
  r.clear();
  if (ch * 8 < K && from >= 0) r.load(x + from * K * (F32 ? 4 : 2), ch * 8);
  const int b = mx_scale_byte<FMT>(dpp_umax_quad(r.top()), rule);
  const uint2 c = mx_codes8<FMT, F32>(r, b);
  // block blk of 32 inputs: step g = blk / 4, j = blk % 4
  const int blk = ch >> 2, j = blk & 3, s = blk >> 2 & 3;
  uint8_t *to, *scale;
  if constexpr (INTERLEAVED) {
    const int64_t b16 = m >> 4;
    const int row = (int)(m & 15);
    if (FMT == kFp4)
      to = codes + (b16 * at.G + (blk >> 2)) * kBlockBytes + (j * 16 + row) * 16 + (ch & 3) * 4;
    else  // 16-byte chunk ch / 2 of the step's eight
      to = codes + ((b16 * at.G + (blk >> 2)) * 2 + (ch >> 3 & 1)) * kBlockBytes + ((ch >> 1 & 3) * 16 + row) * 16 +
           (ch & 1) * 8;
    if (blk >> 2 >= at.G) to = nullptr;
    scale = scales + (b16 * at.Q + (blk >> 4)) * kMxScaleBytes + (j * 16 + row) * 4 + s;
  } else {
    const int byte = ch * (FMT == kFp4 ? 4 : 8);
    to = byte < at.ldx ? codes + m * at.ldx + byte : nullptr;
    scale = scales + m * at.lds + (blk & ~15) + 4 * j + s;
  }
  if (to) {
    if constexpr (FMT == kFp4)
      *reinterpret_cast<uint32_t*>(to) = c.x;
    else
      *reinterpret_cast<uint2*>(to) = c;
  }
  if ((ch & 3) == 0) *scale = (uint8_t)b;
}

// ------------------------------------------------------------ weight layout

// Thread: 16 bytes of a codes block (lane L of block (nb, g)), of a launch whose
// first are unit `first`; blocks that only fill the stride are zero.
__global__ void __launch_bounds__(kThreads)
pack_codes_kernel(const uint8_t* __restrict__ codes, int64_t first, int64_t units, int K, int stride,
                  uint8_t* __restrict__ packed) {
  const int64_t t = first + (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (t >= units) return;
  const int L = (int)(t & 63), j = L >> 4, c = L & 15;
  const int64_t blk = t >> 6, nb = blk / stride;
  const int g = (int)(blk % stride), k = g * kMxStep + j * kMxBlock;
  v4u_rows v = {0, 0, 0, 0};
  if (k < K) v = *reinterpret_cast<const v4u_rows*>(codes + ((nb * 16 + c) * K + k) / 2);
  reinterpret_cast<v4u_rows*>(packed)[t] = v;
}
// Thread: the four scale bytes of lane L of super (nb, q); the last 256
// threads clear the 1024 bytes behind the planes.
__global__ void __launch_bounds__(kThreads)
pack_scales_kernel(const uint8_t* __restrict__ scales, int64_t first, int64_t units, int K, int stride,
                   uint8_t* __restrict__ plane) {
  const int64_t t = first + (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (t >= units + 256) return;
  uint32_t v = 0;
  if (t < units) {
    const int L = (int)(t & 63), j = L >> 4, c = L & 15;
    const int64_t sup = t >> 6, nb = sup / stride;
    const int q = (int)(sup % stride), per = K / kMxBlock;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int b = (4 * q + s) * 4 + j;
      if (b < per) v |= (uint32_t)scales[(nb * 16 + c) * per + b] << (8 * s);
    }
  }
  reinterpret_cast<uint32_t*>(plane)[t] = v;
}
__global__ void __launch_bounds__(kThreads)
unpack_codes_kernel(const uint8_t* __restrict__ packed, int64_t first, int64_t units, int K, int stride,
                    uint8_t* __restrict__ codes) {
  const int64_t t = first + (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (t >= units) return;
  const int L = (int)(t & 63), j = L >> 4, c = L & 15;
  const int64_t blk = t >> 6, nb = blk / stride;
  const int k = (int)(blk % stride) * kMxStep + j * kMxBlock;
  if (k < K)
    *reinterpret_cast<v4u_rows*>(codes + ((nb * 16 + c) * K + k) / 2) = reinterpret_cast<const v4u_rows*>(packed)[t];
}
__global__ void __launch_bounds__(kThreads)
unpack_scales_kernel(const uint8_t* __restrict__ plane, int64_t first, int64_t units, int K, int stride,
                     uint8_t* __restrict__ scales) {
  const int64_t t = first + (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (t >= units) return;
  const int L = (int)(t & 63), j = L >> 4, c = L & 15;
  const int64_t sup = t >> 6, nb = sup / stride;
  const int q = (int)(sup % stride), per = K / kMxBlock;
  const uint32_t v = reinterpret_cast<const uint32_t*>(plane)[t];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int b = (4 * q + s) * 4 + j;
    if (b < per) scales[(nb * 16 + c) * per + b] = (uint8_t)(v >> (8 * s));
  }
}

unsigned blocks_of(int64_t items) { return (unsigned)((items + kThreads - 1) / kThreads); }

// f(format, float) as template arguments.
template <typename F>
void typed(int fmt, int f32, F&& f) {
  using std::integral_constant;
  if (fmt == kFp4) {
    if (f32) f(integral_constant<int, kFp4>{}, integral_constant<bool, true>{});
    else f(integral_constant<int, kFp4>{}, integral_constant<bool, false>{});
  } else {
    if (f32) f(integral_constant<int, kFp8>{}, integral_constant<bool, true>{});
    else f(integral_constant<int, kFp8>{}, integral_constant<bool, false>{});
  }
}

// Chunks of one launch: a launch has fewer than 2^32 threads.
constexpr int64_t kMostChunks = (int64_t)1 << 30;

// f(first, grid) for launches of a thread an item.
template <typename F>
void passes(int64_t items, F&& f) {
  for (int64_t t = 0; t < items; t += kMostChunks)
    f(t, dim3(blocks_of(items - t < kMostChunks ? items - t : kMostChunks)));
}

}  // namespace

hipError_t launch_mx_quant(const MxQuantArgs& a, hipStream_t st) {
  const int64_t total = a.M * a.K / 8;
  passes(total, [&](int64_t t, dim3 grid) {
    typed(a.fmt, a.f32, [&](auto fmt, auto f32) {
      hipLaunchKernelGGL((quant_kernel<decltype(fmt)::value, decltype(f32)::value>), grid, dim3(kThreads), 0, st,
                         static_cast<const uint8_t*>(a.x) + t * 8 * (a.f32 ? 4 : 2), total - t, a.rule,
                         a.codes + t * (a.fmt == kFp4 ? 4 : 8), a.scales + t / 4);
    });
  });
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t M, int64_t K,
                             void* y, int f32, hipStream_t st) {
  const int64_t total = M * K / 8;
  passes(total, [&](int64_t t, dim3 grid) {
    typed(fmt, f32, [&](auto fm, auto fl) {
      hipLaunchKernelGGL((dequant_kernel<decltype(fm)::value, decltype(fl)::value>), grid, dim3(kThreads), 0, st,
                         codes + t * (fmt == kFp4 ? 4 : 8), scales + t / 4, total - t,
                         static_cast<uint8_t*>(y) + t * 8 * (f32 ? 4 : 2));
    });
  });
  return hipGetLastError();
}

hipError_t launch_mx_rows(const MxQuantArgs& a, const MxRowsArgs& r, hipStream_t st) {
  RowPlaces at{};
  at.ldx = (int)mx_row_bytes(a.K, a.fmt);
  at.lds = (int)mx_row_scale_bytes(a.K);
  at.G = (int)mx_steps(a.K);
  at.Q = (int)mx_supers(a.K);
  at.rows = r.rows;
  at.M = a.M;
  // whole supers; of the other layout the stride of the scales.  (Where the
  // supers are odd in number and the last one more than half full, the codes'
  // stride ends 128 bytes behind it.  They stay unwritten, and no stage reads
  // them.)
  at.chunks = r.interleaved ? at.Q * 64 : at.lds * 4;
  const int64_t rows = r.interleaved ? r.P : a.M;
  const int wide = (at.chunks + kThreads - 1) / kThreads;
  const GroupTiles list{r.offsets, r.E, r.bm, r.offsets ? (int)mx_tile_slots(r.P, r.E, r.bm) : 0, r.P, r.ntiles,
                        r.tiles};
  constexpr int64_t kMostItems = (int64_t)1 << 23;  // workgroups of one launch
  const int64_t pass = kMostItems / wide;
  for (int64_t m = 0; m < rows; m += pass) {
    const int64_t n = rows - m < pass ? rows - m : pass;
    GroupTiles g = list;
    if (m) g.offsets = nullptr;  // listed by the first launch
    at.first = m;
    const dim3 grid((unsigned)(n * wide + (g.offsets ? 1 : 0)));
    typed(a.fmt, a.f32, [&](auto fmt, auto f32) {
      constexpr int F = decltype(fmt)::value;
      constexpr bool W = decltype(f32)::value;
      if (r.interleaved)
        hipLaunchKernelGGL((rows_kernel<F, W, true>), grid, dim3(kThreads), 0, st,
                           static_cast<const uint8_t*>(a.x), (int)a.K, a.rule, a.codes, a.scales, wide, at, g);
      else
        hipLaunchKernelGGL((rows_kernel<F, W, false>), grid, dim3(kThreads), 0, st,
                           static_cast<const uint8_t*>(a.x), (int)a.K, a.rule, a.codes, a.scales, wide, at, g);
    });
  }
  return hipGetLastError();
}

hipError_t launch_mx_pack(const uint8_t* codes, const uint8_t* scales, int64_t N, int64_t K, uint8_t* packed,
                          hipStream_t st) {
  const int cs = (int)mx_code_stride(K), ss = (int)mx_scale_stride(K);
  const int64_t uc = N / 16 * cs * 64, us = N / 16 * ss * 64;
  passes(uc, [&](int64_t t, dim3 grid) {
    hipLaunchKernelGGL(pack_codes_kernel, grid, dim3(kThreads), 0, st, codes, t, uc, (int)K, cs, packed);
  });
  passes(us + 256, [&](int64_t t, dim3 grid) {
    hipLaunchKernelGGL(pack_scales_kernel, grid, dim3(kThreads), 0, st, scales, t, us, (int)K, ss,
                       packed + mx_scales_offset(N, K));
  });
  return hipGetLastError();
}

hipError_t launch_mx_unpack(const uint8_t* packed, int64_t N, int64_t K, uint8_t* codes, uint8_t* scales,
                            hipStream_t st) {
  const int cs = (int)mx_code_stride(K), ss = (int)mx_scale_stride(K);
  const int64_t uc = N / 16 * cs * 64, us = N / 16 * ss * 64;
  passes(uc, [&](int64_t t, dim3 grid) {
    hipLaunchKernelGGL(unpack_codes_kernel, grid, dim3(kThreads), 0, st, packed, t, uc, (int)K, cs, codes);
  });
  passes(us, [&](int64_t t, dim3 grid) {
    hipLaunchKernelGGL(unpack_scales_kernel, grid, dim3(kThreads), 0, st, packed + mx_scales_offset(N, K), t, us,
                       (int)K, ss, scales);
  });
  return hipGetLastError();
}

}  // namespace w4a8
