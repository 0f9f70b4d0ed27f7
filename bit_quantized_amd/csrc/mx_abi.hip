// Host entry points of include/w4a8_mx.h: argument checks, the plan of a call,
// workspace layout and launches.  Every check runs before anything is enqueued.
#include <algorithm>
#include <cstdarg>
#include <cstdio>

#include "../../include/w4a8_mx.h"
#include "mx.h"

namespace w4a8 {
namespace {

constexpr int64_t kMostRows = (int64_t)1 << 24;
constexpr int64_t kMostOffset = ((int64_t)1 << 32) - 1;  // bytes that 32 bits of offset reach

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of the tile kernel.  `one` and `two`: microseconds of a step of 128
// inputs where a compute unit has one of them, and where it has as many as fit
// (`fit`), with rows of 4 and of 8 bits; 2048 to 18944 inputs, 33 to 4096 rows,
// +- 20 %.
struct TileShape {
  int bm, bn, fit;
  double one, two;
};
constexpr TileShape kShapes[2][4] = {
    {{64, 128, 2, 0.24, 0.46}, {128, 128, 2, 0.42, 0.80}, {128, 256, 2, 0.66, 1.28}, {256, 256, 1, 1.22, 1.22}},
    {{64, 128, 2, 0.28, 0.54}, {128, 128, 2, 0.48, 0.88}, {128, 256, 1, 0.80, 0.80}, {256, 256, 1, 1.35, 1.35}}};
constexpr int kSplitMost = 16;

// Microseconds of `tiles` tiles of `steps` steps each.
double tile_cost(const TileShape& s, int64_t tiles, double steps) {
  const int64_t cus = device_cus(), round = cus * s.fit;
  const int64_t rest = tiles % round;
  return steps * (double(tiles / round) * s.two + (rest == 0 ? 0.0 : rest <= cus ? s.one : s.two));
}

// The linear's tiles: the shape and split of least cost (over 54 sizes 1 % from
// the fastest of a sweep, at worst 15: 1024 rows 18944 -> 3584 in 8 bits, 88 us
// of 128 x 128, 77 of 128 x 256 in halves).  A split adds a launch and its
// sums, written and read at 4 TB/s (33 rows 18944 -> 3584: 16.8 us of 8 slices,
// 17.6 of 9, 52 unsplit).
double plan_tiles(MxPlan& p, int64_t M, int64_t N, int64_t Q, int fmt) {
  double best = 1e30;
  for (const TileShape& s : kShapes[fmt]) {
    const int64_t tiles = ceil_div(M, s.bm) * ceil_div(N, s.bn);
    for (int64_t k = 1; k == 1 || (k <= kSplitMost && k <= Q / 2 && tiles * k <= device_cus()); ++k) {
      if (ceil_div(Q, ceil_div(Q, k)) != k) continue;  // as long with fewer
      const double cost = tile_cost(s, tiles * k, 4.0 * ceil_div(Q, k)) + (k > 1 ? 3.0 + 8e-6 * k * M * N / 4.0 : 0.0);
      if (cost < best) {
        best = cost;
        p.bm = s.bm;
        p.bn = s.bn;
        p.ksplit = (int)k;
      }
    }
  }
  return best;
}

// Most rows that the stream takes: of the linear; of a group, evenly shared.
constexpr int kStreamRows = 64, kStreamPerGroup = 8;

// Microseconds of the stream for M rows: the weight from memory, or the rows
// through the L1 caches of the compute units, KiB at 45 a microsecond (33 rows
// 18944 -> 3584 in 8 bits: 16 us; 64 rows 4096 -> 4096 in 4: 4).
double stream_cost(int64_t M, int64_t N, int64_t K, int fmt) {
  const double blocks = std::max(1.0, N / 16.0 / device_cus()), G = double(mx_steps(K));
  const double kib = blocks * G * (ceil_div(M, 16) * (fmt == kFp4 ? 1 : 2) + 1);
  return std::max(kib / 45.0, N * K * 0.53 / 6.5e6);
}

// Wavefronts of a stream workgroup: as many as shorten the longest share of
// the supers.
int stream_waves(int64_t Q, int most) {
  int best = 1;
  for (int w = 2; w <= most && w <= Q; ++w)
    if (ceil_div(Q, w) < ceil_div(Q, best)) best = w;
  return best;
}

// Raw rows: every workgroup quantises all of its tile's.  It saves a launch
// (2.5 us) where there are one or two, or the rows that workgroups read again
// are few bytes (8 rows 3584 -> 3584: 8.2 against 9.6 us; 4 rows 3584 ->
// 18944, 34 MB: 12.3 against 11.5).  The bytes are counted at two an input: a
// plan does not know whether the rows are float.
constexpr int64_t kTokenLds = 48 * 1024, kTokenReads = 20 << 20;
bool token_fits(int64_t rows, int64_t N, int64_t K, int fmt) {
  return rows <= 16 && rows * (mx_row_bytes(K, fmt) + mx_row_scale_bytes(K)) <= kTokenLds &&
         (rows <= 2 || N / 16 * rows * K * 2 <= kTokenReads);
}

}  // namespace

MxPlan mx_plan(int64_t M, int64_t P, int E, int64_t N, int64_t K, int fmt) {
  MxPlan p;
  const int64_t Q = mx_supers(K);
  p.bm = p.bn = 16;
  if (token_fits(P, N, K, fmt)) {
    p.path = kMxToken;
  } else if (!E) {
    const double tiles = M > 16 ? plan_tiles(p, M, N, Q, fmt) : 1e30;
    p.path = kMxTile;
    if (M <= 16 || (M <= kStreamRows && stream_cost(M, N, K, fmt) < tiles)) {
      p.path = kMxStream;
      p.ksplit = 1;
      p.bm = (int)ceil_div(M, 16) * 16;
      // (32 rows 4096 -> 8192 in 8 bits: 9.1 against 10.4 us; 20 rows 2048 -> 8192 in 4: 5.8, 6.0)
      p.bn = M > 16 && N / 32 >= device_cus() ? 32 : 16;
    }
  } else {
    // By the rows of a group, evenly shared (the groups' own numbers are on
    // the device), measured with 64 and 128 groups, which fill the compute
    // units whatever the tile.  Few groups do not: 17 rows of one group 3584 ->
    // 3584 take 10.2 us in 28 tiles, 6.4 by the linear's plan.
    // 64 tokens x 8 of 128 (4 rows a group) take 31 us streamed, 256 (16 rows)
    // 47, and 37 in tiles of 64.  With 4-bit rows 64 rows a group take 46 in
    // tiles of 64 x 128, 51 in the next; 96 rows 98, 98 (128 x 128), 90 (128 x
    // 256) and 118 (256 x 256); 576 rows 351, 297, 254 and 292.  With 8-bit
    // rows 192 rows take 167, 162, 163 and 175.
    const double per = double(P) / E;
    p.path = kMxTile;
    if (per <= kStreamPerGroup) {
      p.path = kMxStream;
      p.bn = 32;  // (of the plain product: 27.1 against 29.7 us at 4 rows a group)
    } else if (per <= 80) {
      p.bm = 64, p.bn = 128;
    } else if ((fmt == kFp8 && per <= 256) || N <= 256) {
      p.bm = 128, p.bn = 128;
    } else if (per <= 768) {
      p.bm = 128, p.bn = 256;
    } else {
      p.bm = 256, p.bn = 256;
    }
  }
  if (p.path != kMxTile) p.waves = stream_waves(Q, p.bm > 16 ? 8 : 16);
  auto take = [&](int64_t bytes) {
    const int64_t at = p.bytes;
    p.bytes += round_up256(bytes);
    return at;
  };
  if (p.path != kMxToken) {
    if (p.path == kMxStream) {
      p.codes = take(ceil_div(P, 16) * mx_block_bytes(K, fmt));
      p.scales = take(ceil_div(P, 16) * mx_block_scale_bytes(K));
    } else {
      p.codes = take(M * mx_row_bytes(K, fmt));
      p.scales = take(M * mx_row_scale_bytes(K));
    }
    if (E) {
      p.ntiles = take(sizeof(int));
      p.tiles = take(mx_tile_slots(P, E, p.bm) * (int64_t)sizeof(MxTile));
    }
    if (p.ksplit > 1) p.parts = take(p.ksplit * P * N * 4);
  }
  p.bytes = std::max<int64_t>(p.bytes, 256);
  return p;
}

namespace {

// Bytes that serve M (P) rows and every smaller number of them.
int64_t workspace_bound(int64_t M, int64_t P, int E, int64_t N, int64_t K, int fmt) {
  // rows, or interleaved product rows of the stream
  const int64_t Ps = std::min<int64_t>(P, E ? (int64_t)kStreamPerGroup * E : kStreamRows);
  const int64_t n = std::max(round_up256(M * mx_row_bytes(K, fmt)) + round_up256(M * mx_row_scale_bytes(K)),
                             ceil_div(Ps, 16) * (mx_block_bytes(K, fmt) + mx_block_scale_bytes(K)));
  if (E) return n + 256 + round_up256(mx_tile_slots(P, E, 16) * (int64_t)sizeof(MxTile));
  // ksplit times the tiles is at most the compute units; no split of fewer than four supers
  int64_t parts = 0;
  const int64_t Q = mx_supers(K);
  for (const TileShape& s : kShapes[fmt])
    if (Q >= 4 && ceil_div(N, s.bn) * 2 <= device_cus())  // (else never split)
      parts = std::max(parts, std::min((int64_t)device_cus() * s.bm * s.bn, std::min<int64_t>(kSplitMost, Q / 2) * M * N));
  return std::max<int64_t>(n + round_up256(parts * 4), 256);
}

int fail(int status, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return report_error(status, msg);
}

int finish(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(W4A8_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
  return report_error(W4A8_OK, "");
}

struct Span {
  const void* p;
  size_t bytes;
};

// Every pointer set and aligned; no written buffer meets another one.
template <int NI, int NO>
int check_buffers(const Span (&in)[NI], const Span (&out)[NO]) {
  auto at = [](const Span& s) { return reinterpret_cast<uintptr_t>(s.p); };
  auto meet = [&](const Span& a, const Span& b) {
    return a.bytes && b.bytes && at(a) < at(b) + b.bytes && at(b) < at(a) + a.bytes;
  };
  for (const Span& s : in)
    if (s.bytes && !s.p) return fail(W4A8_ERR_INVALID_ARG, "null input pointer");
  for (const Span& s : out)
    if (s.bytes && !s.p) return fail(W4A8_ERR_INVALID_ARG, "null output pointer");
  for (const Span& s : in)
    if (s.bytes && at(s) % 16) return fail(W4A8_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  for (const Span& s : out)
    if (s.bytes && at(s) % 16) return fail(W4A8_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  for (int o = 0; o < NO; ++o) {
    for (const Span& s : in)
      if (meet(out[o], s)) return fail(W4A8_ERR_INVALID_ARG, "an output or the workspace aliases an input");
    for (int q = o + 1; q < NO; ++q)
      if (meet(out[o], out[q])) return fail(W4A8_ERR_INVALID_ARG, "outputs or the workspace alias each other");
  }
  return W4A8_OK;
}

int check_rows(int64_t M) {
  if (M <= 0 || M > kMostRows) return fail(W4A8_ERR_INVALID_ARG, "%lld rows out of range", (long long)M);
  return W4A8_OK;
}
int check_inputs(int64_t K) {
  if (K <= 0) return fail(W4A8_ERR_INVALID_ARG, "K=%lld out of range", (long long)K);
  if (K % kMxBlock || K > kMxMaxK)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "K=%lld is not a multiple of 32 up to 2^22", (long long)K);
  return W4A8_OK;
}
int check_dtype(int32_t d) {
  if (d != W4A8_BF16 && d != W4A8_F32) return fail(W4A8_ERR_INVALID_ARG, "unknown activation dtype %d", (int)d);
  return W4A8_OK;
}
int check_format(int32_t f) {
  if (f != W4A8_MX_FP4 && f != W4A8_MX_FP8) return fail(W4A8_ERR_INVALID_ARG, "unknown element format %d", (int)f);
  return W4A8_OK;
}
int check_rule(int32_t r) {
  if (r != W4A8_MX_FLOOR && r != W4A8_MX_CEIL) return fail(W4A8_ERR_INVALID_ARG, "unknown scale rule %d", (int)r);
  return W4A8_OK;
}
int check_weight(int64_t N, int64_t K) {
  if (int rc = check_inputs(K)) return rc;
  if (N <= 0 || N > ((int64_t)1 << 31)) return fail(W4A8_ERR_INVALID_ARG, "N=%lld out of range", (long long)N);
  if (N % 16) return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "N=%lld is not a multiple of 16", (long long)N);
  return W4A8_OK;
}
int check_product(int64_t M, int64_t N, int64_t K, int32_t act) {
  if (int rc = check_rows(M)) return rc;
  if (int rc = check_weight(N, K)) return rc;
  if (int rc = check_format(act)) return rc;
  // (with the odd stride at most 1.5 2^31 bytes of codes)
  if (N * mx_steps(K) * kMxStep > kMostOffset)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "the codes are addressed with 32-bit offsets (N=%lld K=%lld)",
                (long long)N, (long long)K);
  return W4A8_OK;
}
// A launch has fewer than 2^32 threads.
int check_launch(const MxPlan& p, int64_t P, int32_t E, int64_t N) {
  const int64_t tiles = E ? mx_tile_slots(P, E, p.bm) : ceil_div(P, p.bm);
  const int64_t threads = p.path == kMxTile ? 512 : 64 * p.waves;
  if (tiles * ceil_div(N, p.bn) * threads >= (int64_t)1 << 32)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "%lld x %lld outputs in one call", (long long)P, (long long)N);
  return W4A8_OK;
}
// The checks of the sizes, and the plan that they give.
int plan_linear(int64_t M, int64_t N, int64_t K, int32_t act, MxPlan& p) {
  if (int rc = check_product(M, N, K, act)) return rc;
  p = mx_plan(M, M, 0, N, K, act);
  return check_launch(p, M, 0, N);
}
int plan_grouped(int64_t M, int64_t P, int32_t E, int64_t N, int64_t K, int32_t act, MxPlan& p) {
  if (int rc = check_rows(M)) return rc;
  if (E < 1 || E > kMxMaxGroups) return fail(W4A8_ERR_INVALID_ARG, "E=%d out of [1, %d]", (int)E, kMxMaxGroups);
  if (int rc = check_product(P, N, K, act)) return rc;
  if (N * E > (int64_t)1 << 31) return fail(W4A8_ERR_INVALID_ARG, "N=%lld times E=%d out of range", (long long)N, (int)E);
  p = mx_plan(M, P, E, N, K, act);
  return check_launch(p, P, E, N);
}

size_t value_bytes(int32_t d) { return d == W4A8_F32 ? 4 : 2; }
size_t code_bytes(int64_t M, int64_t K, int32_t f) { return (size_t)(f == W4A8_MX_FP4 ? M * K / 2 : M * K); }

// Rows to the workspace, then the product.
struct Call {
  const void* x;
  int32_t x_dtype, act, rule;
  const uint8_t* packed;
  const int32_t *offsets, *rows;
  int64_t M, P;
  int32_t E;  // 0: the linear
  int64_t N, K;
  bool gated;
  uint16_t* y;
  uint8_t* ws;
};
hipError_t run(const Call& c, const MxPlan& p, hipStream_t st) {
  const int64_t groups = c.E ? c.E : 1;
  MxArgs a{};
  a.rule = c.rule;
  a.codes = c.packed;
  a.scales = c.packed + mx_scales_offset(groups * c.N, c.K);
  a.offsets = c.offsets;
  a.rows = c.rows;
  a.M = c.M;
  a.P = c.P;
  a.E = c.E;
  a.K = (int)c.K;
  a.G = (int)mx_steps(c.K);
  a.Q = (int)mx_supers(c.K);
  a.gstride = (int)mx_code_stride(c.K);
  a.qstride = (int)mx_scale_stride(c.K);
  a.ldx = (int)mx_row_bytes(c.K, c.act);
  a.lds = (int)mx_row_scale_bytes(c.K);
  a.nb = (int)(c.N / 16);
  a.bm = p.bm;
  a.y = c.y;
  if (p.path == kMxToken) {
    a.x = c.x;
    a.f32 = c.x_dtype == W4A8_F32;
  } else {
    a.qx = c.ws + p.codes;
    a.qs = c.ws + p.scales;
    if (c.E) {
      a.ntiles = reinterpret_cast<int*>(c.ws + p.ntiles);
      a.tiles = reinterpret_cast<MxTile*>(c.ws + p.tiles);
    }
    a.parts = reinterpret_cast<float*>(c.ws + p.parts);
    const MxQuantArgs q{c.x, c.x_dtype == W4A8_F32, c.act, c.rule, c.M, c.K, c.ws + p.codes, c.ws + p.scales};
    const MxRowsArgs r{p.path == kMxStream, c.rows, c.offsets, c.E, p.bm, c.P, const_cast<int*>(a.ntiles),
                       const_cast<MxTile*>(a.tiles)};
    const hipError_t e = launch_mx_rows(q, r, st);
    if (e != hipSuccess) return e;
  }
  if (p.path == kMxTile) {
    a.strips = (int)ceil_div(c.N, p.bn);
    return launch_mx_tile(a, p, c.act, c.gated, st);
  }
  a.strips = c.gated ? a.nb / 2 : (int)ceil_div(c.N, p.bn);
  return launch_mx_stream(a, p, c.act, c.gated, st);
}

int fill_plan(const MxPlan& p, w4a8_mx_plan_t* plan) {
  plan->path = p.path;
  plan->tile_rows = p.bm;
  plan->tile_cols = p.bn;
  plan->ksplit = p.ksplit;
  return report_error(W4A8_OK, "");
}

}  // namespace
}  // namespace w4a8

using namespace w4a8;

extern "C" {

int w4a8_mx_quant(const void* x, int32_t x_dtype, int64_t M, int64_t K, int32_t format, int32_t rule,
                  uint8_t* codes, uint8_t* scales, void* stream) {
  if (int rc = check_rows(M)) return rc;
  if (int rc = check_inputs(K)) return rc;
  if (int rc = check_dtype(x_dtype)) return rc;
  if (int rc = check_format(format)) return rc;
  if (int rc = check_rule(rule)) return rc;
  const Span in[] = {{x, (size_t)M * K * value_bytes(x_dtype)}};
  const Span out[] = {{codes, code_bytes(M, K, format)}, {scales, (size_t)M * K / kMxBlock}};
  if (int rc = check_buffers(in, out)) return rc;
  (void)hipGetLastError();
  const MxQuantArgs a{x, x_dtype == W4A8_F32, format, rule, M, K, codes, scales};
  return finish(launch_mx_quant(a, static_cast<hipStream_t>(stream)), "quantiser launch");
}

int w4a8_mx_dequant(const uint8_t* codes, const uint8_t* scales, int32_t format, int64_t M, int64_t K, void* y,
                    int32_t y_dtype, void* stream) {
  if (int rc = check_rows(M)) return rc;
  if (int rc = check_inputs(K)) return rc;
  if (int rc = check_format(format)) return rc;
  if (int rc = check_dtype(y_dtype)) return rc;
  const Span in[] = {{codes, code_bytes(M, K, format)}, {scales, (size_t)M * K / kMxBlock}};
  const Span out[] = {{y, (size_t)M * K * value_bytes(y_dtype)}};
  if (int rc = check_buffers(in, out)) return rc;
  (void)hipGetLastError();
  return finish(launch_mx_dequant(codes, scales, format, M, K, y, y_dtype == W4A8_F32,
                                  static_cast<hipStream_t>(stream)),
                "dequantiser launch");
}

size_t w4a8_mx_weight_bytes(int64_t N, int64_t K) {
  if (check_weight(N, K)) return 0;
  return (size_t)mx_weight_bytes(N, K);
}

int w4a8_mx_pack_weights(const uint8_t* codes, const uint8_t* scales, int64_t N, int64_t K, void* packed,
                         size_t packed_bytes, void* stream) {
  if (int rc = check_weight(N, K)) return rc;
  const size_t need = (size_t)mx_weight_bytes(N, K);
  if (packed && packed_bytes < need)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "packed buffer %zu bytes, need %zu", packed_bytes, need);
  const Span in[] = {{codes, (size_t)N * K / 2}, {scales, (size_t)N * K / kMxBlock}};
  const Span out[] = {{packed, need}};
  if (int rc = check_buffers(in, out)) return rc;
  (void)hipGetLastError();
  return finish(launch_mx_pack(codes, scales, N, K, static_cast<uint8_t*>(packed), static_cast<hipStream_t>(stream)),
                "pack launch");
}

int w4a8_mx_unpack_weights(const void* packed, size_t packed_bytes, int64_t N, int64_t K, uint8_t* codes,
                           uint8_t* scales, void* stream) {
  if (int rc = check_weight(N, K)) return rc;
  const size_t need = (size_t)mx_weight_bytes(N, K);
  if (packed && packed_bytes < need)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "packed buffer %zu bytes, need %zu", packed_bytes, need);
  const Span in[] = {{packed, need}};
  const Span out[] = {{codes, (size_t)N * K / 2}, {scales, (size_t)N * K / kMxBlock}};
  if (int rc = check_buffers(in, out)) return rc;
  (void)hipGetLastError();
  return finish(launch_mx_unpack(static_cast<const uint8_t*>(packed), N, K, codes, scales,
                                 static_cast<hipStream_t>(stream)),
                "unpack launch");
}

int w4a8_mx_linear_plan(int64_t M, int64_t N, int64_t K, int32_t act, w4a8_mx_plan_t* plan) {
  if (!plan) return fail(W4A8_ERR_INVALID_ARG, "null plan");
  MxPlan p;
  if (int rc = plan_linear(M, N, K, act, p)) return rc;
  return fill_plan(p, plan);
}

size_t w4a8_mx_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t act) {
  MxPlan p;
  if (plan_linear(M, N, K, act, p)) return 0;
  return (size_t)workspace_bound(M, M, 0, N, K, act);
}

int w4a8_mx_linear(const void* x, int32_t x_dtype, int32_t act, int32_t rule, const void* packed,
                   size_t packed_bytes, int64_t M, int64_t N, int64_t K, uint16_t* y, void* workspace,
                   size_t workspace_bytes, void* stream) {
  MxPlan p;
  if (int rc = plan_linear(M, N, K, act, p)) return rc;
  if (int rc = check_dtype(x_dtype)) return rc;
  if (int rc = check_rule(rule)) return rc;
  const size_t wb = (size_t)mx_weight_bytes(N, K);
  if (packed && packed_bytes < wb)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "packed buffer %zu bytes, need %zu", packed_bytes, wb);
  if (!workspace || workspace_bytes < (size_t)p.bytes)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "workspace %zu bytes, need %zu", workspace_bytes, (size_t)p.bytes);
  const Span in[] = {{x, (size_t)M * K * value_bytes(x_dtype)}, {packed, wb}};
  const Span out[] = {{y, (size_t)M * N * 2}, {workspace, (size_t)p.bytes}};
  if (int rc = check_buffers(in, out)) return rc;
  (void)hipGetLastError();
  const Call c{x, x_dtype, act,  rule, static_cast<const uint8_t*>(packed), nullptr, nullptr, M, M, 0, N, K,
               false, y, static_cast<uint8_t*>(workspace)};
  return finish(run(c, p, static_cast<hipStream_t>(stream)), "linear launch");
}

int w4a8_mx_grouped_linear_plan(int64_t M, int64_t P, int32_t E, int64_t N, int64_t K, int32_t act,
                                w4a8_mx_plan_t* plan) {
  if (!plan) return fail(W4A8_ERR_INVALID_ARG, "null plan");
  MxPlan p;
  if (int rc = plan_grouped(M, P, E, N, K, act, p)) return rc;
  return fill_plan(p, plan);
}

size_t w4a8_mx_grouped_linear_workspace_bytes(int64_t M, int64_t P, int32_t E, int64_t N, int64_t K, int32_t act) {
  MxPlan p;
  if (plan_grouped(M, P, E, N, K, act, p)) return 0;
  return (size_t)workspace_bound(M, P, E, N, K, act);
}

int w4a8_mx_grouped_linear(const void* x, int32_t x_dtype, int32_t act, int32_t rule, const void* packed,
                           size_t packed_bytes, const int32_t* offsets, const int32_t* rows, int64_t M, int64_t P,
                           int32_t E, int64_t N, int64_t K, int32_t gated, uint16_t* y, void* workspace,
                           size_t workspace_bytes, void* stream) {
  MxPlan p;
  if (int rc = plan_grouped(M, P, E, N, K, act, p)) return rc;
  if (int rc = check_dtype(x_dtype)) return rc;
  if (int rc = check_rule(rule)) return rc;
  if (gated && N % 32)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "N=%lld gates and values are not a multiple of 32", (long long)N);
  if (!rows && M != P)
    return fail(W4A8_ERR_INVALID_ARG, "without rows M=%lld and P=%lld must agree", (long long)M, (long long)P);
  if (rows && M * mx_row_bytes(K, act) >= kOob)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "rows by index are addressed with 32-bit offsets (M=%lld K=%lld)",
                (long long)M, (long long)K);
  const size_t wb = (size_t)mx_weight_bytes(E * N, K);
  if (packed && packed_bytes < wb)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "packed buffer %zu bytes, need %zu", packed_bytes, wb);
  if (!workspace || workspace_bytes < (size_t)p.bytes)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "workspace %zu bytes, need %zu", workspace_bytes, (size_t)p.bytes);
  const Span in[] = {{x, (size_t)M * K * value_bytes(x_dtype)},
                     {packed, wb},
                     {offsets, ((size_t)E + 1) * 4},
                     {rows, rows ? (size_t)P * 4 : 0}};
  const Span out[] = {{y, (size_t)P * N * (gated ? 1 : 2)}, {workspace, (size_t)p.bytes}};
  if (int rc = check_buffers(in, out)) return rc;
  (void)hipGetLastError();
  const Call c{x, x_dtype, act, rule, static_cast<const uint8_t*>(packed), offsets, rows, M, P, E, N, K,
               gated != 0, y, static_cast<uint8_t*>(workspace)};
  return finish(run(c, p, static_cast<hipStream_t>(stream)), "grouped linear launch");
}

}  // extern "C"
