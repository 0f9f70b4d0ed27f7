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

struct TileShape {
  int bm, bn;
};
constexpr TileShape kSmall{64, 128}, kMiddle{128, 128}, kLarge{256, 256};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Wavefronts of a stream workgroup: those that share the supers most evenly,
// the more the better.
int stream_waves(int64_t Q) {
  int best = 1;
  int64_t best_cost = Q;
  for (int w = 1; w <= 8 && w <= Q; ++w) {
    const int64_t cost = ceil_div(Q, w);
    if (cost < best_cost) {
      best = w;
      best_cost = cost;
    }
  }
  return best;
}

// Raw rows that a token workgroup quantises into LDS.
constexpr int64_t kTokenLds = 48 * 1024;

int split_of(int64_t tiles, int64_t Q) {
  const int64_t room = device_cus() / tiles;
  return (int)std::max<int64_t>(1, std::min(room, Q / 2));
}

}  // namespace

MxPlan mx_plan(int64_t M, int64_t P, int E, int64_t N, int64_t K, int fmt) {
  MxPlan p;
  const int64_t Q = mx_supers(K), cus = device_cus();
  const int64_t row = mx_row_bytes(K, fmt) + mx_row_scale_bytes(K);
  const int64_t per = E ? ceil_div(P, E) : P;  // rows of a group, evenly shared
  const int64_t most = std::min<int64_t>(P, 16);
  if (E ? P <= 16 : P <= 4) p.path = most * row <= kTokenLds ? kMxToken : kMxStream;
  else if (per <= 16) p.path = kMxStream;
  else p.path = kMxTile;
  if (p.path != kMxTile) {
    p.bm = 16;
    p.bn = 16;
    p.waves = stream_waves(Q);
  } else {
    auto work = [&](const TileShape& s) { return (E ? P / s.bm + E / 2 : ceil_div(P, s.bm)) * ceil_div(N, s.bn); };
    TileShape s = kLarge;
    if (per <= 64) s = kSmall;
    else if (per <= 128 || work(kLarge) * 4 < cus * 3) s = kMiddle;
    p.bm = s.bm;
    p.bn = s.bn;
    if (!E) p.ksplit = split_of(work(s), Q);
  }
  auto take = [&](int64_t bytes) {
    const int64_t at = p.bytes;
    p.bytes += round_up256(bytes);
    return at;
  };
  if (p.path != kMxToken) {
    p.codes = take(M * mx_row_bytes(K, fmt));
    p.scales = take(M * mx_row_scale_bytes(K));
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
  int64_t n = round_up256(M * mx_row_bytes(K, fmt)) + round_up256(M * mx_row_scale_bytes(K));
  if (E) return n + 256 + round_up256(mx_tile_slots(P, E, 16) * (int64_t)sizeof(MxTile));
  // ksplit times the tiles is at most the compute units, and at most half the supers a tile
  int64_t parts = 0;
  const int64_t Q = mx_supers(K);
  for (const TileShape& s : {kSmall, kMiddle, kLarge}) {
    const int64_t strips = ceil_div(N, s.bn);
    if (strips * 2 > device_cus() || Q < 4) continue;  // never split
    parts = std::max(parts, std::min<int64_t>((int64_t)device_cus() * s.bm * s.bn, Q / 2 * M * N));
  }
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
  if (N * mx_steps(K) * kMxStep > kMostOffset)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "the codes are addressed with 32-bit offsets (N=%lld K=%lld)",
                (long long)N, (long long)K);
  return W4A8_OK;
}
// A launch has fewer than 2^32 threads.
int check_launch(const MxPlan& p, int64_t P, int32_t E, int64_t N) {
  const int64_t tiles = E ? mx_tile_slots(P, E, p.bm) : ceil_div(P, p.bm);
  const int64_t threads = p.path == kMxTile ? (p.bm == 256 ? 512 : 256) : 64 * p.waves;
  if (tiles * ceil_div(N, p.bn) * threads >= (int64_t)1 << 32)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "%lld x %lld outputs in one call", (long long)P, (long long)N);
  return W4A8_OK;
}
int check_linear(int64_t M, int64_t N, int64_t K, int32_t act) {
  if (int rc = check_product(M, N, K, act)) return rc;
  return check_launch(mx_plan(M, M, 0, N, K, act), M, 0, N);
}
int check_grouped(int64_t M, int64_t P, int32_t E, int64_t N, int64_t K, int32_t act) {
  if (int rc = check_rows(M)) return rc;
  if (E < 1 || E > kMxMaxGroups) return fail(W4A8_ERR_INVALID_ARG, "E=%d out of [1, %d]", (int)E, kMxMaxGroups);
  if (int rc = check_product(P, N, K, act)) return rc;
  if (N * E > (int64_t)1 << 31) return fail(W4A8_ERR_INVALID_ARG, "N=%lld times E=%d out of range", (long long)N, (int)E);
  return check_launch(mx_plan(M, P, E, N, K, act), P, E, N);
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
  a.ldx = (int)mx_row_bytes(c.K, c.act);
  a.lds = (int)mx_row_scale_bytes(c.K);
  a.nb = (int)(c.N / 16);
  a.bm = p.bm;
  a.ksplit = p.ksplit;
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
    const hipError_t e = launch_mx_rows(q, c.offsets, c.E, c.P, p.bm, const_cast<int*>(a.ntiles),
                                        const_cast<MxTile*>(a.tiles), st);
    if (e != hipSuccess) return e;
  }
  if (p.path == kMxTile) {
    a.strips = (int)ceil_div(c.N, p.bn);
    return launch_mx_tile(a, p, c.act, c.gated, st);
  }
  a.strips = a.nb / (c.gated ? 2 : 1);
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
  if (int rc = check_linear(M, N, K, act)) return rc;
  return fill_plan(mx_plan(M, M, 0, N, K, act), plan);
}

size_t w4a8_mx_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t act) {
  if (check_linear(M, N, K, act)) return 0;
  return (size_t)workspace_bound(M, M, 0, N, K, act);
}

int w4a8_mx_linear(const void* x, int32_t x_dtype, int32_t act, int32_t rule, const void* packed,
                   size_t packed_bytes, int64_t M, int64_t N, int64_t K, uint16_t* y, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (int rc = check_linear(M, N, K, act)) return rc;
  if (int rc = check_dtype(x_dtype)) return rc;
  if (int rc = check_rule(rule)) return rc;
  const size_t wb = (size_t)mx_weight_bytes(N, K);
  if (packed && packed_bytes < wb)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "packed buffer %zu bytes, need %zu", packed_bytes, wb);
  const MxPlan p = mx_plan(M, M, 0, N, K, act);
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
  if (int rc = check_grouped(M, P, E, N, K, act)) return rc;
  return fill_plan(mx_plan(M, P, E, N, K, act), plan);
}

size_t w4a8_mx_grouped_linear_workspace_bytes(int64_t M, int64_t P, int32_t E, int64_t N, int64_t K, int32_t act) {
  if (check_grouped(M, P, E, N, K, act)) return 0;
  return (size_t)workspace_bound(M, P, E, N, K, act);
}

int w4a8_mx_grouped_linear(const void* x, int32_t x_dtype, int32_t act, int32_t rule, const void* packed,
                           size_t packed_bytes, const int32_t* offsets, const int32_t* rows, int64_t M, int64_t P,
                           int32_t E, int64_t N, int64_t K, int32_t gated, uint16_t* y, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (int rc = check_grouped(M, P, E, N, K, act)) return rc;
  if (int rc = check_dtype(x_dtype)) return rc;
  if (int rc = check_rule(rule)) return rc;
  if (gated && N % 32)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "N=%lld gates and values are not a multiple of 32", (long long)N);
  if (!rows && M != P)
    return fail(W4A8_ERR_INVALID_ARG, "without rows M=%lld and P=%lld must agree", (long long)M, (long long)P);
  if (rows && M * mx_row_bytes(K, act) > kMostOffset)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "rows by index are addressed with 32-bit offsets (M=%lld K=%lld)",
                (long long)M, (long long)K);
  const size_t wb = (size_t)mx_weight_bytes(E * N, K);
  if (packed && packed_bytes < wb)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "packed buffer %zu bytes, need %zu", packed_bytes, wb);
  const MxPlan p = mx_plan(M, P, E, N, K, act);
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
