// Host entry points of include/w4a8_rows.h: argument checks, workspace layout
// and launches.  Every check runs before anything is enqueued.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/w4a8_rows.h"
#include "experts.h"
#include "lora.h"
#include "route.h"

using namespace w4a8;

namespace {

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

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

// Every pointer set and aligned; no written buffer meets another one.
template <int NI, int NO>
int check_buffers(const Span (&in)[NI], const Span (&out)[NO]) {
  for (const Span& s : in)
    if (s.bytes && !s.p) return fail(W4A8_ERR_INVALID_ARG, "null input pointer");
  for (const Span& s : out)
    if (s.bytes && !s.p) return fail(W4A8_ERR_INVALID_ARG, "null output pointer");
  for (const Span& s : in)
    if (s.bytes && !aligned16(s.p)) return fail(W4A8_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  for (const Span& s : out)
    if (s.bytes && !aligned16(s.p)) return fail(W4A8_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  for (int o = 0; o < NO; ++o) {
    for (const Span& s : in)
      if (overlap(out[o], s)) return fail(W4A8_ERR_INVALID_ARG, "an output or the workspace aliases an input");
    for (int q = o + 1; q < NO; ++q)
      if (overlap(out[o], out[q])) return fail(W4A8_ERR_INVALID_ARG, "outputs or the workspace alias each other");
  }
  return W4A8_OK;
}

int check_rows(int64_t M) {
  if (M <= 0 || M > ((int64_t)1 << 24)) return fail(W4A8_ERR_INVALID_ARG, "M=%lld out of range", (long long)M);
  return W4A8_OK;
}

int check_dtype(int32_t d) {
  if (d != W4A8_BF16 && d != W4A8_F32) return fail(W4A8_ERR_INVALID_ARG, "unknown activation dtype %d", (int)d);
  return W4A8_OK;
}

size_t value_bytes(int32_t d) { return d == W4A8_F32 ? 4 : 2; }

PackedView view(const void* packed, int64_t N, int64_t K) {
  const uint8_t* base = static_cast<const uint8_t*>(packed);
  return PackedView{base, base + zeros_offset(N, K),
                    reinterpret_cast<const float*>(base + scales_offset(N, K))};
}

int check_moe(int64_t M, int32_t k, int32_t E, int64_t I, int64_t K) {
  if (int rc = check_rows(M)) return rc;
  if (k < 1 || k > kMaxTopK) return fail(W4A8_ERR_INVALID_ARG, "k=%d out of [1, %d]", (int)k, kMaxTopK);
  if (E < 1 || E > kMaxExperts) return fail(W4A8_ERR_INVALID_ARG, "E=%d out of [1, %d]", (int)E, kMaxExperts);
  if (I <= 0 || K <= 0 || I > ((int64_t)1 << 24) || K > ((int64_t)1 << 24))
    return fail(W4A8_ERR_INVALID_ARG, "I=%lld K=%lld out of range", (long long)I, (long long)K);
  if (I % kGroup || K % kGroup)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "I=%lld and K=%lld must be multiples of 128", (long long)I,
                (long long)K);
  if (I * K > kPrefillMaxBytes || k * (I > K ? I : K) > kPrefillMaxBytes)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "one expert is addressed with 32-bit offsets (I=%lld K=%lld)",
                (long long)I, (long long)K);
  if (w4a8_packed_weight_bytes(E * 2 * I, K, kGroup) == 0 || w4a8_packed_weight_bytes(E * K, I, kGroup) == 0)
    return W4A8_ERR_INVALID_ARG;  // (its message is set)
  if (moe_plan(M, k, E, I, K).tokens < 1)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "a single token exceeds the 32-bit offsets (k=%d I=%lld K=%lld)",
                (int)k, (long long)I, (long long)K);
  return W4A8_OK;
}

int check_lora(int64_t M, int64_t N, int64_t K, int32_t L, int32_t R) {
  if (w4a8_packed_weight_bytes(N, K, kGroup) == 0)  // (its message is set)
    return N <= 0 || K <= 0 ? W4A8_ERR_INVALID_ARG : W4A8_ERR_UNSUPPORTED_SHAPE;
  if (int rc = check_rows(M)) return rc;
  if (L < 1 || L > 65536) return fail(W4A8_ERR_INVALID_ARG, "L=%d out of [1, 65536]", (int)L);
  if (R < 8 || R > kMaxRank || R % 8)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "rank %d is not a multiple of 8 in [8, %d]", (int)R, kMaxRank);
  if (N * K / 2 > kPrefillMaxBytes || K > kPrefillMaxBytes)
    return fail(W4A8_ERR_UNSUPPORTED_SHAPE, "the codes are addressed with 32-bit offsets (N=%lld K=%lld)",
                (long long)N, (long long)K);
  return W4A8_OK;
}

}  // namespace

extern "C" {

int w4a8_moe_route(const void* logits, int32_t dtype, const float* bias, int64_t M, int32_t E,
                   int32_t k, int32_t score, int32_t n_groups, int32_t topk_groups,
                   int32_t group_top, int32_t renormalize, float scale, int32_t* ids,
                   float* weights, void* stream) {
  if (int rc = check_rows(M)) return rc;
  if (int rc = check_dtype(dtype)) return rc;
  if (E < 1 || E > kMaxExperts) return fail(W4A8_ERR_INVALID_ARG, "E=%d out of [1, %d]", (int)E, kMaxExperts);
  if (score != W4A8_SCORE_SOFTMAX && score != W4A8_SCORE_SIGMOID)
    return fail(W4A8_ERR_INVALID_ARG, "unknown score function %d", (int)score);
  if (n_groups < 1 || n_groups > kMaxGroups || E % n_groups)
    return fail(W4A8_ERR_INVALID_ARG, "%d groups do not divide %d experts (at most %d)", (int)n_groups,
                (int)E, kMaxGroups);
  if (topk_groups < 1 || topk_groups > n_groups)
    return fail(W4A8_ERR_INVALID_ARG, "topk_groups=%d out of [1, %d]", (int)topk_groups, (int)n_groups);
  const int per = E / n_groups;
  if (group_top < 1 || group_top > 2 || group_top > per)
    return fail(W4A8_ERR_INVALID_ARG, "group_top=%d: 1 or 2, at most a group's %d experts", (int)group_top, per);
  if (k < 1 || k > kMaxTopK || k > per * topk_groups)
    return fail(W4A8_ERR_INVALID_ARG, "k=%d out of [1, %d]", (int)k,
                per * topk_groups < kMaxTopK ? per * topk_groups : kMaxTopK);
  if (!std::isfinite(scale)) return fail(W4A8_ERR_INVALID_ARG, "scale is not finite");
  const size_t mk = (size_t)M * k * 4;
  const Span in[] = {{logits, (size_t)M * E * value_bytes(dtype)}, {bias, bias ? (size_t)E * 4 : 0}};
  const Span out[] = {{ids, mk}, {weights, mk}};
  if (int rc = check_buffers(in, out)) return rc;
  (void)hipGetLastError();
  const RouteArgs a{logits, dtype,  bias,        M,         E,     k,   score == W4A8_SCORE_SOFTMAX,
                    renormalize != 0, n_groups, topk_groups, group_top, scale, ids, weights};
  return finish(launch_route(a, static_cast<hipStream_t>(stream)), "route launch");
}

size_t w4a8_moe_mlp_workspace_bytes(int64_t M, int32_t k, int32_t E, int64_t I, int64_t K) {
  if (check_moe(M, k, E, I, K)) return 0;
  return (size_t)moe_plan(M, k, E, I, K).bytes;
}

int w4a8_moe_mlp(const void* x, int32_t x_dtype, const void* up, size_t up_bytes, const void* down,
                 size_t down_bytes, const int32_t* ids, const float* weights, int64_t M, int32_t k,
                 int32_t E, int64_t I, int64_t K, uint16_t* y, void* workspace,
                 size_t workspace_bytes, void* stream) {
  if (int rc = check_moe(M, k, E, I, K)) return rc;
  if (int rc = check_dtype(x_dtype)) return rc;
  const size_t ub = (size_t)packed_bytes(E * 2 * I, K), db = (size_t)packed_bytes(E * K, I);
  if (up && up_bytes < ub)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "up weight %zu bytes, need %zu", up_bytes, ub);
  if (down && down_bytes < db)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "down weight %zu bytes, need %zu", down_bytes, db);
  const MoePlan p = moe_plan(M, k, E, I, K);
  if (!workspace || workspace_bytes < (size_t)p.bytes)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "workspace %zu bytes, need %zu", workspace_bytes, (size_t)p.bytes);
  const size_t vb = value_bytes(x_dtype), mk = (size_t)M * k * 4;
  const Span in[] = {{x, (size_t)M * K * vb}, {up, ub}, {down, db}, {ids, mk}, {weights, mk}};
  const Span out[] = {{y, (size_t)M * K * 2}, {workspace, (size_t)p.bytes}};
  if (int rc = check_buffers(in, out)) return rc;
  (void)hipGetLastError();
  hipError_t e = hipSuccess;
  for (int64_t m0 = 0; m0 < M && e == hipSuccess; m0 += p.tokens) {
    const int64_t mc = M - m0 < p.tokens ? M - m0 : p.tokens;
    const MoeArgs a{static_cast<const uint8_t*>(x) + (size_t)m0 * K * vb,
                    x_dtype,
                    view(up, E * 2 * I, K),
                    view(down, E * K, I),
                    ids + m0 * k,
                    weights + m0 * k,
                    mc,
                    k,
                    E,
                    I,
                    K,
                    y + m0 * K,
                    static_cast<uint8_t*>(workspace)};
    e = launch_moe(a, p, static_cast<hipStream_t>(stream));
  }
  return finish(e, "expert MLP launch");
}

int w4a8_moe_mlp_plan(int64_t M, int32_t k, int32_t E, int64_t I, int64_t K, w4a8_moe_mlp_plan_t* plan) {
  if (!plan) return fail(W4A8_ERR_INVALID_ARG, "null plan");
  if (int rc = check_moe(M, k, E, I, K)) return rc;
  const MoePlan p = moe_plan(M, k, E, I, K);
  plan->tokens = p.tokens;
  plan->tile_rows = p.bm;
  plan->up_path = p.up;
  plan->down_path = p.down;
  plan->down_columns = p.down == kStreamPath || p.down == kRunPath ? down_columns(p, p.tokens * k, E, I, K) : 1;
  return report_error(W4A8_OK, "");
}

size_t w4a8_lora_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t L, int32_t R) {
  if (check_lora(M, N, K, L, R)) return 0;
  return (size_t)lora_workspace(M, N, K, L, R);
}

int w4a8_lora_linear_plan(int64_t M, int64_t N, int64_t K, int32_t L, int32_t R, w4a8_lora_linear_plan_t* plan) {
  if (!plan) return fail(W4A8_ERR_INVALID_ARG, "null plan");
  if (int rc = check_lora(M, N, K, L, R)) return rc;
  const LoraPlan p = lora_plan(M, N, K, L, R);
  plan->rows = p.rows;
  plan->path = p.path;
  plan->ksplit = p.ksplit;
  plan->in_epilogue = p.parts < 0;
  plan->sorted = p.sorted;
  return report_error(W4A8_OK, "");
}

int w4a8_lora_linear(const void* x, int32_t x_dtype, const void* packed, size_t packed_bytes_,
                     const uint16_t* A, const uint16_t* B, const float* scale, const int32_t* ids,
                     int64_t M, int64_t N, int64_t K, int32_t L, int32_t R, uint16_t* y,
                     void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_lora(M, N, K, L, R)) return rc;
  if (int rc = check_dtype(x_dtype)) return rc;
  const size_t wb = (size_t)packed_bytes(N, K);
  if (packed && packed_bytes_ < wb)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "packed buffer %zu bytes, need %zu", packed_bytes_, wb);
  const LoraPlan p = lora_plan(M, N, K, L, R);
  if (!workspace || workspace_bytes < (size_t)p.bytes)
    return fail(W4A8_ERR_BUFFER_TOO_SMALL, "workspace %zu bytes, need %zu", workspace_bytes, (size_t)p.bytes);
  const size_t vb = value_bytes(x_dtype);
  const Span in[] = {{x, (size_t)M * K * vb},           {packed, wb},
                     {A, (size_t)L * R * K * 2},        {B, (size_t)L * N * R * 2},
                     {scale, (size_t)L * 4},            {ids, (size_t)M * 4}};
  const Span out[] = {{y, (size_t)M * N * 2}, {workspace, (size_t)p.bytes}};
  if (int rc = check_buffers(in, out)) return rc;
  (void)hipGetLastError();
  hipError_t e = hipSuccess;
  for (int64_t m0 = 0; m0 < M && e == hipSuccess; m0 += p.rows) {
    const int64_t mc = M - m0 < p.rows ? M - m0 : p.rows;
    const LoraArgs a{static_cast<const uint8_t*>(x) + (size_t)m0 * K * vb,
                     x_dtype,
                     view(packed, N, K),
                     A,
                     B,
                     scale,
                     ids + m0,
                     mc,
                     N,
                     K,
                     L,
                     R,
                     y + m0 * N,
                     static_cast<uint8_t*>(workspace)};
    e = launch_lora(a, p, static_cast<hipStream_t>(stream));
  }
  return finish(e, "adapter linear launch");
}

}  // extern "C"
