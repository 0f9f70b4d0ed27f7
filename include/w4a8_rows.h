/*
 * w4a8_rows.h — C ABI of the operators whose weights depend on the row: a
 * router, the expert MLP it feeds, and a shared projection with a low-rank
 * adapter per row.  The weights of the experts and the projection are W4A8
 * packed weights (w4a8.h); status codes, activation dtypes, alignment, stream,
 * ownership and determinism are as stated there.
 */
#ifndef W4A8_ROWS_H
#define W4A8_ROWS_H

#include "w4a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * How a call runs, chosen from its sizes and the device's compute units (256
 * on MI355X): host only, for tests and tuning; nothing is enqueued.  Kernels:
 */
#define W4A8_ROWS_TOKEN 1  /* a single token's experts, a single adapted row */
#define W4A8_ROWS_STREAM 2 /* weights streamed past activations staged at once */
#define W4A8_ROWS_RUN 3    /* weights streamed, activations in slices */
#define W4A8_ROWS_TILE 4   /* 256 rows x 256 channels on the matrix cores */
typedef struct {
  int64_t tokens;       /* of a pass; more of them run in several */
  int32_t tile_rows;    /* (token, slot) pairs that a tile of one expert holds */
  int32_t up_path;      /* W4A8_ROWS_* of the up and the down product */
  int32_t down_path;
  int32_t down_columns; /* 16-channel columns that a wavefront of the down product
                           takes one after another (STREAM, RUN) */
} w4a8_moe_mlp_plan_t;
typedef struct {
  int64_t rows;         /* of a pass */
  int32_t path;         /* W4A8_ROWS_* of the shared product */
  int32_t ksplit;       /* its slices of the inputs */
  int32_t in_epilogue;  /* the product's kernel adds the adapters, else a reduction does */
  int32_t sorted;       /* rows taken in the order of their adapters */
} w4a8_lora_linear_plan_t;

/* score functions of w4a8_moe_route */
#define W4A8_SCORE_SOFTMAX 0
#define W4A8_SCORE_SIGMOID 1

/*
 * w4a8_moe_route — the k experts of each token and their weights.
 *   logits   device [M][E], bfloat16 (W4A8_BF16) or float (W4A8_F32)
 *   bias     device float [E], or NULL
 *   ids      device int32 [M][k]: the chosen experts, best first; -1 where
 *            fewer than k can be chosen
 *   weights  device float [M][k]: their weights; 0 beside an id of -1
 * With p the softmax (over the experts) or the sigmoid of the logits and
 * c = p + bias (the bias takes part in the choice only):
 *   - n_groups > 1: the E experts form n_groups runs of E / n_groups; a
 *     group's value is the sum of its group_top (1 or 2) largest c, and the
 *     topk_groups groups of largest value stay;
 *   - the k experts of largest c among those that stay are chosen;
 *   - weights = p of the chosen, divided by their sum if renormalize (0 where
 *     that sum is 0), times scale.
 * Ties go to the lowest index.  The choice is made on values of 64 bits (on
 * the logits where no bias and no sum enters); p and the weights are float.
 * An expert whose logit is minus infinity or NaN is off: it is never chosen
 * and its p is 0.  Plus infinity counts as the largest finite value.  A bias
 * of minus infinity or NaN takes its expert out of the choice.
 * Requirements: 1 <= M <= 2^24, 1 <= E <= 1024, 1 <= k <= 64, k <= the
 * experts of topk_groups groups, 1 <= topk_groups <= n_groups <= 64,
 * E % n_groups == 0, group_top 1 or 2 and at most E / n_groups.
 */
int w4a8_moe_route(const void* logits, int32_t dtype, const float* bias, int64_t M, int32_t E,
                   int32_t k, int32_t score, int32_t n_groups, int32_t topk_groups,
                   int32_t group_top, int32_t renormalize, float scale, int32_t* ids,
                   float* weights, void* stream);

/*
 * w4a8_moe_mlp — the gated MLP of each token's experts, summed by weight:
 *   h[m][j] = bf16( silu(gate) * up ),  (gate, up) = W4A8 product of x[m] and
 *             expert ids[m][j]'s up weight
 *   y[m]    = bf16( sum_j weights[m][j] * (W4A8 product of h[m][j] and that
 *             expert's down weight) )
 * Both products quantise their input rows by the rule of w4a8_quant_act; the
 * slots are summed in float32 in slot order.
 *   x        device [M][K], bfloat16 or float
 *   up       packed weight of E * 2 I channels and K inputs: expert e has
 *            channels [2 I e, 2 I (e + 1)), I gate channels, then I up channels
 *   down     packed weight of E * K channels and I inputs: expert e has
 *            channels [K e, K (e + 1))
 *   ids      device int32 [M][k]; a slot whose id lies outside [0, E) adds
 *            nothing (an expert held elsewhere); a token with no slot left
 *            gives zeros
 *   weights  device float [M][k]
 *   y        device bfloat16 bits [M][K]
 *   workspace  device scratch of w4a8_moe_mlp_workspace_bytes(M, k, E, I, K)
 *            bytes; contents on entry are ignored.  The size for M tokens
 *            serves every smaller number of them
 * The result of a token does not depend on the other tokens of the call
 * except through the kernel that their number selects.  The experts' rows are
 * counted on the device: the call never synchronises and can be captured.
 * Requirements: 1 <= M <= 2^24, 1 <= k <= 64, 1 <= E <= 1024, I % 128 == 0,
 * K % 128 == 0, one expert's 2 I K / 2 code bytes below 2^31.
 */
int w4a8_moe_mlp_plan(int64_t M, int32_t k, int32_t E, int64_t I, int64_t K, w4a8_moe_mlp_plan_t* plan);
size_t w4a8_moe_mlp_workspace_bytes(int64_t M, int32_t k, int32_t E, int64_t I, int64_t K);
int w4a8_moe_mlp(const void* x, int32_t x_dtype, const void* up, size_t up_bytes, const void* down,
                 size_t down_bytes, const int32_t* ids, const float* weights, int64_t M, int32_t k,
                 int32_t E, int64_t I, int64_t K, uint16_t* y, void* workspace,
                 size_t workspace_bytes, void* stream);

/*
 * w4a8_lora_linear — a shared W4A8 linear with a low-rank adapter per row:
 *   y[m] = bf16( w4a8 sum of x[m]  +  scale[l] * (x[m] A[l]^T) B[l]^T ),  l = ids[m]
 * where the first term is the unrounded sum of w4a8_gemm on the quantised row
 * and the adapter sees the row as given.  Adapter sums are float32 (the
 * operands of the matrix cores are bf16: exact for A, B and bf16 rows, two
 * bf16 parts, 16 significant bits, for float rows and for x A^T).
 *   x       device [M][K], bfloat16 or float
 *   packed  packed weight of N channels and K inputs
 *   A       device bfloat16 [L][R][K];  B  device bfloat16 [L][N][R]
 *   scale   device float [L]
 *   ids     device int32 [M]; a row whose id lies outside [0, L) has no adapter
 *   y       device bfloat16 bits [M][N]
 *   workspace  device scratch of w4a8_lora_linear_workspace_bytes(M, N, K, L, R) bytes;
 *           contents on entry are ignored.  The size for M rows serves every
 *           smaller number of them (few rows are split further along K and
 *           can take more room than many)
 * Requirements: as w4a8_linear; R % 8 == 0, 8 <= R <= 128, 1 <= L <= 65536,
 * N * K / 2 below 2^31 bytes.
 */
int w4a8_lora_linear_plan(int64_t M, int64_t N, int64_t K, int32_t L, int32_t R, w4a8_lora_linear_plan_t* plan);
size_t w4a8_lora_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t L, int32_t R);
int w4a8_lora_linear(const void* x, int32_t x_dtype, const void* packed, size_t packed_bytes,
                     const uint16_t* A, const uint16_t* B, const float* scale, const int32_t* ids,
                     int64_t M, int64_t N, int64_t K, int32_t L, int32_t R, uint16_t* y,
                     void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A8_ROWS_H */
