/*
 * moe_experts.h -- C ABI of libmoe_dispatch.so, second part: the experts'
 * matrix product over the rows that moe_dispatch placed, and what training
 * needs around it (the router's balance loss, the gradients of the router, of
 * the combine and of the expert product).  moe_dispatch.h holds the path
 * itself and every convention: device pointers, the caller's memory and
 * stream, no allocation, no synchronisation, no state between calls; errors
 * the host can see are returned and launch nothing.  Every call can be
 * captured in a HIP graph; a workspace belongs to one call at a time, so
 * graphs that may run at once need workspaces of their own.  Unless a call
 * says otherwise its outputs overlap none of its other buffers.
 *
 * The gradient of moe_dispatch itself (each token's gradient is the sum of its
 * pairs' rows) is moe_combine with all weights one.
 *
 * Results are deterministic: no order of summation depends on timing.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_dispatch.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of the expert product, y = act(z):
 *   SILU    z / (1 + exp(-z))
 *   GELU    z/2 * (1 + erf(z / sqrt 2))
 *   SWIGLU  silu(gate) * up, gate the first half of z's columns, up the second */
typedef enum {
  MOE_ACT_NONE = 0,
  MOE_ACT_SILU = 1,
  MOE_ACT_GELU = 2,
  MOE_ACT_SWIGLU = 3
} moe_activation;

#define MOE_MAX_FEATURES (1 << 22)
/* A tile's rows past the last one still have a 32-bit number. */
#define MOE_MAX_EXPERT_ROWS (INT32_MAX - 65535)
/* Tokens, and sequences, of the router's calls. */
#define MOE_MAX_ROUTED (1 << 30)

/* One linear layer held by every expert (host struct, read during the call).
 * P below is the number of columns before the activation: 2 * out_features for
 * MOE_ACT_SWIGLU, else out_features.  Neither K nor P exceeds MOE_MAX_FEATURES. */
typedef struct {
  int32_t in_features;  /* K > 0: K % 8 == 0; fp8 payload: K % 128 == 0 */
  int32_t out_features; /* F > 0: F % 8 == 0; fp8 payload: F % 128 == 0 */
  int32_t activation;   /* moe_activation */
} moe_linear;

/*
 * moe_expert_matmul -- every expert multiplies the rows of its segment with
 * its own weights ([EFA] MoE all-to-all over EFA: the grouped GEMM between
 * dispatch and combine), with bias, activation and residual applied before
 * the one rounding of the result:
 *
 *   z = x[row] * weight[e]^T + bias[e],   y[row] = bf16(act(z) + residual[row])
 *
 *   shape         as given to moe_dispatch (after moe_dispatch_sources with
 *                 num_tokens = S*T); its payload says what x holds.  No more
 *                 than num_tokens * top_k rows may be placed: the launch is
 *                 sized for these, rows past them may stay unwritten.
 *                 hidden is checked but not used: the columns are the
 *                 linear's, so the same shape serves both projections.
 *   x, x_scales   [rows][K] in the receive layout: bf16, or e4m3 codes with
 *                 [rows][K/128] fp32 scales (NULL for bf16).
 *   layout        expert_counts and expert_offsets are read (on the device:
 *                 the work follows the counts, not the buffer's size).  NULL
 *                 for a dense product, with num_experts == top_k == 1: all
 *                 num_tokens rows belong to the one expert (a shared expert).
 *   weight        [E][P][K] bf16, or e4m3 codes with weight_scales
 *                 [E][P/128][K/128] fp32, one per 128 x 128 block (NULL for
 *                 bf16).  16-byte aligned, like every row buffer here.
 *   bias          [E][P] fp32, or NULL.
 *   residual      [rows][F] bf16, or NULL; may be y itself.
 *   y             [rows][F] bf16 out (for either payload).
 *   pre           [rows][P] bf16 out, bf16(z), for the backward pass; or NULL.
 * bf16: sums are fp32.  fp8: the products of each 128 columns are summed first
 * and then scaled and added in fp32; that first sum is the matrix instruction's,
 * which cuts products below 2^-13 of the largest among 8 neighbouring columns
 * (each factor was itself rounded to 2^-4).  Rows of no segment are neither read for a result nor
 * written.
 * Errors: MOE_ERR_INVALID_ARG; MOE_ERR_UNSUPPORTED for E, k, features or rows
 * (MOE_MAX_EXPERT_ROWS) past the library's limits, and for outputs of more tiles
 * (16 x 64 or larger) than one launch has: 2^24, fp8 2^23.
 */
moe_status moe_expert_matmul(const moe_shape *shape, const moe_linear *linear, const void *x,
                             const float *x_scales, const moe_layout *layout,
                             const void *weight, const float *weight_scales,
                             const float *bias, const void *residual, void *y, void *pre,
                             hipStream_t stream);

/* Bytes of device workspace moe_expert_matmul_backward needs (0 for invalid
 * arguments or when none is needed).  Host function. */
size_t moe_expert_matmul_backward_workspace_size(const moe_shape *shape,
                                                 const moe_linear *linear);

/*
 * moe_expert_matmul_backward -- gradients of moe_expert_matmul, bf16 payload
 * only (MOE_ERR_UNSUPPORTED for fp8).  With gz = grad_y * act'(pre):
 *
 *   grad_x[row]    = bf16( gz[row] * weight[e] )                 [rows][K]
 *   grad_weight[e] = bf16( sum over e's rows of gz[row]^T x[row] ) [E][P][K]
 *   grad_bias[e]   = sum over e's rows of gz[row], fp32          [E][P]
 *
 *   Any of the three may be NULL (not wanted).  grad_x is written on placed
 *   rows only; an expert without rows gets zeros.  The residual's gradient is
 *   grad_y itself.
 *   pre           as moe_expert_matmul wrote it; NULL (and not read) for
 *                 MOE_ACT_NONE.
 *   x             read for grad_weight only, weight for grad_x only (else NULL
 *                 is allowed).
 *   workspace     moe_expert_matmul_backward_workspace_size bytes, 16-byte
 *                 aligned; contents need no initialisation.  It holds gz
 *                 rounded to bf16, which the two products read (grad_bias is
 *                 summed before that rounding), and parts of those sums.  NULL
 *                 is allowed for MOE_ACT_NONE without grad_bias.
 * Errors as moe_expert_matmul; MOE_ERR_UNSUPPORTED also for a grad_bias of more
 * than 2^31 - 1 entries and a grad_weight of more than 2^31 - 1 tiles.
 */
moe_status moe_expert_matmul_backward(const moe_shape *shape, const moe_linear *linear,
                                      const void *grad_y, const void *x,
                                      const moe_layout *layout, const void *weight,
                                      const void *pre, void *grad_x, void *grad_weight,
                                      float *grad_bias, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream);

/*
 * moe_combine_backward -- gradients of moe_combine, bf16 payload only
 * (MOE_ERR_UNSUPPORTED for fp8):
 *
 *   grad_y[token_row[t][j]] = bf16( w[t][j] * grad_out[t] )
 *   grad_weights[t][j]      = sum over columns of grad_out[t] * expert_y[token_row[t][j]], fp32
 *
 *   A pair with token_row -1 has grad_weights 0 and no row; rows no pair
 *   reaches are not written.  Either output may be NULL (not wanted, not both);
 *   expert_y is read for grad_weights only, topk_weights for grad_y only.
 */
moe_status moe_combine_backward(const moe_shape *shape, const void *grad_out,
                                const void *expert_y, const moe_layout *layout,
                                const float *topk_weights, void *grad_y,
                                float *grad_weights, hipStream_t stream);

/* Bytes of device workspace moe_balance_loss needs; 0 for invalid arguments or
 * when none is needed.  Host function. */
size_t moe_balance_loss_workspace_size(int32_t T, int32_t E, int32_t num_seqs);

/*
 * moe_balance_loss -- per-expert counts of a routed batch and the loss that
 * balances them.  Tokens form num_seqs sequences; per sequence s, over its n_s
 * tokens that have an expert at all (some id in [0, E)),
 *
 *   c[s][i] = its pairs with id i           P[s][i] = mean of p[t][i]
 *   loss    = coef / num_seqs * sum over s, i of  E * c[s][i] / (k * n_s) * P[s][i]
 *
 *   with p[t] the softmax of the biased logits, or for MOE_SCORE_SIGMOID their
 *   sigmoids over their sum.  A uniform routing gives coef; a sequence without
 *   such a token gives 0.
 *
 *   logits, bias  as given to moe_route_topk.
 *   topk_ids      [T][k]; ids outside [0, E) are not counted, and a token
 *                 without any other takes no part (padding).
 *   seq_offsets   [num_seqs + 1] int32 device, not decreasing: sequence s is
 *                 the tokens seq_offsets[s] .. seq_offsets[s+1] - 1 (values are
 *                 cut to [0, T]); tokens outside every sequence take no part.
 *                 NULL: one sequence of all tokens (num_seqs must be 1).
 *   expert_counts [num_seqs][E] int32 out, c.
 *   expert_probs  [num_seqs][E] fp32 out, P (0 for a sequence without tokens).
 *   seq_tokens    [num_seqs] int32 out, n.
 *   loss          [1] fp32 out.
 *   workspace     moe_balance_loss_workspace_size bytes, 16-byte aligned.
 * Errors: MOE_ERR_INVALID_ARG; MOE_ERR_UNSUPPORTED past MOE_MAX_EXPERTS,
 * MOE_MAX_TOP_K, MOE_MAX_ROUTED tokens or sequences, 2^31 - 1 entries of an
 * output or pairs.
 */
moe_status moe_balance_loss(const float *logits, const float *bias, const int32_t *topk_ids,
                            int32_t T, int32_t E, int32_t k, int32_t score,
                            const int32_t *seq_offsets, int32_t num_seqs, float coef,
                            int32_t *expert_counts, float *expert_probs, int32_t *seq_tokens,
                            float *loss, void *workspace, size_t workspace_bytes,
                            hipStream_t stream);

/* Bytes of device workspace moe_route_backward needs (only for grad_bias); 0
 * for invalid arguments or when none is needed.  Host function. */
size_t moe_route_backward_workspace_size(int32_t T, int32_t E);

/*
 * moe_route_backward -- gradient of the router's logits: of the weights that
 * moe_route_topk or moe_route_topk_grouped gave (the choice of experts is
 * constant) and of moe_balance_loss (the counts are constant).  Either part
 * may be left out, not both.
 *
 *   logits, bias, topk_ids, topk_weights, score   as of the forward calls.
 *   grad_weights  [T][k] fp32, or NULL for no routed part (topk_weights may
 *                 then be NULL).  Pairs with an id outside [0, E) have no
 *                 gradient, whatever stands in grad_weights.
 *   expert_counts, seq_tokens   as moe_balance_loss wrote them, or the sums
 *                 over the ranks of a data-parallel group; both NULL for no
 *                 balance part (seq_offsets and num_seqs are then not used).
 *   grad_loss     [1] fp32 device, gradient of the loss value; NULL means 1.
 *   grad_logits   [T][E] fp32 out, every entry written.
 *   grad_bias     [E] fp32 out, the sum of grad_logits over tokens; or NULL.
 *   workspace     moe_route_backward_workspace_size bytes, 16-byte aligned;
 *                 only read with grad_bias (else NULL is allowed).
 * Errors as moe_balance_loss.
 */
moe_status moe_route_backward(const float *logits, const float *bias, const int32_t *topk_ids,
                              const float *topk_weights, const float *grad_weights, int32_t T,
                              int32_t E, int32_t k, int32_t score, const int32_t *seq_offsets,
                              int32_t num_seqs, float coef, const int32_t *expert_counts,
                              const int32_t *seq_tokens, const float *grad_loss,
                              float *grad_logits, float *grad_bias, void *workspace,
                              size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
