/*
 * moe_ffn.h -- C ABI of libmoe_dispatch.so, third part: an expert layer whose
 * products run in 8 bits, served and trained.  The RMS norm in front of the
 * router and its gradient, 8-bit weights from the master weights, and the gated
 * feed-forward block of the experts with its gradient.  moe_dispatch.h holds the
 * path itself and every convention: device pointers, the caller's memory and
 * stream, no allocation, no synchronisation, no state between calls; errors the
 * host can see are returned and launch nothing.  Every call can be captured in a
 * HIP graph; a workspace belongs to one call at a time, so graphs that may run at
 * once need workspaces of their own.  Unless a call says otherwise its outputs
 * overlap none of its other buffers.
 *
 * 8-bit rows and weights are what moe_dispatch and moe_expert_matmul take: OCP
 * e4m3 codes with one fp32 scale for 128 neighbouring columns of a row, or for a
 * 128 x 128 block of a weight:
 *
 *   scale = fp32( max|v| / 448 ),  code = e4m3( fp32( v / scale ) ), to nearest even
 *
 * and zeros where the scale is 0.  A NaN makes its whole block and the scale NaN;
 * an infinity makes the scale infinite, its own code NaN and the others 0.
 *
 * Results are deterministic: no order of summation depends on timing.
 */
#ifndef MOE_FFN_H
#define MOE_FFN_H

#include "moe_dispatch.h"
#include "moe_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_MAX_NORM_COLUMNS 65536

/*
 * moe_rms_norm -- adds the residual and normalises each row:
 *
 *   t = bf16( x + residual ),  r = 1 / sqrt( mean(t^2) + eps ),  v = t * r * weight
 *
 *   x, residual   [T][H] bf16; residual NULL: t = x.
 *   weight        [H] fp32.
 *   total         [T][H] bf16 out, t (the residual stream); or NULL.
 *   y             [T][H] bf16 out, v rounded once (for moe_dispatch and the
 *                 router); or NULL.
 *   codes, scales [T][H] e4m3 and [T][H/128] fp32 out, v in 8 bits, rounded once
 *                 (for a shared expert); both or neither; H % 128 == 0.
 *   inv_rms       [T] fp32 out, r (for the backward pass); or NULL.
 *   total, y may be x or residual themselves (not each other).
 * Squares are summed in fp32, where they leave its range those of the row times
 * 2^80 or 2^-80: any finite row will do.  Without eps a row of zeros, or of less than
 * 2^-127, has no r in fp32.
 * At least one output.  H % 8 == 0; row buffers and weight are 16-byte aligned.
 * Errors: MOE_ERR_INVALID_ARG; MOE_ERR_UNSUPPORTED for H > MOE_MAX_NORM_COLUMNS.
 */
moe_status moe_rms_norm(const void *x, const void *residual, const float *weight, int32_t T,
                        int32_t H, float eps, void *total, void *y, void *codes, float *scales,
                        float *inv_rms, hipStream_t stream);

/* Bytes of device workspace moe_rms_norm_backward needs (only for grad_weight);
 * 0 for invalid arguments or when none is needed.  Host function. */
size_t moe_rms_norm_backward_workspace_size(int32_t T, int32_t H);

/*
 * moe_rms_norm_backward -- gradient of moe_rms_norm.  With n = t * r and
 * a = grad_y * weight:
 *
 *   grad_x      = bf16( r * (a - n * mean(a * n)) + carried )      [T][H]
 *   grad_weight = sum over rows of grad_y * n, fp32                [H]
 *
 *   grad_y        [T][H] bf16, gradient of v (a rounding to bf16 or to 8 bits
 *                 counts as the identity).
 *   total, inv_rms   as moe_rms_norm wrote them (total: x itself without residual).
 *   carried       [T][H] bf16, the gradient that reaches total past the norm, or
 *                 NULL.  grad_x is the gradient of x and of residual alike.
 *   grad_x may be grad_y or carried itself; either output may be NULL (not both).
 *   workspace     moe_rms_norm_backward_workspace_size bytes, 16-byte aligned, no
 *                 initialisation; only used for grad_weight (else NULL is allowed).
 * Errors as moe_rms_norm.
 */
moe_status moe_rms_norm_backward(const void *grad_y, const void *total, const float *weight,
                                 const float *inv_rms, const void *carried, int32_t T, int32_t H,
                                 void *grad_x, float *grad_weight, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream);

typedef enum { MOE_TYPE_BF16 = 0, MOE_TYPE_FP32 = 1 } moe_type;

/*
 * moe_quantize_weight -- E weights of P rows by K columns in 8 bits.
 *   weight        [E][P][K], of `type` (moe_type); P % 128 == 0, K % 128 == 0.
 *   codes, scales [E][P][K] e4m3 and [E][P/128][K/128] fp32 out, as
 *                 moe_expert_matmul and moe_expert_ffn take them.
 * Errors: MOE_ERR_INVALID_ARG; MOE_ERR_UNSUPPORTED for E > MOE_MAX_EXPERTS, P or
 * K > MOE_MAX_FEATURES and more than 2^24 - 1 blocks.
 */
moe_status moe_quantize_weight(const void *weight, int32_t type, int32_t E, int32_t P, int32_t K,
                               void *codes, float *scales, hipStream_t stream);

/* The gated feed-forward block held by every expert (host struct, read during
 * the call).  hidden <= MOE_MAX_FEATURES, intermediate <= MOE_MAX_FEATURES / 2. */
typedef struct {
  int32_t hidden;       /* H > 0, H % 128 == 0: columns of x and y */
  int32_t intermediate; /* I > 0, I % 128 == 0: columns between the projections */
} moe_ffn;

/* Bytes of device workspace moe_expert_ffn needs; 0 for invalid arguments or when
 * none is needed.  Host function. */
size_t moe_expert_ffn_workspace_size(const moe_shape *shape, const moe_ffn *ffn);

/*
 * moe_expert_ffn -- every expert's gated feed-forward block on the rows of its
 * segment, fp8 payload (MOE_ERR_UNSUPPORTED for bf16: that is two calls of
 * moe_expert_matmul).  With e the row's expert, all values those of their codes:
 *
 *   z = x * up[e]^T,  h = silu(z[0..I)) * z[I..2I),  y = bf16( q(h) * down[e]^T + residual )
 *
 *   where q rounds rows to 8 bits in blocks of 128 columns (from the fp32 sums).
 *
 *   shape, layout as moe_expert_matmul takes them (layout NULL: a dense block,
 *                 num_experts == top_k == 1, for a shared expert).
 *   x, x_scales   [rows][H] e4m3 and [rows][H/128] fp32 in the receive layout.
 *   up, down      [E][2I][H] (gate rows first) and [E][H][I] e4m3, with
 *   up_scales, down_scales   [E][2I/128][H/128] and [E][H/128][I/128] fp32.
 *   residual      [rows][H] bf16, or NULL; may be y itself.
 *   y             [rows][H] bf16 out.
 *   pre           [rows][2I] bf16 out, bf16(z), for the backward pass; or NULL.
 *   workspace     moe_expert_ffn_workspace_size bytes, 16-byte aligned, no
 *                 initialisation.
 * Sums as moe_expert_matmul's fp8 ones.  Rows of no segment are neither read for a
 * result nor written.
 * Errors as moe_expert_matmul, for a shape of more tiles than one launch has.
 */
moe_status moe_expert_ffn(const moe_shape *shape, const moe_ffn *ffn, const void *x,
                          const float *x_scales, const moe_layout *layout, const void *up,
                          const float *up_scales, const void *down, const float *down_scales,
                          const void *residual, void *y, void *pre, void *workspace,
                          size_t workspace_bytes, hipStream_t stream);

/* Bytes of device workspace moe_expert_ffn_backward needs; 0 for invalid arguments
 * or when none is needed.  Host function. */
size_t moe_expert_ffn_backward_workspace_size(const moe_shape *shape, const moe_ffn *ffn);

/*
 * moe_expert_ffn_backward -- gradients of moe_expert_ffn (roundings count as the
 * identity).  With g = pre[0..I), u = pre[I..2I), s = 1 / (1 + exp(-g)):
 *
 *   gh = q(grad_y) * down[e]
 *   gz = [ gh * u * s * (1 + g * (1 - s)),  gh * g * s ]
 *   grad_x[row]  = bf16( q(gz) * up[e] )                                  [rows][H]
 *   grad_up[e]   = bf16( sum over e's rows of bf16(gz)^T bf16(x) )        [E][2I][H]
 *   grad_down[e] = bf16( sum over e's rows of grad_y^T bf16(g * s * u) )  [E][H][I]
 *
 *   The products with the weights run in 8 bits as the forward ones; the weights'
 *   gradients, which an optimiser adds up, in bf16 with fp32 sums.
 *   grad_y        [rows][H] bf16; pre as moe_expert_ffn wrote it; the others as it
 *                 was given.  The residual's gradient is grad_y itself.
 *   Any of the three outputs may be NULL (not wanted, not all).  grad_x is written
 *   on placed rows only; an expert without rows gets zeros.
 *   x, x_scales   read for grad_up only (else NULL is allowed), up and up_scales
 *                 for grad_x only, down and down_scales for grad_x and grad_up.
 *   workspace     moe_expert_ffn_backward_workspace_size bytes, 16-byte aligned, no
 *                 initialisation.
 * Errors as moe_expert_ffn; MOE_ERR_UNSUPPORTED also for weights of more than
 * 2^31 - 1 tiles of 128 x 128 and for more than some 2^26 rows.
 */
moe_status moe_expert_ffn_backward(const moe_shape *shape, const moe_ffn *ffn, const void *grad_y,
                                   const void *x, const float *x_scales, const moe_layout *layout,
                                   const void *up, const float *up_scales, const void *down,
                                   const float *down_scales, const void *pre, void *grad_x,
                                   void *grad_up, void *grad_down, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FFN_H */
