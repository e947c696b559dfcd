// capi_experts.hip -- argument checks of moe_experts.h, then launches on the
// caller's stream.  No allocation, no synchronisation, no state.
#include "moe_experts.h"
#include "experts.h"
#include "shape_check.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// present and aligned / absent or aligned
bool rows_ok(const void* p) { return p && aligned16(p); }
bool maybe_rows_ok(const void* p) { return aligned16(p); }

moe_status from_hip(hipError_t e) {
  if (e == hipErrorNotSupported) return MOE_ERR_UNSUPPORTED;  // the launchers' own limits
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// A shape's receive rows.
moe_status check_shape(const moe_shape* s, int* rows) {
  int L;
  int64_t n;
  const moe_status st = moe::check_shape(s, &L, &n);
  if (st != MOE_OK) return st;
  if (n > MOE_MAX_EXPERT_ROWS) return MOE_ERR_UNSUPPORTED;
  *rows = (int)n;
  return MOE_OK;
}

moe_status check_linear(const moe_shape* s, const moe_linear* l, int* P) {
  if (!l || l->in_features <= 0 || l->out_features <= 0) return MOE_ERR_INVALID_ARG;
  if (l->activation < MOE_ACT_NONE || l->activation > MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  const int unit = s->payload == MOE_PAYLOAD_FP8_E4M3_B128 ? 128 : 8;
  if (l->in_features % unit != 0 || l->out_features % unit != 0) return MOE_ERR_INVALID_ARG;
  const int64_t p = (l->activation == MOE_ACT_SWIGLU ? 2 : 1) * (int64_t)l->out_features;
  // a tile's rows are addressed with 32-bit byte offsets
  if (p > MOE_MAX_FEATURES || l->in_features > MOE_MAX_FEATURES) return MOE_ERR_UNSUPPORTED;
  *P = (int)p;
  return MOE_OK;
}

moe_status segments(const moe_shape* s, const moe_layout* lay, int rows, moe::Segments* seg) {
  if (lay) {
    if (!lay->expert_counts || !lay->expert_offsets) return MOE_ERR_INVALID_ARG;
    seg->counts = lay->expert_counts;
    seg->offsets = lay->expert_offsets;
  } else {
    if (s->num_experts != 1 || s->top_k != 1) return MOE_ERR_INVALID_ARG;
    if (s->num_tokens > rows) return MOE_ERR_INVALID_ARG;  // more tokens than rows
    rows = s->num_tokens;
    seg->counts = seg->offsets = nullptr;
  }
  seg->E = s->num_experts;
  seg->L = s->num_experts / s->num_ranks;
  seg->C = s->rank_capacity;
  seg->rows = rows;
  const int64_t pairs = (int64_t)s->num_tokens * s->top_k;
  seg->pairs = (int)(pairs < rows ? pairs : rows);
  if (seg->pairs == 0) seg->rows = 0;  // no segment, whatever the counts say
  return MOE_OK;
}

moe_status check_router(int32_t T, int32_t E, int32_t k, int32_t score, int32_t S) {
  if (T < 0 || E < 1 || k < 1 || k > E || S < 1) return MOE_ERR_INVALID_ARG;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (E > MOE_MAX_EXPERTS || k > MOE_MAX_TOP_K) return MOE_ERR_UNSUPPORTED;
  if (T > MOE_MAX_ROUTED || S > MOE_MAX_ROUTED) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)S * E > INT32_MAX || (int64_t)T * k > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_expert_matmul(const moe_shape* shape, const moe_linear* linear, const void* x,
                             const float* x_scales, const moe_layout* layout, const void* weight,
                             const float* weight_scales, const float* bias, const void* residual,
                             void* y, void* pre, hipStream_t stream) {
  moe::MatmulParams p{};
  int rows;
  moe_status st = check_shape(shape, &rows);
  if (st != MOE_OK) return st;
  if ((st = check_linear(shape, linear, &p.P)) != MOE_OK) return st;
  if ((st = segments(shape, layout, rows, &p.seg)) != MOE_OK) return st;
  if (p.seg.pairs == 0) return MOE_OK;  // nothing can be placed
  const bool fp8 = shape->payload == MOE_PAYLOAD_FP8_E4M3_B128;
  if (!rows_ok(x) || !rows_ok(weight) || !rows_ok(y) || !maybe_rows_ok(residual) ||
      !maybe_rows_ok(pre) || !aligned16(bias))
    return MOE_ERR_INVALID_ARG;
  if (fp8 && (!x_scales || !weight_scales)) return MOE_ERR_INVALID_ARG;
  p.x = x;
  p.x_scales = x_scales;
  p.weight = weight;
  p.weight_scales = weight_scales;
  p.bias = bias;
  p.residual = static_cast<const uint16_t*>(residual);
  p.y = static_cast<uint16_t*>(y);
  p.pre = static_cast<uint16_t*>(pre);
  p.K = linear->in_features;
  p.F = linear->out_features;
  p.act = linear->activation;
  return from_hip(moe::launch_expert_matmul(p, fp8, stream));
}

size_t moe_expert_matmul_backward_workspace_size(const moe_shape* shape,
                                                 const moe_linear* linear) {
  int rows, P;
  if (check_shape(shape, &rows) != MOE_OK || check_linear(shape, linear, &P) != MOE_OK) return 0;
  const int64_t pairs = (int64_t)shape->num_tokens * shape->top_k;
  return moe::expert_matmul_grad_workspace(rows, (int)(pairs < rows ? pairs : rows),
                                           shape->num_experts, P, linear->activation);
}

moe_status moe_expert_matmul_backward(const moe_shape* shape, const moe_linear* linear,
                                      const void* grad_y, const void* x, const moe_layout* layout,
                                      const void* weight, const void* pre, void* grad_x,
                                      void* grad_weight, float* grad_bias, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
  moe::MatmulGradParams p{};
  int rows;
  moe_status st = check_shape(shape, &rows);
  if (st != MOE_OK) return st;
  if ((st = check_linear(shape, linear, &p.P)) != MOE_OK) return st;
  if (shape->payload != MOE_PAYLOAD_BF16) return MOE_ERR_UNSUPPORTED;
  const bool idle = linear->activation == MOE_ACT_NONE && !grad_bias;  // gz is grad_y
  const size_t need = idle ? 0 : moe_expert_matmul_backward_workspace_size(shape, linear);
  if ((st = segments(shape, layout, rows, &p.seg)) != MOE_OK) return st;
  if (!grad_x && !grad_weight && !grad_bias) return MOE_ERR_INVALID_ARG;
  if (!maybe_rows_ok(grad_x) || !maybe_rows_ok(grad_weight) || !aligned16(grad_bias))
    return MOE_ERR_INVALID_ARG;
  if (p.seg.pairs > 0) {
    if (!rows_ok(grad_y) || (grad_weight && !rows_ok(x)) || (grad_x && !rows_ok(weight)))
      return MOE_ERR_INVALID_ARG;
    if (linear->activation != MOE_ACT_NONE && !rows_ok(pre)) return MOE_ERR_INVALID_ARG;
  }
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return MOE_ERR_INVALID_ARG;
  p.grad_y = static_cast<const uint16_t*>(grad_y);
  p.x = static_cast<const uint16_t*>(x);
  p.weight = static_cast<const uint16_t*>(weight);
  p.pre = static_cast<const uint16_t*>(pre);
  p.grad_x = static_cast<uint16_t*>(grad_x);
  p.grad_weight = static_cast<uint16_t*>(grad_weight);
  p.grad_bias = grad_bias;
  p.workspace = workspace;
  p.K = linear->in_features;
  p.F = linear->out_features;
  p.act = linear->activation;
  return from_hip(moe::launch_expert_matmul_grad(p, stream));
}

moe_status moe_combine_backward(const moe_shape* shape, const void* grad_out, const void* expert_y,
                                const moe_layout* layout, const float* topk_weights, void* grad_y,
                                float* grad_weights, hipStream_t stream) {
  int rows;
  moe_status st = check_shape(shape, &rows);
  if (st != MOE_OK) return st;
  if (shape->payload != MOE_PAYLOAD_BF16) return MOE_ERR_UNSUPPORTED;
  if (!grad_y && !grad_weights) return MOE_ERR_INVALID_ARG;
  if (shape->num_tokens == 0) return MOE_OK;
  if (!layout || !layout->token_row || !rows_ok(grad_out) || !maybe_rows_ok(grad_y) ||
      (grad_weights && !rows_ok(expert_y)) || (grad_y && !topk_weights))
    return MOE_ERR_INVALID_ARG;
  return from_hip(moe::launch_combine_grad(grad_out, expert_y, layout->token_row, topk_weights,
                                           grad_y, grad_weights, shape->num_tokens, shape->hidden,
                                           shape->top_k, rows, stream));
}

size_t moe_balance_loss_workspace_size(int32_t T, int32_t E, int32_t num_seqs) {
  if (check_router(T, E, 1, MOE_SCORE_SOFTMAX, num_seqs) != MOE_OK) return 0;
  return moe::balance_workspace(T, E, num_seqs);
}

moe_status moe_balance_loss(const float* logits, const float* bias, const int32_t* topk_ids,
                            int32_t T, int32_t E, int32_t k, int32_t score,
                            const int32_t* seq_offsets, int32_t num_seqs, float coef,
                            int32_t* expert_counts, float* expert_probs, int32_t* seq_tokens,
                            float* loss, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
  const moe_status st = check_router(T, E, k, score, num_seqs);
  if (st != MOE_OK) return st;
  if (T > 0 && (!logits || !topk_ids)) return MOE_ERR_INVALID_ARG;
  if (!seq_offsets && num_seqs != 1) return MOE_ERR_INVALID_ARG;
  if (!expert_counts || !expert_probs || !seq_tokens || !loss) return MOE_ERR_INVALID_ARG;
  const size_t need = moe::balance_workspace(T, E, num_seqs);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return MOE_ERR_INVALID_ARG;
  const moe::BalanceParams p{logits, bias,      topk_ids, seq_offsets, expert_counts, expert_probs,
                             seq_tokens, loss,  workspace, T, E, k, score, num_seqs, coef};
  return from_hip(moe::launch_balance_loss(p, stream));
}

size_t moe_route_backward_workspace_size(int32_t T, int32_t E) {
  if (check_router(T, E, 1, MOE_SCORE_SOFTMAX, 1) != MOE_OK) return 0;
  return moe::route_grad_workspace(T, E);
}

moe_status moe_route_backward(const float* logits, const float* bias, const int32_t* topk_ids,
                              const float* topk_weights, const float* grad_weights, int32_t T,
                              int32_t E, int32_t k, int32_t score, const int32_t* seq_offsets,
                              int32_t num_seqs, float coef, const int32_t* expert_counts,
                              const int32_t* seq_tokens, const float* grad_loss,
                              float* grad_logits, float* grad_bias, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  const bool balance = expert_counts && seq_tokens;
  if (!expert_counts != !seq_tokens) return MOE_ERR_INVALID_ARG;
  if (!balance && !grad_weights) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_router(T, E, k, score, balance ? num_seqs : 1);
  if (st != MOE_OK) return st;
  if (balance && !seq_offsets && num_seqs != 1) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_ids || !grad_logits || (grad_weights && !topk_weights)))
    return MOE_ERR_INVALID_ARG;
  const size_t need = grad_bias ? moe::route_grad_workspace(T, E) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return MOE_ERR_INVALID_ARG;
  const moe::RouteGradParams p{logits,   bias,       topk_ids,
                               topk_weights, grad_weights, balance ? seq_offsets : nullptr,
                               expert_counts, seq_tokens, grad_loss,
                               grad_logits, grad_bias, workspace,
                               T, E, k, score, balance ? num_seqs : 1, coef};
  return from_hip(moe::launch_route_grad(p, stream));
}

}  // extern "C"
