// capi_ffn.hip -- argument checks of moe_ffn.h, then launches on the caller's
// stream.  No allocation, no synchronisation, no state.
#include "moe_ffn.h"
#include "capi_check.h"
#include "ffn.h"

namespace {

using namespace moe::capi;

moe_status check_norm(int32_t T, int32_t H) {
  if (T < 0 || H <= 0 || H % 8 != 0) return MOE_ERR_INVALID_ARG;
  return H > MOE_MAX_NORM_COLUMNS ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// A block's shape, and what of it lies where.
moe_status check_ffn(const moe_shape* shape, const moe_ffn* ffn, int* rows) {
  const moe_status st = check_shape(shape, rows);
  if (st != MOE_OK) return st;
  if (!ffn || ffn->hidden <= 0 || ffn->intermediate <= 0 || ffn->hidden % 128 != 0 ||
      ffn->intermediate % 128 != 0)
    return MOE_ERR_INVALID_ARG;
  if (shape->payload != MOE_PAYLOAD_FP8_E4M3_B128) return MOE_ERR_UNSUPPORTED;
  if (ffn->hidden > MOE_MAX_FEATURES || ffn->intermediate > MOE_MAX_FEATURES / 2)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int pairs_of(const moe_shape* s, int rows) {
  const int64_t pairs = (int64_t)s->num_tokens * s->top_k;
  return (int)(pairs < rows ? pairs : rows);
}

}  // namespace

extern "C" {

moe_status moe_rms_norm(const void* x, const void* residual, const float* weight, int32_t T,
                        int32_t H, float eps, void* total, void* y, void* codes, float* scales,
                        float* inv_rms, hipStream_t stream) {
  const moe_status st = check_norm(T, H);
  if (st != MOE_OK) return st;
  if (!total && !y && !codes && !inv_rms) return MOE_ERR_INVALID_ARG;
  if (!codes != !scales || (codes && H % 128 != 0)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!rows_ok(x) || !maybe_rows_ok(residual) || !rows_ok(weight) || !maybe_rows_ok(total) ||
      !maybe_rows_ok(y) || !maybe_rows_ok(codes))
    return MOE_ERR_INVALID_ARG;
  if (total && total == y) return MOE_ERR_INVALID_ARG;
  moe::NormParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.residual = static_cast<const uint16_t*>(residual);
  p.weight = weight;
  p.total = static_cast<uint16_t*>(total);
  p.y = static_cast<uint16_t*>(y);
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = scales;
  p.inv_rms = inv_rms;
  p.T = T;
  p.H = H;
  p.eps = eps;
  return from_hip(moe::launch_rms_norm(p, stream));
}

size_t moe_rms_norm_backward_workspace_size(int32_t T, int32_t H) {
  return check_norm(T, H) == MOE_OK ? moe::rms_norm_grad_workspace(T, H) : 0;
}

moe_status moe_rms_norm_backward(const void* grad_y, const void* total, const float* weight,
                                 const float* inv_rms, const void* carried, int32_t T, int32_t H,
                                 void* grad_x, float* grad_weight, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  const moe_status st = check_norm(T, H);
  if (st != MOE_OK) return st;
  if (!grad_x && !grad_weight) return MOE_ERR_INVALID_ARG;
  if (T == 0 && !grad_weight) return MOE_OK;
  if (!rows_ok(weight) || !maybe_rows_ok(grad_x) || !aligned16(grad_weight) ||
      !maybe_rows_ok(carried))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!rows_ok(grad_y) || !rows_ok(total) || !inv_rms)) return MOE_ERR_INVALID_ARG;
  const size_t need = grad_weight ? moe::rms_norm_grad_workspace(T, H) : 0;
  if (need > 0 && (!rows_ok(workspace) || workspace_bytes < need)) return MOE_ERR_INVALID_ARG;
  moe::NormGradParams p{};
  p.grad_y = static_cast<const uint16_t*>(grad_y);
  p.total = static_cast<const uint16_t*>(total);
  p.weight = weight;
  p.inv_rms = inv_rms;
  p.carried = static_cast<const uint16_t*>(carried);
  p.grad_x = static_cast<uint16_t*>(grad_x);
  p.grad_weight = grad_weight;
  p.workspace = workspace;
  p.T = T;
  p.H = H;
  return from_hip(moe::launch_rms_norm_grad(p, stream));
}

moe_status moe_quantize_weight(const void* weight, int32_t type, int32_t E, int32_t P, int32_t K,
                               void* codes, float* scales, hipStream_t stream) {
  if (type != MOE_TYPE_BF16 && type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (E < 1 || P < 1 || K < 1 || P % 128 != 0 || K % 128 != 0) return MOE_ERR_INVALID_ARG;
  if (E > MOE_MAX_EXPERTS || P > MOE_MAX_FEATURES || K > MOE_MAX_FEATURES)
    return MOE_ERR_UNSUPPORTED;
  const int64_t blocks = (int64_t)E * (P / 128) * (K / 128);
  if (blocks >= (1 << 24)) return MOE_ERR_UNSUPPORTED;  // of 256 threads
  if (!rows_ok(weight) || !rows_ok(codes) || !scales) return MOE_ERR_INVALID_ARG;
  return from_hip(moe::launch_quantize_weight(weight, type == MOE_TYPE_FP32, (unsigned)blocks,
                                              K / 128, static_cast<uint8_t*>(codes), scales,
                                              stream));
}

size_t moe_expert_ffn_workspace_size(const moe_shape* shape, const moe_ffn* ffn) {
  int rows;
  if (check_ffn(shape, ffn, &rows) != MOE_OK) return 0;
  return moe::expert_ffn_workspace(rows, pairs_of(shape, rows), shape->num_experts, ffn->hidden,
                                   ffn->intermediate);
}

moe_status moe_expert_ffn(const moe_shape* shape, const moe_ffn* ffn, const void* x,
                          const float* x_scales, const moe_layout* layout, const void* up,
                          const float* up_scales, const void* down, const float* down_scales,
                          const void* residual, void* y, void* pre, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  moe::FfnParams p{};
  int rows;
  moe_status st = check_ffn(shape, ffn, &rows);
  if (st != MOE_OK) return st;
  if ((st = segments(shape, layout, rows, &p.seg)) != MOE_OK) return st;
  if (p.seg.pairs == 0) return MOE_OK;  // nothing can be placed
  if (!rows_ok(x) || !x_scales || !rows_ok(up) || !up_scales || !rows_ok(down) || !down_scales ||
      !maybe_rows_ok(residual) || !rows_ok(y) || !maybe_rows_ok(pre))
    return MOE_ERR_INVALID_ARG;
  if (!rows_ok(workspace) || workspace_bytes < moe_expert_ffn_workspace_size(shape, ffn))
    return MOE_ERR_INVALID_ARG;
  p.x = static_cast<const uint8_t*>(x);
  p.x_scales = x_scales;
  p.up = static_cast<const uint8_t*>(up);
  p.up_scales = up_scales;
  p.down = static_cast<const uint8_t*>(down);
  p.down_scales = down_scales;
  p.residual = static_cast<const uint16_t*>(residual);
  p.y = static_cast<uint16_t*>(y);
  p.pre = static_cast<uint16_t*>(pre);
  p.workspace = workspace;
  p.H = ffn->hidden;
  p.I = ffn->intermediate;
  return from_hip(moe::launch_expert_ffn(p, stream));
}

size_t moe_expert_ffn_backward_workspace_size(const moe_shape* shape, const moe_ffn* ffn) {
  int rows;
  if (check_ffn(shape, ffn, &rows) != MOE_OK || shape->num_tokens == 0) return 0;
  return moe::expert_ffn_grad_workspace(rows, ffn->hidden, ffn->intermediate);
}

moe_status moe_expert_ffn_backward(const moe_shape* shape, const moe_ffn* ffn, const void* grad_y,
                                   const void* x, const float* x_scales, const moe_layout* layout,
                                   const void* up, const float* up_scales, const void* down,
                                   const float* down_scales, const void* pre, void* grad_x,
                                   void* grad_up, void* grad_down, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  moe::FfnGradParams p{};
  int rows;
  moe_status st = check_ffn(shape, ffn, &rows);
  if (st != MOE_OK) return st;
  if ((st = segments(shape, layout, rows, &p.seg)) != MOE_OK) return st;
  if (!grad_x && !grad_up && !grad_down) return MOE_ERR_INVALID_ARG;
  if (!maybe_rows_ok(grad_x) || !maybe_rows_ok(grad_up) || !maybe_rows_ok(grad_down))
    return MOE_ERR_INVALID_ARG;
  if (p.seg.pairs > 0) {
    if (!rows_ok(grad_y) || !rows_ok(pre)) return MOE_ERR_INVALID_ARG;
    if (grad_up && (!rows_ok(x) || !x_scales)) return MOE_ERR_INVALID_ARG;
    if (grad_x && (!rows_ok(up) || !up_scales)) return MOE_ERR_INVALID_ARG;
    if ((grad_x || grad_up) && (!rows_ok(down) || !down_scales)) return MOE_ERR_INVALID_ARG;
    if (!rows_ok(workspace) ||
        workspace_bytes < moe_expert_ffn_backward_workspace_size(shape, ffn))
      return MOE_ERR_INVALID_ARG;
  } else if (!grad_up && !grad_down) {
    return MOE_OK;  // no rows at all
  }
  p.grad_y = static_cast<const uint16_t*>(grad_y);
  p.x = static_cast<const uint8_t*>(x);
  p.x_scales = x_scales;
  p.up = static_cast<const uint8_t*>(up);
  p.up_scales = up_scales;
  p.down = static_cast<const uint8_t*>(down);
  p.down_scales = down_scales;
  p.pre = static_cast<const uint16_t*>(pre);
  p.grad_x = static_cast<uint16_t*>(grad_x);
  p.grad_up = static_cast<uint16_t*>(grad_up);
  p.grad_down = static_cast<uint16_t*>(grad_down);
  p.workspace = workspace;
  p.H = ffn->hidden;
  p.I = ffn->intermediate;
  return from_hip(moe::launch_expert_ffn_grad(p, stream));
}

}  // extern "C"
