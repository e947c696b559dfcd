// experts.h -- internal launchers of the expert product, the balance loss and
// the gradients (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// Where the receive rows of each expert lie.  counts and offsets are device
// arrays (NULL: one expert holding all `rows` rows).
struct Segments {
  const int32_t* counts;
  const int32_t* offsets;
  int E, L, C;
  int rows;   // receive rows addressed
  int pairs;  // T*k: no more rows than these can be placed
};

struct MatmulParams {
  Segments seg;
  const void* x;
  const float* x_scales;
  const void* weight;
  const float* weight_scales;
  const float* bias;
  const uint16_t* residual;
  uint16_t* y;
  uint16_t* pre;
  int K, F, P, act;
};

struct MatmulGradParams {
  Segments seg;
  const uint16_t* grad_y;
  const uint16_t* x;
  const uint16_t* weight;
  const uint16_t* pre;
  uint16_t* grad_x;
  uint16_t* grad_weight;
  float* grad_bias;
  void* workspace;
  int K, F, P, act;
};

hipError_t launch_expert_matmul(const MatmulParams& p, bool fp8, hipStream_t st);
size_t expert_matmul_grad_workspace(int rows, int pairs, int E, int P, int act);
hipError_t launch_expert_matmul_grad(const MatmulGradParams& p, hipStream_t st);

hipError_t launch_combine_grad(const void* grad_out, const void* y, const int32_t* token_row,
                               const float* w, void* grad_y, float* grad_w, int T, int H, int k,
                               int rows, hipStream_t st);

struct BalanceParams {
  const float* logits;
  const float* bias;
  const int32_t* ids;
  const int32_t* seq_offsets;
  int32_t* counts;
  float* probs;
  int32_t* tokens;
  float* loss;
  void* workspace;
  int T, E, k, score, S;
  float coef;
};

size_t balance_workspace(int T, int E, int S);
hipError_t launch_balance_loss(const BalanceParams& p, hipStream_t st);

struct RouteGradParams {
  const float* logits;
  const float* bias;
  const int32_t* ids;
  const float* weights;
  const float* grad_weights;
  const int32_t* seq_offsets;
  const int32_t* counts;
  const int32_t* tokens;
  const float* grad_loss;
  float* grad_logits;
  float* grad_bias;
  void* workspace;
  int T, E, k, score, S;
  float coef;
};

size_t route_grad_workspace(int T, int E);
hipError_t launch_route_grad(const RouteGradParams& p, hipStream_t st);

}  // namespace moe
