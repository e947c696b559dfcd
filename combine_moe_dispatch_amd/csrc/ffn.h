// ffn.h -- internal launchers of the expert layer in 8 bits (host side).
#pragma once

#include "experts.h"

namespace moe {

struct NormParams {
  const uint16_t* x;
  const uint16_t* residual;
  const float* weight;
  uint16_t* total;
  uint16_t* y;
  uint8_t* codes;
  float* scales;
  float* inv_rms;
  int T, H;
  float eps;
};
hipError_t launch_rms_norm(const NormParams& p, hipStream_t st);

struct NormGradParams {
  const uint16_t* grad_y;
  const uint16_t* total;
  const float* weight;
  const float* inv_rms;
  const uint16_t* carried;
  uint16_t* grad_x;
  float* grad_weight;
  void* workspace;
  int T, H;
};
size_t rms_norm_grad_workspace(int T, int H);
hipError_t launch_rms_norm_grad(const NormGradParams& p, hipStream_t st);

// blocks: 128 x 128 blocks of all weights together, kb of them along K.
hipError_t launch_quantize_weight(const void* weight, bool fp32, unsigned blocks, int kb,
                                  uint8_t* codes, float* scales, hipStream_t st);

struct FfnParams {
  Segments seg;
  const uint8_t* x;
  const float* x_scales;
  const uint8_t* up;
  const float* up_scales;
  const uint8_t* down;
  const float* down_scales;
  const uint16_t* residual;
  uint16_t* y;
  uint16_t* pre;
  void* workspace;
  int H, I;
};
size_t expert_ffn_workspace(int rows, int pairs, int E, int H, int I);
hipError_t launch_expert_ffn(const FfnParams& p, hipStream_t st);

struct FfnGradParams {
  Segments seg;
  const uint16_t* grad_y;
  const uint8_t* x;
  const float* x_scales;
  const uint8_t* up;
  const float* up_scales;
  const uint8_t* down;
  const float* down_scales;
  const uint16_t* pre;
  uint16_t* grad_x;
  uint16_t* grad_up;
  uint16_t* grad_down;
  void* workspace;
  int H, I;
};
size_t expert_ffn_grad_workspace(int rows, int H, int I);
hipError_t launch_expert_ffn_grad(const FfnGradParams& p, hipStream_t st);

}  // namespace moe
