// quantize_weight.hip -- weights to e4m3 with one scale per 128 x 128 block.
//
// A block of 256 threads holds one 128 x 128 block in registers between its
// largest magnitude and its codes, so the weights are read once: a stream (32 of 4096
// x 7168, fp32: 4.7 GB in 850 us, 5.5 TB/s).
#include "expert_device.h"
#include "ffn.h"
#include "quantize.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 16;  // rows of a pass: 16 threads of 8 columns each
constexpr int kPasses = 128 / kRows;

template <class T>
__global__ void __launch_bounds__(kThreads)
quantize_weight_kernel(const T* weight, int kb, uint8_t* codes, float* scales) {
  __shared__ uint32_t s_largest[kThreads / kWave];
  const size_t K = (size_t)kb * 128;
  const unsigned b = blockIdx.x, row0 = b / kb, col = b % kb;  // row0: block row of all weights
  const size_t at = ((size_t)row0 * 128 + threadIdx.x / 16) * K + col * 128 + threadIdx.x % 16 * 8;
  float v[kPasses][8];
  uint32_t largest = 0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) load8(v[i], weight + at + i * kRows * K);
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) largest = max(largest, magnitude(v[i][j]));
  largest = max_over_rows(max_over_16(largest));
  if (lane_id() == 0) s_largest[threadIdx.x / kWave] = largest;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) largest = max(largest, s_largest[w]);
  const BlockScale block(largest);
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    *reinterpret_cast<uint2*>(codes + at + i * kRows * K) = block.codes(v[i]);
  if (threadIdx.x == 0) scales[b] = block.scale;
}

}  // namespace

hipError_t launch_quantize_weight(const void* weight, bool fp32, unsigned blocks, int kb,
                                  uint8_t* codes, float* scales, hipStream_t st) {
  if (fp32)
    hipLaunchKernelGGL((quantize_weight_kernel<float>), dim3(blocks), dim3(kThreads), 0, st,
                       static_cast<const float*>(weight), kb, codes, scales);
  else
    hipLaunchKernelGGL((quantize_weight_kernel<uint16_t>), dim3(blocks), dim3(kThreads), 0, st,
                       static_cast<const uint16_t*>(weight), kb, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
