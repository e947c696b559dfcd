// combine_grad.hip -- gradients of the combine.
//
// out[t] = sum over slots of w[t][j] y[row(t, j)], so the gradient of a row is
// its weight times its token's output gradient, and the gradient of a weight
// is the dot product of the two rows.  A block owns one (token, slot) pair:
// it reads both rows once, writes one, and sums its products in fp32.  A
// stream: a token's pairs lie in neighbouring blocks, which find its gradient
// row in the caches.  4096 tokens of 7168 columns, top-8: 1.0 GB in 189 us, 5.3
// TB/s, what a large copy reaches; 128 tokens 7.9 us.
#include "device_common.h"
#include "experts.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr unsigned kMaxBlocks = 1u << 23;  // a launch has less than 2^32 threads

__global__ void __launch_bounds__(kThreads)
combine_grad_kernel(const uint4* __restrict__ grad_out, const uint4* __restrict__ y,
                    const int32_t* __restrict__ token_row, const float* __restrict__ w,
                    uint4* __restrict__ grad_y, float* __restrict__ grad_w, int nvec, int k,
                    int rows, unsigned first) {
  __shared__ float s_sum[kThreads / kWave];
  const size_t pair = first + blockIdx.x;
  const int row = token_row[pair];
  if (row < 0 || row >= rows) {
    if (grad_w && threadIdx.x == 0) grad_w[pair] = 0.0f;
    return;
  }
  const float a = grad_y ? w[pair] : 0.0f;
  const uint4* go = grad_out + (pair / k) * nvec;
  float sum = 0.0f;
  for (int v = threadIdx.x; v < nvec; v += kThreads) {
    const uint4 g = go[v];
    const uint32_t gq[4] = {g.x, g.y, g.z, g.w};
    if (grad_y) {
      uint32_t o[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) o[m] = pack_bf16x2(a * bf16_lo(gq[m]), a * bf16_hi(gq[m]));
      grad_y[(size_t)row * nvec + v] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (grad_w) {
      const uint4 r = y[(size_t)row * nvec + v];
      const uint32_t rq[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        sum = fmaf(bf16_lo(gq[m]), bf16_lo(rq[m]), sum);
        sum = fmaf(bf16_hi(gq[m]), bf16_hi(rq[m]), sum);
      }
    }
  }
  if (!grad_w) return;
  for (int d = kWave / 2; d > 0; d /= 2) sum += __shfl_xor(sum, d);
  if (lane_id() == 0) s_sum[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float total = 0.0f;
    for (int i = 0; i < kThreads / kWave; ++i) total += s_sum[i];
    grad_w[pair] = total;
  }
}

}  // namespace

hipError_t launch_combine_grad(const void* grad_out, const void* y, const int32_t* token_row,
                               const float* w, void* grad_y, float* grad_w, int T, int H, int k,
                               int rows, hipStream_t st) {
  const unsigned pairs = (unsigned)T * (unsigned)k;
  for (unsigned first = 0; first < pairs; first += kMaxBlocks) {
    const unsigned left = pairs - first;
    hipLaunchKernelGGL(combine_grad_kernel, dim3(left < kMaxBlocks ? left : kMaxBlocks),
                       dim3(kThreads), 0, st, static_cast<const uint4*>(grad_out),
                       static_cast<const uint4*>(y), token_row, w, static_cast<uint4*>(grad_y),
                       grad_w, H / 8, k, rows, first);
  }
  return hipGetLastError();
}

}  // namespace moe
