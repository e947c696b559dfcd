// expert_matmul.hip -- the experts' matrix product over the placed rows, and
// its gradient.
//
// The experts multiply their tokens with their weights in a grouped GEMM
// between dispatch and combine ("Enabling trillion-parameter models on AWS
// EFA", MoE all-to-all over EFA), sized from the routing counts in device
// memory ("Lower Latency and Higher Throughput with Multi-Node DeepSeek
// Deployment", Quantization).
//
// All three products are D[u][v] = sum over r of A[u][r] B[v][r], u the
// contiguous dimension of the output:
//   y      u = weight row,     v = token row,  r = input feature
//   grad_x u = input feature,  v = token row,  r = weight row (A transposed)
//   grad_w u = input feature,  v = weight row, r = token row (both transposed)
// A block of four waves holds a 64 x 64 tile of D; the operands pass through
// LDS in steps of 32 along r, zeros past their ends.
#include "expert_device.h"

namespace moe {

namespace {

constexpr int kTile = 64;
constexpr int kStep = 32;
constexpr int kPitch = kStep + 8;
constexpr int kThreads = 256;

__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// 64 x 32 operand tile, rows i0.., columns r0.. of a row-major matrix (ld
// elements a row), zeros past rows/red.
__device__ __forceinline__ void stage_rows(uint16_t (*s)[kPitch], const uint16_t* m, size_t ld,
                                           int i0, int i_end, int r0, int red) {
  const int i = threadIdx.x / 4, c = (threadIdx.x % 4) * 8;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (i0 + i < i_end && r0 + c < red) v = load16(m + (size_t)(i0 + i) * ld + r0 + c);
  *reinterpret_cast<uint4*>(&s[i][c]) = v;
}

// The same tile of a matrix that holds it transposed: row r, column i.
__device__ __forceinline__ void stage_cols(uint16_t (*s)[kPitch], const uint16_t* m, size_t ld,
                                           int i0, int i_end, int r0, int red) {
  const int r = threadIdx.x / 8, c = (threadIdx.x % 8) * 8;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (r0 + r < red && i0 + c < i_end) v = load16(m + (size_t)(r0 + r) * ld + i0 + c);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    s[c + 2 * e][r] = (uint16_t)w[e];
    s[c + 2 * e + 1][r] = (uint16_t)(w[e] >> 16);
  }
}

// e4m3 codes widened to bf16 (exact).
__device__ __forceinline__ void stage_codes(uint16_t (*s)[kPitch], const uint8_t* m, size_t ld,
                                            const int row, bool in, int r0) {
  const int i = threadIdx.x / 4, c = (threadIdx.x % 4) * 8;
  uint2 v = make_uint2(0, 0);
  if (in) v = *reinterpret_cast<const uint2*>(m + (size_t)row * ld + r0 + c);
  float f[8];
  e4m3x4_to_f32(v.x, f);
  e4m3x4_to_f32(v.y, f + 4);
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    *reinterpret_cast<uint32_t*>(&s[i][c + e]) = pack_bf16x2(f[e], f[e + 1]);
}

__device__ __forceinline__ bf16x8_t frag(uint16_t (*s)[kPitch], int i0) {
  const int lane = lane_id();
  return *reinterpret_cast<const bf16x8_t*>(&s[i0 + (lane & 15)][(lane >> 4) * 8]);
}

__device__ __forceinline__ void mma_step(f32x4_t (&acc)[4], uint16_t (*sa)[kPitch],
                                         uint16_t (*sb)[kPitch]) {
  const bf16x8_t b = frag(sb, (threadIdx.x / kWave) * 16);
#pragma unroll
  for (int u = 0; u < 4; ++u)
    acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(sa, u * 16), b, acc[u], 0, 0, 0);
}

__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

template <bool FP8, int ACT>
__global__ void __launch_bounds__(kThreads)
matmul_kernel(MatmulParams p) {
  __shared__ __align__(16) uint16_t sa[kTile][kPitch], sb[kTile][kPitch];
  constexpr bool kGated = ACT == kActSwiglu;
  constexpr int kCols = kGated ? kTile / 2 : kTile;  // output columns of a block
  const int e = blockIdx.y;
  const int n0 = blockIdx.x * kCols;
  int begin, end;
  segment_of(p.seg, e, begin, end);
  const int lane = lane_id();
  const int srow = threadIdx.x / 4;  // the tile row this thread stages
  // the weight row behind tile row srow (gate rows, then up rows), or -1
  const int col = n0 + (kGated ? srow % kCols : srow);
  const int wrow = col < p.F ? (kGated && srow >= kCols ? p.F + col : col) : -1;
  for (int m0 = begin; m0 < end; m0 += kTile) {
    f32x4_t acc[4] = {};
    if constexpr (FP8) {
      const uint8_t* w = static_cast<const uint8_t*>(p.weight) + (size_t)e * p.P * p.K;
      const uint8_t* x = static_cast<const uint8_t*>(p.x);
      const int kb = p.K / 128;
      const int m = m0 + (threadIdx.x / kWave) * 16 + (lane & 15);
      for (int b = 0; b < kb; ++b) {
        f32x4_t part[4] = {};
        for (int r0 = b * 128; r0 < b * 128 + 128; r0 += kStep) {
          __syncthreads();
          stage_codes(sa, w, p.K, max(wrow, 0), wrow >= 0, r0);
          stage_codes(sb, x, p.K, min(m0 + srow, end - 1), m0 + srow < end, r0);
          __syncthreads();
          mma_step(part, sa, sb);
        }
        const float sx = m < end ? p.x_scales[(size_t)m * kb + b] : 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int c = n0 + (kGated ? (u % 2) * 16 : u * 16) + (lane >> 4) * 4;
          const int row = min(c, p.F - 1) + (kGated && u >= 2 ? p.F : 0);
          const float s =
              sx * p.weight_scales[((size_t)e * (p.P / 128) + row / 128) * kb + b];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[u][i] = fmaf(part[u][i], s, acc[u][i]);
        }
      }
    } else {
      const uint16_t* w = static_cast<const uint16_t*>(p.weight) + (size_t)e * p.P * p.K;
      for (int r0 = 0; r0 < p.K; r0 += kStep) {
        __syncthreads();
        const int c = (threadIdx.x % 4) * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (wrow >= 0 && r0 + c < p.K) v = load16(w + (size_t)wrow * p.K + r0 + c);
        *reinterpret_cast<uint4*>(&sa[srow][c]) = v;
        stage_rows(sb, static_cast<const uint16_t*>(p.x), p.K, m0, end, r0, p.K);
        __syncthreads();
        mma_step(acc, sa, sb);
      }
    }
    const int m = m0 + (threadIdx.x / kWave) * 16 + (lane & 15);
    if (m >= end) continue;
    float z[4][4];
    int cols[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      cols[u] = n0 + (kGated ? (u % 2) * 16 : u * 16) + (lane >> 4) * 4;
      const int row = cols[u] + (kGated && u >= 2 ? p.F : 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[u][i] = acc[u][i];
        if (p.bias && cols[u] < p.F) z[u][i] += p.bias[(size_t)e * p.P + row + i];
      }
      if (p.pre && cols[u] < p.F) store4(p.pre + (size_t)m * p.P + row, z[u]);
    }
#pragma unroll
    for (int u = 0; u < (kGated ? 2 : 4); ++u) {
      if (cols[u] >= p.F) continue;
      float o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kGated)
          o[i] = z[u][i] * sigmoid_f32(z[u][i]) * z[u + 2][i];
        else
          o[i] = act_f32<ACT>(z[u][i]);
      }
      const size_t at = (size_t)m * p.F + cols[u];
      if (p.residual)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += bf16_f32(p.residual[at + i]);
      store4(p.y + at, o);
    }
  }
}

// gz = grad_y * act'(pre) to bf16, and its column sums in fp32: a thread owns
// one column and the block walks the expert's rows.
template <int ACT>
__global__ void __launch_bounds__(kThreads)
act_grad_kernel(MatmulGradParams p, uint16_t* gz) {
  const int e = blockIdx.y;
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.F) return;
  int begin, end;
  segment_of(p.seg, e, begin, end);
  float sum0 = 0.0f, sum1 = 0.0f;
  for (int m = begin; m < end; ++m) {
    const float gy = bf16_f32(p.grad_y[(size_t)m * p.F + c]);
    const size_t at = (size_t)m * p.P + c;
    if constexpr (ACT == kActSwiglu) {
      const float g = bf16_f32(p.pre[at]), u = bf16_f32(p.pre[at + p.F]);
      const float s = sigmoid_f32(g);
      const float dg = gy * u * s * (1.0f + g * (1.0f - s)), du = gy * g * s;
      gz[at] = (uint16_t)pack_bf16x2(dg, 0.0f);
      gz[at + p.F] = (uint16_t)pack_bf16x2(du, 0.0f);
      sum0 += dg;
      sum1 += du;
    } else {
      float d = gy;
      if constexpr (ACT == kActSilu) {
        const float z = bf16_f32(p.pre[at]);
        const float s = sigmoid_f32(z);
        d = gy * s * (1.0f + z * (1.0f - s));
      } else if constexpr (ACT == kActGelu) {
        const float z = bf16_f32(p.pre[at]);
        d = gy * (0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
                  z * expf(-0.5f * z * z) * 0.39894228040143268f);
      }
      if (gz) gz[at] = (uint16_t)pack_bf16x2(d, 0.0f);
      sum0 += d;
    }
  }
  if (p.grad_bias) {
    p.grad_bias[(size_t)e * p.P + c] = sum0;
    if constexpr (ACT == kActSwiglu) p.grad_bias[(size_t)e * p.P + p.F + c] = sum1;
  }
}

// grad_x: D[input feature][token row], A transposed.
__global__ void __launch_bounds__(kThreads)
grad_x_kernel(MatmulGradParams p, const uint16_t* gz) {
  __shared__ __align__(16) uint16_t sa[kTile][kPitch], sb[kTile][kPitch];
  const int e = blockIdx.y, n0 = blockIdx.x * kTile, lane = lane_id();
  int begin, end;
  segment_of(p.seg, e, begin, end);
  const uint16_t* w = p.weight + (size_t)e * p.P * p.K;
  for (int m0 = begin; m0 < end; m0 += kTile) {
    f32x4_t acc[4] = {};
    for (int r0 = 0; r0 < p.P; r0 += kStep) {
      __syncthreads();
      stage_cols(sa, w, p.K, n0, p.K, r0, p.P);
      stage_rows(sb, gz, p.P, m0, end, r0, p.P);
      __syncthreads();
      mma_step(acc, sa, sb);
    }
    const int m = m0 + (threadIdx.x / kWave) * 16 + (lane & 15);
    if (m >= end) continue;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = n0 + u * 16 + (lane >> 4) * 4;
      const float v[4] = {acc[u][0], acc[u][1], acc[u][2], acc[u][3]};
      if (c < p.K) store4(p.grad_x + (size_t)m * p.K + c, v);
    }
  }
}

// grad_w: D[input feature][weight row], both transposed, summed over rows.
__global__ void __launch_bounds__(kThreads)
grad_w_kernel(MatmulGradParams p, const uint16_t* gz) {
  __shared__ __align__(16) uint16_t sa[kTile][kPitch], sb[kTile][kPitch];
  const int e = blockIdx.z, n0 = blockIdx.x * kTile, p0 = blockIdx.y * kTile, lane = lane_id();
  int begin, end;
  segment_of(p.seg, e, begin, end);
  f32x4_t acc[4] = {};
  for (int r0 = begin; r0 < end; r0 += kStep) {
    __syncthreads();
    stage_cols(sa, p.x, p.K, n0, p.K, r0, end);
    stage_cols(sb, gz, p.P, p0, p.P, r0, end);
    __syncthreads();
    mma_step(acc, sa, sb);
  }
  const int row = p0 + (threadIdx.x / kWave) * 16 + (lane & 15);
  if (row >= p.P) return;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int c = n0 + u * 16 + (lane >> 4) * 4;
    const float v[4] = {acc[u][0], acc[u][1], acc[u][2], acc[u][3]};
    if (c < p.K) store4(p.grad_weight + ((size_t)e * p.P + row) * p.K + c, v);
  }
}

template <bool FP8>
void launch_forward(const MatmulParams& p, hipStream_t st) {
  const int cols = p.act == kActSwiglu ? kTile / 2 : kTile;
  const dim3 grid((p.F + cols - 1) / cols, p.seg.E);
  switch (p.act) {
    case kActSilu: hipLaunchKernelGGL((matmul_kernel<FP8, kActSilu>), grid, dim3(kThreads), 0, st, p); break;
    case kActGelu: hipLaunchKernelGGL((matmul_kernel<FP8, kActGelu>), grid, dim3(kThreads), 0, st, p); break;
    case kActSwiglu: hipLaunchKernelGGL((matmul_kernel<FP8, kActSwiglu>), grid, dim3(kThreads), 0, st, p); break;
    default: hipLaunchKernelGGL((matmul_kernel<FP8, kActNone>), grid, dim3(kThreads), 0, st, p); break;
  }
}

}  // namespace

hipError_t launch_expert_matmul(const MatmulParams& p, bool fp8, hipStream_t st) {
  if (fp8)
    launch_forward<true>(p, st);
  else
    launch_forward<false>(p, st);
  return hipGetLastError();
}

size_t expert_matmul_grad_workspace(int rows, int pairs, int E, int P, int act) {
  return act == kActNone || pairs == 0 ? 0 : ((size_t)rows * P * 2 + 15) / 16 * 16;
}

hipError_t launch_expert_matmul_grad(const MatmulGradParams& p, hipStream_t st) {
  uint16_t* gz = p.act == kActNone ? nullptr : static_cast<uint16_t*>(p.workspace);
  if (p.grad_bias || p.act != kActNone) {
    const dim3 grid((p.F + kThreads - 1) / kThreads, p.seg.E);
    switch (p.act) {
      case kActSilu: hipLaunchKernelGGL((act_grad_kernel<kActSilu>), grid, dim3(kThreads), 0, st, p, gz); break;
      case kActGelu: hipLaunchKernelGGL((act_grad_kernel<kActGelu>), grid, dim3(kThreads), 0, st, p, gz); break;
      case kActSwiglu: hipLaunchKernelGGL((act_grad_kernel<kActSwiglu>), grid, dim3(kThreads), 0, st, p, gz); break;
      default: hipLaunchKernelGGL((act_grad_kernel<kActNone>), grid, dim3(kThreads), 0, st, p, gz); break;
    }
  }
  const uint16_t* g = gz ? gz : p.grad_y;
  const unsigned nt = (p.K + kTile - 1) / kTile, pt = (p.P + kTile - 1) / kTile;
  if (p.grad_x)
    hipLaunchKernelGGL(grad_x_kernel, dim3(nt, p.seg.E), dim3(kThreads), 0, st, p, g);
  if (p.grad_weight)
    hipLaunchKernelGGL(grad_w_kernel, dim3(nt, pt, p.seg.E), dim3(kThreads), 0, st, p, g);
  return hipGetLastError();
}

}  // namespace moe
