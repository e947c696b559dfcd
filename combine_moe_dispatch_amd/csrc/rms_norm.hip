// rms_norm.hip -- the RMS norm in front of the router, with the residual's
// addition and rows in bf16 and in 8 bits, and its gradient.
//
//   t = bf16(x + residual), r = 1 / sqrt(mean t^2 + eps), v = t r w
//   grad_x = r (a - n mean(a n)) + carried, a = g w, n = t r;  grad_w = sum g n
//
// A row stays in a block's registers between the sum over it and its results, so
// every value is read and written once: both are streams.  A block takes row
// after row with the next one's loads on their way, and keeps its columns'
// weights.  The norm is of the rounded sum, which is what the next layer and the
// backward pass see.
#include "expert_device.h"
#include "ffn.h"
#include "quantize.h"

namespace moe {

namespace {

// Sum over a block; the two slots of one use are free again two uses later.
template <int THREADS>
struct BlockSum {
  static constexpr int kWaves = THREADS / kWave;
  float (*slots)[kWaves];  // [2] in LDS
  int turn = 0;

  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) v += __shfl_xor(v, d);
    if constexpr (kWaves == 1) return v;
    if (lane_id() == 0) slots[turn][threadIdx.x / kWave] = v;
    lds_barrier();
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += slots[turn][w];
    turn ^= 1;
    return sum;
  }
};

// V vectors of 8 columns a thread, THREADS apart.
template <int THREADS, int V>
struct Row {
  uint4 q[V];
  // A row that does not exist, or a null buffer, is zeros.
  __device__ __forceinline__ void load(const uint16_t* base, int64_t t, int T, int H) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * THREADS) * 8;
      q[i] = make_uint4(0, 0, 0, 0);
      if (base && t < T && c < H)
        q[i] = *reinterpret_cast<const uint4*>(base + (size_t)t * H + c);
    }
  }
};

template <int THREADS, int V>
__device__ __forceinline__ void load_weights(float (&w)[V][8], const float* weight, int H) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * THREADS) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = 0.0f;
    if (c < H) add8(w[i], weight + c);
  }
}

template <int THREADS, int V>
__global__ void __launch_bounds__(THREADS)
rms_norm_kernel(NormParams p) {
  __shared__ float s_slots[2][THREADS / kWave];
  BlockSum<THREADS> block_sum{s_slots};
  Row<THREADS, V> x, res;
  int64_t t = blockIdx.x;
  x.load(p.x, t, p.T, p.H);
  res.load(p.residual, t, p.T, p.H);
  float w[V][8];
  load_weights<THREADS, V>(w, p.weight, p.H);
  for (; t < p.T; t += gridDim.x) {
    float v[V][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      unpack8(v[i], x.q[i]);
      if (p.residual) {
        float r[8];
        unpack8(r, res.q[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += r[j];
        x.q[i] = pack8(v[i]);
        unpack8(v[i], x.q[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
      const int c = (threadIdx.x + i * THREADS) * 8;
      if (p.total && c < p.H)
        *reinterpret_cast<uint4*>(p.total + (size_t)t * p.H + c) = x.q[i];
    }
    x.load(p.x, t + gridDim.x, p.T, p.H);
    res.load(p.residual, t + gridDim.x, p.T, p.H);
    const float r = 1.0f / sqrtf(block_sum(sum) / (float)p.H + p.eps);
    if (p.inv_rms && threadIdx.x == 0) p.inv_rms[t] = r;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (threadIdx.x + i * THREADS) * 8;
      uint32_t largest = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = v[i][j] * r * w[i][j];
        largest = max(largest, magnitude(v[i][j]));
      }
      const size_t at = (size_t)t * p.H + c;
      if (p.y && c < p.H) *reinterpret_cast<uint4*>(p.y + at) = pack8(v[i]);
      if (p.codes) {
        const BlockScale block(max_over_16(largest));  // 16 lanes: 128 columns
        if (c < p.H) {
          *reinterpret_cast<uint2*>(p.codes + at) = block.codes(v[i]);
          if (threadIdx.x % 16 == 0) p.scales[at / 128] = block.scale;
        }
      }
    }
  }
}

// parts: [gridDim.x][H] sums of this block's rows, or NULL.
template <int THREADS, int V>
__global__ void __launch_bounds__(THREADS)
rms_norm_grad_kernel(NormGradParams p, float* parts) {
  __shared__ float s_slots[2][THREADS / kWave];
  BlockSum<THREADS> block_sum{s_slots};
  Row<THREADS, V> gy, total, carried;
  int64_t t = blockIdx.x;
  gy.load(p.grad_y, t, p.T, p.H);
  total.load(p.total, t, p.T, p.H);
  float r = t < p.T ? p.inv_rms[t] : 0.0f;
  float w[V][8], gw[V][8] = {};
  load_weights<THREADS, V>(w, p.weight, p.H);
  for (; t < p.T; t += gridDim.x) {
    carried.load(p.carried, t, p.T, p.H);
    float a[V][8], n[V][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      unpack8(a[i], gy.q[i]);
      unpack8(n[i], total.q[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[i][j] *= r;
        gw[i][j] = fmaf(a[i][j], n[i][j], gw[i][j]);
        a[i][j] *= w[i][j];
        sum = fmaf(a[i][j], n[i][j], sum);
      }
    }
    const int64_t next = t + gridDim.x;
    gy.load(p.grad_y, next, p.T, p.H);
    total.load(p.total, next, p.T, p.H);
    const float r_next = next < p.T ? p.inv_rms[next] : 0.0f;
    if (p.grad_x) {
      const float mean = block_sum(sum) / (float)p.H;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float c8[8];
        unpack8(c8, carried.q[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[i][j] = fmaf(r, a[i][j] - n[i][j] * mean, c8[j]);
        const int c = (threadIdx.x + i * THREADS) * 8;
        if (c < p.H) *reinterpret_cast<uint4*>(p.grad_x + (size_t)t * p.H + c) = pack8(a[i]);
      }
    }
    r = r_next;
  }
  if (!parts) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (threadIdx.x + i * THREADS) * 8;
    if (c >= p.H) continue;
    float4* out = reinterpret_cast<float4*>(parts + (size_t)blockIdx.x * p.H + c);
    out[0] = make_float4(gw[i][0], gw[i][1], gw[i][2], gw[i][3]);
    out[1] = make_float4(gw[i][4], gw[i][5], gw[i][6], gw[i][7]);
  }
}

// The blocks' sums, 64 columns a block: each of 16 waves adds every 16th part.
constexpr int kJoin = 16;
__global__ void __launch_bounds__(kJoin * kWave)
rms_norm_join_kernel(const float* parts, float* grad_weight, int blocks, int H) {
  __shared__ float s_sum[kJoin][kWave];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int c = blockIdx.x * kWave + lane;
  float sum = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int b = wave; b < blocks; b += kJoin) sum += parts[(size_t)b * H + c];
  }
  s_sum[wave][lane] = sum;
  __syncthreads();
  if (wave > 0 || c >= H) return;
#pragma unroll
  for (int w = 1; w < kJoin; ++w) sum += s_sum[w][lane];
  grad_weight[c] = sum;
}

constexpr int kNormBlocks = 1024;
constexpr int kGradBlocks = 512;

int blocks_of(int T, int most) { return T < 1 ? 1 : T < most ? T : most; }

// Few rows: a block of 1024 threads each; else 256, which leave room for several
// rows to a compute unit.
bool wide_rows(int T, int H) { return H > 256 * 8 * 4 || T <= 256; }

}  // namespace

hipError_t launch_rms_norm(const NormParams& p, hipStream_t st) {
  const dim3 grid(blocks_of(p.T, kNormBlocks));
#define MOE_NORM(THREADS, V) \
  hipLaunchKernelGGL((rms_norm_kernel<THREADS, V>), grid, dim3(THREADS), 0, st, p)
  const int vectors = p.H / 8;
  if (wide_rows(p.T, p.H)) {
    if (vectors <= 1024) MOE_NORM(1024, 1);
    else if (vectors <= 2048) MOE_NORM(1024, 2);
    else if (vectors <= 4096) MOE_NORM(1024, 4);
    else MOE_NORM(1024, 8);
  } else {
    if (vectors <= 256) MOE_NORM(256, 1);
    else if (vectors <= 512) MOE_NORM(256, 2);
    else MOE_NORM(256, 4);
  }
#undef MOE_NORM
  return hipGetLastError();
}

size_t rms_norm_grad_workspace(int T, int H) {
  const int blocks = blocks_of(T, kGradBlocks);
  return blocks > 1 ? (size_t)blocks * H * 4 : 0;
}

hipError_t launch_rms_norm_grad(const NormGradParams& p, hipStream_t st) {
  const int blocks = blocks_of(p.T, kGradBlocks);
  float* parts = !p.grad_weight ? nullptr
                 : blocks > 1   ? static_cast<float*>(p.workspace)
                                : p.grad_weight;
  const dim3 grid(blocks);
#define MOE_NORM_GRAD(THREADS, V) \
  hipLaunchKernelGGL((rms_norm_grad_kernel<THREADS, V>), grid, dim3(THREADS), 0, st, p, parts)
  const int vectors = p.H / 8;
  if (wide_rows(p.T, p.H)) {
    if (vectors <= 1024) MOE_NORM_GRAD(1024, 1);
    else if (vectors <= 2048) MOE_NORM_GRAD(1024, 2);
    else if (vectors <= 4096) MOE_NORM_GRAD(1024, 4);
    else MOE_NORM_GRAD(1024, 8);
  } else {
    if (vectors <= 256) MOE_NORM_GRAD(256, 1);
    else if (vectors <= 512) MOE_NORM_GRAD(256, 2);
    else MOE_NORM_GRAD(256, 4);
  }
#undef MOE_NORM_GRAD
  if (p.grad_weight && blocks > 1)
    hipLaunchKernelGGL(rms_norm_join_kernel, dim3((p.H + kWave - 1) / kWave),
                       dim3(kJoin * kWave), 0, st, parts, p.grad_weight, blocks, p.H);
  return hipGetLastError();
}

}  // namespace moe
