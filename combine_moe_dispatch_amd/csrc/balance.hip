// balance.hip -- the router's balance loss and the router's gradient.
//
// Both walk the logits one wave per token: the wave holds the token's biased
// logits (expert i*64 + lane in register i), its scores and their sum.  The
// loss adds the probabilities of a sequence's tokens up per expert and counts
// the pairs; the gradient needs those counts only.
#include "device_common.h"
#include "experts.h"

namespace moe {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;

__device__ __forceinline__ float wave_sum(float v) {
  for (int d = kWave / 2; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
  for (int d = kWave / 2; d > 0; d /= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// Probabilities of token t in registers (0 past E); r holds 1 - sigmoid for
// sigmoid scores and 1 for softmax, the factor of their gradient.  Where no
// logit is positive the sigmoids are taken relative to the largest one,
// exp(l - top) / (1 + exp(l)), so that their sum cannot vanish.
template <int VPL>
__device__ __forceinline__ void token_probs(const float* logits, const float* bias, int t, int E,
                                            int score, float (&p)[VPL], float (&r)[VPL]) {
  const int lane = lane_id();
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * kWave + lane;
    p[i] = e < E ? logits[(size_t)t * E + e] + (bias ? bias[e] : 0.0f) : -INFINITY;
    top = fmaxf(top, p[i]);
  }
  top = wave_max(top);
  if (score == 1) top = fminf(top, 0.0f);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool in = i * kWave + lane < E;
    r[i] = score == 1 ? 1.0f / (1.0f + expf(p[i])) : 1.0f;
    if (score == 1 && top == 0.0f)
      p[i] = in ? 1.0f / (1.0f + expf(-p[i])) : 0.0f;
    else
      p[i] = in ? expf(p[i] - top) * r[i] : 0.0f;
    sum += p[i];
  }
  sum = wave_sum(sum);
#pragma unroll
  for (int i = 0; i < VPL; ++i) p[i] /= sum;
}

__device__ __forceinline__ void sequence_bounds(const int32_t* off, int s, int T, int& a, int& b) {
  a = off ? min(max(off[s], 0), T) : 0;
  b = off ? min(max(off[s + 1], 0), T) : T;
}

// One block per sequence.
template <int VPL>
__global__ void __launch_bounds__(kThreads)
balance_kernel(BalanceParams q) {
  __shared__ int s_count[kMaxExperts];
  __shared__ float s_prob[kWaves][kMaxExperts];
  __shared__ int s_tokens[kWaves];
  const int s = blockIdx.x, lane = lane_id(), wave = threadIdx.x / kWave;
  for (int e = threadIdx.x; e < q.E; e += kThreads) s_count[e] = 0;
  __syncthreads();
  int a, b;
  sequence_bounds(q.seq_offsets, s, q.T, a, b);
  float acc[VPL] = {};
  int n = 0;
  for (int t = a + wave; t < b; t += kWaves) {
    const int id = lane < q.k ? q.ids[(size_t)t * q.k + lane] : -1;
    const bool real = id >= 0 && id < q.E;
    if (real) atomicAdd(&s_count[id], 1);
    if (__ballot(real) == 0) continue;
    ++n;
    float p[VPL], sc[VPL];
    token_probs<VPL>(q.logits, q.bias, t, q.E, q.score, p, sc);
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] += p[i];
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (i * kWave + lane < q.E) s_prob[wave][i * kWave + lane] = acc[i];
  if (lane == 0) s_tokens[wave] = n;
  __syncthreads();
  int total = 0;
  for (int i = 0; i < kWaves; ++i) total += s_tokens[i];
  for (int e = threadIdx.x; e < q.E; e += kThreads) {
    float sum = 0.0f;
    for (int i = 0; i < kWaves; ++i) sum += s_prob[i][e];
    q.counts[(size_t)s * q.E + e] = s_count[e];
    q.probs[(size_t)s * q.E + e] = sum / (float)max(total, 1);
  }
  if (threadIdx.x == 0) q.tokens[s] = total;
}

__global__ void __launch_bounds__(kThreads)
balance_loss_kernel(BalanceParams q) {
  __shared__ float s_sum[kWaves];
  float sum = 0.0f;
  for (size_t i = threadIdx.x; i < (size_t)q.S * q.E; i += kThreads)
    sum += (float)q.counts[i] / (float)max(q.tokens[i / q.E], 1) * q.probs[i];
  sum = wave_sum(sum);
  if (lane_id() == 0) s_sum[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x != 0) return;
  float total = 0.0f;
  for (int i = 0; i < kWaves; ++i) total += s_sum[i];
  q.loss[0] = total * ((float)q.E / (float)q.k) * (q.coef / (float)q.S);
}

// The sequence of token t: the last one that begins at or before it, if it
// reaches it (-1: none).
__device__ __forceinline__ int sequence_of(const int32_t* off, int S, int t) {
  if (!off) return 0;
  int lo = 0, hi = S;  // off[lo] <= t < off[hi], where such a pair exists
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (off[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return off[lo] <= t && t < off[lo + 1] ? lo : -1;
}

template <int VPL>
__global__ void __launch_bounds__(kThreads)
route_grad_kernel(RouteGradParams q) {
  __shared__ float s_add[kWaves][kMaxExperts];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int t = blockIdx.x * kWaves + wave;
  if (t >= q.T) return;
  float p[VPL], r[VPL], d[VPL];
  const int id = lane < q.k ? q.ids[(size_t)t * q.k + lane] : -1;
  const bool real = id >= 0 && id < q.E;
  if (__ballot(real) == 0) {  // a padded token, whatever its logits hold
    for (int e = lane; e < q.E; e += kWave) q.grad_logits[(size_t)t * q.E + e] = 0.0f;
    return;
  }
  token_probs<VPL>(q.logits, q.bias, t, q.E, q.score, p, r);
  const int seq = q.counts ? sequence_of(q.seq_offsets, q.S, t) : -1;
#pragma unroll
  for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
  if (seq >= 0) {
    const float n = (float)max(q.tokens[seq], 1);
    const float f = (q.grad_loss ? q.grad_loss[0] : 1.0f) * (q.coef / (float)q.S) *
                    ((float)q.E / (float)q.k) / (n * n);
    float mean = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * kWave + lane;
      d[i] = e < q.E ? f * (float)q.counts[(size_t)seq * q.E + e] : 0.0f;
      mean += d[i] * p[i];
    }
    mean = wave_sum(mean);
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = p[i] * (d[i] - mean);
  }
  if (q.grad_weights) {
    float* add = s_add[wave];
    for (int e = lane; e < q.E; e += kWave) add[e] = 0.0f;
    __builtin_amdgcn_wave_barrier();
    const float w = real ? q.weights[(size_t)t * q.k + lane] : 0.0f;
    const float gw = real ? q.grad_weights[(size_t)t * q.k + lane] : 0.0f;
    const float mean = wave_sum(gw * w);
    const float dl = w * (gw - mean);
    // slots in turn, so that a repeated id adds up in slot order
    for (int j = 0; j < q.k; ++j) {
      if (lane == j && real) add[id] += dl;
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i * kWave + lane < q.E) d[i] += add[i * kWave + lane];
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * kWave + lane;
    if (e < q.E) q.grad_logits[(size_t)t * q.E + e] = d[i] * r[i];
  }
}

// One block per 64 experts: column sums of grad_logits.
__global__ void __launch_bounds__(kThreads)
grad_bias_kernel(RouteGradParams q) {
  __shared__ float s_sum[kWaves][kWave];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int e = blockIdx.x * kWave + lane;
  float sum = 0.0f;
  if (e < q.E)
    for (int t = wave; t < q.T; t += kWaves) sum += q.grad_logits[(size_t)t * q.E + e];
  s_sum[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && e < q.E)
    q.grad_bias[e] = s_sum[0][lane] + s_sum[1][lane] + s_sum[2][lane] + s_sum[3][lane];
}

}  // namespace

#define MOE_BY_VPL(KERNEL, GRID)                                                             \
  do {                                                                                       \
    const int vpl = (q.E + kWave - 1) / kWave;                                               \
    if (vpl <= 1)                                                                            \
      hipLaunchKernelGGL(KERNEL<1>, GRID, dim3(kThreads), 0, st, q);                         \
    else if (vpl <= 4)                                                                       \
      hipLaunchKernelGGL(KERNEL<4>, GRID, dim3(kThreads), 0, st, q);                         \
    else                                                                                     \
      hipLaunchKernelGGL(KERNEL<16>, GRID, dim3(kThreads), 0, st, q);                        \
  } while (0)

size_t balance_workspace(int T, int E, int S) { return 0; }

hipError_t launch_balance_loss(const BalanceParams& q, hipStream_t st) {
  MOE_BY_VPL(balance_kernel, dim3((unsigned)q.S));
  hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(kThreads), 0, st, q);
  return hipGetLastError();
}

size_t route_grad_workspace(int T, int E) { return 0; }

hipError_t launch_route_grad(const RouteGradParams& q, hipStream_t st) {
  if (q.T > 0) MOE_BY_VPL(route_grad_kernel, dim3((unsigned)((q.T + kWaves - 1) / kWaves)));
  if (q.grad_bias)
    hipLaunchKernelGGL(grad_bias_kernel, dim3((unsigned)((q.E + kWave - 1) / kWave)),
                       dim3(kThreads), 0, st, q);
  return hipGetLastError();
}

}  // namespace moe
