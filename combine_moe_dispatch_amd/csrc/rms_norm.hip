// rms_norm.hip -- the RMS norm in front of the router, with the residual's
// addition and rows in bf16 and in 8 bits, and its gradient.
//
//   t = bf16(x + residual), r = 1 / sqrt(mean t^2 + eps), v = t r w
//   grad_x = r (a - n mean(a n)) + carried, a = g w, n = t r;  grad_w = sum g n
//
// A row stays in registers (as it came, in bf16) between the sum over it and its
// results, so every value is read and written once: both are streams (4096 rows of
// 7168: 265 MB in 51 us, 5.2 TB/s; the gradient of 16384: 940 MB in 183 us, 5.1 TB/s).
// L threads have a row, 16 to a whole block by its length, and take row after row,
// the next one's loads on their way while this one is summed; they keep their
// columns' weights.  The norm is of the rounded sum, which is what the next layer and
// the backward pass see.
#include "expert_device.h"
#include "ffn.h"
#include "quantize.h"

namespace moe {

namespace {

// L threads to a row, blocks of kThreads.
template <int L>
struct Group {
  static constexpr int kThreads = L < 256 ? 256 : L;
  static constexpr int kRows = kThreads / L;
  static constexpr int kWaves = L > kWave ? L / kWave : 1;
  float (*slots)[kWaves];  // [2] in LDS; one use's are free again two uses later
  int turn = 0;

  // (a whole block's row is the same number in all lanes, and its addresses scalar)
  static __device__ __forceinline__ int lane() { return L >= 256 ? threadIdx.x : threadIdx.x % L; }
  static __device__ __forceinline__ int64_t first() {
    return L >= 256 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kRows + threadIdx.x / L;
  }
  static __device__ __forceinline__ int64_t stride() { return (int64_t)gridDim.x * kRows; }
  // A thread's vector i of 8 columns.
  static __device__ __forceinline__ int column(int i) { return (lane() + i * L) * 8; }

  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int d = 1; d < (L < kWave ? L : kWave); d *= 2) v += __shfl_xor(v, d);
    if constexpr (kWaves == 1) return v;
    if (lane_id() == 0) slots[turn][threadIdx.x / kWave] = v;
    lds_barrier();
    float all = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) all += slots[turn][w];
    turn ^= 1;
    return all;
  }
};

// V vectors of 8 columns a thread.  A row that does not exist, or a null buffer, is
// zeros.
template <int L, int V>
struct Row {
  uint4 q[V];
  __device__ __forceinline__ void load(const uint16_t* base, int64_t t, int T, int H) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = Group<L>::column(i);
      q[i] = make_uint4(0, 0, 0, 0);
      if (base && t < T && c < H)
        q[i] = *reinterpret_cast<const uint4*>(base + (size_t)t * H + c);
    }
  }
};

// A thread's weights: kept, or (KEEP false) loaded for each use.
template <int L, int V, bool KEEP>
struct Weights {
  float w[KEEP ? V : 1][8];
  const float* base;
  int H;
  __device__ __forceinline__ void get(float (&v)[8], int i) const {
    const int c = Group<L>::column(i);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    if (c < H) add8(v, base + c);
  }
  __device__ __forceinline__ Weights(const float* weight, int columns) : base(weight), H(columns) {
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < V; ++i) get(w[i], i);
    }
  }
  __device__ __forceinline__ void operator()(float (&v)[8], int i) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = w[i][j];
    } else {
      get(v, i);
    }
  }
};

// A mean of squares from here on has lost none that count: those below 2^-126.
constexpr float kLeastMean = 0x1p-100f;

// From 32 columns a thread of 1024 on there is no room beside the row at hand: its
// weights are loaded for each use and the next row behind its stores.  (Of the others
// the gradient at 16 columns a thread of 1024 spills 5 registers, of these the norm at 64
// columns 6 and the gradient 34.)
template <int L, int V>
constexpr bool kRoom = L < 1024 || V < 4;

template <int L, int V>
__global__ void __launch_bounds__(Group<L>::kThreads)
rms_norm_kernel(NormParams p) {
  __shared__ float s_slots[2][Group<L>::kWaves];
  Group<L> group{s_slots};
  Row<L, V> x, res;
  int64_t t = Group<L>::first();
  x.load(p.x, t, p.T, p.H);
  res.load(p.residual, t, p.T, p.H);
  const Weights<L, V, kRoom<L, V>> weights(p.weight, p.H);
  for (; t < p.T; t += Group<L>::stride()) {
    Row<L, V> total;
    float wide[kRoom<L, V> ? V : 1][8];  // total in fp32
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v[8];
      unpack8(v, x.q[i]);
      total.q[i] = x.q[i];
      if (p.residual) {
        float r[8];
        unpack8(r, res.q[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += r[j];
        total.q[i] = pack8(v);
        unpack8(v, total.q[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = fmaf(v[j], v[j], sum);
        if constexpr (kRoom<L, V>) wide[i][j] = v[j];
      }
      const int c = Group<L>::column(i);
      if (p.total && c < p.H)
        *reinterpret_cast<uint4*>(p.total + (size_t)t * p.H + c) = total.q[i];
    }
    if constexpr (kRoom<L, V>) {
      x.load(p.x, t + Group<L>::stride(), p.T, p.H);
      res.load(p.residual, t + Group<L>::stride(), p.T, p.H);
    }
    const float mean = group.sum(sum) / (float)p.H + p.eps;
    float r = 1.0f / sqrtf(mean);
    if (mean < kLeastMean || mean == __builtin_inff()) {
      // squares past the range of fp32: those of the values times a power of two
      const float by = mean < 1.0f ? 0x1p80f : 0x1p-80f;
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v[8];
        if constexpr (!kRoom<L, V>) unpack8(v, total.q[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float scaled = (kRoom<L, V> ? wide[kRoom<L, V> ? i : 0][j] : v[j]) * by;
          sum = fmaf(scaled, scaled, sum);
        }
      }
      r = by / sqrtf(group.sum(sum) / (float)p.H + p.eps * by * by);
    }
    if (p.inv_rms && Group<L>::lane() == 0) p.inv_rms[t] = r;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = Group<L>::column(i);
      float w[8];
      float (&v)[8] = wide[kRoom<L, V> ? i : 0];
      if constexpr (!kRoom<L, V>) unpack8(v, total.q[i]);
      weights(w, i);
      uint32_t largest = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = v[j] * r * w[j];
        largest = max(largest, magnitude(v[j]));
      }
      const size_t at = (size_t)t * p.H + c;
      if (p.y && c < p.H) *reinterpret_cast<uint4*>(p.y + at) = pack8(v);
      if (p.codes) {
        const BlockScale block(max_over_16(largest));  // 16 lanes: 128 columns
        if (c < p.H) {
          *reinterpret_cast<uint2*>(p.codes + at) = block.codes(v);
          if (threadIdx.x % 16 == 0) p.scales[at / kFp8Block] = block.scale;
        }
      }
    }
    if constexpr (!kRoom<L, V>) {
      x.load(p.x, t + Group<L>::stride(), p.T, p.H);
      res.load(p.residual, t + Group<L>::stride(), p.T, p.H);
    }
  }
}

__device__ __forceinline__ void store_sums(float* out, const float (&v)[8]) {
  reinterpret_cast<float4*>(out)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(out)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// parts: [gridDim.x * kRows][H] sums of each group's rows, or NULL.  Where the row
// itself fills the registers they are rms_norm_columns_kernel's.
template <int L, int V>
__global__ void __launch_bounds__(Group<L>::kThreads)
rms_norm_grad_kernel(NormGradParams p, float* parts) {
  // else a row is read again for its results (1024 rows of 65536 278 us against 256)
  constexpr bool kHold = V < 8;
  __shared__ float s_slots[2][Group<L>::kWaves];
  Group<L> group{s_slots};
  int64_t t = Group<L>::first();
  Row<L, V> gy, total;
  float r = 0.0f;
  const auto load = [&](int64_t t) {
    gy.load(p.grad_y, t, p.T, p.H);
    total.load(p.total, t, p.T, p.H);
    r = t < p.T ? p.inv_rms[t] : 0.0f;
  };
  load(t);
  const Weights<L, V, kRoom<L, V>> weights(p.weight, p.H);
  float gw[kRoom<L, V> ? V : 1][8] = {};
  for (; t < p.T; t += Group<L>::stride()) {
    const Row<L, V> gy_here = gy, total_here = total;
    const float r_here = r;
    Row<L, kRoom<L, V> ? V : 1> carried;
    if constexpr (kRoom<L, V>) carried.load(p.carried, t, p.T, p.H);
    if constexpr (kRoom<L, V>) load(t + Group<L>::stride());
    // a = g w and n = t r of vector i
    const auto values = [&](float (&g)[8], float (&n)[8], float (&a)[8], int i) {
      float w[8];
      unpack8(g, gy_here.q[i]);
      unpack8(n, total_here.q[i]);
      weights(w, i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[j] *= r_here;
        a[j] = g[j] * w[j];
      }
    };
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float g[8], n[8], a[8];
      values(g, n, a, i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (kRoom<L, V>) gw[i][j] = fmaf(g[j], n[j], gw[i][j]);
        sum = fmaf(a[j], n[j], sum);
      }
    }
    if (p.grad_x) {
      const float mean = group.sum(sum) / (float)p.H;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = Group<L>::column(i);
        if (c >= p.H) continue;
        const size_t at = (size_t)t * p.H + c;
        float g[8], n[8], a[8], more[8] = {};
        if constexpr (kHold) {
          values(g, n, a, i);
        } else {
          float w[8];
          load8(g, p.grad_y + at);
          load8(n, p.total + at);
          weights(w, i);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            n[j] *= r_here;
            a[j] = g[j] * w[j];
          }
        }
        if constexpr (kRoom<L, V>)
          unpack8(more, carried.q[i]);
        else if (p.carried)
          load8(more, p.carried + at);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = fmaf(r_here, a[j] - n[j] * mean, more[j]);
        store8(p.grad_x + at, a);
      }
    }
    if constexpr (!kRoom<L, V>) load(t + Group<L>::stride());
  }
  if constexpr (kRoom<L, V>) {
    if (!parts) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = Group<L>::column(i);
      if (c < p.H) store_sums(parts + (size_t)Group<L>::first() * p.H + c, gw[i]);
    }
  }
}

// Sums over rows of grad_y n for rows of more columns than a block can keep: 2048
// columns a block, rows blockIdx.y, + gridDim.y, ..  It reads both operands a second
// time, where the sums beside the row would spill (2048
// rows of 32768 248 us, so 174; 1024 of 65536 737 and 256).
constexpr int kWideThreads = 256, kWideGroups = 64;
__global__ void __launch_bounds__(kWideThreads)
rms_norm_columns_kernel(NormGradParams p, float* parts) {
  const int c = (blockIdx.x * kWideThreads + threadIdx.x) * 8;
  if (c >= p.H) return;
  float gw[8] = {};
#pragma unroll 4
  for (int64_t t = blockIdx.y; t < p.T; t += gridDim.y) {
    const size_t at = (size_t)t * p.H + c;
    const float r = p.inv_rms[t];
    float g[8], n[8];
    load8(g, p.grad_y + at);
    load8(n, p.total + at);
#pragma unroll
    for (int j = 0; j < 8; ++j) gw[j] = fmaf(g[j], n[j] * r, gw[j]);
  }
  store_sums(parts + (size_t)blockIdx.y * p.H + c, gw);
}

// The groups' sums, 64 columns a block: each of 16 waves adds every 16th part.
constexpr int kJoin = 16;
__global__ void __launch_bounds__(kJoin * kWave)
rms_norm_join_kernel(const float* parts, float* grad_weight, int groups, int H) {
  __shared__ float s_sum[kJoin][kWave];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int c = blockIdx.x * kWave + lane;
  float sum = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int g = wave; g < groups; g += kJoin) sum += parts[(size_t)g * H + c];
  }
  s_sum[wave][lane] = sum;
  __syncthreads();
  if (wave > 0 || c >= H) return;
#pragma unroll
  for (int w = 1; w < kJoin; ++w) sum += s_sum[w][lane];
  grad_weight[c] = sum;
}

// Threads to a row and vectors a thread: narrow rows share a block (65536 rows of 256
// columns, 256 threads each 97 us, 32 each 31 us; the gradient 154 against 42), and a
// row has up to 32 columns a thread where there are many, so that several fit a compute
// unit.
struct Split {
  int threads, vectors;
};
Split split_of(int T, int H) {
  const int n = H / 8;  // vectors of a row
  if (T > 1 && n <= 16) return {16, 1};
  if (T > 1 && n <= 32) return {32, 1};
  if (T > 1 && n <= 128) return {64, n <= 64 ? 1 : 2};
  const int l = n <= 256 || (n <= 1024 && T > 256) ? 256 : 1024;
  return {l, n <= l ? 1 : n <= 2 * l ? 2 : n <= 4 * l ? 4 : 8};
}

// Blocks of a launch: no more than so many, each with its rows.
int blocks_of(int T, Split s, int most) {
  const int rows = s.threads < 256 ? 256 / s.threads : 1;
  const int blocks = (int)(((int64_t)T + rows - 1) / rows);
  return blocks < 1 ? 1 : blocks < most ? blocks : most;
}
constexpr int kNormBlocks = 1024, kGradBlocks = 512;
bool wide(Split s) { return s.threads == 1024 && s.vectors >= 4; }  // as kRoom
int groups_of(int T, int H) {
  const Split s = split_of(T, H);
  if (wide(s)) return T < 1 ? 1 : T < kWideGroups ? T : kWideGroups;
  return blocks_of(T, s, kGradBlocks) * (s.threads < 256 ? 256 / s.threads : 1);
}

// call(L, V) as constants, those of split_of
template <class Call>
void with_split(Split s, const Call& call) {
  const auto vectors = [&](auto l) {
    using std::integral_constant;
    constexpr int kL = decltype(l)::value, kMost = kL < 64 ? 1 : kL < 256 ? 2 : kL < 1024 ? 4 : 8;
    if (s.vectors == 1) return call(l, integral_constant<int, 1>{});
    if constexpr (kMost >= 2)
      if (s.vectors == 2) return call(l, integral_constant<int, 2>{});
    if constexpr (kMost >= 4)
      if (s.vectors == 4) return call(l, integral_constant<int, 4>{});
    if constexpr (kMost >= 8) call(l, integral_constant<int, 8>{});
  };
  switch (s.threads) {
    case 16: vectors(std::integral_constant<int, 16>{}); break;
    case 32: vectors(std::integral_constant<int, 32>{}); break;
    case 64: vectors(std::integral_constant<int, 64>{}); break;
    case 256: vectors(std::integral_constant<int, 256>{}); break;
    default: vectors(std::integral_constant<int, 1024>{}); break;
  }
}

}  // namespace

hipError_t launch_rms_norm(const NormParams& p, hipStream_t st) {
  const Split s = split_of(p.T, p.H);
  const dim3 grid(blocks_of(p.T, s, kNormBlocks));
  with_split(s, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    hipLaunchKernelGGL((rms_norm_kernel<L, V>), grid, dim3(Group<L>::kThreads), 0, st, p);
  });
  return hipGetLastError();
}

size_t rms_norm_grad_workspace(int T, int H) {
  const int groups = groups_of(T, H);
  return groups > 1 ? (size_t)groups * H * 4 : 0;
}

hipError_t launch_rms_norm_grad(const NormGradParams& p, hipStream_t st) {
  const Split s = split_of(p.T, p.H);
  const int groups = groups_of(p.T, p.H);
  float* parts = !p.grad_weight ? nullptr
                 : groups > 1   ? static_cast<float*>(p.workspace)
                                : p.grad_weight;
  const dim3 grid(blocks_of(p.T, s, kGradBlocks));
  if (parts && wide(s))
    hipLaunchKernelGGL(rms_norm_columns_kernel,
                       dim3((p.H / 8 + kWideThreads - 1) / kWideThreads, groups),
                       dim3(kWideThreads), 0, st, p, parts);
  if (p.grad_x || !wide(s))
    with_split(s, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      hipLaunchKernelGGL((rms_norm_grad_kernel<L, V>), grid, dim3(Group<L>::kThreads), 0, st, p,
                         parts);
    });
  if (p.grad_weight && groups > 1)
    hipLaunchKernelGGL(rms_norm_join_kernel, dim3((p.H + kWave - 1) / kWave),
                       dim3(kJoin * kWave), 0, st, parts, p.grad_weight, groups, p.H);
  return hipGetLastError();
}

}  // namespace moe
