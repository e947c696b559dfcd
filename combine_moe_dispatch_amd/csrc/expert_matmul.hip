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
// so that a lane's four accumulators are neighbours in memory.  A block holds
// a tile of D in registers and walks r in steps of 64: while its waves multiply
// one step out of LDS, the loads of the next go straight into another part of
// it.  Sums are fp32, but for the first 128 products of fp8 (see there); results
// are rounded to bf16 once.
//
// What bounds it (32 experts of 4096 x 7168 weights): up to some 100 rows an
// expert the weights' way from memory (1.9 GB: 317 us at 32 rows, 5.9 TB/s; one
// token's eight experts 81 us, 5.8 TB/s), past that the matrix units and the
// power they draw (4096 tokens, 1.75 TFLOP in 1.51 ms back to back, 1.64 on
// average under a profiler; as one dense product 1.36 ms against 1.29 of the
// library's).
#include <type_traits>

#include "expert_product.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// The product for few rows an expert, where the weights' way from memory is
// what counts.  Each of a block's SPLIT waves takes a share of the steps for
// the whole tile, through a ring of its own in LDS: no wave waits for another
// until the shares are added up, and a tile that has a compute unit to itself
// still has SPLIT rings of loads on their way (one expert of 2048 x 7168 and 64
// rows: 21 us, where one ring a block with a barrier a step took 60).
// ---------------------------------------------------------------------------
template <int TU, int TV, int SPLIT, int STAGES>
struct StreamProduct {
  using C = Config<1, 1, TU, TV>;  // of one wave
  using A = OperandTile<C::kBu, 1, false, true>;
  using B = OperandTile<C::kBv, 1, false, false>;
  static constexpr int kThreads = SPLIT * kWave;
  static constexpr int kStage = A::kBytes + B::kBytes;
  static constexpr int kRing = STAGES * kStage;
  static constexpr int kLds = SPLIT * kRing;
  static constexpr int kLoads = A::kLoads + B::kLoads;
  static_assert((STAGES - 2) * kLoads < 64, "counted by the hardware");
  A a;
  B b;
  f32x4_t acc[TU][TV];
  typename A::template Reader<TU> ra;
  typename B::template Reader<TV> rb;

  template <bool TAIL>
  __device__ __forceinline__ void multiply(uint32_t here, int nv, int left) {
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      bf16x8_t fa[TU];
#pragma unroll
      for (int u = 0; u < TU; ++u) fa[u] = ra.template frag<TAIL>(here, u, k, left);
#pragma unroll
      for (int v = 0; v < TV; ++v) {
        if (v >= nv) break;
        const bf16x8_t fb = rb.template frag<TAIL>(here + A::kBytes, v, k, left);
#pragma unroll
        for (int u = 0; u < TU; ++u)
          acc[u][v] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[u], fb, acc[u][v], 0, 0, 0);
      }
    }
  }

  // red > 0 positions along r, `rows` rows along v; ap, bp as in TileProduct.
  // Wave 0 is left with the result.
  __device__ __forceinline__ void run(char* smem, int wave, const char* (&ap)[A::kLoads],
                                      const char* bp, int red, int rows) {
    ra.init(0);
    rb.init(0);
#pragma unroll
    for (int u = 0; u < TU; ++u)
#pragma unroll
      for (int v = 0; v < TV; ++v) acc[u][v] = f32x4_t{};
    const int nv = min((rows + 15) / 16, TV);
    const int steps = (red + kStep - 1) / kStep;
    const int rest = red - (steps - 1) * kStep;  // positions of the last step
    const int share = (steps + SPLIT - 1) / SPLIT;
    const int first = min(wave * share, steps), end = min(first + share, steps);
#pragma unroll
    for (int i = 0; i < A::kLoads; ++i) ap[i] += (size_t)first * (kStep * 2);
    bp += (size_t)first * (kStep * 2);
    const uint32_t lds = lds_address(smem) + wave * kRing, lds_end = lds + kRing;
    uint32_t fill = lds, here = lds;
    auto after = [&](uint32_t slot) { return slot + kStage == lds_end ? lds : slot + kStage; };
    auto load = [&](auto tail) {
      constexpr bool kTail = decltype(tail)::value;
#pragma unroll
      for (int i = 0; i < A::kLoads; ++i) {
        a.template load<kTail>(i, fill, 0, ap[i], 0, rest);
        ap[i] += kStep * 2;
      }
#pragma unroll
      for (int i = 0; i < B::kLoads; ++i)
        b.template load<kTail>(i, fill + A::kBytes, 0, bp, 0, rest);
      bp += kStep * 2;
    };
    auto start = [&](int t) {
      if (t + 1 < steps || rest == kStep)
        load(std::false_type{});
      else
        load(std::true_type{});
      fill = after(fill);
    };
    for (int t = first; t < first + STAGES - 1 && t < end; ++t) start(t);
    for (int t = first; t < end; ++t) {
      if (t + STAGES - 1 <= end)
        wait_vm<(STAGES - 2) * kLoads>();
      else
        wait_vm<0>();
      wait_lds();  // the step before has been read out of the slot to fill
      if (t + STAGES - 1 < end) start(t + STAGES - 1);
      if (t + 1 < steps)
        multiply<false>(here, nv, rest);
      else
        multiply<true>(here, nv, rest);
      here = after(here);
    }
    // the shares, added up in their order
    static_assert(kRing >= TU * TV * 16 * kWave, "a wave's sums fit its ring");
    f32x4_t* sums = reinterpret_cast<f32x4_t*>(smem + wave * kRing) + lane_id();
    wait_lds();
    if (wave > 0) {
#pragma unroll
      for (int u = 0; u < TU; ++u)
#pragma unroll
        for (int v = 0; v < TV; ++v) sums[(u * TV + v) * kWave] = acc[u][v];
    }
    __syncthreads();
    if (wave > 0) return;
    for (int w = 1; w < SPLIT; ++w) {
      const f32x4_t* other = reinterpret_cast<f32x4_t*>(smem + w * kRing) + lane_id();
#pragma unroll
      for (int u = 0; u < TU; ++u)
#pragma unroll
        for (int v = 0; v < TV; ++v) acc[u][v] += other[(u * TV + v) * kWave];
    }
  }

  __device__ __forceinline__ void eight(float (&o)[8], int a, int v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = acc[2 * a + i / 4][v][i % 4];
  }
};

// ---------------------------------------------------------------------------
// gz = grad_y * act'(pre) to bf16, and its column sums in fp32 (summed before
// that rounding).  A stream: a lane owns 8 columns (of the gate and of the up
// half), a block 4 x 512 columns of every split's rows, four rows on their way
// at once; the splits' sums are added by a second launch.  8192 rows of 4096:
// 168 MB in 40 us at best, 4.2 TB/s, 60 on average among other kernels.
//
// gz is bf16 because the matrix units take no more in one pass: the rest of it
// as a second operand would double both products.  Against fp64 the gradients are
// off by 2.3e-3 of their size, 1.7e-3 with the outputs' rounding alone.
// ---------------------------------------------------------------------------
constexpr int kActRows = 4;

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == kActSilu) {
    const float s = sigmoid_f32(z);
    return s * (1.0f + z * (1.0f - s));
  }
  if (ACT == kActGelu)
    return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
           z * expf(-0.5f * z * z) * 0.39894228040143268f;
  return 1.0f;
}

// parts: [gridDim.z][E][P] column sums, or NULL when they are not wanted.
template <int ACT>
__global__ void __launch_bounds__(kThreads)
act_grad_kernel(MatmulGradParams p, uint16_t* gz, float* parts) {
  constexpr bool kGated = ACT == kActSwiglu;
  __shared__ __align__(16) float s_sum[kActRows - 1][kGated ? 2 : 1][kWave * 8];
  const int e = blockIdx.y, lane = lane_id(), wave = threadIdx.x / kWave;
  const int c = (blockIdx.x * kWave + lane) * 8;
  const bool in = c < p.F;
  int begin, end;
  segment_of(p.seg, e, begin, end);
  const int per = (max(end - begin, 0) + gridDim.z - 1) / gridDim.z;
  const int first = begin + blockIdx.z * per, last = min(first + per, end);
  float sum[8] = {}, sum_up[8] = {};
  if (in) {
    for (int m = first + wave; m < last; m += kActRows) {
      float gy[8], z[8], up[8], d[8], du[8];
      load8(gy, p.grad_y + (size_t)m * p.F + c);
      const size_t at = (size_t)m * p.P + c;
      if (ACT != kActNone) load8(z, p.pre + at);
      if (kGated) load8(up, p.pre + at + p.F);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (kGated) {
          const float s = sigmoid_f32(z[i]);
          d[i] = gy[i] * up[i] * s * (1.0f + z[i] * (1.0f - s));
          du[i] = gy[i] * z[i] * s;
          sum_up[i] += du[i];
        } else {
          d[i] = ACT == kActNone ? gy[i] : gy[i] * act_slope<ACT>(z[i]);
        }
        sum[i] += d[i];
      }
      if (ACT != kActNone) store8(gz + at, d);
      if (kGated) store8(gz + at + p.F, du);
    }
  }
  if (!parts) return;
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s_sum[wave - 1][0][lane * 8 + i] = sum[i];
      if (kGated) s_sum[wave - 1][kGated ? 1 : 0][lane * 8 + i] = sum_up[i];
    }
  }
  __syncthreads();
  if (wave > 0 || !in) return;
  float* out = parts + ((size_t)blockIdx.z * p.seg.E + e) * p.P + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    for (int w = 0; w < kActRows - 1; ++w) {
      sum[i] += s_sum[w][0][lane * 8 + i];
      if (kGated) sum_up[i] += s_sum[w][kGated ? 1 : 0][lane * 8 + i];
    }
    out[i] = sum[i];
    if (kGated) out[p.F + i] = sum_up[i];
  }
}

__global__ void __launch_bounds__(kThreads)
bias_grad_kernel(const float* parts, float* grad_bias, size_t n, int splits) {
  const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  float sum = 0.0f;
#pragma unroll 8
  for (int s = 0; s < splits; ++s) sum += parts[(size_t)s * n + i];
  grad_bias[i] = sum;
}

// Splits of an expert's rows: enough blocks to fill the chip, no fewer than 16
// rows to a split on average.
int act_splits(int pairs, int E, int F) {
  const int64_t blocks = (int64_t)E * ((F + 511) / 512);
  const int64_t want = (2048 + blocks - 1) / blocks, most = pairs / E / 16 + 1;
  return (int)(want < most ? want : most);
}

// Bias, activation and residual on the accumulators, then the one rounding.
template <class C, int ACT, class Product>
__device__ __forceinline__ void finish(const Product& prod, const MatmulParams& p, const Tile& t,
                                       int wave) {
  using Cols = Columns<C, ACT>;
  const int wu = wave % C::kWu, wv = wave / C::kWu, lane = lane_id();
#pragma unroll
  for (int a = 0; a < Cols::kPairs; ++a) {
    const int col = t.n * Cols::kTile + wu * Cols::kWave + a * 32 + (lane >> 4) * 8;
    if (col >= p.F) continue;
    float bias[8] = {}, bias_up[8] = {};  // once for all rows
    if (p.bias) {
      const float* b = p.bias + (size_t)t.e * p.P + col;
      add8(bias, b);
      if (Cols::kGated) add8(bias_up, b + p.F);
    }
#pragma unroll
    for (int v = 0; v < C::kTv; ++v) {
      const int m = t.m0 + (v * C::kWv + wv) * 16 + (lane & 15);
      if (m >= t.end) continue;
      float z[8], up[8];
      prod.eight(z, a, v);
      if (Cols::kGated) prod.eight(up, a + Cols::kPairs, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[i] += bias[i];
        if (Cols::kGated) up[i] += bias_up[i];
      }
      if (p.pre) {
        store8(p.pre + (size_t)m * p.P + col, z);
        if (Cols::kGated) store8(p.pre + (size_t)m * p.P + p.F + col, up);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        z[i] = Cols::kGated ? z[i] * sigmoid_short(z[i]) * up[i] : act_f32<ACT>(z[i]);
      const size_t at = (size_t)m * p.F + col;
      if (p.residual) add8(z, p.residual + at);
      store8(p.y + at, z);
    }
  }
}

template <class C, int ACT>
__global__ void __launch_bounds__(C::kThreads)
matmul_kernel(MatmulParams p, int ntiles) {
  extern __shared__ __align__(1024) char smem[];
  Tile t;
  if (!find_tile<C::kBv>(p.seg, ntiles, blockIdx.x, t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = t.n * Columns<C, ACT>::kTile;
  TileProduct<C, false, false> prod;
  prod.setup(smem, wave);
  prod.lda = prod.ldb = (uint32_t)p.K * 2;
  prod.red = p.K;
  weight_loads<C, ACT>(prod.a, prod.ap,
                       static_cast<const char*>(p.weight) + ((size_t)t.e * p.P + n0) * prod.lda,
                       wave, p.F, p.F - n0, prod.lda);
  prod.b.init(wave, prod.ldb, min(C::kBv, t.end - t.m0));
  prod.bp = static_cast<const char*>(p.x) + (size_t)t.m0 * prod.ldb;
  prod.begin_and_run(t.end - t.m0);
  finish<C, ACT>(prod, p, t, wave);
}

template <class Product, int ACT>
__global__ void __launch_bounds__(Product::kThreads)
matmul_stream_kernel(MatmulParams p, int ntiles) {
  using C = typename Product::C;
  extern __shared__ __align__(1024) char smem[];
  Tile t;
  if (!find_tile<C::kBv>(p.seg, ntiles, blockIdx.x, t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = t.n * Columns<C, ACT>::kTile;
  const uint32_t ld = (uint32_t)p.K * 2;
  const int rows = min(C::kBv, t.end - t.m0);
  Product prod;
  const char* ap[Product::A::kLoads];
  weight_loads<C, ACT>(prod.a, ap,
                       static_cast<const char*>(p.weight) + ((size_t)t.e * p.P + n0) * ld, 0, p.F,
                       p.F - n0, ld);
  prod.b.init(0, ld, rows);
  prod.run(smem, wave, ap, static_cast<const char*>(p.x) + (size_t)t.m0 * ld, p.K, rows);
  if (wave == 0) finish<C, ACT>(prod, p, t, 0);
}

template <class C, int STAGES, int ACT>
__global__ void __launch_bounds__(C::kThreads)
matmul_fp8_kernel(MatmulParams p, int ntiles) {
  using Product = Fp8Product<C, STAGES>;
  using Cols = Columns<C, ACT>;
  extern __shared__ __align__(1024) char smem[];
  Tile t;
  if (!find_tile<C::kBv>(p.seg, ntiles, blockIdx.x, t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = t.n * Cols::kTile, kb = p.K / 128;
  const uint32_t ld = (uint32_t)p.K;
  const int rows = min(C::kBv, t.end - t.m0);
  Product prod;
  prod.template weight_rows<Cols::kGated>(
      wave, static_cast<const char*>(p.weight) + ((size_t)t.e * p.P + n0) * ld, ld, p.F - n0,
      (size_t)p.F * ld);
  prod.b.init(wave, ld, rows);
  // the scales of this wave's weight rows (all of one block of 128, or of the
  // gate's and the up's block); past the last column any will do
  static_assert(128 % Cols::kWave == 0, "a wave's columns lie in one block of scales");
  const int block = min(n0 + wave % C::kWu * Cols::kWave, p.F - 1) / 128;
  const int lane = lane_id();
  const size_t up = Cols::kGated && lane % 2 == 1 ? p.F / 128 : 0;
  const float* scale =
      lane < 32 ? p.x_scales + (size_t)(t.m0 + min(wave * 32 + lane, rows - 1)) * kb
                : p.weight_scales + ((size_t)t.e * (p.P / 128) + block + up) * kb;
  const char* bp = static_cast<const char*>(p.x) + (size_t)t.m0 * ld;
  prod.run_rows(smem, wave, bp, scale, kb, rows);
  finish<C, ACT>(prod, p, t, wave);
}

// grad_x: D[input feature][token row].
template <class C>
__global__ void __launch_bounds__(C::kThreads)
grad_x_kernel(MatmulGradParams p, const uint16_t* gz, int ntiles) {
  using Product = TileProduct<C, true, false>;
  extern __shared__ __align__(1024) char smem[];
  Tile t;
  if (!find_tile<C::kBv>(p.seg, ntiles, blockIdx.x, t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = t.n * C::kBu;
  Product prod;
  prod.setup(smem, wave);
  prod.lda = (uint32_t)p.K * 2;
  prod.ldb = (uint32_t)p.P * 2;
  prod.red = p.P;
  prod.a.init(wave, prod.lda, min(C::kBu, p.K - n0));
  prod.b.init(wave, prod.ldb, min(C::kBv, t.end - t.m0));
#pragma unroll
  for (int i = 0; i < Product::A::kLoads; ++i)
    prod.ap[i] = reinterpret_cast<const char*>(p.weight + (size_t)t.e * p.P * p.K + n0);
  prod.bp = reinterpret_cast<const char*>(gz + (size_t)t.m0 * p.P);
  prod.begin_and_run(t.end - t.m0);
  store_tile<C, false>(prod, wave, p.grad_x + (size_t)t.m0 * p.K + n0, p.K, t.end - t.m0,
                       p.K - n0);
}

// grad_w: D[input feature][weight row], summed over the expert's rows.  Every
// expert has nt x pt tiles; one without rows has zeros.  With few rows an
// expert a tile is a handful of steps and a large result, so the blocks stay:
// each takes one tile after another and starts the loads of the next before
// it stores the last, without waiting for those stores.  32 experts of 256 rows,
// 4096 x 7168: 1.9 GB written in 800 us (810 before half steps were left out,
// 575 of them without the stores); a tile's steps take 9.7 us, the next one's
// loads 1.8, the stores 4.4.
// Streaming stores took 1130 us, device-scope ones 1080, 128 x 128 tiles with
// two blocks to a compute unit 936.
template <class C>
__global__ void __launch_bounds__(C::kThreads)
grad_w_kernel(MatmulGradParams p, const uint16_t* gz, unsigned nt, unsigned pt) {
  using Product = TileProduct<C, true, true>;
  extern __shared__ __align__(1024) char smem[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int* seg_begin = reinterpret_cast<int*>(smem + Product::kLds);
  int* seg_rows = seg_begin + kMaxExperts;
  fill_table(seg_begin, seg_rows, p.seg);
  __syncthreads();
  const unsigned total = nt * pt * (unsigned)p.seg.E;
  Product prod;
  prod.setup(smem, wave);
  prod.lda = (uint32_t)p.K * 2;
  prod.ldb = (uint32_t)p.P * 2;
  struct Place {
    int e, n0, p0, rows;
  };
  auto place = [&](unsigned b) {
    const unsigned at = xcd_local_block(b, total), in = at % (nt * pt);
    Place w;
    w.e = (int)(at / (nt * pt));
    // neighbouring blocks write neighbouring columns (897 against 1000 us the
    // other way round at 32 experts, 4096 x 7168)
    w.n0 = (int)(in % nt) * C::kBu;
    w.p0 = (int)(in / nt) * C::kBv;
    w.rows = __builtin_amdgcn_readfirstlane(seg_rows[w.e]);
    return w;
  };
  auto begin = [&](const Place& w) {
    if (w.rows <= 0) return;
    const int first = __builtin_amdgcn_readfirstlane(seg_begin[w.e]);
    prod.red = w.rows;
    prod.a.init(wave, prod.lda, min(C::kBu, p.K - w.n0));
    prod.b.init(wave, prod.ldb, min(C::kBv, p.P - w.p0));
#pragma unroll
    for (int i = 0; i < Product::A::kLoads; ++i)
      prod.ap[i] = reinterpret_cast<const char*>(p.x + (size_t)first * p.K + w.n0);
    prod.bp = reinterpret_cast<const char*>(gz + (size_t)first * p.P + w.p0);
    prod.template begin<C::kTv>();
  };
  Place w = place(blockIdx.x);  // the grid has no more blocks than tiles
  begin(w);
  bool stores = false;  // kStores of them started behind this tile's loads
  for (unsigned b = blockIdx.x;;) {
    if (w.rows > 0)
      prod.template run<C::kTv>(stores ? kStores<C> : 0);
    else
      prod.clear();
    b += gridDim.x;
    const bool more = b < total;
    const Place n = place(more ? b : 0);
    if (more) begin(n);
    uint16_t* out = p.grad_weight + ((size_t)w.e * p.P + w.p0) * p.K + w.n0;
    stores = p.P - w.p0 >= C::kBv && p.K - w.n0 >= C::kBu;
    if (stores)
      store_tile<C, true>(prod, wave, out, p.K, 0, 0);
    else
      store_tile<C, false>(prod, wave, out, p.K, p.P - w.p0, p.K - w.n0);
    if (!more) break;
    w = n;
  }
}

// 256 x 256 tiles for experts of many rows, one block to a compute unit; 128 x
// 128, two blocks to a unit, for the others: the second block works while the
// first waits for its first loads or stores its results (256 x 128 tiles, one
// to a unit, took 371 us against 346 at 64 rows an expert, 32 experts of 4096
// x 7168, and 42 us against 37 for 1021 rows of one expert of 7168 x 2048).
using Large = Config<2, 2, 8, 8>;
using Mid = Config<2, 2, 4, 4>;
// 64 x 16 by four waves that share the steps.
using Few = StreamProduct<4, 1, 4, 3>;
// fp8 where there are few large tiles: 256 token rows by 128 weight rows in three steps
// of LDS.
using FewCodes = Config<2, 4, 4, 4>;

// Large tiles from 112 rows an expert on, where some experts begin to need two
// small ones (32 experts, 4096 x 7168: 96 rows 394 us against 357 on small
// tiles, 128 rows 435 against 501, 256 rows 637 against 668, 512 rows 905
// against 1024), if they give three quarters of the compute units one (one
// expert, 7168 x 2048: 112 tiles 59 us against 36, 168 tiles 61 against 59, 196
// tiles 63 against 66).
bool large_tiles(const Segments& s, int u) {
  return s.pairs / s.E >= 112 && tiles_of(s, u, Large::kBu, Large::kBv) >= kUnits * 3 / 4;
}

// The streaming product for up to 4 rows an expert and 128 in all (one token of
// 8 of 32 experts, 4096 x 7168: 82 us against 110 on 128 x 128 tiles; 128 rows
// of 32 experts, 4 each 316 against 317, in 8 of them 88 against 114; 256 rows of
// 256 experts, one each 2.49 ms for either, in 8 of them 179 us against 106, in
// one 137 against 71: its 16 row tiles read the weights again), and while those
// tiles would leave compute units idle, up to 64 an expert (one expert, 64 rows,
// 2048 x 7168: 21 us against 63).
bool few_rows(const Segments& s, int u) {
  const int64_t rows = s.pairs / s.E;
  return (rows <= 4 && s.pairs <= 128) ||
         (rows <= 64 && tiles_of(s, u, Mid::kBu, Mid::kBv) < kUnits);
}

// The weight gradient has every expert's tiles whatever the counts: large
// ones above 64 rows an expert, if they give three quarters of the compute units
// one (one expert of 2048 x 4096, 4096 rows, 128 large tiles: 100 us against 68;
// 2048 x 6144, 1024 rows, 192 tiles: 36.7 against 37.3; 4096 x 4096, 8192 rows,
// 256 tiles: 202 against 259; 32 experts of 4096 x 7168, 256 rows: 808 against
// 936; 256 of 512 x 512, 32 rows: 35 against 30).
bool large_weight_tiles(const Segments& s, int K, int P) {
  const int64_t tiles = (int64_t)s.E * ((K + Large::kBu - 1) / Large::kBu) *
                        ((P + Large::kBv - 1) / Large::kBv);
  return s.pairs / s.E > 64 && tiles >= kUnits * 3 / 4;
}

// fp8 on 128 x 128 tiles in place of FewCodes': up to 128 rows an expert, where there
// are as many of them, two to a unit (32 experts of 8 rows 159 us against 157; 16 rows
// and 2048 x 7168, 24.5 us against 22), and while they find a compute unit each (4096 x
// 7168, one expert: 200 rows 52 us against 35, 1021 rows 55 against 41, 1500 rows 59
// against 68; 8 experts of 130 rows 56 against 80).  Among several experts chance gives
// some more rows than the mean, and a second tile each (8 experts at random, 104 rows
// 41 us against 48, 112 rows 51 against 64, 128 rows 49 against 69): a quarter more is
// counted.
bool narrow_codes(const Segments& s, int u) {
  const int64_t mean = s.pairs / s.E, rows = s.E > 1 ? mean + mean / 4 : mean;
  const int64_t busy = s.E < s.pairs ? s.E : s.pairs;
  const int64_t tiles = (rows + NarrowCodes::kBv - 1) / NarrowCodes::kBv *
                        ((u + NarrowCodes::kBu - 1) / NarrowCodes::kBu);
  return rows <= NarrowCodes::kBv || busy * tiles <= kUnits;
}

template <class C, int ACT>
hipError_t launch_tiles(const MatmulParams& p, hipStream_t st) {
  constexpr int kCols = Columns<C, ACT>::kTile;
  constexpr int kLds = TileProduct<C, false, false>::kLds;
  const int ntiles = (p.F + kCols - 1) / kCols;
  const int64_t grid = tile_bound(p.seg, C::kBv, ntiles);
  if (!launchable(grid, C::kThreads)) return hipErrorNotSupported;
  const hipError_t e = allow_lds<matmul_kernel<C, ACT>, kLds>();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((matmul_kernel<C, ACT>), dim3((unsigned)grid), dim3(C::kThreads), kLds, st, p,
                     ntiles);
  return hipGetLastError();
}

template <class Product, int ACT>
hipError_t launch_stream(const MatmulParams& p, hipStream_t st) {
  using C = typename Product::C;
  constexpr int kCols = Columns<C, ACT>::kTile;
  const int ntiles = (p.F + kCols - 1) / kCols;
  const int64_t grid = tile_bound(p.seg, C::kBv, ntiles);
  if (!launchable(grid, Product::kThreads)) return hipErrorNotSupported;
  const hipError_t e = allow_lds<matmul_stream_kernel<Product, ACT>, Product::kLds>();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((matmul_stream_kernel<Product, ACT>), dim3((unsigned)grid),
                     dim3(Product::kThreads), Product::kLds, st, p, ntiles);
  return hipGetLastError();
}

template <class C, int STAGES, int ACT>
hipError_t launch_codes(const MatmulParams& p, hipStream_t st) {
  constexpr int kCols = Columns<C, ACT>::kTile;
  constexpr int kLds = Fp8Product<C, STAGES>::kLds;
  const int ntiles = (p.F + kCols - 1) / kCols;
  const int64_t grid = tile_bound(p.seg, C::kBv, ntiles);
  if (!launchable(grid, C::kThreads)) return hipErrorNotSupported;
  const hipError_t e = allow_lds<matmul_fp8_kernel<C, STAGES, ACT>, kLds>();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((matmul_fp8_kernel<C, STAGES, ACT>), dim3((unsigned)grid), dim3(C::kThreads), kLds,
                     st, p, ntiles);
  return hipGetLastError();
}

template <int ACT>
hipError_t launch_forward(const MatmulParams& p, bool fp8, hipStream_t st) {
  if (fp8) {
    if (large_codes(p.seg, p.P)) return launch_codes<Codes, 2, ACT>(p, st);
    if (narrow_codes(p.seg, p.P)) return launch_codes<NarrowCodes, 2, ACT>(p, st);
    return launch_codes<FewCodes, 3, ACT>(p, st);
  }
  if (large_tiles(p.seg, p.P)) return launch_tiles<Large, ACT>(p, st);
  if (few_rows(p.seg, p.P)) return launch_stream<Few, ACT>(p, st);
  return launch_tiles<Mid, ACT>(p, st);
}

template <class C>
hipError_t launch_grad_x(const MatmulGradParams& p, const uint16_t* gz, hipStream_t st) {
  constexpr int kLds = TileProduct<C, true, false>::kLds;
  const int ntiles = (p.K + C::kBu - 1) / C::kBu;
  const int64_t grid = tile_bound(p.seg, C::kBv, ntiles);
  if (!launchable(grid, C::kThreads)) return hipErrorNotSupported;
  const hipError_t e = allow_lds<grad_x_kernel<C>, kLds>();
  if (e != hipSuccess || grid == 0) return e;
  hipLaunchKernelGGL((grad_x_kernel<C>), dim3((unsigned)grid), dim3(C::kThreads), kLds, st, p, gz,
                     ntiles);
  return hipGetLastError();
}

// BLOCKS to a compute unit.
template <class C, int BLOCKS>
hipError_t launch_grad_w(const MatmulGradParams& p, const uint16_t* gz, hipStream_t st) {
  constexpr int kLds = TileProduct<C, true, true>::kLds + kTableBytes;
  const unsigned nt = (p.K + C::kBu - 1) / C::kBu, pt = (p.P + C::kBv - 1) / C::kBv;
  const int64_t tiles = (int64_t)nt * pt * p.seg.E;
  if (tiles > INT32_MAX) return hipErrorNotSupported;
  const hipError_t e = allow_lds<grad_w_kernel<C>, kLds>();
  if (e != hipSuccess) return e;
  constexpr int kMost = kUnits * BLOCKS;
  hipLaunchKernelGGL((grad_w_kernel<C>), dim3((unsigned)(tiles < kMost ? tiles : kMost)),
                     dim3(C::kThreads), kLds, st, p, gz, nt, pt);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_matmul(const MatmulParams& p, bool fp8, hipStream_t st) {
  switch (p.act) {
    case kActSilu: return launch_forward<kActSilu>(p, fp8, st);
    case kActGelu: return launch_forward<kActGelu>(p, fp8, st);
    case kActSwiglu: return launch_forward<kActSwiglu>(p, fp8, st);
    default: return launch_forward<kActNone>(p, fp8, st);
  }
}

size_t gz_bytes(int rows, int P, int act) {
  return act == kActNone ? 0 : ((size_t)rows * P * 2 + 15) / 16 * 16;
}

size_t expert_matmul_grad_workspace(int rows, int pairs, int E, int P, int act) {
  if (pairs == 0) return 0;
  const int splits = act_splits(pairs, E, act == kActSwiglu ? P / 2 : P);
  return gz_bytes(rows, P, act) + (splits > 1 ? (size_t)splits * E * P * 4 : 0);
}

hipError_t launch_expert_matmul_grad(const MatmulGradParams& p, hipStream_t st) {
  if (p.grad_bias && (int64_t)p.seg.E * p.P > INT32_MAX) return hipErrorNotSupported;
  uint16_t* gz = p.act == kActNone ? nullptr : static_cast<uint16_t*>(p.workspace);
  if (p.grad_bias || p.act != kActNone) {
    const int splits = p.seg.pairs == 0 ? 1 : act_splits(p.seg.pairs, p.seg.E, p.F);
    float* parts = !p.grad_bias ? nullptr
                   : splits == 1
                       ? p.grad_bias
                       : reinterpret_cast<float*>(static_cast<char*>(p.workspace) +
                                                  gz_bytes(p.seg.rows, p.P, p.act));
    const dim3 grid((p.F + 511) / 512, p.seg.E, splits);
#define MOE_ACT_GRAD(ACT)                                                                     \
  hipLaunchKernelGGL((act_grad_kernel<ACT>), grid, dim3(kThreads), 0, st, p, gz, parts)
    switch (p.act) {
      case kActSilu: MOE_ACT_GRAD(kActSilu); break;
      case kActGelu: MOE_ACT_GRAD(kActGelu); break;
      case kActSwiglu: MOE_ACT_GRAD(kActSwiglu); break;
      default: MOE_ACT_GRAD(kActNone); break;
    }
#undef MOE_ACT_GRAD
    if (p.grad_bias && splits > 1) {
      const size_t n = (size_t)p.seg.E * p.P;
      hipLaunchKernelGGL(bias_grad_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)),
                         dim3(kThreads), 0, st, parts, p.grad_bias, n, splits);
    }
  }
  const uint16_t* g = gz ? gz : p.grad_y;
  const bool large = large_tiles(p.seg, p.K);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.grad_x)
    e = large ? launch_grad_x<Large>(p, g, st) : launch_grad_x<Mid>(p, g, st);
  if (e == hipSuccess && p.grad_weight)
    e = large_weight_tiles(p.seg, p.K, p.P) ? launch_grad_w<Large, 1>(p, g, st)
                                            : launch_grad_w<Mid, 2>(p, g, st);
  return e;
}

}  // namespace moe
