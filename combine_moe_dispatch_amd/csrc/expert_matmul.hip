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
// a tile of D in registers and walks r in steps of 64: while its four waves
// multiply one step out of LDS, the loads of the next go straight into the
// other half of it.
#include <type_traits>

#include "expert_tile.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// The tile product
// ---------------------------------------------------------------------------
// WU x WV waves of TU x TV fragments of 16 x 16.  A wave's fragments lie side
// by side along u and kWv apart along v, so that the rows of a part tile are
// spread over all waves.
template <int WU, int WV, int TU, int TV>
struct Config {
  static constexpr int kWu = WU, kWv = WV, kTu = TU, kTv = TV;
  static constexpr int kWaves = WU * WV, kThreads = kWaves * kWave;
  static constexpr int kBu = WU * TU * 16, kBv = WV * TV * 16;
};

template <class C, bool AT, bool BT>
struct TileProduct {
  using A = OperandTile<C::kBu, C::kWaves, AT, true>;
  using B = OperandTile<C::kBv, C::kWaves, BT, false>;
  static constexpr int kStage = A::kBytes + B::kBytes;
  static constexpr int kLds = 2 * kStage;
  static constexpr int kLoads = A::kLoads + B::kLoads;
  struct Fragments {
    bf16x8_t a[C::kTu], b[C::kTv];
  };
  A a;
  B b;
  f32x4_t acc[C::kTu][C::kTv];
  typename A::template Reader<C::kTu> ra;
  typename B::template Reader<C::kTv> rb;

  // Fragment i (of kTv + kTu) of part k of the step at lds.
  template <bool TAIL>
  __device__ __forceinline__ void read(Fragments& f, int i, uint32_t lds, int k, int left) const {
    if (i < C::kTv)
      f.b[i] = rb.template frag<TAIL>(lds + A::kBytes, i * (BT ? 1 : C::kWv), k, left);
    else
      f.a[i - C::kTv] = ra.template frag<TAIL>(lds, i - C::kTv, k, left);
  }
  template <bool TAIL>
  __device__ __forceinline__ void read_all(Fragments& f, uint32_t lds, int k, int left) const {
#pragma unroll
    for (int i = 0; i < C::kTv + C::kTu; ++i) read<TAIL>(f, i, lds, k, left);
  }

  // acc += f, row of fragments by row, with before(u) in front of row u: what
  // it issues runs beside the products.
  template <class Before>
  __device__ __forceinline__ void multiply(const Fragments& f, Before before) {
#pragma unroll
    for (int u = 0; u < C::kTu; ++u) {
      before(u);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int v = 0; v < C::kTv; ++v)
        mfma_in_place(acc[u][v], f.a[u], f.b[v]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int u = 0; u < C::kTu; ++u)
#pragma unroll
      for (int v = 0; v < C::kTv; ++v) acc[u][v] = f32x4_t{};
  }

  // red > 0 positions along r.  ap[i] is where load i of this wave starts in A
  // (weight rows of a gated layer lie in two places), bp in B; lda, ldb are
  // the operands' row pitches in bytes.
  __device__ __forceinline__ void run(char* smem, int wave, const char* (&ap)[A::kLoads],
                                      const char* bp, uint32_t lda, uint32_t ldb, int red) {
    static_assert(kParts == 2, "the parts are written out");
    ra.init(wave % C::kWu * C::kTu * 16);
    rb.init(wave / C::kWu * 16, C::kWv);
    clear();
    const size_t sta = AT ? (size_t)kStep * lda : (size_t)kStep * 2;
    const size_t stb = BT ? (size_t)kStep * ldb : (size_t)kStep * 2;
    uint32_t here = lds_address(smem), next = here + kStage;
    const int steps = (red + kStep - 1) / kStep;
    const int rest = red - (steps - 1) * kStep;       // positions of the last step
    const int whole = rest == kStep ? steps : steps - 1;
    auto advance = [&] {
#pragma unroll
      for (int i = 0; i < A::kLoads; ++i) ap[i] += sta;
      bp += stb;
    };
    auto load = [&](int i, uint32_t to, auto tail) {  // load i of the next step
      if (i < A::kLoads)
        a.template load<decltype(tail)::value>(i, to, wave, ap[i], lda, rest);
      else if (i < kLoads)
        b.template load<decltype(tail)::value>(i - A::kLoads, to + A::kBytes, wave, bp, ldb, rest);
    };
    auto start = [&](uint32_t to, bool full) {
      if (full) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load(i, to, std::false_type{});
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load(i, to, std::true_type{});
      }
      advance();
    };
    // Every wave's reads of `here` are in registers and its loads of `next` in
    // LDS: `here` may be filled again and `next` be read.
    auto meet = [&] {
      wait_lds();
      wait_vm<0>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    auto turn = [&] {
      const uint32_t h = here;
      here = next;
      next = h;
    };
    constexpr int kReads = (2 * (C::kTu + C::kTv) + C::kTu - 1) / C::kTu;  // in the first rows
    constexpr int kStarts = (kLoads + C::kTu - 1) / C::kTu;
    auto reading = [&](Fragments& f, uint32_t lds, int k, int u) {
#pragma unroll
      for (int i = u * kReads; i < (u + 1) * kReads; ++i)
        if (i < C::kTu + C::kTv) read<false>(f, i, lds, k, rest);
    };
    const auto nothing = [](int) {};
    Fragments f0, f1;
    start(here, whole > 0);
    if (steps > 1) {
      start(next, whole > 1);
      wait_vm<kLoads>();
    } else {
      wait_vm<0>();
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (steps > 1)
      read_all<false>(f0, here, 0, rest);
    else
      read_all<true>(f0, here, 0, rest);
    // Half a step is multiplied while the next half is read, the second half
    // behind the barrier, so that the matrix units have work on both sides.
    for (int t = 0; t + 2 < whole; ++t) {
      multiply(f0, [&](int u) { reading(f1, here, 1, u); });
      meet();
      multiply(f1, [&](int u) {
        reading(f0, next, 0, u);
#pragma unroll
        for (int i = u * kStarts; i < (u + 1) * kStarts; ++i) load(i, here, std::false_type{});
      });
      advance();
      turn();
    }
    if (whole < steps && steps > 2) {  // the step whose loads are the short ones
      multiply(f0, [&](int u) { reading(f1, here, 1, u); });
      meet();
      start(here, false);
      multiply(f1, [&](int u) { reading(f0, next, 0, u); });
      turn();
    }
    if (steps > 1) {
      multiply(f0, [&](int u) { reading(f1, here, 1, u); });
      meet();
      multiply(f1, nothing);
      read_all<true>(f0, next, 0, rest);
      turn();
    }
    read_all<true>(f1, here, 1, rest);
    multiply(f0, nothing);
    multiply(f1, nothing);
    mfma_results();
#pragma unroll
    for (int u = 0; u < C::kTu; ++u)
#pragma unroll
      for (int v = 0; v < C::kTv; ++v) mfma_result(acc[u][v]);
  }

  // This lane's outputs of fragments 2a and 2a + 1 by v: eight neighbours
  // along u from a * 32 + (lane >> 4) * 8 on, of the fragment's row lane & 15.
  __device__ __forceinline__ void eight(float (&o)[8], int a, int v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = acc[2 * a + i / 4][v][i % 4];
  }
};

// ---------------------------------------------------------------------------
// The same for e4m3 operands with a scale per 128 values along r: one step is
// one block of 128, whose products are summed by one 16 x 16 x 128 matrix
// instruction per fragment and then scaled in fp32, sx of the token times sw
// of the 128 weight rows.  A row of a step is 128 bytes, as in the bf16
// product, so the tiles in LDS are the same; the chunks of a fragment are
// taken in an order of their own, equal for both operands, which a sum does
// not notice.  Eight waves, and three steps in LDS: a serving batch has few
// rows an expert, so the weights stream through once and the loads in flight
// count.
// ---------------------------------------------------------------------------
template <class C>
struct Fp8Product {
  using A = OperandTile<C::kBu, C::kWaves, false, true>;
  using B = OperandTile<C::kBv, C::kWaves, false, false>;
  static constexpr int kScales = C::kWaves * 256;  // one dword a lane
  static_assert(C::kBv == C::kWaves * 32, "a wave brings in the scales of 32 rows");
  static constexpr int kStage = A::kBytes + B::kBytes + kScales;
  static constexpr int kStages = 3, kLds = kStages * kStage;
  static constexpr int kLoads = A::kLoads + B::kLoads + 1;
  A a;
  B b;
  f32x4_t acc[C::kTu][C::kTv];
  typename A::template Reader<C::kTu> ra;
  typename B::template Reader<C::kTv> rb;

  template <class R>
  static __device__ __forceinline__ i32x8_t frag(const R& r, uint32_t lds, int n) {
    union {
      bf16x8_t h[2];
      i32x8_t v;
    } u;
    u.h[0] = r.template frag<false>(lds, n, 0, 0);
    u.h[1] = r.template frag<false>(lds, n, 1, 0);
    return u.v;
  }

  // blocks > 0 steps.  scale: the scale this lane brings in, of step 0: lanes
  // 0-31 one of the wave's 32 x rows, lanes 32 and 33 those of the weight rows
  // behind the first and the second half of the wave's fragments.  (A plain
  // load of them would wait for every load to LDS before it.)  rows: how many
  // the tile has.
  __device__ __forceinline__ void run(char* smem, int wave, const char* (&ap)[A::kLoads],
                                      const char* bp, const float* scale, int blocks, int rows) {
    ra.init(wave % C::kWu * C::kTu * 16);
    rb.init(wave / C::kWu * 16);
#pragma unroll
    for (int u = 0; u < C::kTu; ++u)
#pragma unroll
      for (int v = 0; v < C::kTv; ++v) acc[u][v] = f32x4_t{};
    const uint32_t lds = lds_address(smem), lds_end = lds + kLds;
    uint32_t fill = lds, here = lds;
    auto after = [&](uint32_t slot) { return slot + kStage == lds_end ? lds : slot + kStage; };
    auto start = [&] {
#pragma unroll
      for (int i = 0; i < A::kLoads; ++i) {
        a.template load<false>(i, fill, wave, ap[i], 0, 0);
        ap[i] += 128;
      }
#pragma unroll
      for (int i = 0; i < B::kLoads; ++i)
        b.template load<false>(i, fill + A::kBytes, wave, bp, 0, 0);
      load4_to_lds(fill + A::kBytes + B::kBytes + wave * 256, scale);
      bp += 128;
      scale += 1;
      fill = after(fill);
    };
    start();
    if (blocks > 1) start();
    // the fragments of this wave that hold rows at all
    const int wv = wave / C::kWu;
    const int nv = min((rows - wv * 16 + C::kWv * 16 - 1) / (C::kWv * 16), C::kTv);
    // 32 rows of scales every 256 bytes, this wave's two behind its own 32
    const uint32_t scales = A::kBytes + B::kBytes;
    const uint32_t sw_at = scales + wave * 256 + 128;
    const uint32_t sx_at = scales + wv / 2 * 256 + wv % 2 * 64 + (lane_id() & 15) * 4;
    static_assert(C::kWv % 2 == 0, "a fragment's scales lie 256 bytes per two fragments on");
    auto lds_float = [](uint32_t p) {
      return *(const __attribute__((address_space(3))) float*)(uintptr_t)p;
    };
    for (int t = 0; t < blocks; ++t) {
      if (t + 1 < blocks)
        wait_vm<kLoads>();
      else
        wait_vm<0>();
      wait_lds();  // this wave has read the step before out
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (t + 2 < blocks) start();
      if (nv > 0) {
        const float sw[2] = {lds_float(here + sw_at), lds_float(here + sw_at + 4)};
        i32x8_t fa[C::kTu];
#pragma unroll
        for (int u = 0; u < C::kTu; ++u) fa[u] = frag(ra, here, u);
#pragma unroll
        for (int v = 0; v < C::kTv; ++v) {
          if (v >= nv) break;
          const i32x8_t fb = frag(rb, here + A::kBytes, v * C::kWv);
          const float sx = lds_float(here + sx_at + v * C::kWv / 2 * 256);
          f32x4_t part[C::kTu];
#pragma unroll
          for (int u = 0; u < C::kTu; ++u)
            part[u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[u], fb, f32x4_t{}, 0, 0,
                                                                       0, 0, 0, 0);
#pragma unroll
          for (int u = 0; u < C::kTu; ++u) {
            const float s = sx * sw[u < C::kTu / 2 ? 0 : 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[u][v][i] = fmaf(part[u][i], s, acc[u][v][i]);
          }
        }
      }
      here = after(here);
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
// at once; the splits' sums are added by a second launch.
// ---------------------------------------------------------------------------
constexpr int kActRows = 4;

__device__ __forceinline__ void load8(float (&v)[8], const uint16_t* p) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

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

// y (and pre): u runs over weight rows; a gated layer's wave takes half of its
// fragments from the gate rows and half from the up rows of the same columns.
template <class C, int ACT>
struct Columns {
  static constexpr bool kGated = ACT == kActSwiglu;
  static constexpr int kPairs = (kGated ? C::kTu / 2 : C::kTu) / 2;  // along the output's columns
  static constexpr int kWave = kPairs * 32;                          // output columns of a wave
  static constexpr int kTile = kWave * C::kWu;                       // and of the tile
};

// This wave's loads of weight rows: w is the first of the tile's (gate) rows,
// cols how many columns are left from there, ld the bytes of a row.
template <class C, int ACT, class A>
__device__ __forceinline__ void weight_loads(A& a, const char* (&ap)[A::kLoads], const char* w,
                                             int wave, int F, int cols, uint32_t ld) {
  using Cols = Columns<C, ACT>;
#pragma unroll
  for (int i = 0; i < A::kLoads; ++i) {
    const int q = wave * A::kLoads + i;
    int row, c;
    A::chunk_of(q, row, c);
    const int first = q * A::kRowsPerLoad;  // the load's rows are of one kind
    const bool up = Cols::kGated && first % (2 * Cols::kWave) >= Cols::kWave;
    const int col =
        Cols::kGated ? row / (2 * Cols::kWave) * Cols::kWave + row % Cols::kWave : row;
    a.off[i] = (uint32_t)min(col, cols - 1) * ld + (uint32_t)c * 16;
    a.where[i] = (uint16_t)(c * 8);
    ap[i] = w + (up ? (size_t)F * ld : 0);
  }
}

// Bias, activation and residual on the accumulators, then the one rounding.
template <class C, int ACT, class Product>
__device__ __forceinline__ void finish(const Product& prod, const MatmulParams& p, const Tile& t,
                                       int wave) {
  using Cols = Columns<C, ACT>;
  const int wu = wave % C::kWu, wv = wave / C::kWu, lane = lane_id();
#pragma unroll
  for (int v = 0; v < C::kTv; ++v) {
    const int m = t.m0 + (v * C::kWv + wv) * 16 + (lane & 15);
    if (m >= t.end) continue;
#pragma unroll
    for (int a = 0; a < Cols::kPairs; ++a) {
      const int col = t.n * Cols::kTile + wu * Cols::kWave + a * 32 + (lane >> 4) * 8;
      if (col >= p.F) continue;
      float z[8], up[8];
      prod.eight(z, a, v);
      if (Cols::kGated) prod.eight(up, a + Cols::kPairs, v);
      if (p.bias) {
        const float* b = p.bias + (size_t)t.e * p.P + col;
        add8(z, b);
        if (Cols::kGated) add8(up, b + p.F);
      }
      if (p.pre) {
        store8(p.pre + (size_t)m * p.P + col, z);
        if (Cols::kGated) store8(p.pre + (size_t)m * p.P + p.F + col, up);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        z[i] = Cols::kGated ? z[i] * sigmoid_f32(z[i]) * up[i] : act_f32<ACT>(z[i]);
      const size_t at = (size_t)m * p.F + col;
      if (p.residual) add8(z, p.residual + at);
      store8(p.y + at, z);
    }
  }
}

template <class C, int ACT>
__global__ void __launch_bounds__(C::kThreads)
matmul_kernel(MatmulParams p, int ntiles) {
  using Product = TileProduct<C, false, false>;
  extern __shared__ __align__(1024) char smem[];
  Tile t;
  if (!find_tile<C::kBv>(p.seg, ntiles, blockIdx.x, t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = t.n * Columns<C, ACT>::kTile;
  const uint32_t ld = (uint32_t)p.K * 2;
  Product prod;
  const char* ap[Product::A::kLoads];
  weight_loads<C, ACT>(prod.a, ap,
                       static_cast<const char*>(p.weight) + ((size_t)t.e * p.P + n0) * ld, wave,
                       p.F, p.F - n0, ld);
  prod.b.init(wave, ld, min(C::kBv, t.end - t.m0));
  prod.run(smem, wave, ap, static_cast<const char*>(p.x) + (size_t)t.m0 * ld, ld, ld, p.K);
  finish<C, ACT>(prod, p, t, wave);
}

template <class C, int ACT>
__global__ void __launch_bounds__(C::kThreads)
matmul_fp8_kernel(MatmulParams p, int ntiles) {
  using Product = Fp8Product<C>;
  using Cols = Columns<C, ACT>;
  extern __shared__ __align__(1024) char smem[];
  Tile t;
  if (!find_tile<C::kBv>(p.seg, ntiles, blockIdx.x, t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = t.n * Cols::kTile, kb = p.K / 128;
  const uint32_t ld = (uint32_t)p.K;
  const int rows = min(C::kBv, t.end - t.m0);
  Product prod;
  const char* ap[Product::A::kLoads];
  weight_loads<C, ACT>(prod.a, ap,
                       static_cast<const char*>(p.weight) + ((size_t)t.e * p.P + n0) * ld, wave,
                       p.F, p.F - n0, ld);
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
  prod.run(smem, wave, ap, static_cast<const char*>(p.x) + (size_t)t.m0 * ld, scale, kb, rows);
  finish<C, ACT>(prod, p, t, wave);
}

// The accumulators as bf16 rows: row v of the tile to out + v * ld, for v
// below rows, columns below cols.
template <class C, class Product>
__device__ __forceinline__ void store_tile(const Product& prod, int wave, uint16_t* out, size_t ld,
                                           int rows, int cols) {
  const int wu = wave % C::kWu, wv = wave / C::kWu, lane = lane_id();
#pragma unroll
  for (int v = 0; v < C::kTv; ++v) {
    const int m = (v * C::kWv + wv) * 16 + (lane & 15);
    if (m >= rows) continue;
#pragma unroll
    for (int a = 0; a < C::kTu / 2; ++a) {
      const int c = (wu * C::kTu + 2 * a) * 16 + (lane >> 4) * 8;
      float o[8];
      prod.eight(o, a, v);
      if (c < cols) store8(out + (size_t)m * ld + c, o);
    }
  }
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
  const uint32_t lda = (uint32_t)p.K * 2, ldb = (uint32_t)p.P * 2;
  Product prod;
  prod.a.init(wave, lda, min(C::kBu, p.K - n0));
  prod.b.init(wave, ldb, min(C::kBv, t.end - t.m0));
  const char* ap[Product::A::kLoads];
#pragma unroll
  for (int i = 0; i < Product::A::kLoads; ++i)
    ap[i] = reinterpret_cast<const char*>(p.weight + (size_t)t.e * p.P * p.K + n0);
  prod.run(smem, wave, ap, reinterpret_cast<const char*>(gz) + (size_t)t.m0 * ldb, lda, ldb, p.P);
  store_tile<C>(prod, wave, p.grad_x + (size_t)t.m0 * p.K + n0, p.K, t.end - t.m0, p.K - n0);
}

// grad_w: D[input feature][weight row], summed over the expert's rows.
template <class C>
__global__ void __launch_bounds__(C::kThreads)
grad_w_kernel(MatmulGradParams p, const uint16_t* gz, unsigned nt, unsigned pt) {
  using Product = TileProduct<C, true, true>;
  extern __shared__ __align__(1024) char smem[];
  const unsigned b = xcd_local_block(blockIdx.x, gridDim.x);
  const int e = (int)(b / (nt * pt));
  const unsigned in = b % (nt * pt);
  const int n0 = (int)(in / pt) * C::kBu, p0 = (int)(in % pt) * C::kBv;
  int begin, end;
  segment_of(p.seg, e, begin, end);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t lda = (uint32_t)p.K * 2, ldb = (uint32_t)p.P * 2;
  Product prod;
  if (end > begin) {
    prod.a.init(wave, lda, min(C::kBu, p.K - n0));
    prod.b.init(wave, ldb, min(C::kBv, p.P - p0));
    const char* ap[Product::A::kLoads];
#pragma unroll
    for (int i = 0; i < Product::A::kLoads; ++i)
      ap[i] = reinterpret_cast<const char*>(p.x + (size_t)begin * p.K + n0);
    prod.run(smem, wave, ap, reinterpret_cast<const char*>(gz + (size_t)begin * p.P + p0), lda,
             ldb, end - begin);
  } else {
    prod.clear();
  }
  store_tile<C>(prod, wave, p.grad_weight + ((size_t)e * p.P + p0) * p.K + n0, p.K, p.P - p0,
                p.K - n0);
}

// 256 x 256 tiles for experts of many rows, 256 x 128 for those of few: a part
// tile wastes the products of its missing rows.
using Large = Config<2, 2, 8, 8>;
using Small = Config<2, 2, 8, 4>;

// Large tiles where an expert has more rows than one small tile on average
// and the large tiles alone fill the 256 compute units.
#ifndef GXL
#define GXL Large
#endif
#ifndef GWL
#define GWL Large
#endif
using Mid = Config<2, 2, 4, 4>;
// fp8: 128 weight rows by 256 token rows, so that an expert's weights are read
// once however its 128 or so rows fall.
using Codes = Config<2, 4, 4, 4>;

bool large_tiles(const Segments& s, int u) {
  const int64_t tiles = ((int64_t)s.pairs / Large::kBv) * ((u + Large::kBu - 1) / Large::kBu);
  return s.pairs / s.E > Small::kBv && tiles >= 256;
}

template <class K>
hipError_t allow_lds(K kernel, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <class C, int ACT, class Product, class Kernel>
hipError_t launch_tiles(Kernel kernel, const MatmulParams& p, hipStream_t st) {
  constexpr int kCols = Columns<C, ACT>::kTile;
  const int ntiles = (p.F + kCols - 1) / kCols;
  const int64_t grid = tile_bound(p.seg, C::kBv, ntiles);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  const hipError_t e = allow_lds(kernel, Product::kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(C::kThreads), Product::kLds, st, p, ntiles);
  return hipGetLastError();
}

template <int ACT>
hipError_t launch_forward(const MatmulParams& p, bool fp8, hipStream_t st) {
  if (fp8) return launch_tiles<Codes, ACT, Fp8Product<Codes>>(matmul_fp8_kernel<Codes, ACT>, p, st);
  if (large_tiles(p.seg, p.P))
    return launch_tiles<Large, ACT, TileProduct<Large, false, false>>(matmul_kernel<Large, ACT>, p,
                                                                      st);
  return launch_tiles<Small, ACT, TileProduct<Small, false, false>>(matmul_kernel<Small, ACT>, p,
                                                                    st);
}

template <class C>
hipError_t launch_grad_x(const MatmulGradParams& p, const uint16_t* gz, hipStream_t st) {
  constexpr int kLds = TileProduct<C, true, false>::kLds;
  const int ntiles = (p.K + C::kBu - 1) / C::kBu;
  const int64_t grid = tile_bound(p.seg, C::kBv, ntiles);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  const hipError_t e = allow_lds(grad_x_kernel<C>, kLds);
  if (e != hipSuccess || grid == 0) return e;
  hipLaunchKernelGGL((grad_x_kernel<C>), dim3((unsigned)grid), dim3(C::kThreads), kLds, st, p, gz,
                     ntiles);
  return hipGetLastError();
}

template <class C>
hipError_t launch_grad_w(const MatmulGradParams& p, const uint16_t* gz, hipStream_t st) {
  constexpr int kLds = TileProduct<C, true, true>::kLds;
  const unsigned nt = (p.K + C::kBu - 1) / C::kBu, pt = (p.P + C::kBv - 1) / C::kBv;
  const int64_t grid = (int64_t)nt * pt * p.seg.E;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  const hipError_t e = allow_lds(grad_w_kernel<C>, kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((grad_w_kernel<C>), dim3((unsigned)grid), dim3(C::kThreads), kLds, st, p, gz,
                     nt, pt);
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
    e = large ? launch_grad_x<GXL>(p, g, st) : launch_grad_x<Small>(p, g, st);
  if (e == hipSuccess && p.grad_weight)
    e = (int64_t)p.K * p.P >= 256 * 256 ? launch_grad_w<GWL>(p, g, st)
                                        : launch_grad_w<Small>(p, g, st);
  return e;
}

}  // namespace moe
