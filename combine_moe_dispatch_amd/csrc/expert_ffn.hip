// expert_ffn.hip -- the experts' gated feed-forward block in 8 bits and its
// gradient.
//
//   z = x Wu^T, h = silu(z1) z2, y = q(h) Wd^T
//   gh = q(gy) Wd, gz = act'(z) gh, gx = q(gz) Wu, gWu = gz^T x, gWd = gy^T h
//
// with q the rounding of rows to e4m3 in blocks of 128 columns.  The products
// with the weights are those of expert_product.h, one step one scale block:
//   h      u = gate and up rows of 128 columns, v = token row, r = column of x
//   gh, gx u = weight column, v = token row, r = weight row (weights transposed)
// A tile has all columns of a scale block, so that rows are rounded to 8 bits where
// they are made, from the fp32 sums, and the activation and its slope need no pass
// of their own.  The weights' gradients are expert_matmul's, in bf16: they are
// added up over many steps, and 2^-4 a factor would be their largest error by far.
#include "expert_product.h"
#include "ffn.h"
#include "quantize.h"

namespace moe {

namespace {

// 256 columns of u by 256 token rows in two steps of LDS (Codes), or by 128 in
// three.  NarrowCodes: 128 by 128, two blocks to a compute unit.
using ShortCodes = Config<2, 4, 8, 2>;
// 256 by 64.
using FlatCodes = Config<2, 4, 8, 1>;
template <class C>
constexpr int kStages = C::kTv == 4 || C::kTu == 4 ? 2 : 3;

// ---------------------------------------------------------------------------
// Forward: h
// ---------------------------------------------------------------------------
struct UpParams {
  Segments seg;
  const uint8_t* x;
  const float* x_scales;
  const uint8_t* up;
  const float* up_scales;
  uint16_t* pre;
  uint8_t* h;
  float* h_scales;
  int H, I;
};

// The gated activation on the accumulators, then rows of 128 columns to 8 bits.
// A wave has 64 of the columns; the largest magnitudes meet in LDS.
template <class C, class Product>
__device__ __forceinline__ void finish_up(Product& prod, const UpParams& p, const Tile& t,
                                          int wave, uint32_t* s_largest) {
  using Cols = Columns<C, kActSwiglu>;
  static_assert(Cols::kTile == kFp8Block, "a tile is one block of columns");
  const int wu = wave % C::kWu, wv = wave / C::kWu, lane = lane_id();
  const int col0 = t.n * kFp8Block + wu * Cols::kWave + (lane >> 4) * 8;
#pragma unroll
  for (int v = 0; v < C::kTv; ++v) {
    const int row = (v * C::kWv + wv) * 16 + (lane & 15), m = t.m0 + row;
    uint32_t largest = 0;
#pragma unroll
    for (int a = 0; a < Cols::kPairs; ++a) {
      float z[8], up[8];
      prod.eight(z, a, v);
      prod.eight(up, a + Cols::kPairs, v);
      if (p.pre && m < t.end) {
        uint16_t* pre = p.pre + (size_t)m * (2 * p.I) + col0 + a * 32;
        store8(pre, z);
        store8(pre + p.I, up);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[i] = z[i] * sigmoid_short(z[i]) * up[i];
        largest = max(largest, magnitude(z[i]));
        prod.acc[2 * a + i / 4][v][i % 4] = z[i];
      }
    }
    largest = max_over_rows(largest);
    if (lane < 16) s_largest[wu * C::kBv + row] = largest;
  }
  lds_barrier();
#pragma unroll
  for (int v = 0; v < C::kTv; ++v) {
    const int row = (v * C::kWv + wv) * 16 + (lane & 15), m = t.m0 + row;
    if (m >= t.end) continue;
    uint32_t largest = 0;
#pragma unroll
    for (int w = 0; w < C::kWu; ++w) largest = max(largest, s_largest[w * C::kBv + row]);
    const BlockScale block(largest);
#pragma unroll
    for (int a = 0; a < Cols::kPairs; ++a) {
      float h[8];
      prod.eight(h, a, v);
      *reinterpret_cast<uint2*>(p.h + (size_t)m * p.I + col0 + a * 32) = block.codes(h);
    }
    if (wu == 0 && lane < 16) p.h_scales[(size_t)m * (p.I / kFp8Block) + t.n] = block.scale;
  }
}

template <class C, class Product>
__device__ __forceinline__ void up_product(Product& prod, char* smem, const UpParams& p,
                                           const Tile& t, int wave) {
  using Cols = Columns<C, kActSwiglu>;
  const int kb = p.H / kFp8Block, ib = p.I / kFp8Block, lane = lane_id();
  const int n0 = t.n * Cols::kTile;
  const uint32_t ld = (uint32_t)p.H;
  const int rows = min(C::kBv, t.end - t.m0);
  prod.template weight_rows<true>(
      wave, reinterpret_cast<const char*>(p.up) + ((size_t)t.e * 2 * p.I + n0) * ld, ld, p.I - n0,
      (size_t)p.I * ld);
  prod.b.init(wave, ld, rows);
  const float* scale =
      lane < 32 ? p.x_scales + (size_t)(t.m0 + min(wave * 32 + lane, rows - 1)) * kb
                : p.up_scales +
                      ((size_t)t.e * 2 * ib + n0 / kFp8Block + (lane % 2 == 1 ? ib : 0)) * kb;
  prod.run_rows(smem, wave, reinterpret_cast<const char*>(p.x) + (size_t)t.m0 * ld, scale, kb,
                rows);
}

template <class C>
constexpr int kUpLds = Fp8Product<C, kStages<C>>::kLds + C::kWu * C::kBv * 4;

// 4096 tokens, top-8 of 32 experts of 7168 x 2048: 884 us, 2.2 PFLOP/s (a large
// product with one scale 3.1); the matrix units are 48 % busy.  The sums are scaled by
// vector instructions and so fill the vector registers: eight waves of 128 x 64, which
// read 192 KB out of LDS a step and bring 64 KB in, 2048 cycles at 128 bytes a cycle and
// as many as their products take.  First loads, activation and stores take 163 us.  128
// tokens: the weights' way from memory, 5.5 TB/s in 168 us.
template <class C>
__global__ void __launch_bounds__(C::kThreads)
ffn_up_kernel(UpParams p, int ntiles) {
  using Product = Fp8Product<C, kStages<C>>;
  extern __shared__ __align__(1024) char smem[];
  Tile t;
  if (!find_tile<C::kBv>(p.seg, ntiles, blockIdx.x, t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  Product prod;
  up_product<C>(prod, smem, p, t, wave);
  finish_up<C>(prod, p, t, wave, reinterpret_cast<uint32_t*>(smem + Product::kLds));
}

// ---------------------------------------------------------------------------
// Few tiles: the steps of a tile are shared out over the blocks of gridDim.y, whose
// sums lie behind one another in fp32; a launch of its own adds them up and does
// what comes after the product.  One token's way through one expert is its weights'
// way from memory, and 32 tiles of 56 steps would leave that to 32 compute units.
// The sums lie row behind placed row: a receive buffer of fixed capacity has room for
// many more (128 tokens of 32 ranks of 4096: 131072 rows, of which 1024 are placed).
// ---------------------------------------------------------------------------
// Which of the placed rows the tile's first one is.
__device__ __forceinline__ int placed_row(const Segments& s, const Tile& t) {
  if (s.rows == s.pairs) return t.m0;  // any row will do
  const int lane = lane_id();
  int n = 0;
  for (int base = 0; base <= t.e; base += kWave) {
    if (base + lane > t.e) continue;
    int begin, end;
    segment_of(s, base + lane, begin, end);
    n += base + lane == t.e ? t.m0 - begin : max(end - begin, 0);
  }
  return __builtin_amdgcn_readlane(wave_inclusive_sum_dpp(n), 63);
}

struct SplitParams {
  Segments seg;
  const uint8_t* x;
  const float* x_scales;
  const uint8_t* weight;
  const float* weight_scales;
  float* parts;  // [gridDim.y][seg.pairs][P]
  int K, P;
};

template <class C>
__global__ void __launch_bounds__(C::kThreads)
ffn_split_kernel(SplitParams p, int ntiles) {
  using Product = Fp8Product<C, kStages<C>>;
  static_assert(C::kBu == kFp8Block, "a tile's weight rows are one block of scales");
  extern __shared__ __align__(1024) char smem[];
  Tile t;
  if (!find_tile<C::kBv>(p.seg, ntiles, blockIdx.x, t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const int kb = p.K / kFp8Block, rows = min(C::kBv, t.end - t.m0);
  const int placed = placed_row(p.seg, t);
  // every share has a step (the launch sees to that)
  const int first = (int)((int64_t)kb * blockIdx.y / gridDim.y);
  const int last = (int)((int64_t)kb * (blockIdx.y + 1) / gridDim.y);
  const uint32_t ld = (uint32_t)p.K;
  Product prod;
  prod.template weight_rows<false>(
      wave,
      reinterpret_cast<const char*>(p.weight) + ((size_t)t.e * p.P + t.n * C::kBu) * ld +
          first * kFp8Block,
      ld, p.P - t.n * C::kBu, 0);
  prod.b.init(wave, ld, rows);
  const float* scale =
      lane < 32 ? p.x_scales + (size_t)(t.m0 + min(wave * 32 + lane, rows - 1)) * kb
                : p.weight_scales + ((size_t)t.e * (p.P / kFp8Block) + t.n) * kb;
  prod.run_rows(smem, wave,
                reinterpret_cast<const char*>(p.x) + (size_t)t.m0 * ld + first * kFp8Block,
                scale + first, last - first, rows);
  const int wu = wave % C::kWu, wv = wave / C::kWu;
#pragma unroll
  for (int v = 0; v < C::kTv; ++v) {
    const int row = (v * C::kWv + wv) * 16 + (lane & 15), at = placed + row;
    if (row >= rows || at >= p.seg.pairs) continue;  // (whatever the counts say)
    float* out = p.parts + ((size_t)blockIdx.y * p.seg.pairs + at) * p.P + t.n * C::kBu;
#pragma unroll
    for (int a = 0; a < C::kTu / 2; ++a) {
      float o[8];
      prod.eight(o, a, v);
      float4* q = reinterpret_cast<float4*>(out + Product::column(wu, a));
      q[0] = make_float4(o[0], o[1], o[2], o[3]);
      q[1] = make_float4(o[4], o[5], o[6], o[7]);
    }
  }
}

// Eight neighbouring sums of a row from their shares, in the shares' order.
__device__ __forceinline__ void add_shares(float (&v)[8], const float* parts, size_t apart,
                                           int shares) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < shares; ++s) add8(v, parts + s * apart);
}

constexpr int kJoinRows = 4, kJoinThreads = 256;

// h and its 8 bits from the shares of z.
__global__ void __launch_bounds__(kJoinThreads)
ffn_join_up_kernel(UpParams p, const float* parts, int shares) {
  Tile t;
  if (!find_tile<kJoinRows>(p.seg, 1, blockIdx.x, t)) return;
  const int placed = placed_row(p.seg, t), units = p.I / 8;
  const int rows = min(min(kJoinRows, t.end - t.m0), p.seg.pairs - placed);
  const size_t apart = (size_t)p.seg.pairs * (2 * p.I);
  // units per row are a multiple of 16: the 16 lanes of a scale block stay together
  for (int i = blockIdx.y * kJoinThreads + threadIdx.x; i < rows * units;
       i += gridDim.y * kJoinThreads) {
    const size_t m = t.m0 + i / units;
    const int c = i % units * 8;
    const float* z = parts + ((size_t)placed + i / units) * (2 * p.I) + c;
    float g[8], u[8];
    add_shares(g, z, apart, shares);
    add_shares(u, z + p.I, apart, shares);
    if (p.pre) {
      store8(p.pre + m * (2 * p.I) + c, g);
      store8(p.pre + m * (2 * p.I) + p.I + c, u);
    }
    uint32_t largest = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = g[j] * sigmoid_short(g[j]) * u[j];
      largest = max(largest, magnitude(g[j]));
    }
    const BlockScale block(max_over_16(largest));
    const size_t at = m * p.I + c;
    *reinterpret_cast<uint2*>(p.h + at) = block.codes(g);
    if (threadIdx.x % 16 == 0) p.h_scales[at / kFp8Block] = block.scale;
  }
}

// y from its shares.
__global__ void __launch_bounds__(kJoinThreads)
ffn_join_down_kernel(Segments seg, const float* parts, int shares, const uint16_t* residual,
                     uint16_t* y, int H) {
  Tile t;
  if (!find_tile<kJoinRows>(seg, 1, blockIdx.x, t)) return;
  const int placed = placed_row(seg, t), units = H / 8;
  const int rows = min(min(kJoinRows, t.end - t.m0), seg.pairs - placed);
  for (int i = blockIdx.y * kJoinThreads + threadIdx.x; i < rows * units;
       i += gridDim.y * kJoinThreads) {
    const size_t at = (size_t)t.m0 * H + (size_t)i * 8;
    float v[8];
    add_shares(v, parts + (size_t)placed * H + (size_t)i * 8, (size_t)seg.pairs * H, shares);
    if (residual) add8(v, residual + at);
    store8(y + at, v);
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// Placed rows of grad_y to 8 bits and of x to bf16 (code times scale, half a bf16
// step off: a token's scale cannot be taken out of a sum over tokens, and what the
// rounding leaves would be a second product; NULL: not wanted): a stream, 4 rows a block
// (16384 rows of 7168: 705 MB in 158 us, 4.5 TB/s).
constexpr int kPrepareRows = 4, kPrepareThreads = 256;

struct PrepareParams {
  Segments seg;
  const uint16_t* grad_y;
  uint8_t* gy;
  float* gy_scales;
  const uint8_t* x;
  const float* x_scales;
  uint16_t* wide_x;
  int H;
};

__global__ void __launch_bounds__(kPrepareThreads)
ffn_prepare_kernel(PrepareParams p) {
  Tile t;
  if (!find_tile<kPrepareRows>(p.seg, 1, blockIdx.x, t)) return;
  const int rows = min(kPrepareRows, t.end - t.m0), units = p.H / 8;
  // units per row are a multiple of 16: the 16 lanes of a scale block stay together
  for (int i = threadIdx.x; i < rows * units; i += kPrepareThreads) {
    const size_t at = (size_t)t.m0 * p.H + (size_t)i * 8;
    float v[8];
    load8(v, p.grad_y + at);
    uint32_t largest = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) largest = max(largest, magnitude(v[j]));
    const BlockScale block(max_over_16(largest));
    *reinterpret_cast<uint2*>(p.gy + at) = block.codes(v);
    if (threadIdx.x % 16 == 0) p.gy_scales[at / kFp8Block] = block.scale;
    if (p.wide_x) {
      const uint2 q = *reinterpret_cast<const uint2*>(p.x + at);
      const float s = p.x_scales[at / kFp8Block];
      e4m3x4_to_f32(q.x, v);
      e4m3x4_to_f32(q.y, v + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= s;
      store8(p.wide_x + at, v);
    }
  }
}

// h alone, where only the second weight's gradient is wanted.
__global__ void __launch_bounds__(kPrepareThreads)
ffn_hidden_kernel(Segments seg, const uint16_t* pre, uint16_t* h, int I) {
  Tile t;
  if (!find_tile<kPrepareRows>(seg, 1, blockIdx.x, t)) return;
  const int rows = min(kPrepareRows, t.end - t.m0), units = I / 8;
  for (int i = threadIdx.x; i < rows * units; i += kPrepareThreads) {
    const size_t m = t.m0 + i / units;
    const int c = i % units * 8;
    float g[8], u[8];
    load8(g, pre + m * (2 * I) + c);
    load8(u, pre + m * (2 * I) + I + c);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = g[j] * sigmoid_short(g[j]) * u[j];
    store8(h + m * I + c, g);
  }
}

struct SlopeParams {
  Segments seg;
  const uint8_t* gy;
  const float* gy_scales;
  const uint8_t* down;
  const float* down_scales;
  const uint16_t* pre;
  uint8_t* gz;         // rows of 2I in 8 bits, or NULL
  float* gz_scales;
  uint16_t* wide_gz;   // the same in bf16, or NULL
  uint16_t* h;         // rows of I in bf16, or NULL
  int H, I;
};

// The slope of the activation on the accumulators; a wave has all 128 columns of a
// scale block, of the gate's and of the up half's gradient.  A row's pre-activations
// are loaded in front of the row's before it, whose stores they would else wait for.
// 16384 rows, 32 experts of 7168 x 2048: 454 us, of which the products alone would
// take 154 at a large product's rate; 400 MB are read and written behind them, and a
// block has its compute unit to itself.
template <class C, class Product>
__device__ __forceinline__ void finish_slope(Product& prod, const SlopeParams& p, const Tile& t,
                                             int wave) {
  constexpr int kPairs = C::kTu / 2;
  static_assert(kPairs * 32 == kFp8Block, "a wave's columns are one block");
  const int wu = wave % C::kWu, wv = wave / C::kWu, lane = lane_id();
  const int col0 = (t.n * C::kWu + wu) * kFp8Block;
  if (col0 >= p.I) return;
  const int P = 2 * p.I, pb = P / kFp8Block;
  const auto row_of = [&](int v) { return t.m0 + (v * C::kWv + wv) * 16 + (lane & 15); };
  const auto column = [&](int a) { return t.n * C::kBu + Product::column(wu, a); };
  struct Pre {
    uint4 g[kPairs], u[kPairs];
  };
  const auto load = [&](Pre& q, int v) {
    const uint16_t* pre = p.pre + (size_t)min(row_of(v), t.end - 1) * P;
#pragma unroll
    for (int a = 0; a < kPairs; ++a) {
      q.g[a] = *reinterpret_cast<const uint4*>(pre + column(a));
      q.u[a] = *reinterpret_cast<const uint4*>(pre + column(a) + p.I);
    }
  };
  Pre here, next;
  load(here, 0);
#pragma unroll
  for (int v = 0; v < C::kTv; ++v) {
    if (v + 1 < C::kTv) load(next, v + 1);
    const int m = row_of(v);
    const bool there = m < t.end;
    const size_t at = (size_t)m * P;
    float du[kPairs][8];
    uint32_t largest_g = 0, largest_u = 0;
#pragma unroll
    for (int a = 0; a < kPairs; ++a) {
      float dg[8], g[8], u[8], h[8];
      prod.eight(dg, a, v);
      unpack8(g, here.g[a]);
      unpack8(u, here.u[a]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = sigmoid_short(g[i]), silu = g[i] * s;
        du[a][i] = dg[i] * silu;
        dg[i] = dg[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
        h[i] = silu * u[i];
        largest_g = max(largest_g, magnitude(dg[i]));
        largest_u = max(largest_u, magnitude(du[a][i]));
        prod.acc[2 * a + i / 4][v][i % 4] = dg[i];
      }
      if (there && p.h) store8(p.h + (size_t)m * p.I + column(a), h);
      if (there && p.wide_gz) {
        store8(p.wide_gz + at + column(a), dg);
        store8(p.wide_gz + at + column(a) + p.I, du[a]);
      }
    }
    if (p.gz) {
      const BlockScale gate(max_over_rows(largest_g)), up(max_over_rows(largest_u));
      if (there) {
#pragma unroll
        for (int a = 0; a < kPairs; ++a) {
          float dg[8];
          prod.eight(dg, a, v);
          *reinterpret_cast<uint2*>(p.gz + at + column(a)) = gate.codes(dg);
          *reinterpret_cast<uint2*>(p.gz + at + column(a) + p.I) = up.codes(du[a]);
        }
        if (lane < 16) {
          float* scales = p.gz_scales + (size_t)m * pb + col0 / kFp8Block;
          scales[0] = gate.scale;
          scales[pb / 2] = up.scale;
        }
      }
    }
    here = next;
  }
}

// The product with transposed weights, rows of `cols` columns: sums over `red`
// weight rows.
template <class C, class Product>
__device__ __forceinline__ void transposed_product(Product& prod, char* smem, const Tile& t,
                                                   int wave, const uint8_t* rows_codes,
                                                   const float* row_scales, const uint8_t* weight,
                                                   const float* weight_scales, int red, int cols) {
  const int lane = lane_id(), rb = red / kFp8Block, cb = cols / kFp8Block, n0 = t.n * C::kBu;
  const int rows = min(C::kBv, t.end - t.m0);
  prod.weight_columns(wave, reinterpret_cast<const char*>(weight) + (size_t)t.e * red * cols + n0,
                      (uint32_t)cols, cols - n0);
  prod.b.init(wave, (uint32_t)red, rows);
  // half a wave's columns lie in one block of scales; past the last column any will do
  static_assert(kFp8Block % Product::kHalfRows == 0, "one scale half a wave");
  const int block =
      min(n0 + Product::place(lane % 2, wave % C::kWu * Product::kHalfRows), cols - 1) / kFp8Block;
  const float* scale =
      lane < 32 ? row_scales + (size_t)(t.m0 + min(wave * 32 + lane, rows - 1)) * rb
                : weight_scales + (size_t)t.e * rb * cb + block;
  prod.scale_step = lane < 32 ? 1 : cb;
  prod.run_rows(smem, wave, reinterpret_cast<const char*>(rows_codes) + (size_t)t.m0 * red, scale,
                rb, rows);
  prod.exchange();
}

template <class C>
__global__ void __launch_bounds__(C::kThreads)
ffn_slope_kernel(SlopeParams p, int ntiles) {
  using Product = Fp8Product<C, kStages<C>, true>;
  extern __shared__ __align__(1024) char smem[];
  Tile t;
  if (!find_tile<C::kBv>(p.seg, ntiles, blockIdx.x, t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  Product prod;
  transposed_product<C>(prod, smem, t, wave, p.gy, p.gy_scales, p.down, p.down_scales, p.H, p.I);
  finish_slope<C>(prod, p, t, wave);
}

// Stores alone behind the products: 16384 rows, 32 experts of 7168 x 2048 557 us, the
// matrix units 38 % busy.
struct RowGradParams {
  Segments seg;
  const uint8_t* gz;
  const float* gz_scales;
  const uint8_t* up;
  const float* up_scales;
  uint16_t* grad_x;
  int H, I;
};

template <class C>
__global__ void __launch_bounds__(C::kThreads)
ffn_grad_x_kernel(RowGradParams p, int ntiles) {
  using Product = Fp8Product<C, kStages<C>, true, true>;
  extern __shared__ __align__(1024) char smem[];
  Tile t;
  if (!find_tile<C::kBv>(p.seg, ntiles, blockIdx.x, t)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  Product prod;
  transposed_product<C>(prod, smem, t, wave, p.gz, p.gz_scales, p.up, p.up_scales, 2 * p.I, p.H);
  const int wu = wave % C::kWu, wv = wave / C::kWu, lane = lane_id();
#pragma unroll
  for (int v = 0; v < C::kTv; ++v) {
    const int m = t.m0 + (v * C::kWv + wv) * 16 + (lane & 15);
#pragma unroll
    for (int a = 0; a < C::kTu / 2; ++a) {
      const int col = t.n * C::kBu + Product::column(wu, a);
      float o[8];
      prod.eight(o, a, v);
      if (m < t.end && col < p.H) store8(p.grad_x + (size_t)m * p.H + col, o);
    }
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// u: columns along u in all, cols of them a tile
template <class C, auto KERNEL, int LDS, class Params>
hipError_t launch_product(const Params& p, int u, int cols, hipStream_t st) {
  const int ntiles = (u + cols - 1) / cols;
  const int64_t grid = tile_bound(p.seg, C::kBv, ntiles);
  if (!launchable(grid, C::kThreads)) return hipErrorNotSupported;
  const hipError_t e = allow_lds<KERNEL, LDS>();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(KERNEL, dim3((unsigned)grid), dim3(C::kThreads), LDS, st, p, ntiles);
  return hipGetLastError();
}

template <class C>
struct SlopeKernel {
  static constexpr auto kKernel = ffn_slope_kernel<C>;
};
template <class C>
struct RowGradKernel {
  static constexpr auto kKernel = ffn_grad_x_kernel<C>;
};

// A product with transposed weights, of u columns.  The shortest tiles while longer
// ones would leave half the compute units idle: what a tile's rows take behind its
// products counts as well (602 rows of 6 experts, 640 x 384: slopes 22 us on 12 tiles
// of 128 rows, 14 on twice as many; the rows' gradient 10 against 8).
template <template <class> class Kernel, class Params>
hipError_t launch_transposed(const Params& p, int u, hipStream_t st) {
  const auto launch = [&](auto config) {
    using C = decltype(config);
    constexpr int kLds = Fp8Product<C, kStages<C>, true>::kLds;
    return launch_product<C, Kernel<C>::kKernel, kLds>(p, u, C::kBu, st);
  };
  if (large_codes(p.seg, u)) return launch(Codes{});
  if (tiles_of(p.seg, u, ShortCodes::kBu, ShortCodes::kBv) <= kUnits / 2)
    return launch(FlatCodes{});
  return launch(ShortCodes{});
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

// Pieces of a workspace one after the other.
struct Carver {
  char* at;
  template <class T>
  T* take(size_t n) {
    T* p = reinterpret_cast<T*>(at);
    at += round_up(n * sizeof(T));
    return p;
  }
};

// Products of up to u columns can be launched at all (the smallest tile has 128 x
// 128 of them).
bool launchable_columns(const Segments& s, int u) {
  return launchable(tile_bound(s, 128, (u + 127) / 128), 512);
}

}  // namespace

namespace {

// Tiles of u columns by C's rows, the rows evenly spread.
template <class C>
int64_t even_tiles(int pairs, int E, int u, int cols) {
  const int busy = E < pairs ? E : pairs, rows = (pairs + busy - 1) / busy;
  return (int64_t)busy * ((rows + C::kBv - 1) / C::kBv) * (u / cols);
}

// In how many shares a projection's sums are made (0: whole, in the larger tiles).
// Below 16 steps a tile is short beside the launches (8 tokens of 4 experts, 1024 x
// 512: 17 us whole, 25 in shares).  Up to one 128 x 128 tile for a compute unit the
// shares give each unit one block (one expert of 2048 x 7168 whole and in shares, call
// by call: one token 46 against 26 us, 64 tokens 54 against 32, 512 tokens 76 against
// 46; twice the blocks 31, 41 and 69), and with a few rows an expert such tiles read
// the weights faster than the larger ones (one token of 8 of 32 experts, up projections
// 53 us against 41 + 5).  Up to 4 rows an expert that is one share of more tiles than
// units, about as fast as whole tiles (the block of 7168 x 2048, top-8 of 32 experts: 4
// tokens 171 us against 182, 16 tokens 242 against 239; of 256: 16 tokens 726 against 740,
// 128 tokens 1.82 ms against 1.79).  There is no second reason for one share of a down projection,
// whose tiles are as small, nor of the up projections where tiles of 256 x 64 are as
// many (1021 tokens of one expert 74 us against 69, 600 tokens 63 against 60; but one
// token of 8 experts, which makes half as many, 68 against 80).
struct Shares {
  int up, down;
};
Shares shares_of(int pairs, int E, int H, int I) {
  const auto shares = [&](int P, int K) {
    const int64_t tiles = even_tiles<NarrowCodes>(pairs, E, P, NarrowCodes::kBu);
    const int steps = K / kFp8Block;
    if (steps < 16 || (tiles > kUnits && pairs / E > 4)) return 0;
    const int64_t want = kUnits / tiles, most = steps / 2;
    return (int)(want < 1 ? 1 : want < most ? want : most);
  };
  const int up = shares(2 * I, H), down = shares(H, I);
  const int64_t flat = even_tiles<FlatCodes>(pairs, E, I, kFp8Block);
  const bool whole = up == 1 && flat > kUnits / 2 && flat <= kUnits;
  return {whole ? 0 : up, down > 1 ? down : 0};
}

size_t parts_bytes(size_t pairs, Shares s, int H, int I) {
  const size_t up = (size_t)s.up * 2 * I, down = (size_t)s.down * H;
  return round_up(pairs * (up > down ? up : down) * 4);
}

hipError_t launch_split(const SplitParams& p, int shares, hipStream_t st) {
  using C = NarrowCodes;
  constexpr int kLds = Fp8Product<C, kStages<C>>::kLds;
  const hipError_t e = allow_lds<ffn_split_kernel<C>, kLds>();
  if (e != hipSuccess) return e;
  const int ntiles = p.P / C::kBu;
  hipLaunchKernelGGL((ffn_split_kernel<C>),
                     dim3((unsigned)tile_bound(p.seg, C::kBv, ntiles), shares), dim3(C::kThreads),
                     kLds, st, p, ntiles);
  return hipGetLastError();
}

// Blocks of a join: some 8 columns a thread once, if there are few rows.
dim3 join_grid(const Segments& seg, int columns) {
  const unsigned x = (unsigned)tile_bound(seg, kJoinRows, 1);
  const unsigned most = (unsigned)(kJoinRows * columns / 8 + kJoinThreads - 1) / kJoinThreads;
  return dim3(x, most < 16 ? most : 16);
}

}  // namespace

size_t expert_ffn_workspace(int rows, int pairs, int E, int H, int I) {
  if (pairs == 0) return 0;
  const size_t n = rows;
  return round_up(n * I) + round_up(n * (I / kFp8Block) * 4) +
         parts_bytes(pairs, shares_of(pairs, E, H, I), H, I);
}

hipError_t launch_expert_ffn(const FfnParams& p, hipStream_t st) {
  const Segments& seg = p.seg;
  if (!launchable_columns(seg, 2 * p.I) || !launchable_columns(seg, p.H))
    return hipErrorNotSupported;
  const Shares shares = shares_of(seg.pairs, seg.E, p.H, p.I);
  const size_t n = seg.rows;
  Carver ws{static_cast<char*>(p.workspace)};
  uint8_t* h = ws.take<uint8_t>(n * p.I);
  float* h_scales = ws.take<float>(n * (p.I / kFp8Block));
  float* parts = reinterpret_cast<float*>(ws.at);
  const UpParams up{seg, p.x, p.x_scales, p.up, p.up_scales, p.pre, h, h_scales, p.H, p.I};
  hipError_t e;
  if (shares.up > 0) {
    const SplitParams split{seg, p.x, p.x_scales, p.up, p.up_scales, parts, p.H, 2 * p.I};
    e = launch_split(split, shares.up, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(ffn_join_up_kernel, join_grid(seg, p.I), dim3(kJoinThreads), 0, st, up,
                       parts, shares.up);
    e = hipGetLastError();
  } else if (even_tiles<FlatCodes>(seg.pairs, seg.E, p.I, kFp8Block) <= kUnits) {
    e = launch_product<FlatCodes, ffn_up_kernel<FlatCodes>, kUpLds<FlatCodes>>(up, p.I, 128, st);
  } else if (large_codes(seg, 2 * p.I)) {
    e = launch_product<Codes, ffn_up_kernel<Codes>, kUpLds<Codes>>(up, p.I, 128, st);
  } else {
    e = launch_product<ShortCodes, ffn_up_kernel<ShortCodes>, kUpLds<ShortCodes>>(up, p.I, 128, st);
  }
  if (e != hipSuccess) return e;
  if (shares.down > 0) {
    const SplitParams split{seg, h, h_scales, p.down, p.down_scales, parts, p.I, p.H};
    e = launch_split(split, shares.down, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(ffn_join_down_kernel, join_grid(seg, p.H), dim3(kJoinThreads), 0, st, seg,
                       parts, shares.down, p.residual, p.y, p.H);
    return hipGetLastError();
  }
  MatmulParams down{};
  down.seg = seg;
  down.x = h;
  down.x_scales = h_scales;
  down.weight = p.down;
  down.weight_scales = p.down_scales;
  down.residual = p.residual;
  down.y = p.y;
  down.K = p.I;
  down.F = down.P = p.H;
  down.act = kActNone;
  return launch_expert_matmul(down, true, st);
}

size_t expert_ffn_grad_workspace(int rows, int H, int I) {
  const size_t n = rows, P = 2 * (size_t)I;
  return round_up(n * H) + round_up(n * (H / kFp8Block) * 4) + round_up(n * P) +
         round_up(n * (P / kFp8Block) * 4) + round_up(n * P * 2) + round_up(n * I * 2) +
         round_up(n * H * 2);
}

hipError_t launch_expert_ffn_grad(const FfnGradParams& p, hipStream_t st) {
  const Segments& seg = p.seg;
  const int P = 2 * p.I, hb = p.H / kFp8Block, pb = P / kFp8Block;
  if (!launchable_columns(seg, p.I) || !launchable_columns(seg, p.H) ||
      (int64_t)seg.E * hb * pb > INT32_MAX ||
      !launchable(tile_bound(seg, kPrepareRows, 1), kPrepareThreads))
    return hipErrorNotSupported;
  const size_t n = seg.rows;
  Carver ws{static_cast<char*>(p.workspace)};
  uint8_t* gy = ws.take<uint8_t>(n * p.H);
  float* gy_scales = ws.take<float>(n * hb);
  uint8_t* gz = ws.take<uint8_t>(n * P);
  float* gz_scales = ws.take<float>(n * pb);
  uint16_t* wide_gz = ws.take<uint16_t>(n * P);
  uint16_t* h = ws.take<uint16_t>(n * p.I);
  uint16_t* wide_x = ws.take<uint16_t>(n * p.H);
  hipError_t e = hipSuccess;
  if (seg.pairs > 0 && !p.grad_x && !p.grad_up) {
    hipLaunchKernelGGL(ffn_hidden_kernel, dim3((unsigned)tile_bound(seg, kPrepareRows, 1)),
                       dim3(kPrepareThreads), 0, st, seg, p.pre, h, p.I);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else if (seg.pairs > 0) {
    const PrepareParams prepare{seg,  p.grad_y, gy, gy_scales, p.x, p.x_scales,
                                p.grad_up ? wide_x : nullptr, p.H};
    hipLaunchKernelGGL(ffn_prepare_kernel, dim3((unsigned)tile_bound(seg, kPrepareRows, 1)),
                       dim3(kPrepareThreads), 0, st, prepare);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const SlopeParams slope{seg,   gy,
                            gy_scales, p.down,
                            p.down_scales, p.pre,
                            p.grad_x ? gz : nullptr, gz_scales,
                            p.grad_up ? wide_gz : nullptr, p.grad_down ? h : nullptr,
                            p.H,   p.I};
    e = launch_transposed<SlopeKernel>(slope, p.I, st);
    if (e != hipSuccess) return e;
    if (p.grad_x) {
      const RowGradParams row{seg, gz, gz_scales, p.up, p.up_scales, p.grad_x, p.H, p.I};
      e = launch_transposed<RowGradKernel>(row, p.H, st);
      if (e != hipSuccess) return e;
    }
  }
  MatmulGradParams w{};
  w.seg = seg;
  w.act = kActNone;
  if (p.grad_up) {
    w.grad_y = wide_gz;
    w.x = wide_x;
    w.grad_weight = p.grad_up;
    w.K = p.H;
    w.F = w.P = P;
    if ((e = launch_expert_matmul_grad(w, st)) != hipSuccess) return e;
  }
  if (p.grad_down) {
    w.grad_y = p.grad_y;
    w.x = h;
    w.grad_weight = p.grad_down;
    w.K = p.I;
    w.F = w.P = p.H;
    e = launch_expert_matmul_grad(w, st);
  }
  return e;
}

}  // namespace moe
