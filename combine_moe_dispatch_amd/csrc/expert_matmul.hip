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
#include <atomic>
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

//
// Four waves: with one wave to a SIMD each holds 128 x 128 of a 256 x 256 tile
// and reads a quarter less from LDS per product than eight waves of 128 x 64
// (prefill of 4096 tokens 1.62 against 1.73 ms; in two teams of four that
// read and multiply in turns 1.80 ms, with 32 x 32 x 16 products 1.84 ms).
// The matrix units draw the chip's power, so what counts is less work around
// them rather than fewer idle cycles: the clock falls as those go.
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

  // A tile whose last quarters have no rows (only where B's rows run along r)
  // leaves out their products and B's loads of them: PART is how many of the
  // fragments along v a wave has to do, in quarters of kTv.
  template <int PART>
  static constexpr int kPartLoads = A::kLoads + B::kLoads * PART / C::kTv;

  // Fragment i (of PART + kTu) of part k of the step at lds.
  template <int PART, bool TAIL>
  __device__ __forceinline__ void read(Fragments& f, int i, uint32_t lds, int k, int left) const {
    if (i < PART)
      f.b[i] = rb.template frag<TAIL>(lds + A::kBytes, i * (BT ? 1 : C::kWv), k, left);
    else
      f.a[i - PART] = ra.template frag<TAIL>(lds, i - PART, k, left);
  }
  template <int PART, bool TAIL>
  __device__ __forceinline__ void read_all(Fragments& f, uint32_t lds, int k, int left) const {
#pragma unroll
    for (int i = 0; i < PART + C::kTu; ++i) read<PART, TAIL>(f, i, lds, k, left);
  }

  // acc += f, row of fragments by row, with before(u) in front of row u: what
  // it issues runs beside the products.
  template <int PART, class Before>
  __device__ __forceinline__ void multiply(const Fragments& f, Before before) {
#pragma unroll
    for (int u = 0; u < C::kTu; ++u) {
      before(u);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int v = 0; v < PART; ++v) mfma_in_place(acc[u][v], f.a[u], f.b[v]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int u = 0; u < C::kTu; ++u)
#pragma unroll
      for (int v = 0; v < C::kTv; ++v) acc[u][v] = f32x4_t{};
  }

  // A tile's operands: ap[i] is where load i of this wave starts in A (weight
  // rows of a gated layer lie in two places), bp in B; lda, ldb are the
  // operands' row pitches in bytes, red > 0 the positions along r.
  const char* ap[A::kLoads];
  const char* bp;
  uint32_t lda, ldb;
  int red, wave;
  uint32_t lds;

  __device__ __forceinline__ void setup(char* smem, int wave_) {
    wave = wave_;
    lds = lds_address(smem);
    ra.init(wave % C::kWu * C::kTu * 16);
    rb.init(wave / C::kWu * 16, C::kWv);
  }
  __device__ __forceinline__ int steps() const { return (red + kStep - 1) / kStep; }
  // The next step's load i, and all of them.
  template <bool TAIL>
  __device__ __forceinline__ void load(int i, uint32_t to) {
    const int rest = red % kStep;
    if (i < A::kLoads)
      a.template load<TAIL>(i, to, wave, ap[i], lda, rest);
    else if (i < kLoads)
      b.template load<TAIL>(i - A::kLoads, to + A::kBytes, wave, bp, ldb, rest);
  }
  __device__ __forceinline__ void advance() {
#pragma unroll
    for (int i = 0; i < A::kLoads; ++i) ap[i] += AT ? (size_t)kStep * lda : (size_t)kStep * 2;
    bp += BT ? (size_t)kStep * ldb : (size_t)kStep * 2;
  }
  template <int PART>
  __device__ __forceinline__ void start(uint32_t to, bool full) {
    if (full) {
#pragma unroll
      for (int i = 0; i < kPartLoads<PART>; ++i) load<false>(i, to);
    } else {
#pragma unroll
      for (int i = 0; i < kPartLoads<PART>; ++i) load<true>(i, to);
    }
    advance();
  }
  // Start the first two steps of a tile.  No wave may still read LDS.
  template <int PART>
  __device__ __forceinline__ void begin() {
    const int whole = red / kStep;
    start<PART>(lds, whole > 0);
    if (steps() > 1) start<PART>(lds + kStage, whole > 1);
  }

  // The tile that begin() has started.  Afterwards LDS is free again.  behind:
  // stores that this wave has started since (0, or kStores at least).
  template <int PART>
  __device__ __forceinline__ void run(int behind) {
    constexpr int kLoads = kPartLoads<PART>;
    constexpr int kBehind = C::kTv * C::kTu / 2;
    static_assert(kLoads + kBehind < 64, "counted by the hardware");
    static_assert(kParts == 2, "the parts are written out");
    clear();
    uint32_t here = lds, next = lds + kStage;
    const int steps = this->steps(), whole = red / kStep;
    const int rest = red - (steps - 1) * kStep;  // positions of the last step
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
    constexpr int kReads = (2 * (C::kTu + PART) + C::kTu - 1) / C::kTu;  // in the first rows
    constexpr int kStarts = (kLoads + C::kTu - 1) / C::kTu;
    auto reading = [&](Fragments& f, uint32_t lds, int k, int u) {
#pragma unroll
      for (int i = u * kReads; i < (u + 1) * kReads; ++i)
        if (i < C::kTu + PART) read<PART, false>(f, i, lds, k, rest);
    };
    const auto nothing = [](int) {};
    Fragments f0, f1;
    if (steps > 1 && behind > 0)
      wait_vm<kLoads + kBehind>();
    else if (steps > 1)
      wait_vm<kLoads>();
    else
      wait_vm<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (steps > 1)
      read_all<PART, false>(f0, here, 0, rest);
    else
      read_all<PART, true>(f0, here, 0, rest);
    // Half a step is multiplied while the next half is read, the second half
    // behind the barrier, so that the matrix units have work on both sides.
    for (int t = 0; t + 2 < whole; ++t) {
      multiply<PART>(f0, [&](int u) { reading(f1, here, 1, u); });
      meet();
      multiply<PART>(f1, [&](int u) {
        reading(f0, next, 0, u);
#pragma unroll
        for (int i = u * kStarts; i < (u + 1) * kStarts; ++i)
          if (i < kLoads) load<false>(i, here);
      });
      advance();
      turn();
    }
    if (whole < steps && steps > 2) {  // the step whose loads are the short ones
      multiply<PART>(f0, [&](int u) { reading(f1, here, 1, u); });
      meet();
      start<PART>(here, false);
      multiply<PART>(f1, [&](int u) { reading(f0, next, 0, u); });
      turn();
    }
    if (steps > 1) {
      multiply<PART>(f0, [&](int u) { reading(f1, here, 1, u); });
      meet();
      multiply<PART>(f1, nothing);
      read_all<PART, true>(f0, next, 0, rest);
      turn();
    }
    // the second half of the last step may have no positions (a weight gradient
    // over 256 rows an expert 3% less)
    if (rest > kPart) read_all<PART, true>(f1, here, 1, rest);
    multiply<PART>(f0, nothing);
    wait_lds();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (rest > kPart) multiply<PART>(f1, nothing);
    mfma_results();
#pragma unroll
    for (int u = 0; u < C::kTu; ++u)
#pragma unroll
      for (int v = 0; v < C::kTv; ++v) mfma_result(acc[u][v]);
  }

  // A tile of `rows` along v, from its first load on.
  template <int PART>
  __device__ __forceinline__ void begin_and_run() {
    static_assert(!BT, "the front of a transposed operand's tile is not its first columns");
    begin<PART>();
    run<PART>(0);
  }
  __device__ __forceinline__ void begin_and_run(int rows) {
    if (rows > C::kBv * 3 / 4)
      begin_and_run<C::kTv>();
    else if (rows > C::kBv / 2)
      begin_and_run<C::kTv * 3 / 4>();
    else if (rows > C::kBv / 4)
      begin_and_run<C::kTv / 2>();
    else
      begin_and_run<C::kTv / 4>();
  }

  // This lane's outputs of fragments 2a and 2a + 1 by v: eight neighbours
  // along u from a * 32 + (lane >> 4) * 8 on, of the fragment's row lane & 15.
  __device__ __forceinline__ void eight(float (&o)[8], int a, int v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = acc[2 * a + i / 4][v][i % 4];
  }
};

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
// The same for e4m3 operands with a scale per 128 values along r: one step is
// one block of 128, whose products are summed by one 16 x 16 x 128 matrix
// instruction per fragment and then scaled in fp32, sx of the token times sw
// of the 128 weight rows.  A row of a step is 128 bytes, as in the bf16
// product, so the tiles in LDS are the same; the chunks of a fragment are
// taken in an order of their own, equal for both operands, which a sum does
// not notice.  Eight waves, two on every SIMD: one scales while the other
// multiplies.
//
// The instruction's own sum has fewer bits than fp32: of 8 neighbouring columns
// it cuts every product below 2^-13 of the largest (measured; the 16 x 16 x 32
// instruction does the same), so a sum is off by less than 2^-10 of the groups'
// largest products (2.5 2^-13 at most in 10^5 sums of random codes, 2^-19 of the
// magnitudes in the mean of normal ones).  Both factors of a product were
// rounded to 2^-4 before, and exact sums would need the codes widened to bf16, at
// half the rate.
// ---------------------------------------------------------------------------
template <class C, int STAGES>
struct Fp8Product {
  using A = OperandTile<C::kBu, C::kWaves, false, true>;
  using B = OperandTile<C::kBv, C::kWaves, false, false>;
  static constexpr int kScales = C::kWaves * 256;  // one dword a lane
  static_assert(C::kBv == C::kWaves * 32, "a wave brings in the scales of 32 rows");
  static constexpr int kStage = A::kBytes + B::kBytes + kScales;
  static constexpr int kLds = STAGES * kStage;
  static constexpr int kRows = 4;  // of fragments multiplied at a time
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

  // PART: as in TileProduct.  blocks > 0 steps.  scale: the scale this lane brings in, of step 0: lanes
  // 0-31 one of the wave's 32 x rows, lanes 32 and 33 those of the weight rows
  // behind the first and the second half of the wave's fragments.  (A plain
  // load of them would wait for every load to LDS before it.)  rows: how many
  // the tile has.
  template <int PART>
  __device__ __forceinline__ void run(char* smem, int wave, const char* (&ap)[A::kLoads],
                                      const char* bp, const float* scale, int blocks, int rows) {
    constexpr int kRowLoads = B::kLoads * PART / C::kTv;
    constexpr int kLoads = A::kLoads + kRowLoads + 1;
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
      for (int i = 0; i < kRowLoads; ++i)
        b.template load<false>(i, fill + A::kBytes, wave, bp, 0, 0);
      load4_to_lds(fill + A::kBytes + B::kBytes + wave * 256, scale);
      bp += 128;
      scale += 1;
      fill = after(fill);
    };
    for (int t = 0; t < STAGES - 1 && t < blocks; ++t) start();
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
      if (t + STAGES - 1 <= blocks)
        wait_vm<(STAGES - 2) * kLoads>();
      else
        wait_vm<0>();
      wait_lds();  // this wave has read the step before out
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (t + STAGES - 1 < blocks) start();
      if (nv > 0) {
        const float sw[2] = {lds_float(here + sw_at), lds_float(here + sw_at + 4)};
#pragma unroll
        for (int u0 = 0; u0 < C::kTu; u0 += kRows) {
          i32x8_t fa[kRows];
#pragma unroll
          for (int u = 0; u < kRows; ++u) fa[u] = frag(ra, here, u0 + u);
#pragma unroll
          for (int v = 0; v < PART; ++v) {
            if (v >= nv) break;
            const i32x8_t fb = frag(rb, here + A::kBytes, v * C::kWv);
            const float sx = lds_float(here + sx_at + v * C::kWv / 2 * 256);
            f32x4_t part[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u)
              part[u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[u], fb, f32x4_t{}, 0,
                                                                         0, 0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
              const float s = sx * sw[u0 + u < C::kTu / 2 ? 0 : 1];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[u0 + u][v][i] = fmaf(part[u][i], s, acc[u0 + u][v][i]);
            }
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
// at once; the splits' sums are added by a second launch.  8192 rows of 4096:
// 168 MB in 40 us at best, 4.2 TB/s, 60 on average among other kernels.
//
// gz is bf16 because the matrix units take no more in one pass: the rest of it
// as a second operand would double both products.  Against fp64 the gradients are
// off by 2.3e-3 of their size, 1.7e-3 with the outputs' rounding alone.
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
    const int q = A::load_of(i, wave);
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
  const char* bp = static_cast<const char*>(p.x) + (size_t)t.m0 * ld;
  if (rows > C::kBv * 3 / 4)
    prod.template run<C::kTv>(smem, wave, ap, bp, scale, kb, rows);
  else if (rows > C::kBv / 2)
    prod.template run<C::kTv * 3 / 4>(smem, wave, ap, bp, scale, kb, rows);
  else if (rows > C::kBv / 4)
    prod.template run<C::kTv / 2>(smem, wave, ap, bp, scale, kb, rows);
  else
    prod.template run<C::kTv / 4>(smem, wave, ap, bp, scale, kb, rows);
  finish<C, ACT>(prod, p, t, wave);
}

// The accumulators as bf16 rows: row v of the tile to out + v * ld, for v
// below rows, columns below cols.  A whole tile takes kStores stores a lane.
template <class C>
constexpr int kStores = C::kTv * C::kTu / 2;

template <class C, bool WHOLE, class Product>
__device__ __forceinline__ void store_tile(const Product& prod, int wave, uint16_t* out, size_t ld,
                                           int rows, int cols) {
  const int wu = wave % C::kWu, wv = wave / C::kWu, lane = lane_id();
#pragma unroll
  for (int v = 0; v < C::kTv; ++v) {
    const int m = (v * C::kWv + wv) * 16 + (lane & 15);
    if (!WHOLE && m >= rows) continue;
#pragma unroll
    for (int a = 0; a < C::kTu / 2; ++a) {
      const int c = (wu * C::kTu + 2 * a) * 16 + (lane >> 4) * 8;
      float o[8];
      prod.eight(o, a, v);
      if (WHOLE || c < cols) store8(out + (size_t)m * ld + c, o);
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
// fp8, 256 token rows by 256 weight rows in two steps of LDS or by 128 in
// three: the large tile moves less per product (32 experts of 4096 x 7168: 512
// rows each 444 us against 527, 128 rows 236 against 284), the small one has
// twice the blocks and the deeper ring for few rows (64 rows 201 against 195).
using Codes = Config<2, 4, 8, 4>;
using FewCodes = Config<2, 4, 4, 4>;

constexpr int kUnits = 256;  // compute units

int64_t tiles_of(const Segments& s, int u, int bu, int bv) {
  const int64_t rows = s.pairs / s.E, busy = s.E < s.pairs ? s.E : s.pairs;
  return busy * ((rows + bv - 1) / bv) * ((u + bu - 1) / bu);
}

// Large tiles from 112 rows an expert on, where some experts begin to need two
// small ones (32 experts, 4096 x 7168: 96 rows 394 us against 357 on small
// tiles, 128 rows 435 against 501, 256 rows 637 against 668, 512 rows 905
// against 1024), if they give three quarters of the compute units one (one
// expert, 7168 x 2048: 112 tiles 59 us against 36, 168 tiles 61 against 59, 196
// tiles 63 against 66).
bool large_tiles(const Segments& s, int u) {
  return s.pairs / s.E >= 112 && tiles_of(s, u, Large::kBu, Large::kBv) >= kUnits * 3 / 4;
}

// The large fp8 tile where an expert has more than a quarter of its rows on
// average and every compute unit gets one.
bool large_codes(const Segments& s, int u) {
  return s.pairs / s.E > Codes::kBv / 4 && tiles_of(s, u, Codes::kBu, Codes::kBv) >= kUnits;
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

// A launch has less than 2^32 threads.
bool launchable(int64_t blocks, int threads) { return blocks < (int64_t(1) << 32) / threads; }

// More than 64 KB of LDS has to be asked for, once per kernel and device.
template <auto KERNEL, int BYTES>
hipError_t allow_lds() {
  static std::atomic<uint64_t> done{0};
  int device;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (device & 63);
  if (device < 64 && (done.load(std::memory_order_relaxed) & bit)) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL),
                          hipFuncAttributeMaxDynamicSharedMemorySize, BYTES);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
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
