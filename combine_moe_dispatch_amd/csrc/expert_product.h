// expert_product.h -- the tiled matrix products of the experts' rows: a block
// holds a tile of D[u][v] = sum over r of A[u][r] B[v][r] in registers, in bf16
// or in e4m3 with block scales, and what their kernels and launches share.
#pragma once

#include <atomic>
#include <type_traits>

#include "expert_tile.h"

namespace moe {

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
// Half of an e4m3 operand held transposed: one step is 128 rows along r of SIZE
// columns, [128][SIZE] bytes in LDS, read back through the transposing 8-byte load:
// of 16 lanes, lane j names 8 bytes of row j / 2 (columns 0-7 or 8-15) and receives
// column j of the 8 rows.  As in OperandTile the layout is linear in the lanes and
// chunk c of row i sits in slot c ^ f(i): the 16 rows that half a wave reads from
// (two runs of 8, 16 apart) take 16 different places of the 256 bytes of banks.
// A lane receives its 32 positions in the order of the other operand's chunks,
// 16 (l >> 4) .. + 15 and 64 behind.
// ---------------------------------------------------------------------------
template <int SIZE, int WAVES>
struct TransposedCodes {
  static constexpr int kBytes = SIZE * 128;
  static constexpr int kLoads = kBytes / 1024 / WAVES;
  static_assert(kLoads * WAVES * 1024 == kBytes, "whole wave loads");
  static_assert(SIZE == 128, "the swizzle is that of rows of 128 bytes");
  static constexpr int kSlots = SIZE / 16;
  static constexpr int kRowsPerLoad = 64 / kSlots;
  uint32_t off[kLoads];

  static __device__ __forceinline__ int swizzle(int row) {
    return ((row >> 1) & 3) | ((row >> 4) & 1) << 2;
  }
  static __device__ __forceinline__ int load_of(int i, int wave) { return i * WAVES + wave; }
  // The chunk that this lane brings in with load q, and its row.
  static __device__ __forceinline__ void chunk_of(int q, int& row, int& c) {
    const int lane = lane_id();
    row = q * kRowsPerLoad + lane / kSlots;
    c = (lane % kSlots) ^ swizzle(row);
  }
  template <bool TAIL>
  __device__ __forceinline__ void load(int i, uint32_t lds, int wave, const char* base, uint32_t,
                                       int) const {
    load_to_lds(lds + (uint32_t)load_of(i, wave) * 1024, base, off[i]);
  }

  template <int N>
  struct Reader {
    static constexpr int kAts = N;
    uint32_t at[N];
    __device__ __forceinline__ void init(int i0) {
      const int lane = lane_id(), j = lane & 15, row = (lane >> 4) * 16 + (j >> 1);
#pragma unroll
      for (int n = 0; n < N; ++n)
        at[n] = (uint32_t)(row * SIZE + ((i0 / 16 + n) ^ swizzle(row)) * 16 + (j & 1) * 8);
    }
  };
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
//
// AT: A is held transposed, its rows along r.  Its fragments are not paired, so
// that a lane's eight neighbours come from an exchange between the lanes behind
// the last product.  ACROSS: the waves' first fragments are the tile's first
// half, which is read in whole lines (rows' gradient of 2048 tokens 558 us against
// 610); otherwise a wave has neighbouring columns.
// ---------------------------------------------------------------------------
template <class C, int STAGES, bool AT = false, bool ACROSS = false>
struct Fp8Product {
  // A lies in two halves: of every wave's fragments the first ones, then the others.
  using Half = std::conditional_t<AT, TransposedCodes<C::kBu / 2, C::kWaves>,
                                  OperandTile<C::kBu / 2, C::kWaves, false, true>>;
  using B = OperandTile<C::kBv, C::kWaves, false, false>;
  static constexpr int kHalf = C::kTu / 2, kHalfRows = kHalf * 16;  // of a wave
  static constexpr int kScales = C::kWaves * 256;  // one dword a lane
  static_assert(C::kBv <= C::kWaves * 32, "a wave brings in the scales of 32 rows");
  static constexpr int kStage = 2 * Half::kBytes + B::kBytes + kScales;
  static constexpr int kLds = STAGES * kStage;
  Half a[2];
  B b;
  f32x4_t acc[C::kTu][C::kTv];
  typename Half::template Reader<kHalf> ra;
  typename B::template Reader<C::kTv> rb;
  const char* ap[2];  // the halves' first step,
  size_t a_step;      // the bytes to the next one (AT),
  int scale_step;     // and the entries between this lane's scales (AT)

  // Position along u of place i of a half, in the tile.
  static __device__ __forceinline__ int place(int half, int i) {
    if (ACROSS) return half * (C::kBu / 2) + i;
    return i / kHalfRows * (2 * kHalfRows) + half * kHalfRows + i % kHalfRows;
  }
  // Weight rows w, w + ld, .. of which cols are left; GATED: the first halves are
  // gate rows, the second ones the up rows of the same columns, up bytes on.
  template <bool GATED>
  __device__ __forceinline__ void weight_rows(int wave, const char* w, uint32_t ld, int cols,
                                              size_t up) {
    static_assert(!AT, "rows along r");
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < Half::kLoads; ++i) {
        int row, c;
        Half::chunk_of(Half::load_of(i, wave), row, c);
        const int col = GATED ? row : place(half, row);
        a[half].off[i] = (uint32_t)min(col, cols - 1) * ld + (uint32_t)c * 16;
        a[half].where[i] = 0;
      }
      ap[half] = w + (GATED && half == 1 ? up : 0);
    }
  }
  // Weight columns w, w + 1, .. of which cols are left (a multiple of 16).
  __device__ __forceinline__ void weight_columns(int wave, const char* w, uint32_t ld, int cols) {
    static_assert(AT, "rows along u");
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < Half::kLoads; ++i) {
        int row, c;
        Half::chunk_of(Half::load_of(i, wave), row, c);
        a[half].off[i] = (uint32_t)row * ld + (uint32_t)min(place(half, c * 16), cols - 16);
      }
      ap[half] = w;
    }
    a_step = (size_t)kFp8Block * ld;
  }

  // Where a step's fragments are read from: a reader's addresses in its place in LDS,
  // made once a step, so that the rest is in the instructions' offsets (the compiler
  // would add them up anew for every read: 928 us against 871 for 4096 tokens' up
  // projections).
  template <class R>
  struct Places {
    uint32_t at[R::kAts];
    __device__ __forceinline__ void set(const R& r, uint32_t lds) {
#pragma unroll
      for (int k = 0; k < R::kAts; ++k) {
        at[k] = r.at[k] + lds;
        asm volatile("" : "+v"(at[k]));
      }
    }
  };
  using ReaderA = typename Half::template Reader<kHalf>;
  using ReaderB = typename B::template Reader<C::kTv>;
  template <class T>
  static __device__ __forceinline__ T lds_read(uint32_t p) {
    return *(const __attribute__((address_space(3))) T*)(uintptr_t)p;
  }
  // Fragment v of B, and u of A.
  static __device__ __forceinline__ i32x8_t frag_b(const Places<ReaderB>& p, int v) {
    union {
      bf16x8_t h[2];
      i32x8_t v;
    } f;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      f.h[k] = lds_read<bf16x8_t>(p.at[k] + v * C::kWv * 16 * kFp8Block);
    return f.v;
  }
  static __device__ __forceinline__ i32x8_t frag_a(const Places<ReaderA>& p, int u) {
    const int half = u / kHalf * Half::kBytes, n = u % kHalf;
    union {
      i32x2_t q[4];
      bf16x8_t h[2];
      i32x8_t v;
    } f;
    if constexpr (AT) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        f.q[q] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2_t*)(uintptr_t)(
                p.at[n] + half + (q / 2 * 64 + q % 2 * 8) * (C::kBu / 2)));
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        f.h[k] = lds_read<bf16x8_t>(p.at[k] + half + (n / 2 * 32 + n % 2 * 4) * kFp8Block);
    }
    return f.v;
  }

  // PART: as in TileProduct.  blocks > 0 steps.  scale: the scale this lane brings
  // in, of step 0: lanes 0-31 one of the wave's 32 x rows, lanes 32 and 33 those of
  // the weight rows behind the first and the second half of the wave's fragments.
  // (A plain load of them would wait for every load to LDS before it.)  rows: how
  // many the tile has.
  //
  // A wave multiplies row after row of fragments while it reads the next one, and
  // scales each product behind the second one after it.  B's fragments stay in
  // registers for a step.  All waves meet twice a step: when A's first half, B and
  // the scales are in registers and their place can be filled again, and when the
  // second half is.
  // So a load has one and a half steps to arrive with two steps of LDS (with one
  // meeting a step, and one step to arrive, 4096 tokens' up projections took 955
  // us, with two 918; without any wait for memory 850).
  template <int PART>
  __device__ __forceinline__ void run(char* smem, int wave, const char* bp, const float* scale,
                                      int blocks, int rows) {
    constexpr int kRowLoads = B::kLoads * PART / C::kTv;
    constexpr int kFirst = Half::kLoads + kRowLoads + 1;  // loads of a first half, B and scales
    constexpr int kSecond = Half::kLoads;
    constexpr int kLoads = kFirst + kSecond;
    static_assert((STAGES - 1) * kLoads + kSecond < 64, "counted by the hardware");
    constexpr uint32_t kSecondAt = Half::kBytes, kRowsAt = 2 * Half::kBytes,
                       kScalesAt = kRowsAt + B::kBytes;
    ra.init(wave % C::kWu * kHalfRows);
    rb.init(wave / C::kWu * 16);
#pragma unroll
    for (int u = 0; u < C::kTu; ++u)
#pragma unroll
      for (int v = 0; v < C::kTv; ++v) acc[u][v] = f32x4_t{};
    const uint32_t lds = lds_address(smem), lds_end = lds + kLds;
    uint32_t here = lds;
    auto after = [&](uint32_t slot) { return slot + kStage == lds_end ? lds : slot + kStage; };
    auto load_first = [&](int i, uint32_t slot) {
      if (i < Half::kLoads) {
        a[0].template load<false>(i, slot, wave, ap[0], 0, 0);
      } else if (i + 1 < kFirst) {
        b.template load<false>(i - Half::kLoads, slot + kRowsAt, wave, bp, 0, 0);
      } else {
        load4_to_lds(slot + kScalesAt + wave * 256, scale);
        ap[0] += AT ? a_step : 128;
        bp += 128;
        scale += AT ? scale_step : 1;
      }
    };
    auto start_first = [&](uint32_t slot) {
#pragma unroll
      for (int i = 0; i < kFirst; ++i) load_first(i, slot);
    };
    auto start_second = [&](uint32_t slot) {
#pragma unroll
      for (int i = 0; i < kSecond; ++i)
        a[1].template load<false>(i, slot + kSecondAt, wave, ap[1], 0, 0);
      ap[1] += AT ? a_step : 128;
    };
    for (int t = 0; t < STAGES && t < blocks; ++t) {
      start_first(here);
      start_second(here);
      here = after(here);
    }
    here = lds;
    if (blocks >= STAGES)
      wait_vm<(STAGES - 1) * kLoads + kSecond>();
    else
      wait_vm<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // All waves have read the first half, B and the scales of step t out, and its
    // second half has come.
    auto meet_first = [&](int t) {
      wait_lds();
      if (t + STAGES <= blocks)
        wait_vm<(STAGES - 1) * kLoads>();
      else
        wait_vm<0>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    // They have read its second half out, and what step t + 1 begins with has come.
    auto meet_second = [&](int t) {
      wait_lds();
      if (t + STAGES < blocks)
        wait_vm<(STAGES - 1) * kLoads>();
      else if (t + STAGES == blocks)
        wait_vm<(STAGES - 2) * kLoads + kSecond>();
      else
        wait_vm<0>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    // the fragments of this wave that hold rows at all
    const int wv = wave / C::kWu;
    if (rows <= wv * 16) {
      for (int t = 0; t < blocks; ++t) {
        meet_first(t);
        if (t + STAGES < blocks) start_first(here);
        if (t + 1 == blocks) break;
        meet_second(t);
        if (t + STAGES < blocks) start_second(here);
        here = after(here);
      }
      return;
    }
    // 32 rows of scales every 256 bytes, this wave's two behind its own 32
    const uint32_t sw_at = kScalesAt + wave * 256 + 128;
    const uint32_t sx_at = kScalesAt + wv / 2 * 256 + wv % 2 * 64 + (lane_id() & 15) * 4;
    static_assert(C::kWv % 2 == 0, "a fragment's scales lie 256 bytes per two fragments on");
    constexpr int kProducts = C::kTu * PART, kBehind = 2, kSlots = kBehind + 1;
    static_assert(kBehind <= (C::kTu - 1) * PART, "a step's scales before the next one's");
    // rows of A's fragments read ahead: one where a row is four products, else two
    constexpr int kAhead = PART <= 2 ? 2 : 1, kRows = 2 * kAhead;
    static_assert(C::kTu % kRows == 0 && kAhead <= kHalf, "the same places in every step");
    i32x8_t fa[kRows], fb[PART];
    float sx[PART], sw[2], s[2][PART];
    f32x4_t part[kSlots];
    Places<ReaderA> pa;
    Places<ReaderB> pb;
    uint32_t ps, pw;  // of the rows' scales, and the weight's
    auto set_places = [&] {
      pa.set(ra, here);
      pb.set(rb, here + kRowsAt);
      ps = here + sx_at;
      pw = here + sw_at;
      asm volatile("" : "+v"(ps));
    };
    auto read_a = [&](int u) { fa[u % kRows] = frag_a(pa, u); };
    auto read_b = [&](int v) {
      fb[v] = frag_b(pb, v);
      sx[v] = lds_read<float>(ps + v * C::kWv / 2 * 256);
    };
    auto read_w = [&] {
      sw[0] = lds_read<float>(pw);
      sw[1] = lds_read<float>(pw + 4);
    };
    set_places();
#pragma unroll
    for (int u = 0; u < kAhead; ++u) read_a(u);
#pragma unroll
    for (int v = 0; v < PART; ++v) read_b(v);
    read_w();
    // A first half's loads are started some with each row of products: all at once
    // they hold up the waves.
    constexpr int kSpread = kHalf < 3 ? kHalf : 3;  // all before the next meeting
    constexpr int kChunk = (kFirst + kSpread - 1) / kSpread;
    // LAST: no step follows.
    auto step = [&](int t, auto last) {
      constexpr bool kLast = decltype(last)::value;
      const bool more = !kLast && t + STAGES < blocks;
      const uint32_t slot = here;
#pragma unroll
      for (int i = 0; i < kProducts + kBehind; ++i) {
        const int u = i / PART, v = i % PART;
        const bool row = i < kProducts && v == 0;
        if (row) {
          if (u + kAhead == kHalf) meet_first(t);
          if (u + kAhead < C::kTu) {
            read_a(u + kAhead);
          } else if (!kLast) {
            if (u + kAhead == C::kTu) {
              meet_second(t);
              here = after(here);
              set_places();
            }
            read_a(u + kAhead - C::kTu);
          }
        }
        if (i < kProducts)
          part[i % kSlots] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              fa[u % kRows], fb[v], f32x4_t{}, 0, 0, 0, 0, 0, 0);
        if (row && more) {
          const int n = u + kAhead - kHalf;
          if (n >= 0 && n < kSpread) {
#pragma unroll
            for (int q = 0; q < kChunk; ++q)
              if (n * kChunk + q < kFirst) load_first(n * kChunk + q, slot);
          }
          if (u + kAhead == C::kTu) start_second(slot);
        }
        if (i >= kBehind) {
          const int j = i - kBehind, ju = j / PART, jv = j % PART;
          if (j == 0) {
#pragma unroll
            for (int n = 0; n < 2 * PART; ++n) s[n / PART][n % PART] = sx[n % PART] * sw[n / PART];
          }
          const float scale = s[ju / kHalf][jv];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc[ju][jv][k] = fmaf(part[j % kSlots][k], scale, acc[ju][jv][k]);
          // here and not behind a meeting, where the compiler would move it
          asm volatile("" : "+v"(acc[ju][jv]));
        }
        if (i < kProducts && u + 1 == C::kTu && !kLast) {
          read_b(v);
          if (v == 0) read_w();
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int t = 0; t + 1 < blocks; ++t) step(t, std::false_type{});
    step(blocks - 1, std::true_type{});
  }

  // A tile of `rows` rows: as many quarters (halves) of it as have some.
  __device__ __forceinline__ void run_rows(char* smem, int wave, const char* bp,
                                           const float* scale, int blocks, int rows) {
    if constexpr (C::kTv % 4 == 0) {
      if (rows > C::kBv * 3 / 4)
        run<C::kTv>(smem, wave, bp, scale, blocks, rows);
      else if (rows > C::kBv / 2)
        run<C::kTv * 3 / 4>(smem, wave, bp, scale, blocks, rows);
      else if (rows > C::kBv / 4)
        run<C::kTv / 2>(smem, wave, bp, scale, blocks, rows);
      else
        run<C::kTv / 4>(smem, wave, bp, scale, blocks, rows);
    } else if constexpr (C::kTv == 1) {
      run<1>(smem, wave, bp, scale, blocks, rows);
    } else {
      static_assert(C::kTv % 2 == 0 && B::kLoads % 2 == 0, "whole loads of half a tile");
      if (rows > C::kBv / 2)
        run<C::kTv>(smem, wave, bp, scale, blocks, rows);
      else
        run<C::kTv / 2>(smem, wave, bp, scale, blocks, rows);
    }
  }

  // AT, behind the last product: lanes 16-31 and 48-63 of a fragment for 0-15 and
  // 32-47 of its neighbour, which leaves every lane 8 neighbours along u.
  __device__ __forceinline__ void exchange() {
    static_assert(AT, "paired fragments need none");
#pragma unroll
    for (int v = 0; v < C::kTv; ++v)
#pragma unroll
      for (int a = 0; a < C::kTu / 2; ++a) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const auto r = __builtin_amdgcn_permlane16_swap(
              __float_as_uint(acc[2 * a][v][i]), __float_as_uint(acc[2 * a + 1][v][i]), false,
              false);
          acc[2 * a][v][i] = __uint_as_float(r[0]);
          acc[2 * a + 1][v][i] = __uint_as_float(r[1]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  }

  // This lane's outputs of fragments 2a and 2a + 1 by v: eight neighbours along
  // u, from column(wu, a) of the tile on.
  __device__ __forceinline__ void eight(float (&o)[8], int a, int v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = acc[2 * a + i / 4][v][i % 4];
  }
  static __device__ __forceinline__ int column(int wu, int a) {
    const int g = lane_id() >> 4;
    return place(a * 2 / kHalf, wu * kHalfRows) + a * 2 % kHalf * 16 +
           (AT ? (g & 1) * 16 + (g >> 1) * 8 : g * 8);
  }
};

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

constexpr int kUnits = 256;  // compute units

inline int64_t tiles_of(const Segments& s, int u, int bu, int bv) {
  const int64_t rows = s.pairs / s.E, busy = s.E < s.pairs ? s.E : s.pairs;
  return busy * ((rows + bv - 1) / bv) * ((u + bu - 1) / bu);
}

// e4m3 in 256 x 256 tiles and two steps of LDS, where every compute unit gets one
// and there are 16 rows an expert, so that most experts have some.  It moves less per
// product than smaller tiles (32 experts of 4096 x 7168 against 128 x 256 tiles: 16
// rows each 161 us against 164, 64 rows 169 against 187, 128 rows 196 against 234, 512
// rows 499 against 624; one expert and 2048 rows, which make 128 tiles, with the way
// back to 7168 columns 137 against 117).  Uneven routing gains more (rows by 1 / rank over
// the 32 experts: 16 rows 174 against 196, 64 rows 280 against 395) unless few experts have
// them all and the tiles are few after all (16 rows in one expert 82 against 71, 40 rows in
// eight 69 against 55).
using Codes = Config<2, 4, 8, 4>;
// 128 x 128, two blocks to a compute unit.
using NarrowCodes = Config<2, 4, 4, 2>;
inline bool large_codes(const Segments& s, int u) {
  return s.pairs / s.E >= 16 && tiles_of(s, u, Codes::kBu, Codes::kBv) >= kUnits;
}

// A launch has less than 2^32 threads.
inline bool launchable(int64_t blocks, int threads) { return blocks < (int64_t(1) << 32) / threads; }

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

}  // namespace moe
