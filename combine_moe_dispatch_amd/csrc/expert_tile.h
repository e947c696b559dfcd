// expert_tile.h -- how the tiled products find their work and move their
// operands: tiles of a grouped product numbered from the device counts, and
// loads that go from global memory straight into LDS.
#pragma once

#include "expert_device.h"

namespace moe {

typedef short i16x4_t __attribute__((ext_vector_type(4)));

// One tile of a product over the placed rows: rows [m0, end) of expert e from
// m0 on, column tile n.
struct Tile {
  int e, m0, end, n;
};

// Tiles of one expert run through groups of row tiles, column tile by column
// tile, so that the tiles running together on an XCD share few row and column
// slabs in its L2: groups of 4 row tiles where two tiles share a compute unit,
// equal ones of at most 8 where each has its own (32 experts, 4096 x 7168,
// against groups of 4: 6000 tokens 2.38 -> 2.26 ms, 8192 3.05 -> 3.00; of 16,
// 16384 tokens 6.00 -> 6.16).
template <int BV>
__device__ __forceinline__ unsigned group_rows(unsigned tiles) {
  if (BV < 256) return 4;
  if (tiles <= 8) return tiles;
  const unsigned groups = (tiles + 7) / 8;
  return (tiles + groups - 1) / groups;
}

// Tile `b` of the launch, or false when there are fewer.  Every wave works it
// out for itself: lane i of a pass looks at expert base + i, and a prefix sum
// over the lanes finds the expert whose tiles hold it.  The first pass counts
// all tiles, so that they can be dealt to the XCDs in runs; up to 64 experts
// it is the only one.
template <int BV>
__device__ __forceinline__ bool find_tile(const Segments& s, int ntiles, unsigned b, Tile& t) {
  const int lane = lane_id();
  int begin, end, mt, incl;
  auto look = [&](int base) {
    begin = end = 0;
    if (base + lane < s.E) segment_of(s, base + lane, begin, end);
    mt = end > begin ? (end - begin + BV - 1) / BV : 0;
    incl = wave_inclusive_sum_dpp(mt);
    return (unsigned)__builtin_amdgcn_readlane(incl, 63);
  };
  unsigned total = look(0);
  for (int base = kWave; base < s.E; base += kWave) total += look(base);
  total *= (unsigned)ntiles;
  if (b >= total) return false;
  unsigned left = xcd_local_block(b, total);
  for (int base = 0; base < s.E; base += kWave) {
    if (s.E > kWave) look(base);
    const unsigned here = (unsigned)__builtin_amdgcn_readlane(incl, 63) * (unsigned)ntiles;
    if (left >= here) {
      left -= here;
      continue;
    }
    // the first lane whose inclusive tile count passes `left`
    const uint64_t past = __ballot((unsigned)incl * (unsigned)ntiles > left);
    const int src = __ffsll((unsigned long long)past) - 1;
    const int mts = __builtin_amdgcn_readlane(mt, src);
    left -= (unsigned)(__builtin_amdgcn_readlane(incl, src) - mts) * (unsigned)ntiles;
    t.e = base + src;
    const int first = __builtin_amdgcn_readlane(begin, src);
    t.end = __builtin_amdgcn_readlane(end, src);
    const unsigned most = group_rows<BV>((unsigned)mts);
    const unsigned g = left / (most * (unsigned)ntiles);
    const unsigned rows = min(most, (unsigned)mts - g * most);
    left -= g * most * (unsigned)ntiles;
    t.n = (int)(left / rows);
    t.m0 = first + (int)(g * most + left % rows) * BV;
    return true;
  }
  return false;
}

// Every expert's rows in LDS, for blocks that take one tile after another: a
// look at the counts in memory would wait for the block's loads and stores
// under way.  A barrier has to follow.
constexpr int kTableBytes = 2 * kMaxExperts * 4;
__device__ __forceinline__ void fill_table(int* begin, int* rows, const Segments& s) {
  for (int e = threadIdx.x; e < s.E; e += blockDim.x) {
    int first, end;
    segment_of(s, e, first, end);
    begin[e] = first;
    rows[e] = end - first;
  }
}

// Most tiles a grouped product can have: every expert may end in a part tile.
inline int64_t tile_bound(const Segments& s, int bv, int ntiles) {
  const int64_t busy = s.E < s.pairs ? s.E : s.pairs;
  return ((int64_t)s.pairs / bv + busy) * ntiles;
}

// 16 bytes a lane from base + offset to LDS, lane i at lds + 16 i.  The load
// counts in vmcnt; the compiler does not know it, so wait with wait_vm.
__device__ __forceinline__ void load_to_lds(uint32_t lds, const void* base, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(offset), "s"(base)
               : "memory", "m0");
}
// 4 bytes a lane from an address of its own, lane i at lds + 4 i.
__device__ __forceinline__ void load4_to_lds(uint32_t lds, const void* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds), "v"(p)
               : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// c += a b on the 16 x 16 x 32 matrix unit, the accumulators staying where they
// are: with the builtin the compiler moved them between registers around the
// loops over a tile (as many moves as products at 256 accumulators).  The
// compiler does not see that this is a matrix instruction: after the last one
// mfma_results, then mfma_result on every accumulator, before it is read.
__device__ __forceinline__ void mfma_in_place(f32x4_t& c, bf16x8_t a, bf16x8_t b) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
// A matrix instruction may not read what a vector instruction wrote less than
// two wait states before; mfma_in_place keeps no such distance by itself.  Its
// operands come out of LDS, whose reads are waited for, except where they are
// masked: those pass through here.  (The two states in front of every product
// take 1% of a prefill's time.)
__device__ __forceinline__ void operand_written(bf16x8_t& v) { asm volatile("s_nop 1" : "+v"(v)); }
// The last product's results get written (8 wait states would do).
__device__ __forceinline__ void mfma_results() { asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15"); }
__device__ __forceinline__ void mfma_result(f32x4_t& c) { asm volatile("" : "+a"(c)); }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)reinterpret_cast<const __attribute__((address_space(3))) void*>(
      (uintptr_t)p);
}

// ---------------------------------------------------------------------------
// Operand tiles in LDS.  One step of a product takes kStep values along the
// reduction r.  An operand whose rows run along r lies as [rows][kStep]; one
// held transposed (rows along the other dimension) as [kStep][cols], read back
// through the transposing LDS load.  Both are filled by wave loads of 1 KB, so
// the layout is linear in the lanes and the 16-byte chunks of a row are
// permuted on the global side instead: chunk c of row i sits in slot c ^ f(i),
// which spreads the reads of a fragment over all banks (no conflicts counted),
// but for the transposed paired operand, whose reads meet two by two (8% of the
// row gradient's busy cycles, 4% of the weight gradient's).
// ---------------------------------------------------------------------------
constexpr int kStep = 64;
constexpr int kPart = 32;             // r values of one 16 x 16 x 32 product
constexpr int kParts = kStep / kPart;

// PAIRED, for the operand that makes the output's contiguous dimension: two
// neighbouring fragments share 32 rows, row g * 8 + b * 4 + i being row
// g * 4 + i of fragment b, so that the pair leaves every lane with 8
// neighbouring outputs.
template <int SIZE, int WAVES, bool TRANSPOSED, bool PAIRED>
struct OperandTile {
  static constexpr int kBytes = SIZE * kStep * 2;
  static constexpr int kLoads = kBytes / 1024 / WAVES;  // wave loads per wave and step
  static_assert(kLoads * WAVES * 1024 == kBytes, "whole wave loads");
  static constexpr int kSlots = TRANSPOSED ? SIZE / 8 : kStep / 8;  // chunks in a row
  static constexpr int kRowsPerLoad = 64 / kSlots;
  uint32_t off[kLoads];    // byte offset of this lane's chunk, step 0
  uint16_t where[kLoads];  // its first position along r within a step

  static __device__ __forceinline__ int swizzle(int row) {
    if (TRANSPOSED) return ((row & 3) | ((row >> 3) & 1) << 2) << 1;
    return PAIRED ? ((row >> 1) & 1) | ((row >> 3) & 3) << 1 : (row >> 1) & 7;
  }
  // Load i of a wave among the tile's: the waves' first loads fill its front.
  static __device__ __forceinline__ int load_of(int i, int wave) { return i * WAVES + wave; }
  // The chunk that this lane brings in with load q of the tile, and its row.
  static __device__ __forceinline__ void chunk_of(int q, int& row, int& c) {
    const int lane = lane_id();
    row = q * kRowsPerLoad + lane / kSlots;
    c = (lane % kSlots) ^ swizzle(row);
  }

  // ld: bytes between rows.  valid: rows (columns, when transposed: a multiple
  // of 8) the tile really has, at least one (eight); past them the last one is
  // read again.
  __device__ __forceinline__ void init(int wave, uint32_t ld, int valid) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      int row, c;
      chunk_of(load_of(i, wave), row, c);
      if constexpr (TRANSPOSED) {
        off[i] = (uint32_t)row * ld + (uint32_t)min(c * 8, valid - 8) * 2;
        where[i] = (uint16_t)row;
      } else {
        off[i] = (uint32_t)min(row, valid - 1) * ld + (uint32_t)c * 16;
        where[i] = (uint16_t)(c * 8);
      }
    }
  }
  // Start load i of a step whose first value, for this load, is at base.
  // left < kStep: only that many positions exist, others re-read the first.
  template <bool TAIL>
  __device__ __forceinline__ void load(int i, uint32_t lds, int wave, const char* base,
                                       uint32_t ld, int left) const {
    uint32_t o = off[i];
    if (TAIL && (int)where[i] >= left)
      o -= TRANSPOSED ? (uint32_t)where[i] * ld : (uint32_t)where[i] * 2;
    load_to_lds(lds + (uint32_t)load_of(i, wave) * 1024, base, o);
  }

  // Reading fragments: N of 16 rows each (columns, when transposed) from i0
  // on.  Lane l of a fragment holds its row l & 15 and, of part k of the step,
  // the positions (l >> 4) * 8 .. + 7.  The swizzle depends on the lane alone
  // (and on k, or on n when transposed), so the addresses are made once and
  // the rest is in the instructions' offsets.
  template <int N>
  struct Reader {
    static constexpr int kAts = !TRANSPOSED ? kParts : PAIRED ? N / 2 : N;
    uint32_t at[kAts];
    // apart: fragments of the operand between two of this reader's (transposed
    // only; else the caller numbers them so)
    __device__ __forceinline__ void init(int i0, int apart = 1) {
      const int lane = lane_id(), j = lane & 15;
      if constexpr (TRANSPOSED) {
        // 16 lanes turn a block of 4 positions x 16 columns around: lane j of
        // them names 8 bytes of it and receives column j
        const int row = (lane >> 4) * 8 + (j >> 2);
#pragma unroll
        for (int n = 0; n < kAts; ++n) {
          const int col = i0 + (PAIRED ? n * 32 + (j & 3) * 8 : n * apart * 16 + (j & 3) * 4);
          at[n] = (uint32_t)(row * (SIZE * 2) + ((col / 8) ^ swizzle(row)) * 16 + (col & 4) * 2);
        }
      } else {
        const int row = i0 + (PAIRED ? (j >> 2) * 8 + (j & 3) : j);
#pragma unroll
        for (int k = 0; k < kParts; ++k)
          at[k] = (uint32_t)(row * (kStep * 2) + ((k * 4 + (lane >> 4)) ^ swizzle(row)) * 16);
      }
    }
    // lds: LDS address of the operand's step.  TAIL: positions at or past left
    // are zero.
    template <bool TAIL>
    __device__ __forceinline__ bf16x8_t frag(uint32_t lds, int n, int k, int left) const {
      union {
        bf16x8_t v;
        i16x4_t h[2];
        uint32_t w[4];
      } u;
      if constexpr (TRANSPOSED) {
        const uint32_t p = lds + (PAIRED ? at[n / 2] + n % 2 * 8 : at[n]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) i16x4_t*)(uintptr_t)(
                  p + (k * kPart + h * 4) * (SIZE * 2)));
      } else {
        const int row = PAIRED ? n / 2 * 32 + n % 2 * 4 : n * 16;
        u.v = *(const __attribute__((address_space(3))) bf16x8_t*)(uintptr_t)(
            lds + at[k] + row * (kStep * 2));
      }
      if constexpr (TAIL) {
        const int r = k * kPart + (lane_id() >> 4) * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = r + 2 * j < left ? 0x0000ffffu : 0u;
          const uint32_t hi = r + 2 * j + 1 < left ? 0xffff0000u : 0u;
          u.w[j] &= lo | hi;
        }
        operand_written(u.v);
      }
      return u.v;
    }
  };
};

}  // namespace moe
