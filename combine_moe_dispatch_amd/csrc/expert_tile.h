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

// Tiles of one expert run through groups of kGroupRows row tiles, column tile
// by column tile, so that the tiles running together on an XCD share few row
// and column slabs in its L2 (4 x 8 of them on its 32 compute units).
constexpr int kGroupRows = 4;

// Tile `b` of the launch, or false when there are fewer.  Every wave works it
// out for itself: lane i of a pass looks at expert base + i, and a prefix sum
// over the lanes finds the expert whose tiles hold it.
template <int BV>
__device__ __forceinline__ bool find_tile(const Segments& s, int ntiles, unsigned b, Tile& t) {
  const int lane = lane_id();
  // all tiles, so that the tiles can be dealt to the XCDs in runs
  unsigned total = 0;
  for (int base = 0; base < s.E; base += kWave) {
    int begin = 0, end = 0;
    if (base + lane < s.E) segment_of(s, base + lane, begin, end);
    const int mt = end > begin ? (end - begin + BV - 1) / BV : 0;
    total += (unsigned)__builtin_amdgcn_readlane(wave_inclusive_sum_dpp(mt), 63);
  }
  total *= (unsigned)ntiles;
  if (b >= total) return false;
  unsigned left = xcd_local_block(b, total);
  for (int base = 0; base < s.E; base += kWave) {
    int begin = 0, end = 0;
    if (base + lane < s.E) segment_of(s, base + lane, begin, end);
    const int mt = end > begin ? (end - begin + BV - 1) / BV : 0;
    const int incl = wave_inclusive_sum_dpp(mt);
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
    const unsigned per = kGroupRows * (unsigned)ntiles;
    const unsigned g = left / per;
    const unsigned rows = min((unsigned)kGroupRows, (unsigned)mts - g * kGroupRows);
    left -= g * per;
    t.n = (int)(left / rows);
    t.m0 = first + (int)(g * kGroupRows + left % rows) * BV;
    return true;
  }
  return false;
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
               : "memory");
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

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
// which spreads the reads of a fragment over all banks.
// ---------------------------------------------------------------------------
constexpr int kStep = 64;

template <int SIZE, int WAVES, bool TRANSPOSED>
struct OperandTile {
  static constexpr int kBytes = SIZE * kStep * 2;
  static constexpr int kLoads = kBytes / 1024 / WAVES;  // wave loads per wave and step
  static_assert(kLoads * WAVES * 1024 == kBytes, "whole wave loads");
  uint32_t off[kLoads];   // byte offset of this lane's chunk, step 0
  uint16_t where[kLoads]; // its first position along r within a step

  static __device__ __forceinline__ int swizzle(int row) {
    return TRANSPOSED ? ((row & 3) | ((row >> 3) & 1) << 2) << 1 : (row >> 1) & 7;
  }

  // ld: bytes between rows.  valid: rows (columns, when transposed: a multiple
  // of 8) the tile really has, at least one (eight); past them the last one is
  // read again.
  __device__ __forceinline__ void init(int wave, uint32_t ld, int valid) {
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int q = wave * kLoads + i;
      if constexpr (TRANSPOSED) {
        constexpr int kSlots = SIZE / 8;  // chunks in a row
        const int at = q * 64 + lane;
        const int r = at / kSlots;
        const int c = min(((at % kSlots) ^ swizzle(r)) * 8, valid - 8);
        off[i] = (uint32_t)r * ld + (uint32_t)c * 2;
        where[i] = (uint16_t)r;
      } else {
        const int row = q * 8 + lane / 8;
        const int c = (lane % 8) ^ swizzle(row);
        off[i] = (uint32_t)min(row, valid - 1) * ld + (uint32_t)c * 16;
        where[i] = (uint16_t)(c * 8);
      }
    }
  }
  // Start the loads of one step: base[i] is where load i starts in it.
  // left < kStep: only that many positions exist, others re-read the first.
  template <bool TAIL>
  __device__ __forceinline__ void load(uint32_t lds, int wave, const char* const (&base)[kLoads],
                                       uint32_t ld, int left) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint32_t o = off[i];
      if (TAIL && (int)where[i] >= left)
        o -= TRANSPOSED ? (uint32_t)where[i] * ld : (uint32_t)where[i] * 2;
      load_to_lds(lds + (uint32_t)(wave * kLoads + i) * 1024, base[i], o);
    }
  }
  // Reading fragments: N of 16 rows each (columns, when transposed) from i0
  // on.  Lane l of fragment n holds row l & 15 and, of the 32 values along r
  // from ks * 32 on, (l >> 4) * 8 .. + 7.  The swizzle depends on the lane
  // alone (and, transposed, on n), so the addresses are made once and the rest
  // is in the instructions' offsets.
  template <int N>
  struct Reader {
    uint32_t at[TRANSPOSED ? N : kStep / 32];
    __device__ __forceinline__ void init(int i0) {
      const int lane = lane_id();
      if constexpr (TRANSPOSED) {
        const int row = (lane >> 4) * 8 + ((lane & 15) >> 2);
#pragma unroll
        for (int n = 0; n < N; ++n)
          at[n] = (uint32_t)(row * (SIZE * 2) + ((i0 / 8 + 2 * n) ^ swizzle(row)) * 16 +
                             (lane & 3) * 8);
      } else {
        const int row = i0 + (lane & 15);
#pragma unroll
        for (int ks = 0; ks < kStep / 32; ++ks)
          at[ks] = (uint32_t)(row * (kStep * 2) + ((ks * 4 + (lane >> 4)) ^ swizzle(row)) * 16);
      }
    }
    // lds: LDS address of the operand's step.  TAIL: values at or past left
    // are zero.
    template <bool TAIL>
    __device__ __forceinline__ bf16x8_t frag(uint32_t lds, int n, int ks, int left) const {
      union {
        bf16x8_t v;
        i16x4_t h[2];
        uint32_t w[4];
      } u;
      if constexpr (TRANSPOSED) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          u.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) i16x4_t*)(uintptr_t)(
                  lds + at[n] + (ks * 32 + h * 4) * (SIZE * 2)));
      } else {
        u.v = *(const __attribute__((address_space(3))) bf16x8_t*)(uintptr_t)(
            lds + at[ks] + n * 16 * (kStep * 2));
      }
      if constexpr (TAIL) {
        const int r = ks * 32 + (lane_id() >> 4) * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = r + 2 * j < left ? 0x0000ffffu : 0u;
          const uint32_t hi = r + 2 * j + 1 < left ? 0xffff0000u : 0u;
          u.w[j] &= lo | hi;
        }
      }
      return u.v;
    }
  };
};

}  // namespace moe
