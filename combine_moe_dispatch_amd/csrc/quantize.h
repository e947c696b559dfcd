// quantize.h -- rows and blocks to e4m3 with one scale for 128 columns:
// scale = max|v| / 448 and code = e4m3(v / scale), both IEEE fp32 divisions.
#pragma once

#include "device_common.h"

namespace moe {

// Magnitudes as integers: they order as the values do, and a NaN comes out
// above everything else, so that it reaches the scale.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The largest over the 4 lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ uint32_t max_over_rows(uint32_t m) {
  const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  const uint32_t n = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(n, n, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}
// The largest over each 16 neighbouring lanes (row rotations by 8, 4, 2, 1).
__device__ __forceinline__ uint32_t max_over_16(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xf, 0xf, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xf, 0xf, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xf, 0xf, true));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xf, 0xf, true));
}

// The scale of a block whose largest magnitude is given, and its codes.
//
// v / scale without a division: from the correctly rounded reciprocal r,
// q0 = v r and one remainder correction q0 + r (v - scale q0), both fused, give the
// correctly rounded quotient when nothing underflows (Markstein's division).
// Scales far from 1 are first brought near it, with the values, by a power of two,
// which is exact; then only quotients that round to code 0 can underflow.
// |q| <= 448 (1 + 2^-23)^2, which the packed convert rounds to nearest even, but
// for scales below 2^-126, which are too coarse: those quotients are cut at 448.
struct BlockScale {
  float scale, factor, by, inverse;

  __device__ __forceinline__ explicit BlockScale(uint32_t largest) {
    scale = __uint_as_float(largest) / 448.0f;
    factor = scale < 0x1p-80f ? 0x1p100f : scale > 0x1p80f ? 0x1p-100f : 1.0f;
    by = scale * factor;
    inverse = scale == 0.0f ? 0.0f : 1.0f / by;
    if (by == __builtin_inff()) by = 0.0f;  // then inverse is 0, and inf * 0 a NaN
  }

  // Eight neighbouring codes.
  __device__ __forceinline__ uint2 codes(const float (&v)[8]) const {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = v[i] * factor, q0 = x * inverse;
      // (this way round a remainder of 0 leaves a -0 its sign)
      q[i] = fmaf(-fmaf(by, q0, -x), inverse, q0);
    }
    if (scale < 0x1p-126f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(q[i], -448.0f), 448.0f);
    }
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
      c[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], lo, true);
    }
    return scale == 0.0f ? make_uint2(0, 0) : make_uint2(c[0], c[1]);
  }
};

}  // namespace moe
