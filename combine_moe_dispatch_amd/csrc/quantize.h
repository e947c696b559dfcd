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
struct BlockScale {
  float scale, inverse;
  bool ordinary;

  __device__ __forceinline__ explicit BlockScale(uint32_t largest) {
    scale = __uint_as_float(largest) / 448.0f;
    inverse = 1.0f / scale;
    ordinary = scale >= 0x1p-80f && scale <= 0x1p80f;
  }

  // v / scale without a division: from the correctly rounded reciprocal r,
  // q0 = v r and one remainder correction q0 + r (v - scale q0), both fused,
  // give the correctly rounded quotient when nothing underflows (Markstein's
  // division).  In the ordinary range only quotients that round to code 0 can;
  // |q| <= 448 (1 + 2^-23)^2, which the packed convert rounds to nearest even.
  __device__ __forceinline__ float quotient(float v) const {
    const float q0 = v * inverse;
    return fmaf(fmaf(-scale, q0, v), inverse, q0);
  }

  // Eight neighbouring codes.
  __device__ __forceinline__ uint2 codes(const float (&v)[8]) const {
    uint32_t c[2] = {0, 0};
    if (ordinary) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * i]), quotient(v[4 * i + 1]),
                                                       0, false);
        c[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * i + 2]),
                                                         quotient(v[4 * i + 3]), lo, true);
      }
    } else if (scale != 0.0f) {  // very small or large, infinite or NaN
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i / 4] |= f32_to_e4m3(v[i] / scale) << (8 * (i % 4));
    }
    return make_uint2(c[0], c[1]);
  }
};

}  // namespace moe
