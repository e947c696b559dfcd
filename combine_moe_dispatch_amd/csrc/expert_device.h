// expert_device.h -- device helpers of the expert product and its gradient.
#pragma once

#include "device_common.h"
#include "experts.h"

namespace moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActSwiglu = 3 };

// Rows [begin, end) of expert e that hold placed pairs: its counts cut at its
// rank's capacity, and at the buffer whatever the metadata says.
__device__ __forceinline__ void segment_of(const Segments& s, int e, int& begin, int& end) {
  if (s.counts == nullptr) {
    begin = 0;
    end = s.rows;
    return;
  }
  begin = max(s.offsets[e], 0);
  int64_t last = (int64_t)begin + max(s.counts[e], 0);
  if (s.C > 0) last = min(last, (int64_t)(e / s.L) * s.C + s.C);
  end = (int)min(last, (int64_t)s.rows);
}

// Eight neighbouring bf16 values to and from memory (16 bytes).
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void add8(float (&v)[8], const uint16_t* p) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] += bf16_lo(w[i]);
    v[2 * i + 1] += bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void add8(float (&v)[8], const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] += a.x;
  v[1] += a.y;
  v[2] += a.z;
  v[3] += a.w;
  v[4] += b.x;
  v[5] += b.y;
  v[6] += b.z;
  v[7] += b.w;
}

__device__ __forceinline__ float sigmoid_f32(float v) { return 1.0f / (1.0f + expf(-v)); }

// The same for results that are rounded to bf16 next: the hardware's 2^x and
// reciprocal, off by (1 + |v|) 2^-23 of the value or so where the rounding is
// off by 2^-8.  A tile's activations are thousands of these per lane.
__device__ __forceinline__ float sigmoid_short(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504088896341f));
}

// act(z) for the one-input activations
template <int ACT>
__device__ __forceinline__ float act_f32(float z) {
  if (ACT == kActSilu) return z * sigmoid_short(z);
  if (ACT == kActGelu) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
  return z;
}

}  // namespace moe
