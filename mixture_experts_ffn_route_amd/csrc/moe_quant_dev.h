// e4m3 quantisation of 128-column blocks held by 16 consecutive lanes, eight
// columns each (the norm and the few-token layer).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"

namespace moe {

typedef uint32_t q_u32x2 __attribute__((ext_vector_type(2)));

// Maximum over a DPP row (16 consecutive lanes), in every lane of it.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));   // quad_perm: lane ^ 1
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));   // quad_perm: lane ^ 2
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));  // row_half_mirror: other quad
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true));  // row_mirror: other half
}

// The same over groups of 8 lanes.
__device__ __forceinline__ uint32_t row8_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));
}

// Quotients v / s of 8 values of a block with scale s, finite and not zero:
// from a reciprocal and one correction step; a scale below 2^-90, whose
// remainders could underflow, divides.
__device__ __forceinline__ void quotients8(const float v[8], float s, float q[8]) {
  if (s >= 0x1p-90f) {
    const float inv = 1.0f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q0 = v[i] * inv;
      q[i] = copysignf(fmaf(fmaf(-q0, s, v[i]), inv, q0), v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] / s;
  }
}

// Their e4m3 codes.
__device__ __forceinline__ q_u32x2 codes8(const float q[8]) {
  q_u32x2 w;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int lo = cvt2_e4m3(q[4 * j], q[4 * j + 1], 0, false);
    w[j] = (uint32_t)cvt2_e4m3(q[4 * j + 2], q[4 * j + 3], lo, true);
  }
  return w;
}

// Codes of a block whose scale is zero (all values are), or not finite (it
// holds a NaN or an infinity): zero, NaN.
__device__ __forceinline__ q_u32x2 codes_without_scale(float s) {
  const uint32_t w = s == 0.0f ? 0u : 0x7f7f7f7fu;
  return q_u32x2{w, w};
}

// Codes of 8 values of a block with scale s.
__device__ __forceinline__ q_u32x2 quant8(const float v[8], float s) {
  if (s == 0.0f || !isfinite(s)) return codes_without_scale(s);
  float q[8];
  quotients8(v, s, q);
  return codes8(q);
}

}  // namespace moe
