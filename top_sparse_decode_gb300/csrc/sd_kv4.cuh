// The 4-bit K/V cache's number format (include/sd.h, sd_kv4), shared by its kernels.
#pragma once

#include <cuda_bf16.h>

#include "sd_internal.cuh"

namespace sd {

constexpr int kKv4Row = 64;     // code bytes of a token's K (or V) row
constexpr int kKv4Scales = 8;   // bf16 values of a token's scale record
constexpr uint32_t kKv4NanPair = 0x7FC07FC0u;

// A group's step: bf16((hi - lo) / 15), the fp32 quotient rounded to nearest even; 0
// below 2^-100 (the remainders that kv4_code forms stay exact); NaN when a value of the
// group is not finite or the step overflows.
__device__ __forceinline__ float kv4_step(float lo, float hi) {
  const float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(hi - lo, 15.0f)));
  if (!(s < INFINITY)) return __uint_as_float(0x7FC00000u);
  return s < 7.8886091e-31f ? 0.0f : s;
}

// clamp(rint(d / s), 0, 15) for d >= 0; y = 1 / s correctly rounded (0 for s = 0).  The
// quotient is formed as t = d y, t + y (d - t s), which is the correctly rounded d / s
// (P. W. Markstein, IBM J. Res. Dev. 34(1), 1990): a plain product d y breaks the exact
// ties that coarse bf16 inputs hit often.
__device__ __forceinline__ uint32_t kv4_code(float d, float s, float y) {
  const float t = d * y;
  const float q = fmaf(fmaf(-t, s, d), y, t);
  return (uint32_t)fminf(rintf(q), 15.0f);
}

// Two channels of a word of codes (from bit sh) as packed bf16.
__device__ __forceinline__ uint32_t kv4_pair(uint32_t word, int sh, float s, float m) {
  const float a = fmaf((float)((word >> sh) & 15u), s, m);
  const float b = fmaf((float)((word >> (sh + 4)) & 15u), s, m);
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace sd
