// The 4-bit K/V cache's number format (include/sd.h, sd_kv4), shared by its kernels.
#pragma once

#include <cuda_bf16.h>

#include "sd_internal.cuh"

namespace sd {

constexpr int kKv4Row = 64;     // code bytes of a token's K (or V) row
constexpr int kKv4Scales = 8;   // bf16 values of a token's scale record
constexpr uint32_t kKv4NanPair = 0x7FC07FC0u;

// Short kernels are launched while the kernel before them in the stream ends, and wait for
// it here before they touch memory, which hides a part of the launch's latency (a write
// and a read of 64 x 8 tokens 5.0 us, 5.8 without; a cluster attention 0.3 to 0.7 us less).
__device__ __forceinline__ void kv4_wait_prior() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}
template <class... P, class... A>
int kv4_launch(const char* what, void (*kern)(P...), dim3 grid, int threads, size_t smem,
               int cluster, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return check_launch(what);
  note_launches(1);
  return check_launch(what);
}

// Pairs of fp32 values, one instruction for both.
__device__ __forceinline__ uint64_t f2_make(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// d / s from y = 1 / s, correctly rounded: t = d y, t + y (d - t s) (P. W. Markstein, IBM J.
// Res. Dev. 34(1), 1990).  A plain product d y would break the exact ties that coarse
// bf16 inputs hit often.
__device__ __forceinline__ float kv4_divide(float d, float s, float y) {
  const float t = d * y;
  return fmaf(fmaf(-t, s, d), y, t);
}
__device__ __forceinline__ uint64_t kv4_divide2(uint64_t d, uint64_t neg_s, uint64_t y) {
  const uint64_t t = f2_mul(d, y);
  return f2_fma(f2_fma(t, neg_s, d), y, t);
}

// A group's step: bf16((hi - lo) / 15), the fp32 quotient rounded to nearest even; 0
// below 2^-100 (the remainders of the divisions by it stay exact); NaN when a value of the
// group is not finite or the step overflows.
__device__ __forceinline__ float kv4_step(float lo, float hi) {
  const float q = kv4_divide(hi - lo, 15.0f, 0.0666666701f);  // the fp32 nearest to 1 / 15
  const float s = __bfloat162float(__float2bfloat16_rn(q));
  if (!(s < INFINITY)) return __uint_as_float(0x7FC00000u);
  return s < 7.8886091e-31f ? 0.0f : s;
}

// 1 / s correctly rounded, for a normal s of eight significant bits: the hardware's
// approximation and one Newton step (equal to the IEEE reciprocal for every such s).
__device__ __forceinline__ float kv4_rcp(float s) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(s));
  return fmaf(fmaf(-s, y, 1.0f), y, y);
}

// A word of codes from the octet x: clamp(rint((x - lo) / s), 0, 15) at bits 4 i; y = 1 / s
// correctly rounded, or 0 for s = 0 (codes 0).
__device__ __forceinline__ uint32_t kv4_word(const uint4& x, float lo, float s, float y) {
  const uint64_t l2 = f2_make(-lo, -lo), s2 = f2_make(-s, -s), y2 = f2_make(y, y);
  // adding 1.5 2^23 rounds to a whole number (ties to even): the bits 0x4B400000 + c
  const uint64_t magic = f2_make(12582912.0f, 12582912.0f);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t word = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    float q0, q1;
    f2_split(kv4_divide2(f2_add(f2_make(bf16_lo(w[i]), bf16_hi(w[i])), l2), s2, y2), q0, q1);
    f2_split(f2_add(f2_make(fminf(q0, 15.0f), fminf(q1, 15.0f)), magic), q0, q1);
    word = (word * 16u + __float_as_uint(q1)) * 16u + __float_as_uint(q0);
  }
  return word - 0x4B400000u * 0x11111111u;  // modulo 2^32
}

// Two channels of a word of codes (from bit sh) as packed bf16.
__device__ __forceinline__ uint32_t kv4_pair(uint32_t word, int sh, float s, float m) {
  // a code under the exponent of 2^23 is 2^23 + c
  const float a = __uint_as_float((word >> sh & 15u) | 0x4B000000u) - 8388608.0f;
  const float b = __uint_as_float((word >> (sh + 4) & 15u) | 0x4B000000u) - 8388608.0f;
  const __nv_bfloat162 r = __floats2bfloat162_rn(fmaf(a, s, m), fmaf(b, s, m));
  return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace sd
