// Attention over ranges of the bf16 cache (include/sd.h, sd_window_attend and
// sd_prefix_attend): what its kernels share.
#pragma once

#include "sd_internal.cuh"

namespace sd {

constexpr float kDnLog2e = 1.4426950408889634f;
constexpr float kDnLn2 = 0.6931471805599453f;

// A kernel launched while the one before it in the stream ends waits here for it.
__device__ __forceinline__ void dn_wait_prior() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}
// Launches a kernel that way (it makes no read-only loads), in clusters where cluster > 0.
template <class P>
int dn_launch_early(const char* what, void (*kern)(P), unsigned grid, int threads, size_t smem,
                    int cluster, cudaStream_t st, const P& a, bool early = true) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (early) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return check_launch(what);
  note_launches(1);
  return check_launch(what);
}

// The window call's geometry: query token t of sequence b stands at first + pos[b] + t.
struct DnWindow {
  const int32_t* pos;
  const int32_t* length;
  int64_t first, m, n, window, sink;
  __device__ __forceinline__ int64_t at(int b) const { return first + (pos ? pos[b] : 0); }
  __device__ __forceinline__ int64_t len(int b) const {
    return length ? imax64(0, imin64(m, length[b])) : m;
  }
};

// The tokens that positions [p0, p1] see, as two ranges [0, s1) and [w0, w1), s1 <= w0.
struct DnRanges {
  int64_t s1, w0, w1;
};
__device__ __forceinline__ DnRanges dn_ranges(const DnWindow& w, int64_t p0, int64_t p1) {
  DnRanges r;
  r.w1 = imax64(0, imin64(w.n, p1 + 1));
  r.w0 = p0 - w.window < 0 ? 0 : imin64(p0 - w.window + 1, r.w1);
  r.s1 = imin64(imin64(w.sink, w.n), r.w1);
  if (r.s1 >= r.w0) r.s1 = 0, r.w0 = 0;  // one range
  return r;
}

// One query row's softmax, a warp over a range of tokens: lane l holds channels 4l .. 4l + 3
// of q (times scale log2 e) and of the sum.  m in log2 units.
struct DnRow {
  float4 q, o;
  float m, l;
};
__device__ __forceinline__ float4 dn_ld4(const uint16_t* p) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y));
}
__device__ __forceinline__ void dn_row_begin(DnRow& r, const uint16_t* q, float sl2, int lane) {
  const float4 x = dn_ld4(q + 4 * lane);
  r.q = make_float4(x.x * sl2, x.y * sl2, x.z * sl2, x.w * sl2);
  r.o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  r.m = -INFINITY;
  r.l = 0.0f;
}
__device__ __forceinline__ void dn_row_over(DnRow& r, const uint16_t* K, const uint16_t* V,
                                            int64_t i0, int64_t i1, int lane) {
  for (int64_t i = i0; i < i1; ++i) {
    const float4 k = dn_ld4(K + i * kD + 4 * lane), v = dn_ld4(V + i * kD + 4 * lane);
    float z = fmaf(r.q.x, k.x, fmaf(r.q.y, k.y, fmaf(r.q.z, k.z, r.q.w * k.w)));
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    const float top = fmaxf(r.m, z), mu = top == -INFINITY ? 0.0f : top;
    const float f = exp2f(r.m - mu), p = exp2f(z - mu);
    r.m = top;
    r.l = fmaf(r.l, f, p);
    r.o.x = fmaf(r.o.x, f, p * v.x);
    r.o.y = fmaf(r.o.y, f, p * v.y);
    r.o.z = fmaf(r.o.z, f, p * v.z);
    r.o.w = fmaf(r.o.w, f, p * v.w);
  }
}
__device__ __forceinline__ uint32_t dn_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void dn_row_end(const DnRow& r, uint16_t* out, float* lse, int lane) {
  const float inv = r.l == 0.0f ? 0.0f : 1.0f / r.l;  // a row that sees nothing: 0
  *reinterpret_cast<uint2*>(out + 4 * lane) =
      make_uint2(dn_pack(r.o.x * inv, r.o.y * inv), dn_pack(r.o.z * inv, r.o.w * inv));
  if (lse && lane == 0) *lse = r.l == 0.0f ? -INFINITY : (r.m + log2f(r.l)) * kDnLn2;
}

// sd_dense_stream.cu: one query token per sequence.
int64_t window_stream_parts(const Dims& s, int64_t tokens);
int launch_window_stream(const Dims& s, const uint16_t* q, const sd_strides& qs,
                         const uint16_t* K, const uint16_t* V, const DnWindow& w, bool own,
                         const int32_t* end, int64_t tokens, float scale, const float* pre_o,
                         const float2* pre_ml, int pre, uint16_t* out, const sd_strides& os,
                         float* lse, float* cut_o, float2* cut_ml, int* cut, cudaStream_t st);

}  // namespace sd
