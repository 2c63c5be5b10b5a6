// Attention over ranges of the bf16 cache (include/sd.h, sd_window_attend and
// sd_prefix_attend): what its kernels share.
#pragma once

#include "sd_dense_plan.cuh"
#include "sd_internal.cuh"
#include "sd_mma.cuh"

namespace sd {

constexpr float kDnLog2e = 1.4426950408889634f;
constexpr float kDnLn2 = 0.6931471805599453f;

// A kernel launched while the one before it in the stream ends waits here for it.  (In a place
// and under a name of its own: the kernels that use it are held to ordinary loads by name.)
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
// of q and of the sum.  m in log2 units.
struct DnRow {
  float4 q, o;
  float m, l;
};
__device__ __forceinline__ float4 dn_ld4(const uint16_t* p) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y));
}
__device__ __forceinline__ void dn_row_over(DnRow& r, const uint16_t* K, const uint16_t* V,
                                            int64_t i0, int64_t i1, float sl2, int lane) {
  for (int64_t i = i0; i < i1; ++i) {
    const float4 k = dn_ld4(K + i * kD + 4 * lane), v = dn_ld4(V + i * kD + 4 * lane);
    float z = fmaf(r.q.x, k.x, fmaf(r.q.y, k.y, fmaf(r.q.z, k.z, r.q.w * k.w)));
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    z *= sl2;
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
__device__ __forceinline__ void dn_row_end(const DnRow& r, uint16_t* out, float* lse, int lane) {
  const float inv = r.l == 0.0f ? 0.0f : 1.0f / r.l;  // a row that sees nothing: 0
  *reinterpret_cast<uint2*>(out + 4 * lane) =
      make_uint2(bf16_pack(r.o.x * inv, r.o.y * inv), bf16_pack(r.o.z * inv, r.o.w * inv));
  if (lse && lane == 0) *lse = r.l == 0.0f ? -INFINITY : (r.m + log2f(r.l)) * kDnLn2;
}

// ---- a warp's softmax of eight rows over groups of 16 tokens --------------------------------
// S = Q K^T as m16n8k16 bf16 products (M: the rows, upper half empty), p = 2^(s - m) in fp32,
// O^T += V^T P^T with p as two bf16 parts (16 bits of it) and V^T read by transposing matrix
// loads.  A group's K and V lie in shared memory, chunks of 16 bytes XOR-swizzled by token, so
// that the matrix loads meet no bank twice.
constexpr uint32_t kDnRowBytes = kD * 2;
constexpr uint32_t kDnHalf = kSwGroup * kDnRowBytes;  // a group's K: 4 KB; V behind it
constexpr uint32_t kDnStage = 2 * kDnHalf;

__device__ __forceinline__ uint32_t dn_su32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void dn_ldm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void dn_ldmt(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void dn_cp16(uint32_t dst, const uint16_t* src, bool v) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
               "r"(v ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void dn_cp_commit() {
  asm volatile("cp.async.commit_group;\n" ::: "memory");
}
template <int N>
__device__ __forceinline__ void dn_cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
// Copies of a group whose first token is at element `at` of K and V, `have` of 16 tokens.
__device__ __forceinline__ void dn_fetch(uint32_t stage, const uint16_t* K, const uint16_t* V,
                                         int64_t at, int have, int lane) {
  const int lr = lane >> 4, lc = lane & 15;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int t = 2 * k + lr;
    const uint32_t dst = stage + t * kDnRowBytes + ((lc ^ (t & 7)) << 4);
    const int64_t src = at + 8 * lc + (t < have ? t : 0) * kD;
    dn_cp16(dst, K + src, t < have);
    dn_cp16(dst + kDnHalf, V + src, t < have);
  }
}
// Row gid = lane / 4 of S: m (log2 units) and this lane's share of l; columns 2 tig, 2 tig + 1
// (tig = lane % 4) of O^T.
struct DnEight {
  float o[8][4];
  float m, l;
};
__device__ __forceinline__ void dn_eight_begin(DnEight& x) {
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) x.o[mt][0] = x.o[mt][1] = x.o[mt][2] = x.o[mt][3] = 0.0f;
  x.m = -INFINITY;
  x.l = 0.0f;
}
// A group of `have` tokens; real: this lane's row exists.  m moves when a group's maximum is
// more than `slack` above it.
__device__ __forceinline__ void dn_eight_step(DnEight& x, const uint32_t (&qa)[8][2],
                                              uint32_t at, int have, bool real, float sl2,
                                              float slack, int lane) {
  const int tig = lane & 3;
  float sc[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int t = 8 * n + (lane & 7);
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) {
      uint32_t k[4];
      dn_ldm(k, at + t * kDnRowBytes + (((4 * kp + (lane >> 3)) ^ (t & 7)) << 4));
      mma_bf16(sc[n], qa[2 * kp][0], 0u, qa[2 * kp][1], 0u, k[0], k[1]);
      mma_bf16(sc[n], qa[2 * kp + 1][0], 0u, qa[2 * kp + 1][1], 0u, k[2], k[3]);
    }
  }
  float z[2][2], top = -INFINITY;
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      z[n][e] = real && 8 * n + 2 * tig + e < have ? sc[n][e] * sl2 : -INFINITY;
      top = fmaxf(top, z[n][e]);
    }
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  const bool need = top > x.m + slack;
  if (__any_sync(0xFFFFFFFFu, need)) {
    const float f = need ? exp2f(x.m - top) : 1.0f;  // m = -inf: 0
    // O^T's columns 2tig, 2tig + 1 are rows whose factors the lanes of S's rows hold
    const float fa = __shfl_sync(0xFFFFFFFFu, f, 8 * tig);
    const float fb = __shfl_sync(0xFFFFFFFFu, f, 8 * tig + 4);
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      x.o[mt][0] *= fa;
      x.o[mt][1] *= fb;
      x.o[mt][2] *= fa;
      x.o[mt][3] *= fb;
    }
    x.l *= f;
    if (need) x.m = top;
  }
  const float mu = x.m == -INFINITY ? 0.0f : x.m;
  // a weight as two bf16, its upper half and what that leaves: 16 bits of it.  Neither part is
  // negative, and the second is a 2^17th of the weight at least (0 only below 2^-116), so that
  // an infinity in V stays what it is and a weight of 0 stays 0.
  uint32_t p[2], rest[2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const float u = exp2f(z[n][0] - mu), v = exp2f(z[n][1] - mu);
    x.l += u + v;
    p[n] = __byte_perm(__float_as_uint(u), __float_as_uint(v), 0x7632);
    rest[n] = bf16_pack(fmaxf(u - bf16_lo(p[n]), u * 0x1p-17f),
                        fmaxf(v - bf16_hi(p[n]), v * 0x1p-17f));
  }
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) {
    const int t = (lane & 7) + 8 * (lane >> 4);
    uint32_t v[4];
    dn_ldmt(v, at + kDnHalf + t * kDnRowBytes + (((2 * mt + ((lane >> 3) & 1)) ^ (t & 7)) << 4));
    mma_bf16(x.o[mt], v[0], v[1], v[2], v[3], p[0], p[1]);
    mma_bf16(x.o[mt], v[0], v[1], v[2], v[3], rest[0], rest[1]);
  }
}
// O to shared memory, o[row][d], of the first `rows` rows; each row's l whole in its lanes.
__device__ __forceinline__ void dn_eight_end(DnEight& x, float* o, int rows, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
  x.l += __shfl_xor_sync(0xFFFFFFFFu, x.l, 1);
  x.l += __shfl_xor_sync(0xFFFFFFFFu, x.l, 2);
  __syncwarp();  // o may lie where the last groups did
#pragma unroll
  for (int mt = 0; mt < 8; ++mt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = 2 * tig + (e & 1);
      if (row < rows) o[row * kD + 16 * mt + 8 * (e >> 1) + gid] = x.o[mt][e];
    }
}

// sd_dense_stream.cu: one query token per sequence.
int64_t window_stream_parts(const Dims& s, int64_t tokens);
int launch_window_stream(const Dims& s, const uint16_t* q, const sd_strides& qs,
                         const uint16_t* K, const uint16_t* V, const DnWindow& w, bool own,
                         const int32_t* end, int64_t tokens, float scale, const float* pre_o,
                         const float2* pre_ml, int pre, uint16_t* out, const sd_strides& os,
                         float* lse, float* cut_o, float2* cut_ml, int* cut, cudaStream_t st);

}  // namespace sd
