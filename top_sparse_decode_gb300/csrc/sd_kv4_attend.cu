// Decode attention over the 4-bit K/V cache (HashAttention: Semantic Sparsity for Faster
// Inference, 2.1): z_i = scale <q, k_i>, o = sum e^{z_i - m} v_i / sum e^{z_i - m}, over a
// range of each sequence or over selected tokens.
//
// One CTA per (sequence, KV head); each warp an online softmax over every eighth token,
// four channels per lane, joined at the end.
#include "sd_internal.cuh"
#include "sd_kv4.cuh"

namespace sd {
namespace {

constexpr int kKaWarps = 8;

struct KaArgs {
  const uint16_t* q;
  sd_kv4 c;
  const int32_t* idx;
  int64_t idx_stride;
  const int32_t* count;
  int64_t max_count;
  const int32_t* begin;
  const int32_t* end;
  int Hq, Hkv;
  int64_t n, ncap;
  float scale;
  float* out;
  float* lse;
};

// Four consecutive channels 4 lane .. of a row.
__device__ __forceinline__ void ka_row(float (&x)[4], const uint8_t* code, const uint16_t* scale,
                                       int lane) {
  const int grp = lane >> 4, w = 2 * ((lane & 15) >> 1) + grp;
  const uint32_t word = reinterpret_cast<const uint32_t*>(code)[w] >> (16 * (lane & 1));
  const float s = bf16_to_f32(scale[2 * grp]), m = bf16_to_f32(scale[2 * grp + 1]);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = fmaf((float)((word >> (4 * i)) & 15u), s, m);
}

template <int G>
__global__ void __launch_bounds__(32 * kKaWarps) kv4_attend_kernel(const KaArgs a) {
  const int64_t row = blockIdx.x;
  const int b = (int)(row / a.Hkv), h = (int)(row % a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float q[G][4], o[G][4], m[G], l[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[g][i] = bf16_to_f32(a.q[((int64_t)b * a.Hq + h * G + g) * kD + 4 * lane + i]) * a.scale;
      o[g][i] = 0.0f;
    }
  }
  int64_t t0, t1;
  if (a.idx) {
    t0 = 0;
    t1 = imin64(a.count[row], a.max_count);
  } else {
    t0 = a.begin ? imax64(a.begin[b], 0) : 0;
    t1 = a.end ? imin64(a.end[b], a.n) : a.n;
  }
  for (int64_t t = t0 + warp; t < t1; t += kKaWarps) {
    const int64_t tok = a.idx ? a.idx[row * a.idx_stride + t] : t;
    if (tok < 0 || tok >= a.n) continue;
    const int64_t at = row * a.ncap + tok;
    float k[4], v[4];
    ka_row(k, a.c.k + at * kKv4Row, a.c.scale + at * kKv4Scales, lane);
    ka_row(v, a.c.v + at * kKv4Row, a.c.scale + at * kKv4Scales + 4, lane);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) z = fmaf(q[g][i], k[i], z);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, s);
      const float mn = fmaxf(m[g], z);
      const float w = m[g] == -INFINITY ? 0.0f : expf(m[g] - mn);
      const float p = z == -INFINITY ? 0.0f : expf(z - mn);
      m[g] = mn;
      l[g] = fmaf(l[g], w, p);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[g][i] = fmaf(o[g][i], w, p * v[i]);
    }
  }
  __shared__ float so[kKaWarps][G][kD], sm[kKaWarps][G], sl[kKaWarps][G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int i = 0; i < 4; ++i) so[warp][g][4 * lane + i] = o[g][i];
    if (lane == 0) {
      sm[warp][g] = m[g];
      sl[warp][g] = l[g];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < G * kD; e += 32 * kKaWarps) {
    const int g = e / kD, j = e % kD;
    float mm = -INFINITY, ll = 0.0f, oo = 0.0f;
    for (int w = 0; w < kKaWarps; ++w) mm = fmaxf(mm, sm[w][g]);
    for (int w = 0; w < kKaWarps; ++w) {
      const float f = sl[w][g] == 0.0f ? 0.0f : expf(sm[w][g] - mm);
      ll = fmaf(sl[w][g], f, ll);
      oo = fmaf(so[w][g][j], f, oo);
    }
    const int64_t bq = (int64_t)b * a.Hq + h * G + g;
    a.out[bq * kD + j] = ll != 0.0f ? oo / ll : 0.0f;
    if (a.lse && j == 0) a.lse[bq] = ll != 0.0f ? mm + logf(ll) : -INFINITY;
  }
}

}  // namespace

size_t kv4_attend_workspace_bytes(const Dims&, int64_t) { return 16; }

int launch_kv4_attend(const Dims& s, const uint16_t* q, const sd_kv4& c, const int32_t* idx,
                      int64_t idx_stride, const int32_t* count, int64_t max_count,
                      const int32_t* begin, const int32_t* end, float scale, float* out,
                      float* lse, void*, cudaStream_t st) {
  const KaArgs a{q,    c,     idx, idx_stride, count, max_count, begin, end, s.Hq, s.Hkv, s.n,
                 s.ncap, scale, out, lse};
  const unsigned rows = (unsigned)(s.B * s.Hkv);
  switch (s.G) {
    case 1: kv4_attend_kernel<1><<<rows, 32 * kKaWarps, 0, st>>>(a); break;
    case 2: kv4_attend_kernel<2><<<rows, 32 * kKaWarps, 0, st>>>(a); break;
    case 4: kv4_attend_kernel<4><<<rows, 32 * kKaWarps, 0, st>>>(a); break;
    default: kv4_attend_kernel<8><<<rows, 32 * kKaWarps, 0, st>>>(a); break;
  }
  note_launches(1);
  return check_launch("kv4 attend");
}

}  // namespace sd
