// Queries and keys normed per head and rotated by position on their way from the projection
// into q and the bf16 cache, values copied beside them (HashAttention: Semantic Sparsity for
// Faster Inference, 2.1: the q, k and v that the three stages start from).
//
//   y = x / sqrt(mean(x^2) + eps) * w,  (y_a, y_b) -> (y_a cos t - y_b sin t,
//   y_b cos t + y_a sin t),  t = position * inv_freq[j], pair j = (j, j + rot / 2) or
//   (2j, 2j + 1).
//
// Bound by HBM: every row is read and written once (512 bytes), with some 15 instructions
// per 16 bytes.  A CTA takes kRpTok tokens of a sequence (one, and a share of its heads,
// where there are few): its threads form the tokens' angles first, one each, while the first
// rows' loads are in flight -- in 64 bits up to the fraction of a turn, since position *
// inv_freq reaches 10^6 radians -- and then 16 lanes take a row, 16 bytes a lane, kRpRows
// rows of a lane in flight.  A pair's other channel is in the lane rot / 16 away (or in the
// same lane, `pairs`), the row's sum of squares in a 16-lane shuffle tree.
#include "sd_internal.cuh"

namespace sd {
namespace {

constexpr int kRpThreads = 256;
constexpr int kRpHalves = kRpThreads / 16;  // rows a CTA holds at a time
constexpr int kRpRows = 3;                  // rows of a lane in flight
constexpr int kRpTok = 4;                   // tokens per CTA where there are many

struct RpArgs {
  const uint16_t* q;
  uint16_t* qo;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* K;
  uint16_t* V;
  sd_strides qs, qos, ks, vs;
  const float* qw;
  const float* kw;
  const double* freq;
  float eps;
  int rot;
  int Hq, Hkv;       // heads present (0: that side is absent)
  int Hv, Hcache;    // value heads present; KV heads of the cache
  int64_t n, ncap, m, first;
  const int32_t* pos;
  const int32_t* length;
  const int32_t* rotary;
  int toks;          // tokens per CTA
  int heads_per;     // heads per CTA
  int64_t tiles;     // token tiles per sequence
};

__device__ __forceinline__ uint32_t rp_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// What a lane does with one row: where it comes from and goes to.
struct RpRow {
  const uint16_t* src;
  uint16_t* dst;
  const float* w;
  int tok;    // token of the CTA's tile; -1: no row
  int plain;  // a value row: copied
};

__device__ __forceinline__ RpRow rp_row(const RpArgs& a, int b, int64_t t0, int ntok, int h0,
                                        int nh, int i, int64_t cache0) {
  RpRow r;
  r.tok = -1;
  r.plain = 0;
  r.w = nullptr;
  r.src = nullptr;
  r.dst = nullptr;
  const int tok = i / nh, h = h0 + (i - tok * nh);
  if (tok >= ntok) return r;
  const int64_t t = t0 + tok;
  if (h < a.Hq) {
    r.src = a.q + b * a.qs.seq + h * a.qs.head + t * a.qs.token;
    r.dst = a.qo + b * a.qos.seq + h * a.qos.head + t * a.qos.token;
    r.w = a.qw;
    r.tok = tok;
    return r;
  }
  const int64_t at = cache0 + tok;
  if (at < 0 || at >= a.n) return r;
  const bool val = h >= a.Hq + a.Hkv;
  const int hk = h - a.Hq - (val ? a.Hkv : 0);
  const int64_t to = (((int64_t)b * a.Hcache + hk) * a.ncap + at) * kD;
  if (val) {
    r.src = a.v + b * a.vs.seq + hk * a.vs.head + t * a.vs.token;
    r.dst = a.V + to;
    r.plain = 1;
  } else {
    r.src = a.k + b * a.ks.seq + hk * a.ks.head + t * a.ks.token;
    r.dst = a.K + to;
    r.w = a.kw;
  }
  r.tok = tok;
  return r;
}

template <bool PAIRS>
__global__ void __launch_bounds__(kRpThreads) norm_rope_kernel(RpArgs a) {
  __shared__ float2 cs[kRpTok][kD / 2];  // cos, sin
  const int tid = threadIdx.x, lane16 = tid & 15, half = tid >> 4;
  const int b = (int)(blockIdx.x / a.tiles);
  const int64_t t0 = (blockIdx.x - b * a.tiles) * a.toks;
  const int64_t len = a.length ? imin64(a.m, a.length[b]) : a.m;
  const int ntok = (int)imin64(a.toks, len - t0);
  if (ntok <= 0) return;
  const int heads = a.Hq + a.Hkv + a.Hv;
  const int h0 = blockIdx.y * a.heads_per, nh = min(a.heads_per, heads - h0);
  const int64_t cache0 = a.first + (a.pos ? a.pos[b] : 0) + t0;
  const int rows = ntok * nh;

  RpRow r[kRpRows];
  uint4 x[kRpRows];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < kRpRows; ++u) {
      const int i = base + u * kRpHalves + half;
      r[u] = rp_row(a, b, t0, i < rows ? ntok : 0, h0, nh, i, cache0);
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r[u].tok >= 0) x[u] = *reinterpret_cast<const uint4*>(r[u].src + 8 * lane16);
    }
  };
  load(0);
  const int pairs = a.rot >> 1;
  for (int i = tid; i < ntok * pairs; i += kRpThreads) {
    const int tok = i / pairs, j = i - tok * pairs;
    const int64_t p = a.rotary ? (int64_t)a.rotary[b] + t0 + tok : cache0 + tok;
    // the angle in turns (1 / 2 pi), its whole turns dropped, all in 64 bits
    const double turns = (double)p * a.freq[j] * 0.15915494309189533577;
    const float half_turns = (float)(2.0 * (turns - rint(turns)));
    float s, c;
    sincospif(half_turns, &s, &c);
    cs[tok][j] = make_float2(c, s);
  }
  __syncthreads();

  const int c0 = 8 * lane16, hw = pairs >> 3;  // lanes to a pair's other channel
  const bool turned = c0 < a.rot;
  for (int base = 0;; ) {
#pragma unroll
    for (int u = 0; u < kRpRows; ++u) {
      float f[8];
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
      }
      if (__any_sync(0xFFFFFFFFu, r[u].w != nullptr)) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
        for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        if (r[u].w) {
          const float inv = rsqrtf(ss * (1.0f / kD) + a.eps);
          const float4 w0 = *reinterpret_cast<const float4*>(r[u].w + c0);
          const float4 w1 = *reinterpret_cast<const float4*>(r[u].w + c0 + 4);
          f[0] *= inv * w0.x, f[1] *= inv * w0.y, f[2] *= inv * w0.z, f[3] *= inv * w0.w;
          f[4] *= inv * w1.x, f[5] *= inv * w1.y, f[6] *= inv * w1.z, f[7] *= inv * w1.w;
        }
      }
      const int tok = max(r[u].tok, 0);
      if constexpr (PAIRS) {
        if (turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 e = cs[tok][(c0 >> 1) + i];
            const float p = f[2 * i], q = f[2 * i + 1];
            f[2 * i] = p * e.x - q * e.y;
            f[2 * i + 1] = q * e.x + p * e.y;
          }
        }
      } else if (a.rot) {
        const bool low = c0 < pairs;
        const int other = turned ? (low ? lane16 + hw : lane16 - hw) : lane16;
        const int j0 = low ? c0 : c0 - pairs;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_sync(0xFFFFFFFFu, f[i], other, 16);
          if (turned) {
            const float2 e = cs[tok][j0 + i];
            f[i] = f[i] * e.x + (low ? -o : o) * e.y;
          }
        }
      }
      if (r[u].tok >= 0) {
        const uint4 y = make_uint4(rp_pack(f[0], f[1]), rp_pack(f[2], f[3]),
                                   rp_pack(f[4], f[5]), rp_pack(f[6], f[7]));
        *reinterpret_cast<uint4*>(r[u].dst + c0) = r[u].plain ? x[u] : y;
      }
    }
    base += kRpRows * kRpHalves;
    if (base >= rows) break;
    load(base);
  }
}

}  // namespace

int launch_norm_rope(const Dims& s, const sd_rope& rope, const uint16_t* q, const sd_strides& qs,
                     uint16_t* qo, const sd_strides& qos, const uint16_t* k,
                     const sd_strides& ks, const uint16_t* v, const sd_strides& vs, uint16_t* K,
                     uint16_t* V, int64_t m, int64_t first, const int32_t* pos,
                     const int32_t* length, const int32_t* rotary, cudaStream_t st) {
  RpArgs a;
  a.q = q, a.qo = qo, a.k = k, a.v = v, a.K = K, a.V = V;
  a.qs = qs, a.qos = qos, a.ks = ks, a.vs = vs;
  a.qw = rope.q_weight, a.kw = rope.k_weight, a.freq = rope.inv_freq;
  a.eps = rope.eps, a.rot = rope.rot;
  a.Hq = q ? s.Hq : 0, a.Hkv = k ? s.Hkv : 0, a.Hv = v ? s.Hkv : 0, a.Hcache = s.Hkv;
  a.n = s.n, a.ncap = s.ncap, a.m = m, a.first = first;
  a.pos = pos, a.length = length, a.rotary = rotary;
  const int heads = a.Hq + a.Hkv + a.Hv;
  const int64_t sms = device_sm_count();
  // few tokens: one per CTA, its heads over several CTAs
  a.toks = (int64_t)s.B * m >= 4 * sms * kRpTok ? kRpTok : 1;
  a.tiles = (m + a.toks - 1) / a.toks;
  const int64_t ctas = a.tiles * s.B;
  if (ctas >= (int64_t)1 << 31)
    return fail(SD_ERR_UNSUPPORTED, "sd_qk_norm_rope: batch * m too large");
  a.heads_per = heads;
  if (a.toks == 1 && ctas < 2 * sms) a.heads_per = min(heads, kRpHalves);
  const dim3 grid((unsigned)ctas, (unsigned)((heads + a.heads_per - 1) / a.heads_per));
  if (rope.pairs)
    norm_rope_kernel<true><<<grid, kRpThreads, 0, st>>>(a);
  else
    norm_rope_kernel<false><<<grid, kRpThreads, 0, st>>>(a);
  note_launches(1);
  return check_launch("norm and rotation");
}

}  // namespace sd
