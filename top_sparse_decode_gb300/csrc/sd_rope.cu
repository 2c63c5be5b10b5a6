// Queries and keys normed per head and rotated by position on their way from the projection
// into q and the bf16 cache, values copied beside them (HashAttention: Semantic Sparsity for
// Faster Inference, 2.1: the q, k and v that the three stages start from).
//
//   y = x / sqrt(mean(x^2) + eps) * w,  (y_a, y_b) -> (y_a cos t - y_b sin t,
//   y_b cos t + y_a sin t),  t = position * inv_freq[j], pair j = (j, j + rot / 2) or
//   (2j, 2j + 1).
//
// Bound by HBM: every row is read and written once (512 bytes).  Sixteen lanes take a token
// and walk heads, 16 bytes of a row a lane, kRpRows rows in flight.  What depends on the
// token alone is formed once.  Its angles, since position * inv_freq reaches 10^6 radians as
// the fraction of a turn: a whole number of 2^-64 per position, times the position in 64-bit
// integers, which drop the whole turns by themselves (64-bit floats run at 2 a cycle and SM
// here); a thread forms a few of the CTA's, through shared memory.  And per channel the
// factors A = w cos t and B = -+ w' sin t, w' the pair's other weight, so that a row's channel
// is r (x A + x' B) with r the row's norm: the other channel x' comes as it was loaded, from
// the lane rot / 16 away or (`pairs`) from the same word.
//
// 4 x 32,768 tokens of 48 heads: 536 us, 6.0 TB/s, 89 % of the measured copy rate.  (With the
// angles in 64-bit floats 545.  With the angles read again and applied after the norm for
// every row the arithmetic was the bound: 1,064 us.)  Few tokens pay for it: their first rows
// are loaded behind the angles and two barriers, and queries, keys and values one after the
// other.  64 tokens of 48 heads take 5.9 us, 3 x 1,021 of 12 heads 10.8; the kernel of 1,064 us,
// whose first rows were in flight beside the angles, took 4.8 and 6.0.
#include "sd_internal.cuh"

namespace sd {
namespace {

constexpr int kRpThreads = 256;
constexpr int kRpTok = kRpThreads / 16;  // tokens per CTA
constexpr int kRpRows = 4;               // rows of a lane in flight

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
  int64_t n, ncap, first;
  uint32_t m;
  int64_t tokens;    // B * m
  const int32_t* pos;
  const int32_t* length;
  const int32_t* rotary;
  int heads_per;     // heads per CTA (of queries, then keys, then values)
};

__device__ __forceinline__ uint32_t rp_word(const uint4& x, int i) {
  return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
}

// Heads [h, end) of a token: rows at src + h * sstep to dst + h * dstep.
template <bool PAIRS, bool PLAIN>
__device__ __forceinline__ void rp_heads(const uint16_t* src, int64_t sstep, uint16_t* dst,
                                         int64_t dstep, int h, int end, bool on,
                                         const float (&A)[8], const float (&B)[8], bool norm,
                                         bool turned, int other, float eps) {
  uint4 x[kRpRows];
#pragma unroll
  for (int u = 0; u < kRpRows; ++u) {
    x[u] = make_uint4(0u, 0u, 0u, 0u);
    if (on && h + u < end) x[u] = *reinterpret_cast<const uint4*>(src + (h + u) * sstep);
  }
  for (; h < end; h += kRpRows) {
    uint4 next[kRpRows];
#pragma unroll
    for (int u = 0; u < kRpRows; ++u) {
      next[u] = make_uint4(0u, 0u, 0u, 0u);
      if (on && h + kRpRows + u < end)
        next[u] = *reinterpret_cast<const uint4*>(src + (h + kRpRows + u) * sstep);
    }
#pragma unroll
    for (int u = 0; u < kRpRows; ++u) {
      uint4 y = x[u];
      if (!PLAIN) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = bf16_lo(rp_word(x[u], i));
          f[2 * i + 1] = bf16_hi(rp_word(x[u], i));
        }
        float r = 1.0f;
        if (norm) {
          float ss = 0.0f, st = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            ss = fmaf(f[i], f[i], ss);
            st = fmaf(f[i + 1], f[i + 1], st);
          }
          ss += st;
#pragma unroll
          for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
          r = rsqrtf(ss * (1.0f / kD) + eps);
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t own = rp_word(x[u], i);
          const uint32_t o = PAIRS ? __byte_perm(own, own, 0x1032)
                                   : __shfl_sync(0xFFFFFFFFu, own, other, 16);
          float lo = f[2 * i] * A[2 * i], hi = f[2 * i + 1] * A[2 * i + 1];
          if (turned) {
            lo = fmaf(bf16_lo(o), B[2 * i], lo);
            hi = fmaf(bf16_hi(o), B[2 * i + 1], hi);
          }
          w[i] = bf16_pack(lo * r, hi * r);
        }
        y = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (on && h + u < end) *reinterpret_cast<uint4*>(dst + (h + u) * dstep) = y;
      x[u] = next[u];
    }
  }
}

template <bool PAIRS>
__global__ void __launch_bounds__(kRpThreads) norm_rope_kernel(RpArgs a) {
  __shared__ float2 cs[kRpTok][kD / 2];  // cos, sin
  __shared__ uint64_t turn[kD / 2];      // turns per position, their fraction in 2^-64
  const int tid = threadIdx.x, lane16 = tid & 15, slot = tid >> 4;
  const int64_t t_cta = (int64_t)blockIdx.x * kRpTok;
  const int pairs = a.rot >> 1;
  // the sequence and token of a place among the CTA's
  auto where = [&](int i, int& b, uint32_t& t) {
    const int64_t at = t_cta + i;
    if (at >= a.tokens) return false;
    b = a.tokens < ((int64_t)1 << 32) ? (int)((uint32_t)at / a.m) : (int)(at / a.m);
    t = (uint32_t)(at - (int64_t)b * a.m);
    return !a.length || (int64_t)t < a.length[b];
  };
  if (tid < pairs) {
    const double x = a.freq[tid] * 0.15915494309189533577;  // 1 / 2 pi
    turn[tid] = (uint64_t)__double2ll_rn((x - rint(x)) * 18446744073709551616.0);
  }
  __syncthreads();
  for (int i = tid; i < kRpTok * pairs; i += kRpThreads) {
    const int s = i / pairs, j = i - s * pairs;
    int b;
    uint32_t t;
    if (!where(s, b, t)) continue;
    const int64_t p = (a.rotary ? (int64_t)a.rotary[b] : a.first + (a.pos ? a.pos[b] : 0)) + t;
    // whole turns drop out of the product's upper half
    const float half_turns = (float)(int64_t)((uint64_t)p * turn[j]) * 0x1p-63f;
    float s0, c0;
    sincospif(half_turns, &s0, &c0);
    cs[s][j] = make_float2(c0, s0);
  }
  __syncthreads();

  int b = 0;
  uint32_t t = 0;
  const bool on = where(slot, b, t);
  const int c0 = 8 * lane16;
  const bool turned = c0 < a.rot, low = c0 < pairs;
  const int other = !turned ? lane16 : low ? lane16 + (pairs >> 3) : lane16 - (pairs >> 3);
  const int h0 = blockIdx.y * a.heads_per;
  const int h1 = min(h0 + a.heads_per, a.Hq + a.Hkv + a.Hv);
  const int64_t at = a.first + (a.pos ? a.pos[b] : 0) + t;
  const bool in = on && at >= 0 && at < a.n;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {  // queries, keys
    const int s0 = side ? a.Hq : 0, s1 = side ? a.Hq + a.Hkv : a.Hq;
    const int lo = max(h0, s0) - s0, hi = min(h1, s1) - s0;
    if (lo >= hi) continue;
    const float* w = side ? a.kw : a.qw;
    float A[8], B[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      A[i] = w ? w[c0 + i] : 1.0f;
      B[i] = 0.0f;
      if (turned) {
        const float2 e = cs[slot][PAIRS ? (c0 + i) >> 1 : (low ? c0 : c0 - pairs) + i];
        const float wo = w ? w[PAIRS ? c0 + (i ^ 1) : 8 * other + i] : 1.0f;
        const bool first = PAIRS ? !(i & 1) : low;
        B[i] = (first ? -wo : wo) * e.y;
        A[i] *= e.x;
      }
    }
    const uint16_t* src = side ? a.k + b * a.ks.seq + t * a.ks.token
                               : a.q + b * a.qs.seq + t * a.qs.token;
    uint16_t* dst = side ? a.K + ((int64_t)b * a.Hcache * a.ncap + at) * kD
                         : a.qo + b * a.qos.seq + t * a.qos.token;
    rp_heads<PAIRS, false>(src + c0, side ? a.ks.head : a.qs.head, dst + c0,
                           side ? a.ncap * kD : a.qos.head, lo, hi, side ? in : on, A, B,
                           w != nullptr, turned, other, a.eps);
  }
  const int s0 = a.Hq + a.Hkv;
  const int lo = max(h0, s0) - s0, hi = min(h1, s0 + a.Hv) - s0;
  if (lo < hi) {
    const float none[8] = {};
    rp_heads<PAIRS, true>(a.v + b * a.vs.seq + t * a.vs.token + c0, a.vs.head,
                          a.V + ((int64_t)b * a.Hcache * a.ncap + at) * kD + c0, a.ncap * kD, lo,
                          hi, in, none, none, false, false, lane16, a.eps);
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
  a.n = s.n, a.ncap = s.ncap, a.m = (uint32_t)m, a.first = first;
  a.pos = pos, a.length = length, a.rotary = rotary;
  a.tokens = (int64_t)s.B * m;
  const int heads = a.Hq + a.Hkv + a.Hv;
  const int64_t ctas = (a.tokens + kRpTok - 1) / kRpTok;
  if (ctas >= (int64_t)1 << 31)
    return fail(SD_ERR_UNSUPPORTED, "sd_qk_norm_rope: batch * m too large");
  // few tokens: their heads over several CTAs, down to one round of rows, as long as each of
  // the GPU's SMs has room for them (four CTAs)
  const int64_t want = imax64(1, 4 * (int64_t)device_sm_count() / ctas);
  const int64_t rounds = (heads + kRpRows - 1) / kRpRows;
  a.heads_per = (int)((rounds + imin64(rounds, want) - 1) / imin64(rounds, want)) * kRpRows;
  a.heads_per = max(a.heads_per, (heads + 65534) / 65535);  // a grid's second extent
  const dim3 grid((unsigned)ctas, (unsigned)((heads + a.heads_per - 1) / a.heads_per));
  if (rope.pairs)
    norm_rope_kernel<true><<<grid, kRpThreads, 0, st>>>(a);
  else
    norm_rope_kernel<false><<<grid, kRpThreads, 0, st>>>(a);
  note_launches(1);
  return check_launch("norm and rotation");
}

}  // namespace sd
