// Decode attention over the 4-bit K/V cache (HashAttention: Semantic Sparsity for Faster
// Inference, 2.1): z_i = scale <q, k_i>, o = sum e^{z_i - m} v_i / sum e^{z_i - m}, over a
// range of each sequence's tokens or over selected ones (2.5, rows read in place).
//
// With k_ij = c_ij s_ig + m_ig (g = the group of channel j):
//   z_i = scale sum_g [ s_ig sum_{j in g} q_j c_ij + m_ig sum_{j in g} q_j ]
//   o_j = [ sum_i (p_i s_ig) c_ij + sum_i p_i m_ig ] / sum_i p_i
// so the codes are only ever multiplied as whole numbers, by the tensor cores, and scales
// and minima enter once per token and group, in fp32.
//  * A code needs no conversion: the four bits, masked in place, are an f16 subnormal c
//    2^-24 (bits 0..3 of a half-word) or 16 c 2^-24 (bits 4..7), both exact.  The 16 goes
//    into q (QK^T) and into the outputs at the end (PV).
//  * z: S = K q^T, m16n8k16 with 16 tokens as rows and the heads as columns: 8 MMAs per 16
//    tokens.  q is scaled by a power of two per head to f16; bf16 values stay exact
//    unless they are 2^-36 below the head's largest.
//  * PV: O^T = V^T P^T, 16 channels as rows, heads as columns, 16 tokens deep.  w = p s f is
//    split in two f16 parts (22 bits; f a power of two per head and group that holds the
//    largest w in [2^7, 2^14], raised and lowered as an online softmax moves its
//    maximum).  With G <= 4 the columns 4..7 repeat the heads and take the low parts (8
//    MMAs per 16 tokens), with G = 8 the low parts are 8 more.
//  * p = 2^(z log2 e - m); m, a whole number per head, is raised only when a logit
//    exceeds it by 8.
//
// Each warp pulls 16-token tiles (2,304 bytes) through a ring of its own in shared memory
// with 16-byte asynchronous copies; rows are swizzled there so that both operands read
// without bank conflicts.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "sd_internal.cuh"
#include "sd_kv4.cuh"
#include "sd_mma.cuh"

namespace sd {
namespace {

namespace cg = cooperative_groups;

constexpr int kKaTile = 16;    // tokens per tile
constexpr int kKaWarps = 8;    // warps per CTA
constexpr int kKaThreads = 32 * kKaWarps;
constexpr int kKaDepth = 5;    // tiles in a warp's ring
constexpr int kKaOffV = kKaTile * kKv4Row, kKaOffS = 2 * kKaOffV;
constexpr int kKaOffMask = kKaOffS + kKaTile * 2 * kKv4Scales;
constexpr int kKaStage = kKaOffMask + 16;
constexpr int kKaRing = kKaDepth * kKaStage;
constexpr float kKaLog2e = 1.4426950408889634f;
constexpr float kKaLn2 = 0.6931471805599453f;
constexpr float kKaEmpty = -1e30f;   // m before the first token
constexpr float kKaSlack = 8.0f;     // log2 headroom of p over m
constexpr float kKaWMax = 16384.0f;  // largest w that is not rescaled
constexpr float kKaF0 = 1.2676506e30f;  // 2^100: f before the first token, and its limit

struct KaArgs {
  const uint16_t* q;
  sd_kv4 c;
  const int32_t* idx;
  int64_t idx_stride;
  const int32_t* count;
  int max_count;
  const int32_t* begin;
  const int32_t* end;
  int Hq, Hkv;
  int n;
  int64_t ncap, rows;
  float scale;
  float* out;
  float* lse;
  uint32_t* ticket;  // [rows], zero at launch (balanced kernel)
  float* part_o;     // [2 CTAs][G][kD]
  float2* part_ml;   // [2 CTAs][G]
};

// Tokens of a row: positions [t0, t0 + len) of the sequence, or len entries of idx.
struct KaRow {
  int t0, len;
};
template <bool GATHER>
__device__ __forceinline__ KaRow ka_row(const KaArgs& a, int64_t row, int b) {
  KaRow r;
  if (GATHER) {
    r.t0 = 0;
    r.len = max(min(__ldg(a.count + row), a.max_count), 0);
  } else {
    r.t0 = a.begin ? max(__ldg(a.begin + b), 0) : 0;
    const int e = a.end ? min(__ldg(a.end + b), a.n) : a.n;
    r.len = e > r.t0 ? e - r.t0 : 0;
  }
  return r;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes into shared memory; zeros where v is false.
__device__ __forceinline__ void ka_copy16(uint32_t dst, const void* src, bool v) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
               "r"(v ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ka_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ka_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(a)
               : "memory");
  return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 x;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(x.x), "=r"(x.y) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(x) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ float ka_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// Requests tile `tile` of a row into a stage.  Lane l copies chunk l % 4 of the rows of
// tokens l / 4 and l / 4 + 8 (chunks swizzled by 2 where the token's bit 1 is set) and,
// below 16, the scale record of token l.  Tokens past the row, and indices outside [0,
// n), become zeros; the stage's mask lists the others.
template <bool GATHER>
__device__ __forceinline__ void ka_issue(const KaArgs& a, uint32_t stage, int64_t row,
                                         const KaRow& r, int tile, int lane) {
  const int p = tile * kKaTile + (lane & 15);
  bool ok = p < r.len;
  int tok = 0;
  if (GATHER) {
    if (ok) tok = __ldg(a.idx + row * a.idx_stride + p);
    ok = ok && tok >= 0 && tok < a.n;
    if (!ok) tok = 0;
  } else if (ok) {
    tok = r.t0 + p;
  }
  const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok) & 0xFFFFu;
  const int64_t base = row * a.ncap;
  const int tl = lane >> 2, ch = lane & 3;
  const uint32_t dst = stage + tl * kKv4Row + ((ch ^ (lane >> 2 & 2)) * 16);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = __shfl_sync(0xFFFFFFFFu, tok, tl + 8 * h);
    const bool v = mask >> (tl + 8 * h) & 1u;
    const int64_t off = (base + t) * kKv4Row + ch * 16;
    ka_copy16(dst + h * 8 * kKv4Row, a.c.k + off, v);
    ka_copy16(dst + h * 8 * kKv4Row + kKaOffV, a.c.v + off, v);
  }
  if (lane < kKaTile)
    ka_copy16(stage + kKaOffS + lane * 16, a.c.scale + (base + tok) * kKv4Scales, ok);
  if (lane == 0) sts32(stage + kKaOffMask, mask);
}

// q as the B operand, and per-head constants of the lane's two columns (heads).
struct KaQ {
  uint32_t b[2][4][2];  // [group][k-step][half]
  float ch[2];          // scale log2(e) 2^24 / (q's power of two)
  float qs[2][2];       // [column][group]: scale log2(e) sum of the group's q
};

// The head of column c (c < 8); with G <= 4 columns 4..7 repeat 0..3.
template <int G>
__device__ __forceinline__ int ka_head(int c) {
  return G == 8 ? c : c & 3;
}

template <int G>
__device__ __forceinline__ void ka_load_q(KaQ& Q, const KaArgs& a, int64_t row, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
  const int b = (int)(row / a.Hkv), h = (int)(row % a.Hkv), hd = ka_head<G>(gid);
  const bool real = hd < G;
  const uint16_t* qr = a.q + ((int64_t)b * a.Hq + h * G + (real ? hd : 0)) * kD;
  uint4 w[2][2];
  float top = 0.0f, sum[2] = {0.0f, 0.0f};
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[g][j] = *reinterpret_cast<const uint4*>(qr + 64 * g + 16 * tig + 8 * j);
      if (!real) w[g][j] = make_uint4(0u, 0u, 0u, 0u);
      const uint32_t x[4] = {w[g][j].x, w[g][j].y, w[g][j].z, w[g][j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top = fmaxf(top, fmaxf(fabsf(bf16_lo(x[i])), fabsf(bf16_hi(x[i]))));
        sum[g] += bf16_lo(x[i]) + bf16_hi(x[i]);
      }
    }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    sum[0] += __shfl_xor_sync(0xFFFFFFFFu, sum[0], o);
    sum[1] += __shfl_xor_sync(0xFFFFFFFFu, sum[1], o);
  }
  // 2^k q has its largest value in [2^14, 2^15) (k at most 120: smaller heads are 0 to
  // any cache)
  const int k = top > 0.0f ? min(14 - ((int)(__float_as_uint(top) >> 23) - 127), 120) : 0;
  const float up = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // word 4 tig + 2 j + g: nibbles i and i + 4 of a half-word pair, i = 0..3
      const uint32_t x[4] = {w[g][j].x, w[g][j].y, w[g][j].z, w[g][j].w};
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(x[i]) * up;
        f[2 * i + 1] = bf16_hi(x[i]) * up;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const __half2 lo = __floats2half2_rn(f[2 * s], f[2 * s + 4]);
        const __half2 hi = __floats2half2_rn(f[2 * s + 1] * 0.0625f, f[2 * s + 5] * 0.0625f);
        Q.b[g][2 * j + s][0] = *reinterpret_cast<const uint32_t*>(&lo);
        Q.b[g][2 * j + s][1] = *reinterpret_cast<const uint32_t*>(&hi);
      }
    }
  const float sl = a.scale * kKaLog2e;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int src = 4 * (2 * tig + e);  // a lane that loaded the column's head
    const int kc = __shfl_sync(0xFFFFFFFFu, k, src);
    Q.ch[e] = sl * __uint_as_float((uint32_t)(127 + 24 - kc) << 23);
    Q.qs[e][0] = sl * __shfl_sync(0xFFFFFFFFu, sum[0], src);
    Q.qs[e][1] = sl * __shfl_sync(0xFFFFFFFFu, sum[1], src);
  }
}

// A warp's online softmax.  o: O^T in units of 2^-24 / f (odd channels 16 times that);
// tile 4 g + u holds channels 64 g + 8 gid + 2 u (o[..][e]) and + 1 (o[..][2 + e]) of
// columns 2 tig + e.  l, mo: this lane's tokens only.
struct KaState {
  float o[8][4];
  float m[2], l[2];
  float f[2][2], mo[2][2];  // [column][group]
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[t][i] = 0.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[e] = kKaEmpty;
      l[e] = 0.0f;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        f[e][g] = kKaF0;
        mo[e][g] = 0.0f;
      }
    }
  }
};

// The largest x over the lanes that hold the same columns.
__device__ __forceinline__ float ka_col_max(float x) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

// Raises the columns' m where a logit exceeds it by more than the slack.
__device__ __forceinline__ void ka_raise_m(KaState& S, const float (&z)[2][2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float top = ka_col_max(fmaxf(z[0][e], z[1][e]));
    if (!(top > S.m[e] + kKaSlack)) continue;  // uniform over the column's lanes
    const float up = ceilf(top), d = up - S.m[e], al = ka_exp2(-d);
    S.m[e] = up;
    S.l[e] *= al;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      S.mo[e][g] *= al;
      // what was summed weighs 2^-d now: f takes up the factor, o stays, up to f's limit
      const float fn = fminf(S.f[e][g] * ka_exp2(fminf(d, 126.0f)), kKaF0);
      const float r = (fn / S.f[e][g]) * al;
      S.f[e][g] = fn;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        S.o[4 * g + u][e] *= r;
        S.o[4 * g + u][2 + e] *= r;
      }
    }
  }
}

// Lowers f where p s f exceeds kKaWMax, to bring the largest to [2^7, 2^8).
__device__ __forceinline__ void ka_lower_f(KaState& S, const float (&p)[2][2],
                                        const float (&sv)[2][2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float top = ka_col_max(fmaxf(p[0][e] * sv[0][g], p[1][e] * sv[1][g]));
      if (!(top * S.f[e][g] > kKaWMax) || !(top < INFINITY)) continue;
      const int ex = (int)(__float_as_uint(top) >> 23) - 127;  // top >= 2^-86: normal
      const float fn = __uint_as_float((uint32_t)(127 + max(7 - ex, -126)) << 23);
      const float r = fn / S.f[e][g];
      S.f[e][g] = fn;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        S.o[4 * g + u][e] *= r;
        S.o[4 * g + u][2 + e] *= r;
      }
    }
}

__device__ __forceinline__ uint32_t ka_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// One 16-token tile.  Row r of the score tile is token tau(r) (r < 8: r / 2, odd rows 4 +
// (r / 2 ^ 1)) or tau(r - 8) + 8: with the swizzle, any eight lanes of a K read and any
// sixteen of a V read touch each bank once.
template <int G>
__device__ __forceinline__ void ka_tile(KaState& S, const KaQ& Q, uint32_t st, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
  const int tk = (gid & 1) ? 4 + (gid >> 1 ^ 1) : gid >> 1;
  const uint32_t ak = st + tk * kKv4Row + ((tig ^ (gid >> 1 & 2)) * 16);
  const uint4 ka = lds128(ak), kb = lds128(ak + 8 * kKv4Row);
  const uint32_t as = st + kKaOffS + tk * 16;
  const uint4 sa = lds128(as), sb = lds128(as + 8 * 16);
  const uint32_t mask = lds32(st + kKaOffMask);
  const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
  constexpr uint32_t kLo = 0x000F000Fu, kHi = 0x00F000F0u;
  float acc[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t xa = wa[2 * j + g] >> (8 * s), xb = wb[2 * j + g] >> (8 * s);
        mma_f16(acc[g], xa & kLo, xb & kLo, xa & kHi, xb & kHi, Q.b[g][2 * j + s][0],
                Q.b[g][2 * j + s][1]);
      }
  float z[2][2], sv[2][2], mv[2][2];
  {
    const uint4 sc[2] = {sa, sb};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float s0 = bf16_lo(sc[r].x), m0 = bf16_hi(sc[r].x);
      const float s1 = bf16_lo(sc[r].y), m1 = bf16_hi(sc[r].y);
      sv[r][0] = bf16_lo(sc[r].z);
      mv[r][0] = bf16_hi(sc[r].z);
      sv[r][1] = bf16_lo(sc[r].w);
      mv[r][1] = bf16_hi(sc[r].w);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        z[r][e] = fmaf(fmaf(s1, acc[1][2 * r + e], s0 * acc[0][2 * r + e]), Q.ch[e],
                       fmaf(m1, Q.qs[e][1], m0 * Q.qs[e][0]));
    }
  }
  if (mask != 0xFFFFu) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (!(mask >> (tk + 8 * r) & 1u)) z[r][0] = z[r][1] = -INFINITY;
  }
  const bool raise = fmaxf(z[0][0], z[1][0]) > S.m[0] + kKaSlack ||
                     fmaxf(z[0][1], z[1][1]) > S.m[1] + kKaSlack;
  if (__any_sync(0xFFFFFFFFu, raise)) ka_raise_m(S, z);
  float p[2][2], w[2][2][2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    p[0][e] = ka_exp2(z[0][e] - S.m[e]);
    p[1][e] = ka_exp2(z[1][e] - S.m[e]);
    S.l[e] += p[0][e] + p[1][e];
#pragma unroll
    for (int g = 0; g < 2; ++g)
      S.mo[e][g] = fmaf(p[1][e], mv[1][g], fmaf(p[0][e], mv[0][g], S.mo[e][g]));
  }
  float top = 0.0f;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        w[r][e][g] = p[r][e] * (sv[r][g] * S.f[e][g]);
        top = fmaxf(top, w[r][e][g]);
      }
  if (__any_sync(0xFFFFFFFFu, top > kKaWMax)) {
    ka_lower_f(S, p, sv);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int g = 0; g < 2; ++g) w[r][e][g] = p[r][e] * (sv[r][g] * S.f[e][g]);
  }
  // P^T's high and low f16 parts, as B operands
  uint32_t bh[2][2], bl[2][2];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t hi = ka_pack(w[r][0][g], w[r][1][g]);
      const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      const uint32_t lo = ka_pack(w[r][0][g] - hf.x, w[r][1][g] - hf.y);
      if (G == 8) {
        bh[g][r] = transpose_8x8(hi);
        bl[g][r] = transpose_8x8(lo);
      } else {
        bh[g][r] = transpose_8x8(tig < 2 ? hi : lo);
      }
    }
  // rows 2 tig, 2 tig + 1 (and + 8) of V, 8 bytes from byte 8 gid: channels 8 gid .. + 7 of
  // either group
  const uint32_t av = st + kKaOffV + ((gid >> 1 ^ (tig & 2)) * 16) + (gid & 1) * 8;
  const uint2 v0 = lds64(av + tig * kKv4Row), v1 = lds64(av + (4 + (tig ^ 1)) * kKv4Row);
  const uint2 v2 = lds64(av + (tig + 8) * kKv4Row), v3 = lds64(av + (12 + (tig ^ 1)) * kKv4Row);
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint32_t w0 = g ? v0.y : v0.x, w1 = g ? v1.y : v1.x;
    const uint32_t w2 = g ? v2.y : v2.x, w3 = g ? v3.y : v3.x;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t sel = u < 2 ? 0x5410u : 0x7632u;
      const uint32_t x = __byte_perm(w0, w1, sel) >> (8 * (u & 1));
      const uint32_t y = __byte_perm(w2, w3, sel) >> (8 * (u & 1));
      mma_f16(S.o[4 * g + u], x & kLo, x & kHi, y & kLo, y & kHi, bh[g][0], bh[g][1]);
      if (G == 8)
        mma_f16(S.o[4 * g + u], x & kLo, x & kHi, y & kLo, y & kHi, bl[g][0], bl[g][1]);
    }
  }
}

// The state of a warp in natural units, written to so [G][kD] and sml [G] = (m, l).
template <int G>
__device__ __forceinline__ void ka_flush(KaState& S, float* so, float2* sml, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      S.l[e] += __shfl_xor_sync(0xFFFFFFFFu, S.l[e], o);
      S.mo[e][0] += __shfl_xor_sync(0xFFFFFFFFu, S.mo[e][0], o);
      S.mo[e][1] += __shfl_xor_sync(0xFFFFFFFFu, S.mo[e][1], o);
    }
    const int c = 2 * tig + e, hd = ka_head<G>(c);
    const bool mine = c < G;
    if (mine && gid == 0) sml[hd] = make_float2(S.m[e], S.l[e]);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float k = 16777216.0f / S.f[e][g];
      float x[8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float even = S.o[4 * g + u][e], odd = S.o[4 * g + u][2 + e];
        if (G != 8) {  // the low parts' columns
          even += __shfl_xor_sync(0xFFFFFFFFu, even, 2);
          odd += __shfl_xor_sync(0xFFFFFFFFu, odd, 2);
        }
        x[2 * u] = fmaf(even, k, S.mo[e][g]);
        x[2 * u + 1] = fmaf(odd, k * 0.0625f, S.mo[e][g]);
      }
      if (mine) {
        float4* d = reinterpret_cast<float4*>(so + hd * kD + 64 * g + 8 * gid);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
      }
    }
  }
}

// e^(m - top) in log2 units for a state of sum l (0 for an empty one).
__device__ __forceinline__ float ka_weight(float2 ml, float top) {
  return ml.y == 0.0f ? 0.0f : exp2f(ml.x - top);
}

__device__ __forceinline__ void ka_write(const KaArgs& a, int64_t bq, int j, float o, float m,
                                         float l) {
  a.out[bq * kD + j] = l != 0.0f ? o / l : 0.0f;  // an empty row gives 0
  if (a.lse && j == 0) a.lse[bq] = l != 0.0f ? (m + log2f(l)) * kKaLn2 : -INFINITY;
}

// A few rows: one cluster of CTAs per row, tiles dealt to its warps in turn, the states
// joined through shared and distributed shared memory.
template <int G, bool GATHER>
__global__ void __launch_bounds__(kKaThreads, 2) kv4_cluster_kernel(const KaArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), CS = (int)cl.num_blocks();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.y;
  const int b = (int)(row / a.Hkv), h = (int)(row % a.Hkv);
  const KaRow r = ka_row<GATHER>(a, row, b);
  const int tiles = (r.len + kKaTile - 1) / kKaTile, step = CS * kKaWarps;
  const uint32_t ring = smem_addr(smem) + warp * kKaRing;
  int next = rank * kKaWarps + warp;
#pragma unroll
  for (int d = 0; d < kKaDepth - 1; ++d) {
    if (next < tiles) ka_issue<GATHER>(a, ring + d * kKaStage, row, r, next, lane);
    ka_commit();
    next += step;
  }
  KaQ Q;
  ka_load_q<G>(Q, a, row, lane);
  KaState S;
  S.clear();
  uint32_t slot = 0;
  for (int t = rank * kKaWarps + warp; t < tiles; t += step) {
    const uint32_t put = slot == 0 ? (kKaDepth - 1) * kKaStage : slot - kKaStage;
    if (next < tiles) ka_issue<GATHER>(a, ring + put, row, r, next, lane);
    ka_commit();
    next += step;
    ka_wait<kKaDepth - 1>();
    __syncwarp();
    ka_tile<G>(S, Q, ring + slot, lane);
    __syncwarp();
    slot = slot == (kKaDepth - 1) * kKaStage ? 0 : slot + kKaStage;
  }
  ka_wait<0>();
  __syncthreads();  // the rings become the warps' states
  float* so = reinterpret_cast<float*>(smem);             // [warps][G][kD]
  float2* sml = reinterpret_cast<float2*>(so + kKaWarps * G * kD);  // [warps][G]
  float* co = reinterpret_cast<float*>(sml + kKaWarps * G);  // the CTA's: [G][kD]
  float2* cml = reinterpret_cast<float2*>(co + G * kD);      // [G]
  ka_flush<G>(S, so + warp * G * kD, sml + warp * G, lane);
  __syncthreads();
  for (int e = threadIdx.x; e < G * kD; e += kKaThreads) {
    const int g = e / kD;
    float top = kKaEmpty, l = 0.0f, o = 0.0f;
#pragma unroll
    for (int w = 0; w < kKaWarps; ++w) top = fmaxf(top, sml[w * G + g].x);
#pragma unroll
    for (int w = 0; w < kKaWarps; ++w) {
      const float f = ka_weight(sml[w * G + g], top);
      l = fmaf(sml[w * G + g].y, f, l);
      o = fmaf(so[w * G * kD + e], f, o);
    }
    if (CS == 1) {
      ka_write(a, (int64_t)b * a.Hq + h * G + g, e % kD, o, top, l);
    } else {
      co[e] = o;
      if (e % kD == 0) cml[g] = make_float2(top, l);
    }
  }
  if (CS == 1) return;
  cl.sync();
  const int per = G * kD / CS;
  for (int e = rank * per + threadIdx.x; e < (rank + 1) * per; e += kKaThreads) {
    const int g = e / kD;
    float top = kKaEmpty, l = 0.0f, o = 0.0f;
    for (int c = 0; c < CS; ++c) top = fmaxf(top, cl.map_shared_rank(cml, c)[g].x);
    for (int c = 0; c < CS; ++c) {
      const float2 ml = cl.map_shared_rank(cml, c)[g];
      const float f = ka_weight(ml, top);
      l = fmaf(ml.y, f, l);
      o = fmaf(cl.map_shared_rank(co, c)[e], f, o);
    }
    ka_write(a, (int64_t)b * a.Hq + h * G + g, e % kD, o, top, l);
  }
  cl.sync();  // every CTA's state stays alive until the others have read it
}

template <int G, bool GATHER>
int ka_launch(const Dims& s, const KaArgs& a, int64_t most, cudaStream_t st) {
  const int64_t tiles = (most + kKaTile - 1) / kKaTile;
  int cs = 1;
  while (cs < 8 && a.rows * cs * 2 <= 2 * device_sm_count() && cs * 2 * kKaWarps <= tiles) cs *= 2;
  const size_t bytes = (size_t)kKaWarps * kKaRing;
  auto kern = kv4_cluster_kernel<G, GATHER>;
  if (int rc = set_smem_limit((const void*)kern, bytes, "kv4 attend")) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs, (unsigned)a.rows, 1);
  cfg.blockDim = dim3(kKaThreads, 1, 1);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return check_launch("kv4 attend");
  note_launches(1);
  return check_launch("kv4 attend");
}

template <int G>
int ka_pick(const Dims& s, const KaArgs& a, int64_t most, cudaStream_t st) {
  return a.idx ? ka_launch<G, true>(s, a, most, st) : ka_launch<G, false>(s, a, most, st);
}

}  // namespace

size_t kv4_attend_workspace_bytes(const Dims&, int64_t) { return 16; }

int launch_kv4_attend(const Dims& s, const uint16_t* q, const sd_kv4& c, const int32_t* idx,
                      int64_t idx_stride, const int32_t* count, int64_t max_count,
                      const int32_t* begin, const int32_t* end, float scale, float* out,
                      float* lse, void* ws, cudaStream_t st) {
  KaArgs a = {};
  a.q = q;
  a.c = c;
  a.idx = idx;
  a.idx_stride = idx_stride;
  a.count = count;
  a.max_count = (int)max_count;
  a.begin = begin;
  a.end = end;
  a.Hq = s.Hq;
  a.Hkv = s.Hkv;
  a.n = (int)s.n;
  a.ncap = s.ncap;
  a.rows = (int64_t)s.B * s.Hkv;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  const int64_t most = idx ? max_count : s.n;
  switch (s.G) {
    case 1: return ka_pick<1>(s, a, most, st);
    case 2: return ka_pick<2>(s, a, most, st);
    case 4: return ka_pick<4>(s, a, most, st);
    default: return ka_pick<8>(s, a, most, st);
  }
}

}  // namespace sd
