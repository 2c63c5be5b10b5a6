// Decode attention over the 4-bit K/V cache (HashAttention: Semantic Sparsity for Faster
// Inference, 2.1): z_i = scale <q, k_i>, o = sum e^{z_i - m} v_i / sum e^{z_i - m}, over a
// range of each sequence's tokens or over selected ones (2.5, rows read in place).
//
// With k_ij = c_ij s_ig + m_ig and v_ij = (c_ij - 7.5) s_ig + m'_ig (g = the group of channel
// j, m' = m + 7.5 s the middle of its range):
//   z_i = scale sum_g [ s_ig sum_{j in g} q_j c_ij + m_ig sum_{j in g} q_j ]
//   o_j = [ sum_i (p_i s_ig) (c_ij - 7.5) + sum_i p_i m'_ig ] / sum_i p_i
// so only codes are multiplied by the tensor cores, as small whole (or half) numbers, and
// scales and minima enter once per token and group, in fp32.  Both sums of o are of numbers
// that change sign: with c in place of c - 7.5 they would be large and cancel.
//  * A code becomes an f16 number by a mask and one multiplication (ka_code_lo).
//  * z: S = K q^T, m16n8k16 with 16 tokens as rows and the heads as columns: 8 MMAs per 16
//    tokens.  q is scaled by a power of two per head to f16; bf16 values stay exact
//    unless they are 2^-32 below the head's largest.
//  * PV: O^T = V^T P^T, 16 channels as rows, heads as columns, 16 tokens deep.  w = p s f is
//    split in two f16 parts (22 bits: one rounding to 11 would cost 2^-12 of an output; f
//    a power of two per head and group that holds the largest w in [2^7, 2^14], raised and
//    lowered as an online softmax moves its maximum).  22 bits hold down to 2^-10 of the
//    largest w that the warp has met; below, a w is off by at most 2^-25, 2^-32 of that one,
//    so that a tail of many small weights is off by 2^-32 per token of the warp, where its
//    sum in fp32 may be by 2^-27 (chains of an eighth of the tokens).  With G <= 4 columns
//    0..3 take the high parts and 4..7 the low ones (8 MMAs per 16 tokens), with G = 8 the
//    low parts are 8 more.
//  * p = 2^(z log2 e - m); m, a whole number per head, is raised only when weights
//    exceed 2^8 or so.
//
// Each warp pulls 32-token tiles (4,608 bytes) through a ring of its own in shared memory
// with 16-byte asynchronous copies; rows are swizzled there so that both operands read
// without bank conflicts.  No warp waits for another while it works.
//
// What bounds it: 144 bytes a token and KV head from HBM are 397 cycles of an SM's four
// schedulers per 16 tokens at the measured copy rate; the work on them is ~307
// instructions (G <= 4; 360 with G = 8), half of them integer operations that issue every
// second cycle: ~88 to take the codes apart, 64 to scale and centre them, 16 (24) MMAs of
// 8.4 cycles.  It runs at ~420 cycles (G <= 4).  Measured (GB300): 8 KV heads of 1,048,576
// tokens, G = 4: 199 us, 6.1 TB/s, 89 % of the copy rate; 512 of 16,384, G = 8: 244 us, 5.0
// TB/s.  Tried on the former and slower: six warps a CTA (their 168 registers spill; 5 us
// more), scores of the next tile beside the values of this one (14), e4m3 MMAs for the
// scores (converted to f16 by the compiler on this GPU; 35), the upper codes of a word taken
// down by an integer multiplication instead of a shift (24), three CTAs an SM with scale
// records read twice to save registers (10).  Subnormal codes without the multiplication and
// one running sum on the tensor cores were no faster and took outputs off by up to 1e-2 of
// themselves.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "sd_internal.cuh"
#include "sd_kv4.cuh"
#include "sd_kv4_plan.cuh"
#include "sd_mma.cuh"

namespace sd {
namespace {

namespace cg = cooperative_groups;

constexpr int kKaThreads = 32 * kKaWarps;
constexpr int kKaOffV = kKaTile * kKv4Row, kKaOffS = 2 * kKaOffV;
constexpr int kKaOffMask = kKaOffS + kKaTile * 2 * kKv4Scales;
constexpr int kKaOffQ = kKaOffMask + 16;  // the row's queries, where the tile is its first
template <int G>
constexpr int kKaStage = kKaOffQ + G * kD * 2;
// Tiles in a warp's ring (G = 4: 204 us with 3 when it was 211 with 4, on the longest case
// above; G = 8: 257 and 252).
template <int G>
constexpr int kKaDepth = G == 8 ? 4 : 3;
template <int G>
constexpr int kKaRing = kKaDepth<G> * kKaStage<G>;
constexpr float kKaLog2e = 1.4426950408889634f;
constexpr float kKaLn2 = 0.6931471805599453f;
constexpr float kKaEmpty = -3e38f;   // m before the first token
constexpr float kKaPMax = 512.0f;    // largest sum of a lane's p that leaves m as it is
constexpr float kKaWMax = 16384.0f;  // largest w that leaves f as it is (0x7400 in f16)
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
  int2* meta;       // [rows]: the first warp that holds tiles of the row and how many do
  float* part_o;    // [2 warps][G][kD]
  float2* part_ml;  // [2 warps][G]
};

// Tokens of a row: positions [t0, t0 + len) of the sequence, or len entries of idx.
struct KaRow {
  int t0, len;
};
// An ordinary load of a count, a range or an index: a kernel that is launched early lives
// while the one before it may still write them, so a read-only load (of data that do not
// change while its kernel lives) is not for them.  volatile keeps it behind the wait; the
// compiler may move the others past it, as it may not past a plain load here (199 us; 203
// with *p or __ldcg, 8 KV heads of 1,048,576 tokens).
__device__ __forceinline__ int ka_load(const int32_t* p) {
  int x;
  asm volatile("ld.global.s32 %0, [%1];\n" : "=r"(x) : "l"(p));
  return x;
}
template <bool GATHER>
__device__ __forceinline__ KaRow ka_row(const KaArgs& a, int64_t row, int b) {
  KaRow r;
  if (GATHER) {
    r.t0 = 0;
    r.len = max(min(ka_load(a.count + row), a.max_count), 0);
  } else {
    r.t0 = a.begin ? max(ka_load(a.begin + b), 0) : 0;
    const int e = a.end ? min(ka_load(a.end + b), a.n) : a.n;
    r.len = e > r.t0 ? e - r.t0 : 0;
  }
  return r;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes into shared memory; zeros where v is false.
__device__ __forceinline__ void ka_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
// ... of scattered rows: without more of the neighbourhood than a 64-byte row.
__device__ __forceinline__ void ka_copy16_near(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16;\n" ::"r"(dst), "l"(src)
               : "memory");
}
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

// Where a warp's next tile comes from.  Lane l copies chunk l % 4 of the rows of tokens l / 4
// + 8 h (swizzled by 2 where the token's bit 1 is set) and the scale record of token l.
// Tokens past the row, and indices outside [0, n), become zeros; a gathered stage keeps
// the mask of the others.
template <bool GATHER>
struct KaSrc {
  const uint8_t *k, *v;     // this lane's chunk: of the tile's first token, or of token 0
  const uint16_t* s;        // ... its token's scale record, or token 0's
  const int32_t* idx;       // gathered: the tile's index of this lane
  int left;                 // tokens of the row from the tile on
  int tok;                  // gathered: this lane's index, requested a tile ahead
  __device__ __forceinline__ void fetch(int lane) {
    if (GATHER) tok = lane < left ? ka_load(idx) : -1;
  }
  __device__ __forceinline__ void set(const KaArgs& a, int64_t row, const KaRow& r, int tile,
                                      int lane) {
    left = r.len - tile * kKaTile;
    const int64_t at = row * a.ncap + (GATHER ? 0 : r.t0 + (int64_t)tile * kKaTile);
    const int64_t off = (at + (GATHER ? 0 : lane >> 2)) * kKv4Row + (lane & 3) * 16;
    k = a.c.k + off;
    v = a.c.v + off;
    s = a.c.scale + (at + (GATHER ? 0 : lane)) * kKv4Scales;
    if (GATHER) idx = a.idx + row * a.idx_stride + tile * (int64_t)kKaTile + lane;
    fetch(lane);
  }
  __device__ __forceinline__ void advance(int tiles, int lane) {
    left -= tiles * kKaTile;
    if (GATHER) {
      idx += (int64_t)tiles * kKaTile;
    } else {
      k += (int64_t)tiles * kKaTile * kKv4Row;
      v += (int64_t)tiles * kKaTile * kKv4Row;
      s += (int64_t)tiles * kKaTile * kKv4Scales;
    }
    fetch(lane);
  }
  // p + t bytes
  static __device__ __forceinline__ const uint8_t* at(const uint8_t* p, uint32_t t, int bytes) {
    uint64_t r;
    asm("mad.wide.u32 %0, %1, %2, %3;\n" : "=l"(r) : "r"(t), "r"(bytes), "l"(p));
    return reinterpret_cast<const uint8_t*>(r);
  }
  __device__ __forceinline__ void issue(const KaArgs& a, uint32_t stage, int lane) const {
    const int tl = lane >> 2;
    const uint32_t dst = stage + tl * kKv4Row + (((lane & 3) ^ (tl & 2)) * 16);
    const uint32_t dsts = stage + kKaOffS + lane * 16;
    if (GATHER) {
      const bool ok = (unsigned)tok < (unsigned)a.n;
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
      const uint8_t* sb = reinterpret_cast<const uint8_t*>(s);
      if (mask == 0xFFFFFFFFu) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint32_t t = __shfl_sync(0xFFFFFFFFu, tok, tl + 8 * h);
          ka_copy16_near(dst + h * 8 * kKv4Row, at(k, t, kKv4Row));
          ka_copy16_near(dst + h * 8 * kKv4Row + kKaOffV, at(v, t, kKv4Row));
        }
        ka_copy16_near(dsts, at(sb, tok, 2 * kKv4Scales));
      } else {
        const uint32_t safe = ok ? tok : 0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint32_t t = __shfl_sync(0xFFFFFFFFu, safe, tl + 8 * h);
          const bool val = mask >> (tl + 8 * h) & 1u;
          ka_copy16(dst + h * 8 * kKv4Row, at(k, t, kKv4Row), val);
          ka_copy16(dst + h * 8 * kKv4Row + kKaOffV, at(v, t, kKv4Row), val);
        }
        ka_copy16(dsts, at(sb, safe, 2 * kKv4Scales), ok);
      }
      if (lane == 0) sts32(stage + kKaOffMask, mask);
    } else if (left >= kKaTile) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        ka_copy16(dst + h * 8 * kKv4Row, k + h * 8 * kKv4Row);
        ka_copy16(dst + h * 8 * kKv4Row + kKaOffV, v + h * 8 * kKv4Row);
      }
      ka_copy16(dsts, s);
    } else {  // addresses past the row's last token stay at the tile's first
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const bool val = tl + 8 * h < left;
        const int64_t off = val ? h * 8 * kKv4Row : -(int64_t)tl * kKv4Row;
        ka_copy16(dst + h * 8 * kKv4Row, k + off, val);
        ka_copy16(dst + h * 8 * kKv4Row + kKaOffV, v + off, val);
      }
      ka_copy16(dsts, lane < left ? s : s - (int64_t)lane * kKv4Scales, lane < left);
    }
  }
};

// q as the B operand, and per-head constants of the lane's two columns (heads).
template <int G>
struct KaQ {
  // [columns 0..3 or 4..7 (G = 8: all at once)][group][k-step][half]
  uint32_t b[G == 8 ? 1 : 2][2][4][2];
  float ch[2];          // scale log2(e) 2^9 / (q's power of two)
  float qs[2][2];       // [column][group]: scale log2(e) sum of the group's q
};

// The head of column c (c < 8); with G <= 4 columns 4..7 repeat 0..3.
template <int G>
__device__ __forceinline__ int ka_head(int c) {
  return G == 8 ? c : c & 3;
}

// Requests a row's queries into a stage, with its first tile.
template <int G>
__device__ __forceinline__ void ka_issue_q(const KaArgs& a, uint32_t stage, int row, int lane) {
  const uint16_t* q = a.q + ((int64_t)(row / a.Hkv) * a.Hq + row % a.Hkv * G) * kD;
#pragma unroll
  for (int c = lane; c < G * kD / 8; c += 32) ka_copy16(stage + kKaOffQ + 16 * c, q + 8 * c);
}

template <int G>
__device__ __forceinline__ void ka_load_q(KaQ<G>& Q, const KaArgs& a, uint32_t stage, int lane) {
  const int gid = lane >> 2, tig = lane & 3, hd = ka_head<G>(gid);
  const bool real = hd < G;
  const uint32_t qr = stage + kKaOffQ + (real ? hd : 0) * kD * 2;
  uint4 w[2][2];
  float top = 0.0f, sum[2] = {0.0f, 0.0f};
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[g][j] = lds128(qr + 2 * (64 * g + 16 * tig + 8 * j));
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
  // 2^k q has its largest value in [2^14, 2^15) (k at most 120: smaller heads give 0)
  const int k = top > 0.0f ? min(14 - ((int)(__float_as_uint(top) >> 23) - 127), 120) : 0;
  const float up = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // word 4 tig + 2 j + g: channels i and i + 4 of the octet are a half-word pair
      const uint32_t x[4] = {w[g][j].x, w[g][j].y, w[g][j].z, w[g][j].w};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const __half2 lo = __floats2half2_rn(bf16_lo(x[s]) * up, bf16_lo(x[s + 2]) * up);
        const __half2 hi = __floats2half2_rn(bf16_hi(x[s]) * up, bf16_hi(x[s + 2]) * up);
        const uint32_t x0 = *reinterpret_cast<const uint32_t*>(&lo);
        const uint32_t x1 = *reinterpret_cast<const uint32_t*>(&hi);
        if constexpr (G == 8) {
          Q.b[0][g][2 * j + s][0] = x0;
          Q.b[0][g][2 * j + s][1] = x1;
        } else {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            Q.b[t][g][2 * j + s][0] = gid >> 2 == t ? x0 : 0u;
            Q.b[t][g][2 * j + s][1] = gid >> 2 == t ? x1 : 0u;
          }
        }
      }
    }
  const float sl = a.scale * kKaLog2e;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int src = 4 * (2 * tig + e);  // a lane that loaded the column's head
    const int kc = __shfl_sync(0xFFFFFFFFu, k, src);
    Q.ch[e] = sl * 512.0f * __uint_as_float((uint32_t)(127 - kc) << 23);
    Q.qs[e][0] = sl * __shfl_sync(0xFFFFFFFFu, sum[0], src);
    Q.qs[e][1] = sl * __shfl_sync(0xFFFFFFFFu, sum[1], src);
  }
}

// f16 pairs of the codes that a word holds at bits 0..3 (lo) or 4..7 (hi) of its halves:
// masked in place they are the subnormals c 2^-24 or 16 c 2^-24; a multiplication takes
// them to c 2^-9, normal numbers (the tensor cores align products by their nominal
// exponents and cut the rest, which would cost subnormals up to ten bits).
__device__ __forceinline__ uint32_t ka_code_lo(uint32_t x) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(y) : "r"(x & 0x000F000Fu), "r"(0x78007800u));  // 2^15
  return y;
}
__device__ __forceinline__ uint32_t ka_code_hi(uint32_t x) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(y) : "r"(x & 0x00F000F0u), "r"(0x68006800u));  // 2^11
  return y;
}
// The same, centred: (c - 7.5) 2^-9.
__device__ __forceinline__ uint32_t ka_mid_lo(uint32_t x) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;\n"
      : "=r"(y)
      : "r"(x & 0x000F000Fu), "r"(0x78007800u), "r"(0xA380A380u));  // -7.5 2^-9
  return y;
}
__device__ __forceinline__ uint32_t ka_mid_hi(uint32_t x) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;\n"
      : "=r"(y)
      : "r"(x & 0x00F000F0u), "r"(0x68006800u), "r"(0xA380A380u));
  return y;
}

// A warp's online softmax.  o: sum w (c - 7.5) in units of 2^-9; tile 4 g + u holds channels 64 g + 8 gid + 2 u (o[..][e]) and + 1 (o[..][2 + e]) of
// columns 2 tig + e (G <= 4: columns 4..7 the low parts).  m, f: of those columns' heads;
// mo: sum p (m + 7.5 s); l, mo: this lane's tokens only.
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

// The largest x over the lanes that hold the same heads.
template <int G>
__device__ __forceinline__ float ka_head_max(float x) {
#pragma unroll
  for (int o = G == 8 ? 4 : 2; o <= 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

// Raises m to the whole number above `top`, the tile's largest logit of column e.
__device__ __forceinline__ void ka_raise_m(KaState& S, int e, float top) {
  if (!(top > S.m[e])) return;  // uniform over the column's lanes
  const float up = ceilf(top), d = up - S.m[e], al = ka_exp2(-d);
  S.m[e] = up;
  S.l[e] *= al;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    S.mo[e][g] *= al;
    // what was summed weighs 2^-d now: f takes up the factor, o stays, up to f's limit.  In
    // exponents, as 2^d alone may pass the fp32 range (f then stayed where wide values had
    // left it, and small ones after them became 0).  1 / f is as exact; r is 0 below 2^-49,
    // where f is at its limit and an old sum below 2^-135 of no account.
    const uint32_t fb = __float_as_uint(S.f[e][g]);
    const float fn = __uint_as_float(
        min(fb + ((uint32_t)fminf(d, 217.0f) << 23), __float_as_uint(kKaF0)));
    const float r = fn * (al * __uint_as_float(0x7F000000u - fb));
    S.f[e][g] = fn;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      S.o[4 * g + u][e] *= r;
      S.o[4 * g + u][2 + e] *= r;
    }
  }
}

// Lowers f where it takes `top`, the tile's largest p s of column e and group g, above
// kKaWMax, to bring it to [2^7, 2^8).
__device__ __forceinline__ void ka_lower_f(KaState& S, int e, int g, float top) {
  if (!(top * S.f[e][g] > kKaWMax) || !(top < INFINITY)) return;
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

__device__ __forceinline__ uint32_t ka_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// A tile is worked on as two 16-token halves, in three parts: the scores S = K q^T, the
// weights, and the values O^T += V^T P^T.  Row r of a half's score tile is token tau(r)
// (r < 8: r / 2, odd rows 4 + (r / 2 ^ 1)) or tau(r - 8) + 8: with the swizzle, any eight
// lanes of a K read and any sixteen of a V read touch each bank once.
// G = 8: a lane has the logits of two heads and four tokens.  G <= 4: the first half's
// heads are columns 0..3 and the second's 4..7 (q's other columns are zero), so that a
// lane has two heads and the two tokens of its half, and no logit is computed twice.
template <int G>
struct KaScores {
  float c[G == 8 ? 2 : 1][2][4];  // [half][group]
};

__device__ __forceinline__ int ka_tau(int gid) {
  return (gid & 1) ? 4 + (gid >> 1 ^ 1) : gid >> 1;
}

template <int G>
__device__ __forceinline__ void ka_scores(KaScores<G>& C, const KaQ<G>& Q, uint32_t st, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
  constexpr bool both = G != 8;
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const uint32_t ak =
        st + (16 * hf + ka_tau(gid)) * kKv4Row + ((tig ^ (gid >> 1 & 2)) * 16);
    const uint4 ka = lds128(ak), kb = lds128(ak + 8 * kKv4Row);
    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t xa = wa[2 * j + g] >> (8 * s), xb = wb[2 * j + g] >> (8 * s);
          const uint32_t a0 = ka_code_lo(xa), a1 = ka_code_lo(xb);
          const uint32_t a2 = ka_code_hi(xa), a3 = ka_code_hi(xb);
          const uint32_t(&qb)[2] = Q.b[both ? hf : 0][g][2 * j + s];
          float(&c)[4] = C.c[both ? 0 : hf][g];
          if (j + s == 0 && (!both || hf == 0))
            mma_f16_zero(c, a0, a1, a2, a3, qb[0], qb[1]);
          else
            mma_f16(c, a0, a1, a2, a3, qb[0], qb[1]);
        }
  }
}

// P^T's high and low f16 parts, as B operands: G = 8 h and l; G <= 4 columns 0..3 of h the
// high parts of its half's heads, 4..7 the low parts.
struct KaP {
  uint32_t h[2][2][2], l[2][2][2];  // [half][group][r]
};

// valid: the tile's tokens that count.
template <int G>
__device__ __forceinline__ void ka_weights(KaP& P, KaState& S, const KaScores<G>& C,
                                           const KaQ<G>& Q, uint32_t st, uint32_t valid,
                                           int lane) {
  constexpr int NR = G == 8 ? 4 : 2;  // this lane's tokens
  const int gid = lane >> 2, tig = lane & 3;
  const int side = G == 8 ? 0 : tig >> 1;  // G <= 4: the half of this lane's tokens
  const int tk = ka_tau(gid);
  float cq[NR][2][2];  // [token][column][group]: scale log2(e) sum of q c
  float sk[NR][2], mk[NR][2], sv[NR][2], mv[NR][2];  // [token][group]
  auto token = [&](int i) { return (G == 8 ? 16 * (i >> 1) : 16 * side) + tk + 8 * (i & 1); };
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const uint4 sc = lds128(st + kKaOffS + token(i) * 16);
    sk[i][0] = bf16_lo(sc.x);
    sk[i][1] = bf16_lo(sc.y);
    mk[i][0] = bf16_hi(sc.x);
    mk[i][1] = bf16_hi(sc.y);
    sv[i][0] = bf16_lo(sc.z);
    sv[i][1] = bf16_lo(sc.w);
    mv[i][0] = fmaf(7.5f, sv[i][0], bf16_hi(sc.z));  // the middle of the group's range
    mv[i][1] = fmaf(7.5f, sv[i][1], bf16_hi(sc.w));
    const float(&ac)[2][4] = C.c[i >> 1];
    // out of q's f16 units before the step comes in: a step is up to 2^124, and its product
    // with a sum in those units (up to 2^16) could pass the fp32 range where a logit does not
#pragma unroll
    for (int g = 0; g < 2; ++g)
      f2_split(f2_mul(f2_make(ac[g][2 * (i & 1)], ac[g][2 * (i & 1) + 1]),
                      f2_make(Q.ch[0], Q.ch[1])),
               cq[i][0][g], cq[i][1][g]);
  }
  // log2 of the weight over 2^sub
  auto logit = [&](int i, int e, float sub) {
    const float base = fmaf(mk[i][1], Q.qs[e][1], fmaf(mk[i][0], Q.qs[e][0], -sub));
    return fmaf(sk[i][1], cq[i][e][1], fmaf(sk[i][0], cq[i][e][0], base));
  };
  auto ok = [&](int i) { return valid >> token(i) & 1u; };
  float p[NR][2], sum[2];
  auto weights = [&](int e) {
#pragma unroll
    for (int i = 0; i < NR; ++i) p[i][e] = ka_exp2(logit(i, e, S.m[e]));
    if (valid != 0xFFFFFFFFu) {
#pragma unroll
      for (int i = 0; i < NR; ++i)
        if (!ok(i)) p[i][e] = 0.0f;
    }
    sum[e] = p[0][e] + p[1][e];
    if constexpr (NR == 4) sum[e] += p[2][e] + p[3][e];
  };
  weights(0);
  weights(1);
  // w = (p f) s, in this order: p f is at most 2^109, where s f would be infinite for a wide
  // step while f stands at its start, and p = 0 or a small w would become NaN.  p f below
  // the normal range takes at most 2^-26 from a w.
  float pf[NR][2][2];  // [token][group][column]
  uint32_t hi[NR][2];  // w's high parts, a pair of columns each
  auto weigh = [&]() {
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        pf[i][g][0] = p[i][0] * S.f[0][g];
        pf[i][g][1] = p[i][1] * S.f[1][g];
        hi[i][g] = ka_pack(pf[i][g][0] * sv[i][g], pf[i][g][1] * sv[i][g]);
      }
  };
  weigh();
  __half2 ht = *reinterpret_cast<__half2*>(&hi[0][0]);
#pragma unroll
  for (int i = 1; i < 2 * NR; ++i)
    ht = __hmax2(ht, *reinterpret_cast<__half2*>(&hi[i >> 1][i & 1]));
  const uint32_t hb = *reinterpret_cast<uint32_t*>(&ht);
  const bool over =
      fmaxf(sum[0], sum[1]) > kKaPMax || (hb & 0xFFFFu) > 0x7400u || hb > 0x7400FFFFu;
  if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float zt = -INFINITY;
#pragma unroll
      for (int i = 0; i < NR; ++i)
        if (ok(i)) zt = fmaxf(zt, logit(i, e, 0.0f));
      ka_raise_m(S, e, ka_head_max<G>(zt));
      weights(e);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float wt = 0.0f;
#pragma unroll
        for (int i = 0; i < NR; ++i) wt = fmaxf(wt, p[i][e] * sv[i][g]);
        ka_lower_f(S, e, g, ka_head_max<G>(wt));
      }
    }
    weigh();
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    S.l[e] += sum[e];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int i = 0; i < NR; ++i) S.mo[e][g] = fmaf(p[i][e], mv[i][g], S.mo[e][g]);
  }
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float2 h2 = __half22float2(*reinterpret_cast<const __half2*>(&hi[i][g]));
      const uint32_t lo = ka_pack(fmaf(pf[i][g][0], sv[i][g], -h2.x),
                                  fmaf(pf[i][g][1], sv[i][g], -h2.y));
      if constexpr (G == 8) {
        P.h[i >> 1][g][i & 1] = transpose_8x8(hi[i][g]);
        P.l[i >> 1][g][i & 1] = transpose_8x8(lo);
      } else {  // the first half's low parts move to the lanes of columns 4..7, the
                // second's high parts to those of 0..3
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, side ? hi[i][g] : lo, 2);
        P.h[0][g][i] = transpose_8x8(side ? got : hi[i][g]);
        P.h[1][g][i] = transpose_8x8(side ? lo : got);
      }
    }
}

// V's codes as the MMAs' A operand before unpacking: rows 2 tig, 2 tig + 1 (and + 8) of either
// half, 8 bytes from byte 8 gid (channels 8 gid .. + 7 of either group), the two tokens'
// half-words paired.
struct KaV {
  uint32_t x[2][2][2][2];  // [half][group][low or high half-word][rows + 0 or 8]
};

__device__ __forceinline__ void ka_load_v(KaV& V, uint32_t st, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const uint32_t av = st + kKaOffV + 16 * hf * kKv4Row + ((gid >> 1 ^ (tig & 2)) * 16) +
                        (gid & 1) * 8;
    const uint2 v0 = lds64(av + tig * kKv4Row), v1 = lds64(av + (4 + (tig ^ 1)) * kKv4Row);
    const uint2 v2 = lds64(av + (tig + 8) * kKv4Row), v3 = lds64(av + (12 + (tig ^ 1)) * kKv4Row);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t sel = k ? 0x7632u : 0x5410u;
      V.x[hf][0][k][0] = __byte_perm(v0.x, v1.x, sel);
      V.x[hf][0][k][1] = __byte_perm(v2.x, v3.x, sel);
      V.x[hf][1][k][0] = __byte_perm(v0.y, v1.y, sel);
      V.x[hf][1][k][1] = __byte_perm(v2.y, v3.y, sel);
    }
  }
}

template <int G>
__device__ __forceinline__ void ka_values(KaState& S, const KaP& P, const KaV& V) {
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      // the tensor cores add by truncation: a tile is summed from zero and added by
      // rounding, or the error would grow with the tokens
      float t[4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t x = V.x[hf][g][u >> 1][0] >> (8 * (u & 1));
        const uint32_t y = V.x[hf][g][u >> 1][1] >> (8 * (u & 1));
        const uint32_t a0 = ka_mid_lo(x), a1 = ka_mid_hi(x), a2 = ka_mid_lo(y), a3 = ka_mid_hi(y);
        if (hf == 0)
          mma_f16_zero(t, a0, a1, a2, a3, P.h[hf][g][0], P.h[hf][g][1]);
        else
          mma_f16(t, a0, a1, a2, a3, P.h[hf][g][0], P.h[hf][g][1]);
        if (G == 8) mma_f16(t, a0, a1, a2, a3, P.l[hf][g][0], P.l[hf][g][1]);
      }
      float(&o)[4] = S.o[4 * g + u];
      if constexpr (G == 8) {  // in pairs (2% here; with G <= 4 single additions are 3% faster)
        f2_split(f2_add(f2_make(o[0], o[1]), f2_make(t[0], t[1])), o[0], o[1]);
        f2_split(f2_add(f2_make(o[2], o[3]), f2_make(t[2], t[3])), o[2], o[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += t[i];
      }
    }
}

// The mask of a row's tile whose first token has `left` tokens of the row from it on.
template <bool GATHER>
__device__ __forceinline__ uint32_t ka_valid(uint32_t stage, int left) {
  if (GATHER) return lds32(stage + kKaOffMask);
  return left >= kKaTile ? 0xFFFFFFFFu : (1u << left) - 1u;
}

// The tiles of a row (or a part of one), `tiles` of them, the first in stage `slot` with the
// queries: `issue` requests one more tile into the stage it is given and commits.
template <int G, bool GATHER, class Issue>
__device__ __forceinline__ void ka_tiles(KaState& S, const KaArgs& a, uint32_t ring,
                                         uint32_t& slot, uint32_t& put, int tiles, int left,
                                         int step, Issue issue, int lane) {
  if (tiles <= 0) return;
  KaQ<G> Q;
  ka_wait<kKaDepth<G> - 2>();
  __syncwarp();
  ka_load_q<G>(Q, a, slot, lane);
  for (; tiles > 0; --tiles, left -= step) {
    if constexpr (G != 8) {
      issue(put);
      ka_wait<kKaDepth<G> - 1>();
    } else {
      ka_wait<kKaDepth<G> - 2>();
    }
    __syncwarp();
    KaScores<G> C;
    ka_scores<G>(C, Q, slot, lane);
    KaV V;  // requested here, where the chain of the weights leaves the time
    ka_load_v(V, slot, lane);
    if constexpr (G == 8) issue(put);  // 244 us here, 252 at the top; with G <= 4 213 and 211
    KaP P;
    ka_weights<G>(P, S, C, Q, slot, ka_valid<GATHER>(slot, left), lane);
    ka_values<G>(S, P, V);
    __syncwarp();
    put = slot;
    slot = slot == ring + (kKaDepth<G> - 1) * kKaStage<G> ? ring : slot + kKaStage<G>;
  }
}

// The state of a warp in natural units, written to so [G][kD] and sml [G] = (m, l); with
// DONE it is the whole row's: so is out, divided by l, and lse (or null) takes the place
// of sml.
template <int G, bool DONE>
__device__ __forceinline__ void ka_flush(KaState& S, float* so, float2* sml, float* lse,
                                         int lane) {
  const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int o = G == 8 ? 4 : 2; o <= 16; o <<= 1) {
      S.l[e] += __shfl_xor_sync(0xFFFFFFFFu, S.l[e], o);
      S.mo[e][0] += __shfl_xor_sync(0xFFFFFFFFu, S.mo[e][0], o);
      S.mo[e][1] += __shfl_xor_sync(0xFFFFFFFFu, S.mo[e][1], o);
    }
    const int c = 2 * tig + e, hd = ka_head<G>(c);
    const bool mine = c < G;
    const float l = S.l[e];
    if (mine && gid == 0) {
      if (!DONE)
        sml[hd] = make_float2(S.m[e], l);
      else if (lse)
        lse[hd] = l != 0.0f ? (S.m[e] + log2f(l)) * kKaLn2 : -INFINITY;
    }
    const float inv = !DONE ? 1.0f : l != 0.0f ? 1.0f / l : 0.0f;  // an empty row gives 0
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float k = 512.0f / S.f[e][g];
      float x[8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float even = S.o[4 * g + u][e], odd = S.o[4 * g + u][2 + e];
        if (G != 8) {  // the low parts' columns
          even += __shfl_xor_sync(0xFFFFFFFFu, even, 2);
          odd += __shfl_xor_sync(0xFFFFFFFFu, odd, 2);
        }
        x[2 * u] = fmaf(even, k, S.mo[e][g]) * inv;
        x[2 * u + 1] = fmaf(odd, k, S.mo[e][g]) * inv;
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

// Few tiles: one cluster of CTAs per row, tiles dealt to its warps in turn, the states joined
// through shared and distributed shared memory.  One launch, and the workspace that every
// call brings is left alone: a call of one 4,096-token KV head takes 8.2 us as a graph node
// (9.3 with the streaming kernel), one of a single tile 4.4.
template <int G, bool GATHER>
__global__ void __launch_bounds__(kKaThreads, 2) kv4_cluster_kernel(const KaArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  kv4_wait_prior();
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), CS = (int)cl.num_blocks();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.y;
  const int b = (int)(row / a.Hkv), h = (int)(row % a.Hkv);
  const KaRow r = ka_row<GATHER>(a, row, b);
  const int step = CS * kKaWarps;
  const uint32_t ring = smem_addr(smem) + warp * kKaRing<G>;
  const int first = rank * kKaWarps + warp;
  KaSrc<GATHER> src;
  src.set(a, row, r, first, lane);
#pragma unroll
  for (int d = 0; d < kKaDepth<G> - 1; ++d) {
    if (src.left > 0) {
      if (d == 0) ka_issue_q<G>(a, ring, (int)row, lane);
      src.issue(a, ring + d * kKaStage<G>, lane);
      src.advance(step, lane);
    }
    ka_commit();
  }
  KaState S;
  S.clear();
  uint32_t slot = ring, put = ring + (kKaDepth<G> - 1) * kKaStage<G>;
  const int tiles = (int)(((unsigned)r.len + kKaTile - 1) / kKaTile);
  ka_tiles<G, GATHER>(
      S, a, ring, slot, put, (tiles - first + step - 1) / step, r.len - first * kKaTile,
      step * kKaTile,
      [&](uint32_t stage) {
        if (src.left > 0) {
          src.issue(a, stage, lane);
          src.advance(step, lane);
        }
        ka_commit();
      },
      lane);
  ka_wait<0>();
  __syncthreads();  // the rings become the warps' states
  float* so = reinterpret_cast<float*>(smem);             // [warps][G][kD]
  float2* sml = reinterpret_cast<float2*>(so + kKaWarps * G * kD);  // [warps][G]
  float* co = reinterpret_cast<float*>(sml + kKaWarps * G);  // the CTA's: [G][kD]
  float2* cml = reinterpret_cast<float2*>(co + G * kD);      // [G]
  ka_flush<G, false>(S, so + warp * G * kD, sml + warp * G, nullptr, lane);
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

// Many tokens: the rows' tiles, in row-major order, are cut into equal ranges, one per
// warp of the grid, and each warp's ring runs on across rows.  A row that lies within a
// range is written at once; a row cut by ranges leaves a partial per range, and a second
// kernel joins them in range order.
constexpr int kKaMaxWarps = 320 * kKaWarps;  // partials of the workspace: two per warp

// The ranges are equal shares of the rows' weights: kKaRowCost places that stand for what a
// row costs beside its tiles (queries, output, a last tile that is half empty), then one
// place per tile.  Without them the warps that drew a ragged batch's short rows ended 20 us
// after the others (64 x 8 rows of 1 to 16,384 tokens, G = 4: 127 us; 122, 118, 108, 109
// and 110 with 1, 2, 4, 6 and 8).
constexpr int kKaRowCost = 4;

// Items of the partition: sequences of Hkv rows each, or single rows with counts of
// their own.
template <bool GATHER>
__device__ __forceinline__ int ka_item_tiles(const KaArgs& a, int64_t item) {
  const KaRow r = ka_row<GATHER>(a, item, (int)item);  // either reads its one index only
  return (int)(((unsigned)r.len + kKaTile - 1) / kKaTile);
}
__device__ __forceinline__ int64_t ka_weight_of(int tiles) {
  return tiles > 0 ? (int64_t)tiles + kKaRowCost : 0;
}

// A segment: tiles [a0, a1) of a row; left: places of the range from tile a0's on (a GPU's
// memory holds far fewer than 2^31 tiles a warp).
template <bool GATHER>
struct KaSeg {
  int row, left, a0, a1, tiles;
  KaRow r;
  __device__ __forceinline__ void load(const KaArgs& a) {
    r = ka_row<GATHER>(a, row, row / a.Hkv);
    tiles = (int)(((unsigned)r.len + kKaTile - 1) / kKaTile);
    a1 = min(tiles, a0 + left);
  }
  // The range's next segment; false at its end.
  __device__ __forceinline__ bool next(const KaArgs& a) {
    left -= a1 - a0 + kKaRowCost;
    if (left <= 0) return false;
    a0 = 0;
    do {
      ++row;
      load(a);
    } while (tiles == 0 && row + 1 < (int)a.rows);
    return true;
  }
};

template <int G, bool GATHER>
__global__ void __launch_bounds__(kKaThreads, 2) kv4_stream_kernel(const KaArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ long long ends[kKaThreads], part[kKaWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t gw = (int64_t)blockIdx.x * kKaWarps + warp, W = (int64_t)gridDim.x * kKaWarps;
  // every thread counts the tiles of a run of items, a scan gives where its run ends
  const int64_t items = GATHER ? a.rows : a.rows / a.Hkv, mult = GATHER ? 1 : a.Hkv;
  const int64_t per = (items + kKaThreads - 1) / kKaThreads;
  const int64_t i0 = imin64(threadIdx.x * per, items), i1 = imin64(i0 + per, items);
  long long incl = 0;
#pragma unroll 8
  for (int64_t i = i0; i < i1; ++i) incl += ka_weight_of(ka_item_tiles<GATHER>(a, i)) * mult;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) part[warp] = incl;
  // rows without tokens, dealt to all warps of the grid
  for (int64_t r = gw; r < a.rows; r += W) {
    const int b = (int)(r / a.Hkv);
    if (ka_row<GATHER>(a, r, b).len > 0) continue;
    const int64_t bq = (int64_t)b * a.Hq + (r % a.Hkv) * G;
    for (int e = lane; e < G * kD; e += 32) ka_write(a, bq + e / kD, e % kD, 0.0f, 0.0f, 0.0f);
    if (lane == 0) a.meta[r] = make_int2(0, 0);
  }
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kKaWarps; ++w) {
    if (w < warp) incl += part[w];
    total += part[w];
  }
  ends[threadIdx.x] = incl;
  __syncthreads();
  const int64_t N = imin64(W, total);  // no range is empty
  if (gw >= N) return;
  const int64_t g0 = gw * total / N, g1 = (gw + 1) * total / N;
  KaSeg<GATHER> cur;
  {
    // the run that holds the first tile, then the item in it
    int run = 0;
#pragma unroll
    for (int k = 0; k < kKaWarps; ++k)
      run += __popc(__ballot_sync(0xFFFFFFFFu, ends[32 * k + lane] <= g0));
    int64_t at = run ? ends[run - 1] : 0, item = run * per;
    int64_t w = ka_weight_of(ka_item_tiles<GATHER>(a, item));
    while (g0 >= at + w * mult && item + 1 < items) {
      at += w * mult;
      w = ka_weight_of(ka_item_tiles<GATHER>(a, ++item));
    }
    const int64_t in = (g0 - at) / w, off = g0 - at - in * w - kKaRowCost;
    cur.row = (int)(item * mult + in);
    cur.a0 = (int)imax64(off, 0);
    cur.left = (int)(g1 - g0 + imin64(off, 0));
    if (cur.left <= 0) return;  // only places before the row's first tile
    cur.load(a);
  }
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  KaSeg<GATHER> it = cur;  // runs ahead of cur
  bool more = true;
  int itile = it.a0;
  KaSrc<GATHER> src;
  src.set(a, it.row, it.r, itile, lane);
  const uint32_t ring = smem_addr(smem) + warp * kKaRing<G>;
  ka_issue_q<G>(a, ring, it.row, lane);
  auto issue = [&](uint32_t stage) {
    if (more) {
      src.issue(a, stage, lane);
      if (++itile < it.a1) {
        src.advance(1, lane);
      } else {
        more = it.next(a);
        itile = 0;
        if (more) {
          src.set(a, it.row, it.r, 0, lane);
          // its queries into the stage that its first tile takes next (which may hold the
          // tile being worked on, whose queries are in registers)
          ka_issue_q<G>(a, stage == ring + (kKaDepth<G> - 1) * kKaStage<G> ? ring : stage + kKaStage<G>,
                        it.row, lane);
        }
      }
    }
    ka_commit();
  };
#pragma unroll
  for (int d = 0; d < kKaDepth<G> - 1; ++d) issue(ring + d * kKaStage<G>);
  uint32_t slot = ring, put = ring + (kKaDepth<G> - 1) * kKaStage<G>;
  do {
    KaState S;
    S.clear();
    ka_tiles<G, GATHER>(S, a, ring, slot, put, cur.a1 - cur.a0, cur.r.len - cur.a0 * kKaTile,
                        kKaTile, issue, lane);
    const bool whole = cur.a0 == 0 && cur.a1 == cur.tiles;
    if (cur.a0 == 0 && lane == 0) {
      const int64_t last = ((g1 - cur.left + cur.tiles) * N - 1) / total;
      a.meta[cur.row] = make_int2((int)gw, whole ? 0 : (int)(last - gw) + 1);
    }
    if (whole) {
      const int64_t bq = (int64_t)(cur.row / a.Hkv) * a.Hq + (cur.row % a.Hkv) * G;
      ka_flush<G, true>(S, a.out + bq * kD, nullptr, a.lse ? a.lse + bq : nullptr, lane);
    } else {  // partial 1 of the row's first warp, 0 of the others
      const int64_t p = (2 * gw + (cur.a0 == 0 ? 1 : 0)) * G;
      ka_flush<G, false>(S, a.part_o + p * kD, a.part_ml + p, nullptr, lane);
    }
  } while (cur.next(a));
  ka_wait<0>();
}

// Partials i0, i0 + step, .. of the np of one head of a row whose first warp is `first`:
// their sum over the lanes' four channels each, and (m, l).
template <int G, int FLIGHT>
__device__ __forceinline__ float4 ka_gather_parts(const KaArgs& a, int first, int np, int g, int i0,
                                                  int step, int lane, float& top, float& l) {
  auto at = [&](int i) { return (2 * ((int64_t)first + i) + (i == 0 ? 1 : 0)) * G + g; };
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  top = kKaEmpty;
  l = 0.0f;
  for (; i0 < np; i0 += FLIGHT * step) {  // so many partials in flight
    float2 ml[FLIGHT];
    float4 v[FLIGHT];
    float tb = top;
#pragma unroll
    for (int k = 0; k < FLIGHT; ++k) {
      const int i = i0 + step * k;
      ml[k] = i < np ? a.part_ml[at(i)] : make_float2(kKaEmpty, 0.0f);
      v[k] = i < np ? reinterpret_cast<const float4*>(a.part_o + at(i) * kD)[lane]
                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      tb = fmaxf(tb, ml[k].x);
    }
    const float f0 = exp2f(top - tb);
    top = tb;
    l *= f0;
    o.x *= f0;
    o.y *= f0;
    o.z *= f0;
    o.w *= f0;
#pragma unroll
    for (int k = 0; k < FLIGHT; ++k) {
      const float f = ka_weight(ml[k], top);
      l = fmaf(ml[k].y, f, l);
      o.x = fmaf(v[k].x, f, o.x);
      o.y = fmaf(v[k].y, f, o.y);
      o.z = fmaf(v[k].z, f, o.z);
      o.w = fmaf(v[k].w, f, o.w);
    }
  }
  return o;
}

// Joins the partials of the rows that were cut.  A CTA takes `run` heads of rows at a time,
// a warp each; those of more than kKaAlone partials are summed by all its warps.
constexpr int kKaJoinWarps = 16;
constexpr int kKaAlone = 16;

// FLIGHT: partials that a warp of the latter has in flight.  16 for a few heads (1 us less
// where 8 rows of 32,768 tokens take 18.5); 8, in 64 registers, for many, whose CTAs then
// fit beside the last of the streaming kernel's (with 73 they start 2 us later).
template <int G, int FLIGHT>
__global__ void __launch_bounds__(32 * kKaJoinWarps) kv4_join_kernel(const KaArgs a, int run) {
  __shared__ float4 so[kKaJoinWarps][32];
  __shared__ float2 sml[kKaJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  kv4_wait_prior();  // the streaming kernel
  const int64_t pairs = a.rows * G;
  for (int64_t base = (int64_t)blockIdx.x * run; base < pairs; base += (int64_t)gridDim.x * run) {
    const int64_t mine = base + warp;
    bool wide = false;
    if (warp < run && mine < pairs) {
      const int64_t row = mine / G;
      const int g = (int)(mine % G);
      const int2 mt = a.meta[row];
      wide = mt.y > kKaAlone;
      if (mt.y > 0 && !wide) {
        float top, l;
        const float4 o = ka_gather_parts<G, 8>(a, mt.x, mt.y, g, 0, 1, lane, top, l);
        const int64_t bq = (row / a.Hkv) * a.Hq + (row % a.Hkv) * G + g;
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        reinterpret_cast<float4*>(a.out + bq * kD)[lane] =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (a.lse && lane == 0) a.lse[bq] = l != 0.0f ? (top + log2f(l)) * kKaLn2 : -INFINITY;
      }
    }
    if (!__syncthreads_or(wide)) continue;
    for (int k = 0; k < run && base + k < pairs; ++k) {
      const int64_t row = (base + k) / G;
      const int g = (int)((base + k) % G);
      const int2 mt = a.meta[row];
      if (mt.y <= kKaAlone) continue;  // uniform over the CTA
      float top, l;
      so[warp][lane] = ka_gather_parts<G, FLIGHT>(a, mt.x, mt.y, g, warp, kKaJoinWarps, lane, top, l);
      if (lane == 0) sml[warp] = make_float2(top, l);
      __syncthreads();
      if (threadIdx.x < kD) {
        const int j = threadIdx.x;
        float tt = kKaEmpty, ll = 0.0f, oo = 0.0f;
#pragma unroll
        for (int w = 0; w < kKaJoinWarps; ++w) tt = fmaxf(tt, sml[w].x);
#pragma unroll
        for (int w = 0; w < kKaJoinWarps; ++w) {
          const float f = ka_weight(sml[w], tt);
          ll = fmaf(sml[w].y, f, ll);
          oo = fmaf(reinterpret_cast<const float*>(so[w])[j], f, oo);
        }
        ka_write(a, (row / a.Hkv) * a.Hq + (row % a.Hkv) * G + g, j, oo, tt, ll);
      }
      __syncthreads();
    }
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The largest cluster of the cluster kernel that this device runs (cached per device); 0:
// none, not even of one CTA.
template <int G, bool GATHER>
int ka_max_cluster() {
  static std::atomic<int> most[kMaxDev];
  return per_device_cached(most, [] {
    auto kern = kv4_cluster_kernel<G, GATHER>;
    const size_t bytes = (size_t)kKaWarps * kKaRing<G>;
    if (set_smem_limit((const void*)kern, bytes, "kv4 attend") != SD_OK) return 0;
    int c = 8;
    for (; c > 0; c >>= 1) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(c, 1, 1);
      cfg.blockDim = dim3(kKaThreads, 1, 1);
      cfg.dynamicSmemBytes = bytes;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = c;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int nc = 0;
      if (cudaOccupancyMaxActiveClusters(&nc, kern, &cfg) == cudaSuccess && nc > 0) break;
      cudaGetLastError();
    }
    return c;
  });
}

template <int G, bool GATHER>
int ka_launch(const KaArgs& a, int64_t most, cudaStream_t st) {
  const int64_t tiles = (most + kKaTile - 1) / kKaTile;
  const int cs = fallback_forced() ? 0
                                   : kv4_cluster_of(a.rows, tiles, device_sm_count(),
                                                    ka_max_cluster<G, GATHER>());
  const size_t bytes = (size_t)kKaWarps * kKaRing<G>;
  if (cs == 0) {
    auto kern = kv4_stream_kernel<G, GATHER>;
    if (int rc = set_smem_limit((const void*)kern, bytes, "kv4 attend")) return rc;
    const int grid = (int)imin64(2 * device_sm_count(), kKaMaxWarps / kKaWarps);
    // (launched early like the others it was no faster, and 3 % slower on long rows)
    kern<<<grid, kKaThreads, bytes, st>>>(a);
    note_launches(1);
    if (int rc = check_launch("kv4 attend")) return rc;
    const int64_t pairs = a.rows * G, ctas = 2 * device_sm_count();
    const int run = (int)imin64((pairs + ctas - 1) / ctas, kKaJoinWarps);
    const dim3 jgrid((unsigned)imin64((pairs + run - 1) / run, 8 * ctas));
    auto join = pairs <= device_sm_count() ? kv4_join_kernel<G, 16> : kv4_join_kernel<G, 8>;
    return kv4_launch("kv4 attend join", join, jgrid, 32 * kKaJoinWarps, 0, 0, st, a, run);
  }
  auto kern = kv4_cluster_kernel<G, GATHER>;
  if (int rc = set_smem_limit((const void*)kern, bytes, "kv4 attend")) return rc;
  return kv4_launch("kv4 attend", kern, dim3(cs, (unsigned)a.rows), kKaThreads, bytes, cs, st, a);
}

template <int G>
int ka_pick(const KaArgs& a, int64_t most, cudaStream_t st) {
  return a.idx ? ka_launch<G, true>(a, most, st) : ka_launch<G, false>(a, most, st);
}

}  // namespace

size_t kv4_attend_workspace_bytes(const Dims& s) {
  return align256(sizeof(int2) * s.B * s.Hkv) +
         (size_t)2 * kKaMaxWarps * s.G * (sizeof(float) * kD + sizeof(float2));
}

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
  uint8_t* p = (uint8_t*)ws;
  a.meta = (int2*)p;
  p += align256(sizeof(int2) * a.rows);
  a.part_o = (float*)p;
  a.part_ml = (float2*)(p + sizeof(float) * 2 * kKaMaxWarps * s.G * kD);
  const int64_t most = idx ? max_count : s.n;
  switch (s.G) {
    case 1: return ka_pick<1>(a, most, st);
    case 2: return ka_pick<2>(a, most, st);
    case 4: return ka_pick<4>(a, most, st);
    default: return ka_pick<8>(a, most, st);
  }
}

}  // namespace sd
