// The 4-bit K/V cache: tokens quantised as they are written, and read back as bf16
// (the KV-write path of HashAttention: Semantic Sparsity for Faster Inference, 2.2,
// where the index is computed as keys are written; the 4-bit uniform codes of Fathom:
// Per-Query Read Depth for Sparse Decoding over Offloaded KV Caches, paragraph "store
// as bit planes per channel", taken per token so that a token's row is complete when
// it is written).
//
// A group is 64 channels of one token's K or V: m = min, s = bf16((max - m) / 15),
// c = clamp(rint((x - m) / s), 0, 15), and a channel stands for c s + m.
//
// A warp's lanes 0..15 take a token's K row and lanes 16..31 its V row, 8 channels (one
// 16-byte access of bf16, one 32-bit word of codes) per lane, 8 lanes per group; four
// tokens at a time, the next four requested before the current ones are worked on.
//
// The read is bound by HBM: 4 x 8 x 131,072 tokens, 2.75 GB, in 423 us (6.5 TB/s, 96 % of
// the copy rate).  The write moves the same bytes in 440 us (6.3 TB/s): its ~100
// instructions a token (quotients rounded as a division's, in pairs of fp32) nearly fill
// the schedulers.  With one token a warp and plain divisions the two took 1.87 ms together.
#include "sd_internal.cuh"
#include "sd_kv4.cuh"

namespace sd {
namespace {

constexpr int kKvWarps = 8;
constexpr int kKvRun = 4;                     // tokens a warp has in hand
constexpr int kKvStep = kKvWarps * kKvRun;    // tokens of a CTA's step

struct KvMoveArgs {
  uint16_t* x[2];        // K, V rows (read by the write, written by the read); null: skipped
  int64_t sb[2], sh[2], st[2];  // their strides in elements
  uint8_t* code[2];      // the cache's k, v
  uint16_t* scale;
  int hkv;
  int64_t n, ncap, m, first;
  const int32_t* pos;
  const int32_t* length;
};

// The tokens [0, len) of sequence b that the call moves and their first position.
__device__ __forceinline__ void kv_range(const KvMoveArgs& a, int b, int64_t& len, int64_t& p0) {
  len = a.length ? imin64(a.m, a.length[b]) : a.m;
  p0 = a.first + (a.pos ? a.pos[b] : 0);
}

// Of both bf16 halves; a NaN stays.
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// What a lane moves: its half (0: K, 1: V), octet and row, and the `count` tokens of the
// row that have a place in the cache, numbered from the first of them (tokens that are
// dropped before it cost nothing).  Both are unsigned and a step is taken only where it
// stays below count, so that no sum wraps however long the call.
struct KvLane {
  int half, l;
  unsigned t, count;
  int64_t row, tok;  // tok: the first one's place among the cache's tokens
  int64_t x;         // offset of its octet in the caller's array
  __device__ __forceinline__ KvLane(const KvMoveArgs& a) {
    const int lane = threadIdx.x & 31;
    half = lane >> 4;
    l = lane & 15;
    row = blockIdx.y;
    const int b = (int)(row / a.hkv), h = (int)(row % a.hkv);
    int64_t len, p0;
    kv_range(a, b, len, p0);
    t = blockIdx.x * kKvStep + (threadIdx.x >> 5) * kKvRun;
    const int64_t t0 = imin64(imax64(0, -p0), a.m);
    count = (unsigned)imax64(0, imin64(len, a.n - p0) - t0);
    tok = row * a.ncap + p0 + t0;
    x = b * a.sb[half] + h * a.sh[half] + t0 * a.st[half] + 8 * l;
  }
  __device__ __forceinline__ bool in(unsigned i) const { return i < count; }
};

__global__ void __launch_bounds__(32 * kKvWarps) kv4_write_kernel(const KvMoveArgs a) {
  kv4_wait_prior();
  const KvLane L(a);
  const bool asked = a.x[L.half] != nullptr;
  const int64_t st = a.st[L.half];
  const uint16_t* src = a.x[L.half] + L.x + L.t * st;
  uint32_t* code = reinterpret_cast<uint32_t*>(a.code[L.half] + (L.tok + L.t) * kKv4Row) +
                   2 * (L.l & 7) + (L.l >> 3);
  uint32_t* scale = reinterpret_cast<uint32_t*>(a.scale + (L.tok + L.t) * kKv4Scales) +
                    2 * L.half + (L.l >> 3);
  uint4 next[kKvRun];
  auto fetch = [&](unsigned t) {
#pragma unroll
    for (int k = 0; k < kKvRun; ++k)
      next[k] = asked && L.in(t + k) ? __ldcs(reinterpret_cast<const uint4*>(src + k * st))
                                     : make_uint4(0u, 0u, 0u, 0u);
  };
  const unsigned step = gridDim.x * kKvStep;
  fetch(L.t);
  for (unsigned t = L.t, left; t < L.count; t = left > step ? t + step : L.count) {
    left = L.count - t;  // the same for both halves
    uint4 cur[kKvRun];
#pragma unroll
    for (int k = 0; k < kKvRun; ++k) cur[k] = next[k];
    src += step * st;
    if (left > step) fetch(t + step);
#pragma unroll
    for (int k = 0; k < kKvRun; ++k) {
      const uint4 w = cur[k];
      // (min, -max) in the halves of one word, then over the group's eight lanes
      const uint32_t mn = min2_nan(min2_nan(w.x, w.y), min2_nan(w.z, w.w));
      const uint32_t mx = max2_nan(max2_nan(w.x, w.y), max2_nan(w.z, w.w)) ^ 0x80008000u;
      uint32_t r = min2_nan(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) r = min2_nan(r, __shfl_xor_sync(0xFFFFFFFFu, r, o));
      const float lo = bf16_lo(r), s = kv4_step(lo, -bf16_hi(r));
      uint32_t sm = __byte_perm(__float_as_uint(s), r, 0x5432);
      uint32_t word = kv4_word(w, lo, s, s > 0.0f ? kv4_rcp(s) : 0.0f);
      if (s != s) {  // a value that is not finite: the group reads as NaN
        sm = kKv4NanPair;
        word = 0;
      }
      if (asked && L.in(t + k)) {
        code[k * (kKv4Row / 4)] = word;
        if ((L.l & 7) == 0) scale[k * (kKv4Scales / 2)] = sm;
      }
    }
    code += (int64_t)step * (kKv4Row / 4);
    scale += (int64_t)step * (kKv4Scales / 2);
  }
}

__global__ void __launch_bounds__(32 * kKvWarps) kv4_read_kernel(const KvMoveArgs a) {
  kv4_wait_prior();
  const KvLane L(a);
  const int64_t st = a.st[L.half];
  uint16_t* dst = a.x[L.half] + L.x + L.t * st;
  const uint32_t* code =
      reinterpret_cast<const uint32_t*>(a.code[L.half] + (L.tok + L.t) * kKv4Row) +
      2 * (L.l & 7) + (L.l >> 3);
  const uint32_t* scale =
      reinterpret_cast<const uint32_t*>(a.scale + (L.tok + L.t) * kKv4Scales) + 2 * L.half +
      (L.l >> 3);
  if (!a.x[L.half]) return;  // whole half-warps, which work alone
  uint32_t nw[kKvRun], ns[kKvRun];
  auto fetch = [&](unsigned t) {
#pragma unroll
    for (int k = 0; k < kKvRun; ++k) {
      const bool ok = L.in(t + k);
      nw[k] = ok ? __ldcs(code + k * (kKv4Row / 4)) : 0u;
      ns[k] = ok ? __ldcs(scale + k * (kKv4Scales / 2)) : 0u;
    }
  };
  const unsigned step = gridDim.x * kKvStep;
  fetch(L.t);
  for (unsigned t = L.t, left; t < L.count; t = left > step ? t + step : L.count) {
    left = L.count - t;
    uint32_t cw[kKvRun], cs[kKvRun];
#pragma unroll
    for (int k = 0; k < kKvRun; ++k) {
      cw[k] = nw[k];
      cs[k] = ns[k];
    }
    code += (int64_t)step * (kKv4Row / 4);
    scale += (int64_t)step * (kKv4Scales / 2);
    if (left > step) fetch(t + step);
#pragma unroll
    for (int k = 0; k < kKvRun; ++k) {
      if (!L.in(t + k)) continue;
      const float s = bf16_lo(cs[k]), m = bf16_hi(cs[k]);
      uint4 o;
      o.x = kv4_pair(cw[k], 0, s, m);
      o.y = kv4_pair(cw[k], 8, s, m);
      o.z = kv4_pair(cw[k], 16, s, m);
      o.w = kv4_pair(cw[k], 24, s, m);
      *reinterpret_cast<uint4*>(dst + k * st) = o;
    }
    dst += step * st;
  }
}

}  // namespace

int launch_kv4_move(bool write, const Dims& s, const sd_kv4& c, void* K, const sd_strides& ks,
                    void* V, const sd_strides& vs, int64_t m, int64_t first, const int32_t* pos,
                    const int32_t* length, cudaStream_t st) {
  KvMoveArgs a;
  a.x[0] = (uint16_t*)K;
  a.x[1] = (uint16_t*)V;
  const sd_strides* str[2] = {&ks, &vs};
  for (int i = 0; i < 2; ++i) {
    a.sb[i] = str[i]->seq;
    a.sh[i] = str[i]->head;
    a.st[i] = str[i]->token;
  }
  a.code[0] = c.k;
  a.code[1] = c.v;
  a.scale = c.scale;
  a.hkv = s.Hkv;
  a.n = s.n;
  a.ncap = s.ncap;
  a.m = m;
  a.first = first;
  a.pos = pos;
  a.length = length;
  // a few steps per CTA where there are many tokens: four waves of the GPU
  const int64_t rows = (int64_t)s.B * s.Hkv, steps = (m + kKvStep - 1) / kKvStep;
  const int64_t waves = imax64(1, (int64_t)device_sm_count() * 32 / rows);
  const dim3 grid((unsigned)imin64(steps, waves), (unsigned)rows);
  return write ? kv4_launch("kv4 write", kv4_write_kernel, grid, 32 * kKvWarps, 0, 0, st, a)
               : kv4_launch("kv4 read", kv4_read_kernel, grid, 32 * kKvWarps, 0, 0, st, a);
}

}  // namespace sd
