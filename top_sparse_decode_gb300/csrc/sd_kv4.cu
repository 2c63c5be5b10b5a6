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

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// What a lane moves: its half (0: K, 1: V), octet and row, and the tokens' range.
struct KvLane {
  int half, l;
  int64_t row, t, len, p0, x;  // x: offset of the lane's octet of token 0 in the caller's array
  __device__ __forceinline__ KvLane(const KvMoveArgs& a) {
    const int lane = threadIdx.x & 31;
    half = lane >> 4;
    l = lane & 15;
    row = blockIdx.y;
    const int b = (int)(row / a.hkv), h = (int)(row % a.hkv);
    kv_range(a, b, len, p0);
    t = (int64_t)blockIdx.x * kKvStep + (threadIdx.x >> 5) * kKvRun;
    // tokens [t, len) whose positions lie in the cache, of a half that is asked for
    len = a.x[half] ? imin64(len, a.n - p0) : 0;
    x = b * a.sb[half] + h * a.sh[half] + 8 * l;
  }
  __device__ __forceinline__ bool in(int64_t i) const { return i < len && p0 + i >= 0; }
};

__global__ void __launch_bounds__(32 * kKvWarps) kv4_write_kernel(const KvMoveArgs a) {
  KvLane L(a);
  const uint16_t* src = a.x[L.half] + L.x;
  const int64_t base = L.row * a.ncap + L.p0, st = a.st[L.half];
  uint32_t* code = reinterpret_cast<uint32_t*>(a.code[L.half]) + 2 * (L.l & 7) + (L.l >> 3);
  uint32_t* scale = reinterpret_cast<uint32_t*>(a.scale) + 2 * L.half + (L.l >> 3);
  uint4 next[kKvRun];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int k = 0; k < kKvRun; ++k)
      next[k] = L.in(t + k) ? __ldcs(reinterpret_cast<const uint4*>(src + (t + k) * st))
                            : make_uint4(0u, 0u, 0u, 0u);
  };
  const int64_t step = (int64_t)gridDim.x * kKvStep;
  const int64_t most = a.length ? imin64(a.m, a.length[L.row / a.hkv]) : a.m;  // both halves'
  fetch(L.t);
  for (int64_t t = L.t; t < most; t += step) {
    uint4 cur[kKvRun];
#pragma unroll
    for (int k = 0; k < kKvRun; ++k) cur[k] = next[k];
    fetch(t + step);
#pragma unroll
    for (int k = 0; k < kKvRun; ++k) {
      const uint4 w = cur[k];
      float lo = min_nan(min_nan(min_nan(bf16_lo(w.x), bf16_hi(w.x)), min_nan(bf16_lo(w.y), bf16_hi(w.y))),
                         min_nan(min_nan(bf16_lo(w.z), bf16_hi(w.z)), min_nan(bf16_lo(w.w), bf16_hi(w.w))));
      float hi = fmax_nan(fmax_nan(fmax_nan(bf16_lo(w.x), bf16_hi(w.x)), fmax_nan(bf16_lo(w.y), bf16_hi(w.y))),
                          fmax_nan(fmax_nan(bf16_lo(w.z), bf16_hi(w.z)), fmax_nan(bf16_lo(w.w), bf16_hi(w.w))));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        hi = fmax_nan(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
      }
      const float s = kv4_step(lo, hi);
      uint32_t sm = (__float_as_uint(s) >> 16) | (__float_as_uint(lo) & 0xFFFF0000u);
      uint32_t word = kv4_word(w, lo, s, s > 0.0f ? __frcp_rn(s) : 0.0f);
      if (s != s) {  // a value that is not finite: the group reads as NaN
        sm = kKv4NanPair;
        word = 0;
      }
      if (L.in(t + k)) {
        const int64_t tok = base + t + k;
        code[tok * (kKv4Row / 4)] = word;
        if ((L.l & 7) == 0) scale[tok * (kKv4Scales / 2)] = sm;
      }
    }
  }
}

__global__ void __launch_bounds__(32 * kKvWarps) kv4_read_kernel(const KvMoveArgs a) {
  KvLane L(a);
  uint16_t* dst = a.x[L.half] + L.x;
  const int64_t base = L.row * a.ncap + L.p0, st = a.st[L.half];
  const uint32_t* code =
      reinterpret_cast<const uint32_t*>(a.code[L.half]) + 2 * (L.l & 7) + (L.l >> 3);
  const uint32_t* scale = reinterpret_cast<const uint32_t*>(a.scale) + 2 * L.half + (L.l >> 3);
  uint32_t nw[kKvRun], ns[kKvRun];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int k = 0; k < kKvRun; ++k) {
      const bool ok = L.in(t + k);
      const int64_t tok = base + t + k;
      nw[k] = ok ? __ldcs(code + tok * (kKv4Row / 4)) : 0u;
      ns[k] = ok ? __ldcs(scale + tok * (kKv4Scales / 2)) : 0u;
    }
  };
  const int64_t step = (int64_t)gridDim.x * kKvStep;
  fetch(L.t);
  for (int64_t t = L.t; t < L.len; t += step) {
    uint32_t cw[kKvRun], cs[kKvRun];
#pragma unroll
    for (int k = 0; k < kKvRun; ++k) {
      cw[k] = nw[k];
      cs[k] = ns[k];
    }
    fetch(t + step);
#pragma unroll
    for (int k = 0; k < kKvRun; ++k) {
      if (!L.in(t + k)) continue;
      const float s = bf16_lo(cs[k]), m = bf16_hi(cs[k]);
      uint4 o;
      o.x = kv4_pair(cw[k], 0, s, m);
      o.y = kv4_pair(cw[k], 8, s, m);
      o.z = kv4_pair(cw[k], 16, s, m);
      o.w = kv4_pair(cw[k], 24, s, m);
      *reinterpret_cast<uint4*>(dst + (t + k) * st) = o;
    }
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
  if (write)
    kv4_write_kernel<<<grid, 32 * kKvWarps, 0, st>>>(a);
  else
    kv4_read_kernel<<<grid, 32 * kKvWarps, 0, st>>>(a);
  note_launches(1);
  return check_launch(write ? "kv4 write" : "kv4 read");
}

}  // namespace sd
