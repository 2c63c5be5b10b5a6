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
// One warp per token: lanes 0..15 its K row, lanes 16..31 its V row, 8 channels (one
// 16-byte load, one 32-bit word of codes) per lane, 8 lanes per group.
#include "sd_internal.cuh"
#include "sd_kv4.cuh"

namespace sd {
namespace {

constexpr int kKvWarps = 8;

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

__global__ void __launch_bounds__(32 * kKvWarps) kv4_write_kernel(const KvMoveArgs a) {
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int row = blockIdx.y, b = row / a.hkv, h = row % a.hkv;
  int64_t len, p0;
  kv_range(a, b, len, p0);
  const int64_t t = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  const int64_t p = p0 + t;
  if (t >= len || p < 0 || p >= a.n || !a.x[half]) return;  // whole half-warps
  const unsigned mask = half ? 0xFFFF0000u : 0x0000FFFFu;
  const uint4 w = *reinterpret_cast<const uint4*>(a.x[half] + b * a.sb[half] + h * a.sh[half] +
                                                  t * a.st[half] + 8 * l);
  const float x[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y),
                      bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = fmax_nan(hi, x[i]);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(mask, lo, o));
    hi = fmax_nan(hi, __shfl_xor_sync(mask, hi, o));
  }
  uint32_t sm, word = 0;
  const float s = kv4_step(lo, hi);
  if (s != s) {
    sm = kKv4NanPair;  // a value that is not finite: the group reads as NaN
  } else {
    sm = (__float_as_uint(s) >> 16) | (__float_as_uint(lo) & 0xFFFF0000u);
    const float y = s > 0.0f ? __frcp_rn(s) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) word |= kv4_code(x[i] - lo, s, y) << (4 * i);
  }
  const int64_t tok = (int64_t)row * a.ncap + p;
  reinterpret_cast<uint32_t*>(a.code[half] + tok * kKv4Row)[2 * (l & 7) + (l >> 3)] = word;
  if ((l & 7) == 0)
    reinterpret_cast<uint32_t*>(a.scale + tok * kKv4Scales)[2 * half + (l >> 3)] = sm;
}

__global__ void __launch_bounds__(32 * kKvWarps) kv4_read_kernel(const KvMoveArgs a) {
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int row = blockIdx.y, b = row / a.hkv, h = row % a.hkv;
  int64_t len, p0;
  kv_range(a, b, len, p0);
  const int64_t t = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
  const int64_t p = p0 + t;
  if (t >= len || p < 0 || p >= a.n || !a.x[half]) return;
  const int64_t tok = (int64_t)row * a.ncap + p;
  const uint32_t word =
      reinterpret_cast<const uint32_t*>(a.code[half] + tok * kKv4Row)[2 * (l & 7) + (l >> 3)];
  const uint32_t sm =
      reinterpret_cast<const uint32_t*>(a.scale + tok * kKv4Scales)[2 * half + (l >> 3)];
  const float s = bf16_lo(sm), m = bf16_hi(sm);
  uint4 o;
  o.x = kv4_pair(word, 0, s, m);
  o.y = kv4_pair(word, 8, s, m);
  o.z = kv4_pair(word, 16, s, m);
  o.w = kv4_pair(word, 24, s, m);
  *reinterpret_cast<uint4*>(a.x[half] + b * a.sb[half] + h * a.sh[half] + t * a.st[half] +
                            8 * l) = o;
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
  const int64_t warps = imin64(m, kKvWarps);
  const dim3 grid((unsigned)((m + warps - 1) / warps), (unsigned)(s.B * s.Hkv));
  if (write)
    kv4_write_kernel<<<grid, 32 * kKvWarps, 0, st>>>(a);
  else
    kv4_read_kernel<<<grid, 32 * kKvWarps, 0, st>>>(a);
  note_launches(1);
  return check_launch(write ? "kv4 write" : "kv4 read");
}

}  // namespace sd
