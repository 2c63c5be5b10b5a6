// Softmax attention over ranges of the bf16 cache (HashAttention: Semantic Sparsity for
// Faster Inference, 2.1, the attention that the sparse step approximates; 3.1, the first and
// the latest tokens kept): a window with first tokens, and a prefix that a batch shares.
//
// A warp takes a query row and walks the tokens that it sees, one softmax over them.
#include "sd_dense.cuh"

namespace sd {
namespace {

struct DnArgs {
  const uint16_t* q;
  const uint16_t* K;
  const uint16_t* V;
  const uint16_t* Kp;
  const uint16_t* Vp;
  uint16_t* out;
  float* lse;
  sd_strides qs, os;
  DnWindow w;
  int B, Hq, Hkv, G;
  int64_t ncap, p, pcap;
  const int32_t* end;
  float sl2;
};

__global__ void __launch_bounds__(128) window_rows_kernel(DnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (i >= (int64_t)a.B * a.Hq * a.w.m) return;
  const int64_t t = i % a.w.m;
  const int h = (int)(i / a.w.m % a.Hq), b = (int)(i / a.w.m / a.Hq);
  if (t >= a.w.len(b)) return;
  const int64_t p = a.w.at(b) + t;
  const DnRanges r = dn_ranges(a.w, p, p);
  const int64_t base = ((int64_t)b * a.Hkv + h / a.G) * a.ncap * kD;
  DnRow x;
  dn_row_begin(x, a.q + b * a.qs.seq + h * a.qs.head + t * a.qs.token, a.sl2, lane);
  dn_row_over(x, a.K + base, a.V + base, 0, r.s1, lane);
  dn_row_over(x, a.K + base, a.V + base, r.w0, r.w1, lane);
  dn_row_end(x, a.out + b * a.os.seq + h * a.os.head + t * a.os.token,
             a.lse ? a.lse + ((int64_t)b * a.Hq + h) * a.w.m + t : nullptr, lane);
}

__global__ void __launch_bounds__(128) prefix_rows_kernel(DnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (i >= (int64_t)a.B * a.Hq) return;
  const int h = (int)(i % a.Hq), b = (int)(i / a.Hq);
  const int64_t base = ((int64_t)b * a.Hkv + h / a.G) * a.ncap * kD;
  const int64_t pre = (int64_t)(h / a.G) * a.pcap * kD;
  const int64_t own = !a.K ? 0 : a.end ? imin64(a.w.n, a.end[b]) : a.w.n;
  DnRow x;
  dn_row_begin(x, a.q + i * kD, a.sl2, lane);
  dn_row_over(x, a.Kp + pre, a.Vp + pre, 0, a.p, lane);
  dn_row_over(x, a.K + base, a.V + base, 0, own, lane);
  dn_row_end(x, a.out + i * kD, a.lse ? a.lse + i : nullptr, lane);
}

}  // namespace

size_t window_attend_workspace_bytes(const Dims&, int64_t, int64_t, int64_t) { return 0; }

int launch_window_attend(const Dims& s, const uint16_t* q, const sd_strides& qs,
                         const uint16_t* K, const uint16_t* V, int64_t m, int64_t first,
                         const int32_t* pos, const int32_t* length, int64_t window, int64_t sink,
                         float scale, uint16_t* out, const sd_strides& os, float* lse, void* ws,
                         cudaStream_t st) {
  DnArgs a = {};
  a.q = q, a.K = K, a.V = V, a.out = out, a.lse = lse, a.qs = qs, a.os = os;
  a.w = DnWindow{pos, length, first, m, s.n, window, sink};
  a.B = s.B, a.Hq = s.Hq, a.Hkv = s.Hkv, a.G = s.G, a.ncap = s.ncap, a.sl2 = scale * kDnLog2e;
  const int64_t rows = (int64_t)s.B * s.Hq * m;
  window_rows_kernel<<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(a);
  note_launches(1);
  return check_launch("window attention");
}

size_t prefix_attend_workspace_bytes(const Dims&, int64_t) { return 0; }

int launch_prefix_attend(const Dims& s, const uint16_t* q, const uint16_t* Kp,
                         const uint16_t* Vp, int64_t p, int64_t pcap, const uint16_t* K,
                         const uint16_t* V, const int32_t* end, float scale, uint16_t* out,
                         float* lse, void* ws, cudaStream_t st) {
  DnArgs a = {};
  a.q = q, a.K = K, a.V = V, a.Kp = Kp, a.Vp = Vp, a.out = out, a.lse = lse;
  a.B = s.B, a.Hq = s.Hq, a.Hkv = s.Hkv, a.G = s.G, a.ncap = s.ncap, a.sl2 = scale * kDnLog2e;
  a.p = p, a.pcap = pcap, a.end = end, a.w.n = s.n;
  const int64_t rows = (int64_t)s.B * s.Hq;
  prefix_rows_kernel<<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(a);
  note_launches(1);
  return check_launch("prefix attention");
}

}  // namespace sd
