// Decode attention of one query token per sequence over ranges of its bf16 cache
// (HashAttention: Semantic Sparsity for Faster Inference, 2.1; 3.1, the first and the latest
// tokens kept): single tokens under a window with first tokens, and a sequence's own tokens
// behind a prefix that the batch shares.
//
// Bound by HBM: 512 bytes a token and KV head against 4 G products of 128.  A row, a
// (sequence, KV head) pair, is cut into `parts` CTAs of four warps; warp w takes every fourth
// group of 16 tokens.  Warps work alone: each keeps a ring of kSwStages groups in shared
// memory, filled by 16-byte asynchronous copies (chunks XOR-swizzled by token, so that the
// matrix loads meet no bank twice), 16 KB of a warp in flight, which 8 warps of an SM make
// 128 KB.  S = Q K^T as m16n8k16 bf16 products (M: the group's heads), p = 2^(s - m) in fp32
// with the reference m raised only when a group's maximum exceeds it by more than 2^8, O^T +=
// V^T P^T with p as two bf16 parts (16 bits of it: the products have time to spare) and V^T
// read by transposing matrix loads (dn_eight_step, sd_dense.cuh).
//
// Measured: 64 x 8 rows of up to 4,224 tokens 140 us (7.0 TB/s; a part stays in L2 between
// passes), 64 x 8 of 1,152 with cold caches 49 us (6.2 TB/s, 92 % of the copy rate); 8 rows of
// 1,152 5.7 us, 8 of 32,768 31.6 us (4.2 TB/s: 38 CTAs a row and a kernel that joins them).
//
// Warps of a CTA join through shared memory, CTAs of a row through the cluster's (up to
// eight), longer cuts through a workspace (dense_join_kernel).  A prefix's partial results
// (sd_dense_tile.cu) join in the same place.
#include <atomic>

#include "sd_dense.cuh"

namespace sd {
namespace {

constexpr int kSwThreads = 32 * kSwCtaWarps;
constexpr int kSwStages = 3;
constexpr size_t kSwSmem = (size_t)kSwCtaWarps * kSwStages * kDnStage;  // 96 KB
constexpr float kSwSlack = 8.0f;

struct SwArgs {
  const uint16_t* q;
  const uint16_t* K;
  const uint16_t* V;
  uint16_t* out;
  float* lse;
  float* part_o;      // cut through the workspace: [row][head][parts][d], not divided by l
  float2* part_ml;
  const float* pre_o; // a prefix's parts: [KV head][sequence][head][pre][d]
  const float2* pre_ml;
  int pre;
  int64_t qseq, qhead, oseq, ohead;
  DnWindow w;
  const int32_t* end; // own tokens [0, min(end, n)) instead of a window (own = 1)
  int own;
  int B, Hkv, parts, cut;  // cut: parts joined by dense_join_kernel
  int64_t ncap;
  float sl2;
};

__device__ __forceinline__ uint32_t sw_rank_addr(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 sw_ld_rank2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float4 sw_ld_rank4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sw_cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;\n" ::
          : "memory");
}

// A softmax's state that a warp holds for one head: lane l channels 4l .. 4l + 3.
struct SwHead {
  float top, sum;
  float4 o;
  __device__ __forceinline__ void add(float m, float l, const float4& x, float mu) {
    const float f = exp2f(m - mu);
    sum = fmaf(l, f, sum);
    o.x = fmaf(x.x, f, o.x);
    o.y = fmaf(x.y, f, o.y);
    o.z = fmaf(x.z, f, o.z);
    o.w = fmaf(x.w, f, o.w);
  }
};
__device__ __forceinline__ SwHead sw_head(float top) {
  return SwHead{top, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
}
__device__ __forceinline__ float sw_ref(float top) { return top == -INFINITY ? 0.0f : top; }

// Joins the prefix's parts to a head and writes out and lse.
template <int G>
__device__ __forceinline__ void sw_finish(const SwArgs& a, SwHead x, int b, int h, int g, int lane) {
  if (a.pre) {
    const int64_t pr = (((int64_t)h * a.B + b) * G + g) * a.pre;
    float top = x.top;
    for (int s = lane; s < a.pre; s += 32) top = fmaxf(top, a.pre_ml[pr + s].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float mu = sw_ref(top);
    SwHead y = sw_head(top);
    y.add(x.top, x.sum, x.o, mu);
    for (int s0 = 0; s0 < a.pre; s0 += 32) {
      float2 ml = make_float2(-INFINITY, 0.0f);
      if (s0 + lane < a.pre) ml = a.pre_ml[pr + s0 + lane];
      const int n = min(32, a.pre - s0);
#pragma unroll 8
      for (int s = 0; s < n; ++s) {
        const float4 v = reinterpret_cast<const float4*>(a.pre_o + (pr + s0 + s) * kD)[lane];
        y.add(__shfl_sync(0xFFFFFFFFu, ml.x, s), __shfl_sync(0xFFFFFFFFu, ml.y, s), v, mu);
      }
    }
    x = y;
  }
  const int head = h * G + g;
  const float inv = x.sum == 0.0f ? 0.0f : 1.0f / x.sum;
  *reinterpret_cast<uint2*>(a.out + b * a.oseq + head * a.ohead + 4 * lane) =
      make_uint2(bf16_pack(x.o.x * inv, x.o.y * inv), bf16_pack(x.o.z * inv, x.o.w * inv));
  if (a.lse && lane == 0)
    a.lse[(int64_t)b * a.Hkv * G + head] =
        x.sum == 0.0f ? -INFINITY : (x.top + log2f(x.sum)) * kDnLn2;
}

template <int G>
__global__ void __launch_bounds__(kSwThreads, 2) dense_stream_kernel(SwArgs a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float2 wml[kSwCtaWarps][8];  // a warp's (m, l) of each head
  __shared__ __align__(16) float2 cml[8];    // the CTA's
  __shared__ __align__(16) float co[8][kD];  // and its O
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const bool real = gid < G;
  const int64_t row = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - row * a.parts);
  const int b = (int)(row / a.Hkv), h = (int)(row - (int64_t)b * a.Hkv);

  DnRanges r;
  if (a.own) {
    r = DnRanges{0, 0, a.end ? imax64(0, imin64(a.w.n, a.end[b])) : a.w.n};
  } else {
    if (a.w.len(b) < 1) return;  // every CTA of the row
    const int64_t p = a.w.at(b);
    r = dn_ranges(a.w, p, p);
  }
  const int na = (int)((r.s1 + kSwGroup - 1) / kSwGroup);
  const int all = na + (int)((r.w1 - r.w0 + kSwGroup - 1) / kSwGroup);
  const int g0 = (int)((int64_t)all * part / a.parts) + warp;
  const int g1 = (int)((int64_t)all * (part + 1) / a.parts);

  const uint32_t mine = dn_su32(ring) + warp * kSwStages * kDnStage;
  const int64_t base = row * a.ncap * kD;
  auto group = [&](int i, int& have) {  // its first token
    const int64_t c0 = i < na ? (int64_t)i * kSwGroup : r.w0 + (int64_t)(i - na) * kSwGroup;
    have = (int)imin64(kSwGroup, (i < na ? r.s1 : r.w1) - c0);
    return c0;
  };
  auto fetch = [&](int i, int slot) {
    if (i < g1) {
      int have;
      const int64_t c0 = group(i, have);
      dn_fetch(mine + slot * kDnStage, a.K, a.V, base + c0 * kD, have, lane);
    }
    dn_cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kSwStages - 1; ++s) fetch(g0 + s * kSwCtaWarps, s);

  uint32_t qa[8][2];
  {
    const uint32_t* q =
        reinterpret_cast<const uint32_t*>(a.q + b * a.qseq + (h * G + (real ? gid : 0)) * a.qhead);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      qa[kk][0] = real ? q[8 * kk + tig] : 0u;
      qa[kk][1] = real ? q[8 * kk + 4 + tig] : 0u;
    }
  }
  DnEight x;
  dn_eight_begin(x);
  int slot = 0;
  for (int i = g0; i < g1; i += kSwCtaWarps) {
    __syncwarp();  // the slot filled next is read by all
    fetch(i + (kSwStages - 1) * kSwCtaWarps, slot == 0 ? kSwStages - 1 : slot - 1);
    dn_cp_wait<kSwStages - 1>();
    __syncwarp();
    int have;
    group(i, have);
    dn_eight_step(x, qa, mine + slot * kDnStage, have, real, a.sl2, kSwSlack, lane);
    slot = slot == kSwStages - 1 ? 0 : slot + 1;
  }
  dn_cp_wait<0>();
  // behind a prefix's kernel every CTA waits for it, also where a later kernel joins the
  // parts: that one waits for this kernel only
  if (a.pre) dn_wait_prior();

  // the warp's (m, l, O) into its own part of the ring
  dn_eight_end(x, reinterpret_cast<float*>(ring + warp * kSwStages * kDnStage), G, lane);
  if (tig == 0) wml[warp][gid] = make_float2(x.m, x.l);
  __syncthreads();
  const bool joined = a.parts > 1 && !a.cut;
  const float* all_o = reinterpret_cast<const float*>(ring);
  constexpr int kStep = kSwStages * kDnStage / sizeof(float);
  for (int g = warp; g < G; g += kSwCtaWarps) {  // a warp per head
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSwCtaWarps; ++w) top = fmaxf(top, wml[w][g].x);
    SwHead x = sw_head(top);
#pragma unroll
    for (int w = 0; w < kSwCtaWarps; ++w)
      x.add(wml[w][g].x, wml[w][g].y,
            reinterpret_cast<const float4*>(all_o + w * kStep + g * kD)[lane], sw_ref(top));
    if (a.cut) {
      const int64_t at = (row * G + g) * a.parts + part;
      reinterpret_cast<float4*>(a.part_o + at * kD)[lane] = x.o;
      if (lane == 0) a.part_ml[at] = make_float2(x.top, x.sum);
    } else if (joined) {
      reinterpret_cast<float4*>(co[g])[lane] = x.o;
      if (lane == 0) cml[g] = make_float2(x.top, x.sum);
    } else {
      sw_finish<G>(a, x, b, h, g, lane);
    }
  }
  if (!joined) return;
  sw_cluster_sync();
  // each CTA of the row finishes its share of the heads
  const uint32_t ml_at = dn_su32(cml), o_at = dn_su32(co);
  for (int g = part + a.parts * warp; g < G; g += a.parts * kSwCtaWarps) {
    const float2 mine2 =
        lane < a.parts ? sw_ld_rank2(sw_rank_addr(ml_at + 8 * g, lane)) : make_float2(-INFINITY, 0.0f);
    float top = mine2.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    SwHead x = sw_head(top);
#pragma unroll 8
    for (int s = 0; s < a.parts; ++s)
      x.add(__shfl_sync(0xFFFFFFFFu, mine2.x, s), __shfl_sync(0xFFFFFFFFu, mine2.y, s),
            sw_ld_rank4(sw_rank_addr(o_at + 4 * (g * kD + 4 * lane), s)), sw_ref(top));
    sw_finish<G>(a, x, b, h, g, lane);
  }
  sw_cluster_sync();  // the others' shared memory is read
}

// The largest cluster that this device runs of the kernel (cached per device).
template <int G>
int sw_max_cluster() {
  static std::atomic<int> most[kMaxDev];
  return per_device_cached(most, [] {
    if (set_smem_limit((const void*)dense_stream_kernel<G>, kSwSmem, "stream attention") != SD_OK)
      return 0;
    int c = 8;
    for (; c > 1; c >>= 1) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(c, 1, 1);
      cfg.blockDim = dim3(kSwThreads, 1, 1);
      cfg.dynamicSmemBytes = kSwSmem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = c;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int nc = 0;
      if (cudaOccupancyMaxActiveClusters(&nc, dense_stream_kernel<G>, &cfg) == cudaSuccess &&
          nc > 0)
        break;
      cudaGetLastError();
    }
    return c;
  });
}

template <int G>
int sw_launch(SwArgs& a, int64_t tokens, float* cut_o, float2* cut_ml, int* cut,
              cudaStream_t st) {
  const int64_t rows = (int64_t)a.B * a.Hkv;
  const SwPlan p = sw_plan(rows, tokens, device_sm_count(),
                           fallback_forced() ? 1 : sw_max_cluster<G>());
  a.parts = p.parts;
  a.cut = p.cut;
  if (p.cut) {
    a.part_o = cut_o;
    a.part_ml = cut_ml;
  }
  *cut = p.cut ? p.parts : 0;
  if (int rc = set_smem_limit((const void*)dense_stream_kernel<G>, kSwSmem, "stream attention"))
    return rc;
  // behind a prefix's kernel: started while it ends
  return dn_launch_early("stream attention", dense_stream_kernel<G>, (unsigned)(rows * p.parts),
                         kSwThreads, kSwSmem, p.parts > 1 && !p.cut ? p.parts : 0, st, a,
                         a.pre > 0);
}

int sw_dispatch(SwArgs& a, int G, int64_t tokens, float* cut_o, float2* cut_ml, int* cut,
                cudaStream_t st) {
  switch (G) {
    case 1: return sw_launch<1>(a, tokens, cut_o, cut_ml, cut, st);
    case 2: return sw_launch<2>(a, tokens, cut_o, cut_ml, cut, st);
    case 4: return sw_launch<4>(a, tokens, cut_o, cut_ml, cut, st);
    default: return sw_launch<8>(a, tokens, cut_o, cut_ml, cut, st);
  }
}

}  // namespace

int64_t window_stream_parts(const Dims& s, int64_t tokens) {
  return (int64_t)s.B * s.Hq * sw_cut((int64_t)s.B * s.Hkv, tokens, device_sm_count());
}

// One query token per sequence: under the window, or (own) over [0, min(end, n)) with a
// prefix's parts joined in.  tokens: what a row may see.  *cut: parts left for
// dense_join_kernel in cut_o, cut_ml (0: out and lse are written).
int launch_window_stream(const Dims& s, const uint16_t* q, const sd_strides& qs,
                         const uint16_t* K, const uint16_t* V, const DnWindow& w, bool own,
                         const int32_t* end, int64_t tokens, float scale, const float* pre_o,
                         const float2* pre_ml, int pre, uint16_t* out, const sd_strides& os,
                         float* lse, float* cut_o, float2* cut_ml, int* cut, cudaStream_t st) {
  SwArgs a = {};
  a.q = q, a.K = K, a.V = V, a.out = out, a.lse = lse;
  a.pre_o = pre_o, a.pre_ml = pre_ml, a.pre = pre;
  a.qseq = qs.seq, a.qhead = qs.head, a.oseq = os.seq, a.ohead = os.head;
  a.w = w, a.own = own, a.end = end, a.B = s.B, a.Hkv = s.Hkv, a.ncap = s.ncap;
  a.sl2 = scale * kDnLog2e;
  return sw_dispatch(a, s.G, tokens, cut_o, cut_ml, cut, st);
}

}  // namespace sd
