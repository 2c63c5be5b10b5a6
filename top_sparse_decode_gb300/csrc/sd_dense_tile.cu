// Softmax attention of many query rows over ranges of the bf16 cache on the 5th-generation
// tensor cores (HashAttention: Semantic Sparsity for Faster Inference, 2.1, the attention
// over every cached token; 3.1, the first and the latest tokens kept): prompts and chunks
// under a window with first tokens, and a batch's rows over the prefix that it shares.
//
// Rows.  A KV head's query heads share its K and V, so a row is a (token, head of the group)
// pair, token by token: 256 rows, two tiles of 128, span 256 / G tokens, and what they see is
// little more than the window.  A work item is two row tiles against the token tiles that
// any of their rows sees -- [0, s1) and [w0, w1), each cut into tiles of 128 from its start
// (a TMA load may start at any token) -- or a part of these, whose results join later.  With
// at most 128 rows (`dual`) both softmax groups take the same rows and every second token
// tile each, so that one's softmax hides behind the other's products.
//
// Per token tile and row tile: S = Q K^T (128 x 128 x 128, both operands from shared memory,
// fp32 in tensor memory), p = 2^(s - m) by the softmax group whose thread owns the row, p
// rounded to bf16 into the columns that S held, O += P V (P from tensor memory, V as it
// lies), by halves of 64 tokens: the first half's product runs beside the second half's
// weights.  The rounding of p costs as much as that of the bf16 result (out is 1.4 times as
// far from 64 bits, up to 1.6); l and lse are of the sums before it.  A second product with
// what it cut off (both parts in the columns of S) took that error away and cost every prompt:
// 32,768 tokens under a window of 4,096 2,117 us (1,546 without), 4 x 4,096 causal 588 (447),
// 3 x 257 21.5 (18.5), a prefix of 131,072 for 128 294 (229).
//
// The reference m begins at 0 and stands as long as half a tile's weights sum up to 2^14 at
// most and a row's so far to 2^-40 at least: a weight's rounding is relative to itself, so any
// m in that range is as good as the maximum, which is then not sought (it took 400 of a
// tile's 2,800 cycles).  Where it does not stand, the half's maximum is sought, m set to the
// whole number above it, and O and l moved by a power of two, exactly (tl_fit).
//
// Roles (384 threads, one CTA per SM, persistent over items): warps 0-3 and 4-7 softmax and
// output of the two row tiles, warp 8 issues the products, warp 9 the TMA loads, warps 10
// and 11 load Q.  Products are issued PV(0), QK(0) of the next tile, PV(1), QK(1): while one
// group's scores are in its softmax the tensor cores work for the other.  S and P share
// columns: QK of the next tile follows PV of this one in the tensor cores' queue.
//
// Shared memory: Q 64 KB, a ring of five 32 KB stages for K and V tiles, all in the 128-byte
// swizzle that the TMA writes.  Tensor memory: S 2 x 128 and O 2 x 128 columns, all 512.
//
// What a row does not see reaches nothing of it: scores by selection; V rows of a tile that no
// row sees, behind the first tokens or a sequence's last row, come as zeros or are set to zero
// in shared memory; and a row whose O comes out not finite, as from a weight of 0 times an
// infinity that the row does not see and others of its tile do (0 x inf is not 0), is computed
// again when the CTA's items are done (tl_again).
//
// What bounds it: the chain of a row tile, whose scores' product, two halves of softmax and
// product with V follow each other; two row tiles in flight keep the tensor pipe busy for some
// 60 % of the cycles.  32,768 tokens of 32 heads, window 4,096: 1,549 us, 1.37 PFLOP/s, 72 %
// of the measured bf16 rate; 4 x 4,096 tokens causal: 447 us, 64 % (items go to CTAs by a fixed
// stride from the largest down: the busiest has 1.07 times the mean's work).  What its steps
// measured on the first of these: products issued by one diverged thread 2,479 us, by a warp
// 1,934; no maximum before the weights, products back to back 1,857; rows that are not finite
// found in O, not by a search of V, 1,777; halves 1,757; the masked softmax out of line 1,603
// (before that the code did not fit the instruction cache: its misses ran at 67 % of what the
// cache behind it gives, now 18 %); the products unrolled again 1,549.  Slower: the maximum and
// the weights by 32 columns with a vote each (2,125), the weights again by a loop around the
// same code (2,179), the softmax groups looking for landed tiles in the issuing warp's place
// (1,637), a barrier for PV at an item's end only and stages released behind QK (1,602).
//
// Every wait is bounded: one that runs out sets the library's error word (sd_device_status)
// and ends the CTA's work.
#include <cuda.h>

#include <atomic>

#include "sd_dense.cuh"
#include "sd_dense_plan.cuh"

namespace sd {

__device__ unsigned int g_tile_timeout = 0;  // set when a bounded wait of a tile kernel ran out

namespace {

constexpr int kTlThreads = 384;
constexpr int kTlStages = 5;
constexpr uint32_t kTlTile = kDtKeys * kD * 2;  // bytes of a K, V or Q tile: 32 KB
constexpr uint32_t kTlHalf = kTlTile / 2;       // 64 channels of it
constexpr uint32_t kTlSpin = 1u << 22;          // try_wait rounds before a wait gives up
constexpr float kTlMost = 16384.0f;             // half a tile's weights sum up to this at most,
constexpr float kTlLeast = 0x1p-40f;            // and a row's so far to this at least, or m moves
constexpr float kTlWide = 0x1p26f;
constexpr uint32_t kTlAgainItems = 1024;        // items with a bit of their own in `again`

struct TlSmem {
  uint8_t q[2][kTlTile];
  uint8_t ring[kTlStages][kTlTile];
  unsigned long long full[kTlStages], empty[kTlStages];
  unsigned long long qfull, qempty;
  // (a barrier for each half of a tile's weights and products: a group may be a half ahead)
  unsigned long long sfull[2], pfull[2][2], pvhalf[2], pvdone[2], oempty[2], mlfull, drain;
  float2 ml[kDtRows];   // dual: the second group's (m, l)
  uint32_t tmem;
  int abort;
  uint32_t again[kTlAgainItems / 32];  // items of this CTA with a row to compute again, by number
};
constexpr size_t kTlSmemBytes = sizeof(TlSmem) + 1024;  // the tiles start on 1 KB

struct TlArgs {
  const uint16_t* q;
  const uint16_t* K;
  const uint16_t* V;
  uint16_t* out;      // splits == 1: the result
  float* lse;
  float* part_o;      // parts: [row][splits][d], not divided by l
  float2* part_ml;    // [row][splits]: (m in log2 units, l)
  sd_strides qs, os;
  DnWindow w;         // m: query tokens per sequence
  int causal;         // 0: every row sees [0, w.n)
  int Hkv, G, lg;     // lg: log2 G
  int64_t ncap;
  float sl2;          // scale * log2(e), above 0
  int dual, splits, wide;  // wide: rows of the result on 32 bytes
  int parts_only;          // splits == 1 leaves a partial result, too
  int64_t per;
  uint32_t items, bh;
};

// ---- PTX ---------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t tl_su32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void tl_init(unsigned long long* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(tl_su32(b)), "r"(count)
               : "memory");
}
__device__ __forceinline__ void tl_arrive(unsigned long long* b) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n" ::"r"(tl_su32(b))
               : "memory");
}
__device__ __forceinline__ bool tl_try(unsigned long long* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(tl_su32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase of the given parity to complete; false once the rounds ran out or
// another thread of the CTA gave up.
__device__ __forceinline__ bool tl_wait(int* abort, unsigned long long* b, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < kTlSpin; ++i) {
    if (tl_try(b, parity)) return true;
    if (*(volatile int*)abort) return false;
  }
  *(volatile int*)abort = 1;
  atomicOr(&g_tile_timeout, 1u);
  return false;
}
// ... by a whole warp, with one answer.
__device__ __forceinline__ bool tl_wait_warp(int* abort, unsigned long long* b, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, tl_wait(abort, b, parity));
}
// The same without a look at the others: for copies in flight when the CTA gives up.
__device__ __forceinline__ void tl_drain(unsigned long long* b, uint32_t parity) {
  for (uint32_t i = 0; i < kTlSpin && !tl_try(b, parity); ++i) {
  }
}
__device__ __forceinline__ void tl_tma(void* dst, const CUtensorMap* map, int c, int tok, int row,
                                       unsigned long long* b) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(tl_su32(dst)),
      "l"(map), "r"(c), "r"(tok), "r"(row), "r"(tl_su32(b))
      : "memory");
}
__device__ __forceinline__ void tl_commit(unsigned long long* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(
                   tl_su32(b))
               : "memory");
}
__device__ __forceinline__ void tl_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void tl_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}
// What was loaded may be used (tl_use32: these 32 registers, none earlier than here).
__device__ __forceinline__ void tl_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tl_use32(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :: "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]) :: "memory");
}
__device__ __forceinline__ void tl_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
// 32 columns of the thread's lane
__device__ __forceinline__ void tl_ld32(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tl_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tl_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// Shared-memory operand in the 128-byte swizzle: 8-row groups 1 KB apart; lbo: for an operand
// whose rows are the product's inner dimension (V), its next 64 columns.  The low word moves
// with the address, the high word stands.
__device__ __forceinline__ uint32_t tl_desc(uint32_t addr, uint32_t lbo) {
  return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t kTlDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// bf16 x bf16 -> fp32, 128 x 128; bit 16: B's rows are the inner dimension
constexpr uint32_t kTlInstr = (1u << 4) | (1u << 7) | (1u << 10) | ((128u / 8) << 17) |
                              ((128u / 16) << 24);
constexpr uint32_t kTlInstrV = kTlInstr | (1u << 16);

__device__ __forceinline__ void tl_mma_qk(uint32_t s, uint32_t q, uint32_t k, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}\n" ::"r"(s),
      "r"(q), "r"(k), "r"(kTlDescHi), "r"(kTlInstr), "r"(add)
      : "memory");
}
__device__ __forceinline__ void tl_mma_pv(uint32_t o, uint32_t p, uint32_t v, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}\n" ::"r"(o),
      "r"(p), "r"(v), "r"(kTlDescHi), "r"(kTlInstrV), "r"(add)
      : "memory");
}
// S = Q K^T by one thread: 16 channels a product, 32 bytes of a 64-channel half.  (Unrolled: in
// a loop a product took 90 cycles to issue, and takes 64 to run.)
__device__ __forceinline__ void tl_qk(uint32_t s, uint32_t q, uint32_t k) {
  const uint32_t dq = tl_desc(q, 16), dk = tl_desc(k, 16);
#pragma unroll
  for (uint32_t kk = 0; kk < 8; ++kk) {
    const uint32_t off = (kk >> 2) * (kTlHalf >> 4) + (kk & 3) * 2;
    tl_mma_qk(s, dq + off, dk + off, kk > 0);
  }
}
// O += P V over 64 tokens: 16 a product, two 8-row groups; 8 columns of P.
__device__ __forceinline__ void tl_pv(uint32_t o, uint32_t p, uint32_t v, bool add) {
  const uint32_t dv = tl_desc(v, kTlHalf);
#pragma unroll
  for (uint32_t kk = 0; kk < 4; ++kk)
    tl_mma_pv(o, p + 8 * kk, dv + 128 * kk, add || kk > 0);
}
__device__ __forceinline__ bool tl_elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
               : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float tl_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Pairs of fp32 values, one instruction for both.
__device__ __forceinline__ uint64_t tl_two(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void tl_of(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t tl_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t tl_mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 bytes, on 32 bytes.
__device__ __forceinline__ void tl_st256(void* dst, const uint32_t* y) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(y[0]),
               "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
               : "memory");
}
__device__ __forceinline__ uint64_t tl_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float tl_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// ---- work --------------------------------------------------------------------------------
// One item: rows [r0, r0 + rows) of (sequence, KV head) bh, token tiles [ta, tb) of the
// item's list (tiles of [0, s1), then of [w0, w1)).
struct TlItem {
  int64_t bh, r0;
  int b, h, rows, split;
  int64_t p0;        // position of query token 0
  DnRanges r;
  int na, ta, tb;    // tiles of [0, s1); this part's tiles
  int t[2];          // token tiles of each softmax group
  int nq;            // row tiles (dual: 2 groups of one)
  int64_t behind;    // position behind the sequence's last row
};

__device__ __forceinline__ TlItem tl_item(const TlArgs& a, uint32_t id) {
  TlItem x;  // (32-bit divisions: 64-bit ones took 3,000 cycles of an item)
  const uint32_t rest = a.splits == 1 ? id : id / (uint32_t)a.splits;
  x.split = (int)(id - rest * (uint32_t)a.splits);
  const uint32_t tile_up = rest / (uint32_t)a.bh, bh = rest - tile_up * (uint32_t)a.bh;
  x.bh = bh;
  // the last rows first: under a causal mask they see most
  const int64_t tile = a.per - 1 - (int64_t)tile_up;
  x.b = (int)(bh / (uint32_t)a.Hkv);
  x.h = (int)(bh - (uint32_t)x.b * (uint32_t)a.Hkv);
  const int64_t len = a.causal ? a.w.len(x.b) : a.w.m;
  x.r0 = tile * (a.dual ? kDtRows : kDtPair);
  x.rows = (int)imax64(0, imin64(a.dual ? kDtRows : kDtPair, len * a.G - x.r0));
  x.p0 = a.causal ? a.w.at(x.b) : 0;
  x.behind = x.p0 + len;
  x.ta = x.tb = x.na = 0;
  x.t[0] = x.t[1] = 0;
  x.nq = a.dual || x.rows > kDtRows ? 2 : 1;
  if (!x.rows) return x;
  if (a.causal) {
    const int64_t pa = x.p0 + (x.r0 >> a.lg), pb = x.p0 + ((x.r0 + x.rows - 1) >> a.lg);
    // [0, s1) and [w0, w1) of all rows: the first row's window start, the last row's end
    DnRanges& r = x.r;
    r.w1 = imax64(0, imin64(a.w.n, pb + 1));
    r.w0 = imax64(0, imin64(pa - a.w.window + 1, r.w1));
    r.s1 = imin64(imin64(a.w.sink, a.w.n), r.w1);
    if (r.s1 >= r.w0) r.s1 = 0, r.w0 = 0;
  } else {
    x.r = DnRanges{0, 0, a.w.n};
  }
  x.na = (int)((uint32_t)(x.r.s1 + kDtKeys - 1) / kDtKeys);
  const uint32_t all = x.na + (uint32_t)(x.r.w1 - x.r.w0 + kDtKeys - 1) / kDtKeys;
  x.ta = 0;
  x.tb = (int)all;
  if (a.splits > 1) {  // all * splits < 2^32: 2^24 tiles at most, and a part for an SM
    x.ta = (int)(all * (uint32_t)x.split / (uint32_t)a.splits);
    x.tb = (int)(all * (uint32_t)(x.split + 1) / (uint32_t)a.splits);
  }
  const int t = x.tb - x.ta;
  if (a.dual) {
    x.t[0] = (t + 1) / 2;
    x.t[1] = t / 2;
  } else {
    x.t[0] = t;
    x.t[1] = x.nq == 2 ? t : 0;
  }
  return x;
}
// Tile i of the list: its first token and its range's end.
__device__ __forceinline__ void tl_tile(const TlItem& x, int i, int64_t& c0, int64_t& end) {
  if (i < x.na) {
    c0 = (int64_t)i * kDtKeys;
    end = x.r.s1;
  } else {
    c0 = x.r.w0 + (int64_t)(i - x.na) * kDtKeys;
    end = x.r.w1;
  }
}
// The list's tile that group g takes j-th.
__device__ __forceinline__ int tl_index(const TlArgs& a, const TlItem& x, int g, int j) {
  return x.ta + (a.dual ? 2 * j + g : j);
}
// Ring position (counted from the item's first) of group g's j-th V.  Loads go K, V, K, V, ..;
// dual: K0, K1, V0, V1, ...
__device__ __forceinline__ uint32_t tl_vpos(const TlArgs& a, const TlItem& x, int g, int j) {
  return a.dual ? 4u * j + (j < x.t[1] ? 2 : 1) + g : 2u * j + 1;
}
__device__ __forceinline__ uint32_t tl_loads(const TlArgs& a, const TlItem& x) {
  return 2u * (a.dual ? x.t[0] + x.t[1] : x.t[0]);
}

// Bits [0, n) of a word.
__device__ __forceinline__ uint32_t tl_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}
// Scores [32 c, 32 c + 32) of the thread's row as loaded, -inf where it does not see them.
__device__ __forceinline__ void tl_mask(uint32_t* s, int c, int hi, int lo, int sk) {
  const uint32_t see = tl_below(hi - 32 * c) &
                       (~tl_below(lo + 1 - 32 * c) | tl_below(sk - 32 * c));
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = see & (1u << i) ? s[i] : 0xFF800000u;
}
// The weights 2^(s sl2 - m) of 2 N scores as packed bf16, and their sum.
template <int N>
__device__ __forceinline__ float tl_weights(uint32_t* pk, const uint32_t* s, float sl2, float m) {
  const uint64_t sl = tl_two(sl2, sl2), mm = tl_two(-m, -m);
  uint64_t sum[2] = {0, 0};  // pairs of +0
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float u, v;
    tl_of(tl_fma2(tl_two(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sl, mm), u, v);
    u = tl_exp2(u);
    v = tl_exp2(v);
    sum[i & 1] = tl_add2(sum[i & 1], tl_two(u, v));
    pk[i] = bf16_pack(u, v);
  }
  float u, v;
  tl_of(tl_add2(sum[0], sum[1]), u, v);
  return u + v;
}
struct TlSeen {  // of a tile's tokens the row sees those below hi, and above lo or below sk
  int hi, lo, sk;
  bool cut;      // not all of them
};
// Whether m is far below a score, or far above all scores of the row so far (kTlMost,
// kTlLeast), for any row of the warp.
__device__ __forceinline__ bool tl_off(float sum, float l) {
  return __any_sync(0xFFFFFFFFu, !(sum <= kTlMost) || l + sum < kTlLeast);
}
// The weights of half a tile for a warp whose rows see a part of it, or with a row whose m
// does not fit: where the half's largest score is over 8 above m, or 30 below while the row
// has no weight yet, m becomes the whole number above it, and l and O move by a power of two,
// exactly.  From 2^26 on a score's product with the scale, which the weights take before it is
// rounded, may be far from such an m: the row becomes NaN, and is computed again with scores
// that are rounded first (tl_again).  with_o: O holds products, done when `b` completes its
// phase.
struct TlFit {
  float m, l;
  bool ok;
};
__device__ __noinline__ TlFit tl_fit(int* abort, unsigned long long* b, uint32_t parity, float m,
                                     float l, uint32_t s_at, uint32_t o_at, int half, bool with_o,
                                     TlSeen see, float sl2) {
  if (see.cut) {  // as the whole halves: against m as it stands
    uint32_t pk[32];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t s[32];
      tl_ld32(s, s_at + 64 * half + 32 * c);
      tl_wait_ld();
      tl_use32(s);
      tl_mask(s, 2 * half + c, see.hi, see.lo, see.sk);
      sum += tl_weights<16>(pk + 16 * c, s, sl2, m);
    }
    const int at = 64 * half;
    const bool sees = see.hi > at && (see.lo + 1 < see.hi || see.sk > at);
    if (!tl_off(sum, sees ? l : 1.0f)) {
      tl_st32(s_at + 32 * half, pk);
      return TlFit{m, l + sum, true};
    }
  }
  float mx = -INFINITY;
#pragma unroll 1
  for (int k = 2 * half; k < 2 * half + 2; ++k) {
    uint32_t s[32];
    tl_ld32(s, s_at + 32 * k);
    tl_wait_ld();
    tl_use32(s);
    if (see.cut) tl_mask(s, k, see.hi, see.lo, see.sk);
    float y[2] = {mx, mx};
#pragma unroll
    for (int i = 0; i < 32; i += 4)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        y[h] = tl_max3(y[h], __uint_as_float(s[i + 2 * h]), __uint_as_float(s[i + 2 * h + 1]));
    mx = fmaxf(y[0], y[1]);
  }
  const float top = ceilf(mx * sl2);
  float f = 1.0f;
  if (top > m + 8.0f || (l == 0.0f && top < m - 30.0f && top != -INFINITY)) {
    f = l == 0.0f || m - top < -126.0f ? 0.0f : exp2f(m - top);
    m = fabsf(top) < kTlWide ? top : NAN;
    l *= f;
  }
  if (with_o && __any_sync(0xFFFFFFFFu, f != 1.0f)) {
    if (!tl_wait_warp(abort, b, parity)) return TlFit{m, l, false};
    tl_fence_after();
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      uint32_t o[32];
      tl_ld32(o, o_at + 32 * k);
      tl_wait_ld();
      tl_use32(o);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
      tl_st32(o_at + 32 * k, o);
    }
  }
#pragma unroll 1
  for (int k = 2 * half; k < 2 * half + 2; ++k) {
    uint32_t s[32], pk[16];
    tl_ld32(s, s_at + 32 * k);
    tl_wait_ld();
    tl_use32(s);
    if (see.cut) tl_mask(s, k, see.hi, see.lo, see.sk);
    l += tl_weights<16>(pk, s, sl2, m);
    tl_st16(s_at + 16 * k, pk);
  }
  return TlFit{m, l, true};
}

// Softmax of the item's row tile `g` (dual: of every second token tile), and its result.
__device__ __forceinline__ void tl_softmax(TlSmem& sm, const TlArgs& a, int g, uint32_t tmem) {
  const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t s_at = tmem + lanes + 128 * g, o_at = tmem + lanes + 256 + 128 * g;
  uint32_t base = 0;   // ring position of the item's first load
  uint32_t done = 0;   // tiles of this group so far
  uint32_t done1 = 0;  // dual: tiles of the second group up to this item's end
  uint32_t other_n = 0;  // dual: items in which the second group had tiles
  for (uint32_t id = blockIdx.x; id < a.items; id += gridDim.x) {
    const TlItem x = tl_item(a, id);
    if (!x.rows) continue;
    const int T = x.t[g];
    const int local = (a.dual ? 0 : kDtRows * g) + tid;  // row of the item
    const int64_t row = x.r0 + local;
    const bool mine = local < x.rows;
    const bool warp_on = (a.dual ? 0 : kDtRows * g) + 32 * warp < x.rows;
    const int64_t p = x.p0 + ((x.r0 + min(local, x.rows - 1)) >> a.lg);
    // positions of this row tile's first and last row
    const int64_t pa = x.p0 + ((x.r0 + (a.dual ? 0 : kDtRows * g)) >> a.lg);
    const int64_t pb =
        x.p0 + ((x.r0 + min((a.dual ? 0 : kDtRows * g) + kDtRows, x.rows) - 1) >> a.lg);
    float m = 0.0f, l = 0.0f;
    if (g == 1 && (x.nq == 1 || (a.dual && T == 0))) {  // nothing of the item is this group's
      base += tl_loads(a, x);
      continue;
    }
    if (a.dual && x.t[1] > 0) ++other_n;
    if (a.dual) done1 += x.t[1];
    for (int j = 0; j < T; ++j) {
      int64_t c0, end;
      tl_tile(x, tl_index(a, x, g, j), c0, end);
      const int have = (int)imin64(kDtKeys, end - c0);
      // whether all rows of the tile see all that it holds
      const bool same = !a.causal || (c0 + have - 1 <= pa &&
                                      (c0 + have <= a.w.sink || c0 > pb - a.w.window));
      if (!tl_wait_warp(&sm.abort, &sm.sfull[g], done & 1)) return;
      tl_fence_after();
      if (a.causal && have < kDtKeys && c0 + kDtKeys > x.behind) {
        // behind the sequence's last row the cache may hold anything: V rows become zero
        // (the TMA gives zeros behind the first tokens, by a map that ends there)
        const uint32_t pos = base + tl_vpos(a, x, g, j);
        const uint32_t st = pos % kTlStages;
        if (!tl_wait_warp(&sm.abort, &sm.full[st], (pos / kTlStages) & 1)) return;
        uint8_t* v = sm.ring[st] + (tid >> 3 & 1) * kTlHalf + (tid & 7) * 16;
#pragma unroll 1
        for (int r = have + (tid >> 4); r < kDtKeys; r += 8)
          *reinterpret_cast<uint4*>(v + r * 128) = make_uint4(0u, 0u, 0u, 0u);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      }
      TlSeen see = {have, -1, kDtKeys, !same || have < kDtKeys};
      if (see.cut && a.causal) {
        see.hi = (int)imax64(0, imin64(have, p + 1 - c0));
        see.sk = (int)imax64(0, imin64(kDtKeys, a.w.sink - c0));
        see.lo = (int)imax64(-1, imin64(kDtKeys, p - a.w.window - c0));
      }
      // by halves of 64 tokens, so that the first half's product with V runs beside the second
      // half's weights
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (warp_on) {
          bool fit = see.cut;
          if (!fit) {
            uint32_t s[2][32], pk[32];
            tl_ld32(s[0], s_at + 64 * half);
            tl_wait_ld();
            tl_use32(s[0]);
            tl_ld32(s[1], s_at + 64 * half + 32);  // while these are worked on
            float sum = tl_weights<16>(pk, s[0], a.sl2, m);
            tl_wait_ld();
            tl_use32(s[1]);
            sum += tl_weights<16>(pk + 16, s[1], a.sl2, m);
            fit = tl_off(sum, l);
            if (!fit) {
              l += sum;
              tl_st32(s_at + 32 * half, pk);
            }
          }
          if (fit) {
            const TlFit y = tl_fit(&sm.abort, half ? &sm.pvhalf[g] : &sm.pvdone[g],
                                   (done + half - 1) & 1, m, l, s_at, o_at, half,
                                   j > 0 || half > 0, see, a.sl2);
            if (!y.ok) return;
            m = y.m, l = y.l;
          }
          tl_wait_st();
        }
        tl_fence_before();
        __syncwarp();
        if (lane == 0) tl_arrive(&sm.pfull[g][half]);
      }
      ++done;
    }
    base += tl_loads(a, x);
    if (l == 0.0f) m = -INFINITY;  // no weight
    if (T > 0) {
      if (!tl_wait_warp(&sm.abort, &sm.pvdone[g], (done - 1) & 1)) return;
      tl_fence_after();
    }
    if (a.dual && g == 1) {
      sm.ml[tid] = make_float2(m, l);
      // read by the first group before it gives O back, which this group's next item needs
      __syncwarp();
      if (lane == 0) tl_arrive(&sm.mlfull);
      continue;
    }
    if (a.dual && x.t[1] > 0) {
      if (!tl_wait_warp(&sm.abort, &sm.mlfull, (other_n - 1) & 1)) return;
      if (!tl_wait_warp(&sm.abort, &sm.pvdone[1], (done1 - 1) & 1)) return;
      tl_fence_after();
    }
    float f0 = 1.0f, f1 = 0.0f;
    if (a.dual && x.t[1] > 0) {
      const float2 y = sm.ml[tid];
      const float top = fmaxf(m, y.x), mu = top == -INFINITY ? 0.0f : top;
      f0 = exp2f(m - mu);
      f1 = exp2f(y.x - mu);
      l = l * f0 + y.y * f1;
      m = top;
    }
    const int64_t t = row >> a.lg;
    const int head = x.h * a.G + (int)(row & (a.G - 1));
    const int64_t prow = (x.bh * a.w.m * a.G + row) * a.splits + x.split;
    const int64_t orow = x.b * a.os.seq + head * a.os.head + t * a.os.token;
    const bool final = a.splits == 1 && !a.parts_only;
    if (final) {
      float inv;  // (to 2^-23; what it multiplies is rounded to bf16)
      asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(inv) : "f"(l));
      inv = l == 0.0f ? 0.0f : inv;
      f0 *= inv;
      f1 *= inv;
    }
    uint64_t odd = 0;  // 0 times every value of O: NaN if one is not finite
    if (warp_on) {
      const uint64_t f00 = tl_two(f0, f0), f11 = tl_two(f1, f1);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0u;
        if (x.t[0] > 0) {
          tl_ld32(o, o_at + 32 * c);
          tl_wait_ld();
          tl_use32(o);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float u, v;
            tl_of(tl_mul2(tl_two(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f00), u, v);
            o[i] = __float_as_uint(u);
            o[i + 1] = __float_as_uint(v);
          }
        }
        if (a.dual && x.t[1] > 0) {
          uint32_t o1[32];
          tl_ld32(o1, o_at + 128 + 32 * c);
          tl_wait_ld();
          tl_use32(o1);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float u, v;
            tl_of(tl_fma2(tl_two(__uint_as_float(o1[i]), __uint_as_float(o1[i + 1])), f11,
                          tl_two(__uint_as_float(o[i]), __uint_as_float(o[i + 1]))),
                  u, v);
            o[i] = __float_as_uint(u);
            o[i + 1] = __float_as_uint(v);
          }
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          odd = tl_fma2(tl_two(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), 0ull, odd);
        if (mine && final) {
          uint32_t y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            y[i] = bf16_pack(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
          uint16_t* dst = a.out + orow + 32 * c;
          if (a.wide) {  // whole 32-byte sectors
#pragma unroll
            for (int i = 0; i < 2; ++i) tl_st256(dst + 16 * i, y + 8 * i);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(dst + 8 * i) =
                  make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        } else if (mine) {
          float* dst = a.part_o + prow * kD + 32 * c;
          if (a.wide) {
#pragma unroll
            for (int i = 0; i < 4; ++i) tl_st256(dst + 8 * i, o + 8 * i);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(dst + 4 * i) =
                  make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
      }
    }
    if (mine) {
      if (!final)
        a.part_ml[prow] = make_float2(m, l);
      else if (a.lse)
        a.lse[((int64_t)x.b * a.Hkv * a.G + head) * a.w.m + t] =
            l == 0.0f ? -INFINITY : (m + log2f(l)) * kDnLn2;
    }
    // a row whose O is not finite may owe that to tokens that it does not see (tl_again)
    float odd0, odd1;
    tl_of(odd, odd0, odd1);
    if (__builtin_expect(__any_sync(0xFFFFFFFFu, mine && !(odd0 == 0.0f && odd1 == 0.0f)), 0) &&
        lane == 0) {
      const uint32_t nth = id / gridDim.x;
      atomicOr(&sm.again[nth % kTlAgainItems / 32], 1u << (nth % 32));
    }
    tl_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (T > 0) tl_arrive(&sm.oempty[g]);
      if (a.dual && x.t[1] > 0) tl_arrive(&sm.oempty[1]);
    }
  }
}

// A ring position as stage and round.
struct TlPos {
  uint32_t stage, par;
  __device__ __forceinline__ void next() {
    if (++stage == kTlStages) {
      stage = 0;
      par ^= 1;
    }
  }
  __device__ __forceinline__ TlPos ahead(uint32_t n) const {  // n <= kTlStages
    TlPos p = {stage + n, par};
    if (p.stage >= kTlStages) {
      p.stage -= kTlStages;
      p.par ^= 1;
    }
    return p;
  }
};

// One warp issues every product of the CTA; it stays together (so that addresses and
// descriptors live in uniform registers: issued by one diverged thread, a tile's eight
// products took 700 to 800 cycles) and elects the thread that issues.
__device__ __forceinline__ bool tl_products(TlSmem& sm, const TlArgs& a, uint32_t tmem) {
  const bool leader = tl_elect();
  uint32_t items = 0, par_p[2] = {0, 0}, outs[2] = {0, 0};
  const uint32_t q_at = tl_su32(sm.q[0]), ring = tl_su32(sm.ring[0]);
  TlPos at = {0, 0};
  auto loaded = [&](const TlPos& p) {
    return tl_wait_warp(&sm.abort, &sm.full[p.stage], p.par);
  };
  for (uint32_t id = blockIdx.x; id < a.items; id += gridDim.x) {
    const TlItem x = tl_item(a, id);
    const int t0 = __shfl_sync(0xFFFFFFFFu, x.t[0], 0), t1 = __shfl_sync(0xFFFFFFFFu, x.t[1], 0);
    if (t0 == 0) continue;
    const int groups = t1 > 0 ? 2 : 1;
    if (!tl_wait_warp(&sm.abort, &sm.qfull, items & 1)) return false;
    // the first scores; dual: K0, K1, V0, V1 in the ring, else K, V
    for (int g = 0; g < groups; ++g) {
      const TlPos kp = a.dual ? at.ahead(g) : at;
      if (!loaded(kp)) return false;
      tl_fence_after();
      if (leader) {
        tl_qk(tmem + 128 * g, q_at + (a.dual ? 0 : g * kTlTile), ring + kp.stage * kTlTile);
        tl_commit(&sm.sfull[g]);
        if (a.dual || g == groups - 1) tl_commit(&sm.empty[kp.stage]);
        if (g == groups - 1 && t0 == 1) tl_commit(&sm.qempty);
      }
      __syncwarp();
    }
    for (int j = 0; j < t0; ++j) {
      const int now = a.dual && j < t1 ? 2 : 1;  // K (and V) loads of this step
      for (int g = 0; g < groups; ++g) {
        if (g == 1 && j >= t1) break;
        const bool last = a.dual || g == groups - 1;  // the stage's last reader
        const bool more = j + 1 < (g ? t1 : t0);
        const TlPos vp = at.ahead(now + (a.dual ? g : 0)), kp = at.ahead(2 * now + (a.dual ? g : 0));
        // both tiles first, so that the scores' products follow without a gap
        if (g == 0 || a.dual) {
          if (!loaded(vp)) return false;
          if (more && !loaded(kp)) return false;
        }
        if (j == 0) {  // O of the item before is read
          if (outs[g] && !tl_wait_warp(&sm.abort, &sm.oempty[g], (outs[g] - 1) & 1)) return false;
          ++outs[g];
        }
        const uint32_t o = tmem + 256 + 128 * g, pp = tmem + 128 * g, v = ring + vp.stage * kTlTile;
        if (!tl_wait_warp(&sm.abort, &sm.pfull[g][0], par_p[g])) return false;
        tl_fence_after();
        if (leader) {
          tl_pv(o, pp, v, j > 0);
          tl_commit(&sm.pvhalf[g]);
        }
        __syncwarp();
        if (!tl_wait_warp(&sm.abort, &sm.pfull[g][1], par_p[g])) return false;
        par_p[g] ^= 1;
        tl_fence_after();
        if (leader) {
          tl_pv(o, pp + 32, v + kTlHalf / 2, true);
          tl_commit(&sm.pvdone[g]);
          if (last) tl_commit(&sm.empty[vp.stage]);
          if (more) {
            tl_qk(tmem + 128 * g, q_at + (a.dual ? 0 : g * kTlTile), ring + kp.stage * kTlTile);
            tl_commit(&sm.sfull[g]);
            if (last) tl_commit(&sm.empty[kp.stage]);
            // the item's last scores: Q may go
            const bool done = g == 1 ? j + 2 == t1 && t1 == t0 : j + 2 == t0 && t1 < t0;
            if (done) tl_commit(&sm.qempty);
          }
        }
        __syncwarp();
      }
      for (int i = 0; i < 2 * now; ++i) at.next();
    }
    ++items;
  }
  // arrivals of the last commits are in before the CTA ends
  return !items || tl_wait_warp(&sm.abort, &sm.qempty, (items - 1) & 1);
}

struct TlMaps {
  CUtensorMap k, v, vs;  // vs: V's first tokens, zeros behind them
};

// One thread issues every K and V load of the CTA.
struct TlLoader {
  uint32_t n;
  bool ok;
};
__device__ __forceinline__ void tl_load(TlSmem& sm, TlLoader& ld, const CUtensorMap* map,
                                        const TlItem& x, int tile) {
  if (!ld.ok) return;
  const uint32_t st = ld.n % kTlStages, round = ld.n / kTlStages;
  if (round && !tl_wait(&sm.abort, &sm.empty[st], (round - 1) & 1)) {
    ld.ok = false;
    return;
  }
  int64_t c0, end;
  tl_tile(x, tile, c0, end);
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;\n" ::"r"(
                   tl_su32(&sm.full[st])),
               "r"(kTlTile)
               : "memory");
  tl_tma(sm.ring[st], map, 0, (int)c0, (int)x.bh, &sm.full[st]);
  tl_tma(sm.ring[st] + kTlHalf, map, 64, (int)c0, (int)x.bh, &sm.full[st]);
  ++ld.n;
}
// Steps [j0, j1) of an item's loads.
__device__ __forceinline__ void tl_load_steps(TlSmem& sm, TlLoader& ld, const TlArgs& a,
                                              const TlMaps& t, const TlItem& x, int j0, int j1) {
  for (int j = j0; ld.ok && j < j1; ++j) {
    const int i = tl_index(a, x, 0, j);
    const bool two = a.dual && j < x.t[1];
    tl_load(sm, ld, &t.k, x, i);
    if (two) tl_load(sm, ld, &t.k, x, i + 1);
    tl_load(sm, ld, i < x.na ? &t.vs : &t.v, x, i);
    if (two) tl_load(sm, ld, i + 1 < x.na ? &t.vs : &t.v, x, i + 1);
  }
}
// Steps that fill no more than the ring: loaded before the CTA's warps meet.
__device__ __forceinline__ int tl_early(const TlArgs& a, const TlItem& x) {
  return min(x.t[0], a.dual ? 1 : 2);
}
__device__ __forceinline__ void tl_loader(TlSmem& sm, TlLoader ld, const TlArgs& a,
                                          const TlMaps& t) {
  for (uint32_t id = blockIdx.x; ld.ok && id < a.items; id += gridDim.x) {
    const TlItem x = tl_item(a, id);
    tl_load_steps(sm, ld, a, t, x, id == blockIdx.x ? tl_early(a, x) : 0, x.t[0]);
  }
  // every load has landed and every stage is released before the CTA ends
  const uint32_t first = ld.n > kTlStages ? ld.n - kTlStages : 0;
  for (uint32_t i = first; i < ld.n; ++i) {
    const uint32_t st = i % kTlStages, par = (i / kTlStages) & 1;
    if (ld.ok) ld.ok = tl_wait(&sm.abort, &sm.empty[st], par);
    if (!ld.ok) tl_drain(&sm.full[st], par);
  }
}

// An item's query rows into shared memory, in the swizzle of the products.
__device__ __forceinline__ void tl_load_q(TlSmem& sm, const TlArgs& a, const TlItem& x, int tid,
                                          int threads) {
  const int rows = a.dual ? kDtRows : x.nq * kDtRows;
  const int c = tid & 15;
  const uint16_t* base = a.q + x.b * a.qs.seq + (int64_t)x.h * a.G * a.qs.head + 8 * c;
#pragma unroll 4
  for (int r = tid >> 4; r < rows; r += threads >> 4) {
    const int64_t row = x.r0 + min(r, x.rows - 1);
    const uint16_t* src = base + (row & (a.G - 1)) * a.qs.head + (row >> a.lg) * a.qs.token;
    const uint32_t dst = tl_su32(sm.q[r >> 7]) + (c >> 3) * kTlHalf + (r & 127) * 128 +
                         (((c & 7) ^ (r & 7)) << 4);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
                 "r"(r < x.rows ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;\n" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}
// Two warps load the rows of each item with tiles but the CTA's first item.
__device__ __forceinline__ void tl_queries(TlSmem& sm, const TlArgs& a) {
  uint32_t items = 0;
  for (uint32_t id = blockIdx.x; id < a.items; id += gridDim.x) {
    const TlItem x = tl_item(a, id);
    if (x.tb == x.ta) continue;
    if (items && !tl_wait_warp(&sm.abort, &sm.qempty, (items - 1) & 1)) return;
    if (id != blockIdx.x) tl_load_q(sm, a, x, threadIdx.x - 320, 64);
    tl_arrive(&sm.qfull);
    ++items;
  }
}

// ---- rows that are not finite ------------------------------------------------------------
// Such rows of the CTA's items once more, when all of its items are done: nothing waits for
// this but the end of the kernel, so that no bounded wait can run out over it.  A warp takes
// eight rows: groups of 16 tokens that all of them see by tensor-core products, where no
// weight of 0 meets a value that its row does not see; then, row by row, what is left (the
// edges of the mask), token by token.  All rows of 32 heads x 32,768 tokens, causal: 86 ms
// (6.0 where they are finite), under a window of 4,096 and 128 first tokens 28 ms (1.55).
// Not inlined: in the kernel's own code it cost the rows that are finite 1 to 7 %.
constexpr int kTlCuts = 16, kTlEight = 8, kTlAgainStages = 3;
struct TlAgain {  // a warp's place, 28 KB of the tiles'
  uint8_t ring[kTlAgainStages][kDnStage];
  union {
    uint32_t q[16][32];       // the rows' queries as the products take them
    float o[kTlEight][kD];
  };
};
static_assert(8 * sizeof(TlAgain) <= (2 + kTlStages) * kTlTile, "eight warps share the tiles");

struct TlWalk {  // the item's tiles, and what eight rows see of them (tokens are below 2^31)
  int s1, w0, w1, na, tb;
  int causal, sink;
  int hi0, hi1;    // no row sees a token behind hi1, all see those up to hi0 by their position
  int lo0, lo1;    // ... the window: no row up to lo0, all behind lo1
  int i, g;        // the walk's place: group g of tile i
  int t0, end;     // tile i
  bool whole;      // all rows see all of it
  int cuts;        // tiles passed that some rows see some of

  __device__ __forceinline__ void tile(int at, int& c0, int& c1) const {
    c0 = at < na ? at * kDtKeys : w0 + (at - na) * kDtKeys;
    c1 = min(at < na ? s1 : w1, c0 + kDtKeys);
  }
  // all rows see all of [c0, c1)
  __device__ __forceinline__ bool all(int c0, int c1) const {
    return !causal || (c1 - 1 <= hi0 && (c1 <= sink || c0 > lo1));
  }
  __device__ __forceinline__ bool none(int c0, int c1) const {
    return causal && (c0 > hi1 || (c1 - 1 <= lo0 && c0 >= sink));
  }
  // The next group that all see; false behind the last.
  __device__ __forceinline__ bool next(int& c0, int* cut) {
    for (; i < tb; ++i, g = 0) {
      if (g == 0) {
        tile(i, t0, end);
        whole = end - t0 == kDtKeys && all(t0, end);
        // (at most six: what eight rows see of the first tokens and of the window ends in two
        // tiles each, and the two ranges of the item end in one)
        if (!whole && !none(t0, end) && cuts < kTlCuts) cut[cuts++] = i;
      }
      for (; g < kDtKeys / kSwGroup; ++g) {
        c0 = t0 + g * kSwGroup;
        if (whole || (c0 + kSwGroup <= end && all(c0, c0 + kSwGroup))) {
          ++g;
          return true;
        }
      }
    }
    return false;
  }
  // What the row at p sees of the rest of tile `at`.
  __device__ __forceinline__ void rest(DnRow& r, int at, int64_t p, int64_t window,
                                       const uint16_t* K, const uint16_t* V, float sl2,
                                       int lane) const {
    int c0, t1;
    tile(at, c0, t1);
#pragma unroll 1
    for (; c0 < t1; c0 += kSwGroup) {
      const int c1 = min(t1, c0 + kSwGroup);
      if (c1 - c0 == kSwGroup && all(c0, c1)) continue;
#pragma unroll 1
      for (int c = c0; c < c1; ++c)
        if (!causal || (c <= p && (c < sink || c > p - window)))
          dn_row_over(r, K, V, c, c + 1, sl2, lane);
    }
  }
};

__device__ __noinline__ void tl_again(TlSmem* sm, const TlArgs* args) {
  const TlArgs& a = *args;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  TlAgain& at = reinterpret_cast<TlAgain*>(sm->q[0])[warp];
  const uint32_t ring = dn_su32(at.ring);
  const bool final = a.splits == 1 && !a.parts_only;
  int cut[kTlCuts];
  uint32_t nth = 0;
  for (uint32_t id = blockIdx.x; id < a.items; id += gridDim.x, ++nth) {
    if (!(sm->again[nth % kTlAgainItems / 32] >> (nth % 32) & 1u)) continue;
    const TlItem x = tl_item(a, id);
    const uint16_t* K = a.K + x.bh * a.ncap * kD;
    const uint16_t* V = a.V + x.bh * a.ncap * kD;
    auto head = [&](int64_t row) { return x.h * a.G + (int)(row & (a.G - 1)); };
    auto part = [&](int64_t row) { return (x.bh * a.w.m * a.G + row) * a.splits + x.split; };
    auto result = [&](int64_t row) {
      return a.out + x.b * a.os.seq + head(row) * a.os.head + (row >> a.lg) * a.os.token;
    };
    auto query = [&](int64_t row) {
      return a.q + x.b * a.qs.seq + (int64_t)head(row) * a.qs.head + (row >> a.lg) * a.qs.token;
    };
#pragma unroll 1
    for (int r0 = kTlEight * warp; r0 < x.rows; r0 += kTlEight * 8) {
      const int rows = min(kTlEight, x.rows - r0);
      const int64_t row0 = x.r0 + r0;
      uint32_t odd = 0;  // rows whose result is not finite
#pragma unroll 1
      for (int r = 0; r < rows; ++r) {
        const float4 y =
            final ? dn_ld4(result(row0 + r) + 4 * lane)
                  : reinterpret_cast<const float4*>(a.part_o + part(row0 + r) * kD)[lane];
        if (__any_sync(0xFFFFFFFFu,
                       !(isfinite(y.x) && isfinite(y.y) && isfinite(y.z) && isfinite(y.w))))
          odd |= 1u << r;
      }
      if (!odd) continue;
      const bool real = (lane >> 2) < rows;
      {
        const uint32_t* q =
            reinterpret_cast<const uint32_t*>(query(row0 + (real ? lane >> 2 : 0)));
        __syncwarp();  // the rows before are written
        for (int k = 0; k < 16; ++k) at.q[k][lane] = real ? q[4 * k + (lane & 3)] : 0u;
      }
      auto token = [&](int64_t i) { return (int)imax64(-1, imin64(a.w.n, i)); };
      const int64_t pa = x.p0 + (row0 >> a.lg), pb = x.p0 + ((row0 + rows - 1) >> a.lg);
      TlWalk walk;
      walk.s1 = (int)x.r.s1, walk.w0 = (int)x.r.w0, walk.w1 = (int)x.r.w1;
      walk.na = x.na, walk.tb = x.tb, walk.causal = a.causal;
      walk.sink = token(a.w.sink), walk.hi0 = token(pa), walk.hi1 = token(pb);
      walk.lo0 = token(pa - a.w.window), walk.lo1 = token(pb - a.w.window);
      walk.i = x.ta, walk.g = walk.cuts = 0;
      DnEight y;
      dn_eight_begin(y);
      const float sl2 = a.sl2;
      int ahead = 0, slot = 0, c0;
#pragma unroll 1
      for (int k = 0;; ++k) {  // group k copied, group k - 2 worked on
        __syncwarp();          // what the slot held is read by all
        if (walk.next(c0, cut)) {
          dn_fetch(ring + slot * kDnStage, K, V, (int64_t)c0 * kD, kSwGroup, lane);
          ++ahead;
        }
        dn_cp_commit();
        slot = slot == kTlAgainStages - 1 ? 0 : slot + 1;
        if (k < kTlAgainStages - 1) continue;
        if (!ahead) break;
        dn_cp_wait<kTlAgainStages - 1>();
        __syncwarp();
        uint32_t qa[8][2];
#pragma unroll
        for (int kk = 0; kk < 16; ++kk) qa[kk >> 1][kk & 1] = at.q[kk][lane];
        dn_eight_step(y, qa, ring + slot * kDnStage, kSwGroup, real, sl2, 0.0f, lane);
        --ahead;
      }
      dn_cp_wait<0>();
      dn_eight_end(y, at.o[0], rows, lane);
      __syncwarp();
#pragma unroll 1
      for (int r = 0; r < rows; ++r) {
        const int64_t row = row0 + r, t = row >> a.lg;
        DnRow z;
        z.m = __shfl_sync(0xFFFFFFFFu, y.m, 4 * r);
        z.l = __shfl_sync(0xFFFFFFFFu, y.l, 4 * r);
        if (!(odd >> r & 1u)) continue;
        z.o = reinterpret_cast<const float4*>(at.o[r])[lane];
        z.q = dn_ld4(query(row) + 4 * lane);
        for (int c = 0; c < walk.cuts; ++c)
          walk.rest(z, cut[c], x.p0 + t, a.w.window, K, V, sl2, lane);
        if (final) {
          float* lse =
              a.lse ? a.lse + ((int64_t)x.b * a.Hkv * a.G + head(row)) * a.w.m + t : nullptr;
          dn_row_end(z, result(row), lse, lane);
        } else {
          reinterpret_cast<float4*>(a.part_o + part(row) * kD)[lane] = z.o;
          if (lane == 0) a.part_ml[part(row)] = make_float2(z.m, z.l);
        }
      }
    }
  }
}

// All warps of the CTA, from either side.
__device__ __forceinline__ void tl_meet() {
  asm volatile("barrier.sync 1, %0;\n" ::"n"(kTlThreads) : "memory");
}

__global__ void __launch_bounds__(kTlThreads, 1)
    dense_tile_kernel(const __grid_constant__ TlMaps maps, const __grid_constant__ TlArgs a) {
  extern __shared__ uint8_t raw[];
  TlSmem& sm = *reinterpret_cast<TlSmem*>(raw + ((1024u - (tl_su32(raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5;
  // the kernel behind may start where there is room; it waits before it reads the parts
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  TlLoader ld = {0, true};
  if (threadIdx.x == 288) {  // the loader's thread: the first loads are under way early
    asm volatile("prefetch.tensormap [%0];\n\tprefetch.tensormap [%1];\n" ::"l"(&maps.k),
                 "l"(&maps.v));
    for (int i = 0; i < kTlStages; ++i) {
      tl_init(&sm.full[i], 1);
      tl_init(&sm.empty[i], 1);
    }
    tl_init(&sm.qfull, 64);
    tl_init(&sm.qempty, 1);
    for (int g = 0; g < 2; ++g) {
      tl_init(&sm.sfull[g], 1);
      tl_init(&sm.pfull[g][0], 4);
      tl_init(&sm.pfull[g][1], 4);
      tl_init(&sm.pvhalf[g], 1);
      tl_init(&sm.pvdone[g], 1);
      tl_init(&sm.oempty[g], 4);
    }
    tl_init(&sm.mlfull, 4);
    tl_init(&sm.drain, 1);
    sm.abort = 0;
    for (int i = 0; i < (int)kTlAgainItems / 32; ++i) sm.again[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    const TlItem x = tl_item(a, blockIdx.x);
    tl_load_steps(sm, ld, a, maps, x, 0, tl_early(a, x));
  } else if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                     tl_su32(&sm.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  } else if (warp < 8) {
    const TlItem x = tl_item(a, blockIdx.x);
    if (x.tb > x.ta) tl_load_q(sm, a, x, threadIdx.x, 256);
  }
  tl_fence_before();
  __syncthreads();
  tl_fence_after();
  const uint32_t tmem = sm.tmem;
  // 384 x 168 registers at launch: 256 x 208 + 128 x 80
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
    tl_softmax(sm, a, warp >> 2, tmem);
    tl_fence_before();
    tl_meet();
    static_assert(kTlAgainItems == 32 * 32, "a word a lane");
    const uint32_t some = sm.again[threadIdx.x & 31];
    if (__builtin_expect(!sm.abort && __any_sync(0xFFFFFFFFu, some != 0), 0))
      tl_again(&sm, &a);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
    if (warp == 8) {
      if (!tl_products(sm, a, tmem)) {
        // gave up: the products in flight end before tensor memory goes
        if (tl_elect()) tl_commit(&sm.drain);
        tl_drain(&sm.drain, 0);
      }
    } else if (warp == 9) {
      if ((threadIdx.x & 31) == 0) tl_loader(sm, ld, a, maps);
    } else {
      tl_queries(sm, a);
    }
    __syncwarp();
    tl_fence_before();
    tl_meet();
    tl_fence_after();
    if (warp == 8)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  }
}

// ---- joining parts -----------------------------------------------------------------------
// A warp per row: out and lse of up to two sets of partial results (m, l, O).
struct TlJoin {
  const float* ao;
  const float2* aml;
  const float* bo;
  const float2* bml;
  int na, nb;
  uint16_t* out;
  float* lse;
  sd_strides os;
  DnWindow w;
  int causal;        // rows of tokens behind a sequence's length are left alone
  int Hq, Hkv, G;
  int64_t B, rows;   // rows: B * Hq * m
};

__global__ void __launch_bounds__(128) dense_join_kernel(TlJoin a) {
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  dn_wait_prior();
  if (i >= a.rows) return;
  const int64_t m = a.w.m, bhq = i / m, t = i - bhq * m;
  const int64_t b = bhq / a.Hq;
  const int h = (int)(bhq - b * a.Hq), kv = h / a.G, g = h - kv * a.G;
  if (a.causal && t >= a.w.len((int)b)) return;
  // set A's rows: (sequence, KV head, token, head of the group), or, for a prefix, (KV head,
  // sequence, head); set B's: (sequence, KV head, head)
  const int64_t ra = a.causal ? ((b * a.Hkv + kv) * m + t) * a.G + g : (kv * a.B + b) * a.G + g;
  const int64_t rb = (b * a.Hkv + kv) * a.G + g;
  const int n = a.na + a.nb;
  auto ml = [&](int p) {
    return p < a.na ? a.aml[ra * a.na + p] : a.bml[rb * a.nb + p - a.na];
  };
  float top = -INFINITY;
  for (int p = lane; p < n; p += 32) top = fmaxf(top, ml(p).x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const float mu = top == -INFINITY ? 0.0f : top;
  float l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int p0 = 0; p0 < n; p0 += 32) {
    float f = 0.0f, fl = 0.0f;
    if (p0 + lane < n) {
      const float2 x = ml(p0 + lane);
      f = exp2f(x.x - mu);  // an empty part: 0
      fl = x.x == -INFINITY && x.y == 0.0f ? 0.0f : f * x.y;
    }
    l += fl;
#pragma unroll 4
    for (int p = p0; p < min(n, p0 + 32); ++p) {
      const float w = __shfl_sync(0xFFFFFFFFu, f, p - p0);
      const float* src = p < a.na ? a.ao + (ra * a.na + p) * kD : a.bo + (rb * a.nb + p - a.na) * kD;
      const float4 v = reinterpret_cast<const float4*>(src)[lane];
      o.x = fmaf(v.x, w, o.x);
      o.y = fmaf(v.y, w, o.y);
      o.z = fmaf(v.z, w, o.z);
      o.w = fmaf(v.w, w, o.w);
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, s);
  DnRow r;
  r.o = o, r.m = top, r.l = l;
  dn_row_end(r, a.out + b * a.os.seq + h * a.os.head + t * a.os.token, a.lse ? a.lse + i : nullptr,
             lane);
}

// ---- host --------------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The tensor map of a cache [rows][ncap][d] whose first n tokens exist: boxes of 64 channels
// x 128 tokens, zeros behind n.
int tl_map(CUtensorMap* map, const uint16_t* base, int64_t n, int64_t ncap, int64_t rows) {
  static std::atomic<EncodeFn> known{nullptr};
  EncodeFn fn = known.load(std::memory_order_acquire);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &res) != cudaSuccess ||
        res != cudaDriverEntryPointSuccess || !p) {
      cudaGetLastError();
      return fail(SD_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
    }
    fn = reinterpret_cast<EncodeFn>(p);
    known.store(fn, std::memory_order_release);
  }
  const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)n, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {kD * 2, (cuuint64_t)ncap * kD * 2};
  const cuuint32_t box[3] = {64, kDtKeys, 1}, one[3] = {1, 1, 1};
  const CUresult rc =
      fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, box,
         one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (rc != CUDA_SUCCESS) return fail(SD_ERR_CUDA, "cuTensorMapEncodeTiled: %d", (int)rc);
  return SD_OK;
}

int tl_launch(TlArgs& a, int64_t rows_bh, const DtPlan& p, cudaStream_t st) {
  TlMaps maps;
  if (int rc = tl_map(&maps.k, a.K, a.w.n, a.ncap, rows_bh)) return rc;
  if (int rc = tl_map(&maps.v, a.V, a.w.n, a.ncap, rows_bh)) return rc;
  maps.vs = maps.v;
  const int64_t firsts = imin64(a.w.sink, a.w.n);
  if (firsts % kDtKeys)
    if (int rc = tl_map(&maps.vs, a.V, firsts, a.ncap, rows_bh)) return rc;
  a.lg = a.G == 8 ? 3 : a.G == 4 ? 2 : a.G - 1;
  // scale 0: every score 0, as near as a product with the least factor comes (0 would turn the
  // -inf of unseen tokens into NaN)
  if (a.sl2 == 0.0f) a.sl2 = 1e-45f;
  a.dual = p.dual;
  a.splits = p.splits;
  a.per = p.per;
  a.items = (uint32_t)p.items;
  a.bh = (uint32_t)rows_bh;
  a.wide = a.splits > 1 || a.parts_only
               ? ((uintptr_t)a.part_o & 31) == 0
               : ((uintptr_t)a.out & 31) == 0 && a.os.seq % 16 == 0 && a.os.head % 16 == 0 &&
                     a.os.token % 16 == 0;
  if (int rc = set_smem_limit((const void*)dense_tile_kernel, kTlSmemBytes, "tile attention"))
    return rc;
  const unsigned grid = (unsigned)imin64(p.items, device_sm_count());
  dense_tile_kernel<<<grid, kTlThreads, kTlSmemBytes, st>>>(maps, a);
  note_launches(1);
  return check_launch("tile attention");
}

int tl_join(const TlJoin& j, cudaStream_t st) {
  return dn_launch_early("attention join", dense_join_kernel, (unsigned)((j.rows + 3) / 4), 128, 0,
                         0, st, j);
}

// Partial results in a workspace: O first, then (m, l).
constexpr size_t kTlPart = kD * sizeof(float) + sizeof(float2);

}  // namespace

// Reads this GPU's word after the work on `st`, then clears it (both ordered on `st`; the host
// waits for the stream).
int tile_error_take(cudaStream_t st, unsigned* word) {
  *word = 0;
  unsigned zero = 0;
  if (cudaMemcpyFromSymbolAsync(word, g_tile_timeout, sizeof(unsigned), 0, cudaMemcpyDeviceToHost,
                                st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return check_launch("device status: read");
  if (*word &&
      (cudaMemcpyToSymbolAsync(g_tile_timeout, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice,
                               st) != cudaSuccess ||
       cudaStreamSynchronize(st) != cudaSuccess))
    return check_launch("device status: clear");
  return SD_OK;
}

// Sets the word as a kernel whose bounded wait ran out would (for testing the report).
int tile_error_set(unsigned word, cudaStream_t st) {
  if (cudaMemcpyToSymbolAsync(g_tile_timeout, &word, sizeof(unsigned), 0, cudaMemcpyHostToDevice,
                              st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return check_launch("device status: set");
  return SD_OK;
}

static DtPlan window_plan(const Dims& s, int64_t m, int64_t window, int64_t sink) {
  const int64_t rows = m * s.G;
  const int64_t span = imin64(m, (rows <= kDtRows ? kDtRows : kDtPair) / s.G);
  const int64_t keys = imin64(s.n, imin64(sink, s.n) + imin64(window, s.n) + span - 1);
  return dt_plan((int64_t)s.B * s.Hkv, rows, keys, device_sm_count(), true);
}
// Tokens that a single query token may see.
static int64_t window_tokens(const Dims& s, int64_t window, int64_t sink) {
  return imin64(s.n, imin64(sink, s.n) + imin64(window, s.n));
}

size_t window_attend_workspace_bytes(const Dims& s, int64_t m, int64_t window, int64_t sink) {
  if (m == 1) {
    const int64_t parts = window_stream_parts(s, window_tokens(s, window, sink));
    return parts == (int64_t)s.B * s.Hq ? 0 : parts * kTlPart;
  }
  const DtPlan p = window_plan(s, m, window, sink);
  return p.splits == 1 ? 0 : (size_t)s.B * s.Hq * m * p.splits * kTlPart;
}

int launch_window_attend(const Dims& s, const uint16_t* q, const sd_strides& qs,
                         const uint16_t* K, const uint16_t* V, int64_t m, int64_t first,
                         const int32_t* pos, const int32_t* length, int64_t window, int64_t sink,
                         float scale, uint16_t* out, const sd_strides& os, float* lse, void* ws,
                         cudaStream_t st) {
  const DnWindow w{pos, length, first, m, s.n, window, sink};
  const int64_t rows = (int64_t)s.B * s.Hq * m;
  TlJoin j = {};
  j.out = out, j.lse = lse, j.os = os, j.w = w, j.causal = 1;
  j.Hq = s.Hq, j.Hkv = s.Hkv, j.G = s.G, j.B = s.B, j.rows = rows;
  if (m == 1) {
    const int64_t tokens = window_tokens(s, window, sink);
    j.ao = (float*)ws;
    j.aml = (float2*)((float*)ws + window_stream_parts(s, tokens) * kD);
    if (int rc = launch_window_stream(s, q, qs, K, V, w, false, nullptr, tokens, scale, nullptr,
                                      nullptr, 0, out, os, lse, (float*)ws, (float2*)j.aml, &j.na,
                                      st))
      return rc;
    return j.na ? tl_join(j, st) : SD_OK;
  }
  const DtPlan p = window_plan(s, m, window, sink);
  TlArgs a = {};
  a.q = q, a.K = K, a.V = V, a.out = out, a.lse = lse, a.qs = qs, a.os = os, a.w = w;
  a.causal = 1, a.Hkv = s.Hkv, a.G = s.G, a.ncap = s.ncap, a.sl2 = scale * kDnLog2e;
  a.part_o = (float*)ws;
  a.part_ml = (float2*)(a.part_o + rows * p.splits * kD);
  if (int rc = tl_launch(a, (int64_t)s.B * s.Hkv, p, st)) return rc;
  if (p.splits == 1) return SD_OK;
  j.ao = a.part_o, j.aml = a.part_ml, j.na = p.splits;
  return tl_join(j, st);
}

static DtPlan prefix_plan(const Dims& s, int64_t p) {
  return dt_plan(s.Hkv, (int64_t)s.B * s.G, p, device_sm_count(), false);
}

size_t prefix_attend_workspace_bytes(const Dims& s, int64_t p) {
  const int64_t rows = (int64_t)s.B * s.Hq;
  const int64_t pre = p ? rows * prefix_plan(s, p).splits : 0;
  return (pre + window_stream_parts(s, s.n)) * kTlPart;
}

int launch_prefix_attend(const Dims& s, const uint16_t* q, const uint16_t* Kp,
                         const uint16_t* Vp, int64_t p, int64_t pcap, const uint16_t* K,
                         const uint16_t* V, const int32_t* end, float scale, uint16_t* out,
                         float* lse, void* ws, cudaStream_t st) {
  const int64_t rows = (int64_t)s.B * s.Hq;
  const sd_strides qs{(int64_t)s.Hq * kD, kD, 0};
  TlJoin j = {};
  j.out = out, j.lse = lse, j.os = qs, j.w.m = 1, j.Hq = s.Hq, j.Hkv = s.Hkv, j.G = s.G;
  j.B = s.B, j.rows = rows;
  const DtPlan plan = p ? prefix_plan(s, p) : DtPlan{};
  const int64_t pre = p ? rows * plan.splits : 0, own = window_stream_parts(s, s.n);
  float* ao = (float*)ws;
  float* bo = ao + pre * kD;
  float2* aml = (float2*)(bo + own * kD);
  float2* bml = aml + pre;
  if (p) {
    // the batch's rows as the tokens of one sequence, every one seeing the whole prefix
    TlArgs a = {};
    a.q = q, a.K = Kp, a.V = Vp, a.qs = sd_strides{0, kD, (int64_t)s.Hq * kD};
    a.w.m = s.B, a.w.n = p, a.Hkv = s.Hkv, a.G = s.G, a.ncap = pcap;
    a.sl2 = scale * kDnLog2e, a.part_o = ao, a.part_ml = aml, a.parts_only = 1;
    if (int rc = tl_launch(a, s.Hkv, plan, st)) return rc;
  }
  j.ao = ao, j.aml = aml, j.na = p ? plan.splits : 0;
  if (K) {
    DnWindow w = {};
    w.n = s.n;
    if (int rc = launch_window_stream(s, q, qs, K, V, w, true, end, s.n, scale, ao, aml, j.na, out,
                                      qs, lse, bo, bml, &j.nb, st))
      return rc;
    if (!j.nb) return SD_OK;
    j.bo = bo, j.bml = bml;
  }
  return tl_join(j, st);
}

}  // namespace sd
