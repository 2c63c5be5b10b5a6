// How attention over ranges of the bf16 cache is cut into work (sd_dense_tile.cu,
// sd_dense_stream.cu), by sizes alone.  Plain C++, so that the rules can be tested without a
// GPU.
#pragma once

#include <cstdint>

namespace sd {

constexpr int kDtRows = 128;   // query rows of a tile (tensor-core M)
constexpr int kDtKeys = 128;   // tokens of a tile
constexpr int kDtPair = 2 * kDtRows;

inline int64_t dt_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t dt_min(int64_t a, int64_t b) { return a < b ? a : b; }
inline int64_t dt_max(int64_t a, int64_t b) { return a > b ? a : b; }

// The tile kernel's cut of `rows` query rows (tokens x group) against up to `keys` tokens,
// for each of `heads` (sequence, KV head) pairs.
struct DtPlan {
  int dual;      // at most 128 rows: both softmax groups take the same rows, the item's token
                 // tiles shared between them
  int64_t per;   // items of a pair: tiles of 128 rows or pairs of them
  int splits;    // parts of an item's token tiles, each with a partial result
  int64_t items; // heads * per * splits
};

// Splits where the items are fewer than the SMs: as many as give each SM one, with some token
// tiles for a part.  Where a kernel of its own joins the parts (a window) that takes as long
// as three tiles or so: four for each softmax group (3 x 2 heads x 257 tokens of G = 8 under
// a window of 501: 19.1 us, 21.4 with two).  Where what follows joins them (a prefix), two:
// 17 x 4 heads of G = 8 over 5,003 tokens 19.0 us, 21.0 with one.
inline DtPlan dt_plan(int64_t heads, int64_t rows, int64_t keys, int sms, bool own_join) {
  DtPlan p;
  p.dual = rows <= kDtRows;
  p.per = dt_ceil(rows, p.dual ? kDtRows : kDtPair);
  const int64_t base = heads * p.per;
  const int64_t tiles = dt_ceil(keys, kDtKeys) + 1;  // two ranges may end in a cut tile each
  const int64_t least = !own_join ? 2 : p.dual ? 8 : 4;
  p.splits = (int)dt_max(1, dt_min(sms / base, tiles / least));
  p.items = base * p.splits;
  return p;
}

// The stream kernel's cut of `rows` (sequence, KV head) rows of up to `tokens` tokens: CTAs of
// a row, and whether a kernel of its own joins them (else a cluster does).
constexpr int kSwGroup = 16;   // tokens that a warp takes at a time
constexpr int kSwCtaWarps = 4;
struct SwPlan {
  int parts, cut;
};
// Parts of a row that a kernel of its own joins: a CTA for each of the GPU's places, with two
// groups a warp at least.
inline int sw_cut(int64_t rows, int64_t tokens, int sms) {
  const int64_t groups = dt_ceil(tokens, kSwGroup);
  return (int)dt_max(1, dt_min(2 * sms / rows, groups / (2 * kSwCtaWarps)));
}
// By groups in a row of work for one warp: the waves of CTAs times a warp's groups, and what
// a wave, a cluster's join and a kernel's join add in the same units.
inline SwPlan sw_plan(int64_t rows, int64_t tokens, int sms, int max_cluster) {
  constexpr int kStart = 3, kJoin = 2, kKernel = 8;
  const int64_t slots = 2 * (int64_t)sms, groups = dt_ceil(tokens, kSwGroup);
  SwPlan best = {1, 0};
  int64_t cost = 0;
  for (int c = 1; c <= 8 && (c == 1 || c <= max_cluster); c *= 2) {
    const int64_t waves = dt_ceil(rows * c, slots);
    const int64_t t = waves * (dt_ceil(groups, (int64_t)kSwCtaWarps * c) + kStart) +
                      (c > 1 ? kJoin : 0);
    if (c == 1 || t < cost) {
      cost = t;
      best = {c, 0};
    }
  }
  const int cut = sw_cut(rows, tokens, sms);
  if (cut > 1) {
    const int64_t t = dt_ceil(groups, (int64_t)kSwCtaWarps * cut) + kStart + kKernel;
    if (t < cost) best = {cut, 1};
  }
  return best;
}

}  // namespace sd
