// Which kernel attends over a 4-bit K/V cache, by sizes and by what the GPU can run.  Plain
// C++, so that the rule can be tested without a GPU.
#pragma once

#include <cstdint>

namespace sd {

constexpr int kKaTile = 32;  // tokens per tile
constexpr int kKaWarps = 4;  // warps per CTA

// CTAs per row for the cluster kernel, or 0 for the streaming kernel.  rows of up to `tiles`
// tiles each, a GPU of `sms` SMs whose clusters of this kernel hold max_cluster CTAs at
// most (8, 4, 2, 1; 0: it does not run at all, as where a process has a part of a GPU).
//
// By tiles in a row of work (t), each ~0.6 to 1 us, with what a launch adds in the same
// units.  Clusters: the tiles of a warp, 4 for every wave of CTAs, and what joining c CTAs
// adds; c > 1 only where all CTAs run at once.  Stream: an even share, and 12 for finding
// it and joining.  Measured (us, clusters / stream): 8 rows of 8,192 tokens 11.1 / 11.5, of
// 16,384 16.0 / 13.5; 128 rows of 4,096 22.6 / 23.8, of 16,384 64.0 / 59.9; 512 rows of 128
// 10.1 / 11.5, of 2,064 39.4 / 35.9.  Next to its border it takes clusters where the other
// is up to 8 to 13 % faster: 512 rows of 32 8.8 / 7.8, of 1,024 24.7 / 23.5; 256 rows of
// 8,192, G = 8, 75.4 / 69.6.
inline int kv4_cluster_of(int64_t rows, int64_t tiles, int sms, int max_cluster) {
  const int64_t slots = 2 * (int64_t)sms;
  constexpr int kJoin[4] = {0, 4, 3, 4};  // c = 1, 2, 4, 8
  int64_t best = 0;
  int cs = 0;
  for (int i = 0; i < 4; ++i) {
    const int64_t c = 1 << i, w = c * kKaWarps;
    if (c > max_cluster || (i && rows * c > slots)) break;
    const int64_t waves = (rows * c + slots - 1) / slots;
    const int64_t t = (tiles + w - 1) / w + kJoin[i];
    const int64_t cost = waves > 1 ? waves * (t + 4) : t;
    if (i == 0 || cost <= best) {
      best = cost;
      cs = (int)c;
    }
  }
  return best > rows * tiles / (slots * kKaWarps) + 12 ? 0 : cs;
}

}  // namespace sd
