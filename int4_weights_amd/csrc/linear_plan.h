// linear_plan.h -- which kernel moe_gemm_bf16 takes, by sizes alone (host code that any C++ compiler takes, so that the
// choice can be tested without a GPU).
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kLinCus = 256;  // not asked of the device: the workspace's size must not depend on it, nor need one

// K blocks (of 64) of a workgroup when K is split.
constexpr int lin_split_blocks(int KB, int splits) { return (KB + splits - 1) / splits; }

enum LinKind { kLinStream16, kLinStream32, kLinStream64, kLin64x64, kLin64x128, kLin128x128, kLin128x128two, kLin256x256 };
struct LinPlan {
  LinKind kind;
  int splits;
};

// Tiles, and what a round of them over the 256 compute units takes in us per K block: one workgroup on each, and where two fit,
// both.  The tile and the split with the smallest estimate are taken.  Measured (us; 64x64, 64x128, 128x128, 128x128 two per
// unit, 256x256; K = 7168, 4096 columns): 128 rows 23.7, 33, 42, 52, 133 (64x64 in two shares 17.8); 512 rows 44, 36, 45, 52, 130;
// 1024 rows 85, 71, 55, 63, 133; 2048 rows 196, 176, 128, 112, 139; 4096 rows 256x256 176, 128x128 two 221.
struct LinTile {
  LinKind kind;
  int bm, bn;
  float one, more, two;  // one round; each of several rounds; two workgroups per compute unit (0: one fits)
};
constexpr LinTile kLinTiles[] = {{kLin64x64, 64, 64, 0.19f, 0.0f, 0.35f},
                                 {kLin64x128, 64, 128, 0.31f, 0.31f, 0.0f},
                                 {kLin128x128, 128, 128, 0.44f, 0.55f, 0.0f},
                                 {kLin128x128two, 128, 128, 0.51f, 0.0f, 0.94f},
                                 {kLin256x256, 256, 256, 1.48f, 1.48f, 0.0f}};

inline LinPlan plan_linear(int M, int N, int K, bool transposed) {
  const int KB = (K + 63) / 64;
  LinPlan best{kLin64x64, 1};
  float least = 0.0f;
  for (const LinTile& c : kLinTiles) {
    const int64_t tiles = (int64_t)((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    for (int s = 1; s <= 8; ++s) {
      // shares of at least 4 blocks, none empty, and not more workgroups than fit at once
      const int per = lin_split_blocks(KB, s);
      if (s > 1 && (per < 4 || (KB + per - 1) / per != s || tiles * s > kLinCus)) continue;
      const int64_t w = tiles * s, at_once = c.two > 0.0f ? 2 * kLinCus : kLinCus, rounds = (w + at_once - 1) / at_once;
      const float step = w <= kLinCus ? c.one : c.two > 0.0f ? c.two * (float)rounds : c.more * (float)rounds;
      // a round begins with its first copies and ends with its stores; the shares are joined by a second launch, which reads them
      const float us = (float)per * step + 2.5f + 1.5f * (float)rounds +
                       (s > 1 ? 1.8f + 0.9f * (float)s + (float)(8 * s + 2) * (float)M * (float)N / 8e6f : 0.0f);
      if (least == 0.0f || us < least) {
        least = us;
        best = {c.kind, s};
      }
    }
  }
  if (transposed || M > 64) return best;
  // Few rows: streaming workgroups whose waves share K, of 16 columns while they fit the chip once, else of 32.  us, stream and
  // tile: 16 x 4096 x 7168 11.0, 14.3; 16 x 7168 x 2048 7.2, 9.2; 32 x 256 x 7168 7.6, 9.5.  From 33 rows on a block of K takes a wave
  // longer (4 waves: 0.47 us, 32 columns 0.82), and tiles win where K is long or the columns are many: 64 x 4096 x 7168 15.9, 16.2;
  // 64 x 7168 x 2048 8.6, 9.9; 40 x 1000 x 1000 4.2, 6.2; 64 x 256 x 7168 13.8, 9.8; 64 x 14336 x 4096 33.8, 28.8.
  if (M <= 16) return {kLinStream16, 1};
  if (M <= 32) return {kLinStream32, 1};
  if (N <= 32 * kLinCus && 2.2f + (float)((KB + 3) / 4) * (N <= 16 * kLinCus ? 0.47f : 0.82f) < least) return {kLinStream64, 1};
  return best;
}

}  // namespace moe
