// dense_plan.h -- which kernel moe_gemm_fp8 takes, by sizes alone (host code that any C++ compiler takes, so that the
// choice can be tested without a GPU).
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kXcd = 8;

// K blocks of a workgroup when K is split: whole groups of 4 (a group's scales are copied at once).
constexpr int split_blocks(int KB, int splits) { return ((KB + 3) / 4 + splits - 1) / splits * 4; }

// Times in us per K block of one round of tiles over the 256 compute units, as measured with the whole chip busy (first: one
// workgroup per compute unit; second, where two fit: both); the tile with the smallest sum of rounds is taken.  Measured
// (us, N x K = 4096 x 7168, bf16 output; 64x64, 64x128, 128x128): 256 rows 16.5, 19.4, 26.4; 512 rows 26.5, 22.1, 26.7;
// 1024 rows 48.3, 42.7, 34.5; 64x128, 128x128, 256x256: 2048 rows 84, 69, 82; 4096 rows 128x128 137, 256x256 104.
enum Kind { kStream16, kStream32, kStream64, k64x64, k64x128, k128x128, k128x128two, k256x256 };
struct Plan {
  Kind kind;
  int splits;
};
struct TileCost {
  Kind kind;
  int bm, bn;
  float one, two;  // two = 0: one workgroup per compute unit
};
constexpr int kCus = 256;  // not asked of the device: the workspace's size must not depend on it, nor need one

inline Plan plan_dense(int M, int N, int K, bool wide) {
  if (M <= 16) return {kStream16, 1};
  if (M <= 32) return {kStream32, 1};
  if (M <= 64) return {kStream64, 1};
  constexpr TileCost narrow_t[] = {{k64x64, 64, 64, 0.33f, 0.57f},
                                   {k64x128, 64, 128, 0.5f, 0.0f},
                                   {k128x128, 128, 128, 0.69f, 0.0f},
                                   {k256x256, 256, 256, 1.9f, 0.0f}};
  constexpr TileCost wide_t[] = {{k64x64, 64, 64, 0.5f, 0.76f},
                                 {k64x128, 64, 128, 0.74f, 0.0f},
                                 {k128x128, 128, 128, 1.3f, 0.0f},
                                 {k128x128two, 128, 128, 1.7f, 2.05f}};
  Plan best{k64x64, 1};
  float least = 0.0f;
  int64_t best_tiles = 0;
  auto consider = [&](const TileCost& c) {
    const int64_t t = (int64_t)((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    const float f = c.two == 0.0f ? c.one * (float)((t + kCus - 1) / kCus)
                                  : (t <= kCus ? c.one : c.two * (float)((t + 2 * kCus - 1) / (2 * kCus)));
    if (best_tiles == 0 || f < least) {
      least = f;
      best.kind = c.kind;
      best_tiles = t;
    }
  };
  if (wide)
    for (const TileCost& c : wide_t) consider(c);
  else
    for (const TileCost& c : narrow_t) consider(c);
  // Few tiles and a long K: split it so that the chip fills, where that saves more than the second launch takes (131 x
  // 1000 x 7168, 48 tiles: 14.7 us whole, 12.1 in two, 11.9 in five).  A share is whole groups, at least 8 blocks but for
  // the last one, and only as many shares are launched as get blocks: 52 blocks in six would be 12, 12, 12, 12, 4 and
  // none.  (The costs here count s equal shares, as the measurements that they were fitted to did.)
  const int KB = K / 128;
  int s = (int)(kCus / best_tiles);
  if (s > KB / 8) s = KB / 8;
  if (s > 8) s = 8;
  if (s > 1 && (float)KB * least * (1.0f - 1.0f / (float)s) > 5.0f) {
    const int per = split_blocks(KB, s);
    best.splits = (KB + per - 1) / per;
  } else {
    s = 1;
  }
  // Where its workgroups of 64 x 16 outputs fit the chip once, the streaming kernel, whose waves split K among themselves (0.14
  // us per K block, in fp32 0.18), unless splitting tiles is faster or the activations, which the columns' workgroups on every
  // XCD read anew, take longer (6 TB/s).  us, tiles and streams: 192 x 1000 x 2048 6.9, 5.1, in fp32 10.3, 6.3; 131 x 512 x
  // 7168 (tiles in seven splits) 10.1, 10.9; 4096 x 64 x 7168 12.8, 19.8; more than one round, 300 x 1000 x 2048: 7.0, 8.7.
  const int64_t cols = (N + 15) / 16;
  const float tiles_us = (float)KB * least / (float)s + (s > 1 ? 5.0f : 0.0f);
  const float stream_us = (float)KB * (wide ? 0.18f : 0.14f);
  const float reread_us = (float)M * (float)K * (float)(cols < kXcd ? cols : kXcd) / 6e6f;
  if ((M + 63) / 64 * cols <= kCus && stream_us < tiles_us && reread_us < tiles_us) return {kStream64, 1};
  return best;
}

}  // namespace moe
