// linear_plan.h -- which kernel moe_gemm_bf16 takes, by sizes alone (host code that any C++ compiler takes, so that the
// choice can be tested without a GPU).
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kLinCus = 256;  // not asked of the device: the workspace's size must not depend on it, nor need one

// K blocks (of 64) of a workgroup when K is split.
constexpr int lin_split_blocks(int KB, int splits) { return (KB + splits - 1) / splits; }

enum LinKind { kLinStream16, kLinStream32, kLinStream64, kLin64x64, kLin64x128, kLin128x128, kLin256x256 };
struct LinPlan {
  LinKind kind;
  int splits;
};
struct LinTile {
  LinKind kind;
  int bm, bn;
  float one, two;  // us per K block of one round of tiles over the chip; two workgroups per compute unit (0: one fits)
};

inline LinPlan plan_linear(int M, int N, int K, bool transposed) {
  const int KB = (K + 63) / 64;
  if (!transposed) {
    if (M <= 16) return {kLinStream16, 1};
    if (M <= 32) return {kLinStream32, 1};
    if (M <= 64) return {kLinStream64, 1};
  }
  constexpr LinTile tiles[] = {{kLin64x64, 64, 64, 0.3f, 0.5f},
                               {kLin64x128, 64, 128, 0.45f, 0.0f},
                               {kLin128x128, 128, 128, 0.6f, 0.9f},
                               {kLin256x256, 256, 256, 1.5f, 0.0f}};
  LinPlan best{kLin64x64, 1};
  float least = 0.0f;
  int64_t best_tiles = 0;
  for (const LinTile& c : tiles) {
    const int64_t t = (int64_t)((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    const float f = c.two == 0.0f ? c.one * (float)((t + kLinCus - 1) / kLinCus)
                                  : (t <= kLinCus ? c.one : c.two * (float)((t + 2 * kLinCus - 1) / (2 * kLinCus)));
    if (best_tiles == 0 || f < least) {
      least = f;
      best.kind = c.kind;
      best_tiles = t;
    }
  }
  int s = best_tiles > 0 ? (int)(kLinCus / best_tiles) : 1;
  if (s > KB / 8) s = KB / 8;
  if (s > 8) s = 8;
  if (s > 1 && (float)KB * least * (1.0f - 1.0f / (float)s) > 5.0f) {
    const int per = lin_split_blocks(KB, s);
    best.splits = (KB + per - 1) / per;
  }
  return best;
}

}  // namespace moe
