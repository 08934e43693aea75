// decode_plan.h -- how moe_experts_decode divides its work, by sizes alone (host code that any C++ compiler takes, so that it can be
// tested without a GPU; the kernels take their LDS layouts from here).
#pragma once

#include <stdint.h>

namespace moe {

enum DecodeFormat { kDecBf16 = 0, kDecFp8 = 1, kDecInt4 = 2, kDecFp4 = 3 };
constexpr bool dec_half(int format) { return format == kDecInt4 || format == kDecFp4; }  // two weights a byte
constexpr int dec_block(int format) { return format == kDecBf16 ? 64 : 128; }            // K values of a block

constexpr int kLdsMost = 160 * 1024;
constexpr int kUpRing = 17 * 1024;
constexpr int kDownRing = 13 * 1024, kDownDeep = 19 * 1024, kDownShort = 9 * 1024;

// The grouping of R routes by expert, in either kernel's LDS.
constexpr int dec_plan_bytes(int R) { return 6 * R + 4; }

// Up-projection.  LDS: the waves' rings, their sums of a unit (twice where that leaves room for two workgroups on a compute unit: then
// a unit takes one barrier), the grouping.
constexpr int dec_up_blocks(int format) { return dec_half(format) ? 4 : 2; }      // of 16 weight columns, gates and ups
constexpr int dec_up_cols(int format) { return 8 * dec_up_blocks(format); }       // columns of h per unit
constexpr int dec_up_row(int format) { return 16 * dec_up_blocks(format) + 2; }   // floats
constexpr int dec_up_part(int format, int rows, int waves) { return waves * rows * dec_up_row(format); }
constexpr int dec_up_bufs(int format, int rows, int waves) {
  return 8 * dec_up_part(format, rows, waves) <= (waves == 4 ? 10 : 20) * 1024 ? 2 : 1;
}
constexpr int dec_up_plan_at(int format, int rows, int waves) {
  return waves * kUpRing + dec_up_bufs(format, rows, waves) * dec_up_part(format, rows, waves) * 4;
}
constexpr int dec_up_lds(int format, int rows, int waves, int R) { return dec_up_plan_at(format, rows, waves) + dec_plan_bytes(R); }

// Down-projection.  LDS: the rings, a line of 16 sums per share of K and route, topk_weights, the grouping.
constexpr int dec_down_lds(int waves, int ring, int ksplit, int R) {
  return waves * ring + R * (64 * ksplit + 4) + dec_plan_bytes(R);
}

struct DecodePlan {
  int rows;                      // of a job: an expert and so many of its routes
  int up_waves, up_groups;       // waves of a workgroup; workgroups
  int down_waves, down_ring, ksplit;
};

inline DecodePlan plan_decode(int format, int T, int k, int E, int H, int I, int cus) {
  DecodePlan p{};
  const int R = T * k;
  // what most experts get, so that their weights are read once
  const float mean = (float)T * (float)k / (float)E;
  p.rows = format != kDecBf16 && (mean <= 2.0f || T <= 4) ? 4 : mean <= 5.0f || T <= 8 ? 8 : 16;

  // Up: persistent workgroups of 4 waves, as many as run at once: two on a compute unit where their LDS fits twice (not with 16 rows
  // of two weights a byte, nor from about 600 routes on), else one.  128 tokens, 8 of 128 experts, 4096 x 1536, where it is one: bf16
  // 706 us with two for each compute unit, 701 with one, FP8 453 and 445, 4-bit 330 and 326; 100 tokens, 8 of 64, 2048 x 1408, 4-bit
  // 151 and 144.  (8 waves in that one: FP8 449, and 5% more or less elsewhere.)  Where there is no more than one unit of work for
  // each compute unit, 8 waves share it.
  const int64_t units = (int64_t)R * (I / dec_up_cols(format));
  const bool two = 2 * dec_up_lds(format, p.rows, 4, R) <= kLdsMost;
  p.up_waves = p.rows < 16 && units <= cus ? 8 : 4;
  const int64_t most = two && p.up_waves == 4 ? 2 * cus : cus;
  p.up_groups = (int)(units < most ? units : most);

  // Down: workgroups that have a compute unit to themselves, because there are few or because of the routes' lines, have 8 waves,
  // else 4; few routes leave room for deeper rings, and their K is shared so that every wave has a part.
  const bool few = H / 16 <= cus;
  const int blocks = I / dec_block(format), lines = dec_down_lds(0, 0, 1, R);
  const bool wide = 8 * kDownRing + lines <= kLdsMost && (few || 2 * (4 * kDownRing + lines) > kLdsMost);
  p.down_waves = wide ? 8 : 4;
  p.down_ring = kDownRing;
  if (p.rows < 16) {
    if (wide && 8 * kDownDeep + lines + 64 * 8 <= kLdsMost) p.down_ring = kDownDeep;
    if (!wide && 2 * (4 * kDownDeep + lines + 64 * 8) <= kLdsMost) p.down_ring = kDownDeep;
  }
  if (dec_half(format) && p.rows == 4 && few && 16 * kDownShort + lines + 64 * 16 <= kLdsMost) {
    p.down_waves = 16;
    p.down_ring = kDownShort;
  }
  p.ksplit = 1;
  while (p.ksplit * R < p.down_waves && 2 * p.ksplit <= blocks) p.ksplit *= 2;
  return p;
}

}  // namespace moe
