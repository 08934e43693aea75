// gemm_dense.hip -- moe_gemm_fp8: a dense FP8 product with an fp32 scale per block of 128.
//
//   D[m, n] = C[m, n] + sum_kb (sa[m,kb] * sw[n',kb]) * sum_{k in kb} a[m,k] * w[n,k]
//   n' = n / 128 (weights scaled 128x128) or n (1x128, the weight gradient's second operand)
//
// The scales are any fp32 values, so unlike the grouped GEMM's powers of two they cannot ride the
// matrix instruction: each K block's sum comes out of matrix instructions that start at zero and is promoted into the
// fp32 accumulator with one fused multiply-add.
//
// Which matrix instruction goes by the output's type.  The FP8 ones (v_mfma_f32_16x16x128_f8f6f4 here, and
// 16x16x32_fp8_fp8 alike) add groups of 8 products aligned to the largest and drop what lies below 2^-13 of its
// binade (measured: 1 + 2^-13 is kept, 1 + 2^-14 is not; products 8 apart are added in full): about 1.5e-5 of the
// result on normal data, at most 7 * 2^-13 of the sum of magnitudes.  A bf16 output rounds 100 times coarser, so it
// takes them; an fp32 output (a gradient that is added up over steps) gets its products from the bf16
// instruction, half as fast, in which E4M3 codes are exact and every product counts in full (1e-8).
//
// Tile.  A workgroup of WM x WN waves computes 16*RB*WM rows x 16*CB*WN columns.  The weight tile is the
// instruction's A operand (output columns), the activations its B operand (rows), so a lane holds 4 consecutive
// columns of one row.  Both operands' K blocks are copied global -> LDS (global_load_lds, 16-byte chunks XOR-swizzled
// through the source address) into two slots; block kb + 1 is copied while block kb is multiplied.  The barrier that
// publishes block kb + 1 sits before the promotion of the step's last row block, when every wave holds its last
// fragments of block kb in registers, so the next block's first fragments are read behind matrix instructions and
// promotions.  Scales come 4 K blocks at a time (one 16-byte copy per row).
#include "dense_plan.h"
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

// Workgroups of up to 512 threads are declared as 512: at two waves per SIMD a wave has 256 registers.  Given 512, the
// compiler takes every K block's sums through the same four accumulation registers, each matrix instruction waiting for
// the previous one's sums to be read out (a 64x64 wave tile: 125 clocks per instruction instead of 32).
#define TWO_WAVES __launch_bounds__(512)

// barrier_lds() whose wait the compiler sees: it then knows that fragments read before the barrier are in registers,
// instead of waiting for the reads issued since.
__device__ __forceinline__ void barrier_reads() {
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}

// 64 lanes x 16 bytes global -> LDS: lane i's bytes from base + voff to lds + 16 i.
__device__ __forceinline__ void copy16(uint32_t voff, const void* base, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(voff), "s"(base), "{m0}"(lds) : "memory");
}

// The bf16 values of 8 E4M3 codes (exact).
__device__ __forceinline__ v8bf to_bf16(int lo, int hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A lane's 32 values of one K block of a row, as the matrix instruction takes them.
template <bool WIDE>
struct Frag {
  v8i v;
  __device__ __forceinline__ void load(const v4i lo, const v4i hi) {
    v = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }
  __device__ __forceinline__ void take(const Frag<false>& c) { v = c.v; }
};
template <>
struct Frag<true> {
  v8bf v[4];
  __device__ __forceinline__ void load(const v4i lo, const v4i hi) {
    v[0] = to_bf16(lo[0], lo[1]);
    v[1] = to_bf16(lo[2], lo[3]);
    v[2] = to_bf16(hi[0], hi[1]);
    v[3] = to_bf16(hi[2], hi[3]);
  }
  __device__ __forceinline__ void take(const Frag<false>& c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) take_quarter(c, i);
  }
  __device__ __forceinline__ void take_quarter(const Frag<false>& c, int i) {
    v[i] = to_bf16(c.v[2 * i], c.v[2 * i + 1]);
  }
};
__device__ __forceinline__ v4f block_sum(const Frag<false>& w, const Frag<false>& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7f7f7f7f, 0,
                                                          0x7f7f7f7f);
}
__device__ __forceinline__ v4f block_sum(const Frag<true>& w, const Frag<true>& x) {
  v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], s, 0, 0, 0);
  return s;
}

// Vectors of D and C, whose rows begin at any element (global memory takes them at any address).
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t v2u_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t v4u_any __attribute__((ext_vector_type(4), aligned(2)));

// Four consecutive columns n .. n + 3 of row m; NT: fp32 past the caches.
template <bool NT>
__device__ __forceinline__ void store4(const DenseArgs& a, int m, int n, v4f v) {
  if (m >= a.M || n >= a.N) return;
  const int64_t at = (int64_t)m * a.ldd + n;
  if (n + 4 <= a.N) {
    if (a.f32) {
      if (a.C) v += *(const v4f_any*)(a.C + (int64_t)m * a.ldc + n);
      if constexpr (NT) __builtin_nontemporal_store(v, (v4f_any*)((float*)a.D + at));
      else *(v4f_any*)((float*)a.D + at) = v;
    } else {
      *(v2u_any*)((uint16_t*)a.D + at) = v2u_any{f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16),
                                                 f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16)};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.N) return;
    if (a.f32)
      ((float*)a.D)[at + i] = a.C ? v[i] + a.C[(int64_t)m * a.ldc + n + i] : v[i];
    else
      ((uint16_t*)a.D)[at + i] = (uint16_t)f32_to_bf16_rne(v[i]);
  }
}

// Eight columns n .. n + 7 of row m as bf16 pairs.
__device__ __forceinline__ void store8(const DenseArgs& a, int m, int n, const v4f v) {
  if (m >= a.M || n >= a.N) return;
  uint16_t* d = (uint16_t*)a.D + (int64_t)m * a.ldd + n;
  v4u_any p;
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = __float_as_uint(v[i]);
  if (n + 8 <= a.N) {
    *(v4u_any*)d = p;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (n + e < a.N) d[e] = (uint16_t)(p[e >> 1] >> 16 * (e & 1));
}

// Lanes 8 .. 15 of each row of 16 get b of lane - 8 in a; lanes 0 .. 7 get a of lane + 8 in b.
__device__ __forceinline__ void swap8(v4f& a, v4f& b) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int x = __float_as_int(a[e]), y = __float_as_int(b[e]);
    a[e] = __int_as_float(__builtin_amdgcn_update_dpp(x, y, 0x128, 0xF, 0xC, false));  // row_ror:8, lanes 8 .. 15
    b[e] = __int_as_float(__builtin_amdgcn_update_dpp(y, x, 0x128, 0xF, 0x3, false));
  }
}

// Of the lanes' 4 columns in two neighbouring 16-column blocks, rounded to bf16: lane group lg gets 8 columns, of block lg & 1,
// from 8 (lg >> 1) on.
__device__ __forceinline__ v4f join_columns(const v4f a, const v4f b) {
  v4f o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t x = f32_to_bf16_rne(a[2 * h]) | (f32_to_bf16_rne(a[2 * h + 1]) << 16);
    const uint32_t y = f32_to_bf16_rne(b[2 * h]) | (f32_to_bf16_rne(b[2 * h + 1]) << 16);
    const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);  // x of groups 1, 3 for y of groups 0, 2
    o[h] = __uint_as_float(r[0]);
    o[2 + h] = __uint_as_float(r[1]);
  }
  return o;
}

template <int RB, int CB, int WM, int WN, int S>
struct TileCfg {
  static constexpr int NW = WM * WN;
  static constexpr int BM = 16 * RB * WM, BN = 16 * CB * WN;
  static constexpr int kPieces = (BM + BN) / 8;  // 1 KB copies (8 rows) per K block
  static constexpr int kPw = kPieces / NW;       // per wave
  static constexpr int kSlot = (BM + BN) * 128;
  static constexpr int kScale = (BM + BN) * 16;  // one group of 4 K blocks
  // Scale groups are copied kAhead groups before their first block: at least 3 blocks' copies are issued after a
  // group's and before the wait that precedes its first use, more than that wait leaves in flight (S - 2 blocks).
  static constexpr int kAhead = S > 5 ? 2 : 1, kScBufs = 2 * kAhead;
  static constexpr int kScOff = S * kSlot;
  static constexpr int kLds = kScOff + kScBufs * kScale;
  static_assert(kPieces % NW == 0, "every wave copies the same number of pieces");
  static_assert(S >= 2 && S <= 4 * kAhead + 1 && kPw * (S - 1) < 64, "scales ahead of their use; vmcnt's range");
  static_assert((BM + BN) % 64 == 0 && BM % 64 == 0, "scale rows in whole waves");
  static_assert(kLds <= 160 * 1024, "LDS");
};

// A workgroup's tile: where it lies, the copies of its operands and scales into LDS, and the reads of them.
template <bool GRAN1, int RB, int CB, int WM, int WN, int S>
struct Tile {
  using C = TileCfg<RB, CB, WM, WN, S>;
  const DenseArgs& a;
  uint8_t* sm;
  uint32_t lds0;
  int lane, wv, l16, lg, KB, kb0, kb1, m0, n0, wm, wn;
  const uint8_t *abase, *wbase;
  uint32_t voff[C::kPw];
  int off_lo, off_hi;
  bool sc_vec;

  __device__ __forceinline__ Tile(const DenseArgs& args, uint8_t* smem) : a(args), sm(smem) {
    lane = lane_id();
    wv = uniform(threadIdx.x >> 6);
    l16 = lane & 15;
    lg = lane >> 4;
    lds0 = lds_offset(sm);
    KB = a.K / 128;
    // this workgroup's K blocks (split K: a multiple of 4 per split)
    const int per_split = split_blocks(KB, a.splits);
    kb0 = uniform(min((int)blockIdx.y * per_split, KB));
    kb1 = uniform(min(kb0 + per_split, KB));
    // Workgroup b runs on XCD b % 8: consecutive tiles go to one XCD, and consecutive tiles are blocks of up to 8
    // column tiles by a few row tiles, so an XCD's workgroups share both operands in its L2.
    const int mt = (a.M + C::BM - 1) / C::BM, nt = (a.N + C::BN - 1) / C::BN, tiles = mt * nt;
    const int per = tiles / kXcd, rem = tiles % kXcd, x = blockIdx.x % kXcd;
    const int t = x * per + min(x, rem) + blockIdx.x / kXcd;
    const int gn = 8, g = t / (mt * gn), gw = min(gn, nt - g * gn), r = t - g * mt * gn;
    m0 = uniform(r / gw * C::BM);
    n0 = uniform((g * gn + r % gw) * C::BN);
    wm = (wv / WN) * 16 * RB;
    wn = (wv % WN) * 16 * CB;
    // copies: this wave's pieces q = wv, wv + NW, ...; rows of the A tile, then of the W tile
    abase = a.A + (int64_t)m0 * a.lda;
    wbase = a.W + (int64_t)n0 * a.ldw;
#pragma unroll
    for (int i = 0; i < C::kPw; ++i) {
      const int row = 8 * (wv + C::NW * i) + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
      voff[i] = row < C::BM ? (uint32_t)min(row, a.M - 1 - m0) * (uint32_t)a.lda + 16u * c
                            : (uint32_t)min(row - C::BM, a.N - 1 - n0) * (uint32_t)a.ldw + 16u * c;
    }
    // fragment read offsets: row l16 of a 16-row block at 128 l16, its chunk c at position c ^ ((row >> 1) & 7)
    const int fsw = (l16 >> 1) & 7;
    off_lo = l16 * 128 + 16 * (lg ^ fsw);
    off_hi = l16 * 128 + 16 * ((4 + lg) ^ fsw);
    sc_vec = KB % 4 == 0 && (((uintptr_t)a.SFA | (uintptr_t)a.SFW) & 15) == 0;
  }

  __device__ __forceinline__ void copy_piece(int kb, int i) const {
    const int q = wv + C::NW * i;
    const uint8_t* base = (8 * q < C::BM ? abase : wbase) + (int64_t)kb * 128;
    copy16(voff[i], base, uniform(lds0 + (kb % S) * C::kSlot + 1024 * q));
  }
  // The K block that a0 and w0 point at, a wave's piece i, into slot SLOT.  (The copy's offset field moves its LDS address
  // too, so the block's offset is in the pointers.)
  template <int SLOT>
  __device__ __forceinline__ void copy_piece_at(const uint8_t* a0, const uint8_t* w0, int i) const {
    const int q = wv + C::NW * i;
    copy16(voff[i], 8 * q < C::BM ? a0 : w0, uniform(lds0 + SLOT * C::kSlot + 1024 * q));
  }
  // the scales of K blocks 4 g4 .. of row r of the tiles at 16 r of a group buffer
  __device__ __forceinline__ int scale_buf(int g4) const { return C::kScOff + (g4 & (C::kScBufs - 1)) * C::kScale; }
  __device__ __forceinline__ void copy_scales(int g4) const {
#pragma unroll
    for (int q = 0; q < (C::BM + C::BN) / 64; q += C::NW) {
      const int p = q + wv;
      if (p * 64 >= C::BM + C::BN) break;
      const int row = 64 * p + lane;
      const bool is_a = 64 * p < C::BM;
      const float* base = is_a ? a.SFA : a.SFW;
      const int sr = is_a ? min(m0 + row, a.M - 1) : min(n0 + row - C::BM, a.N - 1) / (GRAN1 ? 1 : 128);
      if (sc_vec) {
        const int sr0 = is_a ? m0 : n0 / (GRAN1 ? 1 : 128);
        copy16((uint32_t)(sr - sr0) * (uint32_t)KB * 4u, base + (int64_t)sr0 * KB + 4 * g4,
               uniform(lds0 + scale_buf(g4) + 1024 * p));
      } else {
        const float* s = base + (int64_t)sr * KB;
        v4f v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = s[min(4 * g4 + j, KB - 1)];
        *(v4f*)(sm + scale_buf(g4) + 16 * row) = v;
      }
    }
  }
  // before step kb: the group that is first used kAhead groups later
  __device__ __forceinline__ void copy_scales_at(int kb) const {
    if ((kb & 3) == 0 && kb + 4 * C::kAhead < kb1) copy_scales((kb >> 2) + C::kAhead);
  }

  template <typename F>
  __device__ __forceinline__ void frag(F& f, int kb, int row) const {
    const uint8_t* p = sm + (kb % S) * C::kSlot + row * 128;
    f.load(*(const v4i*)(p + off_lo), *(const v4i*)(p + off_hi));
  }
  __device__ __forceinline__ void read_scales(int kb, float (&sa)[RB], v4f (&sw)[GRAN1 ? CB : 1]) const {
    const float* s = (const float*)(sm + scale_buf(kb >> 2)) + (kb & 3);
#pragma unroll
    for (int i = 0; i < RB; ++i) sa[i] = s[4 * (wm + 16 * i + l16)];
    if constexpr (GRAN1) {
#pragma unroll
      for (int j = 0; j < CB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sw[j][e] = s[4 * (C::BM + wn + 16 * j + 4 * lg + e)];
    } else {
      sw[0][0] = s[4 * (C::BM + wn)];
    }
  }

  // A lane's sums are 4 columns of one row per 16x16 block; stored so, an instruction writes 16 rows in pieces of 32 bytes (bf16)
  // or 64. Lanes exchange columns first, so that it writes whole 128-byte lines of 8 rows (bf16 tiles of 32 columns a wave: 64
  // bytes of 16 rows); C is read in the same order.  (4096 x 4096 x 128 in bf16: 16.7 -> 15.4 us; 4096 x 7168 x 128
  // in fp32: 38.4 -> 28.6 us.)
  __device__ __forceinline__ void store(v4f (&acc)[RB][CB]) const {
    static_assert(CB == 2 || CB == 4, "columns are exchanged in pairs");
    // The sums are whole before any lane's store is masked off: without this the compiler moves the last matrix
    // instructions, and the loads of their operands, under the stores' masks, where the other lanes' operands are stale.
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < CB; ++j) asm volatile("" : "+v"(acc[i][j]));
    DenseArgs o = a;
    if (a.splits > 1) {  // this split's sums, whole rows of 4
      o.f32 = 1;
      o.C = nullptr;
      o.N = (a.N + 3) & ~3;
      o.ldd = o.N;
      o.D = a.ws + (int64_t)blockIdx.y * a.M * o.N;
    }
    const int hi = l16 >> 3, l8 = l16 & 7, m = m0 + wm, n = n0 + wn;
    if (o.f32) {
      // past the caches where lines are written whole (4096 x 4096 x 1024: 40.5 us without, 35.9 with); rows that share their
      // lines with their neighbours' pieces meet them in the L2 (4096 x 4095 x 1024: 41.4 us, past it 45.6)
      auto put = [&](auto nt) {
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
          for (int j = 0; j < CB; j += 2) {
            v4f v[2] = {acc[i][j], acc[i][j + 1]};
            swap8(v[0], v[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              store4<decltype(nt)::value != 0>(o, m + 16 * i + 8 * h + l8, n + 16 * (j + hi) + 4 * lg, v[h]);
          }
      };
      if (o.ldd % 4 == 0) put(IntC<1>{});
      else put(IntC<0>{});
      return;
    }
    const int n8 = n + 16 * (lg & 1) + 8 * (lg >> 1);
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      v4f v[CB / 2];  // 8 columns of bf16 each
#pragma unroll
      for (int j = 0; j < CB; j += 2) v[j / 2] = join_columns(acc[i][j], acc[i][j + 1]);
      if constexpr (CB == 4) {
        swap8(v[0], v[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) store8(o, m + 16 * i + 8 * h + l8, n8 + 32 * hi, v[h]);
      } else {
        store8(o, m + 16 * i + l16, n8, v[0]);
      }
    }
  }
};

// One K block's sum into the accumulator.
template <bool GRAN1>
__device__ __forceinline__ void promote(v4f& acc, const v4f sum, float sa, const v4f sw) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(sum[e], GRAN1 ? sa * sw[e] : sa, acc[e]);
}

// Tiles whose fragments fit the registers twice: block kb + 1's fragments and scales are read while block kb is
// multiplied, and block kb + 4 is copied meanwhile into the slot that block kb left when it was read.  With few matrix
// instructions per step a wave's time is its instruction count, so the loop is unrolled over the 4 slots (and the 4 blocks of
// a scale group): slots, offsets and scale positions are constants.  Measured per K block with the chip full: 64x64 0.33 us
// (two workgroups on a compute unit 0.57), 64x128 0.50, 128x128 0.69.  131 x 7168 x 2048, 168 tiles of 64x128, weights from
// HBM: 11.0 us (9.0 where the caches hold them); the steps wait for copies: with every tile reading the same operands 8.8.
template <bool WIDE, bool GRAN1, int RB, int CB, int WM, int WN>
__global__ TWO_WAVES void gemm_dense_small_kernel(const DenseArgs a) {
  constexpr int S = 4;
  using C = TileCfg<RB, CB, WM, WN, S>;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[C::kLds];
  const Tile<GRAN1, RB, CB, WM, WN, S> T(a, sm);
  const int kb0 = T.kb0, kb1 = T.kb1;  // kb0 is a multiple of 4: block kb lies in slot (kb - kb0) & 3 = kb & 3
  v4f acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  struct Regs {
    Frag<false> w[CB], x[RB];  // codes; widened when multiplied
    float sa[RB];
    v4f sw[GRAN1 ? CB : 1];
  } reg[2];
  const uint8_t* pa = sm + T.wm * 128;
  const uint8_t* pw = sm + (C::BM + T.wn) * 128;
  // fragment f (columns first, then rows) of a block in slot `slot`
  auto read_frag = [&](Regs& r, int slot, int f) {
    const uint8_t* p = f < CB ? pw + slot * C::kSlot + 2048 * f : pa + slot * C::kSlot + 2048 * (f - CB);
    Frag<false>& to = f < CB ? r.w[f < CB ? f : 0] : r.x[f < CB ? 0 : f - CB];
    to.load(*(const v4i*)(p + T.off_lo), *(const v4i*)(p + T.off_hi));
  };
  auto read_scales = [&](Regs& r, int slot, const float* sc) {  // sc: the block's scale group
#pragma unroll
    for (int i = 0; i < RB; ++i) r.sa[i] = sc[4 * (T.wm + 16 * i + T.l16) + slot];
    if constexpr (GRAN1) {
#pragma unroll
      for (int j = 0; j < CB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) r.sw[j][e] = sc[4 * (C::BM + T.wn + 16 * j + 4 * T.lg + e) + slot];
    } else {
      r.sw[0][0] = sc[4 * (C::BM + T.wn) + slot];
    }
  };
  // Multiply a block; beside its matrix instructions, one piece of the other work after each: fragments of the next
  // block (more), copies (copies), promotions two tiles behind.  Issued in one go, the reads, the copies and the matrix
  // instructions take turns instead of overlapping: every wave waits at the same queue.
  auto multiply = [&](const Regs& r, bool more, Regs& next, int next_slot, const float* next_sc, bool copies,
                      auto copy) {
    constexpr int NM = RB * CB, NF = RB + CB, D = NM > 2 ? 2 : 1;
    Frag<WIDE> w[CB], x;
#pragma unroll
    for (int j = 0; j < CB; ++j) w[j].take(r.w[j]);
    v4f sum[D + 1];
    static_for<0, NM + D>([&](auto mc) {
      constexpr int m = decltype(mc)::value;
      if constexpr (m < NM) {
        if constexpr (m % CB == 0) x.take(r.x[m / CB]);
        sum[m % (D + 1)] = block_sum(w[m % CB], x);
        if (more) {
#pragma unroll
          for (int f = 0; f < NF; ++f)
            if (f * NM / NF == m) read_frag(next, next_slot, f);
          if (m == NM - 1) read_scales(next, next_slot, next_sc);
        }
        if (copies) {
#pragma unroll
          for (int i = 0; i < C::kPw; ++i)
            if (i * NM / C::kPw == m) copy(i);
        }
      }
      if constexpr (m >= D) {
        constexpr int o = m - D, oi = o / CB, oj = o % CB;
        promote<GRAN1>(acc[oi][oj], sum[o % (D + 1)], GRAN1 ? r.sa[oi] : r.sa[oi] * r.sw[0][0], r.sw[GRAN1 ? oj : 0]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  auto scale_group = [&](int kb) { return (const float*)(sm + T.scale_buf(kb >> 2)); };

  if (kb0 < kb1) {
    const uint8_t *a0 = T.abase + (int64_t)kb0 * 128, *w0 = T.wbase + (int64_t)kb0 * 128;
    T.copy_scales(kb0 >> 2);
    static_for<0, S>([&](auto u) {
      if (kb0 + decltype(u)::value < kb1) {
#pragma unroll
        for (int i = 0; i < C::kPw; ++i) T.template copy_piece_at<decltype(u)::value>(a0, w0, i);
      }
      a0 += 128;
      w0 += 128;
    });
    const bool full = kb0 + S <= kb1;
    if (full)
      wait_vmcnt<C::kPw*(S - 1)>();
    else
      wait_vmcnt<0>();
    barrier_reads();
#pragma unroll
    for (int f = 0; f < RB + CB; ++f) read_frag(reg[0], 0, f);
    read_scales(reg[0], 0, scale_group(kb0));
    if (full) wait_vmcnt<C::kPw*(S - 2)>();
    barrier_reads();  // block kb0 is in registers, block kb0 + 1 in LDS
    // kind 2: block k + S is copied; 1: no more copies, but a next block; 0: the last block
    auto step = [&](int k, auto uc, auto kind) {
      constexpr int u = decltype(uc)::value;
      constexpr bool more = decltype(kind)::value > 0, copies = decltype(kind)::value == 2;
      if constexpr (u == 0) T.copy_scales_at(k);
      multiply(reg[u & 1], more, reg[(u + 1) & 1], (u + 1) & 3, scale_group(k + 1), copies,
               [&](int i) { T.template copy_piece_at<u>(a0, w0, i); });
      if constexpr (copies) {
        a0 += 128;
        w0 += 128;
      }
      if constexpr (more) {
        wait_vmcnt<copies ? C::kPw*(S - 2) : 0>();
        barrier_reads();
      }
    };
    int kb = kb0;
    for (; kb + 2 * S <= kb1; kb += S)  // whole rounds of the ring
      static_for<0, S>([&](auto u) { step(kb + decltype(u)::value, u, IntC<2>{}); });
    for (; kb < kb1; kb += S)
      static_for<0, S>([&](auto u) {
        const int k = kb + decltype(u)::value;
        if (k + S < kb1) step(k, u, IntC<2>{});
        else if (k + 1 < kb1) step(k, u, IntC<1>{});
        else if (k < kb1) step(k, u, IntC<0>{});
      });
  }
  T.store(acc);
}

// The 256x256 tile (8 waves of 128x64: two per SIMD, so that one wave's promotions run beside the other's matrix
// instructions; a wave's 128 accumulators leave room for its fragments once), and in bf16 instructions the 128x128 tile (4
// waves of 64x64, two workgroups per compute unit).  A 256x256 tile copies 64 KB in and reads 192 KB per K block.
// 4096 x 4096 x 7168: 106 us, 2.26 PFLOP/s; 1.6 us per K block and 13 us at the ends (first copies, stores).  Counters of
// that run: matrix instructions 52% of the time at 2.03 GHz, other vector instructions 35%, LDS 26%: the first two overlap
// little, although two waves a SIMD that do nothing else overlap them (16 clocks a matrix instruction in bf16, with four others
// beside it 26).  Memory is not what bounds it: with every tile reading the same operands it takes 5% less.  4096 x 7168 x 4096
// with 1x128 scales, fp32 output and an addend: 246 to 265 us, 0.91 to 0.98 PFLOP/s; beside each 16-clock matrix instruction 4.4 others are
// issued (conversions and promotions; 128x128 scales save one: 221 us).
// The step:
//  * row blocks 0 .. RB-3 in turn, their fragments read two blocks ahead;
//  * then the barrier that publishes block kb + 1, every fragment of block kb being in registers, and the last two row
//    blocks column by column: after column j's two matrix instructions its weight fragment is read anew for block kb + 1;
//  * block kb + 2 is copied into the half slots that block kb leaves: its weights from the first row block of step kb on (a
//    second barrier says that every wave has read them), its activations from the barrier on, so that a copy has about 1.75 and one
//    step to arrive.
template <bool WIDE, bool GRAN1, int RB, int CB, int WM, int WN>
__global__ TWO_WAVES void gemm_dense_kernel(const DenseArgs a) {
  constexpr int S = 2;
  using C = TileCfg<RB, CB, WM, WN, S>;
  static_assert(RB >= 4 && RB % 4 == 0 && C::kPw == 2 * CB && C::BM == 8 * C::NW * CB,
                "fragment ring; a wave's first CB pieces are rows of A, its last CB rows of W");
  static_assert(!WIDE || CB == 4, "a row's 4 quarters are widened beside 4 columns");
  __shared__ __attribute__((aligned(1024))) uint8_t sm[C::kLds];
  const Tile<GRAN1, RB, CB, WM, WN, S> T(a, sm);
  const int kb0 = T.kb0, kb1 = T.kb1;
  v4f acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  Frag<false> xr[4];          // row fragments as read, in a ring
  Frag<WIDE> w[CB], xw[2];    // as multiplied (xw: WIDE only)
  auto x = [&](int i) -> const Frag<WIDE>& {
    if constexpr (WIDE) return xw[i & 1];
    else return xr[i & 3];
  };

  // kind 2: block kb + 2 exists; 1: block kb + 1 does; 0: the last block
  auto step = [&](int kb, auto kind) {
    constexpr int more = decltype(kind)::value;
    float sa[RB];
    v4f sw[GRAN1 ? CB : 1];
    T.read_scales(kb, sa, sw);
    v4f sum[2][CB];
    auto prom = [&](int i, int j) {
      promote<GRAN1>(acc[i][j], sum[i & 1][j], GRAN1 ? sa[i] : sa[i] * sw[0][0], sw[GRAN1 ? j : 0]);
    };
#pragma unroll
    for (int i = 0; i < RB - 2; ++i) {
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        sum[i & 1][j] = block_sum(w[j], x(i));
        if (j == 0) T.frag(xr[(i + 2) & 3], kb, T.wm + 16 * (i + 2));
        if constexpr (WIDE) xw[(i + 1) & 1].take_quarter(xr[(i + 1) & 3], j);
        if constexpr (more == 2) {  // the weights of block kb + 2
          const int c = RB >= 8 ? (j == 2 ? i - 1 : -1) : (i == 1 ? j : -1);
          if (c >= 0 && c < CB) T.copy_piece(kb + 2, CB + c);
        }
        if (i > 0) prom(i - 1, j);
        __builtin_amdgcn_sched_barrier(0);  // one piece of the other work after each matrix instruction
      }
      // every wave has used its weight fragments of block kb, i.e. read them: their half of the slot is free
      if constexpr (more == 2)
        if (i == 0) asm volatile("s_barrier" ::: "memory");
    }
    if constexpr (more > 0) {
      wait_vmcnt<more == 2 ? CB : 0>();  // all but block kb + 2's weights
      barrier_reads();
    }
    Frag<WIDE> xl = x(RB - 2), xm;  // the last two rows
    xm.take(xr[(RB - 1) & 3]);
    Frag<false> wr[2];
    if constexpr (more > 0) {
      T.frag(xr[0], kb + 1, T.wm);
      T.frag(xr[1], kb + 1, T.wm + 16);
    }
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      const v4f s0 = block_sum(w[j], xl), s1 = block_sum(w[j], xm);
      prom(RB - 3, j);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (more > 0) T.frag(wr[j & 1], kb + 1, C::BM + T.wn + 16 * j);
      if constexpr (more == 2) T.copy_piece(kb + 2, j);
      if constexpr (more > 0)
        if (j > 0) w[j - 1].take(wr[(j - 1) & 1]);
      sum[(RB - 2) & 1][j] = s0;
      prom(RB - 2, j);
      sum[(RB - 1) & 1][j] = s1;
      prom(RB - 1, j);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (more > 0) {
      w[CB - 1].take(wr[(CB - 1) & 1]);
      if constexpr (WIDE) xw[0].take(xr[0]);
    }
  };

  if (kb0 < kb1) {
    T.copy_scales(kb0 >> 2);
#pragma unroll
    for (int i = 0; i < C::kPw; ++i) T.copy_piece(kb0, i);
    wait_vmcnt<0>();
    barrier_reads();
    T.frag(xr[0], kb0, T.wm);
    T.frag(xr[1], kb0, T.wm + 16);
    if constexpr (WIDE) xw[0].take(xr[0]);
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      Frag<false> f;
      T.frag(f, kb0, C::BM + T.wn + 16 * j);
      w[j].take(f);
    }
    if (kb0 + 1 < kb1) {
#pragma unroll
      for (int i = 0; i < C::kPw; ++i) T.copy_piece(kb0 + 1, i);
    }
    int kb = kb0;
    for (; kb + 2 < kb1; ++kb) {
      T.copy_scales_at(kb);
      step(kb, IntC<2>{});
    }
    if (kb + 1 < kb1) {
      T.copy_scales_at(kb);
      step(kb, IntC<1>{});
      ++kb;
    }
    step(kb, IntC<0>{});
  }
  T.store(acc);
}

// Split K: the splits' partial sums, added in split order, and the addend.
__global__ __launch_bounds__(256) void gemm_dense_join_kernel(const DenseArgs a) {
  const int np = (a.N + 3) / 4;
  const int64_t total = (int64_t)a.M * np;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total; q += (int64_t)gridDim.x * 256) {
    v4f v = *(const v4f*)(a.ws + 4 * q);
    for (int k = 1; k < a.splits; ++k) v += *(const v4f*)(a.ws + 4 * (q + k * total));
    store4<false>(a, (int)(q / np), 4 * (int)(q % np), v);
  }
}

hipError_t launch_join(const DenseArgs& a, hipStream_t s) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t need = ((int64_t)a.M * ((a.N + 3) / 4) + 255) / 256, cap = (int64_t)device_info().cus * 16;
  gemm_dense_join_kernel<<<(unsigned)(need < cap ? need : cap), 256, 0, s>>>(a);
  return hipGetLastError();
}
template <bool WIDE, bool GRAN1, int RB, int CB, int WM, int WN>
hipError_t launch_small(const DenseArgs& a, hipStream_t s) {
  using C = TileCfg<RB, CB, WM, WN, 4>;
  const dim3 grid(((a.M + C::BM - 1) / C::BM) * ((a.N + C::BN - 1) / C::BN), a.splits);
  gemm_dense_small_kernel<WIDE, GRAN1, RB, CB, WM, WN><<<grid, WM * WN * 64, 0, s>>>(a);
  return launch_join(a, s);
}
template <bool WIDE, bool GRAN1, int RB, int CB, int WM, int WN>
hipError_t launch_big(const DenseArgs& a, hipStream_t s) {
  using C = TileCfg<RB, CB, WM, WN, 2>;
  const dim3 grid(((a.M + C::BM - 1) / C::BM) * ((a.N + C::BN - 1) / C::BN), a.splits);
  gemm_dense_kernel<WIDE, GRAN1, RB, CB, WM, WN><<<grid, WM * WN * 64, 0, s>>>(a);
  return launch_join(a, s);
}

// Few rows (a decode step) or few outputs: every weight byte is used by one wave, so waves need nothing from one another.  A
// workgroup takes 16 CB columns and all 16 RB rows; its KS waves split K into runs of groups of 4 blocks, each
// with a ring of S blocks of its own in LDS (no barrier in the loop), and meet once at the end, where the partial
// sums are added in wave order.  The way through LDS is for the load path: a fragment's lanes hold 16 different
// rows, and loads in that order (4 lanes on 4 cache lines) pass a quarter of the bytes per clock that rows copied
// whole do (64 rows x 4096 x 7168: 22 us with direct fragment loads).  Scales come like the rows, a group's 4 blocks
// with one 16-byte copy per row.
template <int RB, int CB, int KS, int S>
struct StreamCfg {
  static constexpr int kBlock = (RB + CB) * 2048, kPieces = 2 * (RB + CB);
  static constexpr int kScRows = 16 * (RB + CB);                 // rows with scales: activations, then columns
  static constexpr int kScCopies = (kScRows + 63) / 64, kScale = kScCopies * 1024;
  static constexpr int kWave = S * kBlock + 2 * kScale;
  static constexpr int kPart = 16 * RB * (16 * CB + 4) * 4;      // a wave's partial sums, over its ring
  static constexpr int kLds = KS * kWave;
  static_assert(kPart <= kWave && kLds <= 160 * 1024, "LDS");
  static_assert(S >= 2 && S <= 4, "a group's scales are copied at most one group ahead");
};

template <bool WIDE, bool GRAN1, int RB, int CB, int KS, int S>
__global__ TWO_WAVES void gemm_stream_kernel(const DenseArgs a) {
  using C = StreamCfg<RB, CB, KS, S>;
  constexpr int kRows = 16 * RB, kCols = 16 * CB;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[C::kLds];
  const int lane = lane_id(), wv = uniform(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int KB = a.K / 128, groups = (KB + 3) / 4;
  const int n0 = blockIdx.x * kCols, m0 = blockIdx.y * kRows;
  const int per = (groups + KS - 1) / KS;
  const int kb0 = min(4 * wv * per, KB), nb = min(kb0 + 4 * per, KB) - kb0;
  const bool sc_vec = KB % 4 == 0 && (((uintptr_t)a.SFA | (uintptr_t)a.SFW) & 15) == 0;
  uint8_t* ring = sm + wv * C::kWave;
  uint8_t* scl = ring + S * C::kBlock;

  // sources of this lane's copies: piece q (1 KB) is rows 8q .. 8q + 7 of the activations, then of the columns
  const uint8_t* src[C::kPieces];
#pragma unroll
  for (int q = 0; q < C::kPieces; ++q) {
    const int row = 8 * q + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
    src[q] = 8 * q < kRows ? a.A + (int64_t)min(m0 + row, a.M - 1) * a.lda : a.W + (int64_t)min(n0 + row - kRows, a.N - 1) * a.ldw;
    src[q] += (int64_t)kb0 * 128 + 16 * c;
  }
  const float* ssrc[C::kScCopies];
#pragma unroll
  for (int q = 0; q < C::kScCopies; ++q) {
    const int row = min(64 * q + lane, C::kScRows - 1);
    ssrc[q] = row < kRows ? a.SFA + (int64_t)min(m0 + row, a.M - 1) * KB
                          : a.SFW + (int64_t)(min(n0 + row - kRows, a.N - 1) / (GRAN1 ? 1 : 128)) * KB;
    ssrc[q] += kb0;
  }
  auto issue = [&](int b) {  // block b of this wave's run
    if ((b & 3) == 0) {
      uint8_t* dst = scl + ((b >> 2) & 1) * C::kScale;
      // float u of row r: at 4 r + u where rows can be copied as vectors, else at 64 u + r (per 64 rows)
#pragma unroll
      for (int q = 0; q < C::kScCopies; ++q) {
        if (sc_vec) {
          dma16(ssrc[q] + b, dst + 1024 * q);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) dma4(ssrc[q] + min(b + u, KB - 1 - kb0), dst + 1024 * q + 256 * u);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < C::kPieces; ++q) dma16(src[q] + (int64_t)b * 128, ring + (b % S) * C::kBlock + 1024 * q);
  };

  const int fsw = (l16 >> 1) & 7;
  const int off_lo = l16 * 128 + 16 * (lg ^ fsw), off_hi = l16 * 128 + 16 * ((4 + lg) ^ fsw);
  v4f acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int b = 0; b < S - 1; ++b)
    if (b < nb) issue(b);
  for (int b = 0; b < nb; ++b) {
    if (b + S - 1 < nb) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot's last reads are in registers
      issue(b + S - 1);
      wait_vmcnt<(S - 1) * C::kPieces>();
    } else {
      wait_vmcnt<0>();
    }
    asm volatile("" ::: "memory");  // reads below stay behind the wait
    const uint8_t* blk = ring + (b % S) * C::kBlock;
    const float* sc = (const float*)(scl + ((b >> 2) & 1) * C::kScale);
    auto scale = [&](int row) { return sc_vec ? sc[4 * row + (b & 3)] : sc[(row & ~63) * 4 + 64 * (b & 3) + (row & 63)]; };
    Frag<WIDE> x[RB];
    float sa[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      x[i].load(*(const v4i*)(blk + 2048 * i + off_lo), *(const v4i*)(blk + 2048 * i + off_hi));
      sa[i] = scale(16 * i + l16);
    }
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      Frag<WIDE> w;
      w.load(*(const v4i*)(blk + 2048 * (RB + j) + off_lo), *(const v4i*)(blk + 2048 * (RB + j) + off_hi));
      float sw[GRAN1 ? 4 : 1];
#pragma unroll
      for (int e = 0; e < (GRAN1 ? 4 : 1); ++e) sw[e] = scale(kRows + 16 * j + (GRAN1 ? 4 * lg + e : 0));
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const v4f p = block_sum(w, x[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e], sa[i] * sw[GRAN1 ? e : 0], acc[i][j][e]);
      }
    }
  }
  // over the wave's own ring, whose copies have all landed and been read; lane: columns 4 lg .. + 3 of row l16
  float* part = (float*)ring;
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) *(v4f*)(part + (16 * i + l16) * (kCols + 4) + 16 * j + 4 * lg) = acc[i][j];
  __syncthreads();
  for (int q = threadIdx.x; q < kRows * kCols / 4; q += KS * 64) {
    const int m = q / (kCols / 4), n = 4 * (q % (kCols / 4));
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KS; ++k) v += *(const v4f*)((const float*)(sm + k * C::kWave) + m * (kCols + 4) + n);
    store4<false>(a, m0 + m, n0 + n, v);
  }
}

template <bool WIDE, bool GRAN1, int RB, int CB, int KS, int S>
hipError_t launch_stream(const DenseArgs& a, hipStream_t s) {
  const dim3 grid((a.N + 16 * CB - 1) / (16 * CB), (a.M + 16 * RB - 1) / (16 * RB));
  gemm_stream_kernel<WIDE, GRAN1, RB, CB, KS, S><<<grid, KS * 64, 0, s>>>(a);
  return hipGetLastError();
}

template <bool WIDE, bool GRAN1>
hipError_t launch_dense(DenseArgs a, hipStream_t s) {
  const Plan p = plan_dense(a.M, a.N, a.K, WIDE);
  a.splits = p.splits;
  // streaming workgroups: 16 columns and 8 waves while they fit the chip once, else 32 columns and 4 waves (7168 x 2048,
  // 16 rows: 8.0 and 5.9 us)
  const bool many = (a.N + 15) / 16 > kCus;
  switch (p.kind) {
    case kStream16:
      return many ? launch_stream<WIDE, GRAN1, 1, 2, 4, 4>(a, s) : launch_stream<WIDE, GRAN1, 1, 1, 8, 3>(a, s);
    case kStream32:
      return many ? launch_stream<WIDE, GRAN1, 2, 2, 4, 4>(a, s) : launch_stream<WIDE, GRAN1, 2, 1, 8, 3>(a, s);
    case kStream64:
      return many ? launch_stream<WIDE, GRAN1, 4, 2, 4, 2>(a, s) : launch_stream<WIDE, GRAN1, 4, 1, 4, 3>(a, s);
    case k64x64: return launch_small<WIDE, GRAN1, 2, 2, 2, 2>(a, s);
    case k64x128: return launch_small<WIDE, GRAN1, 2, 2, 2, 4>(a, s);
    case k128x128: return launch_small<WIDE, GRAN1, 4, 2, 2, 4>(a, s);
    default:  // the largest of either list
      if constexpr (WIDE) return launch_big<WIDE, GRAN1, 4, 4, 2, 2>(a, s);
      else return launch_big<WIDE, GRAN1, 8, 4, 2, 4>(a, s);
  }
}

}  // namespace

int64_t dense_workspace_bytes(int M, int N, int K) {
  // either output type may be asked for: the larger need
  const int a = plan_dense(M, N, K, false).splits, b = plan_dense(M, N, K, true).splits, s = a > b ? a : b;
  return s > 1 ? 4ll * s * M * ((N + 3) & ~3) : 0;
}

hipError_t launch_gemm_dense(const DenseArgs& a, hipStream_t s) {
  const bool g1 = a.gran_n == 1;
  if (a.f32) return g1 ? launch_dense<true, true>(a, s) : launch_dense<true, false>(a, s);
  return g1 ? launch_dense<false, true>(a, s) : launch_dense<false, false>(a, s);
}

}  // namespace moe
