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
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kXcd = 8;

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

// Four consecutive columns n .. n + 3 of row m (vec: they may be accessed as one vector where all four exist).
__device__ __forceinline__ void store4(const DenseArgs& a, int m, int n, v4f v, bool vec) {
  if (m >= a.M || n >= a.N) return;
  const int64_t at = (int64_t)m * a.ldd + n;
  if (vec && n + 4 <= a.N) {
    if (a.f32) {
      if (a.C) v += *(const v4f*)(a.C + (int64_t)m * a.ldc + n);
      *(v4f*)((float*)a.D + at) = v;
    } else {
      uint2 o;
      o.x = f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16);
      o.y = f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16);
      *(uint2*)((uint16_t*)a.D + at) = o;
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

template <int RB, int CB, int WM, int WN, int S>
struct TileCfg {
  static constexpr int NW = WM * WN;
  static constexpr int BM = 16 * RB * WM, BN = 16 * CB * WN;
  static constexpr int kPieces = (BM + BN) / 8;         // 1 KB copies (8 rows) per K block
  static constexpr int kPw = (kPieces + NW - 1) / NW;   // per wave
  static constexpr int kSlot = (BM + BN) * 128;
  static constexpr int kScale = (BM + BN) * 16;         // one group of 4 K blocks
  // Scale groups are copied kAhead groups early: their copies are older than the kPw * (S - 2) newest that the wait
  // before their first use leaves in flight (4 blocks' copies are issued per group).
  static constexpr int kAhead = S > 6 ? 2 : 1, kScBufs = 2 * kAhead;
  static constexpr int kLds = S * kSlot + kScBufs * kScale;
  static_assert(kPieces % NW == 0, "every wave copies the same number of pieces");
  static_assert(S >= 2 && S <= 4 * kAhead + 2 && kPw * (S - 2) < 64, "scales ahead of their use; vmcnt's range");
  static_assert((BM + BN) % 64 == 0 && BM % 64 == 0, "scale rows in whole waves");
  static_assert(kLds <= 160 * 1024, "LDS");
};

template <bool WIDE, bool GRAN1, int RB, int CB, int WM, int WN, int S>
__global__ __launch_bounds__(WM* WN * 64) void gemm_dense_kernel(const DenseArgs a) {
  using C = TileCfg<RB, CB, WM, WN, S>;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[C::kLds];
  const int lane = lane_id(), wv = uniform(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int KB = a.K / 128;
  // this workgroup's K blocks (split K: a multiple of 4 per split)
  const int per_split = ((KB + 3) / 4 + a.splits - 1) / a.splits * 4;
  const int kb0 = uniform(min((int)blockIdx.y * per_split, KB)), kb1 = uniform(min(kb0 + per_split, KB));

  // Workgroup b runs on XCD b % 8: consecutive tiles go to one XCD, and consecutive tiles are blocks of up to 8
  // column tiles by a few row tiles, so an XCD's workgroups share both operands in its L2.
  const int mt = (a.M + C::BM - 1) / C::BM, nt = (a.N + C::BN - 1) / C::BN;
  const int tiles = mt * nt;
  int t = blockIdx.x;
  {
    const int per = tiles / kXcd, rem = tiles % kXcd, x = t % kXcd, i = t / kXcd;
    t = x * per + min(x, rem) + i;
  }
  const int gn = 8, g = t / (mt * gn), gw = min(gn, nt - g * gn), r = t - g * mt * gn;
  const int m0 = uniform(r / gw * C::BM), n0 = uniform((g * gn + r % gw) * C::BN);

  const int wm = (wv / WN) * 16 * RB, wn = (wv % WN) * 16 * CB;
  const uint32_t lds0 = lds_offset(sm);

  // copies: this wave's pieces q = wv, wv + NW, ...; rows of the A tile, then of the W tile
  const uint8_t* abase = a.A + (int64_t)m0 * a.lda;
  const uint8_t* wbase = a.W + (int64_t)n0 * a.ldw;
  uint32_t voff[C::kPw];
#pragma unroll
  for (int i = 0; i < C::kPw; ++i) {
    const int q = wv + C::NW * i;
    int row = 8 * q + (lane >> 3);
    const int c = (lane & 7) ^ ((row >> 1) & 7);
    if (row < C::BM)
      voff[i] = (uint32_t)min(row, a.M - 1 - m0) * (uint32_t)a.lda + 16u * c;
    else
      voff[i] = (uint32_t)min(row - C::BM, a.N - 1 - n0) * (uint32_t)a.ldw + 16u * c;
  }
  auto copy_piece = [&](int kb, int i) {
    const int q = wv + C::NW * i;
    const uint8_t* base = (8 * q < C::BM ? abase : wbase) + (int64_t)kb * 128;
    copy16(voff[i], base, uniform(lds0 + (kb % S) * C::kSlot + 1024 * q));
  };

  // scales: group g4 (K blocks 4 g4 ..) of row r of the tiles at 16 r of buffer g4 & 1
  const bool sc_vec = KB % 4 == 0 && (((uintptr_t)a.SFA | (uintptr_t)a.SFW) & 15) == 0;
  auto scales = [&](int g4) {
#pragma unroll
    for (int q = 0; q < (C::BM + C::BN) / 64; q += C::NW) {
      const int p = q + wv;
      if (p * 64 >= C::BM + C::BN) break;
      const int row = 64 * p + lane;
      const bool is_a = 64 * p < C::BM;
      const float* base = is_a ? a.SFA : a.SFW;
      const int64_t sr = is_a ? min(m0 + row, a.M - 1) : (GRAN1 ? min(n0 + row - C::BM, a.N - 1)
                                                                 : min(n0 + row - C::BM, a.N - 1) / 128);
      const uint32_t dst = lds0 + S * C::kSlot + (g4 & (C::kScBufs - 1)) * C::kScale;
      if (sc_vec) {
        const int64_t sr0 = is_a ? m0 : (GRAN1 ? n0 : n0 / 128);
        copy16((uint32_t)(sr - sr0) * (uint32_t)KB * 4u, base + sr0 * KB + 4 * g4, uniform(dst + 1024 * p));
      } else {
        const float* s = base + sr * KB;
        v4f v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = s[min(4 * g4 + j, KB - 1)];
        *(v4f*)(sm + S * C::kSlot + (g4 & (C::kScBufs - 1)) * C::kScale + 16 * row) = v;
      }
    }
  };

  // fragment read offsets: row l16 of a 16-row block at 128 l16, its chunk c at position c ^ ((row >> 1) & 7)
  const int fsw = (l16 >> 1) & 7;
  const int off_lo = l16 * 128 + 16 * (lg ^ fsw), off_hi = l16 * 128 + 16 * ((4 + lg) ^ fsw);
  auto frag = [&](Frag<WIDE>& f, int kb, int row) {
    const uint8_t* p = sm + (kb % S) * C::kSlot + row * 128;
    f.load(*(const v4i*)(p + off_lo), *(const v4i*)(p + off_hi));
  };

  v4f acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  Frag<WIDE> wf[CB], xf[2];
  float sa[RB];
  v4f sw[GRAN1 ? CB : 1];

  // the first fragments and the scales of block kb
  auto first = [&](int kb) {
#pragma unroll
    for (int j = 0; j < CB; ++j) frag(wf[j], kb, C::BM + wn + 16 * j);
    frag(xf[0], kb, wm);
    const float* s = (const float*)(sm + S * C::kSlot + ((kb >> 2) & (C::kScBufs - 1)) * C::kScale) + (kb & 3);
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
  };

  if (kb0 < kb1) {
#pragma unroll
  for (int g4 = 0; g4 < C::kAhead; ++g4)
    if (kb0 + 4 * g4 < kb1) scales((kb0 >> 2) + g4);
#pragma unroll
  for (int b = 0; b < S - 1; ++b)
    if (kb0 + b < kb1) {
#pragma unroll
      for (int i = 0; i < C::kPw; ++i) copy_piece(kb0 + b, i);
    }
  if (kb0 + S - 1 <= kb1)
    wait_vmcnt<C::kPw * (S - 2)>();
  else
    wait_vmcnt<0>();
  barrier_lds();
  first(kb0);

  // One K block.  Row block i's matrix instructions alternate with the promotion of row block i - 1.
  // kind 2: block kb + S - 1 is copied meanwhile; 1: no more copies, but a next block; 0: the last block.
  auto step = [&](int kb, auto kind) {
    constexpr bool copies = decltype(kind)::value == 2, more = decltype(kind)::value > 0;
    v4f sum[2][CB];
    float sax[RB];
    v4f swx[GRAN1 ? CB : 1];
#pragma unroll
    for (int i = 0; i < RB; ++i) sax[i] = GRAN1 ? sa[i] : sa[i] * sw[0][0];
    if constexpr (GRAN1) {
#pragma unroll
      for (int j = 0; j < CB; ++j) swx[j] = sw[j];
    }
    auto promote = [&](int i, int j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float s = GRAN1 ? sax[i] * swx[j][e] : sax[i];
        acc[i][j][e] = __builtin_fmaf(sum[i & 1][j][e], s, acc[i][j][e]);
      }
    };
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      if (i + 1 < RB) frag(xf[(i + 1) & 1], kb, wm + 16 * (i + 1));
      if constexpr (copies) {  // spread over the first row blocks
        constexpr int kSpread = RB > 1 ? (RB + 1) / 2 : 1, kEach = (C::kPw + kSpread - 1) / kSpread;
#pragma unroll
        for (int c = i * kEach; c < (i + 1) * kEach && c < C::kPw; ++c) copy_piece(kb + S - 1, c);
      }
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        sum[i & 1][j] = block_sum(wf[j], xf[i & 1]);
        if (i > 0) promote(i - 1, j);
      }
      __builtin_amdgcn_sched_barrier(0);  // keep the row blocks' order (hoisted fragments would spill)
    }
    if constexpr (more) {
      wait_vmcnt<copies ? C::kPw*(S - 2) : 0>();
      barrier_lds();
      first(kb + 1);
    }
#pragma unroll
    for (int j = 0; j < CB; ++j) promote(RB - 1, j);
    __builtin_amdgcn_sched_barrier(0);
  };
  int kb = kb0;
  for (; kb + S - 1 < kb1; ++kb) {
    if ((kb & 3) == 0 && kb + 4 * C::kAhead < kb1) scales((kb >> 2) + C::kAhead);
    step(kb, IntC<2>{});
  }
  if constexpr (S > 2) {
    for (; kb + 1 < kb1; ++kb) {
      if ((kb & 3) == 0 && kb + 4 * C::kAhead < kb1) scales((kb >> 2) + C::kAhead);
      step(kb, IntC<1>{});
    }
  }
  step(kb1 - 1, IntC<0>{});
  }

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
  const bool vec = o.ldd % 4 == 0 && ((uintptr_t)o.D & (o.f32 ? 15 : 7)) == 0 &&
                   (!o.C || (o.ldc % 4 == 0 && ((uintptr_t)o.C & 15) == 0));
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) store4(o, m0 + wm + 16 * i + l16, n0 + wn + 16 * j + 4 * lg, acc[i][j], vec);
}

// Split K: the splits' partial sums, added in split order, and the addend.
__global__ __launch_bounds__(256) void gemm_dense_join_kernel(const DenseArgs a) {
  const int np = (a.N + 3) / 4;
  const int64_t total = (int64_t)a.M * np;
  const bool vec = a.ldd % 4 == 0 && ((uintptr_t)a.D & (a.f32 ? 15 : 7)) == 0 &&
                   (!a.C || (a.ldc % 4 == 0 && ((uintptr_t)a.C & 15) == 0));
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total; q += (int64_t)gridDim.x * 256) {
    v4f v = *(const v4f*)(a.ws + 4 * q);
    for (int k = 1; k < a.splits; ++k) v += *(const v4f*)(a.ws + 4 * (q + k * total));
    store4(a, (int)(q / np), 4 * (int)(q % np), v, vec);
  }
}

template <bool WIDE, bool GRAN1, int RB, int CB, int WM, int WN, int S>
hipError_t launch_tile(const DenseArgs& a, hipStream_t s) {
  using C = TileCfg<RB, CB, WM, WN, S>;
  const int tiles = ((a.M + C::BM - 1) / C::BM) * ((a.N + C::BN - 1) / C::BN);
  gemm_dense_kernel<WIDE, GRAN1, RB, CB, WM, WN, S><<<dim3(tiles, a.splits), WM * WN * 64, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t need = ((int64_t)a.M * ((a.N + 3) / 4) + 255) / 256, cap = (int64_t)device_info().cus * 16;
  gemm_dense_join_kernel<<<(unsigned)(need < cap ? need : cap), 256, 0, s>>>(a);
  return hipGetLastError();
}

// Few rows (a decode step): every weight byte is used by one wave, so waves need nothing from one another.  A
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
__global__ __launch_bounds__(KS * 64) void gemm_stream_kernel(const DenseArgs a) {
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
  const bool vec = a.ldd % 4 == 0 && ((uintptr_t)a.D & (a.f32 ? 15 : 7)) == 0 &&
                   (!a.C || (a.ldc % 4 == 0 && ((uintptr_t)a.C & 15) == 0));
  for (int q = threadIdx.x; q < kRows * kCols / 4; q += KS * 64) {
    const int m = q / (kCols / 4), n = 4 * (q % (kCols / 4));
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KS; ++k) v += *(const v4f*)((const float*)(sm + k * C::kWave) + m * (kCols + 4) + n);
    store4(a, m0 + m, n0 + n, v, vec);
  }
}

template <bool WIDE, bool GRAN1, int RB, int CB, int KS, int S>
hipError_t launch_stream(const DenseArgs& a, hipStream_t s) {
  const dim3 grid((a.N + 16 * CB - 1) / (16 * CB), (a.M + 16 * RB - 1) / (16 * RB));
  gemm_stream_kernel<WIDE, GRAN1, RB, CB, KS, S><<<grid, KS * 64, 0, s>>>(a);
  return hipGetLastError();
}

#ifndef V1
#define V1 1, 1, 8, 4
#define V2 2, 1, 8, 3
#define V4 4, 1, 4, 3
#define TW 4, 4, 2, 2, 2
#define TN 8, 4, 2, 4, 2
#define SP 1
#define MS 64
#endif
template <bool WIDE, bool GRAN1>
hipError_t launch_dense(DenseArgs a, hipStream_t s) {
  a.splits = 1;
  if (a.M <= 16) return launch_stream<WIDE, GRAN1, V1>(a, s);
  if (a.M <= 32 && MS >= 32) return launch_stream<WIDE, GRAN1, V2>(a, s);
  if (a.M <= 64 && MS >= 64) return launch_stream<WIDE, GRAN1, V4>(a, s);
  a.splits = SP;
  if constexpr (WIDE) return launch_tile<WIDE, GRAN1, TW>(a, s);
  else return launch_tile<WIDE, GRAN1, TN>(a, s);
}

}  // namespace

int64_t dense_workspace_bytes(int M, int N, int K) { return SP > 1 ? 4ll * SP * M * ((N + 3) & ~3) : 0; }

hipError_t launch_gemm_dense(const DenseArgs& a, hipStream_t s) {
  const bool g1 = a.gran_n == 1;
  if (a.f32) return g1 ? launch_dense<true, true>(a, s) : launch_dense<true, false>(a, s);
  return g1 ? launch_dense<false, true>(a, s) : launch_dense<false, false>(a, s);
}

}  // namespace moe
