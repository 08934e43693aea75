// gemm_linear.hip -- moe_gemm_bf16: a dense bf16 product with bias, activation and residual in its epilogue, and the
// products of its gradient.
//
//   D[m, n] = C[m, n] + act( sum_k a[m, k] w[n, k] + bias[n] )
//   gated:    D[m, j] = C[m, j] + act(v[m, j]) * v[m, N/2 + j],   v = the product plus bias, w's rows gate then up
//
// Operands come in the order they are stored in: rows with K contiguous, or (ta, tw) rows of one k with m (n) contiguous, as
// the gradients' products need them: dX = dP W has W's n as its k, dW = dP^T X contracts over the tokens.  No transpose goes
// through memory: both orders are copied global -> LDS as they lie, and a fragment of the second order is read with
// ds_read_b64_tr_b16, which hands 16 lanes the columns of 4 rows.
//
// Tile.  A workgroup of WM x WN waves computes 16 RB WM rows x 16 CB WN columns, 64 K values a step.  w is the matrix
// instruction's A operand (output columns), a its B operand (rows), so a lane holds 4 consecutive columns of one row, and the
// epilogue sees each value in fp32 once.  Copies are buffer loads into the LDS, whose range check turns what lies outside the
// matrices (rows, columns, the last K block's rest) into zeros.
//
// Measured (us): 4096 x 4096 x 7168 176 (1.36 PFLOP/s; the library's plain product 155 to 160), with GELU, bias and pre 189 to
// 202; 8192^3 764 (1.44); 4096 x 7168 x 4096 in the gradients' orders 198 (library 200, 221); 1024 x 4096 x 7168 55 (60); 131 x
// 7168 x 2048 13.4 (19); 1 x 4096 x 7168 12.1 from HBM (4.9 TB/s).
#include "linear_act.h"
#include "linear_plan.h"
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr uint32_t kOut = 0x80000000u;  // an offset past every buffer: its copy writes zeros
constexpr int kXcds8 = 8;

__device__ __forceinline__ void barrier_reads() {
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), which the compiler sees
  asm volatile("s_barrier" ::: "memory");
}

// 64 lanes x 16 bytes global -> LDS, lane i's from base + voff to lds + 16 i; offsets from 2^31 on write zeros.
__device__ __forceinline__ void copy16(uint32_t voff, const void* base, uint32_t lds) {
  const uint64_t b = (uint64_t)base;
  const v4i r = {(int)(uint32_t)b, (int)(uint32_t)(b >> 32) & 0xffff, 0x7fffffff, 0x00020000};
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(voff), "s"(r), "{m0}"(lds) : "memory");
}

// The same for what one workgroup alone reads.
__device__ __forceinline__ void copy16_once(uint32_t voff, const void* base, uint32_t lds) {
  const uint64_t b = (uint64_t)base;
  const v4i r = {(int)(uint32_t)b, (int)(uint32_t)(b >> 32) & 0xffff, 0x7fffffff, 0x00020000};
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds" : : "v"(voff), "s"(r), "{m0}"(lds) : "memory");
}

__device__ __forceinline__ v4f mma(const v8bf w, const v8bf x, const v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
}

// -------------------------------------------------------------- epilogue --
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t v2u_any __attribute__((ext_vector_type(2), aligned(2)));

__device__ __forceinline__ v2u_any bf16x4(const v4f v) {
  return v2u_any{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
}
// Elements at .. at + 3 (cnt of them are there) of an fp32 or bf16 row.
__device__ __forceinline__ v4f load4(const void* p, bool f32, int64_t at, int cnt) {
  v4f v = {0.f, 0.f, 0.f, 0.f};
  if (f32) {
    const float* q = (const float*)p + at;
    if (cnt == 4) return *(const v4f_any*)q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cnt) v[i] = q[i];
  } else {
    const uint16_t* q = (const uint16_t*)p + at;
    if (cnt == 4) {
      const v2u_any u = *(const v2u_any*)q;
      return v4f{bf16_to_f32(u[0] & 0xffffu), bf16_to_f32(u[0] >> 16), bf16_to_f32(u[1] & 0xffffu), bf16_to_f32(u[1] >> 16)};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cnt) v[i] = bf16_to_f32(q[i]);
  }
  return v;
}
__device__ __forceinline__ void store4(void* p, bool f32, int64_t at, int cnt, const v4f v) {
  if (f32) {
    float* q = (float*)p + at;
    if (cnt == 4) {
      *(v4f_any*)q = v;
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cnt) q[i] = v[i];
  } else {
    uint16_t* q = (uint16_t*)p + at;
    if (cnt == 4) {
      *(v2u_any*)q = bf16x4(v);
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cnt) q[i] = (uint16_t)bf16_pair(v[i], 0.f);
  }
}

// Eight bf16 columns.
__device__ __forceinline__ void store8(uint16_t* p, const v4f v) {
  typedef float v4b_any __attribute__((ext_vector_type(4), aligned(2)));
  *(v4b_any*)p = v;
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
    const auto r = __builtin_amdgcn_permlane16_swap(bf16_pair(a[2 * h], a[2 * h + 1]), bf16_pair(b[2 * h], b[2 * h + 1]),
                                                    false, false);  // the first of groups 1, 3 for the second of groups 0, 2
    o[h] = __uint_as_float(r[0]);
    o[2 + h] = __uint_as_float(r[1]);
  }
  return o;
}

// Columns n .. n + 3 of row m; NO: how many columns D has.  v: the product (gated: gate and up).
template <bool GATED>
__device__ __forceinline__ void epilogue4(const LinearArgs& a, int m, int n, v4f v, v4f up) {
  const int NO = GATED ? a.N / 2 : a.N;
  if (m >= a.M || n >= NO) return;
  const int cnt = min(4, NO - n);
  if (a.bias) {
    v += load4(a.bias, a.bias_f32, n, cnt);
    if (GATED) up += load4(a.bias, a.bias_f32, NO + n, cnt);
  }
  if (a.pre) {
    store4(a.pre, false, (int64_t)m * a.ldp + n, cnt, v);
    if (GATED) store4(a.pre, false, (int64_t)m * a.ldp + NO + n, cnt, up);
  }
  v = act4(a.act, v);
  if (GATED) v *= up;
  if (a.C) v += load4(a.C, a.c_f32, (int64_t)m * a.ldc + n, cnt);
  store4(a.D, a.d_f32, (int64_t)m * a.ldd + n, cnt, v);
}

// Split K: this share's sums, in rows of ws_cols() floats (gated: the up columns begin at half of them).
__host__ __device__ inline int ws_half(const LinearArgs& a) { return ((a.gated ? a.N / 2 : a.N) + 3) & ~3; }
__host__ __device__ inline int ws_cols(const LinearArgs& a) { return a.gated ? 2 * ws_half(a) : ws_half(a); }

template <bool GATED>
__device__ __forceinline__ void finish4(const LinearArgs& a, int m, int n, const v4f v, const v4f up) {
  if (a.splits == 1) return epilogue4<GATED>(a, m, n, v, up);
  const int half = ws_half(a);
  if (m >= a.M || n >= half) return;
  float* w = a.ws + ((int64_t)blockIdx.y * a.M + m) * ws_cols(a) + n;
  *(v4f*)w = v;
  if (GATED) *(v4f*)(w + half) = up;
}

// ---------------------------------------------------------------- operand --
// One operand's B rows (m or n) x 64 K values in LDS, B * 128 bytes, and its copies.
// K contiguous: row r at 128 r, its 16-byte chunk c at position c ^ ((r >> 1) & 7).
// TR: row k at 2 B k, its 32-byte segment s at position s ^ f(k); f takes the 8 rows that 32 lanes read at once to 8 places.
template <bool TR, int B>
struct Operand {
  static constexpr int kRowsPerCopy = TR ? 512 / B : 8;
  __device__ static __forceinline__ int f(int k) {
    return B == 64 ? ((k >> 1) & 1) | ((k >> 3) & 1) << 1 : (k & 3) | ((k >> 3) & 1) << 2;
  }
  // this lane's place in copy q: k offset within the step, and the row (m or n) in the tile
  __device__ static __forceinline__ void place(int q, int lane, int& k, int& row) {
    if (TR) {
      k = kRowsPerCopy * q + lane / (B / 8);
      const int pos = lane % (B / 8);
      row = ((pos >> 1) ^ f(k)) * 16 + (pos & 1) * 8;
    } else {
      row = 8 * q + (lane >> 3);
      k = 8 * ((lane & 7) ^ ((row >> 1) & 7));
    }
  }
  // byte offset of that place from the tile's first element
  __device__ static __forceinline__ uint32_t offset(int k, int row, int64_t ld) {
    return 2u * (TR ? (uint32_t)k * (uint32_t)ld + (uint32_t)row : (uint32_t)row * (uint32_t)ld + (uint32_t)k);
  }
  // fragment reads: block blk of 16 rows, half h of the step
  int o0, o1;
  __device__ __forceinline__ void init(int lane, int first_blk) {
    const int i = lane & 15, g = lane >> 4;
    if (TR) {
      const int k = 8 * g + (i >> 2);
      o0 = k * 2 * B + 8 * (i & 3);
      o1 = (first_blk ^ f(k)) * 32;
    } else {
      const int sw = (i >> 1) & 7;
      o0 = first_blk * 2048 + i * 128 + 16 * (g ^ sw);
      o1 = first_blk * 2048 + i * 128 + 16 * ((4 + g) ^ sw);
    }
  }
  // blk counts from first_blk, which is a multiple of the wave's blocks (a power of two), so that it can be xor-ed
  __device__ __forceinline__ v8bf frag(const uint8_t* s, int blk, int h) const {
    if constexpr (TR) {
      typedef short v4s __attribute__((ext_vector_type(4)));
      typedef short v8s __attribute__((ext_vector_type(8)));
      const uint8_t* p = s + o0 + (o1 ^ (blk * 32)) + h * 64 * B;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p + 8 * B));
      return __builtin_bit_cast(v8bf, v8s{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    } else {
      return __builtin_bit_cast(v8bf, *(const v4i*)(s + (h ? o1 : o0) + blk * 2048));
    }
  }
};

// ------------------------------------------------------------------- tile --
template <int RB, int CB, int WM, int WN, int S>
struct LinCfg {
  static constexpr int NW = WM * WN, BM = 16 * RB * WM, BN = 16 * CB * WN;
  static constexpr int kCopies = (BM + BN) / 8, kPw = kCopies / NW;
  static constexpr int kSlot = (BM + BN) * 128, kLds = S * kSlot;
  static_assert(kCopies % NW == 0 && kLds <= 160 * 1024 && (S - 1) * kPw < 64, "copies in equal shares; LDS; vmcnt");
};

template <bool TA, bool TW, bool GATED, int RB, int CB, int WM, int WN, int S>
struct LinTileT {
  using C = LinCfg<RB, CB, WM, WN, S>;
  static_assert(!GATED || (!TW && CB % 2 == 0), "gate and up blocks in turn");
  const LinearArgs& a;
  uint8_t* sm;
  uint32_t lds0;
  int lane, wv, l16, lg, KB, kb0, kb1, m0, n0, wm, wn;  // n0: first column of D
  const uint8_t *abase, *wbase;
  uint32_t voff[C::kPw];
  Operand<TA, C::BM> xa;
  Operand<TW, C::BN> xw;

  __device__ __forceinline__ LinTileT(const LinearArgs& args, uint8_t* smem) : a(args), sm(smem) {
    lane = lane_id();
    wv = uniform(threadIdx.x >> 6);
    l16 = lane & 15;
    lg = lane >> 4;
    lds0 = lds_offset(sm);
    KB = (a.K + 63) / 64;
    const int per = lin_split_blocks(KB, a.splits);
    kb0 = uniform(min((int)blockIdx.y * per, KB));
    kb1 = uniform(min(kb0 + per, KB));
    // Workgroup b runs on XCD b % 8: consecutive tiles go to one XCD, and consecutive tiles are blocks of up to 8 column
    // tiles by a few row tiles, so an XCD's workgroups share both operands in its L2.
    const int NO = GATED ? a.N / 2 : a.N, BNO = GATED ? C::BN / 2 : C::BN;
    const int mt = (a.M + C::BM - 1) / C::BM, nt = (NO + BNO - 1) / BNO, tiles = mt * nt;
    const int share = tiles / kXcds8, rem = tiles % kXcds8, x = blockIdx.x % kXcds8;
    const int t = x * share + min(x, rem) + blockIdx.x / kXcds8;
    const int gn = 8, g = t / (mt * gn), gw = min(gn, nt - g * gn), r = t - g * mt * gn;
    m0 = uniform(r / gw * C::BM);
    n0 = uniform((g * gn + r % gw) * BNO);
    wm = (wv / WN) * 16 * RB;
    wn = (wv % WN) * 16 * CB;
    abase = (const uint8_t*)(a.A + (TA ? (int64_t)m0 : m0 * a.lda)) + (int64_t)kb0 * astep();
    wbase = (const uint8_t*)(a.W + (TW ? (int64_t)n0 : n0 * a.ldw)) + (int64_t)kb0 * wstep();
#pragma unroll
    for (int i = 0; i < C::kPw; ++i) {
      int k, row;
      voff[i] = where(i, k, row);
    }
    xa.init(lane, wm / 16);
    xw.init(lane, wn / 16);
  }
  __device__ __forceinline__ int64_t astep() const { return TA ? 128 * a.lda : 128; }
  __device__ __forceinline__ int64_t wstep() const { return TW ? 128 * a.ldw : 128; }
  // copy i of this wave: this lane's k and row, and its offset (kOut where the matrix has no such row)
  __device__ __forceinline__ uint32_t where(int i, int& k, int& row) const {
    const int q = wv + C::NW * i;
    if (8 * q < C::BM) {
      Operand<TA, C::BM>::place(q, lane, k, row);
      return m0 + row < a.M ? Operand<TA, C::BM>::offset(k, row, a.lda) : kOut;
    }
    Operand<TW, C::BN>::place(q - C::BM / 8, lane, k, row);
    if (GATED) {  // 16 gate rows, then the 16 up rows of the same outputs
      const int j = (row >> 5) * 16 + (row & 15);
      row = j + (row & 16 ? a.N / 2 : 0);
      return n0 + j < a.N / 2 ? Operand<TW, C::BN>::offset(k, row, a.ldw) : kOut;
    }
    return n0 + row < a.N ? Operand<TW, C::BN>::offset(k, row, a.ldw) : kOut;
  }
  // before the copies of block kb: if K ends inside it, what lies behind becomes zeros (it is the last block that is copied)
  // (of one operand: of_a, else of w)
  template <bool of_a>
  __device__ __forceinline__ void end_of_k(int kb) {
    if (64 * kb + 64 <= a.K) return;
#pragma unroll
    for (int i = 0; i < C::kPw; ++i) {
      if ((8 * (wv + C::NW * i) < C::BM) != of_a) continue;
      int k, row;
      where(i, k, row);
      if (64 * kb + k >= a.K) voff[i] = kOut;
    }
  }
  // copy i of a block to `at` in the LDS; base: abase or wbase of the block
  __device__ __forceinline__ void copy_to(int i, const uint8_t* base, int at) const {
    copy16(voff[i], base, (uint32_t)uniform((int)lds0 + at));
  }
  __device__ __forceinline__ void store(v4f (&acc)[RB][CB]) const {
    // The sums are whole before any lane's store is masked off.
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < CB; ++j) asm volatile("" : "+v"(acc[i][j]));
    const int NO = GATED ? a.N / 2 : a.N;
    if (a.splits == 1 && m0 + C::BM <= a.M && n0 + (GATED ? C::BN / 2 : C::BN) <= NO) return store_whole(acc);
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int m = m0 + wm + 16 * i + l16;
      if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < CB; j += 2) finish4<true>(a, m, n0 + wn / 2 + 8 * j + 4 * lg, acc[i][j], acc[i][j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < CB; ++j) finish4<false>(a, m, n0 + wn + 16 * j + 4 * lg, acc[i][j], v4f{0.f, 0.f, 0.f, 0.f});
      }
    }
  }
  // A tile inside the matrix: no lane is masked; the bias is read once per column block, a row block's addends before they are
  // needed, and lanes exchange columns so that stores write whole lines.
  __device__ __forceinline__ void store_whole(v4f (&acc)[RB][CB]) const {
    constexpr int OB = GATED ? CB / 2 : CB;  // column blocks of D
    const int NO = GATED ? a.N / 2 : a.N, n = n0 + (GATED ? wn / 2 : wn);
    v4f bias[CB];
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < CB; ++j)
        bias[j] = load4(a.bias, a.bias_f32, GATED ? n + 8 * (j & ~1) + 4 * lg + (j & 1 ? NO : 0) : n + 16 * j + 4 * lg, 4);
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int m = m0 + wm + 16 * i;
      v4f c[OB], o[OB];
      if (a.C) {
#pragma unroll
        for (int j = 0; j < OB; ++j) c[j] = load4(a.C, a.c_f32, (int64_t)(m + l16) * a.ldc + n + 16 * j + 4 * lg, 4);
      }
      if (a.bias) {
#pragma unroll
        for (int j = 0; j < CB; ++j) acc[i][j] += bias[j];
      }
#pragma unroll
      for (int j = 0; j < OB; ++j) o[j] = acc[i][GATED ? 2 * j : j];
      if (a.pre) {
        put<OB>(a.pre, false, a.ldp, m, n, o);
        if constexpr (GATED) {
          v4f up[OB];
#pragma unroll
          for (int j = 0; j < OB; ++j) up[j] = acc[i][2 * j + 1];
          put<OB>(a.pre, false, a.ldp, m, NO + n, up);
        }
      }
#pragma unroll
      for (int j = 0; j < OB; ++j) {
        o[j] = act4(a.act, o[j]);
        if (GATED) o[j] *= acc[i][GATED ? 2 * j + 1 : 0];
        if (a.C) o[j] += c[j];
      }
      put<OB>(a.D, a.d_f32, a.ldd, m, n, o);
    }
  }
  // 16 rows from m on of B 16-column blocks from n on; v[j]: columns 4 lg .. + 3 of block j of row l16.  As they are, an
  // instruction would write 16 rows in pieces of 32 bytes (bf16) or 64.
  template <int B>
  __device__ __forceinline__ void put(void* p, bool f32, int64_t ld, int m, int n, const v4f (&v)[B]) const {
    const int hi = l16 >> 3, l8 = l16 & 7;
    if constexpr (B == 1) {
      store4(p, f32, (int64_t)(m + l16) * ld + n + 4 * lg, 4, v[0]);
    } else if (f32) {
#pragma unroll
      for (int j = 0; j < B; j += 2) {
        v4f x[2] = {v[j], v[j + 1]};
        swap8(x[0], x[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v4f_any* q = (v4f_any*)((float*)p + (int64_t)(m + 8 * h + l8) * ld + n + 16 * (j + hi) + 4 * lg);
          // past the caches where whole lines are written; rows that share lines with their neighbours meet them in the L2
          if (ld % 4 == 0) __builtin_nontemporal_store(x[h], q);
          else *q = x[h];
        }
      }
    } else {
      v4f x[B / 2];  // 8 columns of bf16 each
#pragma unroll
      for (int j = 0; j < B; j += 2) x[j / 2] = join_columns(v[j], v[j + 1]);
      const int n8 = n + 16 * (lg & 1) + 8 * (lg >> 1);
      if constexpr (B == 4) {
        swap8(x[0], x[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) store8((uint16_t*)p + (int64_t)(m + 8 * h + l8) * ld + n8 + 32 * hi, x[h]);
      } else {
        store8((uint16_t*)p + (int64_t)(m + l16) * ld + n8, x[0]);
      }
    }
  }
};

// Smaller tiles: fragments fit the registers twice, so block kb + 1's are read while block kb is multiplied, and block kb + 4 is copied
// meanwhile into the slot that block kb left when it was read.  The loop is unrolled over the 4 slots, so that slots and offsets are
// constants; reads and copies are laid out between the matrix instructions (in one go each, they take turns instead of
// overlapping: 64x64 0.34 us a step).
template <bool TA, bool TW, bool GATED, int RB, int CB, int WM, int WN>
__global__ __launch_bounds__(512) void gemm_linear_small_kernel(const LinearArgs a) {
  constexpr int S = 4;
  using C = LinCfg<RB, CB, WM, WN, S>;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[C::kLds];
  LinTileT<TA, TW, GATED, RB, CB, WM, WN, S> T(a, sm);
  const int kb0 = T.kb0, kb1 = T.kb1;
  v4f acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  struct Regs {
    v8bf w[CB][2], x[RB][2];
  } reg[2];
  // read r of a block in slot `slot`: halves of the weights' fragments, then of the rows'
  auto read = [&](Regs& to, int slot, int r) {
    const uint8_t* p = sm + slot * C::kSlot;
    if (r < 2 * CB) to.w[r < 2 * CB ? r / 2 : 0][r & 1] = T.xw.frag(p + C::BM * 128, r / 2, r & 1);
    else to.x[r < 2 * CB ? 0 : r / 2 - CB][r & 1] = T.xa.frag(p, r / 2 - CB, r & 1);
  };
  auto copy = [&](int slot, int i) {
    const int q = T.wv + C::NW * i;
    T.copy_to(i, 8 * q < C::BM ? T.abase : T.wbase, slot * C::kSlot + 1024 * q);
  };
  auto next_block = [&]() {
    T.abase += T.astep();
    T.wbase += T.wstep();
  };
  // block k in slot u (k - kb0 = u mod 4).  kind 2: block k + 4 is copied; 1: no more copies, but a next block; 0: the last block
  auto step = [&](int k, auto uc, auto kind) {
    constexpr int u = decltype(uc)::value, kd = decltype(kind)::value;
    constexpr int NM = 2 * RB * CB, NF = 2 * (RB + CB);
    const Regs& r = reg[u & 1];
    Regs& next = reg[(u + 1) & 1];
    if constexpr (kd == 2) {
      T.template end_of_k<true>(k + S);
      T.template end_of_k<false>(k + S);
    }
    static_for<0, NM>([&](auto mc) {
      constexpr int m = decltype(mc)::value, h = m / (RB * CB), i = m / CB % RB, j = m % CB;
      acc[i][j] = mma(r.w[j][h], r.x[i][h], acc[i][j]);
      if constexpr (kd > 0) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
          if (f * NM / NF == m) read(next, (u + 1) & 3, f);
      }
      if constexpr (kd == 2) {
#pragma unroll
        for (int c = 0; c < C::kPw; ++c)
          if (c * NM / C::kPw == m) copy(u, c);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (kd == 2) next_block();
    if constexpr (kd > 0) {
      wait_vmcnt<kd == 2 ? C::kPw*(S - 2) : 0>();  // block k + 2 is in the LDS
      barrier_reads();                              // and block k + 1 in registers
    }
  };
  if (kb0 < kb1) {
    static_for<0, S>([&](auto u) {
      const int k = kb0 + decltype(u)::value;
      if (k < kb1) {
        T.template end_of_k<true>(k);
        T.template end_of_k<false>(k);
#pragma unroll
        for (int c = 0; c < C::kPw; ++c) copy(decltype(u)::value, c);
        next_block();
      }
    });
    const bool full = kb0 + S <= kb1;
    if (full) wait_vmcnt<C::kPw*(S - 1)>();
    else wait_vmcnt<0>();
    barrier_reads();
#pragma unroll
    for (int f = 0; f < 2 * (RB + CB); ++f) read(reg[0], 0, f);
    if (full) wait_vmcnt<C::kPw*(S - 2)>();
    barrier_reads();  // block kb0 is in registers, block kb0 + 1 in the LDS
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

// The large tiles (256x256: 8 waves of 128x64, two per SIMD; 128x128: 4 waves of 64x64, two workgroups per compute unit), with the
// other work of a step laid out between the matrix instructions of its own wave:
//  * row blocks 0 .. RB-3 in turn, their fragments read two ahead;
//  * then the barrier that publishes block kb + 1, every fragment of block kb being in registers, and the last two row blocks
//    column by column: after column j's matrix instructions its weight fragment is read anew for block kb + 1;
//  * three slots for rows, two for weights (all of the LDS): a slot of rows is free from that barrier on, so block kb + 3's rows
//    are copied behind it and have two steps to arrive; weights stay in registers from there on, so block kb + 2's are copied from the
//    second row block of step kb on (a barrier says that every wave has read block kb's) and have one and a half.
// 4096 x 4096 x 7168, all tiles at once: 1.48 us a step, of which its matrix instructions are 1.0 at the 2.0 GHz under load; with two
// slots each and copies one step ahead 2.3 us.  Not the memory: with every tile reading the same operands it takes as long.
template <bool TA, bool TW, bool GATED, int RB, int CB, int WM, int WN>
__global__ __launch_bounds__(512) void gemm_linear_big_kernel(const LinearArgs a) {
  using C = LinCfg<RB, CB, WM, WN, 2>;
  constexpr int kA = C::BM * 128, kW = C::BN * 128;
  static_assert(RB >= 4 && RB % 4 == 0 && C::kPw == 2 * CB && C::BM == 8 * C::NW * CB,
                "fragment ring; a wave's first CB copies are of A, its last CB of W");
  __shared__ __attribute__((aligned(1024))) uint8_t sm[3 * kA + 2 * kW];
  LinTileT<TA, TW, GATED, RB, CB, WM, WN, 2> T(a, sm);
  const int kb0 = T.kb0, kb1 = T.kb1;
  v4f acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  v8bf w[CB][2], x[4][2];
  auto read_x = [&](int slot, int i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) x[i & 3][h] = T.xa.frag(sm + slot * kA, i, h);
  };
  auto read_w = [&](int kb, int j) {
#pragma unroll
    for (int h = 0; h < 2; ++h) w[j][h] = T.xw.frag(sm + 3 * kA + (kb & 1) * kW, j, h);
  };
  auto copy_x = [&](int slot, int i) { T.copy_to(i, T.abase, slot * kA + 1024 * (T.wv + C::NW * i)); };
  auto copy_w = [&](int kb, int i) {
    T.copy_to(CB + i, T.wbase, 3 * kA + (kb & 1) * kW + 1024 * (T.wv + C::NW * (CB + i)) - kA);
  };
  int s0 = 0, s1 = 1, s2 = 2;  // the slots of the rows of blocks kb, kb + 1, kb + 2
  // ahead: how many blocks follow block kb, at most 3
  auto step = [&](int kb, auto ahead_c) {
    constexpr int ahead = decltype(ahead_c)::value;
    if constexpr (ahead >= 2) T.template end_of_k<false>(kb + 2);
#pragma unroll
    for (int i = 0; i < RB - 2; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < CB; ++j) {
          acc[i][j] = mma(w[j][h], x[i & 3][h], acc[i][j]);
          if (h == 0 && j == 0) read_x(s0, i + 2);
          if constexpr (ahead >= 2) {  // the weights of block kb + 2
            const int c = RB >= 8 ? (h == 1 && j == 1 ? i - 1 : -1) : (i == 1 && h == 1 ? j : -1);
            if (c >= 0 && c < CB) copy_w(kb, c);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      if constexpr (ahead >= 2)
        if (i == 0) asm volatile("s_barrier" ::: "memory");
    }
    if constexpr (ahead > 0) {
      wait_vmcnt<ahead >= 2 ? 2 * CB : 0>();  // all but block kb + 2
      barrier_reads();
    }
    if constexpr (ahead >= 2) T.wbase += T.wstep();
    if constexpr (ahead == 3) T.template end_of_k<true>(kb + 3);
    v8bf xl[2] = {x[(RB - 2) & 3][0], x[(RB - 2) & 3][1]}, xm[2] = {x[(RB - 1) & 3][0], x[(RB - 1) & 3][1]};
    if constexpr (ahead > 0) {
      read_x(s1, 0);
      read_x(s1, 1);
    }
#pragma unroll
    for (int j = 0; j < CB; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        acc[RB - 2][j] = mma(w[j][h], xl[h], acc[RB - 2][j]);
        acc[RB - 1][j] = mma(w[j][h], xm[h], acc[RB - 1][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (ahead > 0) read_w(kb + 1, j);
      if constexpr (ahead == 3) copy_x(s0, j);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (ahead == 3) T.abase += T.astep();
    const int s = s0;
    s0 = s1;
    s1 = s2;
    s2 = s;
  };
  if (kb0 < kb1) {
    const int n = kb1 - kb0;
    auto issue_x = [&](int kb, int slot) {
      T.template end_of_k<true>(kb);
#pragma unroll
      for (int i = 0; i < CB; ++i) copy_x(slot, i);
      T.abase += T.astep();
    };
    auto issue_w = [&](int kb) {
      T.template end_of_k<false>(kb);
#pragma unroll
      for (int i = 0; i < CB; ++i) copy_w(kb, i);
      T.wbase += T.wstep();
    };
    // in the loop's order: rows are copied before the weights of the block before
    issue_x(kb0, 0);
    issue_w(kb0);
    if (n > 1) issue_x(kb0 + 1, 1);
    if (n > 1) issue_w(kb0 + 1);
    if (n > 2) issue_x(kb0 + 2, 2);
    if (n > 2) wait_vmcnt<3 * CB>();
    else if (n > 1) wait_vmcnt<2 * CB>();
    else wait_vmcnt<0>();
    barrier_reads();
    read_x(0, 0);
    read_x(0, 1);
#pragma unroll
    for (int j = 0; j < CB; ++j) read_w(kb0, j);
    int kb = kb0;
    for (; kb + 3 < kb1; ++kb) step(kb, IntC<3>{});
    if (kb + 2 < kb1) step(kb++, IntC<2>{});
    if (kb + 1 < kb1) step(kb++, IntC<1>{});
    step(kb, IntC<0>{});
  }
  T.store(acc);
}

// Split K: the shares' sums, added in order, then the epilogue.
template <bool GATED>
__global__ __launch_bounds__(256) void gemm_linear_join_kernel(const LinearArgs a) {
  const int half = ws_half(a), cols = ws_cols(a), np = half / 4;
  const int64_t total = (int64_t)a.M * np, plane = (int64_t)a.M * cols;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total; q += (int64_t)gridDim.x * 256) {
    const int m = (int)(q / np), n = 4 * (int)(q % np);
    const float* w = a.ws + (int64_t)m * cols + n;
    v4f v = *(const v4f*)w, up = {0.f, 0.f, 0.f, 0.f};
    if (GATED) up = *(const v4f*)(w + half);
    for (int k = 1; k < a.splits; ++k) {
      v += *(const v4f*)(w + k * plane);
      if (GATED) up += *(const v4f*)(w + k * plane + half);
    }
    epilogue4<GATED>(a, m, n, v, up);
  }
}

template <bool TA, bool TW, bool GATED, int RB, int CB, int WM, int WN, bool BIG = false>
hipError_t launch_tile(const LinearArgs& a, hipStream_t s) {
  using C = LinCfg<RB, CB, WM, WN, 2>;
  const int NO = GATED ? a.N / 2 : a.N, BNO = GATED ? C::BN / 2 : C::BN;
  const dim3 grid(((a.M + C::BM - 1) / C::BM) * ((NO + BNO - 1) / BNO), a.splits);
  if constexpr (BIG) gemm_linear_big_kernel<TA, TW, GATED, RB, CB, WM, WN><<<grid, WM * WN * 64, 0, s>>>(a);
  else gemm_linear_small_kernel<TA, TW, GATED, RB, CB, WM, WN><<<grid, WM * WN * 64, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t need = ((int64_t)a.M * (ws_half(a) / 4) + 255) / 256, cap = (int64_t)device_info().cus * 16;
  gemm_linear_join_kernel<GATED><<<(unsigned)(need < cap ? need : cap), 256, 0, s>>>(a);
  return hipGetLastError();
}

// ----------------------------------------------------------------- stream --
// Few rows (a decode step): every weight byte is used by one wave, so waves need nothing from one another.  A workgroup takes
// 16 CB columns (gated: blocks of 8 gates and their 8 ups) and all 16 RB rows; its KS waves split K, each with a ring of S blocks
// of its own in LDS (no barrier in the loop; all S in flight while a block is multiplied), and meet once at the end, where the partial sums are added in wave order.
template <int RB, int CB, int KS, int S>
struct LinStreamCfg {
  static constexpr int kBlock = (RB + CB) * 2048, kCopies = 2 * (RB + CB), kWave = S * kBlock;
  static constexpr int kPart = 16 * RB * (16 * CB + 4) * 4;  // a wave's partial sums, over its ring
  static constexpr int kLds = KS * kWave;
  static_assert(kPart <= kWave && kLds <= 160 * 1024 && (S - 1) * kCopies < 64, "LDS; vmcnt");
};

template <bool GATED, int RB, int CB, int KS, int S>
__global__ __launch_bounds__(512) void gemm_linear_stream_kernel(const LinearArgs a) {
  using C = LinStreamCfg<RB, CB, KS, S>;
  constexpr int kRows = 16 * RB, kCols = 16 * CB, kOuts = GATED ? kCols / 2 : kCols;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[C::kLds];
  const int lane = lane_id(), wv = uniform(threadIdx.x >> 6), l16 = lane & 15, lg = lane >> 4;
  const int KB = (a.K + 63) / 64, NO = GATED ? a.N / 2 : a.N;
  const int n0 = blockIdx.x * kOuts;
  const int kb0 = wv * KB / KS, nb = (wv + 1) * KB / KS - kb0;
  uint8_t* ring = sm + wv * C::kWave;
  const uint32_t lds0 = (uint32_t)uniform((int)lds_offset(ring));
  const uint8_t* abase = (const uint8_t*)a.A + (int64_t)kb0 * 128;
  const uint8_t* wbase = (const uint8_t*)(a.W + (int64_t)n0 * a.ldw) + (int64_t)kb0 * 128;
  uint32_t voff[C::kCopies];
  const int ck = 8 * ((lane & 7) ^ (lane >> 4));  // this lane's k in even copies; odd ones: ^ 32
#pragma unroll
  for (int q = 0; q < C::kCopies; ++q) {
    const int row = 8 * q + (lane >> 3), k = q & 1 ? ck ^ 32 : ck;
    if (8 * q < kRows) {
      voff[q] = row < a.M ? Operand<false, 64>::offset(k, row, a.lda) : kOut;
    } else {
      int n = row - kRows;
      bool in = n0 + n < NO;
      if (GATED) {
        const int j = (n >> 4) * 8 + (n & 7);
        in = n0 + j < NO;
        n = j + (n & 8 ? NO : 0);
      }
      voff[q] = in ? Operand<false, 64>::offset(k, n, a.ldw) : kOut;
    }
  }
  // Few rows and weights that the caches would not keep until the next step: past their replacement (1 x 4096 x 7168 13.1 -> 12.1
  // us from HBM; but 16 x 256 x 7168, which they keep, 7.5 -> 11.0, and 32 x 4096 x 7168 from the Infinity Cache 11.7 -> 15.4).
  const bool once = a.M <= 8 && (int64_t)a.N * a.K >= 8 << 20;
  int slot = 0;
  auto issue = [&](int b) {
    const bool rest = 64 * (kb0 + b) + 64 > a.K;
#pragma unroll
    for (int q = 0; q < C::kCopies; ++q) {
      uint32_t v = voff[q];
      if (rest && 64 * (kb0 + b) + (q & 1 ? ck ^ 32 : ck) >= a.K) v = kOut;
      const uint32_t to = (uint32_t)uniform((int)(lds0 + slot * C::kBlock + 1024 * q));
      if (8 * q < kRows) copy16(v, abase, to);
      else if (once) copy16_once(v, wbase, to);
      else copy16(v, wbase, to);
    }
    abase += 128;
    wbase += 128;
    slot = slot + 1 == S ? 0 : slot + 1;
  };
  Operand<false, 64> op;
  op.init(lane, 0);
  v4f acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int b = 0; b < S; ++b)
    if (b < nb) issue(b);
  int cs = 0;
  for (int b = 0; b < nb; ++b) {
    if (b + S <= nb) wait_vmcnt<(S - 1) * C::kCopies>();
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    const uint8_t* blk = ring + cs * C::kBlock;
    cs = cs + 1 == S ? 0 : cs + 1;
    v8bf x[2][RB], w[2][CB];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < RB; ++i) x[h][i] = op.frag(blk, i, h);
#pragma unroll
      for (int j = 0; j < CB; ++j) w[h][j] = op.frag(blk, RB + j, h);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the fragments are in registers: the slot is filled anew
    if (b + S < nb) issue(b + S);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < CB; ++j)
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[i][j] = mma(w[h][j], x[h][i], acc[i][j]);
  }
  // over the wave's own ring, whose copies have all landed and been read; lane: columns 4 lg .. + 3 of row l16
  float* part = (float*)ring;
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) *(v4f*)(part + (16 * i + l16) * (kCols + 4) + 16 * j + 4 * lg) = acc[i][j];
  __syncthreads();
  for (int q = threadIdx.x; q < kRows * kOuts / 4; q += KS * 64) {
    const int m = q / (kOuts / 4), n = 4 * (q % (kOuts / 4));
    const int c = GATED ? (n >> 3) * 16 + (n & 7) : n;
    v4f v = {0.f, 0.f, 0.f, 0.f}, up = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const float* p = (const float*)(sm + k * C::kWave) + m * (kCols + 4) + c;
      v += *(const v4f*)p;
      if (GATED) up += *(const v4f*)(p + 8);
    }
    epilogue4<GATED>(a, m, n0 + n, v, up);
  }
}

template <bool GATED, int RB, int CB, int KS, int S>
hipError_t launch_stream(const LinearArgs& a, hipStream_t s) {
  const int NO = GATED ? a.N / 2 : a.N, outs = GATED ? 8 * CB : 16 * CB;
  gemm_linear_stream_kernel<GATED, RB, CB, KS, S><<<(NO + outs - 1) / outs, KS * 64, 0, s>>>(a);
  return hipGetLastError();
}

template <bool TA, bool TW, bool GATED>
hipError_t launch_order(LinearArgs a, hipStream_t s) {
  const LinPlan p = plan_linear(a.M, a.N, a.K, TA || TW);
  a.splits = p.splits;
  if constexpr (!TA && !TW) {
    const bool many = a.N > 16 * kLinCus;
    if (p.kind == kLinStream16) return many ? launch_stream<GATED, 1, 2, 4, 6>(a, s) : launch_stream<GATED, 1, 1, 8, 5>(a, s);
    if (p.kind == kLinStream32) return many ? launch_stream<GATED, 2, 2, 4, 5>(a, s) : launch_stream<GATED, 2, 1, 8, 3>(a, s);
    if (p.kind == kLinStream64) return many ? launch_stream<GATED, 4, 2, 4, 3>(a, s) : launch_stream<GATED, 4, 1, 4, 4>(a, s);
  }
  switch (p.kind) {
    case kLin64x64: return launch_tile<TA, TW, GATED, 2, 2, 2, 2>(a, s);
    case kLin64x128: return launch_tile<TA, TW, GATED, 2, 2, 2, 4>(a, s);
    case kLin128x128: return launch_tile<TA, TW, GATED, 4, 2, 2, 4>(a, s);
    case kLin128x128two: return launch_tile<TA, TW, GATED, 4, 4, 2, 2, true>(a, s);
    default: return launch_tile<TA, TW, GATED, 8, 4, 2, 4, true>(a, s);
  }
}

}  // namespace

int64_t linear_workspace_bytes(int M, int N, int K) {
  // any order and a gated epilogue may be asked for: the largest need
  const int x = plan_linear(M, N, K, false).splits, y = plan_linear(M, N, K, true).splits, s = x > y ? x : y;
  return s > 1 ? 4ll * s * M * (((N + 3) & ~3) + 4) : 0;
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  if (a.gated) return launch_order<false, false, true>(a, s);
  if (!a.ta) return a.tw ? launch_order<false, true, false>(a, s) : launch_order<false, false, false>(a, s);
  return launch_order<true, true, false>(a, s);
}

}  // namespace moe
