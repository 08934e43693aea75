// decode.hip -- moe_experts_decode: the experts of a few tokens, in two kernels.
//
//   up:    h[t,r,j] = silu(sum_k Wg[e,j,k] x[t,k]) * (sum_k Wu[e,j,k] x[t,k]),   e = topk_ids[t,r]
//   down:  Z[t,n]   = C[t,n] + sum_r p[t,r] * sum_j W2[e,n,j] h[t,r,j]
//
// With few tokens the step is the reading of the active experts' weights, each byte once.  So nothing is packed or
// requantised: every workgroup finds the active experts and their tokens from topk_ids itself (plan()), and the waves stream
// weights.  Weights and the rows that meet them are copied global -> LDS, block by block, into a ring that belongs to one
// wave: no barrier in the stream, and the ring runs on across experts and column blocks, so that it is never drained.
//
// Both kernels multiply with v_mfma_f32_16x16x32_bf16, rows (tokens) as its A operand and 16 weight columns as its B operand:
// a lane holds one column of 4 rows.  FP8 codes are widened to bf16 (exact), 4-bit codes become 128 + q in bf16 (exact), with
// -136 times the row's sum from an instruction against a constant; a block's sum of 128 products is scaled in fp32.  MXFP4
// codes are widened together with their power-of-two scale (exact) and need no block sum; a unit with one of the two largest scales,
// which take codes past bf16's range, is added up a second time.  h is rounded to bf16 once (it is
// the matrix instruction's operand; everything else up to Z stays in fp32).
//
// A job is an expert and up to BR of its routes.  Up-projection: a unit is a job and 16 (4-bit and MXFP4: 32) columns of h, whose
// K the 4 (8) waves share; persistent workgroups walk over the units.  Down-projection: a workgroup owns 16 columns of Z and takes every
// job, its waves in turn; the rows' sums meet in LDS as one line per route, so the sum over a token's slots runs in slot order
// whatever wave was first, and no partial result goes through memory.
//
// Measured (us; TB/s of the active experts' weights): 1 token, 8 of 256 experts, 7168 x 2048, FP8 59.4 (5.9); 61 tokens, 8 of 128,
// 4096 x 1536, bf16 679 to 694 (6.8 to 7.0), FP8 368 (6.4); 16 tokens, 4096 x 768, 4-bit packed 80 (5.0), row-major 120
// (copied in pieces of 64 bytes), MXFP4 packed 80, row-major 124.  A plain read of memory reaches 7.3 TB/s.  What bounds it: bytes
// in flight (the rings, 64 to 110 KB a compute unit), the start and the last round of units, and for 4-bit codes the widening beside
// the stream.  Two things cost more than the active experts' bytes: an expert with more than BR routes is read once for each of its jobs
// (Zipf routing of 61 tokens, 8 of 256, 4096 x 1024, FP8: 206 jobs of 149 experts, 4.8 TB/s of the active bytes where uniform
// routing has 6.1), and from about 600 routes on the routes' tables and lines leave room for fewer rings (128 tokens, 8 of 128, 4096 x
// 1536: FP8 445, 5.4 TB/s).
#include "decode_plan.h"
#include "linear_act.h"
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kBf16 = kDecBf16, kFp8 = kDecFp8, kInt4 = kDecInt4, kFp4 = kDecFp4;
constexpr int kRoutes = kDecodeMaxRoutes;

template <int F>
struct Fmt {
  static constexpr int BK = dec_block(F);                   // K values of a block
  static constexpr bool kHalf = dec_half(F);                // two weights a byte
  static constexpr int kPieces = kHalf ? 1 : 2;             // 1 KB copies per 16 columns and block
  static constexpr int kRowBytes = kHalf ? 64 : 128;        // of a weight row's block
  static constexpr int kXRow = 2 * BK;                      // bytes of an activation row's block
  static constexpr int kXChunks = kXRow / 16;
  static constexpr int kRowsPerPiece = 1024 / kXRow;
  static constexpr int kScaled = F != kBf16;
  __device__ static __forceinline__ int row_bytes(int K) { return kHalf ? K / 2 : F == kFp8 ? K : 2 * K; }
};

struct DecodeSide {      // one projection
  const uint8_t* W;      // [E, N, K] in the format
  const uint8_t* S;      // scales: fp32 [E, N/128, K/128], fp16 [E, N, K/128], E8M0 [E, N, K/32], or none
  int N, K;
};

__device__ __forceinline__ void copy16(uint32_t voff, const void* base, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(voff), "s"(base), "{m0}"(lds) : "memory");
}
// Weights, past the caches' replacement: each is read once (61 tokens in bf16: 808 us without, 731 with).
__device__ __forceinline__ void copy16_once(uint32_t voff, const void* base, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" : : "v"(voff), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t voff, const void* base, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" : : "v"(voff), "s"(base), "{m0}"(lds) : "memory");
}

// The bf16 values of 8 E4M3 codes (exact).
__device__ __forceinline__ v8bf widen_fp8(int lo, int hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// The bf16 values of 8 E2M1 codes times a power of two (exact below 2^128; its E8M0 byte is the scale's exponent: byte 0 is 2^-127,
// 255 NaN, and bf16's subnormals hold the smallest ones).
__device__ __forceinline__ v8bf widen_fp4(uint32_t w, float scale) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// The two scales (2^126 and 2^127) that take codes past the largest bf16 number.
constexpr uint32_t kFarScale = 253, kNanScale = 255;
// 128 + q of a dword's 8 nibbles, in the order of nibbles 0 4 1 5 2 6 3 7.  magic: 0x43004300 in a vector register, so that mask
// and exponent take one instruction.
__device__ __forceinline__ v8bf widen_int4(uint32_t w, uint32_t magic) {
  constexpr uint32_t m = 0x000f000fu;
  const v4i v = {(int)((w & m) | magic), (int)(((w >> 4) & m) | magic), (int)(((w >> 8) & m) | magic),
                 (int)(((w >> 12) & m) | magic)};
  return __builtin_bit_cast(v8bf, v);
}
// 8 values in that order.
__device__ __forceinline__ v4i nibble_order(const v4i x) {
  return v4i{(int)__builtin_amdgcn_perm((uint32_t)x[2], (uint32_t)x[0], 0x05040100u),
             (int)__builtin_amdgcn_perm((uint32_t)x[2], (uint32_t)x[0], 0x07060302u),
             (int)__builtin_amdgcn_perm((uint32_t)x[3], (uint32_t)x[1], 0x05040100u),
             (int)__builtin_amdgcn_perm((uint32_t)x[3], (uint32_t)x[1], 0x07060302u)};
}
__device__ __forceinline__ v4f mma(const v4i x, const v8bf w, const v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), w, c, 0, 0, 0);
}

// ------------------------------------------------------------------ plan --
struct Plan {
  uint32_t* job;    // [R] expert | rows << 10 | (first place in order) << 15
  uint16_t* order;  // [R] routes grouped by expert
  int* njobs;
  __device__ __forceinline__ Plan(uint8_t* mem, int R) {
    njobs = (int*)mem;
    job = (uint32_t*)(mem + 4);
    order = (uint16_t*)(job + R);
  }
  __device__ __forceinline__ static int expert(uint32_t j) { return j & 1023; }
  __device__ __forceinline__ static int rows(uint32_t j) { return j >> 10 & 31; }
  __device__ __forceinline__ int route(uint32_t j, int i) const { return order[(j >> 15) + i]; }
};

// Sums of v over this lane and the lanes before it, inside the VALU: within rows of 16 lanes, then over the rows.
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);  // row_bcast:15 to rows 1, 3
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);  // row_bcast:31 to rows 2, 3
  return v;
}

constexpr int kFewRoutes = 64;  // so many routes are grouped by one wave, with one barrier

// Every thread of the workgroup calls it.  count: kMaxExperts ints, used before anything else in LDS is.  A route's place among
// its expert's is first whatever the atomics make it; SORTED: then the order of the routes, the same in every workgroup, as it has
// to be where several of them share a job.  (A row's sums do not depend on the rows beside it.)
template <int BR, int NT, bool SORTED>
__device__ void plan(const Plan& p, int* count, const DecodeArgs& a, bool report) {
  const int R = a.T * a.k;
  if (R <= kFewRoutes) {  // a lane per route: its expert's routes are counted lane by lane
    if (threadIdx.x < kWave) {
      const int lane = lane_id();
      int id = lane < R ? a.ids[lane] : -1;
      if (report && __ballot(id >= a.E) != 0 && lane == 0) atomicOr(a.status, 1);
      if (id >= a.E) id = -1;
      int n = 0, before = 0, first = 0;
#pragma unroll 4
      for (int j = 0; j < R; ++j) {
        const bool same = id == __builtin_amdgcn_readlane(id, j);
        if (same && n == 0) first = j;
        n += same;
        before += same && j < lane;
      }
      const bool lead = id >= 0 && before == 0;
      const uint32_t mine = lead ? (uint32_t)n | (uint32_t)((n + BR - 1) / BR) << 16 : 0u, pre = wave_prefix(mine);
      const uint32_t base = pre - mine;
      const int at = __shfl((int)(base & 0xffff), first);
      if (id >= 0) p.order[at + before] = (uint16_t)lane;
      if (lead)
        for (int b = 0; b * BR < n; ++b)
          p.job[(base >> 16) + b] = (uint32_t)id | (uint32_t)min(n - b * BR, BR) << 10 | (uint32_t)(at + b * BR) << 15;
      if (lane == kWave - 1) *p.njobs = (int)(pre >> 16);
    }
    __syncthreads();
    return;
  }
  for (int e = threadIdx.x; e < a.E; e += NT) count[e] = 0;
  int id[kRoutes / NT], place[kRoutes / NT];
#pragma unroll
  for (int q = 0; q < kRoutes / NT; ++q) {
    const int i = threadIdx.x + NT * q;
    id[q] = i < R ? a.ids[i] : -1;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kRoutes / NT; ++q) {
    if (id[q] >= a.E) {
      if (report) atomicOr(a.status, 1);  // MOE_DEV_ID_RANGE
      id[q] = -1;
    }
    if (id[q] >= 0) place[q] = atomicAdd(count + id[q], 1);
  }
  __syncthreads();
  if (threadIdx.x < kWave) {
    uint32_t base = 0;  // routes | jobs << 16
    for (int c = 0; c < a.E; c += kWave) {
      const int e = c + lane_id(), n = e < a.E ? count[e] : 0, jobs = (n + BR - 1) / BR;
      const uint32_t pre = wave_prefix((uint32_t)n | (uint32_t)jobs << 16);
      const uint32_t mine = base + pre - ((uint32_t)n | (uint32_t)jobs << 16);
      const int at = mine & 0xffff;
      if (n > 0) count[e] = at | n << 16;
      for (int b = 0; b < jobs; ++b)
        p.job[(mine >> 16) + b] = (uint32_t)e | (uint32_t)min(n - b * BR, BR) << 10 | (uint32_t)(at + b * BR) << 15;
      base += (uint32_t)__builtin_amdgcn_readlane((int)pre, kWave - 1);
    }
    if (threadIdx.x == 0) *p.njobs = (int)(base >> 16);
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kRoutes / NT; ++q) {
    const int i = threadIdx.x + NT * q;
    if (id[q] >= 0) p.order[(count[id[q]] & 0xffff) + place[q]] = (uint16_t)i;
  }
  __syncthreads();
  if (!SORTED) return;
#pragma unroll
  for (int q = 0; q < kRoutes / NT; ++q) {
    if (id[q] < 0) continue;
    const int at = count[id[q]] & 0xffff, n = count[id[q]] >> 16, i = threadIdx.x + NT * q;
    place[q] = at;
    for (int j = 0; j < n; ++j) place[q] += p.order[at + j] < i;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kRoutes / NT; ++q) {
    const int i = threadIdx.x + NT * q;
    if (id[q] >= 0) p.order[place[q]] = (uint16_t)i;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- stream --
// One wave's ring: S blocks of NCB x 16 weight columns and BR rows, all of them in flight while a block is multiplied (its
// fragments go to registers first, so that its slot is filled anew at once).
template <int F, bool PACKED, int NCB, int BR, int RING>
struct Stream {
  using T = Fmt<F>;
  static constexpr int XP = (BR + T::kRowsPerPiece - 1) / T::kRowsPerPiece;
  static constexpr int kWBytes = NCB * T::kPieces * 1024, kXBytes = XP * 1024;
  // copies of 256 bytes with a block's scales (packed MXFP4: those of 64 columns each)
  static constexpr int kScales = !T::kScaled ? 0 : F == kFp4 && PACKED && NCB > 1 ? 2 : 1;
  static constexpr int kSlot = kWBytes + kXBytes + 256 * kScales;
  static constexpr int kCopies = NCB * T::kPieces + XP + kScales;
  static constexpr int S0 = RING / kSlot, S = S0 > 8 ? 8 : S0;
  static_assert(S >= 2 && (S - 1) * kCopies < 64, "ring; vmcnt's range");
  static_assert(BR == XP * T::kRowsPerPiece && BR <= 16, "rows in whole copies");

  const DecodeSide side;
  const uint8_t* x;        // rows of K bf16
  uint8_t* ring;
  uint32_t lds0;
  int lane, l16, lg;
  uint32_t wvoff[T::kPieces];
  uint32_t wstep;          // weight bytes from block to block
  // producer: where the next block comes from
  const uint8_t* wbase[NCB];
  const uint8_t* sbase;
  uint32_t xvoff[XP], svoff[2], sstep;
  int pkb, pend, pslot;
  int cslot;
  uint32_t top;            // MXFP4: the largest scale byte of this lane's since begin()

  __device__ __forceinline__ Stream(const DecodeSide& s, const uint8_t* rows, uint8_t* mem) : side(s), x(rows), ring(mem) {
    lane = lane_id();
    l16 = lane & 15;
    lg = lane >> 4;
    lds0 = (uint32_t)uniform((int)lds_offset(mem));
    const uint32_t rowb = T::row_bytes(side.K);
#pragma unroll
    for (int p = 0; p < T::kPieces; ++p) {
      if (PACKED) {
        wvoff[p] = 1024 * p + 16 * lane;
      } else if (T::kHalf) {
        wvoff[p] = (uint32_t)(lane >> 2) * rowb + 16u * ((lane & 3) ^ ((lane >> 4) & 3));
      } else {
        const int row = 8 * p + (lane >> 3);
        wvoff[p] = (uint32_t)row * rowb + 16u * ((lane & 7) ^ ((row >> 1) & 7));
      }
    }
    wstep = PACKED ? (uint32_t)side.N * T::kRowBytes : T::kRowBytes;
    pslot = cslot = 0;
    pkb = pend = 0;
  }

  // Blocks kb0 .. kb1 of columns n(cb) = col0 + 16 cb for cb < NCB/2, col1 + 16 (cb - NCB/2) above (NCB 1: col0), for the
  // job's rows of x: its tokens' (TOKENS; per_k = ceil(2^16 / k): route / k in one product, exact for routes below 2^10 and k up to 64)
  // or its routes'.
  template <bool TOKENS>
  __device__ __forceinline__ void produce(const Plan& p, uint32_t job, uint32_t per_k, int col0, int col1, int kb0, int kb1) {
    const int e = p.expert(job), m = p.rows(job);
    const int64_t rowb = T::row_bytes(side.K);
    const uint8_t* we = side.W + (int64_t)e * side.N * rowb;
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) {
      const int n = NCB == 1 ? col0 : cb < NCB / 2 ? col0 + 16 * cb : col1 + 16 * (cb - NCB / 2);
      wbase[cb] = we + (PACKED ? (int64_t)(n / 16) * (T::kPieces * 1024) : n * rowb) + (int64_t)kb0 * wstep;
    }
#pragma unroll
    for (int q = 0; q < XP; ++q) {
      const int row = T::kRowsPerPiece * q + lane / T::kXChunks, c = lane % T::kXChunks;
      const int sw = F == kBf16 ? (row >> 1) & 7 : row & 15;
      const uint32_t r = (uint32_t)p.route(job, min(row, m - 1));
      xvoff[q] = (TOKENS ? r * per_k >> 16 : r) * (uint32_t)side.K * 2u + 16u * (c ^ sw) + (uint32_t)kb0 * T::kXRow;
    }
    if constexpr (F == kFp8) {  // lane: the scale of column block lane % NCB
      const int cb = lane % NCB, KB = side.K / 128;
      const int n = NCB == 1 ? col0 : cb < NCB / 2 ? col0 + 16 * cb : col1 + 16 * (cb - NCB / 2);
      sbase = side.S + (int64_t)e * (side.N / 128) * KB * 4;
      svoff[0] = (uint32_t)((n / 128) * KB + kb0) * 4u;
      sstep = 4;
    } else if constexpr (F == kInt4) {  // lane: that of column l16 of column block lg % NCB, and its neighbour in the dword
      const int cb = lg % NCB, KG = side.K / 128;
      const int n = (NCB == 1 ? col0 : cb < NCB / 2 ? col0 + 16 * cb : col1 + 16 * (cb - NCB / 2)) + l16;
      sbase = side.S + (int64_t)e * side.N * KG * 2;
      svoff[0] = 2u * (uint32_t)(PACKED ? (kb0 * (side.N / 64) + n / 64) * 64 + (n & 15) * 4 + (n & 63) / 16 : n * KG + kb0);
      sstep = PACKED ? 2u * side.N : 2u;
    } else if constexpr (F == kFp4) {  // a dword: the 4 scales of a column's block, or packed the lane's own of 4 column blocks
      const int cb = lg % NCB, KG = side.K / 128;
      sbase = side.S + (int64_t)e * side.N * KG * 4;
      if (PACKED) {
        svoff[0] = 4u * (uint32_t)((kb0 * (side.N / 64) + col0 / 64) * 64 + lane);
        svoff[1] = 4u * (uint32_t)((kb0 * (side.N / 64) + col1 / 64) * 64 + lane);
        sstep = 4u * side.N;
      } else {
        const int n = (NCB == 1 ? col0 : cb < NCB / 2 ? col0 + 16 * cb : col1 + 16 * (cb - NCB / 2)) + l16;
        svoff[0] = 4u * (uint32_t)(n * KG + kb0);
        sstep = 4u;
      }
    }
    pkb = kb0;
    pend = kb1;
  }

  __device__ __forceinline__ void issue() {
    const uint32_t to = lds0 + (uint32_t)pslot * kSlot;
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) {
#pragma unroll
      for (int p = 0; p < T::kPieces; ++p)
        copy16_once(wvoff[p], wbase[cb], (uint32_t)uniform((int)(to + (cb * T::kPieces + p) * 1024)));
      wbase[cb] += wstep;
    }
#pragma unroll
    for (int q = 0; q < XP; ++q) {
      copy16(xvoff[q], x, (uint32_t)uniform((int)(to + kWBytes + 1024 * q)));
      xvoff[q] += T::kXRow;
    }
#pragma unroll
    for (int q = 0; q < kScales; ++q) {
      copy4(svoff[q] & ~3u, sbase, (uint32_t)uniform((int)(to + kWBytes + kXBytes + 256 * q)));
      svoff[q] += sstep;
    }
    pslot = pslot + 1 == S ? 0 : pslot + 1;
    ++pkb;
  }

  // The oldest block's fragments, in registers.
  struct Frags {
    v4i w[NCB][T::kPieces], x[F == kBf16 ? 2 : 4];
    uint32_t s[NCB];  // FP8: the scale; 4-bit: a dword with the scale in either half; MXFP4: with it in one of its bytes
  };
  __device__ __forceinline__ void read(Frags& f) {
    const uint8_t* w = ring + cslot * kSlot;
    const uint8_t* xs = w + kWBytes;
    const uint8_t* sc = xs + kXBytes;
    const int row = l16 & (BR - 1);  // the rows past BR repeat; nobody reads their sums
    if constexpr (F == kBf16) {
#pragma unroll
      for (int h = 0; h < 2; ++h) f.x[h] = *(const v4i*)(xs + row * 128 + 16 * ((4 * h + lg) ^ ((row >> 1) & 7)));
    } else if constexpr (F == kFp8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f.x[i] = *(const v4i*)(xs + row * 256 + 16 * ((8 * (i >> 1) + 2 * lg + (i & 1)) ^ row));
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d) f.x[d] = *(const v4i*)(xs + row * 256 + 16 * ((PACKED && F == kInt4 ? 4 * d + lg : 4 * lg + d) ^ row));
    }
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) {
#pragma unroll
      for (int h = 0; h < T::kPieces; ++h) {
        const int at = PACKED ? 1024 * h + 16 * lane
                              : T::kHalf ? l16 * 64 + 16 * (lg ^ (l16 >> 2)) : l16 * 128 + 16 * ((4 * h + lg) ^ ((l16 >> 1) & 7));
        f.w[cb][h] = *(const v4i*)(w + cb * T::kPieces * 1024 + at);
      }
      if constexpr (F == kFp8) f.s[cb] = *(const uint32_t*)(sc + 4 * cb);
      if constexpr (F == kInt4 || (F == kFp4 && !PACKED)) f.s[cb] = *(const uint32_t*)(sc + 4 * (16 * cb + l16));
      if constexpr (F == kFp4 && PACKED) f.s[cb] = *(const uint32_t*)(sc + (NCB > 1 && cb >= NCB / 2 ? 256 : 0) + 4 * lane);
    }
    cslot = cslot + 1 == S ? 0 : cslot + 1;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot may be filled anew
  }
  // acc += the block.  kb and col0/col1 are the consumer's (4-bit scales lie in either half of a dword).
  __device__ __forceinline__ void multiply(const Frags& f, v4f (&acc)[NCB], int kb, int col0, int col1) {
    if constexpr (F == kBf16) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb) acc[cb] = mma(f.x[h], __builtin_bit_cast(v8bf, f.w[cb][h]), acc[cb]);
    } else if constexpr (F == kFp8) {
      v4f s[NCB];
#pragma unroll
      for (int cb = 0; cb < NCB; ++cb) s[cb] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb)
          s[cb] = mma(f.x[i], widen_fp8(f.w[cb][i >> 1][2 * (i & 1)], f.w[cb][i >> 1][2 * (i & 1) + 1]), s[cb]);
#pragma unroll
      for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[cb][i] = __builtin_fmaf(__uint_as_float(f.s[cb]), s[cb][i], acc[cb][i]);
    } else if constexpr (F == kFp4) {
      // E2M1 times a power of two is a bf16 number: widened with its scale, products add up without a block sum of their own
#pragma unroll
      for (int cb = 0; cb < NCB; ++cb) {
        const uint32_t e8m0 = f.s[cb] >> (8 * scale_byte(column(cb, col0, col1))) & 0xffu;
        const float scale = __uint_as_float(e8m0 << 23);
        top = max(top, e8m0);
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[cb] = mma(f.x[d], widen_fp4((uint32_t)f.w[cb][0][d], scale), acc[cb]);
      }
    } else {
      const v8bf m136 = {(__bf16)-136.f, (__bf16)-136.f, (__bf16)-136.f, (__bf16)-136.f,
                         (__bf16)-136.f, (__bf16)-136.f, (__bf16)-136.f, (__bf16)-136.f};
      uint32_t magic = 0x43004300u;
      asm("" : "+v"(magic));
      v4i x[4];
      v4f s[NCB], fix = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        x[d] = PACKED ? f.x[d] : nibble_order(f.x[d]);
        fix = mma(x[d], m136, fix);
      }
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb) s[cb] = mma(x[d], widen_int4((uint32_t)f.w[cb][0][d], magic), d == 0 ? fix : s[cb]);
#pragma unroll
      for (int cb = 0; cb < NCB; ++cb) {
        const int n = (NCB == 1 ? col0 : cb < NCB / 2 ? col0 + 16 * cb : col1 + 16 * (cb - NCB / 2)) + l16;
        // (packed: the column block's parity; NCB / 2 blocks from a multiple of 32 on)
        const int half = PACKED ? (NCB == 1 ? col0 / 16 : cb) & 1 : (n * (side.K / 128) + kb) & 1;
        const float q = (float)__builtin_bit_cast(_Float16, (uint16_t)(half ? f.s[cb] >> 16 : f.s[cb]));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[cb][i] = __builtin_fmaf(q, s[cb][i], acc[cb][i]);
      }
    }
  }

  // The first weight column of block cb; the byte of a scale dword that is this lane's for it (MXFP4).
  __device__ __forceinline__ static int column(int cb, int col0, int col1) {
    return NCB == 1 ? col0 : cb < NCB / 2 ? col0 + 16 * cb : col1 + 16 * (cb - NCB / 2);
  }
  __device__ __forceinline__ int scale_byte(int n) const { return PACKED ? (n & 63) / 16 : lg; }

  __device__ __forceinline__ void begin(v4f (&acc)[NCB]) {
    top = 0;
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) acc[cb] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  // After blocks kb0 .. kb1 of produce()'s arguments.  MXFP4: if a scale among them was a far one, acc is nothing yet; they are added up
  // again, out of memory, products under such scales with the scale 2^8 lower and in a sum of their own.  (The stream's copies do not
  // mind: they only make waits longer.  Keeping `top` costs the stream nothing that shows, where a branch in every block cost up to
  // 7%: 128 tokens, 8 of 256 experts, 4096 x 1024 packed 354 us, with the branch 378.)
  template <bool TOKENS>
  __device__ __forceinline__ void end(v4f (&acc)[NCB], const Plan& p, uint32_t job, uint32_t per_k, int col0, int col1, int kb0, int kb1) {
    if constexpr (F == kFp4) {
      if (__builtin_expect(__ballot(top >= kFarScale) == 0, 1)) return;
      begin(acc);
      const int64_t rowb = T::row_bytes(side.K), e = p.expert(job);
      const int KG = side.K / 128;
      const uint32_t r = (uint32_t)p.route(job, min(l16 & (BR - 1), p.rows(job) - 1));
      const uint8_t* xr = x + (int64_t)(TOKENS ? r * per_k >> 16 : r) * side.K * 2;
#pragma unroll 1
      for (int kb = kb0; kb < kb1; ++kb) {
        v4i xf[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) xf[d] = *(const v4i*)(xr + kb * T::kXRow + 16 * (4 * lg + d));
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb) {
          const int n = column(cb, col0, col1);
          const uint8_t* w = side.W + e * side.N * rowb + (PACKED ? (int64_t)(n / 16) * 1024 + (int64_t)kb * wstep + 16 * lane
                                                                  : (n + l16) * rowb + (int64_t)kb * wstep + 16 * lg);
          const v4i wf = *(const v4i*)w;
          const int at = PACKED ? (kb * (side.N / 64) + n / 64) * 64 + lane : (n + l16) * KG + kb;
          const uint32_t s4 = *(const uint32_t*)(side.S + e * side.N * KG * 4 + 4 * (int64_t)at);
          const uint32_t e8m0 = s4 >> (8 * scale_byte(n)) & 0xffu;
          const bool far = e8m0 >= kFarScale && e8m0 != kNanScale;
          const float scale = __uint_as_float((far ? e8m0 - 8 : e8m0) << 23);
          v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            s = mma(xf[d], widen_fp4(far ? (uint32_t)wf[d] : 0u, scale), s);
            acc[cb] = mma(xf[d], widen_fp4(far ? 0u : (uint32_t)wf[d], scale), acc[cb]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[cb][i] = __builtin_fmaf(256.f, s[i], acc[cb][i]);
        }
      }
    }
  }

  // Wait for the oldest block; `full`: S - 1 blocks were issued after it.
  __device__ __forceinline__ void arrive(bool full) {
    if (full) wait_vmcnt<(S - 1) * kCopies>();
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");
  }
};

// -------------------------------------------------------------------- up --
template <int F, int BR, int NW>
struct UpCfg {
  static constexpr int NCB = dec_up_blocks(F), kCols = dec_up_cols(F), kRow = dec_up_row(F);
  static constexpr int kPart = dec_up_part(F, BR, NW), kBufs = dec_up_bufs(F, BR, NW), kPlanAt = dec_up_plan_at(F, BR, NW);
  static_assert(dec_up_lds(F, BR, NW, kRoutes) <= kLdsMost, "any number of routes");
};

template <int F, bool PACKED, int BR, int NW>
__global__ __launch_bounds__(NW < 8 ? 512 : NW * 64) void decode_up_kernel(const DecodeArgs a) {
  using C = UpCfg<F, BR, NW>;
  constexpr int NCB = C::NCB, kCols = C::kCols;
  using St = Stream<F, PACKED, NCB, BR, kUpRing>;
  extern __shared__ __attribute__((aligned(1024))) uint8_t dyn[];
  uint8_t* ring = dyn;
  float* part = (float*)(dyn + NW * kUpRing);
  const Plan p(dyn + C::kPlanAt, a.T * a.k);
  static_assert(NW * kUpRing >= kMaxExperts * (int)sizeof(int), "the plan's table lies in the rings");
  plan<BR, NW * 64, true>(p, (int*)ring, a, blockIdx.x == 0 && a.status);
  const int wv = uniform(threadIdx.x >> 6);
  const DecodeSide side{(const uint8_t*)a.W13, (const uint8_t*)a.S13, 2 * a.I, a.H};
  St st(side, (const uint8_t*)a.x, ring + wv * kUpRing);
  const int ncol = a.I / kCols, units = *p.njobs * ncol;
  const int nb = a.H / Fmt<F>::BK, kb0 = wv * nb / NW, kb1 = (wv + 1) * nb / NW;

  // Workgroup b runs on XCD b % 8: consecutive units, which share their rows, go to one XCD.
  const int xs = gridDim.x / 8, xr = gridDim.x % 8, xcd = blockIdx.x % 8;
  const int first = xcd * xs + min(xcd, xr) + blockIdx.x / 8;
  int pu = first;       // the producer's unit
  auto feed = [&]() {   // one block into the ring, if there is one
    if (st.pkb == st.pend) {
      if (pu >= units || kb0 == kb1) return false;
      const int col = pu % ncol * kCols;
      st.template produce<true>(p, (uint32_t)uniform((int)p.job[pu / ncol]), a.per_k, col, a.I + col, kb0, kb1);
      pu += gridDim.x;
    }
    st.issue();
    return true;
  };
  bool full = true;  // S blocks were issued from the oldest on
#pragma unroll 1
  for (int i = 0; i < St::S; ++i) full = feed();
  int buf = 0;
  for (int u = first; u < units; u += gridDim.x) {
    const uint32_t job = (uint32_t)uniform((int)p.job[u / ncol]);
    const int col = u % ncol * kCols, m = p.rows(job);
    v4f acc[NCB];
    st.begin(acc);
#pragma unroll 1
    for (int kb = kb0; kb < kb1; ++kb) {
      typename St::Frags f;
      st.arrive(full);
      st.read(f);
      full = feed();
      st.multiply(f, acc, kb, col, a.I + col);
    }
    st.template end<true>(acc, p, job, a.per_k, col, a.I + col, kb0, kb1);
    float* sums = part + buf * C::kPart;
    float* mine = sums + wv * BR * C::kRow;
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * st.lg + i < BR) mine[(4 * st.lg + i) * C::kRow + 16 * cb + st.l16] = acc[cb][i];
    barrier_lds();  // with two buffers the only one: the other is written before this one's readers' next barrier
    for (int q = threadIdx.x; q < BR * kCols; q += NW * 64) {
      const int row = q / kCols, c = q % kCols;
      if (row < m) {
        float g = 0.f, up = 0.f;
#pragma unroll
        for (int v = 0; v < NW; ++v) {
          g += sums[(v * BR + row) * C::kRow + c];
          up += sums[(v * BR + row) * C::kRow + kCols + c];
        }
        a.h[(int64_t)p.route(job, row) * a.I + col + c] = (uint16_t)f32_to_bf16_rne(g * sigmoid_f32(g) * up);
      }
    }
    if (C::kBufs == 1) barrier_lds();
    else buf ^= 1;
  }
}

// ------------------------------------------------------------------ down --
static_assert(dec_down_lds(4, kDownRing, 1, kRoutes) <= kLdsMost, "any number of routes fits four waves' rings");

// LDS: NW rings, then a line of 16 sums per share of K and route, then topk_weights and the plan.
template <int F, bool PACKED, int BR, int NW, int RING>
__global__ __launch_bounds__(NW < 8 ? 512 : NW * 64) void decode_down_kernel(const DecodeArgs a) {
  using St = Stream<F, PACKED, 1, BR, RING>;
  extern __shared__ __attribute__((aligned(1024))) uint8_t dyn[];
  static_assert(NW * RING >= kMaxExperts * (int)sizeof(int), "the plan's table lies in the rings");
  float* y = (float*)(dyn + NW * RING);
  const int R = a.T * a.k, KS = a.ksplit;
  float* share = y + 16 * KS * R;  // topk_weights, 0 for skipped slots, whose lines of sums are 0 too
  const Plan p((uint8_t*)(share + R), R);
  plan<BR, NW * 64, false>(p, (int*)dyn, a, false);
  const int wv = uniform(threadIdx.x >> 6);
  const DecodeSide side{(const uint8_t*)a.W2, (const uint8_t*)a.S2, a.H, a.I};
  St st(side, (const uint8_t*)a.h, dyn + wv * RING);
  const int n0 = blockIdx.x * 16, items = *p.njobs * KS, nb = a.I / Fmt<F>::BK;

  int pi = wv;
  auto feed = [&]() {
    if (st.pkb == st.pend) {
      if (pi >= items) return false;
      const int ks = pi % KS;
      st.template produce<false>(p, (uint32_t)uniform((int)p.job[pi / KS]), 0, n0, n0, ks * nb / KS, (ks + 1) * nb / KS);
      pi += NW;
    }
    st.issue();
    return true;
  };
  bool full = true;
#pragma unroll 1
  for (int i = 0; i < St::S; ++i) full = feed();
  for (int i = threadIdx.x; i < R; i += NW * 64) {
    const bool on = (uint32_t)a.ids[i] < (uint32_t)a.E;
    share[i] = on ? a.p[i] : 0.f;
    if (!on)
      for (int c = 0; c < 16 * KS; ++c) y[(c / 16 * R + i) * 16 + c % 16] = 0.f;
  }
  for (int it = wv; it < items; it += NW) {
    const uint32_t job = (uint32_t)uniform((int)p.job[it / KS]);
    const int ks = it % KS, m = p.rows(job);
    v4f acc[1];
    const int kb0 = ks * nb / KS, kb1 = (ks + 1) * nb / KS;
    st.begin(acc);
#pragma unroll 1
    for (int kb = kb0; kb < kb1; ++kb) {
      typename St::Frags f;
      st.arrive(full);
      st.read(f);
      full = feed();
      st.multiply(f, acc, kb, n0, n0);
    }
    st.template end<false>(acc, p, job, 0, n0, n0, kb0, kb1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * st.lg + i < m) y[(ks * R + p.route(job, 4 * st.lg + i)) * 16 + st.l16] = acc[0][i];
  }
  __syncthreads();
  for (int q = threadIdx.x; q < a.T * 16; q += NW * 64) {
    const int t = q >> 4, c = q & 15;
    const int64_t at = (int64_t)t * a.H + n0 + c;
    float z = 0.f;
    for (int r = 0; r < a.k; ++r) {
      const int i = t * a.k + r;
      float v = y[i * 16 + c];
      for (int s = 1; s < KS; ++s) v += y[(s * R + i) * 16 + c];
      z = __builtin_fmaf(share[i], v, z);
    }
    if (a.C) z += bf16_to_f32(a.C[at]);
    a.Z[at] = (uint16_t)f32_to_bf16_rne(z);
  }
}

template <int F, bool PACKED, int BR, int NW>
hipError_t launch_up(const DecodeArgs& a, int groups, hipStream_t s) {
  decode_up_kernel<F, PACKED, BR, NW><<<groups, NW * 64, dec_up_lds(F, BR, NW, a.T * a.k), s>>>(a);
  return hipGetLastError();
}

template <int F, bool PACKED, int BR, int NW, int RING>
hipError_t launch_down(const DecodeArgs& a, hipStream_t s) {
  decode_down_kernel<F, PACKED, BR, NW, RING><<<a.H / 16, NW * 64, dec_down_lds(NW, RING, a.ksplit, a.T * a.k), s>>>(a);
  return hipGetLastError();
}

template <int F, bool PACKED, int BR>
hipError_t launch_rows(const DecodeArgs& a, const DecodePlan& p, hipStream_t s) {
  hipError_t e;
  if constexpr (BR < 16) e = p.up_waves == 8 ? launch_up<F, PACKED, BR, 8>(a, p.up_groups, s) : launch_up<F, PACKED, BR, 4>(a, p.up_groups, s);
  else e = launch_up<F, PACKED, BR, 4>(a, p.up_groups, s);
  if (e != hipSuccess) return e;
  if constexpr (Fmt<F>::kHalf && BR == 4)
    if (p.down_waves == 16) return launch_down<F, PACKED, BR, 16, kDownShort>(a, s);
  if constexpr (BR < 16) {
    if (p.down_ring == kDownDeep) {
      if constexpr (!(Fmt<F>::kHalf && BR == 4))
        if (p.down_waves == 8) return launch_down<F, PACKED, BR, 8, kDownDeep>(a, s);
      return launch_down<F, PACKED, BR, 4, kDownDeep>(a, s);
    }
  }
  return p.down_waves == 8 ? launch_down<F, PACKED, BR, 8, kDownRing>(a, s) : launch_down<F, PACKED, BR, 4, kDownRing>(a, s);
}

template <int F, bool PACKED>
hipError_t launch_format(DecodeArgs a, hipStream_t s) {
  const DecodePlan p = plan_decode(F, a.T, a.k, a.E, a.H, a.I, device_info().cus);
  a.per_k = (65536 + a.k - 1) / a.k;
  a.ksplit = p.ksplit;
  if constexpr (F != kBf16)
    if (p.rows == 4) return launch_rows<F, PACKED, 4>(a, p, s);
  return p.rows == 8 ? launch_rows<F, PACKED, 8>(a, p, s) : launch_rows<F, PACKED, 16>(a, p, s);
}

}  // namespace

int64_t decode_workspace_bytes(int T, int k, int I) { return (int64_t)T * k * I * 2; }

hipError_t launch_experts_decode(const DecodeArgs& a, hipStream_t s) {
  switch (a.format) {
    case kBf16: return a.packed ? launch_format<kBf16, true>(a, s) : launch_format<kBf16, false>(a, s);
    case kFp8: return a.packed ? launch_format<kFp8, true>(a, s) : launch_format<kFp8, false>(a, s);
    case kInt4: return a.packed ? launch_format<kInt4, true>(a, s) : launch_format<kInt4, false>(a, s);
    default: return a.packed ? launch_format<kFp4, true>(a, s) : launch_format<kFp4, false>(a, s);
  }
}

}  // namespace moe
