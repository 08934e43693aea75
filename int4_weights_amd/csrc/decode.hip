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
// -136 times the row's sum from an instruction against a constant; a block's sum of 128 products is scaled in fp32.  h is
// rounded to bf16 once (it is the matrix instruction's operand; everything else up to Z stays in fp32).
//
// A job is an expert and up to BR of its routes.  Up-projection: a unit is a job and 16 (4-bit: 32) columns of h, whose K the 4
// waves share; persistent workgroups walk over the units.  Down-projection: a workgroup owns 16 columns of Z and takes every
// job, its waves in turn; the rows' sums meet in LDS as one line per route, so the sum over a token's slots runs in slot order
// whatever wave was first, and no partial result goes through memory.
#include "linear_act.h"
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kBf16 = 0, kFp8 = 1, kInt4 = 2;
constexpr int kRoutes = kDecodeMaxRoutes;
constexpr int kUpWaves = 4;

template <int F>
struct Fmt {
  static constexpr int BK = F == kBf16 ? 64 : 128;          // K values of a block
  static constexpr int kPieces = F == kInt4 ? 1 : 2;        // 1 KB copies per 16 columns and block
  static constexpr int kRowBytes = F == kInt4 ? 64 : 128;   // of a weight row's block
  static constexpr int kXRow = 2 * BK;                      // bytes of an activation row's block
  static constexpr int kXChunks = kXRow / 16;
  static constexpr int kRowsPerPiece = 1024 / kXRow;
  static constexpr int kScaled = F != kBf16;
};

struct DecodeSide {      // one projection
  const uint8_t* W;      // [E, N, K] in the format
  const uint8_t* S;      // scales: fp32 [E, N/128, K/128], fp16 [E, N, K/128], or none
  int N, K;
};

__device__ __forceinline__ void copy16(uint32_t voff, const void* base, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(voff), "s"(base), "{m0}"(lds) : "memory");
}
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
// 128 + q of a dword's 8 nibbles, in the order of nibbles 0 4 1 5 2 6 3 7.
__device__ __forceinline__ v8bf widen_int4(uint32_t w) {
  const v4i v = {(int)((w & 0x000f000fu) | 0x43004300u), (int)(((w >> 4) & 0x000f000fu) | 0x43004300u),
                 (int)(((w >> 8) & 0x000f000fu) | 0x43004300u), (int)(((w >> 12) & 0x000f000fu) | 0x43004300u)};
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
  int16_t id[kRoutes];      // expert of each route, -1 if none
  int32_t job[kRoutes];     // expert | row block << 16, experts in order of their first route
  int njobs;
};

// Every thread of the workgroup calls it.  first/count: kMaxExperts ints each, used before anything else in LDS is.
template <int BR>
__device__ void plan(Plan& p, int* first, int* count, const int32_t* ids, int R, int E, int32_t* status) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    first[e] = 0x7fffffff;
    count[e] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < R; i += blockDim.x) {
    const int id = ids[i];
    const bool ok = (uint32_t)id < (uint32_t)E;
    p.id[i] = (int16_t)(ok ? id : -1);
    if (ok) {
      atomicMin(first + id, i);  // integers: the order does not matter
      atomicAdd(count + id, 1);
    } else if (id >= E && status) {
      atomicOr(status, 1);       // MOE_DEV_ID_RANGE
    }
  }
  __syncthreads();
  if (threadIdx.x < kWave) {
    int base = 0;
    for (int c = 0; c < R; c += kWave) {
      const int i = c + lane_id();
      const int id = i < R ? p.id[i] : -1;
      const int n = id >= 0 && first[id] == i ? (count[id] + BR - 1) / BR : 0;
      int pre = n;
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const int v = __shfl_up(pre, d);
        if (lane_id() >= d) pre += v;
      }
      for (int b = 0; b < n; ++b) p.job[base + pre - n + b] = id | (b << 16);
      base += __shfl(pre, kWave - 1);
    }
    if (threadIdx.x == 0) p.njobs = base;
  }
  __syncthreads();
}

// The routes of a job in route order into list[0 .. BR) (wave-private LDS); returns how many.
template <int BR>
__device__ __forceinline__ int job_rows(const Plan& p, int job, int R, int* list) {
  const int e = job & 0xffff, lo = (job >> 16) * BR;
  int seen = 0;
  for (int c = 0; c < R; c += kWave) {
    const int i = c + lane_id();
    const bool hit = i < R && p.id[i] == e;
    const uint64_t m = __ballot(hit);
    const int rank = seen + __popcll(m & lanemask_lt()) - lo;
    if (hit && rank >= 0 && rank < BR) list[rank] = i;
    seen += __popcll(m);
    if (seen >= lo + BR) break;
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  return min(uniform(seen) - lo, BR);
}

// ---------------------------------------------------------------- stream --
// One wave's ring: blocks of NCB x 16 weight columns and BR rows, kAhead = S - 1 blocks in flight.
template <int F, bool PACKED, int NCB, int BR, int RING>
struct Stream {
  using T = Fmt<F>;
  static constexpr int XP = (BR + T::kRowsPerPiece - 1) / T::kRowsPerPiece;
  static constexpr int kWBytes = NCB * T::kPieces * 1024, kXBytes = XP * 1024;
  static constexpr int kSlot = kWBytes + kXBytes + (T::kScaled ? 256 : 0);
  static constexpr int kCopies = NCB * T::kPieces + XP + T::kScaled;
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
  uint32_t xvoff[XP], svoff, sstep;
  int pkb, pend, pslot;
  int cslot;

  __device__ __forceinline__ Stream(const DecodeSide& s, const uint8_t* rows, uint8_t* mem) : side(s), x(rows), ring(mem) {
    lane = lane_id();
    l16 = lane & 15;
    lg = lane >> 4;
    lds0 = (uint32_t)uniform((int)lds_offset(mem));
    const uint32_t rowb = F == kInt4 ? side.K / 2 : F == kFp8 ? side.K : 2 * side.K;
#pragma unroll
    for (int p = 0; p < T::kPieces; ++p) {
      if (PACKED) {
        wvoff[p] = 1024 * p + 16 * lane;
      } else if (F == kInt4) {
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
  // rows list[0 .. m) >> shift of x.
  __device__ __forceinline__ void produce(int e, int col0, int col1, int kb0, int kb1, const int* list, int m, bool tokens,
                                          int k) {
    const int64_t rowb = F == kInt4 ? side.K / 2 : F == kFp8 ? side.K : 2 * side.K;
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
      int r = list[min(row, m - 1)];
      if (tokens) r /= k;
      xvoff[q] = (uint32_t)r * (uint32_t)side.K * 2u + 16u * (c ^ sw) + (uint32_t)kb0 * T::kXRow;
    }
    if constexpr (F == kFp8) {  // lane: the scale of column block lane % NCB
      const int cb = lane % NCB, KB = side.K / 128;
      const int n = NCB == 1 ? col0 : cb < NCB / 2 ? col0 + 16 * cb : col1 + 16 * (cb - NCB / 2);
      sbase = side.S + (int64_t)e * (side.N / 128) * KB * 4;
      svoff = (uint32_t)((n / 128) * KB + kb0) * 4u;
      sstep = 4;
    } else if constexpr (F == kInt4) {  // lane: that of column l16 of column block lg % NCB, and its neighbour in the dword
      const int cb = lg % NCB, KG = side.K / 128;
      const int n = (NCB == 1 ? col0 : cb < NCB / 2 ? col0 + 16 * cb : col1 + 16 * (cb - NCB / 2)) + l16;
      sbase = side.S + (int64_t)e * side.N * KG * 2;
      svoff = 2u * (uint32_t)(PACKED ? (kb0 * (side.N / 64) + n / 64) * 64 + (n & 15) * 4 + (n & 63) / 16 : n * KG + kb0);
      sstep = PACKED ? 2u * side.N : 2u;
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
    if constexpr (T::kScaled) {
      copy4(svoff & ~3u, sbase, (uint32_t)uniform((int)(to + kWBytes + kXBytes)));
      svoff += sstep;
    }
    pslot = pslot + 1 == S ? 0 : pslot + 1;
    ++pkb;
  }

  // Multiply the oldest block into acc.  kb and col0/col1 are the consumer's (4-bit scales lie in either half of a dword).
  __device__ __forceinline__ void consume(v4f (&acc)[NCB], int kb, int col0, int col1) {
    const uint8_t* w = ring + cslot * kSlot;
    const uint8_t* xs = w + kWBytes;
    const uint8_t* sc = xs + kXBytes;
    const int row = l16 & (BR - 1);  // the rows past BR repeat; nobody reads their sums
    if constexpr (F == kBf16) {
      const int fx = (row >> 1) & 7, fw = (l16 >> 1) & 7;
      v4i xf[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) xf[h] = *(const v4i*)(xs + row * 128 + 16 * ((4 * h + lg) ^ fx));
#pragma unroll
      for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4i wf = *(const v4i*)(w + cb * 2048 + (PACKED ? 1024 * h + 16 * lane : l16 * 128 + 16 * ((4 * h + lg) ^ fw)));
          acc[cb] = mma(xf[h], __builtin_bit_cast(v8bf, wf), acc[cb]);
        }
    } else if constexpr (F == kFp8) {
      const int fw = (l16 >> 1) & 7;
      v4i xf[4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) xf[2 * h + i] = *(const v4i*)(xs + row * 256 + 16 * ((8 * h + 2 * lg + i) ^ row));
#pragma unroll
      for (int cb = 0; cb < NCB; ++cb) {
        v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4i wf = *(const v4i*)(w + cb * 2048 + (PACKED ? 1024 * h + 16 * lane : l16 * 128 + 16 * ((4 * h + lg) ^ fw)));
          s = mma(xf[2 * h], widen_fp8(wf[0], wf[1]), s);
          s = mma(xf[2 * h + 1], widen_fp8(wf[2], wf[3]), s);
        }
        const float f = *(const float*)(sc + 4 * cb);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[cb][i] = __builtin_fmaf(f, s[i], acc[cb][i]);
      }
    } else {
      v4i xf[4];
      const v8bf m136 = {(__bf16)-136.f, (__bf16)-136.f, (__bf16)-136.f, (__bf16)-136.f,
                         (__bf16)-136.f, (__bf16)-136.f, (__bf16)-136.f, (__bf16)-136.f};
      v4f fix = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        xf[d] = *(const v4i*)(xs + row * 256 + 16 * ((PACKED ? 4 * d + lg : 4 * lg + d) ^ row));
        if (!PACKED) xf[d] = nibble_order(xf[d]);
        fix = mma(xf[d], m136, fix);
      }
#pragma unroll
      for (int cb = 0; cb < NCB; ++cb) {
        const v4i wf = *(const v4i*)(w + cb * 1024 + (PACKED ? 16 * lane : l16 * 64 + 16 * (lg ^ (l16 >> 2))));
        v4f s = fix;
#pragma unroll
        for (int d = 0; d < 4; ++d) s = mma(xf[d], widen_int4((uint32_t)wf[d]), s);
        const int n = (NCB == 1 ? col0 : cb < NCB / 2 ? col0 + 16 * cb : col1 + 16 * (cb - NCB / 2)) + l16;
        const int half = PACKED ? ((n & 63) / 16) & 1 : (n * (side.K / 128) + kb) & 1;
        const uint32_t two = *(const uint32_t*)(sc + 4 * (16 * cb + l16));
        const float f = (float)__builtin_bit_cast(_Float16, (uint16_t)(half ? two >> 16 : two));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[cb][i] = __builtin_fmaf(f, s[i], acc[cb][i]);
      }
    }
    cslot = cslot + 1 == S ? 0 : cslot + 1;
  }

  // Wait for the oldest block; `full`: S - 1 blocks were issued after it.
  __device__ __forceinline__ void arrive(bool full) {
    if (full) wait_vmcnt<(S - 1) * kCopies>();
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");
  }
};

// -------------------------------------------------------------------- up --
constexpr int kUpRing = 17 * 1024;

template <int F, bool PACKED, int BR>
__global__ __launch_bounds__(kUpWaves * 64) void decode_up_kernel(const DecodeArgs a) {
  constexpr int NCB = F == kInt4 ? 4 : 2, kCols = 8 * NCB;  // columns of h per unit
  using St = Stream<F, PACKED, NCB, BR, kUpRing>;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kUpWaves * kUpRing];
  __shared__ float part[2][kUpWaves][BR][16 * NCB + 4];
  __shared__ Plan p;
  __shared__ int lists[kUpWaves][2][16];
  static_assert(sizeof(ring) >= 2 * kMaxExperts * sizeof(int), "the plan's tables lie in the rings");
  const int R = a.T * a.k;
  plan<BR>(p, (int*)ring, (int*)ring + kMaxExperts, a.ids, R, a.E, blockIdx.x == 0 ? a.status : nullptr);
  const int wv = uniform(threadIdx.x >> 6);
  const DecodeSide side{(const uint8_t*)a.W13, (const uint8_t*)a.S13, 2 * a.I, a.H};
  St st(side, (const uint8_t*)a.x, ring + wv * kUpRing);
  const int ncol = a.I / kCols, units = p.njobs * ncol;
  const int nb = a.H / Fmt<F>::BK, kb0 = wv * nb / kUpWaves, kb1 = (wv + 1) * nb / kUpWaves;
  int *plist = lists[wv][0], *clist = lists[wv][1];

  int pu = blockIdx.x;  // the producer's unit
  auto feed = [&]() {   // one block into the ring, if there is one
    if (st.pkb == st.pend) {
      if (pu >= units || kb0 == kb1) return false;
      const int job = uniform(p.job[pu / ncol]), col = pu % ncol * kCols;
      const int m = job_rows<BR>(p, job, R, plist);
      st.produce(job & 0xffff, col, a.I + col, kb0, kb1, plist, m, true, a.k);
      pu += gridDim.x;
    }
    st.issue();
    return true;
  };
#pragma unroll 1
  for (int i = 0; i < St::S - 1; ++i) feed();
  int buf = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x, buf ^= 1) {
    const int job = uniform(p.job[u / ncol]), col = u % ncol * kCols;
    v4f acc[NCB];
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) acc[cb] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int kb = kb0; kb < kb1; ++kb) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot that is filled next has been read
      st.arrive(feed());
      st.consume(acc, kb, col, a.I + col);
    }
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * st.lg + i < BR) part[buf][wv][4 * st.lg + i][16 * cb + st.l16] = acc[cb][i];
    const int m = job_rows<BR>(p, job, R, clist);
    barrier_lds();  // one per unit: the other buffer is written before its readers' next barrier
    for (int q = threadIdx.x; q < BR * kCols; q += kUpWaves * 64) {
      const int row = q / kCols, c = q % kCols;
      if (row < m) {
        float g = 0.f, up = 0.f;
#pragma unroll
        for (int v = 0; v < kUpWaves; ++v) {
          g += part[buf][v][row][c];
          up += part[buf][v][row][kCols + c];
        }
        a.h[(int64_t)clist[row] * a.I + col + c] = (uint16_t)f32_to_bf16_rne(g * sigmoid_f32(g) * up);
      }
    }
  }
}

// ------------------------------------------------------------------ down --
constexpr int kDownRing = 13 * 1024;
constexpr int kLdsMost = 150 * 1024;  // beside the plan
static_assert(4 * kDownRing + 64 * kRoutes <= kLdsMost, "any number of routes fits four waves' rings");

// LDS: NW rings, then a line of 16 sums per share of K and route.
template <int F, bool PACKED, int BR, int NW>
__global__ __launch_bounds__(NW * 64) void decode_down_kernel(const DecodeArgs a) {
  using St = Stream<F, PACKED, 1, BR, kDownRing>;
  extern __shared__ __attribute__((aligned(1024))) uint8_t dyn[];
  __shared__ Plan p;
  __shared__ int lists[NW][2][16];
  static_assert(NW * kDownRing >= 2 * kMaxExperts * (int)sizeof(int), "the plan's tables lie in the rings");
  float* y = (float*)(dyn + NW * kDownRing);
  const int R = a.T * a.k, KS = a.ksplit;
  plan<BR>(p, (int*)dyn, (int*)dyn + kMaxExperts, a.ids, R, a.E, nullptr);
  const int wv = uniform(threadIdx.x >> 6);
  const DecodeSide side{(const uint8_t*)a.W2, (const uint8_t*)a.S2, a.H, a.I};
  St st(side, (const uint8_t*)a.h, dyn + wv * kDownRing);
  const int n0 = blockIdx.x * 16, items = p.njobs * KS, nb = a.I / Fmt<F>::BK;
  int *plist = lists[wv][0], *clist = lists[wv][1];

  int pi = wv;
  auto feed = [&]() {
    if (st.pkb == st.pend) {
      if (pi >= items) return false;
      const int job = uniform(p.job[pi / KS]), ks = pi % KS;
      const int m = job_rows<BR>(p, job, R, plist);
      st.produce(job & 0xffff, n0, n0, ks * nb / KS, (ks + 1) * nb / KS, plist, m, false, 1);
      pi += NW;
    }
    st.issue();
    return true;
  };
#pragma unroll 1
  for (int i = 0; i < St::S - 1; ++i) feed();
  for (int it = wv; it < items; it += NW) {
    const int job = uniform(p.job[it / KS]), ks = it % KS;
    v4f acc[1] = {v4f{0.f, 0.f, 0.f, 0.f}};
    const int kb1 = (ks + 1) * nb / KS;
#pragma unroll 1
    for (int kb = ks * nb / KS; kb < kb1; ++kb) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      st.arrive(feed());
      st.consume(acc, kb, n0, n0);
    }
    const int m = job_rows<BR>(p, job, R, clist);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * st.lg + i < m) y[(ks * R + clist[4 * st.lg + i]) * 16 + st.l16] = acc[0][i];
  }
  __syncthreads();
  for (int q = threadIdx.x; q < a.T * 16; q += NW * 64) {
    const int t = q >> 4, c = q & 15;
    const int64_t at = (int64_t)t * a.H + n0 + c;
    float z = 0.f;
    for (int r = 0; r < a.k; ++r) {
      const int i = t * a.k + r;
      if (p.id[i] < 0) continue;
      float v = y[i * 16 + c];
      for (int s = 1; s < KS; ++s) v += y[(s * R + i) * 16 + c];
      z = __builtin_fmaf(a.p[i], v, z);
    }
    if (a.C) z += bf16_to_f32(a.C[at]);
    a.Z[at] = (uint16_t)f32_to_bf16_rne(z);
  }
}

template <int F, bool PACKED, int BR, int NW>
hipError_t launch_down(const DecodeArgs& a, hipStream_t s) {
  const size_t lds = NW * kDownRing + (size_t)a.ksplit * a.T * a.k * 64;
  // more than 64 KB of LDS asked for at the launch
  const hipError_t e = hipFuncSetAttribute((const void*)decode_down_kernel<F, PACKED, BR, NW>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLdsMost);
  if (e != hipSuccess) return e;
  decode_down_kernel<F, PACKED, BR, NW><<<a.H / 16, NW * 64, lds, s>>>(a);
  return hipGetLastError();
}

template <int F, bool PACKED, int BR>
hipError_t launch_rows(DecodeArgs a, hipStream_t s) {
  const int R = a.T * a.k, nb = a.I / Fmt<F>::BK;
  const int64_t units = (int64_t)R * (a.I / (F == kInt4 ? 32 : 16));
  const int64_t cap = 2 * device_info().cus;
  decode_up_kernel<F, PACKED, BR><<<(unsigned)(units < cap ? units : cap), kUpWaves * 64, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // few routes: their K is shared so that every wave has a part
  const bool wide = a.H / 16 <= 256 && 8 * kDownRing + 64 * R <= kLdsMost;
  const int nw = wide ? 8 : 4;
  a.ksplit = 1;
  while (a.ksplit * R < nw && 2 * a.ksplit <= nb) a.ksplit *= 2;
  return wide ? launch_down<F, PACKED, BR, 8>(a, s) : launch_down<F, PACKED, BR, 4>(a, s);
}

template <int F, bool PACKED>
hipError_t launch_format(const DecodeArgs& a, hipStream_t s) {
  // rows of a job: what most experts get, so that their weights are read once
  const float mean = (float)a.T * (float)a.k / (float)a.E;
  const int most = a.T;
  if constexpr (F != kBf16)
    if (mean <= 2.0f || most <= 4) return launch_rows<F, PACKED, 4>(a, s);
  if (mean <= 5.0f || most <= 8) return launch_rows<F, PACKED, 8>(a, s);
  return launch_rows<F, PACKED, 16>(a, s);
}

}  // namespace

int64_t decode_workspace_bytes(int T, int k, int I) { return (int64_t)T * k * I * 2; }

hipError_t launch_experts_decode(const DecodeArgs& a, hipStream_t s) {
  switch (a.format) {
    case kBf16: return a.packed ? launch_format<kBf16, true>(a, s) : launch_format<kBf16, false>(a, s);
    case kFp8: return a.packed ? launch_format<kFp8, true>(a, s) : launch_format<kFp8, false>(a, s);
    default: return a.packed ? launch_format<kInt4, true>(a, s) : launch_format<kInt4, false>(a, s);
  }
}

}  // namespace moe
