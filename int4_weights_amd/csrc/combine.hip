// combine.hip -- moe_unpermute_combine: z[t] = sum_r p[t,r] * y[output_index[t,r]].
// (rainlin, "GEMM 执行方式", sec. 4.4 and 4.6: the gather reads only the packed
// rows named by output_index and weights them by topk_weights; CuTeDSL bei
// Perplexity: the combine accumulates in registers with vectorised loads.)
//
// One thread per (token, 8 columns): 16-byte loads of each routed row, fp32
// fma in slot order r = 0..k-1, one 16-byte bf16 store.  HBM-bound: every
// routed row is read once and every output row written once, so both go
// nontemporal (streamed past the caches; about 13% faster on the Qwen3-shaped
// combine than cached accesses).
//
// moe_unpermute_combine_bwd: its gradient, dY[output_index[t,r]] = p[t,r] * dZ[t]
// and dp[t,r] = <dZ[t], Y[output_index[t,r]]>.
// One workgroup per token and batch of slots: the token's dZ row is read once per
// batch, every named row of Y is streamed once and its gradient row written
// once (nontemporal).  HBM-bound: 8192 x 8 slots x 4096 232 us, 4.92 TB/s, of which 10 us are the table's two kernels
// (clear, claim); 61 x 8 x 7168 6.9 us, two trips to memory and the launch.
// A row is normally named by one slot (moe_route_pack gives every route a row
// of its own).  A row named by several slots gets the sum over them in route
// order: its lowest slot writes it, in fp32 until the one rounding.  Who names a row is
// found by a scan of output_index in each workgroup (up to 4096 routes, no
// workspace), or beforehand with one integer count and minimum per row in the
// workspace (order-free, so results do not depend on timing).
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* __restrict__ Y, int64_t y_rows,
                                                      const int32_t* __restrict__ oi, const float* __restrict__ w,
                                                      int T, int k, int N, uint16_t* __restrict__ Z) {
  const int chunks = N / 8;
  const int64_t total = (int64_t)T * chunks;
  for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < total;
       idx += (int64_t)gridDim.x * blockDim.x) {
    const int t = (int)(idx / chunks), c = (int)(idx - (int64_t)t * chunks);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    // slots in batches of 8: every index, then every row load, then the sums
    // in slot order (two memory round trips per batch instead of two per slot)
    for (int r0 = 0; r0 < k; r0 += 8) {
      int p[8];
      float wt[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = r0 + j < k ? oi[(int64_t)t * k + r0 + j] : -1;
        wt[j] = r0 + j < k ? w[(int64_t)t * k + r0 + j] : 0.0f;
      }
      v4i y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        y[j] = (p[j] >= 0 && p[j] < y_rows) ? __builtin_nontemporal_load((const v4i*)(Y + (int64_t)p[j] * N + 8 * c))
                                            : v4i{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (p[j] < 0 || p[j] >= y_rows) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = (uint32_t)y[j][i];
          acc[2 * i] = __builtin_fmaf(wt[j], bf16_to_f32(u & 0xffffu), acc[2 * i]);
          acc[2 * i + 1] = __builtin_fmaf(wt[j], bf16_to_f32(u >> 16), acc[2 * i + 1]);
        }
      }
    }
    v4i o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (int)(f32_to_bf16_rne(acc[2 * i]) | (f32_to_bf16_rne(acc[2 * i + 1]) << 16));
    __builtin_nontemporal_store(o, (v4i*)(Z + (int64_t)t * N + 8 * c));
  }
}

hipError_t launch_combine(const uint16_t* Y, int64_t y_rows, const int32_t* oi, const float* w, int T, int k,
                          int N, uint16_t* Z, hipStream_t s) {
  const int64_t total = (int64_t)T * (N / 8);
  if (total == 0) return hipSuccess;
  int64_t grid = (total + 255) / 256;
  const int64_t cap = (int64_t)device_info().cus * 32;
  if (grid > cap) grid = cap;
  combine_kernel<<<(unsigned)grid, 256, 0, s>>>(Y, y_rows, oi, w, T, k, N, Z);
  return hipGetLastError();
}

// ------------------------------------------------------------- backward --
// workspace of the large path: per row of Y the number of slots naming it and the lowest of them
__global__ __launch_bounds__(256) void combine_bwd_clear_kernel(int2* __restrict__ who, int64_t y_rows) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < y_rows; i += (int64_t)gridDim.x * 256)
    who[i] = int2{0, 0x7fffffff};
}
__global__ __launch_bounds__(256) void combine_bwd_claim_kernel(const int32_t* __restrict__ oi, int64_t R,
                                                                int64_t y_rows, int2* __restrict__ who) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < R; i += (int64_t)gridDim.x * 256) {
    const int p = oi[i];
    if (p >= 0 && p < y_rows) {
      atomicAdd(&who[p].x, 1);
      atomicMin(&who[p].y, (int)i);
    }
  }
}

__device__ __forceinline__ void unpack8(const v4i r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32((uint32_t)r[i] & 0xffffu);
    f[2 * i + 1] = bf16_to_f32((uint32_t)r[i] >> 16);
  }
}
__device__ __forceinline__ v4i pack8(const float (&f)[8]) {
  v4i o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (int)(f32_to_bf16_rne(f[2 * i]) | (f32_to_bf16_rne(f[2 * i + 1]) << 16));
  return o;
}

// dY of a row named by `cnt` slots, the lowest of them `own`: the whole workgroup sums them in route order, searching
// the table NT entries at a time (a thread searching alone would take R / 2 dependent loads for a row named twice).
template <int NT>
__device__ __forceinline__ void shared_row(const CombineBwdArgs& a, int p, int own, int cnt) {
  __shared__ uint64_t s_hit[NT / 64];
  const int64_t R = (int64_t)a.T * a.k;
  const int chunks = a.N / 8;
  for (int c0 = 0; c0 < chunks; c0 += NT) {
    const int c = c0 + (int)threadIdx.x;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    int left = cnt;
    for (int64_t i0 = own; i0 < R && left > 0; i0 += NT) {
      const bool hit = i0 + threadIdx.x < R && a.oi[i0 + threadIdx.x] == p;
      const uint64_t m = __ballot(hit);
      __syncthreads();  // the previous entries' hits are used up
      if ((threadIdx.x & 63) == 0) s_hit[threadIdx.x >> 6] = m;
      __syncthreads();
      for (int v = 0; v < NT / 64; ++v)
        for (uint64_t h = s_hit[v]; h; h &= h - 1) {
          const int64_t i = i0 + 64 * v + __builtin_ctzll(h);
          --left;
          if (c >= chunks) continue;
          float dz[8];
          unpack8(*(const v4i*)(a.dZ + i / a.k * a.N + 8 * c), dz);
          const float w = a.w[i];
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = __builtin_fmaf(w, dz[j], acc[j]);
        }
    }
    if (c < chunks) *(v4i*)(a.dY + (int64_t)p * a.N + 8 * c) = pack8(acc);
  }
}

// NT threads per B slots of a token.  Pairs of slots while the chip holds all of them at once: 1024 threads each (a row of
// up to 8192 columns in flight) where every one has a compute unit, 512 where four share one; beyond that 256 threads and 4
// slots, or 8 where a second batch of 4 would hold one or two.  us, k x N, 1024 and 2, 512 and 2, 256 and 4, 256 and 8:
// 61 x 8 x 7168 7.4, 7.8, 14.1, 22.7; 128 x 8 x 4096 10.4, 8.1, 10.9, 17.2; 451 x 8 x 4096 34.8, 22.8, 18.4, 23.2;
// 4096 x 8 x 4096 257, 164, 122, 128; 4096 x 5 x 6560 228, 160, 152, 135; 2166 x 2 x 1312 34.7, 23.3, 20.5, 29.0.
template <int NT, int B>
__global__ __launch_bounds__(NT) void combine_bwd_kernel(const CombineBwdArgs a) {
  constexpr int kScan = (kRouteSmallMax + NT - 1) / NT;
  __shared__ int s_cnt[B], s_own[B];
  __shared__ float s_sum[NT / 64][B];
  const int tid = threadIdx.x, lane = lane_id(), wv = tid >> 6;
  const int chunks = a.N / 8;
  const int R = a.T * a.k;
  const bool scan = a.dY && !a.who;
  const int batches = (a.k + B - 1) / B;
  const int64_t total = (int64_t)a.T * batches;
  for (int64_t q = blockIdx.x; q < total; q += gridDim.x) {  // uniform in the workgroup, as all that decides shared_row is
    const int t = (int)(q / batches), r0 = (int)(q % batches) * B, i0 = t * a.k + r0;
    int p[B];
    float w[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      p[j] = r0 + j < a.k ? a.oi[i0 + j] : -1;
      if (p[j] >= a.y_rows) p[j] = -1;
      w[j] = r0 + j < a.k && a.dY ? a.w[i0 + j] : 0.0f;
    }
    int o[kScan];  // this thread's share of output_index: loaded with the batch's own, compared below
#pragma unroll
    for (int u = 0; u < kScan; ++u) o[u] = scan && tid + NT * u < R ? a.oi[tid + NT * u] : -1;
    bool write[B], shared = false;
#pragma unroll
    for (int j = 0; j < B; ++j) write[j] = a.dY && p[j] >= 0;
    if (a.dY && a.who) {
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (p[j] >= 0 && a.who[p[j]].x != 1) {
          write[j] = false;
          shared = true;
        }
    }
    float dot[B];
#pragma unroll
    for (int j = 0; j < B; ++j) dot[j] = 0.0f;
    v4i dzv = {0, 0, 0, 0}, y[B];
    auto load = [&](int c) {
      dzv = *(const v4i*)(a.dZ + (int64_t)t * a.N + 8 * c);
#pragma unroll
      for (int j = 0; j < B; ++j)
        y[j] = a.dw && p[j] >= 0 ? __builtin_nontemporal_load((const v4i*)(a.Y + (int64_t)p[j] * a.N + 8 * c))
                                 : v4i{0, 0, 0, 0};
    };
    if (tid < chunks) load(tid);
    if (scan) {  // behind the first rows' loads
      if (tid < B) {
        s_cnt[tid] = 0;
        s_own[tid] = 0x7fffffff;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kScan; ++u)
#pragma unroll
        for (int j = 0; j < B; ++j)
          if (o[u] >= 0 && o[u] == p[j]) {
            atomicAdd(&s_cnt[j], 1);
            atomicMin(&s_own[j], tid + NT * u);
          }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (p[j] >= 0 && s_cnt[j] != 1) {
          write[j] = false;
          shared = true;
        }
    }
    for (int c = tid; c < chunks; c += NT) {
      if (c != tid) load(c);
      float dz[8];
      unpack8(dzv, dz);
#pragma unroll
      for (int j = 0; j < B; ++j) {
        float f[8];
        unpack8(y[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[j] = __builtin_fmaf(f[i], dz[i], dot[j]);
      }
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (!write[j]) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[j] * dz[i];
        __builtin_nontemporal_store(pack8(v), (v4i*)(a.dY + (int64_t)p[j] * a.N + 8 * c));
      }
    }
    if (shared) {
      for (int j = 0; j < B; ++j) {
        const int pj = r0 + j < a.k ? a.oi[i0 + j] : -1;
        if (pj < 0 || pj >= a.y_rows) continue;
        const int cnt = a.who ? a.who[pj].x : s_cnt[j];
        const int own = a.who ? a.who[pj].y : s_own[j];
        if (cnt > 1 && own == i0 + j) shared_row<NT>(a, pj, own, cnt);
      }
    }
    if (a.dw) {
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (p[j] < 0) dot[j] = 0.0f;  // a skipped slot's zeros met dZ, which may hold Inf or NaN
#pragma unroll
        for (int off = 32; off; off >>= 1) dot[j] += __shfl_xor(dot[j], off, 64);
        if (lane == 0) s_sum[wv][j] = dot[j];
      }
      __syncthreads();
      if (tid < B && r0 + tid < a.k) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NT / 64; ++v) s += s_sum[v][tid];
        a.dw[i0 + tid] = s;
      }
    }
    __syncthreads();  // s_cnt, s_own and s_sum are reused
  }
}

int64_t combine_bwd_workspace_bytes(int64_t R, int64_t y_rows) { return R <= kRouteSmallMax ? 0 : 8 * y_rows; }

hipError_t launch_combine_bwd(const CombineBwdArgs& a, hipStream_t s) {
  const int64_t cap = (int64_t)device_info().cus * 32;
  if (a.who) {
    const int64_t R = (int64_t)a.T * a.k;
    const int64_t gr = (a.y_rows + 255) / 256, gc = (R + 255) / 256;
    combine_bwd_clear_kernel<<<(unsigned)(gr < cap ? gr : cap), 256, 0, s>>>(a.who, a.y_rows);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    combine_bwd_claim_kernel<<<(unsigned)(gc < cap ? gc : cap), 256, 0, s>>>(a.oi, R, a.y_rows, a.who);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t pairs = (int64_t)a.T * ((a.k + 1) / 2), cus = device_info().cus;
  if (pairs <= cus) {
    combine_bwd_kernel<1024, 2><<<(unsigned)pairs, 1024, 0, s>>>(a);
  } else if (pairs <= 4 * cus) {
    combine_bwd_kernel<512, 2><<<(unsigned)pairs, 512, 0, s>>>(a);
  } else if (a.k % 8 == 5 || a.k % 8 == 6) {
    const int64_t total = (int64_t)a.T * ((a.k + 7) / 8);
    combine_bwd_kernel<256, 8><<<(unsigned)(total < cap ? total : cap), 256, 0, s>>>(a);
  } else {
    const int64_t total = (int64_t)a.T * ((a.k + 3) / 4);
    combine_bwd_kernel<256, 4><<<(unsigned)(total < cap ? total : cap), 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
