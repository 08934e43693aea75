// act_bwd.hip -- moe_act_bwd: the gradient of moe_gemm_bf16's bias and activation.
//
//   dP[m, n] = dD[m, n] * act'(pre[m, n])
//   gated:     dP[m, j] = dD[m, j] * up * act'(gate),   dP[m, N/2 + j] = dD[m, j] * act(gate)
//   dbias[n] (+)= sum_m dP[m, n], of the fp32 values before dP's rounding
//
// One pass: 8 columns per lane (16-byte loads and stores), kRowsAhead rows' loads in flight per lane; the column sums stay in
// registers, meet across lanes and waves in a fixed order, and where the rows are cut into several chunks one line of sums per
// chunk goes to the workspace, where a second launch adds the lines.  A launch costs more than a few hundred rows do, so up to
// kOneChunk rows are one chunk: narrow strips, 16 waves each, no second launch.  333 x 1536 GELU 5.9 us in a graph out of the
// caches, 7.3 out of HBM (two launches of chunks took 14); 4096 x 2 * 2048 SwiGLU 22 us with the bias, 19 without (84 MB: 4.4 TB/s);
// 16384 rows 63 us, 5.3 TB/s.
#include "linear_act.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kOneChunk = 1024;   // rows
constexpr int kRowsAhead = 4;
constexpr int kJoinCols = 64, kJoinParts = 16;

struct Eight {
  float v[8];
};
__device__ __forceinline__ Eight unpack8(const v4i w) {
  Eight r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = bf16_to_f32((uint32_t)w[i] & 0xffffu);
    r.v[2 * i + 1] = bf16_to_f32((uint32_t)w[i] >> 16);
  }
  return r;
}
__device__ __forceinline__ v4i pack8(const Eight& e) {
  v4i w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (int)bf16_pair(e.v[2 * i], e.v[2 * i + 1]);
  return w;
}

// Columns at .. at + 7 of a row, of which cnt are there (rows begin at any element: global memory takes vectors at any address).
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ v4i load8(const uint16_t* p, int cnt) {
  if (cnt == 8) return *(const v4i_any*)p;
  v4i w = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < cnt) w[i >> 1] |= (int)((uint32_t)p[i] << 16 * (i & 1));
  return w;
}
__device__ __forceinline__ void store8(uint16_t* p, int cnt, const v4i w) {
  if (cnt == 8) {
    *(v4i_any*)p = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < cnt) p[i] = (uint16_t)((uint32_t)w[i >> 1] >> 16 * (i & 1));
}

// LPR lanes per row: a workgroup of TPB threads owns 8 LPR columns (of each half, if gated) and the rows of chunk blockIdx.y.
template <int ACT, bool GATED, int LPR, int TPB>
__global__ __launch_bounds__(TPB) void act_bwd_kernel(const ActBwdArgs a) {
  constexpr int kCols = 8 * LPR, kWaves = TPB / 64, kRows = TPB / LPR, H = GATED ? 2 : 1;
  __shared__ float part[kWaves][H][kCols];
  const int lr = threadIdx.x % LPR, wv = threadIdx.x >> 6;
  const int half = GATED ? a.N / 2 : a.N, n = blockIdx.x * kCols + 8 * lr;
  const int r0 = blockIdx.y * a.rows, r1 = min(r0 + a.rows, a.M);
  float s[H][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int h = 0; h < H; ++h) s[h][i] = 0.f;
  const int cnt = min(8, half - n);
  if (cnt > 0) {
    for (int m0 = r0 + threadIdx.x / LPR; m0 < r1; m0 += kRowsAhead * kRows) {
      v4i d[kRowsAhead], g[kRowsAhead], u[kRowsAhead];
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j) {
        const int64_t m = min(m0 + j * kRows, r1 - 1);
        d[j] = load8(a.dD + m * a.ldd + n, cnt);
        if (GATED || ACT != kActNone) g[j] = load8(a.pre + m * a.ldp + n, cnt);
        if (GATED) u[j] = load8(a.pre + m * a.ldp + half + n, cnt);
      }
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j) {
        const int64_t m = m0 + j * kRows;
        if (m >= r1) break;
        const Eight dv = unpack8(d[j]);
        Eight gv{}, uv{}, o, p;
        if (GATED || ACT != kActNone) gv = unpack8(g[j]);
        if (GATED) uv = unpack8(u[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float slope;
          const float act = act_and_slope(ACT, gv.v[i], slope);
          o.v[i] = dv.v[i] * (GATED ? slope * uv.v[i] : slope);
          s[0][i] += o.v[i];
          if (GATED) {
            p.v[i] = dv.v[i] * act;
            s[H - 1][i] += p.v[i];
          }
        }
        if (a.dP) {
          store8(a.dP + m * a.ldo + n, cnt, pack8(o));
          if (GATED) store8(a.dP + m * a.ldo + half + n, cnt, pack8(p));
        }
      }
    }
  }
  if (!a.dbias) return;
#pragma unroll
  for (int h = 0; h < H; ++h) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int x = LPR; x < 64; x <<= 1) s[h][i] += __shfl_xor(s[h][i], x);
      if ((threadIdx.x & 63) < LPR) part[wv][h][8 * lr + i] = s[h][i];
    }
  }
  __syncthreads();
  for (int q = threadIdx.x; q < H * kCols; q += TPB) {
    const int h = q / kCols, c = q % kCols, col = blockIdx.x * kCols + c;
    if (col >= half) continue;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += part[w][h][c];
    const int at = h * half + col;
    if (gridDim.y > 1) a.ws[(int64_t)blockIdx.y * a.N + at] = sum;
    else a.dbias[at] = a.accumulate ? a.dbias[at] + sum : sum;
  }
}

// dbias from the chunks' lines: kJoinParts threads per column take the lines in turn, then meet in order.
__global__ __launch_bounds__(kJoinCols* kJoinParts) void act_bwd_join_kernel(const ActBwdArgs a, int lines) {
  __shared__ float part[kJoinParts][kJoinCols];
  const int c = threadIdx.x % kJoinCols, p = threadIdx.x / kJoinCols, n = blockIdx.x * kJoinCols + c;
  float s = 0.f;
  if (n < a.N) {
#pragma unroll 4
    for (int i = p; i < lines; i += kJoinParts) s += a.ws[(int64_t)i * a.N + n];
  }
  part[p][c] = s;
  __syncthreads();
  if (p || n >= a.N) return;
#pragma unroll
  for (int i = 1; i < kJoinParts; ++i) s += part[i][c];
  a.dbias[n] = a.accumulate ? a.dbias[n] + s : s;
}

// Row chunks: one up to kOneChunk rows; else chunks that give the chip two workgroups per compute unit, of 32 rows at least.
// (By the columns of dP, so that gated calls have half as many workgroups.)
int chunks(int M, int N) {
  if (M <= kOneChunk) return 1;
  const int strips = (N + 511) / 512, c = (1024 + strips - 1) / strips, most = (M + 31) / 32;
  return c < most ? c : most;
}

template <int ACT, bool GATED>
hipError_t launch_gated(ActBwdArgs a, hipStream_t s) {
  const int half = GATED ? a.N / 2 : a.N, c = chunks(a.M, a.N);
  a.rows = a.M > c ? (a.M + c - 1) / c : 1;
  if (c == 1) {
    act_bwd_kernel<ACT, GATED, 4, 1024><<<(half + 31) / 32, 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  const int lines = (a.M + a.rows - 1) / a.rows;
  act_bwd_kernel<ACT, GATED, 64, 256><<<dim3((half + 511) / 512, lines), 256, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dbias) return e;
  act_bwd_join_kernel<<<(a.N + kJoinCols - 1) / kJoinCols, kJoinCols * kJoinParts, 0, s>>>(a, lines);
  return hipGetLastError();
}
template <int ACT>
hipError_t launch_act(const ActBwdArgs& a, hipStream_t s) {
  return a.gated ? launch_gated<ACT, true>(a, s) : launch_gated<ACT, false>(a, s);
}

}  // namespace

int64_t act_bwd_workspace_bytes(int M, int N) {
  const int c = chunks(M, N);
  return c > 1 ? 4ll * c * N : 0;
}

hipError_t launch_act_bwd(const ActBwdArgs& a, hipStream_t s) {
  switch (a.act) {
    case kActRelu: return launch_act<kActRelu>(a, s);
    case kActSilu: return launch_act<kActSilu>(a, s);
    case kActGelu: return launch_act<kActGelu>(a, s);
    case kActGeluTanh: return launch_act<kActGeluTanh>(a, s);
    default: return launch_act<kActNone>(a, s);
  }
}

}  // namespace moe
