// act_bwd.hip -- moe_act_bwd: the gradient of moe_gemm_bf16's bias and activation.
//
//   dP[m, n] = dD[m, n] * act'(pre[m, n])
//   gated:     dP[m, j] = dD[m, j] * up * act'(gate),   dP[m, N/2 + j] = dD[m, j] * act(gate)
//   dbias[n] (+)= sum_m dP[m, n], of the fp32 values before dP's rounding
//
// One pass: 8 columns per lane (16-byte loads and stores), rows in turn; a workgroup's column sums stay in registers, meet in
// LDS, and one line per workgroup goes to the workspace, where a second launch adds the lines in order.
#include "linear_act.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kStrip = 512;  // columns of a workgroup: 64 lanes x 8

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
  for (int i = 0; i < 4; ++i) w[i] = (int)(f32_to_bf16_rne(e.v[2 * i]) | (f32_to_bf16_rne(e.v[2 * i + 1]) << 16));
  return w;
}

template <int ACT, bool GATED>
__global__ __launch_bounds__(256) void act_bwd_kernel(const ActBwdArgs a) {
  __shared__ float part[4][GATED ? 2 : 1][kStrip];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int half = GATED ? a.N / 2 : a.N, n = blockIdx.x * kStrip + 8 * lane;
  const int r0 = blockIdx.y * a.rows, r1 = min(r0 + a.rows, a.M);
  float s0[8], s1[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s0[i] = s1[i] = 0.f;
  if (n < half) {
    for (int m = r0 + wv; m < r1; m += 4) {
      const Eight d = unpack8(*(const v4i*)(a.dD + (int64_t)m * a.ldd + n));
      Eight g{}, u{}, o, p;
      if (GATED || ACT != kActNone) g = unpack8(*(const v4i*)(a.pre + (int64_t)m * a.ldp + n));
      if (GATED) u = unpack8(*(const v4i*)(a.pre + (int64_t)m * a.ldp + half + n));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o.v[i] = d.v[i] * slope1(ACT, g.v[i]);
        if (GATED) {
          o.v[i] *= u.v[i];
          p.v[i] = d.v[i] * act1(ACT, g.v[i]);
          s1[i] += p.v[i];
        }
        s0[i] += o.v[i];
      }
      if (a.dP) {
        *(v4i*)(a.dP + (int64_t)m * a.ldo + n) = pack8(o);
        if (GATED) *(v4i*)(a.dP + (int64_t)m * a.ldo + half + n) = pack8(p);
      }
    }
  }
  if (!a.dbias) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    part[wv][0][8 * lane + i] = s0[i];
    if (GATED) part[wv][GATED ? 1 : 0][8 * lane + i] = s1[i];
  }
  __syncthreads();
  for (int q = threadIdx.x; q < (GATED ? 2 : 1) * kStrip; q += 256) {
    const int which = q / kStrip, c = q % kStrip, col = blockIdx.x * kStrip + c;
    if (col >= half) continue;
    const float s = (part[0][which][c] + part[1][which][c]) + (part[2][which][c] + part[3][which][c]);
    const int at = which * half + col;
    if (gridDim.y > 1) a.ws[(int64_t)blockIdx.y * a.N + at] = s;
    else a.dbias[at] = a.accumulate ? a.dbias[at] + s : s;
  }
}

// dbias from the workgroups' lines, in order.
__global__ __launch_bounds__(256) void act_bwd_join_kernel(const ActBwdArgs a, int lines) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= a.N) return;
  float s = 0.f;
  for (int i = 0; i < lines; ++i) s += a.ws[(int64_t)i * a.N + n];
  a.dbias[n] = a.accumulate ? a.dbias[n] + s : s;
}

// Row chunks: enough workgroups for the chip, at least 16 rows each.
int chunks(int M, int N) {
  const int strips = (N + kStrip - 1) / kStrip;
  int c = (2048 + strips - 1) / strips;
  const int most = M > 16 ? (M + 15) / 16 : 1;
  return c < most ? c : most;
}

template <int ACT>
hipError_t launch_act(ActBwdArgs a, hipStream_t s) {
  const int half = a.gated ? a.N / 2 : a.N;
  const int c = chunks(a.M, a.N);
  a.rows = a.M > c ? (a.M + c - 1) / c : 1;
  const int lines = a.M > a.rows ? (a.M + a.rows - 1) / a.rows : 1;
  const dim3 grid((half + kStrip - 1) / kStrip, lines);
  if (a.gated) act_bwd_kernel<ACT, true><<<grid, 256, 0, s>>>(a);
  else act_bwd_kernel<ACT, false><<<grid, 256, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dbias || lines == 1) return e;
  act_bwd_join_kernel<<<(a.N + 255) / 256, 256, 0, s>>>(a, lines);
  return hipGetLastError();
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
