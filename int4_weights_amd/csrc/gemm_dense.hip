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
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kTile = 128;

__device__ __forceinline__ v4f mfma_fp8(const v8i w, const v8i x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7f7f7f7f, 0,
                                                          0x7f7f7f7f);
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
__device__ __forceinline__ v4f block_sum(const Frag<false>& w, const Frag<false>& x) { return mfma_fp8(w.v, x.v); }
__device__ __forceinline__ v4f block_sum(const Frag<true>& w, const Frag<true>& x) {
  v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], s, 0, 0, 0);
  return s;
}

// Four consecutive columns n .. n + 3 of row m.
__device__ __forceinline__ void store4(const DenseArgs& a, int m, int n, v4f v) {
  if (m >= a.M) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.N) return;
    float o = v[i];
    if (a.C) o += a.C[(int64_t)m * a.ldc + n + i];
    if (a.f32)
      ((float*)a.D)[(int64_t)m * a.ldd + n + i] = o;
    else
      ((uint16_t*)a.D)[(int64_t)m * a.ldd + n + i] = (uint16_t)f32_to_bf16_rne(o);
  }
}

template <bool WIDE>
__global__ __launch_bounds__(256) void gemm_dense_kernel(const DenseArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t sA[kTile * 128], sW[kTile * 128];
  __shared__ float s_sa[kTile], s_sw[kTile];
  const int tid = threadIdx.x, lane = lane_id(), wv = uniform(tid >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int KB = a.K / 128;
  const int nt = (a.N + kTile - 1) / kTile;
  const int m0 = (int)(blockIdx.x / nt) * kTile, n0 = (int)(blockIdx.x % nt) * kTile;
  const int wm = (wv >> 1) * 64, wn = (wv & 1) * 64;
  v4f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int kb = 0; kb < KB; ++kb) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = tid + 256 * i, r = q >> 3, c = (q & 7) ^ ((r >> 1) & 7);
      *(v4i*)(sA + 16 * q) = *(const v4i*)(a.A + (int64_t)min(m0 + r, a.M - 1) * a.lda + (int64_t)kb * 128 + 16 * c);
      *(v4i*)(sW + 16 * q) = *(const v4i*)(a.W + (int64_t)min(n0 + r, a.N - 1) * a.ldw + (int64_t)kb * 128 + 16 * c);
    }
    if (tid < kTile)
      s_sa[tid] = a.SFA[(int64_t)min(m0 + tid, a.M - 1) * KB + kb];
    else
      s_sw[tid - kTile] = a.SFW[(int64_t)(min(n0 + tid - kTile, a.N - 1) / a.gran_n) * KB + kb];
    __syncthreads();
    Frag<WIDE> xf[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = wm + 16 * i + l16, sw = (r >> 1) & 7;
      const v4i lo = *(const v4i*)(sA + r * 128 + 16 * (lg ^ sw)), hi = *(const v4i*)(sA + r * 128 + 16 * ((4 + lg) ^ sw));
      xf[i].load(lo, hi);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = wn + 16 * j + l16, sw = (r >> 1) & 7;
      const v4i lo = *(const v4i*)(sW + r * 128 + 16 * (lg ^ sw)), hi = *(const v4i*)(sW + r * 128 + 16 * ((4 + lg) ^ sw));
      Frag<WIDE> wf;
      wf.load(lo, hi);
      const v4f sw4 = *(const v4f*)(s_sw + wn + 16 * j + 4 * lg);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v4f p = block_sum(wf, xf[i]);
        const float sa = s_sa[wm + 16 * i + l16];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e], sa * sw4[e], acc[i][j][e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) store4(a, m0 + wm + 16 * i + l16, n0 + wn + 16 * j + 4 * lg, acc[i][j]);
}

}  // namespace

int64_t dense_workspace_bytes(int, int, int) { return 0; }

hipError_t launch_gemm_dense(const DenseArgs& a, hipStream_t s) {
  const int64_t tiles = (int64_t)((a.M + kTile - 1) / kTile) * ((a.N + kTile - 1) / kTile);
  if (a.f32)
    gemm_dense_kernel<true><<<(unsigned)tiles, 256, 0, s>>>(a);
  else
    gemm_dense_kernel<false><<<(unsigned)tiles, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
