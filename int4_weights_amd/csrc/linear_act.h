// linear_act.h -- the activations of moe_gemm_bf16's epilogue and their slopes, in fp32.
#pragma once

#include "moe_device.h"

namespace moe {

enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// Phi(v) = erfc(-v / sqrt 2) / 2: no cancellation for negative v.
__device__ __forceinline__ float normal_cdf(float v) { return 0.5f * erfcf(v * -0.70710678118654752f); }
// 1 / (1 + exp(-2u)), u = sqrt(2/pi) (v + 0.044715 v^3): gelu_tanh(v) = v times it.
__device__ __forceinline__ float gelu_gate(float v) {
  const float u2 = 1.5957691216057308f * v * __builtin_fmaf(0.044715f * v, v, 1.0f);
  return 1.0f / (1.0f + expf(-u2));
}

// silu_f32 for any finite v: its exponent overflows past 2.3e38, and from 64 on silu(v) is v in fp32.
__device__ __forceinline__ float silu_any(float v) { return v > 64.0f ? v : silu_f32(v); }

__device__ __forceinline__ float act1(int act, float v) {
  switch (act) {
    case kActRelu: return v < 0.0f ? 0.0f : v;
    case kActSilu: return silu_any(v);
    case kActGelu: return v * normal_cdf(v);
    case kActGeluTanh: return v * gelu_gate(v);
    default: return v;
  }
}
__device__ __forceinline__ v4f act4(int act, v4f v) {  // act: the same for every lane
  if (act == kActNone) return v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = act1(act, v[i]);
  return v;
}

// The derivative (ReLU's at 0: 0).
__device__ __forceinline__ float slope1(int act, float v) {
  switch (act) {
    case kActRelu: return v > 0.0f ? 1.0f : 0.0f;
    case kActSilu: {
      const float s = 1.0f / (1.0f + expf(-v));
      return s * __builtin_fmaf(v, 1.0f - s, 1.0f);
    }
    case kActGelu: return __builtin_fmaf(v * 0.3989422804014327f, expf(-0.5f * v * v), normal_cdf(v));
    case kActGeluTanh: {
      const float s = gelu_gate(v);
      return __builtin_fmaf(v * s * (1.0f - s) * 1.5957691216057308f, __builtin_fmaf(0.134145f * v, v, 1.0f), s);
    }
    default: return 1.0f;
  }
}

// Both, from one evaluation of their common part: returns the slope.
__device__ __forceinline__ float act_and_slope(int act, float v, float& value) {
  switch (act) {
    case kActSilu: {
      const float s = 1.0f / (1.0f + expf(-v));
      value = v * s;
      return s * __builtin_fmaf(v, 1.0f - s, 1.0f);
    }
    case kActGelu: {
      const float c = normal_cdf(v);
      value = v * c;
      return __builtin_fmaf(v * 0.3989422804014327f, expf(-0.5f * v * v), c);
    }
    case kActGeluTanh: {
      const float s = gelu_gate(v);
      value = v * s;
      return __builtin_fmaf(v * s * (1.0f - s) * 1.5957691216057308f, __builtin_fmaf(0.134145f * v, v, 1.0f), s);
    }
    default:
      value = act1(act, v);
      return slope1(act, v);
  }
}

}  // namespace moe
