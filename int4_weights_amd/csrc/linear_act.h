// linear_act.h -- the activations of moe_gemm_bf16's epilogue and their slopes, in fp32.
#pragma once

#include "moe_device.h"

namespace moe {

enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// v within [lo, hi].  (NaN becomes lo: the callers multiply by v itself, so that NaN comes out all the same.)
__device__ __forceinline__ float within(float v, float lo, float hi) { return __builtin_amdgcn_fmed3f(v, lo, hi); }

// exp(a): the hardware exp2 of the rounded product with log2(e), times 1 + the product's error to first order.
__device__ __forceinline__ float exp_f32(float a) {
  constexpr float kLog2e = 1.44269504088896341f, kLog2eLo = 1.92596299e-08f, kLn2 = 0.693147180559945309f;
  const float hi = a * kLog2e;
  const float lo = __builtin_fmaf(a, kLog2eLo, __builtin_fmaf(a, kLog2e, -hi));
  return __builtin_amdgcn_exp2f(hi) * __builtin_fmaf(lo, kLn2, 1.0f);
}

// 1 / (1 + exp(-v)): 0 from -88 down, 1 from 17 up; the bounds keep what overflows from becoming NaN.
__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.0f + exp_f32(within(-v, -64.0f, 128.0f)));
}

// Phi(v) and exp(-v^2 / 2).  Phi(-|v|) = exp(-v^2 / 2) t P(t), t = 1 / (1 + 0.31 |v|), P the polynomial of degree 9 with the
// smallest relative error (1.2e-8 for |v| <= 41; t P(t) 3e-7 as evaluated in fp32), fitted to erfcx(|v| / sqrt 2) / (2 t): no
// cancellation for negative v, and one exponential for the function and its slope.  The exponent's rounding adds up to 2^-24 v^2 / 2
// in relative terms: the tail is off by 4e-7 at |v| = 4, 1e-6 at 6, 4e-6 at 13.
__device__ __forceinline__ float normal_cdf(float v, float& e) {
  const float x = fabsf(v), t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.31f, x, 1.0f));
  e = exp_f32(fmaxf(-0.5f * x * x, -200.0f));
  float p = -0.02082189917564392f;
  p = __builtin_fmaf(p, t, 0.10342404991388321f);
  p = __builtin_fmaf(p, t, -0.1837586760520935f);
  p = __builtin_fmaf(p, t, 0.11884111911058426f);
  p = __builtin_fmaf(p, t, -0.034121375530958176f);
  p = __builtin_fmaf(p, t, 0.07190302759408951f);
  p = __builtin_fmaf(p, t, 0.08510398119688034f);
  p = __builtin_fmaf(p, t, 0.11210367828607559f);
  p = __builtin_fmaf(p, t, 0.12365353852510452f);
  p = __builtin_fmaf(p, t, 0.12367255240678787f);
  const float tail = e * t * p;
  return v > 0.0f ? 1.0f - tail : tail;
}

// sqrt(2/pi) (v + 0.044715 v^3), doubled: gelu_tanh(v) = v sigmoid of it.
__device__ __forceinline__ float gelu_arg(float v) {
  return 1.5957691216057308f * v * __builtin_fmaf(0.044715f * v, v, 1.0f);
}

// Two fp32 values as bf16, rounded to nearest even by the hardware (NaN stays NaN).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// The activation's value, and its slope (ReLU's at 0: 0).  act: the same for every lane.
__device__ __forceinline__ float act_and_slope(int act, float v, float& slope) {
  switch (act) {
    case kActRelu:
      slope = v > 0.0f ? 1.0f : 0.0f;
      return v < 0.0f ? 0.0f : v;
    case kActSilu: {
      const float s = sigmoid_f32(v);
      slope = s * __builtin_fmaf(v, 1.0f - s, 1.0f);
      return v * s;
    }
    case kActGelu: {
      float e;
      const float c = normal_cdf(v, e);
      slope = __builtin_fmaf(v * 0.3989422804014327f, e, c);
      return v * c;
    }
    case kActGeluTanh: {
      const float w = within(v, -16.0f, 16.0f), s = sigmoid_f32(gelu_arg(w));  // its gate is 0 or 1 from there on
      slope = __builtin_fmaf(w * s * (1.0f - s) * 1.5957691216057308f, __builtin_fmaf(0.134145f * w, w, 1.0f), s);
      slope = v == v ? slope : v;  // NaN stays
      return v * s;
    }
    default:
      slope = 1.0f;
      return v;
  }
}
__device__ __forceinline__ float act1(int act, float v) {
  float slope;
  return act_and_slope(act, v, slope);
}
__device__ __forceinline__ v4f act4(int act, v4f v) {
  if (act == kActNone) return v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = act1(act, v[i]);
  return v;
}

}  // namespace moe
