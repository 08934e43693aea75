// router.hip -- moe_router_topk and its gradient: the router between the gate
// projection's logits and moe_route_pack's topk_ids / topk_weights.
//
// Forward, per token (row of E logits x):
//   score   s_e = 1 / (1 + exp(-x_e)) or exp(x_e - m) / sum exp(x - m)
//   key     x_e without a bias (every score is increasing in x), else s_e + b_e
//   groups  G groups of E/G consecutive experts, the best topk_group of them by
//           their largest key, or by the sum of their two largest keys
//   slots   the k largest keys of the kept groups, ties to the lowest expert
//   weight  scale * s, or scale * s / (sum of the selected s)
// One wave per token, the row in registers: lane group g holds expert group g
// (G rounded up to a power of two divides the wave), each lane VPL consecutive
// experts, so a lane's order is the experts' order and a tie goes to the lowest
// lane, then its lowest register.
//
// Exact choice from 32-bit keys.  Experts are ordered by key in 64 bits
// (scores of two experts can lie closer together than fp32 resolves, and a
// different order is a different result), but nearly every row is decided by
// fp32 keys: they carry a bound es + 2^-23 |key| on their error (es: 2^-20 for
// sigmoid scores, 2^-18 times the largest probability for softmax ones; the
// evaluation below stays within half of that), and a row whose neighbouring
// candidates are closer than the bounds allow has its candidates (those down to the
// first clear gap after the k-th) ordered by fp64 keys, one per lane; a row whose
// groups around the last kept one are that close has its group scores summed in
// fp64; only a row with more than 64 close candidates is selected again
// with fp64 keys throughout.  (A whole second selection for every such row cost 6 to 14 us, the
// kernel's tail, with about 12 of them in 4096.)  Without a bias the keys are the logits
// themselves and need no check.
//
// Measured: 4096 x 256, sigmoid, bias, 4 of 8 groups, k 8: 8.6 us; softmax without bias 5.6 us; 16 x 128: 3.8 us, the launch.
// Memory (4.5 MB, 0.9 us) does not bound it: each of the k rounds waits for a maximum over the wave, seven dependent
// cross-lane steps.
//
// A logit of -inf or NaN marks an expert that this token may not use; slots
// left over get id -1 and weight 0, which moe_route_pack skips.
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kNone = (int)0x80000000;  // key of an expert that cannot be chosen

// exp(x) for x <= 0 (and any x below overflow) to about two fp32 ulps: the product x * log2(e) is carried as
// hi + lo, the hardware exp2 takes hi, and lo enters to first order.  0 at -inf.
__device__ __forceinline__ float exp_f32(float x) {
  constexpr float kLog2e = 1.44269504088896341f, kLog2eLo = 1.92596299e-08f, kLn2 = 0.693147180559945309f;
  const float hi = x * kLog2e;
  const float lo = __builtin_fmaf(x, kLog2e, -hi) + x * kLog2eLo;
  const float r = __builtin_amdgcn_exp2f(hi);
  return fabsf(hi) < 200.0f ? r * __builtin_fmaf(lo, kLn2, 1.0f) : r;
}

__device__ __forceinline__ float sigmoid_f32(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_f32(-x)); }

// signed integer in the order of the float (x + 0 turns -0 into +0: equal floats have equal keys)
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x + 0.0f);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

template <int CTRL>
__device__ __forceinline__ int dpp(int old, int v) {
  return __builtin_amdgcn_update_dpp(old, v, CTRL, 0xF, 0xF, false);
}

// Maximum over the wave, in every lane (as a scalar): five steps inside the rows of 16 lanes, two across them.
__device__ __forceinline__ int wave_max_i32(int v) {
  v = max(v, dpp<0xB1>(v, v));
  v = max(v, dpp<0x4E>(v, v));
  v = max(v, dpp<0x141>(v, v));
  v = max(v, dpp<0x140>(v, v));
  v = max(v, dpp<0x142>(v, v));  // lane 15 of a row to the next row
  v = max(v, dpp<0x143>(v, v));  // lane 31 to rows 2 and 3
  return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ float wave_max_f32(float v) { return unordered(wave_max_i32(ordered(v))); }

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float old, float v) {
  return __int_as_float(dpp<CTRL>(__float_as_int(old), __float_as_int(v)));
}

// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += dpp_f32<0xB1>(v, v);
  v += dpp_f32<0x4E>(v, v);
  v += dpp_f32<0x141>(v, v);
  v += dpp_f32<0x140>(v, v);
  v += dpp_f32<0x142>(0.0f, v);
  v += dpp_f32<0x143>(0.0f, v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__device__ __forceinline__ float readlane_f32(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
  if constexpr (sizeof(T) == 2)
    return bf16_to_f32(*p);
  else
    return *p;
}

// Orders one wave's LDS accesses: what a lane wrote before it, every lane of the wave reads after it.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A lane's candidates in descending order: keys, and their positions j packed 4 bits each (first candidate lowest).
// Equal keys keep the lower position first (the comparison is of (key, -j) as one 64-bit integer).  Popping the lane's
// best is then a shift, and no round of the selection searches the lane again (8 rounds over 256 experts: 55
// instructions a round with the search, 28 with the shift).
template <int VPL>
struct Sorted {
  int key[VPL];
  uint32_t pos;
  static __device__ __forceinline__ void order(int64_t& a, int64_t& b) {
    const int64_t hi = a > b ? a : b, lo = a > b ? b : a;
    a = hi;
    b = lo;
  }
  __device__ __forceinline__ void sort(const int (&ik)[VPL]) {
    static_assert(VPL == 1 || VPL == 2 || VPL == 4 || VPL == 8, "sorting networks below");
    int64_t v[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) v[j] = (int64_t)((uint64_t)(uint32_t)ik[j] << 32 | (uint32_t)(VPL - 1 - j));
    // odd-even merge sort
#pragma unroll
    for (int p = 1; p < VPL; p *= 2)
#pragma unroll
      for (int q = p; q >= 1; q /= 2)
#pragma unroll
        for (int j = q % p; j + q < VPL; j += 2 * q)
#pragma unroll
          for (int i = 0; i < q; ++i)
            if (i + j + q < VPL && (i + j) / (2 * p) == (i + j + q) / (2 * p)) order(v[i + j], v[i + j + q]);
    pos = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      key[j] = (int)(v[j] >> 32);
      pos |= (VPL - 1 - (uint32_t)v[j]) << (4 * j);
    }
  }
  __device__ __forceinline__ int best() const { return key[0]; }
  __device__ __forceinline__ int best_pos(int) const { return (int)(pos & 15); }
  __device__ __forceinline__ void pop(int) {
#pragma unroll
    for (int j = 0; j + 1 < VPL; ++j) key[j] = key[j + 1];
    key[VPL - 1] = kNone;
    pos >>= 4;
  }
};
// More candidates per lane than are worth sorting: searched again in every round.
template <int VPL>
struct Unsorted {
  int key[VPL];
  __device__ __forceinline__ void sort(const int (&ik)[VPL]) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = ik[j];
  }
  __device__ __forceinline__ int best() const {
    int b = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) b = max(b, key[j]);
    return b;
  }
  __device__ __forceinline__ int best_pos(int mk) const {
    int p = 0;
#pragma unroll
    for (int j = VPL - 1; j >= 0; --j) p = key[j] == mk ? j : p;
    return p;
  }
  __device__ __forceinline__ void pop(int p) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = j == p ? kNone : key[j];
  }
};
template <int VPL, bool SMALL>
struct Cands : Sorted<VPL> {};
template <int VPL>
struct Cands<VPL, false> : Unsorted<VPL> {};

// Where this lane's experts are: expert base + j for j < n.
struct LaneExperts {
  int base, n, lpg;  // lpg: lanes per group
};
__device__ __forceinline__ LaneExperts lane_experts(int E, int G, int lane) {
  const int S = E / G;
  const int lg = G > 1 ? 32 - __builtin_clz(G - 1) : 0;  // log2 of G rounded up
  const int lpg = 64 >> lg;
  const int cnt = (S + lpg - 1) / lpg;
  const int g = lane >> (6 - lg), l = lane & (lpg - 1);
  LaneExperts r;
  r.lpg = lpg;
  r.base = g * S + l * cnt;
  r.n = g < G ? max(0, min(cnt, S - l * cnt)) : 0;
  return r;
}

struct Pick {
  int id;   // lane r < k: the expert of slot r, -1 if none
  float x;  // and its logit
};

// Two largest of the group's keys, in all its lanes: pairs, quads, 8 and 16 lanes meet inside the VALU (a mirror
// reaches the other half where each half is uniform), wider groups through the lane crossbar.
__device__ __forceinline__ void meet_top2(float& a1, float& a2, float b1, float b2) {
  a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
  a1 = fmaxf(a1, b1);
}
__device__ __forceinline__ void group_top2(float& a1, float& a2, int lpg) {
  if (lpg > 1) meet_top2(a1, a2, dpp_f32<0xB1>(a1, a1), dpp_f32<0xB1>(a2, a2));
  if (lpg > 2) meet_top2(a1, a2, dpp_f32<0x4E>(a1, a1), dpp_f32<0x4E>(a2, a2));
  if (lpg > 4) meet_top2(a1, a2, dpp_f32<0x141>(a1, a1), dpp_f32<0x141>(a2, a2));
  if (lpg > 8) meet_top2(a1, a2, dpp_f32<0x140>(a1, a1), dpp_f32<0x140>(a2, a2));
  if (lpg > 16) meet_top2(a1, a2, __shfl_xor(a1, 16, 64), __shfl_xor(a2, 16, 64));
}

// What follows in 64 bits is for a few rows in a thousand: it reads the row again, one expert per lane and turn, and
// keeps its keys in LDS, so that it costs the other rows no registers (inlined with its keys in registers the kernel
// held 108 of them and 4 waves a SIMD).

template <typename T>
__device__ __forceinline__ float logit_or_none(const T* row, int e) {
  const float x = load_logit(row + e);
  return x > -__builtin_huge_valf() ? x : -__builtin_huge_valf();
}

// Largest logit and the sum of exponentials of the row (softmax).
template <typename T>
__device__ __forceinline__ void softmax_f64(const T* row, int E, int lane, double& m, double& den) {
  float mf = -__builtin_huge_valf();
#pragma unroll 1
  for (int e = lane; e < E; e += 64) mf = fmaxf(mf, logit_or_none(row, e));
  mf = wave_max_f32(mf);
  m = (double)mf;
  double s = 0.0;
#pragma unroll 1
  for (int e = lane; e < E; e += 64) {
    const float x = logit_or_none(row, e);
    if (x > -__builtin_huge_valf()) s += x == mf ? 1.0 : exp((double)x - m);
  }
  den = wave_sum_f64(s);
}
__device__ __forceinline__ double score_f64(int score, double x, double m, double den) {
  const double t = exp(score == 0 ? x - m : -x);
  return score == 0 ? (x == m ? 1.0 : t) / den : 1.0 / (1.0 + t);
}

// Order in 64 bits of the candidates in lanes 0 .. c - 1 (one expert each, none outside them can be among the best k):
// each counts those ahead of it and moves to that lane.
template <typename T>
__device__ __forceinline__ Pick order_f64(const RouterArgs& a, const T* row, Pick p, int c, int lane) {
  double m = 0.0, den = 1.0;
  if (a.score == 0) softmax_f64(row, a.E, lane, m, den);
  const double key = lane < c ? score_f64(a.score, (double)p.x, m, den) + (double)a.bias[p.id] : 0.0;
  int ahead = 0;
  for (int j = 0; j < c; ++j) {
    const int lo = __builtin_amdgcn_readlane((int)(__double_as_longlong(key)), j);
    const int hi = __builtin_amdgcn_readlane((int)(__double_as_longlong(key) >> 32), j);
    const double kj = __longlong_as_double(((long long)hi << 32) | (uint32_t)lo);
    const int ij = __builtin_amdgcn_readlane(p.id, j);
    ahead += kj > key || (kj == key && ij < p.id);
  }
  const int to = 4 * (lane < c ? ahead : lane);
  Pick o;
  o.id = __builtin_amdgcn_ds_permute(to, p.id);
  o.x = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(p.x)));
  if (lane >= a.k) o.id = -1;
  return o;
}

// Whether this lane's expert group is among the kept ones, by group scores in 64 bits.
template <typename T>
__device__ __forceinline__ bool group_kept_f64(const RouterArgs& a, const T* row, const LaneExperts& le, int lane) {
  const double ninf = -__builtin_huge_val();
  double den = 1.0, m = 0.0, a1 = ninf, a2 = ninf;
  if (a.score == 0) softmax_f64(row, a.E, lane, m, den);
#pragma unroll 1
  for (int j = 0; j < le.n; ++j) {
    const float x = logit_or_none(row, le.base + j);
    double v = score_f64(a.score, (double)x, m, den);
    if (a.bias) v += (double)a.bias[le.base + j];
    v = x > -__builtin_huge_valf() && v > ninf ? v : ninf;
    const double lo = v < a1 ? v : a1;
    a1 = v > a1 ? v : a1;
    a2 = lo > a2 ? lo : a2;
  }
#pragma unroll 1
  for (int off = 1; off < le.lpg; off <<= 1) {
    const double b1 = __shfl_xor(a1, off, 64), b2 = __shfl_xor(a2, off, 64);
    const double lo = a1 < b1 ? a1 : b1, m2 = a2 > b2 ? a2 : b2;
    a1 = a1 > b1 ? a1 : b1;
    a2 = lo > m2 ? lo : m2;
  }
  const double gs = a.gtop == 1 || !(a2 > ninf) ? a1 : a1 + a2;
  const int g = lane / le.lpg;
  int better = 0;
#pragma unroll 1
  for (int o = 0; o < a.G; ++o) {
    const double go = __shfl(gs, o * le.lpg, 64);
    better += go > gs || (go == gs && o < g);
  }
  return better < a.TG;
}

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll 1
  for (int off = 1; off < 64; off <<= 1) {
    const double o = __shfl_xor(v, off, 64);
    v = o > v ? o : v;
  }
  return v;
}

// The whole choice in 64 bits, with a bias (every lane of the wave calls it): lane l holds experts l, l + 64, ... in
// key[] (LDS).
template <typename T>
__device__ __forceinline__ Pick select_f64(const RouterArgs& a, const T* row, double* key, int lane) {
  const double ninf = -__builtin_huge_val();
  double den = 1.0, m = 0.0;
  if (a.score == 0) softmax_f64(row, a.E, lane, m, den);
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const float x = logit_or_none(row, e);
    double v = score_f64(a.score, (double)x, m, den);
    v += (double)a.bias[e];
    key[e] = x > -__builtin_huge_valf() && v > ninf ? v : ninf;
  }
  wave_fence();
  if (a.G > 1) {
    // lane g: group g (at most 64)
    const int S = a.E / a.G;
    double a1 = ninf, a2 = ninf;
    if (lane < a.G) {
#pragma unroll 1
      for (int e = lane * S; e < (lane + 1) * S; ++e) {
        const double v = key[e];
        const double lo = v < a1 ? v : a1;
        a1 = v > a1 ? v : a1;
        a2 = lo > a2 ? lo : a2;
      }
    }
    const double gs = a.gtop == 1 || !(a2 > ninf) ? a1 : a1 + a2;
    int better = 0;
#pragma unroll 1
    for (int o = 0; o < a.G; ++o) {
      const double go = __shfl(gs, o, 64);
      better += go > gs || (go == gs && o < lane);
    }
    const uint64_t kept = __ballot(lane < a.G && better < a.TG);
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64)
      if (!(kept >> (e / S) & 1)) key[e] = ninf;
  }
  Pick p{-1, 0.0f};
#pragma unroll 1
  for (int r = 0; r < a.k; ++r) {
    double best = ninf;
    int be = a.E;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
      if (key[e] > best) {
        best = key[e];
        be = e;
      }
    }
    const double mk = wave_max_f64(best);
    if (!(mk > ninf)) break;
    int we = best == mk ? be : a.E;  // the lowest expert of the lanes that hold the largest key
#pragma unroll 1
    for (int off = 1; off < 64; off <<= 1) we = min(we, __shfl_xor(we, off, 64));
    if (we == be && best == mk) key[we] = ninf;
    if (lane == r) {
      p.id = we;
      p.x = load_logit(row + we);
    }
  }
  wave_fence();  // key[] is rewritten by the next row
  return p;
}

// The weights of the selected slots (lane r: slot r; lanes >= k and empty slots hold on = false).
__device__ __forceinline__ float slot_weight(int score, int norm, float scale, bool on, float x, float row_m,
                                             float row_den) {
  if (norm) {
    const float m = wave_max_f32(on ? x : -__builtin_huge_valf());
    float q;
    if (score == 0)
      q = x == m ? 1.0f : exp_f32(x - m);
    else  // s / s_max without underflow: exp(min(x, 0)) / (1 + exp(-|x|)) is the sigmoid for either sign
      q = exp_f32(fminf(x, 0.0f) - fminf(m, 0.0f)) / (1.0f + exp_f32(-fabsf(x)));
    q = on ? q : 0.0f;
    const float sum = wave_sum_f32(q);
    return on ? scale * (q / sum) : 0.0f;
  }
  float s;
  if (score == 0)
    s = (x == row_m ? 1.0f : exp_f32(x - row_m)) / row_den;
  else
    s = exp_f32(fminf(x, 0.0f)) / (1.0f + exp_f32(-fabsf(x)));
  return on ? scale * s : 0.0f;
}

}  // namespace

// BIAS and GROUPS (a.bias, a.G > 1) are compiled apart: a scalar branch per round costs as much as the round's work.
template <typename T, int VPL, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(256) void router_topk_kernel(const RouterArgs a) {
  __shared__ double s_key[4][BIAS ? 64 * (VPL < 16 ? VPL : 16) : 1];  // E <= 1024
  const int lane = lane_id();
  const float ninf = -__builtin_huge_valf();
  const LaneExperts le = lane_experts(a.E, GROUPS ? a.G : 1, lane);
  const bool by_score = BIAS || (GROUPS && a.gtop == 2);
  float b[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    b[j] = 0.0f;
    if constexpr (BIAS) b[j] = a.bias[min(le.base + j, a.E - 1)];
  }
  for (int64_t t = blockIdx.x * 4 + uniform(threadIdx.x >> 6); t < a.T; t += gridDim.x * 4) {
    const T* row = (const T*)a.logits + t * a.ld;
    float x[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = load_logit(row + min(le.base + j, a.E - 1));
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = j < le.n && x[j] > ninf ? x[j] : ninf;  // NaN is -inf

    float row_m = 0.0f, row_den = 1.0f, ex[VPL];
    if (a.score == 0 && (by_score || !a.norm)) {
      float mf = ninf;
#pragma unroll
      for (int j = 0; j < VPL; ++j) mf = fmaxf(mf, x[j]);
      row_m = wave_max_f32(mf);
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        ex[j] = x[j] > ninf ? (x[j] == row_m ? 1.0f : exp_f32(x[j] - row_m)) : 0.0f;
        s += ex[j];
      }
      s = wave_sum_f32(s);
      row_den = s > 0.0f ? s : 1.0f;  // 0 only where no expert is available
    }

    float key[VPL];
    float es = 0.0f;
    if (by_score) {
      const float inv = 1.0f / row_den;
      es = a.score == 0 ? 0x1p-18f * inv : 0x1p-20f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const float s = a.score == 0 ? ex[j] * inv : sigmoid_f32(x[j]);
        key[j] = s + b[j];
        if (!(x[j] > ninf) || !(key[j] > ninf)) key[j] = ninf;
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = x[j];
    }

    bool kept = true;
    if constexpr (GROUPS) {
      float a1 = ninf, a2 = ninf;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const float v = key[j], lo = fminf(v, a1);
        a1 = fmaxf(v, a1);
        a2 = fmaxf(lo, a2);
      }
      group_top2(a1, a2, le.lpg);
      const bool two = a.gtop == 2 && a2 > ninf;
      const float gs = two ? a1 + a2 : a1;
      const int g = lane / le.lpg;
      if (by_score) {
        // 0 for a group without available experts (its infinite key says nothing about precision)
        const float eg = a1 > ninf ? 2.0f * es + 0x1p-22f * (fabsf(a1) + (two ? fabsf(a2) : 0.0f)) : 0.0f;
        const float lo = gs - eg, hi = gs + eg;
        int above = 0, maybe = -1;  // groups surely above this one; possibly above (this one itself counts once)
        for (int o = 0; o < a.G; ++o) {
          above += readlane_f32(lo, o * le.lpg) > hi;
          maybe += !(readlane_f32(hi, o * le.lpg) < lo);
        }
        kept = above < a.TG;
        if (__any(kept && maybe >= a.TG && gs > ninf)) kept = group_kept_f64(a, row, le, lane);
      } else {
        int better = 0;
        for (int o = 0; o < a.G; ++o) {
          const float go = readlane_f32(gs, o * le.lpg);
          better += go > gs || (go == gs && o < g);
        }
        kept = better < a.TG;
      }
    }

    Pick p{-1, 0.0f};
    bool unsure = false;  // more close candidates than lanes
    {
      int ik[VPL];
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        // without a bias the experts' order is the logits'
        const float v = BIAS ? key[j] : x[j];
        ik[j] = kept && key[j] > ninf ? ordered(v) : kNone;
      }
      // With a bias, extraction goes on until the next key is clearly below (r counts the candidates by then); where
      // two of them were too close, their order is settled in 64 bits.
      Cands<VPL, (VPL <= 8)> cand;
      cand.sort(ik);
      float prev = 0.0f;
      bool close = false;
      int r = 0;
      for (;; ++r) {
        const int best = cand.best();
        const int mk = wave_max_i32(best);
        if (mk == kNone) break;
        if constexpr (BIAS) {
          const float v = unordered(mk);
          if (r > 0 && !(prev - v > 2.0f * es + 0x1p-23f * (fabsf(prev) + fabsf(v))))
            close = true;
          else if (r >= a.k)
            break;
          if (r == 64) {
            unsure = true;
            break;
          }
          prev = v;
        } else if (r == a.k) {
          break;
        }
        const int wl = __builtin_ctzll(__ballot(best == mk));
        const int pos = cand.best_pos(mk);
        const int ew = __builtin_amdgcn_readlane(le.base + pos, wl);
        if (lane == wl) cand.pop(pos);
        if (lane == r) {
          p.id = ew;
          p.x = unordered(mk);
        }
      }
      if (BIAS && lane < r) p.x = load_logit(row + p.id);  // the key is not the logit
      if constexpr (BIAS)
        if (close && !unsure) p = order_f64(a, row, p, r, lane);
    }
    if constexpr (BIAS)
      if (unsure) p = select_f64(a, row, s_key[threadIdx.x >> 6], lane);

    const bool on = p.id >= 0;
    const float w = slot_weight(a.score, a.norm, a.scale, on, p.x, row_m, row_den);
    if (lane < a.k) {
      a.ids[t * a.k + lane] = p.id;
      a.w[t * a.k + lane] = w;
    }
  }
}

// Gradient, per token, with g_r = d weight_r, w_r the weight and s_r the score of slot r:
//   renormalised:       d x_r = w_r (g_r - sum_j g_j w_j / scale), times 1 - s_r for sigmoid scores
//   sigmoid as it is:   d x_r = scale g_r s_r (1 - s_r)
//   softmax as it is:   d x_e = scale p_e ([e selected] g_e - sum_j g_j p_j), for every expert
// One wave per token; slots in lanes, the row assembled in LDS so that it is written once, whole (4096 x 256 in fp32: 5.3 us;
// 8191 x 128 in bf16, softmax as it is: 6.9 us; the launch takes 4.4 of either).  An expert
// named by two slots gets the sum over them, in slot order.
template <typename T, int VPL>
__global__ __launch_bounds__(256) void router_topk_bwd_kernel(const RouterBwdArgs a) {
  __shared__ float s_row[4][64 * VPL];
  const int lane = lane_id(), wv = uniform(threadIdx.x >> 6);
  const float ninf = -__builtin_huge_valf();
  float* srow = s_row[wv];
  const bool dense = a.score == 0 && !a.norm;
  const int base = lane * VPL;
  for (int64_t t = blockIdx.x * 4 + wv; t < a.T; t += gridDim.x * 4) {
    const T* row = (const T*)a.logits + t * a.ld;
    int id = -1;
    float g = 0.0f, x = ninf;
    if (lane < a.k) {
      id = a.ids[t * a.k + lane];
      if (id < 0 || id >= a.E) id = -1;
      if (id >= 0) {
        x = load_logit(row + id);
        g = a.dw[t * a.k + lane];
      }
    }
    const bool on = x > ninf;  // an empty slot, or an expert that was not available: no gradient
    g = on ? g : 0.0f;
    float row_m = 0.0f, row_den = 1.0f, ex[VPL];
    if (dense) {
      float mf = ninf;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const float v = base + j < a.E ? load_logit(row + base + j) : ninf;
        ex[j] = v > ninf ? v : ninf;
        mf = fmaxf(mf, ex[j]);
      }
      row_m = wave_max_f32(mf);
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        ex[j] = ex[j] > ninf ? (ex[j] == row_m ? 1.0f : exp_f32(ex[j] - row_m)) : 0.0f;
        s += ex[j];
      }
      s = wave_sum_f32(s);
      row_den = s > 0.0f ? s : 1.0f;  // 0 only where no expert is available
    }
    const float w = slot_weight(a.score, a.norm, 1.0f, on, x, row_m, row_den);
    const float sg = a.scale * g;
    float d, mean = 0.0f;
    if (a.norm || dense) mean = wave_sum_f32(sg * w);
    if (a.norm)
      d = w * (sg - mean);
    else
      d = sg * w;  // dense: the -p_e * mean part is added to every expert below
    if (a.score != 0) {
      const float ax = fabsf(x);  // 1 - s = exp(min(-x, 0)) / (1 + exp(-|x|))
      d *= exp_f32(fminf(-x, 0.0f)) / (1.0f + exp_f32(-ax));
    }
    d = on ? d : 0.0f;
    // slots of the same expert: the first one carries the sum
    bool first = on;
    float sum = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      const int ij = __builtin_amdgcn_readlane(id, j);
      const float dj = readlane_f32(d, j);
      if (ij == id) {
        sum += dj;
        if (j < lane) first = false;
      }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) srow[base + j] = 0.0f;
    wave_fence();
    if (first) srow[id] = sum;
    wave_fence();
    T* out = (T*)a.dlogits + t * a.ldd;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      float v = srow[base + j];
      if (dense) v -= ex[j] / row_den * mean;
      if (base + j < a.E) {
        if constexpr (sizeof(T) == 2)
          out[base + j] = (T)f32_to_bf16_rne(v);
        else
          out[base + j] = v;
      }
    }
    wave_fence();  // the row is rewritten for the next token
  }
}

namespace {

int row_grid(int T) {
  const int64_t need = ((int64_t)T + 3) / 4, cap = (int64_t)device_info().cus * 32;
  return (int)(need < cap ? need : cap);
}

template <typename T, int VPL>
void launch_topk_vpl(const RouterArgs& a, hipStream_t s) {
  const int g = row_grid(a.T);
  if (a.bias && a.G > 1) router_topk_kernel<T, VPL, true, true><<<g, 256, 0, s>>>(a);
  else if (a.bias) router_topk_kernel<T, VPL, true, false><<<g, 256, 0, s>>>(a);
  else if (a.G > 1) router_topk_kernel<T, VPL, false, true><<<g, 256, 0, s>>>(a);
  else router_topk_kernel<T, VPL, false, false><<<g, 256, 0, s>>>(a);
}
template <typename T>
hipError_t launch_topk(const RouterArgs& a, int cnt, hipStream_t s) {
  if (cnt <= 1) launch_topk_vpl<T, 1>(a, s);
  else if (cnt <= 2) launch_topk_vpl<T, 2>(a, s);
  else if (cnt <= 4) launch_topk_vpl<T, 4>(a, s);
  else if (cnt <= 8) launch_topk_vpl<T, 8>(a, s);
  else if (cnt <= 16) launch_topk_vpl<T, 16>(a, s);
  else launch_topk_vpl<T, 32>(a, s);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_bwd(const RouterBwdArgs& a, hipStream_t s) {
  const int g = row_grid(a.T), cnt = (a.E + 63) / 64;
  if (cnt <= 1) router_topk_bwd_kernel<T, 1><<<g, 256, 0, s>>>(a);
  else if (cnt <= 2) router_topk_bwd_kernel<T, 2><<<g, 256, 0, s>>>(a);
  else if (cnt <= 4) router_topk_bwd_kernel<T, 4><<<g, 256, 0, s>>>(a);
  else if (cnt <= 8) router_topk_bwd_kernel<T, 8><<<g, 256, 0, s>>>(a);
  else router_topk_bwd_kernel<T, 16><<<g, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router_topk(const RouterArgs& a, hipStream_t s) {
  int gp = 1;
  while (gp < a.G) gp *= 2;
  const int lpg = 64 / gp, cnt = (a.E / a.G + lpg - 1) / lpg;
  return a.bf16 ? launch_topk<uint16_t>(a, cnt, s) : launch_topk<float>(a, cnt, s);
}

hipError_t launch_router_topk_bwd(const RouterBwdArgs& a, hipStream_t s) {
  return a.bf16 ? launch_bwd<uint16_t>(a, s) : launch_bwd<float>(a, s);
}

}  // namespace moe
