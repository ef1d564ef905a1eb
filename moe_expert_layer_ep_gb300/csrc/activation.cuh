// The activations of the experts' products (moe_act_t) and their derivatives,
// in fp32, for the epilogues: by the hardware's base-2 exponential and
// reciprocal, both within 2 ulp, because an epilogue is bound by the
// instructions it issues (an IEEE quotient costs as much as the rest) and its
// results are rounded to bf16.  The exponential's argument v log2(e) is rounded
// first, which is what is left of exp(v) far from 0: (4 + 3 |v|) 2^-23 of it.
//
//   silu       z s,  s = 1 / (1 + exp(-z));          s (1 + z (1 - s))
//   gelu       z P,  P = (1 + erf(z / sqrt 2)) / 2;  P + z exp(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z s,  s = (1 + tanh v) / 2 = 1 / (1 + exp(-2 v)),
//              v = sqrt(2 / pi) (z + 0.044715 z^3);  s + z s (1 - s) 2 v'
//   relu       max(z, 0);                            1 above 0, else 0
//   relu2      max(z, 0)^2;                          2 max(z, 0)
//
// P: the rational approximation 7.1.26 of Abramowitz and Stegun's handbook,
// erfc(a) = t (a1 + t (a2 + ...)) exp(-a^2) with t = 1 / (1 + p a), whose error is
// at most 1.5e-7; the tail below 0 is taken as it is, not as 1 minus the rest.
// NaN stays NaN in all of them, values and derivatives.  A product is rounded before something is added to it
// (__fmul_rn, __fadd_rn where a compiler might join them), so that kernels of different
// shapes give the same bits.
#pragma once

#include "common.cuh"

namespace moe {

template <int kAct>
struct ActTag {
  static constexpr int value = kAct;
};

// f(tag) for the activation `act`, with the tag's value known to the compiler:
// the choice is made once for many elements.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case MOE_ACT_SILU: f(ActTag<MOE_ACT_SILU>{}); break;
    case MOE_ACT_GELU: f(ActTag<MOE_ACT_GELU>{}); break;
    case MOE_ACT_GELU_TANH: f(ActTag<MOE_ACT_GELU_TANH>{}); break;
    case MOE_ACT_RELU: f(ActTag<MOE_ACT_RELU>{}); break;
    case MOE_ACT_RELU2: f(ActTag<MOE_ACT_RELU2>{}); break;
    default: f(ActTag<MOE_ACT_NONE>{}); break;
  }
}

__device__ __forceinline__ float ex2_fast(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + exp(-x)); 0 below x = -87.3, where it is less than 2^-126.
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_fast(1.0f + ex2_fast(x * -1.44269504f)); }

// max(z, 0), NaN for NaN (z <= 0 ? 0 : z in one instruction).
__device__ __forceinline__ float not_below_0(float z) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));
  return r;
}

// The activation's value and, where it is asked for, its slope at z.
template <int kAct, bool kSlope>
__device__ __forceinline__ float act_at(float z, float* slope) {
  if constexpr (kAct == MOE_ACT_SILU) {
    const float s = sigmoid_fast(z);
    if constexpr (kSlope) *slope = s * fmaf(z, 1.0f - s, 1.0f);
    return z * s;
  } else if constexpr (kAct == MOE_ACT_GELU) {
    const float q = ex2_fast(z * z * -0.72134752f);            // exp(-z^2 / 2)
    const float t = rcp_fast(fmaf(0.23164189f, fabsf(z), 1.0f));   // p / sqrt 2 = 0.3275911 / sqrt 2
    float poly = fmaf(t, 1.061405429f, -1.453152027f);
    poly = fmaf(t, poly, 1.421413741f);
    poly = fmaf(t, poly, -0.284496736f);
    poly = fmaf(t, poly, 0.254829592f);
    const float tail = __fmul_rn(0.5f * t * poly, q);          // erfc(|z| / sqrt 2) / 2
    const float cdf = z >= 0.0f ? 1.0f - tail : tail;
    if constexpr (kSlope) *slope = fmaf(z * q, 0.39894228f, cdf);
    return z * cdf;
  } else if constexpr (kAct == MOE_ACT_GELU_TANH) {
    const float zz = fminf(z * z, 1e30f);                      // (no infinity times 0 in the slope)
    const float s = sigmoid_fast(z * fmaf(zz, 0.07135481f, 1.59576912f));   // 2 sqrt(2 / pi) (1, 0.044715)
    const float v = z * s;
    if constexpr (kSlope) *slope = fmaf(v * (1.0f - s), fmaf(zz, 0.21406444f, 1.59576912f), s);
    return v;
  } else if constexpr (kAct == MOE_ACT_RELU) {
    const float r = not_below_0(z);
    if constexpr (kSlope) *slope = r > 0.0f ? 1.0f : r;
    return r;
  } else if constexpr (kAct == MOE_ACT_RELU2) {
    const float r = not_below_0(z);
    if constexpr (kSlope) *slope = 2.0f * r;
    return r * r;
  } else {
    if constexpr (kSlope) *slope = 1.0f;
    return z;
  }
}

}  // namespace moe
