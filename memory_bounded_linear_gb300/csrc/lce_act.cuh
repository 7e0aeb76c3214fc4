// The activations of the feed-forward operators and their derivatives, in fp32.
//   relu(x) = max(x, 0)                      silu(x) = x s(x),  s(x) = 1 / (1 + e^-x)
//   gelu(x) = x Phi(x), Phi the normal distribution function
//   gelu_tanh(x) = x (1 + tanh(w)) / 2 = x s(2 w),  w = sqrt(2/pi) (x + 0.044715 x^3)
// FAST (bf16 inputs): the exponential and the quotient are the hardware approximations, whose error of
// a few 2^-22 is far below the rounding of the result to 8 bits, and Phi is a short polynomial; fp32
// inputs take the accurate functions.  The FAST formulas take one value or two (V = float, float2: one
// packed instruction for both where the hardware has it).
#pragma once

#include <cuda_runtime.h>
#include <math.h>

#include "lce.h"
#include "ptx.cuh"

namespace lce {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float all(float c, float) { return c; }
__device__ __forceinline__ float2 all(float c, float2) { return make_float2(c, c); }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 vmul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float2 vadd(float2 a, float2 b) { return __fadd2_rn(a, b); }
// f of every value
template <typename F>
__device__ __forceinline__ float each(float x, F&& f) { return f(x); }
template <typename F>
__device__ __forceinline__ float2 each(float2 x, F&& f) { return make_float2(f(x.x), f(x.y)); }
template <typename V>
__device__ __forceinline__ V vex2(V x) { return each(x, [](float v) { return ptx::ex2_approx(v); }); }
template <typename V>
__device__ __forceinline__ V vrcp(V x) { return each(x, [](float v) { return ptx::rcp_approx(v); }); }
__device__ __forceinline__ float where_positive(float x, float a, float b) { return x > 0.f ? a : b; }
__device__ __forceinline__ float2 where_positive(float2 x, float2 a, float2 b) {
  return make_float2(x.x > 0.f ? a.x : b.x, x.y > 0.f ? a.y : b.y);
}

// s(c x) for the constant c; x below about -88 / c: e^-cx is huge or inf and the quotient 0
template <typename V>
__device__ __forceinline__ V fast_sigmoid(V x, float c = 1.f) {
  return vrcp(vadd(vex2(vmul(x, all(-kLog2e * c, x))), all(1.f, x)));
}

// Phi(x) and e = exp(-x^2 / 2), for bf16 results.  The upper tail Q(y) = erfc(y / sqrt 2) / 2 is
// e t P(t) / 2 with t = 1 / (1 + 0.46 y / sqrt 2), Hastings' form; the degree-5 P was fitted to exp(z^2)
// erfc(z) / t on z >= 0 (least squares in t, reweighted towards the largest relative error as in
// Lawson's algorithm; 1.8e-5).  One exponential
// and one quotient serve Phi and the density in its derivative.
template <typename V>
__device__ __forceinline__ V normal_cdf(V x, V& e) {
  const V y = each(x, [](float v) { return fabsf(v); });
  const V t = vrcp(vfma(all(0.46f * kSqrtHalf, x), y, all(1.f, x)));
  e = vex2(vmul(vmul(x, x), all(-0.5f * kLog2e, x)));
  V p = all(0.5f * -0.12635274f, x);  // P / 2
  p = vfma(p, t, all(0.5f * 0.24180298f, x));
  p = vfma(p, t, all(0.5f * 0.12544967f, x));
  p = vfma(p, t, all(0.5f * 0.24052443f, x));
  p = vfma(p, t, all(0.5f * 0.25903428f, x));
  p = vfma(p, t, all(0.5f * 0.25953171f, x));
  const V q = vmul(e, vmul(t, p));
  return where_positive(x, vfma(q, all(-1.f, x), all(1.f, x)), q);
}

// act(x) and, if asked for, d = act'(x) (they share their exponential).
template <int ACT, bool GRAD, typename V>
__device__ __forceinline__ V fast_act(V x, V& d) {
  V a = x;
  if constexpr (ACT == LCE_ACT_RELU) {
    a = each(x, [](float v) { return v > 0.f ? v : (v == v ? 0.f : v); });
    if constexpr (GRAD) d = each(x, [](float v) { return v <= 0.f ? 0.f : 1.f; });
  } else if constexpr (ACT == LCE_ACT_SILU) {
    const V s = fast_sigmoid(x);
    a = vmul(x, s);
    if constexpr (GRAD) d = vfma(a, vfma(s, all(-1.f, x), all(1.f, x)), s);
  } else if constexpr (ACT == LCE_ACT_GELU) {
    V e;
    const V c = normal_cdf(x, e);
    a = vmul(x, c);
    // e is 0 long before x overflows the product
    if constexpr (GRAD) d = vfma(vmul(x, all(kInvSqrt2Pi, x)), e, c);
  } else if constexpr (ACT == LCE_ACT_GELU_TANH) {
    const V x2 = vmul(x, x);
    const V s = fast_sigmoid(vmul(x, vfma(x2, all(0.044715f, x), all(1.f, x))), 2.f * kSqrt2OverPi);
    a = vmul(x, s);
    if constexpr (GRAD) {
      // a (1 - s) is 0 from |x| = 16 on, where x^2 must not turn it into 0 inf
      const V c2 = each(x2, [](float v) { return fminf(v, 256.f); });
      const V w = vfma(c2, all(6.f * kSqrt2OverPi * 0.044715f, x), all(2.f * kSqrt2OverPi, x));
      d = vfma(vmul(a, vfma(s, all(-1.f, x), all(1.f, x))), w, s);
    }
  } else if constexpr (GRAD) {
    d = all(1.f, x);
  }
  return a;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }
// By erfc: 1 + erf(x / sqrt 2) loses Phi's small values (3e-4 of it at x = -4, 4% at -5, all below -5.4).
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(x * -kSqrtHalf); }

template <int ACT, bool FAST>
__device__ __forceinline__ float act(float x) {
  float d;
  if constexpr (FAST || ACT == LCE_ACT_NONE || ACT == LCE_ACT_RELU) return fast_act<ACT, false>(x, d);
  if constexpr (ACT == LCE_ACT_SILU) return x * sigmoid(x);
  if constexpr (ACT == LCE_ACT_GELU) return x * normal_cdf(x);
  return x * sigmoid(2.f * kSqrt2OverPi * (x + 0.044715f * x * x * x));
}

// a = act(x) and d = act'(x) together.
template <int ACT, bool FAST>
__device__ __forceinline__ void act_grad(float x, float& a, float& d) {
  if constexpr (FAST || ACT == LCE_ACT_NONE || ACT == LCE_ACT_RELU) {
    a = fast_act<ACT, true>(x, d);
  } else if constexpr (ACT == LCE_ACT_SILU) {
    const float s = sigmoid(x);
    a = x * s;
    d = s + a * (1.f - s);
  } else if constexpr (ACT == LCE_ACT_GELU) {
    const float c = normal_cdf(x);
    a = x * c;
    d = c + x * expf(-0.5f * x * x) * kInvSqrt2Pi;
  } else {
    const float s = sigmoid(2.f * kSqrt2OverPi * (x + 0.044715f * x * x * x));
    a = x * s;
    const float xc = fminf(fmaxf(x, -16.f), 16.f);  // as in fast_act
    d = s + a * (1.f - s) * (2.f * kSqrt2OverPi) * (1.f + 3.f * 0.044715f * xc * xc);
  }
}

// Two values at once.
template <int ACT, bool FAST>
__device__ __forceinline__ float2 act(float2 x) {
  float2 d;
  if constexpr (FAST) return fast_act<ACT, false>(x, d);
  else return make_float2(act<ACT, false>(x.x), act<ACT, false>(x.y));
}
template <int ACT, bool FAST>
__device__ __forceinline__ void act_grad(float2 x, float2& a, float2& d) {
  if constexpr (FAST) {
    a = fast_act<ACT, true>(x, d);
  } else {
    act_grad<ACT, false>(x.x, a.x, d.x);
    act_grad<ACT, false>(x.y, a.y, d.y);
  }
}

// g act'(x) for act'(x) = d: what the ReLU masks is 0 also where g is an infinity or NaN.
template <int ACT>
__device__ __forceinline__ float2 chain(float2 g, float2 d) {
  if (ACT == LCE_ACT_RELU) return make_float2(d.x != 0.f ? g.x : 0.f, d.y != 0.f ? g.y : 0.f);
  return vmul(g, d);
}

// Calls f(integral_constant<int, activation>) for a run-time activation.
template <int A>
struct ActTag {
  static constexpr int value = A;
};
template <typename F>
__host__ __device__ __forceinline__ void dispatch_act(int a, F&& f) {
  switch (a) {
    case LCE_ACT_RELU: f(ActTag<LCE_ACT_RELU>{}); break;
    case LCE_ACT_SILU: f(ActTag<LCE_ACT_SILU>{}); break;
    case LCE_ACT_GELU: f(ActTag<LCE_ACT_GELU>{}); break;
    case LCE_ACT_GELU_TANH: f(ActTag<LCE_ACT_GELU_TANH>{}); break;
    default: f(ActTag<LCE_ACT_NONE>{});
  }
}

}  // namespace lce
