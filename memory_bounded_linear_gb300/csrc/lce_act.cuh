// The activations of the feed-forward operators and their derivatives, in fp32.
//   relu(x) = max(x, 0)                      silu(x) = x s(x),  s(x) = 1 / (1 + e^-x)
//   gelu(x) = x Phi(x), Phi the normal distribution function
//   gelu_tanh(x) = x (1 + tanh(w)) / 2 = x s(2 w),  w = sqrt(2/pi) (x + 0.044715 x^3)
// FAST (bf16 inputs): the exponential and the quotient are the hardware approximations, whose error of
// a few 2^-22 is far below the rounding of the result to 8 bits, and Phi is a short polynomial; fp32
// inputs take the accurate functions.
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

template <bool FAST>
__device__ __forceinline__ float sigmoid(float x) {
  // x below about -88: e^-x is huge or inf and the quotient 0
  if (FAST) return ptx::rcp_approx(1.f + ptx::ex2_approx(-kLog2e * x));
  return 1.f / (1.f + expf(-x));
}

// Phi(x) and e = exp(-x^2 / 2), for bf16 results.  The upper tail Q(y) = erfc(y / sqrt 2) / 2 is
// e t P(t) / 2 with t = 1 / (1 + 0.46 y / sqrt 2); the degree-5 P was fitted to exp(z^2) erfc(z) / t on
// z >= 0 (least squares in t, reweighted towards the largest relative error, 1.8e-5).  One exponential
// and one quotient serve Phi and the density in its derivative.
__device__ __forceinline__ float normal_cdf(float x, float& e) {
  const float t = ptx::rcp_approx(fmaf(0.46f * kSqrtHalf, fabsf(x), 1.f));
  e = ptx::ex2_approx(-0.5f * kLog2e * x * x);
  float p = 0.5f * -0.12635274f;  // P / 2
  p = fmaf(p, t, 0.5f * 0.24180298f);
  p = fmaf(p, t, 0.5f * 0.12544967f);
  p = fmaf(p, t, 0.5f * 0.24052443f);
  p = fmaf(p, t, 0.5f * 0.25903428f);
  p = fmaf(p, t, 0.5f * 0.25953171f);
  const float q = e * (t * p);
  return x > 0.f ? 1.f - q : q;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act(float x) {
  if constexpr (ACT == LCE_ACT_RELU) return x > 0.f ? x : (x == x ? 0.f : x);
  if constexpr (ACT == LCE_ACT_SILU) return x * sigmoid<FAST>(x);
  if constexpr (ACT == LCE_ACT_GELU) {
    if constexpr (FAST) {
      float e;
      return x * normal_cdf(x, e);
    }
    return 0.5f * x * (1.f + erff(x * kSqrtHalf));
  }
  if constexpr (ACT == LCE_ACT_GELU_TANH)
    return x * sigmoid<FAST>(2.f * kSqrt2OverPi * (x + 0.044715f * x * x * x));
  return x;
}

// a = act(x) and d = act'(x) together (they share their exponential).
template <int ACT, bool FAST>
__device__ __forceinline__ void act_grad(float x, float& a, float& d) {
  if constexpr (ACT == LCE_ACT_RELU) {
    a = x > 0.f ? x : (x == x ? 0.f : x);
    d = x <= 0.f ? 0.f : 1.f;
  } else if constexpr (ACT == LCE_ACT_SILU) {
    const float s = sigmoid<FAST>(x);
    a = x * s;
    d = s + a * (1.f - s);
  } else if constexpr (ACT == LCE_ACT_GELU) {
    float c, e;
    if constexpr (FAST) {
      c = normal_cdf(x, e);
    } else {
      c = 0.5f * (1.f + erff(x * kSqrtHalf));
      e = expf(-0.5f * x * x);
    }
    a = x * c;
    // e is 0 long before x overflows the product
    d = c + x * e * kInvSqrt2Pi;
  } else if constexpr (ACT == LCE_ACT_GELU_TANH) {
    const float s = sigmoid<FAST>(2.f * kSqrt2OverPi * (x + 0.044715f * x * x * x));
    a = x * s;
    // a (1 - s) is 0 from |x| = 16 on, where x^2 must not turn it into 0 inf
    const float xc = fminf(fmaxf(x, -16.f), 16.f);
    d = s + a * (1.f - s) * (2.f * kSqrt2OverPi) * (1.f + 3.f * 0.044715f * xc * xc);
  } else {
    a = x;
    d = 1.f;
  }
}

// g act'(x) for act'(x) = d: what the ReLU masks is 0 also where g is an infinity or NaN.
template <int ACT>
__device__ __forceinline__ float chain(float g, float d) {
  return ACT == LCE_ACT_RELU ? (d != 0.f ? g : 0.f) : g * d;
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
