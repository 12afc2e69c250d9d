// activation.cuh -- the activations of the products with an epilogue (MOE_ACT_*) and their
// derivatives, in binary32.
#pragma once

#include "moe_common.cuh"

namespace moe {
namespace act {

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2).  erfc from Abramowitz &
// Stegun, Handbook of Mathematical Functions, 7.1.26: erfc(x) = (a1 t + .. + a5 t^5) exp(-x^2),
// t = 1 / (1 + p x), x >= 0, off by at most 1.5e-7, which is below bf16's half step of any
// value that counts beside its row; two special-function operations instead of a library erf.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float x = fabsf(z) * 0.70710678f;
  const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
  e = __expf(-x * x);
  float q = fmaf(t, 1.061405429f, -1.453152027f);
  q = fmaf(t, q, 1.421413741f);
  q = fmaf(t, q, -0.284496736f);
  q = fmaf(t, q, 0.254829592f);
  const float tail = 0.5f * q * t * e;           // Phi(-|z|)
  return z < 0.0f ? tail : 1.0f - tail;          // NaN stays NaN through tail
}

// 1 / (1 + exp(-v)); the quotient of an overflowed exponential is 0
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

constexpr float kTanhScale = 0.79788456f;   // sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

template <int kAct>
__device__ __forceinline__ float apply(float z) {
  if (kAct == MOE_ACT_RELU) return z < 0.0f ? 0.0f : z;   // keeps NaN
  if (kAct == MOE_ACT_RELU2) {
    const float r = z < 0.0f ? 0.0f : z;
    return r * r;
  }
  if (kAct == MOE_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  if (kAct == MOE_ACT_GELU_TANH)   // 0.5 (1 + tanh u) = logistic(2 u)
    return z * logistic(2.0f * kTanhScale * z * fmaf(kTanhCube * z, z, 1.0f));
  if (kAct == MOE_ACT_SILU) return z * logistic(z);
  return z;
}

// d act / d z, and act(z)
template <int kAct>
__device__ __forceinline__ float slope(float z, float& y) {
  if (kAct == MOE_ACT_RELU) {
    y = z < 0.0f ? 0.0f : z;
    return z > 0.0f ? 1.0f : 0.0f;
  }
  if (kAct == MOE_ACT_RELU2) {
    const float r = z < 0.0f ? 0.0f : z;
    y = r * r;
    return 2.0f * r;
  }
  if (kAct == MOE_ACT_GELU) {
    float e;
    const float c = normal_cdf(z, e);
    y = z * c;
    return fmaf(z * 0.39894228f, e, c);            // Phi(z) + z phi(z)
  }
  if (kAct == MOE_ACT_GELU_TANH) {
    const float s = logistic(2.0f * kTanhScale * z * fmaf(kTanhCube * z, z, 1.0f));
    y = z * s;
    return fmaf(2.0f * kTanhScale * z * s * (1.0f - s), fmaf(3.0f * kTanhCube * z, z, 1.0f), s);
  }
  if (kAct == MOE_ACT_SILU) {
    const float s = logistic(z);
    y = z * s;
    return s * fmaf(z, 1.0f - s, 1.0f);
  }
  y = z;
  return 1.0f;
}

// f(std::integral_constant<int, activation>) for a run-time activation
template <typename F>
__device__ __forceinline__ void dispatch(int activation, F&& f) {
  switch (activation) {
    case MOE_ACT_RELU: f(std::integral_constant<int, MOE_ACT_RELU>{}); break;
    case MOE_ACT_RELU2: f(std::integral_constant<int, MOE_ACT_RELU2>{}); break;
    case MOE_ACT_GELU: f(std::integral_constant<int, MOE_ACT_GELU>{}); break;
    case MOE_ACT_GELU_TANH: f(std::integral_constant<int, MOE_ACT_GELU_TANH>{}); break;
    case MOE_ACT_SILU: f(std::integral_constant<int, MOE_ACT_SILU>{}); break;
    default: break;
  }
}

}  // namespace act
}  // namespace moe
