// activation.cuh -- the activations of the products with an epilogue (MOE_ACT_*) and their
// derivatives, in binary32.
#pragma once

#include "moe_common.cuh"
#include "sm100_ptx_fp8.cuh"

namespace moe {
namespace act {

constexpr float kTanhScale = 0.79788456f;   // sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

// act(z) and d act / d z of two values at once, in pairs of f32 (one instruction for both of a pair's
// additions, multiplications and multiply-adds): their instructions bound the epilogue's gradient
// (70.7 us with single values, 51.2 with pairs and four rows in flight; 32768 x 768, GELU).
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t each(float (*f)(float), uint64_t v) {
  const float2 u = ptx::unpair(v);
  return ptx::pair(__float_as_uint(f(u.x)), __float_as_uint(f(u.y)));
}
__device__ __forceinline__ float exp2_fast(float v) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
  return y;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
  return y;
}
constexpr float kLog2e = 1.44269504f;

// 1 / (1 + 2^v): the logistic function of -v / log2(e)
__device__ __forceinline__ uint64_t logistic2(uint64_t v) {
  return each(rcp_fast, add2(each(exp2_fast, v), ptx::pair(1.0f)));
}

template <int kAct>
__device__ __forceinline__ void slope2(uint64_t z, uint64_t& y, uint64_t& s) {
  using ptx::fma2;
  using ptx::mul2;
  using ptx::pair;
  if (kAct == MOE_ACT_RELU || kAct == MOE_ACT_RELU2) {
    const float2 u = ptx::unpair(z);
    const float a = u.x < 0.0f ? 0.0f : u.x, b = u.y < 0.0f ? 0.0f : u.y;       // keeps NaN
    const uint64_t r = pair(__float_as_uint(a), __float_as_uint(b));
    if (kAct == MOE_ACT_RELU) {
      y = r;
      s = pair(__float_as_uint(u.x > 0.0f ? 1.0f : 0.0f), __float_as_uint(u.y > 0.0f ? 1.0f : 0.0f));
    } else {
      y = mul2(r, r);
      s = add2(r, r);
    }
  } else if (kAct == MOE_ACT_GELU) {
    // Phi(-|z|) = (c1 t + .. + c6 t^6) exp(-z^2 / 2), t = 1 / (1 + p |z|): the form of Abramowitz & Stegun,
    // Handbook of Mathematical Functions, 7.1.26, with coefficients fitted here (least squares, reweighted towards
    // the largest error) so that the series is off by at most 0.7e-7 and by 2^-14 of Phi(-|z|), as far as exp's
    // range goes: theirs holds the first bound only and has no digit left at z = -5.25.  A negative z takes the tail
    // as it is (1/2 - (1/2 - tail) would cut it off), a positive one what is left of 1.  With the roundings
    // Phi is off by at most 3e-7, and below z = -4 by 2^-14 of itself.
    const uint64_t x = z & 0x7FFFFFFF7FFFFFFFull;
    const uint64_t t = each(rcp_fast, fma2(x, pair(0.292f), pair(1.0f)));
    const uint64_t e = each(exp2_fast, mul2(mul2(z, z), pair(-0.5f * kLog2e)));
    uint64_t q = fma2(t, pair(-0.086436026f), pair(0.2696572f));
    q = fma2(t, q, pair(-0.0747589f));
    q = fma2(t, q, pair(0.16993603f));
    q = fma2(t, q, pair(0.10418754f));
    q = fma2(t, q, pair(0.11741414f));
    const uint64_t tail = mul2(mul2(q, t), e);
    const float2 u = ptx::unpair(z), lo = ptx::unpair(tail), hi = ptx::unpair(fma2(tail, pair(-1.0f), pair(1.0f)));
    const uint64_t phi = pair(__float_as_uint(u.x < 0.0f ? lo.x : hi.x), __float_as_uint(u.y < 0.0f ? lo.y : hi.y));
    y = mul2(z, phi);
    s = fma2(mul2(z, pair(0.39894228f)), e, phi);            // Phi(z) + z phi(z)
  } else if (kAct == MOE_ACT_GELU_TANH) {
    const uint64_t zz = mul2(z, z);
    const uint64_t p = logistic2(mul2(mul2(z, pair(-2.0f * kTanhScale * kLog2e)), fma2(zz, pair(kTanhCube), pair(1.0f))));
    y = mul2(z, p);
    // p + 2 c z p (1 - p) (1 + 3 b z^2), z^2 last: beyond 2^64 it is infinite, where p (1 - p) is 0
    const uint64_t d = mul2(y, fma2(p, pair(-1.0f), pair(1.0f)));
    s = fma2(fma2(mul2(mul2(d, z), z), pair(3.0f * kTanhCube), d), pair(2.0f * kTanhScale), p);
  } else if (kAct == MOE_ACT_SILU) {
    const uint64_t p = logistic2(mul2(z, pair(-kLog2e)));
    y = mul2(z, p);
    s = fma2(y, fma2(p, pair(-1.0f), pair(1.0f)), p);        // p + z p (1 - p)
  } else {
    y = z;
    s = pair(1.0f);
  }
}

// act of a pair (what of slope2 its result does not need is not computed)
template <int kAct>
__device__ __forceinline__ uint64_t apply2(uint64_t z) {
  uint64_t y, s;
  slope2<kAct>(z, y, s);
  return y;
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
