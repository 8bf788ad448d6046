// The activations of the feed-forward operators and their derivatives, in
// fp32. Sigmoid and tanh are both taken from one exponential, e^-|y| (never
// overflows), and one reciprocal:
//   sigmoid(x) = 1 / (1 + e^-x),  (1 + tanh u) / 2 = sigmoid(2 u).
// The normal distribution's Phi is taken from e^(-x^2 / 2), which its density
// needs too, by the Chebyshev fit of erfc(z) e^(z^2) in t = 1 / (1 + z / 2) of
// "Numerical Recipes" (erfcc; fractional error below 1.2e-7 everywhere): about
// 20 instructions where the library's erfc takes 60, in kernels that are bound
// by memory otherwise.
#pragma once

#include "common.hpp"

namespace lora4 {

enum Act : int { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3 };

// 1 / (1 + e^-x): e^-|x| in (0, 1], so neither it nor the sum overflows. The
// exponential and the reciprocal are the hardware's (about one unit in the
// last place each, far below the bf16 rounding of what they feed).
__device__ __forceinline__ float sigmoid_f32(float x) {
  const float e = __expf(-fabsf(x));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  return x >= 0.0f ? r : e * r;
}

constexpr float GELU_K = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float GELU_C = 0.044715f;
constexpr float SQRT_HALF = 0.7071067811865476f;
constexpr float INV_SQRT_2PI = 0.3989422804014327f;

// Phi(x) of the normal distribution, with e = e^(-x^2 / 2) given.
__device__ __forceinline__ float normal_cdf_f32(float x, float e) {
  const float z = fabsf(x) * SQRT_HALF;
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.5f * z);
  float q = 0.17087277f;
  q = q * t - 0.82215223f;
  q = q * t + 1.48851587f;
  q = q * t - 1.13520398f;
  q = q * t + 0.27886807f;
  q = q * t - 0.18628806f;
  q = q * t + 0.09678418f;
  q = q * t + 0.37409196f;
  q = q * t + 1.00002368f;
  q = q * t - 1.26551223f;
  const float half_erfc = 0.5f * t * e * __expf(q);   // Phi(-|x|)
  return x >= 0.0f ? 1.0f - half_erfc : half_erfc;
}

// act(x). An infinite x gives the limit: x at +inf; at -inf 0 (the finite
// factor is taken first, so no 0 * inf).
__device__ __forceinline__ float act_value(float x, int act) {
  if (act == ACT_NONE) return x;
  float p;
  if (act == ACT_SILU) p = sigmoid_f32(x);
  else if (act == ACT_GELU) p = normal_cdf_f32(x, __expf(-0.5f * x * x));
  else p = sigmoid_f32(2.0f * GELU_K * (x + GELU_C * x * x * x));
  return p == 0.0f ? 0.0f : x * p;
}

// Eight values at once; the choice of activation is outside the loop.
__device__ __forceinline__ void act_value8(float (&v)[8], int act) {
  if (act == ACT_SILU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = act_value(v[e], ACT_SILU);
  } else if (act == ACT_GELU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = act_value(v[e], ACT_GELU);
  } else if (act == ACT_GELU_TANH) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = act_value(v[e], ACT_GELU_TANH);
  }
}

// act(x) and act'(x).
__device__ __forceinline__ void act_value_slope(float x, int act, float &v, float &d) {
  if (act == ACT_NONE) {
    v = x;
    d = 1.0f;
    return;
  }
  float p, xdp;   // act(x) = x p(x); xdp = x p'(x)
  if (act == ACT_SILU) {
    p = sigmoid_f32(x);
    const float q = p * sigmoid_f32(-x);   // p (1 - p), without cancellation
    xdp = q == 0.0f ? 0.0f : x * q;
  } else if (act == ACT_GELU) {
    const float e = __expf(-0.5f * x * x);
    p = normal_cdf_f32(x, e);
    const float q = INV_SQRT_2PI * e;
    xdp = q == 0.0f ? 0.0f : x * q;
  } else {
    const float u2 = 2.0f * GELU_K * (x + GELU_C * x * x * x);
    p = sigmoid_f32(u2);
    const float q = p * sigmoid_f32(-u2);
    xdp = q == 0.0f ? 0.0f : x * q * (2.0f * GELU_K) * (1.0f + 3.0f * GELU_C * x * x);
  }
  v = p == 0.0f ? 0.0f : x * p;
  d = p + xdp;
}

}  // namespace lora4
