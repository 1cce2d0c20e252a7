// Activations of the product's epilogue and their slopes, in float32.
//
// Phi(z), the normal distribution's integral that GELU takes, comes from
//   Q(a) = 1 - Phi(a) = E(a) exp(-a^2 / 2),  E(a) = t P(t),  t = 1 / (1 + 0.305 a)   (a >= 0)
// with P the polynomial of degree 7 that makes the largest relative error over
// 0 <= a <= 14 least (9.8e-8 with the constants below; fitted against the scaled
// complementary error function), 4.3e-7 as evaluated in float32.  Beside it stands
// the exponential, whose argument loses 1.5 2^-24 of its size: Q is good to 1.6e-6
// for a <= 8 and 3.8e-6 up to 13, where it leaves float32's normal numbers.  So the
// tail keeps its relative precision, which 1 + erf does not, and the exponential is
// shared with the slope's density.  One reciprocal and one exponential, no branch.
#pragma once

#include "nf4_device.h"

namespace nf4i {

enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

constexpr float kLog2e = 1.44269504088896341f;

// exp(v) where 2^x of the scaled argument is precise enough (|v| up to 88; relative error 1e-5 at most there,
// 2e-7 at |v| <= 1).
__device__ __forceinline__ float exp_fast(float v) { return __builtin_amdgcn_exp2f(v * kLog2e); }

// 1 / (1 + exp(-v)): 0 and 1 at the ends.
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + exp_fast(-v)); }

// exp(-z^2 / 2) and Phi(z).
__device__ __forceinline__ void normal_cdf(float z, float& e, float& phi) {
  const float a = fabsf(z);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.305f, a, 1.0f));
  float p = 0.036699176f;
  p = fmaf(p, t, -0.15298824f);
  p = fmaf(p, t, 0.18571676f);
  p = fmaf(p, t, -0.037976712f);
  p = fmaf(p, t, 0.12102162f);
  p = fmaf(p, t, 0.10342088f);
  p = fmaf(p, t, 0.12246682f);
  p = fmaf(p, t, 0.121639736f);
  e = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e));
  const float q = p * t * e;
  phi = z < 0.0f ? q : 1.0f - q;
}

constexpr float kTanhScale = 0.797884560802865356f;  // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

template <int A>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (A == kActRelu) return z > 0.0f ? z : (z != z ? z : 0.0f);
  if constexpr (A == kActSilu) return z * sigmoid(z);
  if constexpr (A == kActGelu) {
    float e, phi;
    normal_cdf(z, e, phi);
    return z * phi;
  }
  // .5 z (1 + tanh u) = z sigmoid(2 u),  u = sqrt(2 / pi) (z + .044715 z^3)
  if constexpr (A == kActGeluTanh) return z * sigmoid(2.0f * kTanhScale * z * fmaf(kTanhCubic * z, z, 1.0f));
  return z;
}

// Where |z| is large the slope is 0 or 1 and its second term, a product of
// something that overflows and something that vanishes, is left out; NaN stays NaN.
template <int A>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (A == kActRelu) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if constexpr (A == kActSilu) {
    const float s = sigmoid(z);
    const float t = z * s * (1.0f - s);
    return s + (fabsf(z) > 100.0f ? 0.0f : t);
  }
  if constexpr (A == kActGelu) {
    float e, phi;
    normal_cdf(z, e, phi);
    const float t = z * e * 0.398942280401432678f;  // 1 / sqrt(2 pi)
    return phi + (fabsf(z) > 20.0f ? 0.0f : t);
  }
  if constexpr (A == kActGeluTanh) {
    const float zz = z * z;
    const float s = sigmoid(2.0f * kTanhScale * z * fmaf(kTanhCubic, zz, 1.0f));
    const float t = 2.0f * kTanhScale * z * fmaf(3.0f * kTanhCubic, zz, 1.0f) * s * (1.0f - s);
    return s + (fabsf(z) > 20.0f ? 0.0f : t);
  }
  return 1.0f;
}

}  // namespace nf4i
