// act.cuh -- the activations of the a8w8 GEMM's epilogue and their
// derivatives (hq_activation), in f32.  sm_100a only.
//
// sigmoid(x) = 1 / (1 + e^-x) through the hardware exp2 and reciprocal, each
// within 2 ulp.  The tanh form of GELU is z * sigmoid(2u): the same value as
// z/2 (1 + tanh u) without the difference 1 + tanh, which cancels for
// negative u.  The erf form takes Phi(z) = 1/2 erfc(-z / sqrt 2) from
// Abramowitz and Stegun 7.1.26 (Handbook of Mathematical Functions; |error|
// <= 1.5e-7 in erf, so 7.5e-8 in Phi): erfc(x) = (a1 t + .. + a5 t^5) e^-x^2
// with t = 1 / (1 + 0.3275911 x), x >= 0.  Its e^-x^2 is also the density
// that the derivative needs, so both cost one exp2 and one reciprocal.
#pragma once

#include <cstdint>

namespace hq {
namespace {

// hq_activation values
enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

constexpr float kLog2e = 1.44269504f;
constexpr float kTanhC1 = 1.59576912f;               // 2 sqrt(2 / pi)
constexpr float kTanhC2 = 1.59576912f * 0.044715f;

__device__ __forceinline__ float act_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float act_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 1 / (1 + e^-x); 0 and 1 in the limits
__device__ __forceinline__ float act_sigmoid(float x) { return act_rcp(1.0f + act_exp2(-kLog2e * x)); }

// Phi(z) of the standard normal, and e^(-z^2 / 2)
__device__ __forceinline__ float act_phi(float z, float& e) {
  const float x = fabsf(z) * 0.70710678f;
  const float t = act_rcp(fmaf(0.3275911f, x, 1.0f));
  float p = fmaf(t, 1.061405429f, -1.453152027f);
  p = fmaf(t, p, 1.421413741f);
  p = fmaf(t, p, -0.284496736f);
  p = fmaf(t, p, 0.254829592f);
  e = act_exp2(-0.5f * kLog2e * (z * z));
  const float h = 0.5f * (t * p) * e;  // Phi(-|z|)
  return z > 0.0f ? 1.0f - h : h;
}

template <int ACT>
__device__ __forceinline__ float act_forward(float z) {
  if (ACT == kActRelu) return z > 0.0f ? z : (z != z ? z : 0.0f);
  if (ACT == kActGelu) {
    float e;
    return z * act_phi(z, e);
  }
  if (ACT == kActGeluTanh) return z * act_sigmoid(z * fmaf(kTanhC2, z * z, kTanhC1));
  if (ACT == kActSilu) return z * act_sigmoid(z);
  return z;
}

// d act / dz.  With s = 1 / (1 + e) and e = e^-x, the factor s (1 - s) of a
// sigmoid's slope is (e s) s: no difference of nearly equal numbers.  Beyond
// |z| = kLim every derivative is 0 or 1 to within 1e-26, so z is held there
// (NaN passes): e stays finite (kLim = 10 gives x = 87 in the tanh form) and
// no product meets infinity * 0.
template <int ACT>
__device__ __forceinline__ float act_backward(float z) {
  if (ACT == kActRelu) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  constexpr float kLim = ACT == kActGeluTanh ? 10.0f : 64.0f;
  asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %1, %2;\n\tmax.NaN.f32 %0, t, %3;\n\t}" : "=f"(z) : "f"(z), "f"(kLim), "f"(-kLim));
  if (ACT == kActGelu) {
    float e;
    const float phi = act_phi(z, e);
    return fmaf(z * 0.39894228f, e, phi);
  }
  float x = z, zdu = z;  // sigmoid's argument, and z dx/dz
  if (ACT == kActGeluTanh) {
    const float z2 = z * z;
    x = z * fmaf(kTanhC2, z2, kTanhC1);
    zdu = z * fmaf(3.0f * kTanhC2, z2, kTanhC1);
  }
  const float e = act_exp2(-kLog2e * x);
  const float s = act_rcp(1.0f + e);
  return fmaf(zdu * (e * s), s, s);
}

}  // namespace
}  // namespace hq
