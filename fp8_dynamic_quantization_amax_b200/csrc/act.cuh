// act.cuh -- the activations of the a8w8 GEMM's epilogue and their
// derivatives (hq_activation), in f32, two elements at a time.  sm_100a only.
//
// sigmoid(x) = 1 / (1 + e^-x) through the hardware exp2 and reciprocal, each
// within 2 ulp.  The tanh form of GELU is z * sigmoid(2u): the same value as
// z/2 (1 + tanh u) without the difference 1 + tanh, which cancels for
// negative u.
//
// The erf form, with a = |z| and e = e^(-z^2 / 2):
//   gelu(z)  = max(z, 0) - a e P(a),  P(a) ~ erfcx(a / sqrt 2) / 2
//   gelu'(z) = e Q(a) for z < 0, 1 - e Q(a) for z > 0,
//              Q(a) ~ P(a) - a / sqrt(2 pi)
// (Phi(-a) = e erfcx(a / sqrt 2) / 2, and the density is e / sqrt(2 pi)).
// P and Q are polynomials on [0, 5.6] (Phi(-5.6) = 1.1e-8; a is held there),
// fitted by iteratively reweighted least squares in Chebyshev form to the
// smallest maximum of e |error|; the figures are of the coefficients as they
// stand, in f32.  P has degree 11 (3.0e-8), for the value's small results at
// negative z (4e-4 of itself at z = -4).  Q, whose slope is O(1), has two
// forms.  Gradients in f32 take degree 12 with Q(0) = 1/2 exact (1.1e-8): over
// z ~ 1.5 N(0, 1) the slope is off by 4.5e-8 of its norm, plain f32 erf and exp
// by 4.2e-8.  Gradients in bf16 and f16 take degree 9 (2.7e-7; their half steps
// are 3.9e-3 and 4.9e-4).  At bf16's memory rate the backward kernel has 28
// cycles per warp-wide element, at f32's 50.  A rational form (Abramowitz and
// Stegun 7.1.26) has fewer terms but a reciprocal more, and the
// special-function unit takes 8 cycles of its quarter of an SM for a warp's
// exp2 or reciprocal.
#pragma once

#include "elem.cuh"

#include <cstdint>

namespace hq {
namespace {

// hq_activation values
enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

constexpr float kLog2e = 1.44269504f;
constexpr float kTanhC1 = 1.59576912f;               // 2 sqrt(2 / pi)
constexpr float kTanhC2 = 1.59576912f * 0.044715f;
constexpr float kPhiEnd = 5.6f;                       // Phi(-5.6) = 1.1e-8

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
__device__ __forceinline__ float2 act_both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 act_rcp2(float2 x) { return make_float2(act_rcp(x.x), act_rcp(x.y)); }
__device__ __forceinline__ float2 act_exp2_2(float2 x) { return make_float2(act_exp2(x.x), act_exp2(x.y)); }
// 1 / (1 + e^-x); 0 and 1 in the limits
__device__ __forceinline__ float2 act_sigmoid2(float2 x) {
  return act_rcp2(f2_add(act_exp2_2(f2_mul(x, act_both(-kLog2e))), act_both(1.0f)));
}

// |z| up to kPhiEnd, and e^(-z^2 / 2): 0 at infinity, NaN at NaN
__device__ __forceinline__ float2 act_gauss(float2 z, float2& e) {
  e = act_exp2_2(f2_mul(f2_mul(z, z), act_both(-0.5f * kLog2e)));
  return make_float2(fminf(fabsf(z.x), kPhiEnd), fminf(fabsf(z.y), kPhiEnd));
}

__device__ __forceinline__ float act_relu(float z) { return z > 0.0f ? z : (z != z ? z : 0.0f); }

template <int ACT>
__device__ __forceinline__ float2 act_forward(float2 z) {
  if (ACT == kActRelu) return make_float2(act_relu(z.x), act_relu(z.y));
  if (ACT == kActGelu) {
    float2 e;
    const float2 a = act_gauss(z, e);
    float2 q = f2_fma(act_both(-3.1554319e-07f), a, act_both(7.7087816e-06f));
    q = f2_fma(q, a, act_both(-8.4771018e-05f));
    q = f2_fma(q, a, act_both(0.000563652837f));
    q = f2_fma(q, a, act_both(-0.00259009073f));
    q = f2_fma(q, a, act_both(0.00900384784f));
    q = f2_fma(q, a, act_both(-0.0254718177f));
    q = f2_fma(q, a, act_both(0.0619239323f));
    q = f2_fma(q, a, act_both(-0.13280578f));
    q = f2_fma(q, a, act_both(0.249972567f));
    q = f2_fma(q, a, act_both(-0.398940593f));
    q = f2_fma(q, a, act_both(0.49999997f));
    const float2 t = f2_mul(e, a);  // NaN where z is
    return f2_fma(make_float2(-t.x, -t.y), q, make_float2(fmaxf(z.x, 0.0f), fmaxf(z.y, 0.0f)));
  }
  if (ACT == kActGeluTanh)
    return f2_mul(z, act_sigmoid2(f2_mul(z, f2_fma(act_both(kTanhC2), f2_mul(z, z), act_both(kTanhC1)))));
  if (ACT == kActSilu) return f2_mul(z, act_sigmoid2(z));
  return z;
}

// z held in [-lim, lim]: the smaller of |z| and lim with z's sign; NaN passes
__device__ __forceinline__ float act_clamp(float z, float lim) {
  float r;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(lim));
  return r;
}

// d act / dz.  With s = 1 / (1 + e) and e = e^-x, the factor s (1 - s) of a
// sigmoid's slope is (e s) s: no difference of nearly equal numbers.  Beyond
// |z| = lim every derivative is 0 or 1 to within 1e-7 (1e-26 in the sigmoid
// forms), so z is held there (NaN passes): e stays finite (lim = 10 gives
// x = 87 in the tanh form) and no product meets infinity * 0.
// F32: the result stays in f32 (the erf form's polynomial, above).
template <int ACT, bool F32>
__device__ __forceinline__ float2 act_backward(float2 z) {
  if (ACT == kActRelu)
    return make_float2(z.x > 0.0f ? 1.0f : (z.x != z.x ? z.x : 0.0f), z.y > 0.0f ? 1.0f : (z.y != z.y ? z.y : 0.0f));
  if (ACT == kActGelu) {
    float2 e;
    const float2 a = act_gauss(z, e);
    float2 q;
    if (F32) {
      q = f2_fma(act_both(5.99616286e-08f), a, act_both(-1.63705761e-06f));
      q = f2_fma(q, a, act_both(2.02306855e-05f));
      q = f2_fma(q, a, act_both(-0.000151731801f));
      q = f2_fma(q, a, act_both(0.000786682474f));
      q = f2_fma(q, a, act_both(-0.00307194889f));
      q = f2_fma(q, a, act_both(0.00968592428f));
      q = f2_fma(q, a, act_both(-0.0260962807f));
      q = f2_fma(q, a, act_both(0.0622803979f));
      q = f2_fma(q, a, act_both(-0.132924139f));
      q = f2_fma(q, a, act_both(0.249992698f));
      q = f2_fma(q, a, act_both(-0.797884226f));
      q = f2_fma(q, a, act_both(0.5f));
    } else {
      q = f2_fma(act_both(-8.06304979e-06f), a, act_both(0.000151941553f));
      q = f2_fma(q, a, act_both(-0.00127115997f));
      q = f2_fma(q, a, act_both(0.00638279831f));
      q = f2_fma(q, a, act_both(-0.0222308636f));
      q = f2_fma(q, a, act_both(0.059496779f));
      q = f2_fma(q, a, act_both(-0.131772876f));
      q = f2_fma(q, a, act_both(0.249752298f));
      q = f2_fma(q, a, act_both(-0.797864914f));
      q = f2_fma(q, a, act_both(0.499999732f));
    }
    // 1/2 +- (1/2 - e Q), the sign that of z
    const float2 d = f2_fma(make_float2(-e.x, -e.y), q, act_both(0.5f));
    return f2_add(make_float2(copysignf(d.x, z.x), copysignf(d.y, z.y)), act_both(0.5f));
  }
  constexpr float kLim = ACT == kActGeluTanh ? 10.0f : 64.0f;
  z = make_float2(act_clamp(z.x, kLim), act_clamp(z.y, kLim));
  float2 x = z, zdu = z;  // sigmoid's argument, and z dx/dz
  if (ACT == kActGeluTanh) {
    const float2 z2 = f2_mul(z, z);
    x = f2_mul(z, f2_fma(act_both(kTanhC2), z2, act_both(kTanhC1)));
    zdu = f2_mul(z, f2_fma(act_both(3.0f * kTanhC2), z2, act_both(kTanhC1)));
  }
  const float2 e = act_exp2_2(f2_mul(x, act_both(-kLog2e)));
  const float2 s = act_rcp2(f2_add(e, act_both(1.0f)));
  return f2_fma(zdu, f2_mul(f2_mul(e, s), s), s);
}

}  // namespace
}  // namespace hq
