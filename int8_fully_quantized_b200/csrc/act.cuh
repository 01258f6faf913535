// Device-side activation functions shared by the standalone non-linear kernels and the GEMM epilogue.
#pragma once
#include "kernels.h"  // GemmAct
#include "quant.cuh"  // fma_x2

namespace jf {

// erfc(z) for z >= 0 by the Chebyshev fit of Numerical Recipes (Press, Teukolsky, Vetterling and
// Flannery, 2nd ed., section 6.2, "erfcc"): erfc(z) = t exp(-z^2 + P(t)), t = 1 / (1 + z / 2), with a
// fractional error below 1.2e-7 everywhere in exact arithmetic; in fp32 the exponent's rounding adds
// a relative error of about z^2 * 2^-24 (below 5e-6 where erfc is still a normal float).
__device__ __forceinline__ float erfc_nonneg(float z) {
  const float t = __frcp_rn(fmaf(0.5f, z, 1.0f));
  float p = 0.17087277f;
  p = fmaf(p, t, -0.82215223f);
  p = fmaf(p, t, 1.48851587f);
  p = fmaf(p, t, -1.13520398f);
  p = fmaf(p, t, 0.27886807f);
  p = fmaf(p, t, -0.18628806f);
  p = fmaf(p, t, 0.09678418f);
  p = fmaf(p, t, 0.37409196f);
  p = fmaf(p, t, 1.00002368f);
  p = fmaf(p, t, -1.26551223f);
  return t * expf(fmaf(-z, z, p));
}

// erfc_nonneg of two arguments, the Horner chain of both in packed fp32x2 FMAs (each lane rounded
// as fmaf): results bit-identical to two erfc_nonneg calls, in fewer issue slots.
__device__ __forceinline__ void erfc_nonneg_x2(float z0, float z1, float& e0, float& e1) {
  const float t0 = __frcp_rn(fmaf(0.5f, z0, 1.0f)), t1 = __frcp_rn(fmaf(0.5f, z1, 1.0f));
  constexpr float c[10] = {0.17087277f, -0.82215223f, 1.48851587f, -1.13520398f, 0.27886807f,
                           -0.18628806f, 0.09678418f, 0.37409196f, 1.00002368f, -1.26551223f};
  float p0 = c[0], p1 = c[0];
#pragma unroll
  for (int i = 1; i < 10; ++i) fma_x2(p0, p1, t0, t1, c[i], c[i], p0, p1);
  float a0, a1;
  fma_x2(-z0, -z1, z0, z1, p0, p1, a0, a1);
  e0 = t0 * expf(a0);
  e1 = t1 * expf(a1);
}

// GELU(x) = x Phi(x) = 0.5 x (1 + erf(x / sqrt 2)), the exact (erf) form, evaluated through
// e = erfc(|x| / sqrt 2): GELU(x) = 0.5 x (2 - e) for x >= 0 and 0.5 x e for x < 0 (the erfc form
// keeps its relative accuracy for negative x, where 1 + erf cancels).
__device__ __forceinline__ float gelu_f32(float x) {
  const float e = erfc_nonneg(fabsf(x) * 0.70710678118654752440f);
  return 0.5f * x * (x >= 0.0f ? 2.0f - e : e);
}

// GELU'(x) = Phi(x) + x phi(x), with Phi(x) = 0.5 erfc(-x / sqrt 2) and phi(x) = exp(-x^2 / 2) / sqrt(2 pi).
// For x -> -inf both terms vanish (the sum is about phi(x) (1/|x| - |x|), no cancellation that matters).
__device__ __forceinline__ float gelu_grad_f32(float x) {
  const float e = erfc_nonneg(fabsf(x) * 0.70710678118654752440f);
  const float Phi = 0.5f * (x >= 0.0f ? 2.0f - e : e);
  return fmaf(x * 0.39894228040143267794f, expf(-0.5f * x * x), Phi);
}

// GELU'(x) and GELU'(-x) for x >= 0 from one erfc and one exp: Phi(-x) = 1 - Phi(x) and phi is even,
// so both share e = erfc(x / sqrt 2) and exp(-x^2 / 2). Each result is bit-identical to
// gelu_grad_f32 of the same argument (the sign flips involved are exact).
__device__ __forceinline__ void gelu_grad_pair_f32(float x, float& at_pos, float& at_neg) {
  const float e = erfc_nonneg(x * 0.70710678118654752440f);
  const float ex = expf(-0.5f * x * x);
  const float xc = x * 0.39894228040143267794f;
  at_pos = fmaf(xc, ex, 0.5f * (2.0f - e));
  at_neg = fmaf(-xc, ex, 0.5f * e);
}

// gelu_f32 of two values, the erfc chains packed (bit-identical to two gelu_f32 calls).
__device__ __forceinline__ void gelu_f32_x2(float& x0, float& x1) {
  float e0, e1;
  erfc_nonneg_x2(fabsf(x0) * 0.70710678118654752440f, fabsf(x1) * 0.70710678118654752440f, e0, e1);
  x0 = 0.5f * x0 * (x0 >= 0.0f ? 2.0f - e0 : e0);
  x1 = 0.5f * x1 * (x1 >= 0.0f ? 2.0f - e1 : e1);
}

// The hardware's approximate reciprocal (1 ulp) and power of two (2 ulp; results below 2^-126 become 0).
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634074f;

// GELU of two values for the linear layers' epilogues, where the activation competes for issue slots with
// the product itself: erfc_nonneg's fit with the approximate reciprocal and power of two (14 instructions
// a value against 22), GELU(x) = max(x, 0) - |x e / 2|. The exponent -z^2 + P, z = |x| / sqrt 2, carries the roundings of
// z (its constant's and its own, twice: z^2), of the sum and of the product with log2 e, each z^2 2^-24, which are e's
// relative error: measured 1.5e-6 at most for |x| < 3, 5.6e-6 below 7, 8.1e-6 below 9.
__device__ __forceinline__ void gelu_epilogue_x2(float& x0, float& x1) {
  constexpr float c[10] = {0.17087277f, -0.82215223f, 1.48851587f, -1.13520398f, 0.27886807f,
                           -0.18628806f, 0.09678418f, 0.37409196f, 1.00002368f, -1.26551223f};
  float z0, z1, t0, t1, p0 = c[0], p1 = c[0], h0, h1;
  mul_x2(fabsf(x0), fabsf(x1), 0.70710678118654752440f, 0.70710678118654752440f, z0, z1);
  fma_x2(z0, z1, 0.5f, 0.5f, 1.0f, 1.0f, t0, t1);
  t0 = rcp_approx(t0);
  t1 = rcp_approx(t1);
#pragma unroll
  for (int i = 1; i < 10; ++i) fma_x2(p0, p1, t0, t1, c[i], c[i], p0, p1);
  fma_x2(-z0, -z1, z0, z1, p0, p1, p0, p1);
  fma_x2(p0, p1, kLog2e, kLog2e, -1.0f, -1.0f, p0, p1);   // e / 2
  // e is 0 from x = 32 on; held there, the factor of an infinite x does not make its product with 0 a NaN
  mul_x2(fminf(x0, 32.0f), fminf(x1, 32.0f), t0, t1, h0, h1);
  mul_x2(h0, h1, exp2_approx(p0), exp2_approx(p1), h0, h1);
  x0 = fmaxf(x0, 0.0f) - fabsf(h0);
  x1 = fmaxf(x1, 0.0f) - fabsf(h1);
}

// SiLU(x) = x / (1 + exp(-x)). The power overflows to infinity for very negative x, where the quotient is 0.
__device__ __forceinline__ float silu_f32(float x) { return x * rcp_approx(1.0f + exp2_approx(-kLog2e * x)); }

// The tanh form of GELU, 0.5 x (1 + tanh u) with u = sqrt(2 / pi) (x + 0.044715 x^3). Since
// 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)), it is evaluated as x / (1 + exp(-2 u)), which does not cancel.
constexpr float kGeluTanhC0 = 1.5957691216057307117f;                  // 2 sqrt(2 / pi)
constexpr float kGeluTanhC1 = 1.5957691216057307117f * 0.044715f;
__device__ __forceinline__ float gelu_tanh_f32(float x) {
  return x * rcp_approx(1.0f + exp2_approx(-x * fmaf(kLog2e * kGeluTanhC1, x * x, kLog2e * kGeluTanhC0)));
}

// act'(x) and act'(-x) for x >= 0 of every activation of the linear layers' epilogues, with the approximate
// functions. Both sides are formed from the same two small terms, never as 1 minus the other: act'(-x) keeps its
// relative accuracy where it vanishes (a block of strongly negative pre-activations takes its INT8 scale from it).
// GELU: Phi(x) + x phi(x) with e = erfc(x / sqrt 2) of erfc_nonneg's fit: 1 - e / 2 + x phi and e / 2 - x phi.
// The logistic ones, act = x sigmoid(z(x)) with z odd, from t = exp(-z) <= 1, r = 1 / (1 + t) = sigmoid(z) and
// t r = sigmoid(-z): r + x z' t r^2 and t r - x z' t r^2. Beyond x = 20 the tanh form's are 1 and 0.
__device__ __forceinline__ void act_grad_pair_epilogue(float x, int act, float& at_pos, float& at_neg) {
  if (act == kActRelu) {
    at_pos = x > 0.0f ? 1.0f : 0.0f;
    at_neg = 0.0f;
    return;
  }
  if (act == kActGeluEpi) {
    constexpr float c[10] = {0.17087277f, -0.82215223f, 1.48851587f, -1.13520398f, 0.27886807f,
                             -0.18628806f, 0.09678418f, 0.37409196f, 1.00002368f, -1.26551223f};
    const float z = x * 0.70710678118654752440f;
    const float t = rcp_approx(fmaf(0.5f, z, 1.0f));
    float p = c[0];
#pragma unroll
    for (int i = 1; i < 10; ++i) p = fmaf(p, t, c[i]);
    const float h = -0.5f * x;
    const float e = t * exp2_approx(kLog2e * fmaf(h, x, p)), xphi = x * 0.39894228040143267794f * exp2_approx(kLog2e * h * x);
    at_pos = fmaf(-0.5f, e, 1.0f) + xphi;
    at_neg = fmaf(0.5f, e, -xphi);
    return;
  }
  float z = x, dz = 1.0f;
  if (act == kActGeluTanh) {
    x = fminf(x, 20.0f);
    z = x * fmaf(kGeluTanhC1, x * x, kGeluTanhC0);
    dz = fmaf(3.0f * kGeluTanhC1, x * x, kGeluTanhC0);
  }
  const float t = exp2_approx(-kLog2e * z), r = rcp_approx(1.0f + t), u = t * r;
  at_pos = fmaf(x * dz, u * r, r);
  at_neg = fmaf(-x * dz, u * r, u);
}

}  // namespace jf
