// Activations of two fp32 accumulator values at a time, and their derivatives.
#pragma once

#include "common.cuh"

namespace dmoe {
namespace act {

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float2 f2_splat(float v) { return make_float2(v, v); }

__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The exact (erf) GELU, gelu(x) = x Phi(x), and its derivative
// gelu'(x) = Phi(x) + x phi(x), of two accumulator values with packed
// arithmetic.  Phi comes from the erfc approximation of Abramowitz & Stegun,
// Handbook of Mathematical Functions, formula 7.1.26 (|error| <= 1.5e-7; of
// Phi(x) itself 0.05% at x = -4, 0.36% at -6, 1% at -8):
//   erfc(z) ~= t (a1 + t (a2 + t (a3 + t (a4 + t a5)))) exp(-z^2),
//   t = 1 / (1 + p z),  z = |x| / sqrt(2) >= 0,
// with the coefficients halved so that the product is Phi(-|x|) directly.
// exp(-z^2) = exp(-x^2 / 2) = 2^(-x^2 log2(e) / 2) also gives the density
// phi(x) = exp(-x^2 / 2) / sqrt(2 pi).  Phi(x) = 1 - Phi(-|x|) for x >= 0
// and Phi(-|x|) for x < 0, chosen by a select (no cancellation in the left
// tail).
__device__ __forceinline__ void gelu_pair(float2 x, float2& gelu, float2& dgelu) {
  const float2 ax = make_float2(fabsf(x.x), fabsf(x.y));
  const float2 u = f2_fma(ax, f2_splat(0.3275911f * 0.70710678118654752f), f2_splat(1.f));
  const float2 t = make_float2(rcp_approx(u.x), rcp_approx(u.y));
  float2 q = f2_fma(t, f2_splat(0.5f * 1.061405429f), f2_splat(0.5f * -1.453152027f));
  q = f2_fma(t, q, f2_splat(0.5f * 1.421413741f));
  q = f2_fma(t, q, f2_splat(0.5f * -0.284496736f));
  q = f2_fma(t, q, f2_splat(0.5f * 0.254829592f));
  q = f2_mul(q, t);
  const float2 s = f2_mul(f2_mul(x, x), f2_splat(-0.5f * 1.44269504088896341f));
  const float2 e = make_float2(ex2_approx(s.x), ex2_approx(s.y));
  const float2 h = f2_mul(q, e);                                  // Phi(-|x|)
  const float2 omh = f2_fma(h, f2_splat(-1.f), f2_splat(1.f));     // 1 - Phi(-|x|)
  const float2 cdf = make_float2(x.x < 0.f ? h.x : omh.x, x.y < 0.f ? h.y : omh.y);
  dgelu = f2_fma(f2_mul(x, f2_splat(0.39894228040143268f)), e, cdf);  // Phi + x phi
  gelu = f2_mul(x, cdf);
}

// silu(x) = x sigmoid(x) and silu'(x) = sigmoid(x) (1 + x (1 - sigmoid(x))).
__device__ __forceinline__ void silu_pair(float2 x, float2& silu, float2& dsilu) {
  const float2 q = f2_mul(x, f2_splat(-1.44269504088896341f));
  const float2 s = make_float2(rcp_approx(1.f + ex2_approx(q.x)), rcp_approx(1.f + ex2_approx(q.y)));
  const float2 rest = f2_fma(s, f2_splat(-1.f), f2_splat(1.f));
  dsilu = f2_mul(s, f2_fma(x, rest, f2_splat(1.f)));
  silu = f2_mul(x, s);
}

}  // namespace act
}  // namespace dmoe
