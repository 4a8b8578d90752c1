// gelu2.cuh -- GeLU in its exact form and its derivative, two values at a time.
//
// With u = |x|, t = 1 / (1 + p u / sqrt 2) and e = exp(-u^2 / 2), Abramowitz & Stegun, Handbook of Mathematical
// Functions, formula 7.1.26 gives the upper tail of the normal distribution Q(u) = (1 - erf(u / sqrt 2)) / 2 = g e,
// g = (a1 t + a2 t^2 + a3 t^3 + a4 t^4 + a5 t^5) / 2, with |error| <= 7.5e-8.  So
//   x Phi(x) = max(x, 0) - u g e,     Phi(x) + x phi(x) = [x > 0] + e (x / sqrt(2 pi) - sign(x) g).
// u is cut at 64, where e is 0 already, so that infinities have their limits; NaN stays NaN.  8.5 issue slots and two
// special-function operations a value: half of a scalar evaluation through Phi.
#pragma once
#include "f32x2.cuh"

namespace dm {

__device__ __forceinline__ float gelu_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float gelu_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// max(a, b) that keeps NaN (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// g and e of u0, u1 >= 0.
__device__ __forceinline__ void normal_tail_f2(float u0, float u1, uint64_t& g, uint64_t& e) {
  const uint64_t u = f2(u0, u1);
  float d0, d1, s0, s1;
  f2_split(fma_f2(u, f2(0.23164188f, 0.23164188f), f2(1.0f, 1.0f)), d0, d1);
  f2_split(mul_f2(mul_f2(u, u), f2(-0.72134752f, -0.72134752f)), s0, s1);  // log2(exp(-u^2 / 2))
  const uint64_t t = f2(gelu_rcp(d0), gelu_rcp(d1));
  e = f2(gelu_ex2(s0), gelu_ex2(s1));
  uint64_t q = fma_f2(t, f2(0.5307027145f, 0.5307027145f), f2(-0.7265760135f, -0.7265760135f));
  q = fma_f2(t, q, f2(0.7107068705f, 0.7107068705f));
  q = fma_f2(t, q, f2(-0.142248368f, -0.142248368f));
  q = fma_f2(t, q, f2(0.127414796f, 0.127414796f));
  g = mul_f2(t, q);
}

__device__ __forceinline__ void gelu_f2(float x0, float x1, float& y0, float& y1) {
  const float u0 = min_nan(fabsf(x0), 64.0f), u1 = min_nan(fabsf(x1), 64.0f);
  uint64_t g, e;
  normal_tail_f2(u0, u1, g, e);
  f2_split(fma_f2(mul_f2(f2(-u0, -u1), e), g, f2(fmaxf(x0, 0.0f), fmaxf(x1, 0.0f))), y0, y1);
}

__device__ __forceinline__ void gelu_grad_f2(float x0, float x1, float& d0, float& d1) {
  const float u0 = min_nan(fabsf(x0), 64.0f), u1 = min_nan(fabsf(x1), 64.0f);
  uint64_t g, e;
  normal_tail_f2(u0, u1, g, e);
  float g0, g1;
  f2_split(fma_f2(f2(u0, u1), f2(-0.39894228f, -0.39894228f), g), g0, g1);  // x > 0: 1 - e (g - u phi(0)), else e (g - u phi(0))
  const bool up0 = x0 > 0.0f, up1 = x1 > 0.0f;
  f2_split(fma_f2(f2(up0 ? -g0 : g0, up1 ? -g1 : g1), e, f2(up0 ? 1.0f : 0.0f, up1 ? 1.0f : 0.0f)), d0, d1);
}

}  // namespace dm
