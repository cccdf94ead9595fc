// The logistic function of a gate, in a form that keeps products with it right over all of FP32's range.
#pragma once

namespace mfr {

// p = 1 / (1 + exp(-g)) is m * m * r: with h = exp(-|g| / 2), r = 1 / (1 + h * h), which lies in [1/2, 1], and m is 1, or h below
// g = 0.  p alone leaves FP32's normal numbers below g = -87, where its product with a large factor does not: each factor of a
// product takes an m of its own, and no intermediate value is much smaller or larger than the result.
struct Logistic {
  float m, r;
};
__device__ __forceinline__ Logistic logistic(float g) {
  const float h = exp2f(fabsf(g) * -0.72134752f);  // (log2(e) / 2)
  Logistic p;
  p.m = g < 0.0f ? h : 1.0f;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p.r) : "f"(fmaf(h, h, 1.0f)));  // (a NaN stays one)
  return p;
}

// g / (1 + exp(-g)) * u; the first form from kNearGate on, where the quotient stays inside FP32's normal numbers.
constexpr float kNearGate = -80.0f;
__device__ __forceinline__ float swiglu_near(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950409f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r * u;
}
__device__ __forceinline__ float swiglu(float g, float u) {
  const Logistic p = logistic(g);
  return g * p.m * p.r * (u * p.m);
}

// a * b * m * k, m at most 1 and k little more: in an order in which nothing overflows or vanishes on the way unless the result does.
// The larger of a and b takes m.  A smaller one up to 1 can be multiplied in next, since only k follows; above 1 it takes k first.
__device__ __forceinline__ float scaled_product(float a, float b, float m, float k) {
  const bool first = fabsf(a) >= fabsf(b);
  const float t = (first ? a : b) * m, small = first ? b : a;
  return fabsf(small) <= 1.0f ? t * small * k : t * (small * k);
}

}  // namespace mfr
