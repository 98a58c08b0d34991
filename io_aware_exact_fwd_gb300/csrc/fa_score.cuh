// Device pieces shared by the scored-attention kernels: the mask's intervals and the
// tanh cap.
#pragma once

#include <stdint.h>

#include "fa_device.cuh"
#include "fa_internal.h"

namespace fa {

// The interval of keys that query i sees, and of queries that see key j.  Clamped to the
// row: a plan made for longer rows gives a wrong mask, but no position outside the tensors.
__device__ __forceinline__ int2 in_row(int2 x, int N) { return make_int2(min(max(x.x, 0), N), min(max(x.y, 0), N)); }
__device__ __forceinline__ int2 keys_of(const MaskPlan& p, int causal, int b, int i, int N) {
  if (p.q) return in_row(__ldg(p.q + static_cast<size_t>(b) * N + i), N);
  return make_int2(0, causal ? i + 1 : N);
}
__device__ __forceinline__ int2 queries_of(const MaskPlan& p, int causal, int b, int j, int N) {
  if (p.k) return in_row(__ldg(p.k + static_cast<size_t>(b) * N + j), N);
  return make_int2(causal ? j : 0, N);
}

// Bits a .. e - 1 of 32 (a and e clamped to [0, 32]).
__device__ __forceinline__ uint32_t bits_between(int a, int e) {
  a = min(max(a, 0), 32);
  e = min(max(e, 0), 32);
  return static_cast<uint32_t>((1ull << e) - 1ull) & ~static_cast<uint32_t>((1ull << a) - 1ull);
}

// tanh for the cap.  A capped score is softcap * tanh(u); tanh.approx, off by up to
// 2^-11 relative, would move scores by up to hundredths and their weights by percents.
// The kernels work with x = 4 u, whose bits say which of two forms applies: |x| < 2
// exactly when bit 30 of the fp32 is clear (it is set in infinities and NaN too), so one
// OR over a thread's values finds whether any |u| reaches 1/2.
//
// |u| < 1/2: u p(u^2) with p of degree 3 of the smallest relative error on [0, 1/4]
// (5.4e-7, found by linear programming on 4001 points; the score is a dot product of 64 or
// 128 terms, whose own fp32 error is larger).  On the FMA pipe in pairs, none of it on the
// MUFU that the exponentials need.  The coefficients come with a factor and the powers
// of two of x (CapPoly).
__host__ __device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }
struct CapPoly {
  float2 c[4];
};
inline CapPoly cap_poly(float factor) {
  const float c[4] = {0.999999463558197f, -0.33326318860054016f, 0.13190294802188873f, -0.04440207779407501f};
  CapPoly p;
  float f = 0.25f * factor;
  for (int i = 0; i < 4; ++i, f *= 0.0625f) p.c[i] = pair(c[i] * f);
  return p;
}
// factor * tanh(x / 4) / x, |x| < 2.
__device__ __forceinline__ float2 tanh_over_x(float2 x, const CapPoly& k) {
  const float2 w = __fmul2_rn(x, x);
  float2 p = __ffma2_rn(k.c[3], w, k.c[2]);
  p = __ffma2_rn(p, w, k.c[1]);
  return __ffma2_rn(p, w, k.c[0]);
}
__device__ __forceinline__ uint32_t or_bits(uint32_t acc, float2 x) {
  return acc | __float_as_uint(x.x) | __float_as_uint(x.y);
}
constexpr uint32_t kReachesTwo = 0x40000000u;
// The bound on softcap log2(e) up to which builds of the kernels may count on small caps.
constexpr float kBoundedCap = 80.0f;
// factor * tanh(x / 4) + add, any x: 1 - 2 / (1 + e^2u), which keeps its absolute error
// (about 2^-22 factor) at both ends (e^2u -> 0 or infinity gives -1 or 1).  Fit for arguments that come
// near the cap, and for any under a cap of kBoundedCap or less (an error of 2e-5 in the exponent); above it
// small arguments need the other form.
__device__ __forceinline__ float2 tanh_any(float2 x, float factor, float2 add) {
  const float2 a = __fmul2_rn(x, pair(0.7213475204444817f));
  const float2 e = __fadd2_rn(make_float2(ex2_approx(a.x), ex2_approx(a.y)), pair(1.f));
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  return __ffma2_rn(r, pair(-2.f * factor), __fadd2_rn(add, pair(factor)));
}

}  // namespace fa
