// Device pieces shared by the scored-attention kernels: the mask's intervals and the
// tanh cap.
#pragma once

#include <stdint.h>

#include "fa_device.cuh"
#include "fa_internal.h"

namespace fa {

// The interval of keys that query i sees, and of queries that see key j.
__device__ __forceinline__ int2 keys_of(const MaskPlan& p, int causal, int b, int i, int N) {
  if (p.q) return __ldg(p.q + static_cast<size_t>(b) * N + i);
  return make_int2(0, causal ? i + 1 : N);
}
__device__ __forceinline__ int2 queries_of(const MaskPlan& p, int causal, int b, int j, int N) {
  if (p.k) return __ldg(p.k + static_cast<size_t>(b) * N + j);
  return make_int2(causal ? j : 0, N);
}

// tanh for the cap.  A capped score is softcap * tanh(u); tanh.approx, off by up to
// 2^-11 relative, would move scores by up to hundredths and their weights by percents.
//
// |u| <= 1: u p(u^2) with p of degree 5 of the smallest relative error on [0, 1] (5.6e-7,
// found by linear programming on 4001 points; the score is a dot product of 64 or 128
// terms, whose own fp32 error is larger).  On the FMA pipe in pairs, none of it on the
// MUFU that the exponentials need.  The coefficients come with a factor (CapPoly), the
// result is factor * tanh(u).
__host__ __device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }
struct CapPoly {
  float2 c[6];
};
inline CapPoly cap_poly(float factor) {
  const float c[6] = {0.999999463558197f,     -0.33328977227211f,    0.13280832767486572f,
                      -0.05158914253115654f, 0.016724668443202972f, -0.0030597823206335306f};
  CapPoly p;
  for (int i = 0; i < 6; ++i) p.c[i] = pair(c[i] * factor);
  return p;
}
// tanh(u) * factor / u.
__device__ __forceinline__ float2 tanh_over_u(float2 u, const CapPoly& k) {
  const float2 w = __fmul2_rn(u, u);
  float2 p = __ffma2_rn(k.c[5], w, k.c[4]);
  p = __ffma2_rn(p, w, k.c[3]);
  p = __ffma2_rn(p, w, k.c[2]);
  p = __ffma2_rn(p, w, k.c[1]);
  return __ffma2_rn(p, w, k.c[0]);
}
// Any u: 1 - 2 / (1 + e^2u), which keeps its absolute error at both ends (e^2u -> 0 or
// infinity gives -1 or 1).
__device__ __forceinline__ float tanh_any(float u) {
  const float e = ex2_approx(u * 2.885390081777927f);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return fmaf(-2.f, r, 1.f);
}

}  // namespace fa
