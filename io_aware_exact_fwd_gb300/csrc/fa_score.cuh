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

// tanh for the cap, to an absolute error of about 2^-23 (the cap's scores are
// cap * tanh, so tanh.approx, off by up to 2^-11 relative, would move a capped score by
// percents of 1 and its weight with it).
//
// |u| <= 1: u p(u^2), p of degree 6 with the smallest relative error on [0, 1] (3.5e-8,
// found by linear programming on 4001 points).  Pairs, on the FMA pipe: 8 packed
// operations, none on the MUFU that the exponentials need.
__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 tanh_small(float2 u) {
  const float2 w = __fmul2_rn(u, u);
  float2 p = pair(0.001009133062325418f);
  p = __ffma2_rn(p, w, pair(-0.0061064367182552814f));
  p = __ffma2_rn(p, w, pair(0.0201801136136055f));
  p = __ffma2_rn(p, w, pair(-0.05340071767568588f));
  p = __ffma2_rn(p, w, pair(0.13323982059955597f));
  p = __ffma2_rn(p, w, pair(-0.33332768082618713f));
  p = __ffma2_rn(p, w, pair(0.9999999403953552f));
  return __fmul2_rn(u, p);
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
