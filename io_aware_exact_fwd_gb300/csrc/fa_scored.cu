// Scored attention: the mask plan, and the backward in its simplest form, one warp per
// row on the CUDA cores (the formulas: include/fa.h).
#include <cuda_bf16.h>
#include <math.h>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "fa_score.cuh"

namespace fa {
namespace {

// One thread per position.  Position i of row b: the last document that starts at or
// before i (binary search in the offsets) holds it if it ends after i.  Padding gets
// empty intervals that keep both ends nondecreasing along the row: at the first
// document's start before it, else at the end of the document before it.  Everything
// is clamped to [0, N], so offsets that break the contract still give intervals inside
// the row.
__global__ void __launch_bounds__(256) mask_plan_kernel(const int32_t* __restrict__ cu_docs,
                                                        const int32_t* __restrict__ prefix, int n_docs,
                                                        int2* __restrict__ qi, int2* __restrict__ ki, int N,
                                                        long long rows, int causal) {
  const long long r = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (r >= rows) return;
  const int b = static_cast<int>(r / N), i = static_cast<int>(r % N);
  int s = 0, e = N, p = 0;
  if (cu_docs) {
    const int32_t* cu = cu_docs + static_cast<size_t>(b) * (n_docs + 1);
    int lo = 0, hi = n_docs + 1;  // the number of offsets <= i
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (cu[mid] <= i) lo = mid + 1;
      else hi = mid;
    }
    if (lo == 0) {
      s = e = min(max(cu[0], 0), N);
    } else if (lo == n_docs + 1) {
      s = e = min(max(cu[n_docs], 0), N);
    } else {
      s = min(max(cu[lo - 1], 0), N);
      e = min(max(cu[lo], s), N);
      if (prefix) p = max(prefix[static_cast<size_t>(b) * n_docs + lo - 1], 0);
    }
  } else if (prefix) {
    p = max(prefix[b], 0);
  }
  if (s >= e) {
    qi[r] = ki[r] = make_int2(s, s);
    return;
  }
  const int reach = p >= e - s ? e : s + p;  // the prefix's end
  qi[r] = make_int2(s, causal ? max(i + 1, reach) : e);
  ki[r] = make_int2(causal && i >= reach ? i : s, e);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

template <int E>
__device__ __forceinline__ void load_row(float (&x)[E], const void* base, const Strides& st, int b, int h, int n) {
  const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + b * st.s[2] + h * st.s[1] +
                           static_cast<int64_t>(n) * st.s[0] + (threadIdx.x & 31) * E;
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = __bfloat162float(p[e]);
}
template <int E>
__device__ __forceinline__ void store_row(const float (&x)[E], void* base, const Strides& st, int b, int h, int n) {
  __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + b * st.s[2] + h * st.s[1] +
                     static_cast<int64_t>(n) * st.s[0] + (threadIdx.x & 31) * E;
#pragma unroll
  for (int e = 0; e < E; ++e) p[e] = __float2bfloat16_rn(x[e]);
}
template <int E>
__device__ __forceinline__ float dot(const float (&x)[E], const float (&y)[E]) {
  float a = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) a = fmaf(x[e], y[e], a);
  return warp_sum(a);
}

// The score of a pair and the cap's derivative 1 - tanh^2 there.
__device__ __forceinline__ float score(float qk, const ScoreArgs& sc, float slope, int i, int j, float& bend) {
  float a = sc.scale * qk;
  bend = 1.f;
  if (sc.softcap > 0.f) {
    const float t = tanhf(a / sc.softcap);
    a = sc.softcap * t;
    bend = 1.f - t * t;
  }
  return a - slope * fabsf(static_cast<float>(i - j));
}

// One warp per query row: dQ.
template <int D>
__global__ void __launch_bounds__(128) bwd_dq_rows_kernel(BwdArgs a, ScoreArgs sc, long long rows) {
  constexpr int E = D / 32;
  const long long r = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int i = static_cast<int>(r % a.N), h = static_cast<int>(r / a.N % a.H), b = static_cast<int>(r / a.N / a.H);
  const int hk = h / (a.H / sc.Hkv);
  const float slope = sc.slopes ? sc.slopes[h] : 0.f;
  const int2 see = keys_of(sc.plan, sc.causal, b, i, a.N);
  float q[E], k[E], v[E], g[E], o[E], dq[E] = {}, bend;
  load_row(q, a.q, a.sq, b, h, i);
  load_row(g, a.dout, a.sdo, b, h, i);
  load_row(o, a.o, a.so, b, h, i);
  const float D_i = dot(g, o), lse = a.lse[r];
  for (int j = see.x; j < see.y; ++j) {
    load_row(k, a.k, a.sk, b, hk, j);
    load_row(v, a.v, a.sv, b, hk, j);
    const float s = score(dot(q, k), sc, slope, i, j, bend);
    const float ds = expf(s - lse) * (dot(g, v) - D_i) * bend * a.scale;
#pragma unroll
    for (int e = 0; e < E; ++e) dq[e] = fmaf(ds, k[e], dq[e]);
  }
  store_row(dq, a.dq, a.sdq, b, h, i);
}

// One warp per key row: dK and dV over the group's heads.
template <int D>
__global__ void __launch_bounds__(128) bwd_dkv_rows_kernel(BwdArgs a, ScoreArgs sc, long long rows) {
  constexpr int E = D / 32;
  const long long r = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int j = static_cast<int>(r % a.N), hk = static_cast<int>(r / a.N % sc.Hkv);
  const int b = static_cast<int>(r / a.N / sc.Hkv), group = a.H / sc.Hkv;
  const int2 by = queries_of(sc.plan, sc.causal, b, j, a.N);
  float q[E], k[E], v[E], g[E], o[E], dk[E] = {}, dv[E] = {}, bend;
  load_row(k, a.k, a.sk, b, hk, j);
  load_row(v, a.v, a.sv, b, hk, j);
  for (int h = hk * group; h < hk * group + group; ++h) {
    const float slope = sc.slopes ? sc.slopes[h] : 0.f;
    for (int i = by.x; i < by.y; ++i) {
      load_row(q, a.q, a.sq, b, h, i);
      load_row(g, a.dout, a.sdo, b, h, i);
      load_row(o, a.o, a.so, b, h, i);
      const float s = score(dot(q, k), sc, slope, i, j, bend);
      const float p = expf(s - a.lse[(static_cast<size_t>(b) * a.H + h) * a.N + i]);
      const float ds = p * (dot(g, v) - dot(g, o)) * bend * a.scale;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        dk[e] = fmaf(ds, q[e], dk[e]);
        dv[e] = fmaf(p, g[e], dv[e]);
      }
    }
  }
  store_row(dk, a.dk, a.sdk, b, hk, j);
  store_row(dv, a.dv, a.sdv, b, hk, j);
}

unsigned blocks_of(long long rows) { return static_cast<unsigned>((rows + 3) / 4); }

}  // namespace

cudaError_t launch_mask_plan(const int32_t* cu_docs, const int32_t* prefix, int n_docs, void* plan, int B, int N,
                             int causal, cudaStream_t stream) {
  const long long rows = static_cast<long long>(B) * N;
  int2* qi = static_cast<int2*>(plan);
  mask_plan_kernel<<<static_cast<unsigned>((rows + 255) / 256), 256, 0, stream>>>(cu_docs, prefix, n_docs, qi,
                                                                                  qi + rows, N, rows, causal);
  return cudaGetLastError();
}

cudaError_t launch_bwd_scored(const BwdArgs& a, const ScoreArgs& sc, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.B) * a.H * a.N, kv_rows = static_cast<long long>(a.B) * sc.Hkv * a.N;
  auto kq = a.d == 64 ? bwd_dq_rows_kernel<64> : bwd_dq_rows_kernel<128>;
  auto kkv = a.d == 64 ? bwd_dkv_rows_kernel<64> : bwd_dkv_rows_kernel<128>;
  kq<<<blocks_of(rows), 128, 0, stream>>>(a, sc, rows);
  cudaError_t e = cudaGetLastError();
  if (e) return e;
  kkv<<<blocks_of(kv_rows), 128, 0, stream>>>(a, sc, kv_rows);
  return cudaGetLastError();
}

}  // namespace fa
