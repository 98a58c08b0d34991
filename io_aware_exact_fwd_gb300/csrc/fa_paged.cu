// The paged key/value cache: appending new tokens, and attention of one token a
// sequence over the cache (include/fa.h states both).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "fa_device.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

__device__ __forceinline__ int tokens_of(const PagedCache& c, int b) {
  return min(max(c.seq_lens[b], 0), c.max_pages * c.page_size);
}

// Append: one row of d values of K and of V per d / 8 lanes, 16 bytes each.  A row's
// sequence is found by a binary search in cu_new.
__global__ void __launch_bounds__(256) paged_append_kernel(PagedAppendArgs a, long long chunks) {
  const int per_row = a.c.d / 8;
  const long long x = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (x >= chunks) return;
  const int col = static_cast<int>(x % per_row) * 8;
  const int h = static_cast<int>(x / per_row % a.c.Hkv), t = static_cast<int>(x / per_row / a.c.Hkv);
  int lo = 0, hi = a.c.B + 1;  // the number of offsets <= t
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (a.cu_new[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  if (lo == 0 || lo == a.c.B + 1) return;  // a row of no sequence
  const int b = lo - 1;
  const long long pos = static_cast<long long>(a.c.seq_lens[b]) - (static_cast<long long>(a.cu_new[lo]) - t);
  if (pos < 0 || pos >= static_cast<long long>(a.c.max_pages) * a.c.page_size) return;
  const int at = static_cast<int>(pos) / a.c.page_size, off = static_cast<int>(pos) % a.c.page_size;
  const int page = a.c.page_table[b * a.c.table_stride + at];
  if (page < 0 || page >= a.c.n_pages) return;
  const uint4 kv = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k) + t * a.sk.s[1] + h * a.sk.s[0] + col);
  const uint4 vv = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.v) + t * a.sv.s[1] + h * a.sv.s[0] + col);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.c.k) + page * a.c.sk.s[2] + h * a.c.sk.s[1] + off * a.c.sk.s[0] + col) = kv;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.c.v) + page * a.c.sv.s[2] + h * a.c.sv.s[1] + off * a.c.sv.s[0] + col) = vv;
}

template <bool FP16>
__device__ __forceinline__ float to_f32(uint16_t x) {
  return FP16 ? __half2float(__ushort_as_half(x)) : __bfloat162float(__ushort_as_bfloat16(x));
}
template <bool FP16>
__device__ __forceinline__ uint16_t from_f32(float x) {
  return FP16 ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// Decode, the simplest form: one warp per (sequence, query head) walks the tokens.
template <int D, bool FP16>
__global__ void __launch_bounds__(128) decode_rows_kernel(PagedDecodeArgs a, long long rows) {
  constexpr int E = D / 32;
  const long long r = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int lane = threadIdx.x & 31;
  const int h = static_cast<int>(r % a.H), b = static_cast<int>(r / a.H), hk = h / (a.H / a.c.Hkv);
  const int n = tokens_of(a.c, b);
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + b * a.sq.s[1] + h * a.sq.s[0] + lane * E;
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) q[e] = to_f32<FP16>(qp[e]);
  for (int j = 0; j < n; ++j) {
    const int page = a.c.page_table[b * a.c.table_stride + j / a.c.page_size], off = j % a.c.page_size;
    const bool in = page >= 0 && page < a.c.n_pages;
    const uint16_t* kp = static_cast<const uint16_t*>(a.c.k) + page * a.c.sk.s[2] + hk * a.c.sk.s[1] + off * a.c.sk.s[0] + lane * E;
    const uint16_t* vp = static_cast<const uint16_t*>(a.c.v) + page * a.c.sv.s[2] + hk * a.c.sv.s[1] + off * a.c.sv.s[0] + lane * E;
    float s = 0.f, v[E];
    for (int e = 0; e < E; ++e) {
      s = fmaf(q[e], in ? to_f32<FP16>(kp[e]) : 0.f, s);
      v[e] = in ? to_f32<FP16>(vp[e]) : 0.f;
    }
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= a.scale;
    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    s -= slope * static_cast<float>(n - 1 - j);
    const float mn = fmaxf(m, s), w = expf(m - mn), p = expf(s - mn);
    l = l * w + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * w + p * v[e];
    m = mn;
  }
  uint16_t* op = static_cast<uint16_t*>(a.o) + b * a.so.s[1] + h * a.so.s[0] + lane * E;
  for (int e = 0; e < E; ++e) op[e] = from_f32<FP16>(l > 0.f ? o[e] / l : 0.f);
  if (lane == 0) a.lse[r] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  const long long chunks = static_cast<long long>(a.T) * a.c.Hkv * (a.c.d / 8);
  paged_append_kernel<<<static_cast<unsigned>((chunks + 255) / 256), 256, 0, stream>>>(a, chunks);
  return cudaGetLastError();
}

size_t paged_decode_workspace(int, int, int, int) { return 256; }

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.c.B) * a.H;
  auto kern = a.c.d == 64 ? (a.fp16 ? decode_rows_kernel<64, true> : decode_rows_kernel<64, false>)
                          : (a.fp16 ? decode_rows_kernel<128, true> : decode_rows_kernel<128, false>);
  kern<<<static_cast<unsigned>((rows + 3) / 4), 128, 0, stream>>>(a, rows);
  return cudaGetLastError();
}

}  // namespace fa
