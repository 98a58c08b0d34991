// C entry points of the norm and rotation of queries and keys: argument validation and
// dispatch to the kernels.  Their contract: include/fa.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fa.h"
#include "fa_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
constexpr long long kIntMax = 0x7fffffffLL;

// FA_OK, a status, or -1 for "valid, but nothing to do".
int validate(int B, int H, int Hkv, int N, int d, int rot, const void* q_weight, const void* k_weight,
             const float* inv_freq, const int32_t* positions, int norm, float eps, int weight_dtype, int interleaved,
             int dtype) {
  if (B < 0 || H < 0 || Hkv < 0 || N < 0) return FA_ERR_INVALID_ARG;
  if ((norm != 0 && norm != 1) || (interleaved != 0 && interleaved != 1)) return FA_ERR_INVALID_ARG;
  if (dtype != 1 && dtype != 2) return FA_ERR_INVALID_ARG;
  if (weight_dtype < 0 || weight_dtype > 2) return FA_ERR_INVALID_ARG;
  if (norm ? !(eps > 0.f) || !isfinite(eps) : q_weight || k_weight) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rot < 0 || rot > d || (rot > 0) != (inv_freq != nullptr)) return FA_ERR_INVALID_ARG;
  if (rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  const uintptr_t wa = weight_dtype == 0 ? 4 : 2;
  if (!aligned(q_weight, wa) || !aligned(k_weight, wa) || !aligned(inv_freq, 4) || !aligned(positions, 4))
    return FA_ERR_MISALIGNED;
  if (static_cast<long long>(B) * N > kIntMax / 2 || static_cast<long long>(H) + Hkv > kIntMax / 16) return FA_ERR_UNSUPPORTED;
  if (B == 0 || N == 0 || (H == 0 && Hkv == 0)) return -1;
  return FA_OK;
}

// One tensor of `heads` heads: its strides, and that it is there and aligned (none is needed of no heads).
int take(fa::Strides* s, const void* p, const int64_t* strides, int heads, int N, int d) {
  *s = fa::dense_strides(heads, N, d);
  if (heads == 0) return FA_OK;
  if (!p) return FA_ERR_INVALID_ARG;
  const int st = fa::strides_or(s, strides, 3, *s, d);
  if (st != FA_OK) return st;
  return aligned(p, 16) ? FA_OK : FA_ERR_MISALIGNED;
}

}  // namespace

extern "C" {

int fa_qk_norm_rope(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                    const void* q_weight, const void* k_weight, const float* inv_freq, const int32_t* positions,
                    void* q_out, const int64_t* q_out_strides, void* k_out, const int64_t* k_out_strides, int B, int H,
                    int Hkv, int N, int d, int rot, int norm, float eps, int weight_dtype, int interleaved, int dtype,
                    fa_stream_t stream) {
  const int vs = validate(B, H, Hkv, N, d, rot, q_weight, k_weight, inv_freq, positions, norm, eps, weight_dtype,
                          interleaved, dtype);
  if (vs < 0) return FA_OK;
  if (vs != FA_OK) return vs;
  fa::QkArgs a{};
  int st = take(&a.sq, q, q_strides, H, N, d);
  if (st == FA_OK) st = take(&a.sk, k, k_strides, Hkv, N, d);
  if (st == FA_OK) st = take(&a.sq_out, q_out, q_out_strides, H, N, d);
  if (st == FA_OK) st = take(&a.sk_out, k_out, k_out_strides, Hkv, N, d);
  if (st != FA_OK) return st;
  fa::CallContext c;
  if ((st = fa::call_context(&c)) != FA_OK) return st;
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.weight_type = weight_dtype;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.N = N;
  a.d = d;
  a.rot = rot;
  a.norm = norm;
  a.pairs = interleaved;
  a.fp16 = dtype == 2;
  a.eps = eps;
  return fa::launch_qk_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_qk_norm_rope_bwd_workspace_size(int d) {
  return d == 64 || d == 128 ? fa::qk_norm_rope_bwd_workspace(d) : 0;
}

int fa_qk_norm_rope_bwd(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                        const void* dq_out, const int64_t* dq_out_strides, const void* dk_out,
                        const int64_t* dk_out_strides, const void* q_weight, const void* k_weight,
                        const float* inv_freq, const int32_t* positions, void* dq, const int64_t* dq_strides, void* dk,
                        const int64_t* dk_strides, float* dq_weight, float* dk_weight, void* workspace, size_t ws_bytes,
                        int B, int H, int Hkv, int N, int d, int rot, int norm, float eps, int weight_dtype,
                        int interleaved, int dtype, fa_stream_t stream) {
  const int vs = validate(B, H, Hkv, N, d, rot, q_weight, k_weight, inv_freq, positions, norm, eps, weight_dtype,
                          interleaved, dtype);
  if (vs > 0) return vs;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return FA_ERR_INVALID_ARG;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return FA_ERR_MISALIGNED;
  if (vs < 0 && !dq_weight && !dk_weight) return FA_OK;
  fa::QkArgs a{};
  int st = FA_OK;
  if (vs == FA_OK) {
    if (norm) {  // without a norm the gradient does not depend on q and k
      st = take(&a.sq, q, q_strides, H, N, d);
      if (st == FA_OK) st = take(&a.sk, k, k_strides, Hkv, N, d);
    }
    if (st == FA_OK) st = take(&a.sdq_in, dq_out, dq_out_strides, H, N, d);
    if (st == FA_OK) st = take(&a.sdk_in, dk_out, dk_out_strides, Hkv, N, d);
    if (st == FA_OK) st = take(&a.sq_out, dq, dq_strides, H, N, d);
    if (st == FA_OK) st = take(&a.sk_out, dk, dk_strides, Hkv, N, d);
    if (st != FA_OK) return st;
  }
  if (dq_weight || dk_weight) {
    if (!workspace || ws_bytes < fa::qk_norm_rope_bwd_workspace(d)) return FA_ERR_WORKSPACE;
    if (!aligned(workspace, 4)) return FA_ERR_MISALIGNED;
  }
  fa::CallContext c;
  if ((st = fa::call_context(&c)) != FA_OK) return st;
  if (vs < 0) B = 0;  // no rows: the weights' gradients are 0
  a.q = q;
  a.k = k;
  a.dq_in = dq_out;
  a.dk_in = dk_out;
  a.q_out = dq;
  a.k_out = dk;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.weight_type = weight_dtype;
  a.dq_weight = dq_weight;
  a.dk_weight = dk_weight;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.workspace = workspace;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.N = N;
  a.d = d;
  a.rot = rot;
  a.norm = norm;
  a.pairs = interleaved;
  a.fp16 = dtype == 2;
  a.eps = eps;
  return fa::launch_qk_norm_rope_bwd(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
