// C entry points of scored attention and of the paged caches: argument validation and
// dispatch to the kernels.  Their contract: include/fa.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "fa.h"
#include "fa_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int status_of(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }
constexpr long long kIntMax = 0x7fffffffLL;

// The kernels multiply products by 4 scale / softcap and tanh by softcap log2(e): both have to be finite, and
// the first a normal number (a subnormal one has lost bits).
bool bad_score(float scale, float softcap) {
  return !(scale > 0.f) || !isfinite(scale) || !(softcap >= 0.f) || !isfinite(2.f * softcap) ||
         (softcap > 0.f && !isnormal(4.f * scale / softcap));
}

// FA_OK, a status, or -1 for "valid, but nothing to do".
int validate_scored(int B, int H, int Hkv, int N, int d, int causal, float scale, float softcap) {
  if (B < 0 || H < 0 || Hkv < 0 || N < 0) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (bad_score(scale, softcap)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (B == 0 || H == 0 || N == 0) return -1;
  if (Hkv == 0 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  // B H N (rows, and with them tiles and blocks of the grids) stays inside int; the
  // group's query blocks of one key block are counted in int as well.
  const long long rows = static_cast<long long>(B) * H * ((static_cast<long long>(N) + 255) / 256 * 256);
  if (static_cast<long long>(B) * H > kIntMax || rows > kIntMax) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int validate_plan(const void* plan, size_t plan_bytes, int B, int N, int causal) {
  if (!plan) return FA_OK;
  if (causal) return FA_ERR_INVALID_ARG;
  if (plan_bytes < fa_mask_plan_size(B, N)) return FA_ERR_WORKSPACE;
  return aligned(plan, 16) ? FA_OK : FA_ERR_MISALIGNED;
}

fa::ScoreArgs score_args(const void* plan, int B, int N, int Hkv, int causal, float scale, float softcap,
                         const float* slopes) {
  return fa::ScoreArgs{fa::mask_plan_of(plan, B, N), causal, scale, softcap, slopes, Hkv};
}

}  // namespace

extern "C" {

size_t fa_mask_plan_size(int B, int N) {
  if (B < 1 || N < 1 || static_cast<long long>(B) * N > kIntMax) return 0;
  return static_cast<size_t>(B) * N * 2 * sizeof(int2);
}

int fa_mask_plan(const int32_t* cu_docs, const int32_t* prefix, int n_docs, void* plan, size_t plan_bytes, int B,
                 int N, int causal, fa_stream_t stream) {
  if (B < 0 || N < 0 || n_docs < 1 || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  if (!cu_docs && n_docs != 1) return FA_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return FA_OK;
  const size_t need = fa_mask_plan_size(B, N);
  if (need == 0) return FA_ERR_UNSUPPORTED;
  if (!plan || plan_bytes < need) return FA_ERR_WORKSPACE;
  if (!aligned(plan, 16) || !aligned(cu_docs, 4) || !aligned(prefix, 4)) return FA_ERR_MISALIGNED;
  fa::CallContext c;
  const int st = fa::call_context(&c);
  if (st != FA_OK) return st;
  return status_of(fa::launch_mask_plan(cu_docs, prefix, n_docs, plan, B, N, causal,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

int fa_fwd_scored(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides, const void* v,
                  const int64_t* v_strides, void* o, const int64_t* o_strides, float* lse, int B, int H, int Hkv,
                  int N, int d, const void* plan, size_t plan_bytes, int causal, float scale, float softcap,
                  const float* slopes, fa_stream_t stream) {
  const int vs = validate_scored(B, H, Hkv, N, d, causal, scale, softcap);
  if (vs < 0) return FA_OK;
  if (vs != FA_OK) return vs;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  int st = validate_plan(plan, plan_bytes, B, N, causal);
  if (st != FA_OK) return st;
  fa::FwdArgs a{};
  const fa::Strides dq = fa::dense_strides(H, N, d), dkv = fa::dense_strides(Hkv, N, d);
  if ((st = fa::strides_or(&a.sq, q_strides, 3, dq, d)) != FA_OK) return st;
  if ((st = fa::strides_or(&a.sk, k_strides, 3, dkv, d)) != FA_OK) return st;
  if ((st = fa::strides_or(&a.sv, v_strides, 3, dkv, d)) != FA_OK) return st;
  if ((st = fa::strides_or(&a.so, o_strides, 3, dq, d)) != FA_OK) return st;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(slopes, 4))
    return FA_ERR_MISALIGNED;
  fa::CallContext c;
  if ((st = fa::call_context(&c)) != FA_OK) return st;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  a.B = B;
  a.H = H;
  a.N = N;
  a.d = d;
  a.causal = causal;
  a.scale = scale;
  a.err_word = c.err_word;
  a.dbg = c.dbg;
  return status_of(fa::launch_fwd_scored(a, score_args(plan, B, N, Hkv, causal, scale, softcap, slopes),
                                         reinterpret_cast<cudaStream_t>(stream)));
}

size_t fa_bwd_scored_workspace_size(int B, int H, int Hkv, int N, int d) {
  if (validate_scored(B, H, Hkv, N, d, 0, 1.f, 0.f) != FA_OK) return 0;
  return fa::bwd_scored_workspace(B, H, Hkv, N, d);
}

int fa_bwd_scored(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides, const void* v,
                  const int64_t* v_strides, const void* o, const int64_t* o_strides, const void* dout,
                  const int64_t* dout_strides, const float* lse, void* dq, const int64_t* dq_strides, void* dk,
                  const int64_t* dk_strides, void* dv, const int64_t* dv_strides, void* workspace, size_t ws_bytes,
                  int B, int H, int Hkv, int N, int d, const void* plan, size_t plan_bytes, int causal, float scale,
                  float softcap, const float* slopes, int deterministic, fa_stream_t stream) {
  if (deterministic != 0 && deterministic != 1) return FA_ERR_INVALID_ARG;
  const int vs = validate_scored(B, H, Hkv, N, d, causal, scale, softcap);
  if (vs < 0) return FA_OK;
  if (vs != FA_OK) return vs;
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  int st = validate_plan(plan, plan_bytes, B, N, causal);
  if (st != FA_OK) return st;
  if (deterministic && static_cast<long long>(B) * Hkv > 65535) return FA_ERR_UNSUPPORTED;  // a grid's second axis
  if (!workspace || ws_bytes < fa::bwd_scored_workspace(B, H, Hkv, N, d)) return FA_ERR_WORKSPACE;
  fa::BwdArgs a{};
  const fa::Strides ds = fa::dense_strides(H, N, d), dkv = fa::dense_strides(Hkv, N, d);
  const struct {
    fa::Strides* out;
    const int64_t* in;
    const fa::Strides& dense;
  } each[8] = {{&a.sq, q_strides, ds},       {&a.sk, k_strides, dkv},  {&a.sv, v_strides, dkv},  {&a.so, o_strides, ds},
               {&a.sdo, dout_strides, ds},   {&a.sdq, dq_strides, ds}, {&a.sdk, dk_strides, dkv}, {&a.sdv, dv_strides, dkv}};
  for (const auto& e : each)
    if ((st = fa::strides_or(e.out, e.in, 3, e.dense, d)) != FA_OK) return st;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(dout, 16) ||
      !aligned(lse, 4) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(workspace, 256) ||
      !aligned(slopes, 4))
    return FA_ERR_MISALIGNED;
  fa::CallContext c;
  if ((st = fa::call_context(&c)) != FA_OK) return st;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.dout = dout;
  a.lse = lse;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.workspace = workspace;
  a.B = B;
  a.H = H;
  a.N = N;
  a.d = d;
  a.causal = causal;
  a.deterministic = deterministic;
  a.scale = scale;
  a.err_word = c.err_word;
  a.dbg = c.dbg;
  return status_of(fa::launch_bwd_scored(a, score_args(plan, B, N, Hkv, causal, scale, softcap, slopes),
                                         reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

constexpr int kBf16 = 1, kFp16 = 2;  // the dtype argument

int validate_paged(int B, int Hkv, int d, int page_size, int n_pages, int max_pages, int64_t table_stride, int dtype) {
  if (B < 0 || Hkv < 0 || n_pages < 0 || max_pages < 0) return FA_ERR_INVALID_ARG;
  if (dtype != kBf16 && dtype != kFp16) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (page_size < 16 || page_size > 1024 || page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (B == 0) return -1;
  if (Hkv == 0 || max_pages == 0 || n_pages == 0) return FA_ERR_INVALID_ARG;
  if (table_stride < max_pages) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * page_size > kIntMax / 2 || B > 65535 ||
      static_cast<long long>(B) * Hkv > kIntMax)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int paged_cache(fa::PagedCache* c, const void* k, const int64_t* sk, const void* v, const int64_t* sv,
                const int32_t* page_table, int64_t table_stride, const int32_t* seq_lens, int B, int Hkv, int d,
                int page_size, int n_pages, int max_pages) {
  if (!k || !v || !page_table || !seq_lens) return FA_ERR_INVALID_ARG;
  const fa::Strides dense{{d, static_cast<int64_t>(page_size) * d, static_cast<int64_t>(Hkv) * page_size * d}};
  int st = fa::strides_or(&c->sk, sk, 3, dense, d);
  if (st == FA_OK) st = fa::strides_or(&c->sv, sv, 3, dense, d);
  if (st != FA_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4)) return FA_ERR_MISALIGNED;
  c->k = const_cast<void*>(k);
  c->v = const_cast<void*>(v);
  c->page_table = page_table;
  c->table_stride = table_stride;
  c->seq_lens = seq_lens;
  c->B = B;
  c->Hkv = Hkv;
  c->d = d;
  c->page_size = page_size;
  c->per_page = fa::Div(page_size);
  c->n_pages = n_pages;
  c->max_pages = max_pages;
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_paged_append(const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides, void* k_cache,
                    const int64_t* k_cache_strides, void* v_cache, const int64_t* v_cache_strides,
                    const int32_t* page_table, int64_t table_stride, const int32_t* seq_lens, const int32_t* cu_new,
                    int B, int T, int Hkv, int d, int page_size, int n_pages, int max_pages, int dtype,
                    fa_stream_t stream) {
  if (T < 0) return FA_ERR_INVALID_ARG;
  const int vs = validate_paged(B, Hkv, d, page_size, n_pages, max_pages, table_stride, dtype);
  if (vs < 0) return FA_OK;
  if (vs != FA_OK) return vs;
  if (T == 0) return FA_OK;
  if (static_cast<long long>(T) * Hkv > kIntMax) return FA_ERR_UNSUPPORTED;
  if (!k || !v || !cu_new) return FA_ERR_INVALID_ARG;
  fa::PagedAppendArgs a{};
  int st = paged_cache(&a.c, k_cache, k_cache_strides, v_cache, v_cache_strides, page_table, table_stride, seq_lens,
                       B, Hkv, d, page_size, n_pages, max_pages);
  const fa::Strides dense{{d, static_cast<int64_t>(Hkv) * d, 0}};
  if (st == FA_OK) st = fa::strides_or(&a.sk, k_strides, 2, dense, d);
  if (st == FA_OK) st = fa::strides_or(&a.sv, v_strides, 2, dense, d);
  if (st != FA_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_new, 4)) return FA_ERR_MISALIGNED;
  fa::CallContext c;
  if ((st = fa::call_context(&c)) != FA_OK) return st;
  a.k = k;
  a.v = v;
  a.cu_new = cu_new;
  a.T = T;
  return status_of(fa::launch_paged_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fa_paged_decode_workspace_size(int B, int H, int Hkv, int d) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || (d != 64 && d != 128)) return 0;
  if (B > 65535 || static_cast<long long>(B) * H > kIntMax) return 0;
  return std::max(fa::paged_decode_workspace(B, d), fa::paged_decode_fp8_workspace(B, H, Hkv, d));
}

int fa_paged_decode(const void* q, const int64_t* q_strides, const void* k_cache, const int64_t* k_cache_strides,
                    const void* v_cache, const int64_t* v_cache_strides, const int32_t* page_table,
                    int64_t table_stride, const int32_t* seq_lens, void* o, const int64_t* o_strides, float* lse,
                    void* workspace, size_t ws_bytes, int B, int H, int Hkv, int d, int page_size, int n_pages,
                    int max_pages, int dtype, float scale, float softcap, const float* slopes, fa_stream_t stream) {
  if (H < 0 || bad_score(scale, softcap)) return FA_ERR_INVALID_ARG;
  const int vs = validate_paged(B, Hkv, d, page_size, n_pages, max_pages, table_stride, dtype);
  if (vs < 0 || (vs == FA_OK && H == 0)) return FA_OK;
  if (vs != FA_OK) return vs;
  if (H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H > kIntMax) return FA_ERR_UNSUPPORTED;
  if (!q || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < fa::paged_decode_workspace(B, d)) return FA_ERR_WORKSPACE;
  fa::PagedDecodeArgs a{};
  int st = paged_cache(&a.c, k_cache, k_cache_strides, v_cache, v_cache_strides, page_table, table_stride, seq_lens,
                       B, Hkv, d, page_size, n_pages, max_pages);
  const fa::Strides dense{{d, static_cast<int64_t>(H) * d, 0}};
  if (st == FA_OK) st = fa::strides_or(&a.sq, q_strides, 2, dense, d);
  if (st == FA_OK) st = fa::strides_or(&a.so, o_strides, 2, dense, d);
  if (st != FA_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 256) || !aligned(slopes, 4))
    return FA_ERR_MISALIGNED;
  fa::CallContext c;
  if ((st = fa::call_context(&c)) != FA_OK) return st;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.workspace = workspace;
  a.H = H;
  a.fp16 = dtype == kFp16;
  a.scale = scale;
  a.softcap = softcap;
  a.slopes = slopes;
  a.err_word = c.err_word;
  a.dbg = c.dbg;
  return status_of(fa::launch_paged_decode(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// The strides and scales of a cache of codes: rows start on 16 bytes, as TMA needs them.
int codes_of(fa::PagedCache* c, float* k_scales, float* v_scales) {
  for (int i = 0; i < 3; ++i)
    if (c->sk.s[i] % 16 != 0 || c->sv.s[i] % 16 != 0) return FA_ERR_MISALIGNED;
  if (!k_scales || !v_scales) return FA_ERR_INVALID_ARG;
  if (!aligned(k_scales, 4) || !aligned(v_scales, 4)) return FA_ERR_MISALIGNED;
  c->k_scales = k_scales;
  c->v_scales = v_scales;
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_paged_append_fp8(const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides, void* k_cache,
                        const int64_t* k_cache_strides, void* v_cache, const int64_t* v_cache_strides, float* k_scales,
                        float* v_scales, const int32_t* page_table, int64_t table_stride, const int32_t* seq_lens,
                        const int32_t* cu_new, int B, int T, int Hkv, int d, int page_size, int n_pages, int max_pages,
                        int dtype, fa_stream_t stream) {
  if (T < 0) return FA_ERR_INVALID_ARG;
  const int vs = validate_paged(B, Hkv, d, page_size, n_pages, max_pages, table_stride, dtype);
  if (vs < 0) return FA_OK;
  if (vs != FA_OK) return vs;
  if (T == 0) return FA_OK;
  if (static_cast<long long>(T) * Hkv > kIntMax) return FA_ERR_UNSUPPORTED;
  if (!k || !v || !cu_new) return FA_ERR_INVALID_ARG;
  fa::PagedAppendArgs a{};
  int st = paged_cache(&a.c, k_cache, k_cache_strides, v_cache, v_cache_strides, page_table, table_stride, seq_lens,
                       B, Hkv, d, page_size, n_pages, max_pages);
  const fa::Strides dense{{d, static_cast<int64_t>(Hkv) * d, 0}};
  if (st == FA_OK) st = codes_of(&a.c, k_scales, v_scales);
  if (st == FA_OK) st = fa::strides_or(&a.sk, k_strides, 2, dense, d);
  if (st == FA_OK) st = fa::strides_or(&a.sv, v_strides, 2, dense, d);
  if (st != FA_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_new, 4)) return FA_ERR_MISALIGNED;
  fa::CallContext c;
  if ((st = fa::call_context(&c)) != FA_OK) return st;
  a.k = k;
  a.v = v;
  a.cu_new = cu_new;
  a.T = T;
  a.fp16 = dtype == kFp16;
  return status_of(fa::launch_paged_append_fp8(a, reinterpret_cast<cudaStream_t>(stream)));
}

int fa_paged_decode_fp8(const void* q, const int64_t* q_strides, const void* k_cache, const int64_t* k_cache_strides,
                        const void* v_cache, const int64_t* v_cache_strides, const float* k_scales,
                        const float* v_scales, const int32_t* page_table, int64_t table_stride,
                        const int32_t* seq_lens, void* o, const int64_t* o_strides, float* lse, void* workspace,
                        size_t ws_bytes, int B, int H, int Hkv, int d, int page_size, int n_pages, int max_pages,
                        int dtype, float scale, float softcap, const float* slopes, fa_stream_t stream) {
  if (H < 0 || bad_score(scale, softcap)) return FA_ERR_INVALID_ARG;
  const int vs = validate_paged(B, Hkv, d, page_size, n_pages, max_pages, table_stride, dtype);
  if (vs < 0 || (vs == FA_OK && H == 0)) return FA_OK;
  if (vs != FA_OK) return vs;
  if (H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H > kIntMax) return FA_ERR_UNSUPPORTED;
  if (!q || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < fa_paged_decode_workspace_size(B, H, Hkv, d)) return FA_ERR_WORKSPACE;
  fa::PagedDecodeArgs a{};
  int st = paged_cache(&a.c, k_cache, k_cache_strides, v_cache, v_cache_strides, page_table, table_stride, seq_lens,
                       B, Hkv, d, page_size, n_pages, max_pages);
  const fa::Strides dense{{d, static_cast<int64_t>(H) * d, 0}};
  if (st == FA_OK) st = codes_of(&a.c, const_cast<float*>(k_scales), const_cast<float*>(v_scales));
  if (st == FA_OK) st = fa::strides_or(&a.sq, q_strides, 2, dense, d);
  if (st == FA_OK) st = fa::strides_or(&a.so, o_strides, 2, dense, d);
  if (st != FA_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 256) || !aligned(slopes, 4))
    return FA_ERR_MISALIGNED;
  fa::CallContext c;
  if ((st = fa::call_context(&c)) != FA_OK) return st;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.workspace = workspace;
  a.H = H;
  a.fp16 = dtype == kFp16;
  a.scale = scale;
  a.softcap = softcap;
  a.slopes = slopes;
  a.err_word = c.err_word;
  a.dbg = c.dbg;
  return status_of(fa::launch_paged_decode_fp8(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fa_paged_resize_workspace_size(int B) { return B < 0 || B > 65535 ? 0 : fa::paged_resize_workspace(B); }

int fa_paged_resize(int32_t* page_table, int64_t table_stride, const int32_t* seq_lens, const int32_t* delta,
                    int32_t* free_pages, int capacity, const int32_t* free_count, int32_t* seq_lens_out,
                    int32_t* free_count_out, int32_t* cu_new, int32_t* status, int64_t* slots, int32_t* positions, int T,
                    void* workspace, size_t ws_bytes, int B, int page_size, int max_pages, fa_stream_t stream) {
  if (B < 0 || T < 0 || capacity < 0 || max_pages < 0) return FA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 1024 || page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || static_cast<long long>(max_pages) * page_size > kIntMax / 2) return FA_ERR_UNSUPPORTED;
  if (!free_count || !free_count_out || !cu_new || !status || (capacity > 0 && !free_pages)) return FA_ERR_INVALID_ARG;
  if (B > 0 && (!page_table || !seq_lens || !delta || !seq_lens_out || max_pages == 0 || table_stride < max_pages))
    return FA_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < fa::paged_resize_workspace(B)) return FA_ERR_WORKSPACE;
  const void* words[] = {page_table, seq_lens, delta,  free_pages, free_count, seq_lens_out,
                         free_count_out, cu_new, status, positions, workspace};
  for (const void* p : words)
    if (!aligned(p, 4)) return FA_ERR_MISALIGNED;
  if (!aligned(slots, 8)) return FA_ERR_MISALIGNED;
  fa::CallContext c;
  const int st = fa::call_context(&c);
  if (st != FA_OK) return st;
  fa::PagedResizeArgs a{};
  a.page_table = page_table;
  a.table_stride = table_stride;
  a.seq_lens = seq_lens;
  a.delta = delta;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.lens_out = seq_lens_out;
  a.count_out = free_count_out;
  a.cu_new = cu_new;
  a.status = status;
  a.slots = slots;
  a.positions = positions;
  a.workspace = workspace;
  a.B = B;
  a.page_size = page_size;
  a.per_page = fa::Div(page_size);
  a.max_pages = max_pages;
  a.capacity = capacity;
  a.T = slots || positions ? T : 0;
  return status_of(fa::launch_paged_resize(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
