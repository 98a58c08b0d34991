// Binding of scored attention, of the paged caches and of the norm and rotation of queries
// and keys to PyTorch tensors, for calls made once a layer and token: checks, output allocation and the C call in one step.  In
// Python with ctypes a decode took 27 us of the GB300's host where its kernels take 12.  Here a whole call, its
// launches among it, takes 2.6 us (an append) to 5.5 (a decode: two launches, two tensor maps) and 7 (the gradient of norm
// and rotation); each output or workspace that it has to allocate adds about 1.
//
// Each function takes every argument by position (io_aware_exact_fwd_gb300/__init__.py
// has the keywords and the documentation), raises TypeError or ValueError for tensors
// that do not fit, and returns the C status as an int if the call refused, else the
// outputs.  Tensors are only described to the library, never touched.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>

#include "fa.h"

namespace {

using at::Tensor;

// A tensor that does not fit: its Python exception's type and text.
struct Unfit {
  PyObject* type;
  std::string text;
};
[[noreturn]] void unfit(PyObject* type, const std::string& text) { throw Unfit{type, text}; }

const Tensor& tensor(PyObject* x, const char* name) {
  if (!THPVariable_Check(x)) unfit(PyExc_TypeError, c10::str(name, " must be a torch.Tensor"));
  return THPVariable_Unpack(x);
}

// The GPU index of the tensor a call goes by, and that the rest have to share.
int gpu_of(const Tensor& t, const char* name) {
  if (!t.is_cuda()) unfit(PyExc_ValueError, c10::str(name, " must be a CUDA tensor, got ", t.device()));
  return t.get_device();
}

// The attention tensors' type is the call's (TypeError); that of indices, statistics and
// slopes is fixed (ValueError), as in the ctypes binding.
void check(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int gpu,
           PyObject* wrong_type = PyExc_ValueError) {
  if (t.scalar_type() != type) unfit(wrong_type, c10::str(name, " must be ", type, ", got ", t.scalar_type()));
  if (t.sizes() != shape) unfit(PyExc_ValueError, c10::str(name, " must have shape ", shape, ", got ", t.sizes()));
  if (!t.is_cuda() || t.get_device() != gpu)
    unfit(PyExc_ValueError, c10::str(name, " must be on cuda:", gpu, ", got ", t.device()));
}

// A tensor in any layout whose last dimension is contiguous: its address, and its strides
// from the second-to-last dimension outwards, or NULL when dense (dimensions of one
// element, whose stride means nothing, count as dense).
struct Layout {
  void* p;
  int64_t st[3];
  bool dense;
  const int64_t* strides() const { return dense ? nullptr : st; }
};
Layout layout(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int gpu) {
  check(t, name, type, shape, gpu, PyExc_TypeError);
  Layout x{t.data_ptr(), {0, 0, 0}, t.is_contiguous()};
  if (x.dense) return x;
  const int n = static_cast<int>(shape.size());
  if (t.stride(n - 1) != 1) unfit(PyExc_ValueError, c10::str(name, " must have a contiguous last dimension"));
  int64_t dense = shape[n - 1];
  for (int i = n - 2; i >= 0; --i) {
    x.st[n - 2 - i] = shape[i] == 1 ? dense : t.stride(i);
    dense *= shape[i];
  }
  return x;
}

// A dense tensor's address; None: NULL.
template <class T>
T* flat(PyObject* x, const char* name, at::ScalarType type, at::IntArrayRef shape, int gpu) {
  if (x == Py_None) return nullptr;
  const Tensor& t = tensor(x, name);
  check(t, name, type, shape, gpu);
  if (!t.is_contiguous()) unfit(PyExc_ValueError, c10::str(name, " must be contiguous"));
  return static_cast<T*>(t.data_ptr());
}

// A plan or workspace: a dense tensor of any type.
struct Bytes {
  void* p = nullptr;
  size_t n = 0;
};
Bytes bytes(PyObject* x, const char* name, int gpu) {
  if (x == Py_None) return {};
  const Tensor& t = tensor(x, name);
  if (!t.is_cuda() || t.get_device() != gpu || !t.is_contiguous())
    unfit(PyExc_ValueError, c10::str(name, " must be a contiguous tensor on cuda:", gpu));
  return {t.data_ptr(), t.nbytes()};
}

// A new tensor on the GPU of `like`, from the current stream's memory.  (at::empty comes to the same
// function through the dispatcher, a microsecond later.)
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}
Tensor given_or_new(PyObject* x, const char* name, at::IntArrayRef shape, const Tensor& like, at::ScalarType type) {
  return x != Py_None ? tensor(x, name) : fresh(shape, type, like);
}

float number(PyObject* x) {
  const double v = PyFloat_AsDouble(x);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}
float scale_of(PyObject* x, int64_t d) { return x == Py_None ? static_cast<float>(std::pow(d, -0.5)) : number(x); }
int truth(PyObject* x) {
  const int t = PyObject_IsTrue(x);
  if (t < 0) throw python_error();
  return t;
}

// The caller's stream (its handle), or the GPU's current one.  A given stream is the current one while the
// call allocates: an output, or a workspace let go when the call returns, comes from the memory of the
// stream that uses it, so that what other streams still do with freed memory cannot meet it, and what
// that stream gets the memory for next runs after the call.
class CallStream {
 public:
  CallStream(PyObject* x, int gpu) {
    if (x == Py_None) {
      handle_ = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(gpu)).stream();
      return;
    }
    void* p = PyLong_AsVoidPtr(x);
    if (!p && PyErr_Occurred()) throw python_error();
    handle_ = static_cast<cudaStream_t>(p);
    guard_.reset_stream(c10::cuda::getStreamFromExternal(handle_, static_cast<c10::DeviceIndex>(gpu)));
  }
  operator fa_stream_t() const { return reinterpret_cast<fa_stream_t>(handle_); }

 private:
  cudaStream_t handle_ = nullptr;
  c10::cuda::OptionalCUDAStreamGuard guard_;
};

// The sizes the library takes as int.
int whole(int64_t n, const char* name) {
  if (n > INT32_MAX || n < INT32_MIN) unfit(PyExc_ValueError, c10::str(name, " is too large: ", n));
  return static_cast<int>(n);
}

// fn() with the GPU current, and without the interpreter's lock (nothing in fn may throw).
template <class F>
int call(int gpu, F fn) {
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(gpu));
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = fn();
  Py_END_ALLOW_THREADS;
  return st;
}

PyObject* tuple_of(std::initializer_list<Tensor> ts) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!out) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* x = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (!x) {
      Py_DECREF(out);
      throw python_error();
    }
    PyTuple_SET_ITEM(out, i++, x);
  }
  return out;
}

void sizes4(const Tensor& t, const char* name) {
  if (t.dim() != 4) unfit(PyExc_ValueError, c10::str(name, " must have four dimensions, got shape ", t.sizes()));
}

// B, N, cu_docs, prefix, causal, plan (a tensor), stream
PyObject* mask_plan(PyObject* const* a) {
  const Tensor& plan = tensor(a[5], "plan");
  const int gpu = gpu_of(plan, "plan");
  const int64_t B = PyLong_AsLongLong(a[0]), N = PyLong_AsLongLong(a[1]);
  if (PyErr_Occurred()) throw python_error();
  int64_t docs = 1;
  if (a[2] != Py_None) {
    const Tensor& cu = tensor(a[2], "cu_docs");
    docs = cu.dim() == 2 ? cu.size(1) - 1 : 0;
  }
  const int32_t* cu = flat<const int32_t>(a[2], "cu_docs", at::kInt, {B, docs + 1}, gpu);
  const int32_t* prefix = flat<const int32_t>(a[3], "prefix", at::kInt, {B, docs}, gpu);
  const Bytes p = bytes(a[5], "plan", gpu);
  const int t = whole(docs, "cu_docs"), b = whole(B, "B"), n = whole(N, "N"), causal = truth(a[4]);
  const CallStream s(a[6], gpu);
  const int st = call(gpu, [&] { return fa_mask_plan(cu, prefix, t, p.p, p.n, b, n, causal, s); });
  if (st) return PyLong_FromLong(st);
  Py_RETURN_NONE;
}

// q, k, v, o, lse, causal, scale, softcap, slopes, plan, stream
PyObject* fwd_scored(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  sizes4(q, "q");
  sizes4(k, "k");
  const auto type = at::kBFloat16;
  if (q.scalar_type() != type) unfit(PyExc_TypeError, c10::str("q must be ", type, ", got ", q.scalar_type()));
  const int gpu = gpu_of(q, "q");
  const int64_t B = q.size(0), H = q.size(1), N = q.size(2), d = q.size(3), Hkv = k.size(1);
  const Layout lq = layout(q, "q", type, {B, H, N, d}, gpu), lk = layout(k, "k", type, {B, Hkv, N, d}, gpu),
               lv = layout(v, "v", type, {B, Hkv, N, d}, gpu);
  const CallStream s(a[10], gpu);
  const Tensor o = given_or_new(a[3], "o", {B, H, N, d}, q, type);
  const Tensor lse = given_or_new(a[4], "lse", {B, H, N}, q, at::kFloat);
  const Layout lo = layout(o, "o", type, {B, H, N, d}, gpu);
  check(lse, "lse", at::kFloat, {B, H, N}, gpu);
  if (!lse.is_contiguous()) unfit(PyExc_ValueError, "lse must be contiguous");
  const float* slopes = flat<const float>(a[8], "slopes", at::kFloat, {H}, gpu);
  const Bytes plan = bytes(a[9], "plan", gpu);
  const float scale = scale_of(a[6], d), cap = number(a[7]);
  const int causal = truth(a[5]), b = whole(B, "B"), h = whole(H, "H"), hkv = whole(Hkv, "Hkv"), n = whole(N, "N"),
            dim = whole(d, "d");
  const int st = call(gpu, [&] {
    return fa_fwd_scored(lq.p, lq.strides(), lk.p, lk.strides(), lv.p, lv.strides(), lo.p, lo.strides(),
                         static_cast<float*>(lse.data_ptr()), b, h, hkv, n, dim, plan.p, plan.n, causal,
                         scale, cap, slopes, s);
  });
  return st ? PyLong_FromLong(st) : tuple_of({o, lse});
}

// q, k, v, o, do, lse, dq, dk, dv, workspace, causal, scale, softcap, slopes, plan, stream, deterministic
PyObject* bwd_scored(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &o = tensor(a[3], "o"),
               &go = tensor(a[4], "do");
  sizes4(q, "q");
  sizes4(k, "k");
  const auto type = at::kBFloat16;
  if (q.scalar_type() != type) unfit(PyExc_TypeError, c10::str("q must be ", type, ", got ", q.scalar_type()));
  const int gpu = gpu_of(q, "q");
  const int64_t B = q.size(0), H = q.size(1), N = q.size(2), d = q.size(3), Hkv = k.size(1);
  const std::array<int64_t, 4> qs{B, H, N, d}, ks{B, Hkv, N, d};
  const Layout lq = layout(q, "q", type, qs, gpu), lk = layout(k, "k", type, ks, gpu), lv = layout(v, "v", type, ks, gpu),
               lo = layout(o, "o", type, qs, gpu), lg = layout(go, "do", type, qs, gpu);
  if (a[5] == Py_None) unfit(PyExc_TypeError, "lse must be a torch.Tensor");
  const float* lse = flat<const float>(a[5], "lse", at::kFloat, {B, H, N}, gpu);
  const CallStream s(a[15], gpu);
  const Tensor dq = given_or_new(a[6], "dq", qs, q, type), dk = given_or_new(a[7], "dk", ks, q, type),
               dv = given_or_new(a[8], "dv", ks, q, type);
  const Layout ldq = layout(dq, "dq", type, qs, gpu), ldk = layout(dk, "dk", type, ks, gpu),
               ldv = layout(dv, "dv", type, ks, gpu);
  const int b = whole(B, "B"), h = whole(H, "H"), hkv = whole(Hkv, "Hkv"), n = whole(N, "N"), dim = whole(d, "d");
  Tensor own;
  Bytes ws = bytes(a[9], "workspace", gpu);
  if (a[9] == Py_None) {
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(gpu));
    ws.n = fa_bwd_scored_workspace_size(b, h, hkv, n, dim);
    own = fresh({static_cast<int64_t>(ws.n)}, at::kByte, q);
    ws.p = own.data_ptr();
  }
  const float* slopes = flat<const float>(a[13], "slopes", at::kFloat, {H}, gpu);
  const Bytes plan = bytes(a[14], "plan", gpu);
  const float scale = scale_of(a[11], d), cap = number(a[12]);
  const int causal = truth(a[10]), deterministic = truth(a[16]);
  const int st = call(gpu, [&] {
    return fa_bwd_scored(lq.p, lq.strides(), lk.p, lk.strides(), lv.p, lv.strides(), lo.p, lo.strides(), lg.p,
                         lg.strides(), lse, ldq.p, ldq.strides(), ldk.p, ldk.strides(), ldv.p, ldv.strides(), ws.p, ws.n,
                         b, h, hkv, n, dim, plan.p, plan.n, causal, scale, cap, slopes, deterministic, s);
  });
  return st ? PyLong_FromLong(st) : tuple_of({dq, dk, dv});
}

// What the calls on a paged cache share.
struct Cache {
  at::ScalarType type;
  int code, gpu;
  Layout k, v;
  const int32_t *table, *lens;
  int64_t table_stride, B;
  int hkv, d, page, pages, width;
};
Cache cache_of(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo, bool codes = false) {
  const Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache"), &t = tensor(to, "page_table");
  Cache c;
  c.type = k.scalar_type();
  if (codes ? c.type != at::kFloat8_e4m3fn : c.type != at::kBFloat16 && c.type != at::kHalf)
    unfit(PyExc_TypeError, c10::str("k_cache must be ", codes ? "Float8_e4m3fn" : "BFloat16 or Half", ", got ", c.type));
  c.code = c.type == at::kBFloat16 ? 1 : 2;
  c.gpu = gpu_of(k, "k_cache");
  sizes4(k, "k_cache");
  if (t.dim() != 2) unfit(PyExc_ValueError, "page_table must be [B, max_pages]");
  c.k = layout(k, "k_cache", c.type, k.sizes(), c.gpu);
  c.v = layout(v, "v_cache", c.type, k.sizes(), c.gpu);
  c.B = t.size(0);
  check(t, "page_table", at::kInt, t.sizes(), c.gpu);
  if (t.size(1) > 1 && t.stride(1) != 1) unfit(PyExc_ValueError, "page_table must have contiguous rows");
  c.table = static_cast<const int32_t*>(t.data_ptr());
  c.table_stride = c.B > 1 ? t.stride(0) : std::max<int64_t>(t.size(1), t.stride(0));
  if (lo == Py_None) unfit(PyExc_TypeError, "seq_lens must be a torch.Tensor");
  c.lens = flat<const int32_t>(lo, "seq_lens", at::kInt, {c.B}, c.gpu);
  c.pages = whole(k.size(0), "n_pages");
  c.hkv = whole(k.size(1), "Hkv");
  c.page = whole(k.size(2), "page_size");
  c.d = whole(k.size(3), "d");
  c.width = whole(t.size(1), "max_pages");
  return c;
}

// k, v, k_cache, v_cache, page_table, seq_lens, cu_new, stream
PyObject* paged_append(PyObject* const* a) {
  const Cache c = cache_of(a[2], a[3], a[4], a[5]);
  const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  if (k.dim() != 3) unfit(PyExc_ValueError, "k must be [T, Hkv, d]");
  const int64_t T = k.size(0);
  const Layout lk = layout(k, "k", c.type, {T, c.hkv, c.d}, c.gpu), lv = layout(v, "v", c.type, {T, c.hkv, c.d}, c.gpu);
  if (a[6] == Py_None) unfit(PyExc_TypeError, "cu_new must be a torch.Tensor");
  const int32_t* cu = flat<const int32_t>(a[6], "cu_new", at::kInt, {c.B + 1}, c.gpu);
  const int b = whole(c.B, "B"), t = whole(T, "T");
  const CallStream s(a[7], c.gpu);
  const int st = call(c.gpu, [&] {
    return fa_paged_append(lk.p, lk.strides(), lv.p, lv.strides(), c.k.p, c.k.strides(), c.v.p, c.v.strides(), c.table,
                           c.table_stride, c.lens, cu, b, t, c.hkv, c.d, c.page, c.pages, c.width, c.code, s);
  });
  if (st) return PyLong_FromLong(st);
  Py_RETURN_NONE;
}

// q, k_cache, v_cache, page_table, seq_lens, o, lse, workspace, scale, softcap, slopes, stream
PyObject* paged_decode(PyObject* const* a) {
  const Cache c = cache_of(a[1], a[2], a[3], a[4]);
  const Tensor& q = tensor(a[0], "q");
  if (q.dim() != 3) unfit(PyExc_ValueError, "q must be [B, H, d]");
  const int64_t H = q.size(1);
  const Layout lq = layout(q, "q", c.type, {c.B, H, c.d}, c.gpu);
  const CallStream s(a[11], c.gpu);
  const Tensor o = given_or_new(a[5], "o", {c.B, H, c.d}, q, c.type);
  const Tensor lse = given_or_new(a[6], "lse", {c.B, H}, q, at::kFloat);
  const Layout lo = layout(o, "o", c.type, {c.B, H, c.d}, c.gpu);
  check(lse, "lse", at::kFloat, {c.B, H}, c.gpu);
  if (!lse.is_contiguous()) unfit(PyExc_ValueError, "lse must be contiguous");
  const int b = whole(c.B, "B"), h = whole(H, "H");
  Tensor own;
  Bytes ws = bytes(a[7], "workspace", c.gpu);
  if (a[7] == Py_None) {
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.gpu));
    ws.n = fa_paged_decode_workspace_size(b, h, c.hkv, c.d);
    own = fresh({static_cast<int64_t>(ws.n)}, at::kByte, q);
    ws.p = own.data_ptr();
  }
  const float* slopes = flat<const float>(a[10], "slopes", at::kFloat, {H}, c.gpu);
  const float scale = scale_of(a[8], c.d), cap = number(a[9]);
  const int st = call(c.gpu, [&] {
    return fa_paged_decode(lq.p, lq.strides(), c.k.p, c.k.strides(), c.v.p, c.v.strides(), c.table, c.table_stride,
                           c.lens, lo.p, lo.strides(), static_cast<float*>(lse.data_ptr()), ws.p, ws.n, b, h, c.hkv, c.d,
                           c.page, c.pages, c.width, c.code, scale, cap, slopes, s);
  });
  return st ? PyLong_FromLong(st) : tuple_of({o, lse});
}

// What the two calls on a cache of codes share with the 16-bit one's, and its scales.
struct Cache8 {
  Cache c;
  at::ScalarType type;  // of the 16-bit tensors
  float *k_scales, *v_scales;
};
Cache8 cache8_of(const Tensor& x, const char* name, PyObject* ko, PyObject* vo, PyObject* ks, PyObject* vs, PyObject* to,
                 PyObject* lo) {
  Cache8 r;
  r.type = x.scalar_type();
  if (r.type != at::kBFloat16 && r.type != at::kHalf)
    unfit(PyExc_TypeError, c10::str(name, " must be BFloat16 or Half, got ", r.type));
  r.c = cache_of(ko, vo, to, lo, true);
  r.c.code = r.type == at::kBFloat16 ? 1 : 2;
  const std::array<int64_t, 3> shape{r.c.pages, r.c.hkv, r.c.page / 16};
  if (ks == Py_None || vs == Py_None) unfit(PyExc_TypeError, "k_scales and v_scales must be torch.Tensors");
  r.k_scales = flat<float>(ks, "k_scales", at::kFloat, shape, r.c.gpu);
  r.v_scales = flat<float>(vs, "v_scales", at::kFloat, shape, r.c.gpu);
  return r;
}

// k, v, k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, cu_new, stream
PyObject* paged_append_fp8(PyObject* const* a) {
  const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  const Cache8 x = cache8_of(k, "k", a[2], a[3], a[4], a[5], a[6], a[7]);
  const Cache& c = x.c;
  if (k.dim() != 3) unfit(PyExc_ValueError, "k must be [T, Hkv, d]");
  const int64_t T = k.size(0);
  const Layout lk = layout(k, "k", x.type, {T, c.hkv, c.d}, c.gpu), lv = layout(v, "v", x.type, {T, c.hkv, c.d}, c.gpu);
  if (a[8] == Py_None) unfit(PyExc_TypeError, "cu_new must be a torch.Tensor");
  const int32_t* cu = flat<const int32_t>(a[8], "cu_new", at::kInt, {c.B + 1}, c.gpu);
  const int b = whole(c.B, "B"), t = whole(T, "T");
  const CallStream s(a[9], c.gpu);
  const int st = call(c.gpu, [&] {
    return fa_paged_append_fp8(lk.p, lk.strides(), lv.p, lv.strides(), c.k.p, c.k.strides(), c.v.p, c.v.strides(),
                               x.k_scales, x.v_scales, c.table, c.table_stride, c.lens, cu, b, t, c.hkv, c.d, c.page,
                               c.pages, c.width, c.code, s);
  });
  if (st) return PyLong_FromLong(st);
  Py_RETURN_NONE;
}

// q, k_cache, v_cache, k_scales, v_scales, page_table, seq_lens, o, lse, workspace, scale, softcap, slopes, stream
PyObject* paged_decode_fp8(PyObject* const* a) {
  const Tensor& q = tensor(a[0], "q");
  const Cache8 x = cache8_of(q, "q", a[1], a[2], a[3], a[4], a[5], a[6]);
  const Cache& c = x.c;
  if (q.dim() != 3) unfit(PyExc_ValueError, "q must be [B, H, d]");
  const int64_t H = q.size(1);
  const Layout lq = layout(q, "q", x.type, {c.B, H, c.d}, c.gpu);
  const CallStream s(a[13], c.gpu);
  const Tensor o = given_or_new(a[7], "o", {c.B, H, c.d}, q, x.type);
  const Tensor lse = given_or_new(a[8], "lse", {c.B, H}, q, at::kFloat);
  const Layout lo = layout(o, "o", x.type, {c.B, H, c.d}, c.gpu);
  check(lse, "lse", at::kFloat, {c.B, H}, c.gpu);
  if (!lse.is_contiguous()) unfit(PyExc_ValueError, "lse must be contiguous");
  const int b = whole(c.B, "B"), h = whole(H, "H");
  Tensor own;
  Bytes ws = bytes(a[9], "workspace", c.gpu);
  if (a[9] == Py_None) {
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.gpu));
    ws.n = fa_paged_decode_workspace_size(b, h, c.hkv, c.d);
    own = fresh({static_cast<int64_t>(ws.n)}, at::kByte, q);
    ws.p = own.data_ptr();
  }
  const float* slopes = flat<const float>(a[12], "slopes", at::kFloat, {H}, c.gpu);
  const float scale = scale_of(a[10], c.d), cap = number(a[11]);
  const int st = call(c.gpu, [&] {
    return fa_paged_decode_fp8(lq.p, lq.strides(), c.k.p, c.k.strides(), c.v.p, c.v.strides(), x.k_scales, x.v_scales,
                               c.table, c.table_stride, c.lens, lo.p, lo.strides(), static_cast<float*>(lse.data_ptr()),
                               ws.p, ws.n, b, h, c.hkv, c.d, c.page, c.pages, c.width, c.code, scale, cap, slopes, s);
  });
  return st ? PyLong_FromLong(st) : tuple_of({o, lse});
}

// n elements of a dense tensor from one on, as a tensor of its own on the same memory.  (A slice through the dispatcher takes
// longer than an allocation.)
Tensor part_of(const Tensor& all, int64_t from, int64_t n) {
  Tensor r = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(all.storage()), all.key_set(), all.dtype());
  r.unsafeGetTensorImpl()->set_storage_offset(all.storage_offset() + from);
  r.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return r;
}

// page_table, seq_lens, delta, free_pages, free_count, page_size, slots, positions, seq_lens_out, free_count_out, cu_new,
// status, workspace, stream
PyObject* paged_resize(PyObject* const* a) {
  const Tensor& t = tensor(a[0], "page_table");
  const int gpu = gpu_of(t, "page_table");
  if (t.dim() != 2) unfit(PyExc_ValueError, "page_table must be [B, max_pages]");
  const int64_t B = t.size(0), width = t.size(1);
  check(t, "page_table", at::kInt, t.sizes(), gpu);
  if (width > 1 && t.stride(1) != 1) unfit(PyExc_ValueError, "page_table must have contiguous rows");
  const int64_t stride = B > 1 ? t.stride(0) : std::max<int64_t>(width, t.stride(0));
  const char* needed[] = {"seq_lens", "delta", "free_pages", "free_count"};
  for (int i = 0; i < 4; ++i) tensor(a[1 + i], needed[i]);
  const int32_t* lens = flat<const int32_t>(a[1], "seq_lens", at::kInt, {B}, gpu);
  const int32_t* delta = flat<const int32_t>(a[2], "delta", at::kInt, {B}, gpu);
  const Tensor& list = tensor(a[3], "free_pages");
  int32_t* pages = flat<int32_t>(a[3], "free_pages", at::kInt, {list.numel()}, gpu);
  const int32_t* count = flat<const int32_t>(a[4], "free_count", at::kInt, {1}, gpu);
  const int64_t page = PyLong_AsLongLong(a[5]);
  if (PyErr_Occurred()) throw python_error();
  int64_t T = 0;
  if (a[6] != Py_None) T = tensor(a[6], "slots").numel();
  else if (a[7] != Py_None) T = tensor(a[7], "positions").numel();
  int64_t* slots = flat<int64_t>(a[6], "slots", at::kLong, {T}, gpu);
  int32_t* positions = flat<int32_t>(a[7], "positions", at::kInt, {T}, gpu);
  const CallStream s(a[13], gpu);
  // The outputs that are not given and the workspace are parts of one allocation (five take longer than the kernel).
  const int64_t words[5] = {B, 1, B + 1, 2, a[12] == Py_None ? static_cast<int64_t>(fa_paged_resize_workspace_size(whole(B, "B"))) / 4 : 0};
  int64_t total = words[4];
  for (int i = 0; i < 4; ++i) total += a[8 + i] == Py_None ? words[i] : 0;
  const Tensor all = fresh({total}, at::kInt, t);
  int64_t at_word = 0;
  auto out = [&](int i, const char* name) {
    Tensor r;
    if (a[8 + i] == Py_None) {
      r = part_of(all, at_word, words[i]);
      at_word += words[i];
    } else {
      r = tensor(a[8 + i], name);
      check(r, name, at::kInt, {words[i]}, gpu);
      if (!r.is_contiguous()) unfit(PyExc_ValueError, c10::str(name, " must be contiguous"));
    }
    return r;
  };
  const Tensor lens_out = out(0, "seq_lens_out"), count_out = out(1, "free_count_out"), cu = out(2, "cu_new"), status = out(3, "status");
  const int b = whole(B, "B"), w = whole(width, "max_pages"), n = whole(T, "T"), cap = whole(list.numel(), "free_pages"),
            ps = whole(page, "page_size");
  Bytes ws = bytes(a[12], "workspace", gpu);
  if (a[12] == Py_None) {
    ws.n = static_cast<size_t>(words[4]) * 4;
    ws.p = static_cast<int32_t*>(all.data_ptr()) + at_word;
  }
  const int st = call(gpu, [&] {
    auto ints = [](const Tensor& x) { return static_cast<int32_t*>(x.data_ptr()); };
    return fa_paged_resize(static_cast<int32_t*>(t.data_ptr()), stride, lens, delta, pages, cap, count, ints(lens_out),
                           ints(count_out), ints(cu), ints(status), slots, positions, n, ws.p, ws.n, b, ps, w, s);
  });
  return st ? PyLong_FromLong(st) : tuple_of({lens_out, cu, count_out, status});
}

// A new tensor of x's shape and type; heads beside each other in a token where x has them so.
Tensor fresh_like(const Tensor& x) {
  const int64_t B = x.size(0), H = x.size(1), N = x.size(2), d = x.size(3);
  if (H > 1 && N > 1 ? x.stride(1) < x.stride(2) : N > 1 && x.stride(2) > d)
    return at::detail::empty_strided_cuda({B, H, N, d}, {N * H * d, d, H * d, 1}, x.scalar_type(), x.device());
  return fresh({B, H, N, d}, x.scalar_type(), x);
}

// What the norm and rotation and its gradient share: q, k (tensors that give the sizes), the weights, frequencies and positions.
struct Qk {
  at::ScalarType type;
  int code, gpu, weight_code, b, h, hkv, n, d, rot, norm, pairs;
  int64_t B, H, Hkv, N, D;
  const void *qw, *kw;
  const float* freq;
  const int32_t* pos;
  float eps;
};
Qk qk_of(const Tensor& q, const char* qname, const Tensor& k, const char* kname, PyObject* qw, PyObject* kw, PyObject* freq,
         PyObject* pos, PyObject* eps, PyObject* norm, PyObject* pairs) {
  Qk x;
  sizes4(q, qname);
  sizes4(k, kname);
  x.type = q.scalar_type();
  if (x.type != at::kBFloat16 && x.type != at::kHalf)
    unfit(PyExc_TypeError, c10::str(qname, " must be BFloat16 or Half, got ", x.type));
  x.code = x.type == at::kBFloat16 ? 1 : 2;
  x.gpu = gpu_of(q, qname);
  x.B = q.size(0);
  x.H = q.size(1);
  x.N = q.size(2);
  x.D = q.size(3);
  x.Hkv = k.size(1);
  x.weight_code = 0;
  auto weight = [&](PyObject* w, const char* name) -> const void* {
    if (w == Py_None) return nullptr;
    const Tensor& t = tensor(w, name);
    const at::ScalarType type = t.scalar_type();
    if (type != at::kFloat && type != x.type)
      unfit(PyExc_ValueError, c10::str(name, " must be Float or ", x.type, ", got ", type));
    x.weight_code = type == at::kFloat ? 0 : x.code;
    return flat<void>(w, name, type, {x.D}, x.gpu);
  };
  x.qw = weight(qw, "q_weight");
  const int first = x.weight_code;
  x.kw = weight(kw, "k_weight");
  if (x.qw && x.kw && first != x.weight_code) unfit(PyExc_ValueError, "q_weight and k_weight must have the same dtype");
  if (x.qw && !x.kw) x.weight_code = first;
  const int64_t half = freq == Py_None ? 0 : tensor(freq, "inv_freq").numel();
  x.freq = half ? flat<const float>(freq, "inv_freq", at::kFloat, {half}, x.gpu) : nullptr;
  x.pos = flat<const int32_t>(pos, "positions", at::kInt, {x.B, x.N}, x.gpu);
  x.eps = number(eps);
  x.norm = truth(norm);
  x.pairs = truth(pairs);
  x.b = whole(x.B, "B");
  x.h = whole(x.H, "H");
  x.hkv = whole(x.Hkv, "Hkv");
  x.n = whole(x.N, "N");
  x.d = whole(x.D, "d");
  x.rot = whole(2 * half, "inv_freq");
  return x;
}

// q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out, eps, norm, interleaved, stream
PyObject* qk_norm_rope(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const Qk x = qk_of(q, "q", k, "k", a[2], a[3], a[4], a[5], a[8], a[9], a[10]);
  const std::array<int64_t, 4> qs{x.B, x.H, x.N, x.D}, ks{x.B, x.Hkv, x.N, x.D};
  const Layout lq = layout(q, "q", x.type, qs, x.gpu), lk = layout(k, "k", x.type, ks, x.gpu);
  const CallStream s(a[11], x.gpu);
  const Tensor qo = a[6] != Py_None ? tensor(a[6], "q_out") : fresh_like(q),
               ko = a[7] != Py_None ? tensor(a[7], "k_out") : fresh_like(k);
  const Layout lqo = layout(qo, "q_out", x.type, qs, x.gpu), lko = layout(ko, "k_out", x.type, ks, x.gpu);
  const int st = call(x.gpu, [&] {
    return fa_qk_norm_rope(lq.p, lq.strides(), lk.p, lk.strides(), x.qw, x.kw, x.freq, x.pos, lqo.p, lqo.strides(), lko.p,
                           lko.strides(), x.b, x.h, x.hkv, x.n, x.d, x.rot, x.norm, x.eps, x.weight_code, x.pairs, x.code, s);
  });
  return st ? PyLong_FromLong(st) : tuple_of({qo, ko});
}

// q, k, dq_out, dk_out, q_weight, k_weight, inv_freq, positions, dq, dk, workspace, eps, norm, interleaved, stream
PyObject* qk_norm_rope_bwd(PyObject* const* a) {
  const Tensor &gq = tensor(a[2], "dq_out"), &gk = tensor(a[3], "dk_out");
  const Qk x = qk_of(gq, "dq_out", gk, "dk_out", a[4], a[5], a[6], a[7], a[11], a[12], a[13]);
  const std::array<int64_t, 4> qs{x.B, x.H, x.N, x.D}, ks{x.B, x.Hkv, x.N, x.D};
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const Layout lq = layout(q, "q", x.type, qs, x.gpu), lk = layout(k, "k", x.type, ks, x.gpu),
               lgq = layout(gq, "dq_out", x.type, qs, x.gpu), lgk = layout(gk, "dk_out", x.type, ks, x.gpu);
  const CallStream s(a[14], x.gpu);
  const Tensor dq = a[8] != Py_None ? tensor(a[8], "dq") : fresh_like(gq),
               dk = a[9] != Py_None ? tensor(a[9], "dk") : fresh_like(gk);
  const Layout ldq = layout(dq, "dq", x.type, qs, x.gpu), ldk = layout(dk, "dk", x.type, ks, x.gpu);
  Tensor dqw, dkw, own;
  if (x.qw || x.kw) {
    const Tensor both = fresh({2 * x.D}, at::kFloat, gq);
    if (x.qw) dqw = part_of(both, 0, x.D);
    if (x.kw) dkw = part_of(both, x.D, x.D);
  }
  Bytes ws = bytes(a[10], "workspace", x.gpu);
  if (a[10] == Py_None && (x.qw || x.kw)) {
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(x.gpu));
    ws.n = fa_qk_norm_rope_bwd_workspace_size(x.d);
    own = fresh({static_cast<int64_t>(ws.n)}, at::kByte, gq);
    ws.p = own.data_ptr();
  }
  const int st = call(x.gpu, [&] {
    return fa_qk_norm_rope_bwd(lq.p, lq.strides(), lk.p, lk.strides(), lgq.p, lgq.strides(), lgk.p, lgk.strides(), x.qw,
                               x.kw, x.freq, x.pos, ldq.p, ldq.strides(), ldk.p, ldk.strides(),
                               x.qw ? static_cast<float*>(dqw.data_ptr()) : nullptr,
                               x.kw ? static_cast<float*>(dkw.data_ptr()) : nullptr, ws.p, ws.n, x.b, x.h, x.hkv, x.n, x.d,
                               x.rot, x.norm, x.eps, x.weight_code, x.pairs, x.code, s);
  });
  return st ? PyLong_FromLong(st) : tuple_of({dq, dk, dqw, dkw});
}

// No C++ exception leaves a function: its own become the Python exceptions they name,
// PyTorch's (an allocation that fails) those of PyTorch.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments given, %zd taken", n, N);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Unfit& e) {
    PyErr_SetString(e.type, e.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<mask_plan, 7>("mask_plan"),       method<fwd_scored, 11>("fwd_scored"),
                           method<bwd_scored, 17>("bwd_scored"),    method<paged_append, 8>("paged_append"),
                           method<paged_decode, 12>("paged_decode"),
                           method<paged_append_fp8, 10>("paged_append_fp8"),
                           method<paged_decode_fp8, 14>("paged_decode_fp8"), method<paged_resize, 14>("paged_resize"),
                           method<qk_norm_rope, 12>("qk_norm_rope"), method<qk_norm_rope_bwd, 15>("qk_norm_rope_bwd"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch(void) { return PyModule_Create(&g_module); }
