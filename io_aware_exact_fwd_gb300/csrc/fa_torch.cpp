// Binding of scored attention and of the paged cache to PyTorch tensors, for calls made
// once a layer and token: checks, output allocation and the C call in one step.  In
// Python with ctypes the same work takes 20 us a call on the GB300's host (a decode step
// 27 us where its kernels take 12), here about 1.
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
    PyObject* x = THPVariable_Wrap(t);
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

// What the two calls on a paged cache share.
struct Cache {
  at::ScalarType type;
  int code, gpu;
  Layout k, v;
  const int32_t *table, *lens;
  int64_t table_stride, B;
  int hkv, d, page, pages, width;
};
Cache cache_of(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo) {
  const Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache"), &t = tensor(to, "page_table");
  Cache c;
  c.type = k.scalar_type();
  if (c.type != at::kBFloat16 && c.type != at::kHalf)
    unfit(PyExc_TypeError, c10::str("k_cache must be BFloat16 or Half, got ", c.type));
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
                           method<paged_decode, 12>("paged_decode"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch(void) { return PyModule_Create(&g_module); }
