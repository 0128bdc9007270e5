// binding.cpp -- the packed and cache calls of the Python binding, compiled: checks
// of the tensors, outputs and workspace from torch's allocator, and one call of the
// C ABI.  A step of one sequence is 5 us of GPU work; with these checks and
// allocations written in Python a call took 19 us, so it takes 6.5 (a packed prompt
// of short turns 24 -> 10.5, an eviction read back 52 -> 26).  Arguments are
// positional, as the wrappers in __init__.py pass them (None where they have a
// default).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <string>

#include "fa.h"

namespace {

PyObject* g_error = nullptr;  // FAError(function, code)

struct Raised {};  // a Python error is set

[[noreturn]] void raise(PyObject* type, const std::string& message) {
  PyErr_SetString(type, message.c_str());
  throw Raised{};
}
[[noreturn]] void type_error(const std::string& message) { raise(PyExc_TypeError, message); }
[[noreturn]] void value_error(const std::string& message) { raise(PyExc_ValueError, message); }

void check(const char* function, int code) {
  if (code == FA_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "si", function, code);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

// One call of the C ABI, other Python threads running meanwhile (a launch can wait for
// room in its queue).
struct Unlocked {
  PyThreadState* threads = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(threads); }
};

template <typename F>
void call(const char* function, F f) {
  int code;
  {
    const Unlocked unlocked;
    code = f();
  }
  check(function, code);
}

// ------------------------------------------------------------------ arguments

int to_int(PyObject* o) {
  PyObject* i = PyNumber_Index(o);
  if (!i) throw Raised{};
  int over = 0;
  const long x = PyLong_AsLongAndOverflow(i, &over);
  Py_DECREF(i);
  if (over || x < INT_MIN || x > INT_MAX) raise(PyExc_OverflowError, "integer out of range");
  return (int)x;
}

float to_scale(PyObject* o, int D) {
  if (o == Py_None) return (float)(1.0 / std::sqrt((double)D));
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)x;
}

bool to_bool(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raised{};
  return x != 0;
}

const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

std::string shape_text(at::IntArrayRef s) {
  std::string x = "(";
  for (size_t i = 0; i < s.size(); ++i) x += (i ? ", " : "") + std::to_string(s[i]);
  return x + (s.size() == 1 ? ",)" : ")");
}

// A packed [T, H, D] bf16 CUDA tensor and its strides.
struct Packed {
  const at::Tensor* t;
  fa_packed_stride s;
  bool plain;  // contiguous
  const fa_packed_stride* stride() const { return plain ? nullptr : &s; }
  int64_t size(int d) const { return t->size(d); }
  int device() const { return t->get_device(); }
};

Packed packed(PyObject* o, const char* name, const Packed* like = nullptr) {
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->scalar_type() != at::kBFloat16)
    type_error(std::string(name) + " must be a bfloat16 CUDA tensor");
  if (t->dim() != 3)
    value_error(std::string(name) + " must be [tokens, heads, head dimension]");
  if (like && (t->sizes() != like->t->sizes() || t->get_device() != like->device()))
    value_error(std::string(name) + " must be " + shape_text(like->t->sizes()) + " on the same device");
  for (int d = 0; d < 3; ++d)
    if (t->size(d) > INT_MAX) value_error(std::string(name) + " is too large");
  Packed p{t, {0, 0}, t->is_contiguous()};
  if (p.plain) return p;
  const int64_t T = t->size(0), H = t->size(1), D = t->size(2);
  if (D > 1 && t->stride(2) != 1) value_error(std::string(name) + " must have contiguous elements");
  // the stride of a dimension of one element is arbitrary: give the kernel a valid one
  p.s.head = H > 1 ? t->stride(1) : D;
  p.s.token = T > 1 ? t->stride(0) : std::max(H * D, p.s.head);
  return p;
}

// A contiguous tensor of the caller.
const at::Tensor& given(PyObject* o, at::IntArrayRef shape, at::ScalarType dtype, int device,
                        const char* name) {
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->scalar_type() != dtype || t->get_device() != device ||
      t->sizes() != shape || !t->is_contiguous())
    value_error(std::string(name) + " must be a contiguous " + c10::toString(dtype) + " tensor " +
                shape_text(shape) + " on the inputs' device");
  return *t;
}

// The device and the stream of a call made current: memory that the call allocates
// comes from the pool of the stream that writes it, so nothing queued elsewhere still
// uses it, and what the call drops (a workspace) goes back there behind its kernels.
struct Place {
  int device;
  c10::cuda::OptionalCUDAGuard on_device;
  c10::cuda::CUDAStream caller;  // the current stream of the device before the call
  c10::cuda::OptionalCUDAStreamGuard on_stream;
  fa_stream_t stream;
  Place(int d, PyObject* s) : device(d), caller(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)d)) {
    if (c10::cuda::current_device() != d) on_device.set_index((c10::DeviceIndex)d);
    stream = caller.stream();
    if (s == Py_None) return;
    PyObject* h = PyObject_GetAttrString(s, "cuda_stream");
    if (!h) throw Raised{};
    stream = reinterpret_cast<fa_stream_t>(PyLong_AsUnsignedLongLong(h));
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Raised{};
    if (stream != caller.stream())
      on_stream.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream),
                                                              (c10::DeviceIndex)d));
  }
  bool elsewhere() const { return stream != static_cast<fa_stream_t>(caller.stream()); }
};

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const Place& place) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(c10::Device(at::kCUDA, place.device)));
}

// The same, or for None a new one, whose memory stays until the caller's stream, where
// it is used next, has passed.
at::Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType dtype, const Place& place,
                  const char* name) {
  if (o != Py_None) return given(o, shape, dtype, place.device, name);
  at::Tensor t = fresh(shape, dtype, place);
  if (place.elsewhere()) t.record_stream(place.caller.unwrap());
  return t;
}

at::Tensor workspace(PyObject* o, size_t bytes, const Place& place) {
  if (o == Py_None) return fresh({(int64_t)(bytes ? bytes : 1)}, at::kByte, place);
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->get_device() != place.device || !t->is_contiguous())
    value_error("workspace must be a contiguous tensor on the inputs' device");
  return *t;
}

// An int32 CUDA vector of n elements (n < 0: any number).
const int* int32s(PyObject* o, int64_t n, int device, const char* name, int64_t* size = nullptr) {
  const at::Tensor* t = tensor(o);
  if (!t || t->get_device() != device || t->scalar_type() != at::kInt || t->dim() != 1 ||
      !t->is_contiguous())
    type_error(std::string(name) + " must be a contiguous int32 vector on the inputs' device");
  if ((n >= 0 && t->size(0) != n) || t->size(0) > INT_MAX)
    value_error(std::string(name) + " must have " + std::to_string(n) + " elements");
  if (size) *size = t->size(0);
  return static_cast<const int*>(t->data_ptr());
}

struct Cache {
  void* p;
  int pages, Hkv, page, device;
};

// A 4-bit cache tensor for head dimension D.
Cache cache4(PyObject* o, int64_t D) {
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->scalar_type() != at::kByte) type_error("cache must be a uint8 CUDA tensor");
  if (t->dim() != 3 || !t->is_contiguous() || (D != 64 && D != 128))
    value_error("cache must be a contiguous [pages, Hkv, bytes] tensor of cache4_empty, with head "
                "dimension 64 or 128");
  const int64_t bytes = t->size(2), page = bytes / (D + D / 4);
  if (bytes % (D + D / 4) || (page != 16 && page != 32 && page != 64 && page != 128))
    value_error("cache pages of " + std::to_string(bytes) + " bytes do not hold tokens of " +
                std::to_string(D) + " elements");
  if (t->size(0) > INT_MAX || t->size(1) > INT_MAX) value_error("cache is too large");
  return {t->data_ptr(), (int)t->size(0), (int)t->size(1), (int)page, t->get_device()};
}

const int* page_table(PyObject* o, int64_t B, int device, int* width, const char* name = "page_table") {
  const at::Tensor* t = tensor(o);
  if (!t || t->get_device() != device || t->scalar_type() != at::kInt || !t->is_contiguous())
    type_error(std::string(name) + " must be a contiguous int32 tensor on the cache's device");
  if (t->dim() != 2 || t->size(0) != B || t->size(1) < 1 || t->size(1) > INT_MAX)
    value_error(std::string(name) + " must be [" + std::to_string(B) + ", pages per sequence]");
  *width = (int)t->size(1);
  return static_cast<const int*>(t->data_ptr());
}

float* weights(PyObject* o, int64_t B, int Hkv, int device, int* slots, const char* name) {
  const at::Tensor* t = tensor(o);
  if (!t || t->get_device() != device || t->scalar_type() != at::kFloat || !t->is_contiguous())
    type_error(std::string(name) + " must be a contiguous fp32 tensor on the cache's device");
  if (t->dim() != 3 || t->size(0) != B || t->size(1) != Hkv || t->size(2) < 1 || t->size(2) > INT_MAX)
    value_error(std::string(name) + " must be [" + std::to_string(B) + ", " + std::to_string(Hkv) +
                ", slots]");
  *slots = (int)t->size(2);
  return static_cast<float*>(t->data_ptr());
}

template <typename... T>
PyObject* tuple(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(t));
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  bool ok = true;
  ((ok = ok && [&] {
      PyObject* w = THPVariable_Wrap(t);
      if (w) PyTuple_SET_ITEM(r, i++, w);
      return w != nullptr;
    }()),
   ...);
  if (!ok) {
    Py_DECREF(r);
    throw Raised{};
  }
  return r;
}

// ------------------------------------------------------------------ packed sequences

struct PackedInputs {
  Packed q, k, v;
  int T, Hq, Hkv, D, device;
};

PackedInputs packed_inputs(PyObject* const* a) {
  const Packed q = packed(a[0], "q"), k = packed(a[1], "k");
  if (k.size(0) != q.size(0) || k.size(2) != q.size(2) || k.device() != q.device())
    value_error("k must have q's tokens, head dimension and device");
  const Packed v = packed(a[2], "v", &k);
  return {q, k, v, (int)q.size(0), (int)q.size(1), (int)k.size(1), (int)q.size(2), q.device()};
}

// q, k, v, cu_seqlens, window left, right, scale, out, lse, workspace, stream
PyObject* fwd_varlen(PyObject* const* a) {
  const PackedInputs x = packed_inputs(a);
  const Place place(x.device, a[10]);
  int64_t n;
  const int* cu = int32s(a[3], -1, x.device, "cu_seqlens", &n);
  const int B = (int)n - 1, wl = to_int(a[4]), wr = to_int(a[5]);
  const float scale = to_scale(a[6], x.D);
  const at::Tensor o = output(a[7], {x.T, x.Hq, x.D}, at::kBFloat16, place, "out");
  const at::Tensor lse = output(a[8], {x.Hq, x.T}, at::kFloat, place, "lse");
  const size_t need = a[9] == Py_None ? fa_varlen_workspace_bytes(B, x.T, x.Hq, x.Hkv, x.D, 0, 0) : 0;
  const at::Tensor ws = workspace(a[9], need, place);
  call("fa_fwd_varlen", [&] {
    return fa_fwd_varlen(x.q.t->data_ptr(), x.k.t->data_ptr(), x.v.t->data_ptr(), o.data_ptr(),
                         static_cast<float*>(lse.data_ptr()), cu, B, x.T, x.Hq, x.Hkv, x.D,
                         x.q.stride(), x.k.stride(), x.v.stride(), wl, wr, scale, ws.data_ptr(),
                         ws.nbytes(), place.stream);
  });
  return tuple(o, lse);
}

// q, k, v, o, do, lse, cu_seqlens, window left, right, scale, deterministic,
// workspace, dq, dk, dv, stream
PyObject* bwd_varlen(PyObject* const* a) {
  const PackedInputs x = packed_inputs(a);
  PyObject* const stream = a[15];
  const Place place(x.device, stream);
  const auto q_shape = x.q.t->sizes(), k_shape = x.k.t->sizes();
  const at::Tensor& o = given(a[3], q_shape, at::kBFloat16, x.device, "o");
  const at::Tensor& dO = given(a[4], q_shape, at::kBFloat16, x.device, "do");
  const at::Tensor& lse = given(a[5], {x.Hq, x.T}, at::kFloat, x.device, "lse");
  int64_t n;
  const int* cu = int32s(a[6], -1, x.device, "cu_seqlens", &n);
  const int B = (int)n - 1, wl = to_int(a[7]), wr = to_int(a[8]);
  const float scale = to_scale(a[9], x.D);
  const int det = to_bool(a[10]) ? 1 : 0;
  const size_t need = a[11] == Py_None ? fa_varlen_workspace_bytes(B, x.T, x.Hq, x.Hkv, x.D, 1, det) : 0;
  const at::Tensor ws = workspace(a[11], need, place);
  const at::Tensor dq = output(a[12], q_shape, at::kBFloat16, place, "dq");
  const at::Tensor dk = output(a[13], k_shape, at::kBFloat16, place, "dk");
  const at::Tensor dv = output(a[14], k_shape, at::kBFloat16, place, "dv");
  call("fa_bwd_varlen", [&] {
    return fa_bwd_varlen(x.q.t->data_ptr(), x.k.t->data_ptr(), x.v.t->data_ptr(), o.data_ptr(),
                         dO.data_ptr(), static_cast<const float*>(lse.data_ptr()), dq.data_ptr(),
                         dk.data_ptr(), dv.data_ptr(), cu, B, x.T, x.Hq, x.Hkv, x.D, x.q.stride(),
                         x.k.stride(), x.v.stride(), wl, wr, scale, ws.data_ptr(), ws.nbytes(),
                         det, place.stream);
  });
  return tuple(dq, dk, dv);
}

// ------------------------------------------------------------------ 4-bit cache

// cache, k, v, page_table, cache_lens, cu_seqlens, stream
PyObject* cache4_append(PyObject* const* a) {
  const Packed k = packed(a[1], "k"), v = packed(a[2], "v", &k);
  const int T = (int)k.size(0), Hkv = (int)k.size(1), D = (int)k.size(2), device = k.device();
  const Cache c = cache4(a[0], D);
  if (c.Hkv != Hkv || c.device != device) value_error("cache and k must have the same kv heads and device");
  const Place place(device, a[6]);
  int64_t B;
  const int* lens = int32s(a[4], -1, device, "cache_lens", &B);
  int width;
  const int* table = page_table(a[3], B, device, &width);
  const int* cu = a[5] == Py_None ? nullptr : int32s(a[5], B + 1, device, "cu_seqlens");
  call("fa_cache4_append", [&] {
    return fa_cache4_append(c.p, c.pages, c.page, k.t->data_ptr(), v.t->data_ptr(), k.stride(),
                            v.stride(), (int)B, T, Hkv, D, cu, lens, table, width, place.stream);
  });
  Py_RETURN_NONE;
}

// cache, page_table, first, count, S, D, k, v, stream
PyObject* cache4_read(PyObject* const* a) {
  const int S = to_int(a[4]), D = to_int(a[5]);
  const Cache c = cache4(a[0], D);
  const Place place(c.device, a[8]);
  int64_t B;
  const int* count = int32s(a[3], -1, c.device, "count", &B);
  int width;
  const int* table = page_table(a[1], B, c.device, &width);
  const int* first = a[2] == Py_None ? nullptr : int32s(a[2], B, c.device, "first");
  if (S < 0) check("fa_cache4_read", 1);
  const at::Tensor k = output(a[6], {B, c.Hkv, S, D}, at::kBFloat16, place, "k");
  const at::Tensor v = output(a[7], {B, c.Hkv, S, D}, at::kBFloat16, place, "v");
  call("fa_cache4_read", [&] {
    return fa_cache4_read(c.p, c.pages, c.page, k.data_ptr(), v.data_ptr(), (int)B, c.Hkv, S, D,
                          first, count, table, width, place.stream);
  });
  return tuple(k, v);
}

// q, cache, page_table, cache_lens, scale, weights, weights_out, out, lse, workspace,
// stream
PyObject* cache4_attend(PyObject* const* a) {
  const Packed q = packed(a[0], "q");
  const int B = (int)q.size(0), Hq = (int)q.size(1), D = (int)q.size(2), device = q.device();
  const Cache c = cache4(a[1], D);
  if (c.device != device) value_error("cache and q must be on one device");
  PyObject* const stream = a[10];
  const Place place(device, stream);
  const int* lens = int32s(a[3], B, device, "cache_lens");
  int width, slots = 0;
  const int* table = page_table(a[2], B, device, &width);
  const float scale = to_scale(a[4], D);
  float *w_in = nullptr, *w_out = nullptr;
  if (a[5] != Py_None) w_in = w_out = weights(a[5], B, c.Hkv, device, &slots, "weights");
  if (a[6] != Py_None) {
    int n;
    w_out = weights(a[6], B, c.Hkv, device, &n, "weights_out");
    if (w_in && n != slots) value_error("weights_out must have weights' shape");
    slots = n;
  }
  const at::Tensor o = output(a[7], {B, Hq, D}, at::kBFloat16, place, "out");
  const at::Tensor lse = output(a[8], {B, Hq}, at::kFloat, place, "lse");
  const size_t need =
      a[9] == Py_None ? fa_cache4_attend_workspace_bytes(B, Hq, c.Hkv, D, slots) : 0;
  const at::Tensor ws = workspace(a[9], need, place);
  // the stride of a dimension of one element is arbitrary
  call("fa_cache4_attend", [&] {
    return fa_cache4_attend(q.t->data_ptr(), B > 1 ? q.t->stride(0) : 0,
                            Hq > 1 ? q.t->stride(1) : 0, c.p, c.pages, c.page, o.data_ptr(),
                            static_cast<float*>(lse.data_ptr()), B, Hq, c.Hkv, D, lens, table,
                            width, scale, w_in, w_out, slots, ws.data_ptr(), ws.nbytes(),
                            place.stream);
  });
  return tuple(o, lse);
}

// cache, page_table, cache_lens, weights, out_page_table, D, budget, recent, src,
// weights_out, lens_out, stream
PyObject* cache4_evict(PyObject* const* a) {
  const int D = to_int(a[5]), budget = to_int(a[6]), recent = to_int(a[7]);
  const Cache c = cache4(a[0], D);
  PyObject* const stream = a[11];
  const Place place(c.device, stream);
  int64_t B;
  const int* lens = int32s(a[2], -1, c.device, "cache_lens", &B);
  int width, out_width, cap;
  const int* table = page_table(a[1], B, c.device, &width);
  const int* out_table = page_table(a[4], B, c.device, &out_width, "out_page_table");
  const float* w = weights(a[3], B, c.Hkv, c.device, &cap, "weights");
  if (budget < 1 || recent < 0 || recent > budget || (int64_t)out_width * c.page < budget)
    value_error("budget must be positive, at least recent and within out_page_table");
  const at::Tensor src = output(a[8], {B, c.Hkv, budget}, at::kInt, place, "src");
  const at::Tensor w_out = output(a[9], {B, c.Hkv, budget}, at::kFloat, place, "weights_out");
  const at::Tensor lens_out = output(a[10], {B}, at::kInt, place, "lens_out");
  call("fa_cache4_evict", [&] {
    return fa_cache4_evict(c.p, c.pages, c.page, w, cap, lens, table, width, (int)B, c.Hkv, D,
                           budget, recent, out_table, out_width, static_cast<int*>(src.data_ptr()),
                           static_cast<float*>(w_out.data_ptr()),
                           static_cast<int*>(lens_out.data_ptr()), place.stream);
  });
  return tuple(src, w_out, lens_out);
}

// ------------------------------------------------------------------ module

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != N) type_error("expected " + std::to_string(N) + " arguments");
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL,
          nullptr};
}

PyMethodDef g_methods[] = {method<fwd_varlen, 11>("fwd_varlen"),
                           method<bwd_varlen, 16>("bwd_varlen"),
                           method<cache4_append, 7>("cache4_append"),
                           method<cache4_read, 9>("cache4_read"),
                           method<cache4_attend, 11>("cache4_attend"),
                           method<cache4_evict, 12>("cache4_evict"),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
