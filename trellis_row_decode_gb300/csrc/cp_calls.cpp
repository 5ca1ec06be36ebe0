// cp_calls.cpp -- the projection's and dropout's calls from Python in their common form: contiguous
// tensors on the current device, outputs made here, the current stream.  What ctypes and
// interpreted checks cost, 5 to 9 us a call, is as much as the smallest kernels take.
//
// Each function answers NotImplemented for every other form and for whatever the library refuses;
// the caller (projection.py) then takes its own way, which checks, explains and raises, as it does for
// every call where this file is not built.  Tensors are read through their Python attributes: nothing
// here depends on PyTorch's C++ interface.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include "cp.h"

namespace {

// Objects of torch, found once when the module is made.
PyObject *t_empty, *t_f32, *t_f16, *t_bf16, *t_u8, *t_i64, *t_get_device, *t_get_stream;
PyObject *s_shape, *s_dtype, *s_device, *s_contiguous, *s_data_ptr, *s_get_device, *s_kwnames;

// A reference that is given back.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* q = nullptr) : p(q) {}
  ~Ref() { Py_XDECREF(p); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  PyObject* take() {
    PyObject* q = p;
    p = nullptr;
    return q;
  }
};

// A call that is not of the common form: whatever went wrong on the way here is found again, and
// explained, on the caller's own way.
PyObject* other_way() {
  PyErr_Clear();
  Py_RETURN_NOTIMPLEMENTED;
}

int type_code(PyObject* dtype) {
  return dtype == t_f32 ? CP_F32 : dtype == t_f16 ? CP_F16 : dtype == t_bf16 ? CP_BF16 : -1;
}

bool whole_number(PyObject* x, long long* out) {
  if (x == nullptr || !PyLong_Check(x)) return false;
  *out = PyLong_AsLongLong(x);
  return *out != -1 || !PyErr_Occurred();
}

constexpr int kMostDims = 16;

// A contiguous CUDA tensor as the calls want it.
struct Tensor {
  long long dims[kMostDims];
  int n_dims = 0;
  void* data = nullptr;
  long long device = -1;
  Ref dtype;
  long long last() const { return dims[n_dims - 1]; }
  long long rows() const {
    long long r = 1;
    for (int i = 0; i + 1 < n_dims; ++i) r *= dims[i];
    return r;
  }
};

bool read_tensor(PyObject* o, Tensor* t) {
  Ref whole(PyObject_CallMethodNoArgs(o, s_contiguous));
  if (whole.p != Py_True) return false;
  Ref device(PyObject_CallMethodNoArgs(o, s_get_device)), data(PyObject_CallMethodNoArgs(o, s_data_ptr));
  Ref shape(PyObject_GetAttr(o, s_shape));
  t->dtype.p = PyObject_GetAttr(o, s_dtype);
  if (device.p == nullptr || data.p == nullptr || shape.p == nullptr || t->dtype.p == nullptr ||
      !PyTuple_Check(shape.p) || !whole_number(device.p, &t->device) || t->device < 0)
    return false;
  t->data = reinterpret_cast<void*>(PyLong_AsUnsignedLongLong(data.p));
  const Py_ssize_t n = PyTuple_GET_SIZE(shape.p);
  if (PyErr_Occurred() || n < 1 || n > kMostDims) return false;
  t->n_dims = static_cast<int>(n);
  for (Py_ssize_t i = 0; i < n; ++i)
    if (!whole_number(PyTuple_GET_ITEM(shape.p, i), &t->dims[i]) || t->dims[i] < 0) return false;
  return true;
}

// The same rows: x's leading dimensions, `last` columns.
bool has_shape(const Tensor& t, const Tensor& x, long long last) {
  if (t.n_dims != x.n_dims || t.last() != last) return false;
  for (int i = 0; i + 1 < x.n_dims; ++i)
    if (t.dims[i] != x.dims[i]) return false;
  return true;
}

PyObject* empty(const long long* dims, int n, PyObject* dtype, PyObject* device, void** data) {
  Ref shape(PyTuple_New(n));
  if (shape.p == nullptr) return nullptr;
  for (int i = 0; i < n; ++i) {
    PyObject* d = PyLong_FromLongLong(dims[i]);
    if (d == nullptr) return nullptr;
    PyTuple_SET_ITEM(shape.p, i, d);
  }
  PyObject* args[4] = {nullptr, shape.p, dtype, device};
  Ref out(PyObject_Vectorcall(t_empty, args + 1, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, s_kwnames));
  if (out.p == nullptr) return nullptr;
  Ref at(PyObject_CallMethodNoArgs(out.p, s_data_ptr));
  if (at.p == nullptr) return nullptr;
  *data = reinterpret_cast<void*>(PyLong_AsUnsignedLongLong(at.p));
  return PyErr_Occurred() ? nullptr : out.take();
}
PyObject* empty_like_rows(const Tensor& x, long long last, PyObject* dtype, PyObject* device,
                          void** data) {
  long long dims[kMostDims];
  for (int i = 0; i + 1 < x.n_dims; ++i) dims[i] = x.dims[i];
  dims[x.n_dims - 1] = last;
  return empty(dims, x.n_dims, dtype, device, data);
}

// The current stream of x's device, which has to be the current one.
bool stream_of(const Tensor& x, void** stream) {
  Ref current(PyObject_CallNoArgs(t_get_device));
  long long dev = -1;
  if (current.p == nullptr || !whole_number(current.p, &dev) || dev != x.device) return false;
  Ref s(PyObject_CallOneArg(t_get_stream, current.p));
  if (s.p == nullptr) return false;
  *stream = reinterpret_cast<void*>(PyLong_AsUnsignedLongLong(s.p));
  return !PyErr_Occurred();
}

// p, seed, offset and rng of dropout.
struct Drop {
  double p = 0.0;
  unsigned long long seed = 0, offset = 0;
  const uint64_t* rng = nullptr;
};
bool read_drop(PyObject* const* a, const Tensor& x, Drop* d) {
  if ((!PyFloat_Check(a[0]) && !PyLong_Check(a[0])) || !PyLong_Check(a[1]) || !PyLong_Check(a[2]))
    return false;
  d->p = PyFloat_AsDouble(a[0]);
  d->seed = PyLong_AsUnsignedLongLong(a[1]);
  d->offset = PyLong_AsUnsignedLongLong(a[2]);
  if (PyErr_Occurred()) return false;
  if (a[3] == Py_None) return true;
  Tensor r;
  if (!read_tensor(a[3], &r) || r.dtype.p != t_i64 || r.n_dims != 1 || r.dims[0] != 2 ||
      r.device != x.device)
    return false;
  d->rng = static_cast<const uint64_t*>(r.data);
  return true;
}

constexpr long long kMostRow = (1ll << 32) - 1;

// The library's call, other threads running meanwhile: a launch waits where the stream's queue is
// full, and what it waits for may itself want the interpreter.
template <typename F>
cp_status unlocked(F call) {
  PyThreadState* state = PyEval_SaveThread();
  const cp_status status = call();
  PyEval_RestoreThread(state);
  return status;
}

// dropout(x, residual, p, seed, offset, rng)
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Tensor x, r;
  Drop d;
  void *stream = nullptr, *data = nullptr;
  if (n != 6 || !read_tensor(a[0], &x) || !read_drop(a + 2, x, &d) || x.last() > kMostRow ||
      !stream_of(x, &stream))
    return other_way();
  const int code = type_code(x.dtype.p);
  if (code < 0) return other_way();
  if (a[1] != Py_None && (!read_tensor(a[1], &r) || r.dtype.p != x.dtype.p ||
                          r.device != x.device || !has_shape(r, x, x.last())))
    return other_way();
  Ref device(PyObject_GetAttr(a[0], s_device));
  Ref out(device.p == nullptr ? nullptr : empty(x.dims, x.n_dims, x.dtype.p, device.p, &data));
  if (out.p == nullptr) return other_way();
  const uint64_t width = static_cast<uint64_t>(x.last());
  const uint64_t rows = static_cast<uint64_t>(x.rows());
  if (unlocked([&] {
        return cp_dropout(x.data, width, r.data, width, code, rows, static_cast<uint32_t>(width), d.p,
                          d.seed, d.offset, d.rng, data, width, stream);
      }) != CP_OK)
    return other_way();
  return out.take();
}

// linear(x, weight, bias, activation, residual, dtype, keep, p, seed, offset, rng); activation a
// number of cp.h, dtype None for x's; (out, pre) where keep is True
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Tensor x, w, b, r;
  Drop d;
  void *stream = nullptr, *out_data = nullptr, *pre_data = nullptr, *ws_data = nullptr;
  long long act = 0;
  if (n != 11 || !read_tensor(a[0], &x) || !read_tensor(a[1], &w) || !whole_number(a[3], &act) ||
      !read_drop(a + 7, x, &d) || !stream_of(x, &stream))
    return other_way();
  const int code = type_code(x.dtype.p);
  PyObject* out_type = a[5] == Py_None ? x.dtype.p : a[5];
  const int out_code = type_code(out_type);
  if ((code != CP_F16 && code != CP_BF16) || out_code < 0 || w.dtype.p != x.dtype.p ||
      w.n_dims != 2 || w.device != x.device || w.dims[1] != x.last())
    return other_way();
  const long long width = w.dims[0];
  int bias_code = 0;
  if (a[2] != Py_None) {
    if (!read_tensor(a[2], &b) || b.n_dims != 1 || b.dims[0] != width || b.device != x.device ||
        (bias_code = type_code(b.dtype.p)) < 0)
      return other_way();
  }
  if (a[4] != Py_None && (!read_tensor(a[4], &r) || r.dtype.p != out_type ||
                          r.device != x.device || !has_shape(r, x, width)))
    return other_way();
  const uint64_t m = static_cast<uint64_t>(x.rows()), wide = static_cast<uint64_t>(width),
                 k = static_cast<uint64_t>(x.last());
  Ref device(PyObject_GetAttr(a[0], s_device)), pre, ws;
  if (device.p == nullptr) return other_way();
  Ref out(empty_like_rows(x, width, out_type, device.p, &out_data));
  if (out.p == nullptr) return other_way();
  if (a[6] == Py_True) {
    pre.p = empty_like_rows(x, width, x.dtype.p, device.p, &pre_data);
    if (pre.p == nullptr) return other_way();
  }
  const uint64_t bytes = cp_linear_workspace_bytes(x.data, k, w.data, k, m, wide, k);
  if (bytes != 0) {
    const long long size = static_cast<long long>(bytes);
    ws.p = empty(&size, 1, t_u8, device.p, &ws_data);
    if (ws.p == nullptr) return other_way();
  }
  if (unlocked([&] {
        return cp_linear(x.data, k, w.data, k, code, m, wide, k, b.data, bias_code,
                         static_cast<int>(act), d.p, d.seed, d.offset, d.rng, r.data, wide, out_data,
                         out_code, wide, pre_data, wide, ws_data, bytes, stream);
      }) != CP_OK)
    return other_way();
  return pre.p == nullptr ? out.take() : PyTuple_Pack(2, out.p, pre.p);
}

// linear_grad(dy, x, weight, activation, pre, dw_dtype, db_dtype, p, seed, offset, rng): all three
// gradients, newly made
PyObject* linear_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Tensor dy, x, w, z;
  Drop d;
  void *stream = nullptr, *dx_data = nullptr, *dw_data = nullptr, *db_data = nullptr,
       *ws_data = nullptr;
  long long act = 0;
  if (n != 11 || !read_tensor(a[0], &dy) || !read_tensor(a[1], &x) || !read_tensor(a[2], &w) ||
      !whole_number(a[3], &act) || !read_drop(a + 7, x, &d) || !stream_of(x, &stream))
    return other_way();
  const int code = type_code(x.dtype.p), dy_code = type_code(dy.dtype.p);
  if ((code != CP_F16 && code != CP_BF16) || (dy_code != code && dy_code != CP_F32) ||
      w.dtype.p != x.dtype.p || w.n_dims != 2 || w.device != x.device || dy.device != x.device ||
      w.dims[1] != x.last() || !has_shape(dy, x, w.dims[0]) || (act != 0) != (a[4] != Py_None))
    return other_way();
  if (a[4] != Py_None && (!read_tensor(a[4], &z) || z.dtype.p != x.dtype.p ||
                          z.device != x.device || !has_shape(z, x, w.dims[0])))
    return other_way();
  PyObject* dw_type = a[5] == Py_None ? w.dtype.p : a[5];
  PyObject* db_type = a[6] == Py_None ? w.dtype.p : a[6];
  const int dw_code = type_code(dw_type), db_code = type_code(db_type);
  if (dw_code < 0 || db_code < 0) return other_way();
  const uint64_t m = static_cast<uint64_t>(x.rows()), wide = static_cast<uint64_t>(w.dims[0]),
                 k = static_cast<uint64_t>(x.last());
  const uint64_t bytes = cp_linear_grad_call_bytes(dy.data, dy_code, wide, x.data, k, w.data, k, code,
                                                   m, wide, k, static_cast<int>(act), d.p);
  const long long size = static_cast<long long>(bytes);
  Ref device(PyObject_GetAttr(a[1], s_device)), ws;
  if (device.p == nullptr) return other_way();
  Ref dx(empty(x.dims, x.n_dims, x.dtype.p, device.p, &dx_data));
  if (dx.p == nullptr) return other_way();
  Ref dw(empty(w.dims, 2, dw_type, device.p, &dw_data));
  if (dw.p == nullptr) return other_way();
  Ref db(empty(w.dims, 1, db_type, device.p, &db_data));
  if (db.p == nullptr) return other_way();
  if (bytes != 0) {
    ws.p = empty(&size, 1, t_u8, device.p, &ws_data);
    if (ws.p == nullptr) return other_way();
  }
  if (unlocked([&] {
        return cp_linear_grad(dy.data, dy_code, wide, x.data, k, w.data, k, code, z.data, wide, m,
                              wide, k, static_cast<int>(act), d.p, d.seed, d.offset, d.rng, 0,
                              dx_data, k, dw_data, dw_code, k, db_data, db_code, ws_data, bytes,
                              stream);
      }) != CP_OK)
    return other_way();
  return PyTuple_Pack(3, dx.p, dw.p, db.p);
}

// A function of C as Python's table wants it.
template <typename F>
PyCFunction as_method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"dropout", as_method(&dropout), METH_FASTCALL, nullptr},
                         {"linear", as_method(&linear), METH_FASTCALL, nullptr},
                         {"linear_grad", as_method(&linear_grad), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
  Ref torch(PyImport_ImportModule("torch"));
  if (torch.p == nullptr) return nullptr;
  Ref core(PyObject_GetAttrString(torch.p, "_C"));
  if (core.p == nullptr) return nullptr;
  const struct {
    PyObject** to;
    PyObject* from;
    const char* name;
  } found[] = {{&t_empty, torch.p, "empty"},
               {&t_f32, torch.p, "float32"},
               {&t_f16, torch.p, "float16"},
               {&t_bf16, torch.p, "bfloat16"},
               {&t_u8, torch.p, "uint8"},
               {&t_i64, torch.p, "int64"},
               {&t_get_device, core.p, "_cuda_getDevice"},
               {&t_get_stream, core.p, "_cuda_getCurrentRawStream"}};
  for (const auto& f : found)
    if ((*f.to = PyObject_GetAttrString(f.from, f.name)) == nullptr) return nullptr;
  const struct {
    PyObject** to;
    const char* name;
  } names[] = {{&s_shape, "shape"},         {&s_dtype, "dtype"},
               {&s_device, "device"},       {&s_contiguous, "is_contiguous"},
               {&s_data_ptr, "data_ptr"},   {&s_get_device, "get_device"}};
  for (const auto& f : names)
    if ((*f.to = PyUnicode_InternFromString(f.name)) == nullptr) return nullptr;
  s_kwnames = Py_BuildValue("(ss)", "dtype", "device");
  return s_kwnames == nullptr ? nullptr : PyModule_Create(&module);
}
