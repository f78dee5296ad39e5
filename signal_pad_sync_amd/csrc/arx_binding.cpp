// arx_binding.cpp — the compiled half of the Python binding's layer operators:
// checks the tensors, allocates outputs and workspaces through torch on the
// current stream, and calls the C ABI of arx.h through the addresses that
// bind() is given. A call of the smallest sizes is bound by the host, and the
// same checks in Python cost it two to three times as much.
//
// Every function takes its arguments by position, first the current device and
// its stream; signal_pad_sync_amd/arx.py documents and names them.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>
#include <utility>

#include "arx.h"

namespace {

// ---- what bind() is given ----------------------------------------------------

PyObject* g_error = nullptr;   // ArxError
struct {
  decltype(&arx_linear) linear;
  decltype(&arx_linear_workspace) linear_workspace;
  decltype(&arx_linear_backward) linear_backward;
  decltype(&arx_linear_backward_workspace) linear_backward_workspace;
  decltype(&arx_layer_norm) layer_norm;
  decltype(&arx_layer_norm_backward) layer_norm_backward;
  decltype(&arx_dropout_add) dropout_add;
  decltype(&arx_dropout_add_backward) dropout_add_backward;
  decltype(&arx_dropout_add_norm) dropout_add_norm;
  decltype(&arx_dropout_add_norm_backward) dropout_add_norm_backward;
  decltype(&arx_rows_workspace) rows_workspace;
  decltype(&arx_strerror) strerror;
} g_arx;

// An argument that the binding or the library refuses.
struct Refused {
  int code;
  std::string why;
};

[[noreturn]] void refuse(const char* fmt, ...) {
  char buf[320];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  throw Refused{ARX_EINVAL, buf};
}

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t n : t.sizes()) s += std::to_string(n) + ", ";
  s += "), strides (";
  for (int64_t n : t.strides()) s += std::to_string(n) + ", ";
  return s + ")";
}

int code_of(at::ScalarType t) {
  return t == at::kBFloat16 ? ARX_BF16 : t == at::kHalf ? ARX_F16 : t == at::kFloat ? ARX_F32 : -1;
}

struct Plane {
  void* p = nullptr;
  size_t ld = 0;
};

// One call: its first plane sets the type; every tensor is on the current
// device.
struct Call {
  PyObject* const* args;
  Py_ssize_t count;
  Py_ssize_t at = 2;
  int64_t device;
  hipStream_t stream;
  at::ScalarType type{};
  int dtype = -1;
  at::Tensor first;

  Call(PyObject* const* a, Py_ssize_t n, Py_ssize_t wanted) : args(a), count(n) {
    if (n != wanted) refuse("%zd arguments, %zd wanted", n, wanted);
    device = PyLong_AsLongLong(a[0]);
    stream = reinterpret_cast<hipStream_t>(PyLong_AsSize_t(a[1]));
    if (PyErr_Occurred()) throw python_error();
  }

  PyObject* next() { return args[at++]; }
  bool flag() {
    const int v = PyObject_IsTrue(next());
    if (v < 0) throw python_error();
    return v != 0;
  }
  int number() {
    const long v = PyLong_AsLong(next());
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return (int)v;
  }
  double real() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
  }
  uint64_t bits(const char* name) {
    PyObject* const o = next();
    const unsigned long long v = PyLong_Check(o) ? PyLong_AsUnsignedLongLong(o) : (unsigned long long)-1;
    if (v == (unsigned long long)-1 && (PyErr_Occurred() || !PyLong_Check(o))) {
      PyErr_Clear();
      refuse("%s must be an unsigned 64-bit number", name);
    }
    return v;
  }

  // The next argument as a tensor, or null for None.
  const at::Tensor* tensor(const char* name, bool optional) {
    PyObject* const o = next();
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
    return &THPVariable_Unpack(o);
  }

  void on_device(const at::Tensor& t, const char* name) const {
    if (!t.is_cuda()) refuse("%s must be a GPU tensor", name);
    if (t.get_device() != device) refuse("%s is on GPU %d, not on the current one", name, (int)t.get_device());
  }

  // The first plane: any shape of two dimensions, one of the call's types.
  const at::Tensor& lead(const char* name, bool matrix) {
    const at::Tensor& t = *tensor(name, false);
    type = t.scalar_type();
    dtype = code_of(type);
    if (dtype < 0 || (matrix && dtype == ARX_F32))
      refuse("%s is of type %s, not %s", name, toString(type), matrix ? "BFloat16 or Half" : "BFloat16, Half or Float");
    if (t.dim() != 2) refuse("%s has shape %s, not two dimensions", name, shape_of(t).c_str());
    first = t;
    return t;
  }

  Plane plane(const at::Tensor* t, const char* name, int64_t rows, int64_t cols) const {
    if (!t) return {};
    if (t->scalar_type() != type) refuse("%s is of type %s, not %s", name, toString(t->scalar_type()), toString(type));
    if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols)
      refuse("%s has shape %s, not (%lld, %lld)", name, shape_of(*t).c_str(), (long long)rows, (long long)cols);
    const int64_t ld = t->stride(0);
    if ((t->stride(1) != 1 && cols > 1) || (ld < cols && rows > 1))
      refuse("%s has shape %s: its rows must be contiguous and apart", name, shape_of(*t).c_str());
    on_device(*t, name);
    return {t->data_ptr(), (size_t)(rows > 1 || ld > cols ? ld : cols)};
  }

  void* vector(const at::Tensor* t, const char* name, int64_t n, at::ScalarType want) const {
    if (!t) return nullptr;
    if (t->scalar_type() != want) refuse("%s is of type %s, not %s", name, toString(t->scalar_type()), toString(want));
    if (t->dim() != 1 || t->size(0) != n || (n > 1 && t->stride(0) != 1))
      refuse("%s has shape %s, not (%lld,) in a row", name, shape_of(*t).c_str(), (long long)n);
    on_device(*t, name);
    return t->data_ptr();
  }

  at::Tensor empty(at::IntArrayRef shape) const { return at::empty(shape, first.options()); }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const { return at::empty(shape, first.options().dtype(t)); }
  // Two vectors of n that are kept and dropped together (a row's statistics), in
  // one allocation: one saves 0.7 us of the host's time.
  std::pair<at::Tensor, at::Tensor> two(int64_t n, at::ScalarType t) const {
    at::Tensor a = empty({2 * n}, t);
    at::Tensor b = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(a.storage()), a.key_set(), a.dtype());
    a.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    b.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    b.unsafeGetTensorImpl()->set_storage_offset(n);
    return {a, b};
  }
  at::Tensor space(size_t bytes) const {
    return bytes ? at::empty({(int64_t)bytes}, first.options().dtype(at::kByte)) : at::Tensor();
  }
};

void* address(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

void must(int rc) {
  if (rc != ARX_OK) throw Refused{rc, g_arx.strerror(rc)};
}

PyObject* tuple(std::initializer_list<at::Tensor> items) {
  PyObject* const t = PyTuple_New((Py_ssize_t)items.size());
  if (!t) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& x : items) {
    PyObject* o = Py_None;
    if (x.defined()) o = THPVariable_Wrap(x);
    else Py_INCREF(o);
    if (!o) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// Type of a norm's weight and shift: what is given, or the rows' own.
at::ScalarType norm_type(const Call& c, const at::Tensor* weight, const at::Tensor* shift) {
  const at::Tensor* const t = weight ? weight : shift;
  const at::ScalarType w = t ? t->scalar_type() : c.type;
  if (w != c.type && w != at::kFloat)
    refuse("%s is of type %s, not %s or Float", weight ? "weight" : "shift", toString(w), toString(c.type));
  return w;
}

bool on_lines(const Plane& a) { return ((uintptr_t)a.p & 15u) == 0 && a.ld % 8 == 0 && a.ld < ((size_t)1 << 22); }

// Whether p rounds to no dropout at all (arx.h, arx_dropout_add).
bool keeps_all(double p) { return p >= 0.0 && 65536.0 * p <= 0.5; }

// ---- the operators -----------------------------------------------------------

// (device, stream, x, w, bias, residual, act, save_z, out)
PyObject* linear(Call& c) {
  const at::Tensor& x = c.lead("x", true);
  const at::Tensor& w = *c.tensor("w", false);
  const at::Tensor* const bias = c.tensor("bias", true);
  const at::Tensor* const residual = c.tensor("residual", true);
  const int act = c.number();
  const bool save_z = c.flag();
  const at::Tensor* const given = c.tensor("out", true);
  const int64_t m = x.size(0), k = x.size(1), n = w.dim() == 2 ? w.size(0) : -1;
  const Plane wp = c.plane(&w, "w", n, k), rp = c.plane(residual, "residual", m, n);
  void* const bp = c.vector(bias, "bias", n, c.type);
  const Plane gp = c.plane(given, "out", m, n), xp = c.plane(&x, "x", m, k);
  const at::Tensor y = given ? *given : c.empty({m, n}), z = save_z ? c.empty({m, n}) : at::Tensor();
  const size_t bytes = g_arx.linear_workspace(m, n, k, on_lines(xp) && on_lines(wp));
  const at::Tensor space = c.space(bytes);
  must(g_arx.linear(xp.p, wp.p, bp, rp.p, y.data_ptr(), address(z), m, n, k, xp.ld, wp.ld, rp.ld, given ? gp.ld : n, n,
                    act, c.dtype, address(space), bytes, c.stream));
  return save_z ? tuple({y, z}) : THPVariable_Wrap(y);
}

// (device, stream, dy, x, w, z, act, dx, dw, dbias)
PyObject* linear_backward(Call& c) {
  const at::Tensor& dy = c.lead("dy", true);
  const at::Tensor& x = *c.tensor("x", false);
  const at::Tensor& w = *c.tensor("w", false);
  const at::Tensor* const z = c.tensor("z", true);
  const int act = c.number();
  const bool want_dx = c.flag(), want_dw = c.flag(), want_db = c.flag();
  const int64_t m = dy.size(0), n = dy.size(1), k = w.dim() == 2 ? w.size(1) : -1;
  const Plane wp = c.plane(&w, "w", n, k), xp = c.plane(&x, "x", m, k);
  if (act != ARX_ACT_NONE && !z) refuse("this activation needs z");
  const Plane zp = act == ARX_ACT_NONE ? Plane{} : c.plane(z, "z", m, n), dyp = c.plane(&dy, "dy", m, n);
  const at::Tensor none, dx = want_dx ? c.empty({m, k}) : none, dw = want_dw ? c.empty({n, k}) : none,
                         db = want_db ? c.empty({n}) : none;
  const size_t bytes =
      g_arx.linear_backward_workspace(m, n, k, act, on_lines(dyp) && on_lines(xp) && on_lines(wp));
  const at::Tensor space = c.space(bytes);
  must(g_arx.linear_backward(dyp.p, xp.p, wp.p, zp.p, address(dx), address(dw), address(db), m, n, k, dyp.ld, xp.ld,
                             wp.ld, zp.ld, k, k, act, c.dtype, address(space), bytes, c.stream));
  return tuple({dx, dw, db});
}

// (device, stream, x, weight, shift, eps, out)
PyObject* layer_norm(Call& c) {
  const at::Tensor& x = c.lead("x", false);
  const at::Tensor* const weight = c.tensor("weight", true);
  const at::Tensor* const shift = c.tensor("shift", true);
  const double eps = c.real();
  const at::Tensor* const given = c.tensor("out", true);
  const int64_t rows = x.size(0), cols = x.size(1);
  const at::ScalarType wt = norm_type(c, weight, shift);
  void *const wp = c.vector(weight, "weight", cols, wt), *const sp = c.vector(shift, "shift", cols, wt);
  const Plane gp = c.plane(given, "out", rows, cols), xp = c.plane(&x, "x", rows, cols);
  const at::Tensor y = given ? *given : c.empty({rows, cols});
  const auto [mean, rstd] = c.two(rows, at::kFloat);
  must(g_arx.layer_norm(xp.p, wp, sp, y.data_ptr(), (float*)address(mean), (float*)address(rstd), rows, cols, xp.ld,
                        given ? gp.ld : cols, eps, c.dtype, code_of(wt), c.stream));
  return tuple({y, mean, rstd});
}

// (device, stream, dy, x, mean, rstd, weight)
PyObject* layer_norm_backward(Call& c) {
  const at::Tensor& dy = c.lead("dy", false);
  const at::Tensor* const x = c.tensor("x", false);
  const at::Tensor* const mean = c.tensor("mean", false);
  const at::Tensor* const rstd = c.tensor("rstd", false);
  const at::Tensor* const weight = c.tensor("weight", true);
  const int64_t rows = dy.size(0), cols = dy.size(1);
  const at::ScalarType wt = norm_type(c, weight, nullptr);
  const Plane xp = c.plane(x, "x", rows, cols);
  const float *const mp = (float*)c.vector(mean, "mean", rows, at::kFloat),
              *const rp = (float*)c.vector(rstd, "rstd", rows, at::kFloat);
  void* const wp = c.vector(weight, "weight", cols, wt);
  const Plane dyp = c.plane(&dy, "dy", rows, cols);
  const at::Tensor dx = c.empty({rows, cols}), dw = c.empty({cols}, wt), ds = c.empty({cols}, wt);
  const size_t bytes = g_arx.rows_workspace(rows, cols, 2);
  const at::Tensor space = c.space(bytes);
  must(g_arx.layer_norm_backward(dyp.p, xp.p, mp, rp, wp, dx.data_ptr(), dw.data_ptr(), ds.data_ptr(), rows, cols,
                                 dyp.ld, xp.ld, cols, c.dtype, code_of(wt), address(space), bytes, c.stream));
  return tuple({dx, dw, ds});
}

// (device, stream, x, residual, bias, p, seed, offset, out)
PyObject* dropout_add(Call& c) {
  const at::Tensor& x = c.lead("x", false);
  const at::Tensor* const residual = c.tensor("residual", true);
  const at::Tensor* const bias = c.tensor("bias", true);
  const double p = c.real();
  const uint64_t seed = c.bits("seed"), offset = c.bits("offset");
  const at::Tensor* const given = c.tensor("out", true);
  const int64_t rows = x.size(0), cols = x.size(1);
  const Plane rp = c.plane(residual, "residual", rows, cols);
  void* const bp = c.vector(bias, "bias", cols, c.type);
  const Plane gp = c.plane(given, "out", rows, cols), xp = c.plane(&x, "x", rows, cols);
  const at::Tensor h = given ? *given : c.empty({rows, cols});
  must(g_arx.dropout_add(xp.p, bp, rp.p, h.data_ptr(), rows, cols, xp.ld, rp.ld, given ? gp.ld : cols, p, seed, offset,
                         c.dtype, c.stream));
  return THPVariable_Wrap(h);
}

// (device, stream, dh, p, seed, offset, dbias, share)
PyObject* dropout_add_backward(Call& c) {
  const at::Tensor& dh = c.lead("dh", false);
  const double p = c.real();
  const uint64_t seed = c.bits("seed"), offset = c.bits("offset");
  const bool want_db = c.flag(), share = c.flag();
  const int64_t rows = dh.size(0), cols = dh.size(1);
  const Plane dhp = c.plane(&dh, "dh", rows, cols);
  const bool same = share && keeps_all(p);   // dx is dh then
  const at::Tensor dx = same ? dh : c.empty({rows, cols}), db = want_db ? c.empty({cols}) : at::Tensor();
  const size_t bytes = want_db ? g_arx.rows_workspace(rows, cols, 1) : 0;
  const at::Tensor space = c.space(bytes);
  must(g_arx.dropout_add_backward(dhp.p, same ? nullptr : dx.data_ptr(), address(db), rows, cols, dhp.ld, cols, p, seed,
                                  offset, c.dtype, address(space), bytes, c.stream));
  return tuple({dx, db});
}

// (device, stream, x, residual, weight, shift, bias, p, seed, offset, eps, out)
PyObject* dropout_add_norm(Call& c) {
  const at::Tensor& x = c.lead("x", false);
  const at::Tensor* const residual = c.tensor("residual", true);
  const at::Tensor* const weight = c.tensor("weight", true);
  const at::Tensor* const shift = c.tensor("shift", true);
  const at::Tensor* const bias = c.tensor("bias", true);
  const double p = c.real();
  const uint64_t seed = c.bits("seed"), offset = c.bits("offset");
  const double eps = c.real();
  const at::Tensor* const given = c.tensor("out", true);
  const int64_t rows = x.size(0), cols = x.size(1);
  const at::ScalarType wt = norm_type(c, weight, shift);
  const Plane rp = c.plane(residual, "residual", rows, cols);
  void *const wp = c.vector(weight, "weight", cols, wt), *const sp = c.vector(shift, "shift", cols, wt),
             *const bp = c.vector(bias, "bias", cols, c.type);
  const Plane gp = c.plane(given, "out", rows, cols), xp = c.plane(&x, "x", rows, cols);
  const at::Tensor h = given ? *given : c.empty({rows, cols}), y = c.empty({rows, cols});
  const auto [mean, rstd] = c.two(rows, at::kFloat);
  must(g_arx.dropout_add_norm(xp.p, bp, rp.p, wp, sp, h.data_ptr(), y.data_ptr(), (float*)address(mean),
                              (float*)address(rstd), rows, cols, xp.ld, rp.ld, given ? gp.ld : cols, cols, eps, p, seed,
                              offset, c.dtype, code_of(wt), c.stream));
  return tuple({h, y, mean, rstd});
}

// (device, stream, dy, dh, h, mean, rstd, weight, p, seed, offset, dbias, share)
PyObject* dropout_add_norm_backward(Call& c) {
  const at::Tensor& dy = c.lead("dy", false);
  const at::Tensor* const dh = c.tensor("dh", true);
  const at::Tensor* const h = c.tensor("h", false);
  const at::Tensor* const mean = c.tensor("mean", false);
  const at::Tensor* const rstd = c.tensor("rstd", false);
  const at::Tensor* const weight = c.tensor("weight", true);
  const double p = c.real();
  const uint64_t seed = c.bits("seed"), offset = c.bits("offset");
  const bool want_db = c.flag(), share = c.flag();
  const int64_t rows = dy.size(0), cols = dy.size(1);
  const at::ScalarType wt = norm_type(c, weight, nullptr);
  const Plane dhp = c.plane(dh, "dh", rows, cols), hp = c.plane(h, "h", rows, cols);
  const float *const mp = (float*)c.vector(mean, "mean", rows, at::kFloat),
              *const rp = (float*)c.vector(rstd, "rstd", rows, at::kFloat);
  void* const wp = c.vector(weight, "weight", cols, wt);
  const Plane dyp = c.plane(&dy, "dy", rows, cols);
  const bool same = share && keeps_all(p);   // dresidual is dx then
  const at::Tensor dx = c.empty({rows, cols}), dr = same ? dx : c.empty({rows, cols}),
                   db = want_db ? c.empty({cols}) : at::Tensor(), dw = c.empty({cols}, wt), ds = c.empty({cols}, wt);
  const size_t bytes = g_arx.rows_workspace(rows, cols, 3);
  const at::Tensor space = c.space(bytes);
  must(g_arx.dropout_add_norm_backward(dyp.p, dhp.p, hp.p, mp, rp, wp, dx.data_ptr(), same ? nullptr : dr.data_ptr(),
                                       address(db), dw.data_ptr(), ds.data_ptr(), rows, cols, dyp.ld, dhp.ld, hp.ld, cols, cols, p,
                                       seed, offset, c.dtype, code_of(wt), address(space), bytes, c.stream));
  return tuple({dx, dr, db, dw, ds});
}

// ---- the module --------------------------------------------------------------

// A refusal becomes ArxError; any other C++ exception the one that torch makes
// of it.
template <PyObject* (*OP)(Call&), Py_ssize_t WANTED>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  try {
    Call c(args, count, WANTED);
    return OP(c);
  } catch (const Refused& r) {
    if (PyObject* const e = PyObject_CallFunction(g_error, "is", r.code, r.why.c_str())) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind(ArxError, {name: address}): where the library's functions stand.
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *error, *table;
  if (!PyArg_ParseTuple(args, "OO!", &error, &PyDict_Type, &table)) return nullptr;
  const auto set = [&](const char* name, auto* f) {
    PyObject* const v = PyDict_GetItemString(table, name);
    void* const p = v ? PyLong_AsVoidPtr(v) : nullptr;
    if (!p && !PyErr_Occurred()) PyErr_Format(PyExc_KeyError, "%s", name);
    *f = reinterpret_cast<std::remove_reference_t<decltype(*f)>>(p);
    return p != nullptr;
  };
  const bool ok = set("arx_linear", &g_arx.linear) && set("arx_linear_workspace", &g_arx.linear_workspace) &&
                  set("arx_linear_backward", &g_arx.linear_backward) &&
                  set("arx_linear_backward_workspace", &g_arx.linear_backward_workspace) &&
                  set("arx_layer_norm", &g_arx.layer_norm) &&
                  set("arx_layer_norm_backward", &g_arx.layer_norm_backward) &&
                  set("arx_dropout_add", &g_arx.dropout_add) &&
                  set("arx_dropout_add_backward", &g_arx.dropout_add_backward) &&
                  set("arx_dropout_add_norm", &g_arx.dropout_add_norm) &&
                  set("arx_dropout_add_norm_backward", &g_arx.dropout_add_norm_backward) &&
                  set("arx_rows_workspace", &g_arx.rows_workspace) && set("arx_strerror", &g_arx.strerror);
  if (!ok) return nullptr;
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

template <PyObject* (*OP)(Call&), Py_ssize_t WANTED>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<OP, WANTED>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    method<linear, 9>("linear"),
    method<linear_backward, 10>("linear_backward"),
    method<layer_norm, 7>("layer_norm"),
    method<layer_norm_backward, 7>("layer_norm_backward"),
    method<dropout_add, 9>("dropout_add"),
    method<dropout_add_backward, 8>("dropout_add_backward"),
    method<dropout_add_norm, 12>("dropout_add_norm"),
    method<dropout_add_norm_backward, 13>("dropout_add_norm_backward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
