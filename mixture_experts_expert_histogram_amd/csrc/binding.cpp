// Native half of the Python binding for the operators around the routed
// experts: checks, outputs and the call of the C ABI.  These calls take a few
// microseconds on the GPU, and their checks in Python took longer (residual_fwd
// 13.9 us a call); the functions here are those of _lib.py with every argument
// given by position.  A wrong tensor raises ValueError, a status of the library
// MoeError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/moe.h"

namespace {

using at::Tensor;
using Shape = std::vector<int64_t>;

PyObject *g_check = nullptr, *g_stream = nullptr;   // _lib._check(status, where), _lib._raw_stream(device index)

struct PythonError {};   // an exception is set already

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

std::string list(at::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
void need(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dtype, c10::Device device) {
  if (t.scalar_type() == dtype && t.sizes() == shape && t.device() == device && t.is_contiguous()) return;
  std::ostringstream o;
  o << name << " must be a contiguous " << dtype << " tensor of shape " << list(shape) << " on " << device << ", got "
    << t.scalar_type() << " " << list(t.sizes()) << " on " << t.device() << (t.is_contiguous() ? "" : ", not contiguous");
  refuse(o.str());
}
void* data(const Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }

// The pointer of an optional input, checked.
const void* input(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dtype, c10::Device device) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, name);
  need(t, name, shape, dtype, device);
  return t.data_ptr();
}
// An output: the given tensor, checked, or a new one.
Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dtype, c10::Device device) {
  if (o == Py_None) return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
  const Tensor& t = tensor(o, name);
  need(t, name, shape, dtype, device);
  return t;
}
Tensor workspace(PyObject* o, size_t bytes, c10::Device device) {
  if (o == Py_None)
    return at::empty({(int64_t)(bytes < 256 ? 256 : bytes)}, at::TensorOptions().dtype(at::kByte).device(device));
  const Tensor& t = tensor(o, "ws");
  if (t.device() != device || !t.is_contiguous()) refuse("ws must be contiguous, on " + device.str());
  return t;
}
int32_t kind(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return MOE_BF16;
  if (t.scalar_type() == at::kFloat) return MOE_F32;
  std::ostringstream o;
  o << name << ": unsupported dtype " << t.scalar_type();
  refuse(o.str());
}
at::ScalarType scalar(int32_t k) { return k == MOE_BF16 ? at::kBFloat16 : at::kFloat; }
// A contiguous device tensor [T, H].
const Tensor& rows(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.dim() != 2) refuse(std::string(name) + " must be a device tensor [T, H]");
  need(t, name, t.sizes(), t.scalar_type(), t.device());
  return t;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}
int32_t integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return (int32_t)v;
}

void check(moe_status_t st, const char* where) {
  if (st == MOE_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", (int)st, where);
  Py_XDECREF(r);
  if (PyErr_Occurred()) throw PythonError{};
}
// f(stream) with the device current and its current stream.
template <class F>
void launch(c10::Device device, const char* where, F f) {
  const c10::DeviceGuard guard(device);
  PyObject* i = PyLong_FromLong(device.index());
  PyObject* s = PyObject_CallOneArg(g_stream, i);
  Py_XDECREF(i);
  if (!s) throw PythonError{};
  void* stream = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!stream && PyErr_Occurred()) throw PythonError{};
  moe_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f((hipStream_t)stream);
  Py_END_ALLOW_THREADS
  check(st, where);
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap(const std::optional<Tensor>& t) {
  if (t) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}
// Steals each object.
PyObject* tuple(std::initializer_list<PyObject*> v) {
  PyObject* t = PyTuple_New((Py_ssize_t)v.size());
  Py_ssize_t i = 0;
  for (PyObject* o : v) PyTuple_SET_ITEM(t, i++, o);
  return t;
}

// Runs a function body with its exceptions turned into Python's.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) return PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
  try {
    return f();
  } catch (const PythonError&) {
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ------------------------------------------------------------ norms
moe_norm_desc_t norm_desc(const Tensor& x, int32_t gate, double scale, double eps) {
  return {x.size(0), x.size(1), kind(x, "x"), gate, (float)scale, (float)eps};
}

// norm_fwd(x, w, eps, out) -> y
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    const Tensor& x = rows(a[0], "x");
    const moe_norm_desc_t d = norm_desc(x, MOE_GATE_NONE, 1.0, number(a[2]));
    const Tensor& w = tensor(a[1], "w");
    need(w, "w", {x.size(1)}, x.scalar_type(), x.device());
    const Tensor y = output(a[3], "out", x.sizes(), x.scalar_type(), x.device());
    launch(x.device(), "moe_norm_fwd", [&](hipStream_t s) { return moe_norm_fwd(&d, data(x), data(w), data(y), s); });
    return wrap(y);
  });
}

// norm_bwd(x, w, d_y, d_add, eps, ws, d_x, d_w) -> (d_x, d_w, ws)
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Tensor& x = rows(a[0], "x");
    const auto dt = x.scalar_type();
    const auto dev = x.device();
    const moe_norm_desc_t d = norm_desc(x, MOE_GATE_NONE, 1.0, number(a[4]));
    const Shape H = {x.size(1)};
    const Tensor &w = tensor(a[1], "w"), &dy = tensor(a[2], "d_y");
    need(w, "w", H, dt, dev);
    need(dy, "d_y", x.sizes(), dt, dev);
    const void* add = input(a[3], "d_add", x.sizes(), dt, dev);
    size_t bytes = 0;
    check(moe_norm_workspace_size(&d, &bytes), "moe_norm_workspace_size");
    const Tensor ws = workspace(a[5], bytes, dev), dx = output(a[6], "d_x", x.sizes(), dt, dev),
                 dw = output(a[7], "d_w", H, at::kFloat, dev);
    launch(dev, "moe_norm_bwd", [&](hipStream_t s) {
      return moe_norm_bwd(&d, data(x), data(w), data(dy), add, data(dx), (float*)data(dw), data(ws), ws.nbytes(), s);
    });
    return tuple({wrap(dx), wrap(dw), wrap(ws)});
  });
}

int32_t gate_kind(PyObject* o, const Tensor& x) {
  if (o == Py_None) return MOE_GATE_NONE;
  const Tensor& g = tensor(o, "gate");
  const int64_t T = x.size(0), H = x.size(1);
  const Shape forms[] = {{T, 1}, {H}, {T, H}};
  for (int i = 0; i < 3; ++i)
    if (g.sizes() == at::IntArrayRef(forms[i])) {
      need(g, "gate", forms[i], x.scalar_type(), x.device());
      return MOE_GATE_ROW + i;
    }
  refuse("gate must be [T, 1], [H] or [T, H], got " + list(g.sizes()));
}

// residual_fwd(x, h, w_post, gate, scale, w_next, eps, x_new, y) -> (x_new, y)
PyObject* residual_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const Tensor& x = rows(a[0], "x");
    const auto dt = x.scalar_type();
    const auto dev = x.device();
    const moe_norm_desc_t d = norm_desc(x, gate_kind(a[3], x), number(a[4]), number(a[6]));
    const Shape H = {x.size(1)};
    const Tensor& h = tensor(a[1], "h");
    need(h, "h", x.sizes(), dt, dev);
    const void *post = input(a[2], "w_post", H, dt, dev), *next = input(a[5], "w_next", H, dt, dev);
    const void* gate = a[3] == Py_None ? nullptr : tensor(a[3], "gate").data_ptr();
    const Tensor x_new = output(a[7], "x_new", x.sizes(), dt, dev);
    std::optional<Tensor> y;
    if (next) y = output(a[8], "y", x.sizes(), dt, dev);
    if (x.size(0))   // without rows there is nothing to do, and a gate of none has no address
      launch(dev, "moe_residual_fwd", [&](hipStream_t s) {
        return moe_residual_fwd(&d, data(x), data(h), post, gate, next, data(x_new), y ? data(*y) : nullptr, s);
      });
    return tuple({wrap(x_new), wrap(y)});
  });
}

// residual_bwd(x_new, h, d_x_new, d_y, w_post, gate, scale, w_next, eps, ws, d_x, d_h, d_gate, d_w_post, d_w_next)
//   -> (d_x, d_h, d_gate, d_w_post, d_w_next, ws)
PyObject* residual_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const Tensor& x = rows(a[0], "x_new");
    const auto dt = x.scalar_type();
    const auto dev = x.device();
    moe_norm_desc_t d = norm_desc(x, gate_kind(a[5], x), number(a[6]), number(a[8]));
    const Shape H = {x.size(1)};
    const Tensor& h = tensor(a[1], "h");
    need(h, "h", x.sizes(), dt, dev);
    if ((a[7] == Py_None) != (a[3] == Py_None)) refuse("d_y goes with w_next");
    const void *post = input(a[4], "w_post", H, dt, dev), *next = input(a[7], "w_next", H, dt, dev);
    const void *dnew = input(a[2], "d_x_new", x.sizes(), dt, dev), *dy = input(a[3], "d_y", x.sizes(), dt, dev);
    size_t bytes = 0;
    check(moe_norm_workspace_size(&d, &bytes), "moe_norm_workspace_size");
    const Tensor ws = workspace(a[9], bytes, dev), dx = output(a[10], "d_x", x.sizes(), dt, dev),
                 dh = output(a[11], "d_h", x.sizes(), dt, dev);
    std::optional<Tensor> dg, dpost, dnext;
    const void* gate = nullptr;
    if (d.gate_kind != MOE_GATE_NONE) {
      const Tensor& g = tensor(a[5], "gate");
      dg = output(a[12], "d_gate", g.sizes(), d.gate_kind == MOE_GATE_FULL ? dt : at::kFloat, dev);
      gate = g.data_ptr();
      if (!gate) d.gate_kind = MOE_GATE_NONE;   // no rows: nothing but zero sums to write
    }
    if (post) dpost = output(a[13], "d_w_post", H, at::kFloat, dev);
    if (next) dnext = output(a[14], "d_w_next", H, at::kFloat, dev);
    launch(dev, "moe_residual_bwd", [&](hipStream_t s) {
      return moe_residual_bwd(&d, data(x), data(h), post, gate, next, x.size(0) ? dnew : nullptr, x.size(0) ? dy : nullptr,
                              data(dx), data(dh), dg && gate ? data(*dg) : nullptr, dpost ? (float*)data(*dpost) : nullptr,
                              dnext ? (float*)data(*dnext) : nullptr, data(ws), ws.nbytes(), s);
    });
    return tuple({wrap(dx), wrap(dh), wrap(dg), wrap(dpost), wrap(dnext), wrap(ws)});
  });
}

// ------------------------------------------------------------ feed-forward block
// The descriptor of a call with x, w_gate_up, w_down, gate at a[0..3] and act, layout, limit, alpha at c[0..3].
struct Ffn {
  moe_desc_t d;
  size_t fwd, bwd, saved;
};
Ffn ffn(PyObject* const* a, PyObject* const* c, int32_t grad) {
  const Tensor& x = rows(a[0], "x");
  const Tensor &gu = tensor(a[1], "w_gate_up"), &dn = tensor(a[2], "w_down");
  const int32_t k = kind(x, "x");
  if (gu.dim() != 2 || gu.size(0) % 2) refuse("w_gate_up must be [2I, H]");
  const int64_t T = x.size(0), H = x.size(1), I = gu.size(0) / 2;
  need(gu, "w_gate_up", {2 * I, H}, x.scalar_type(), x.device());
  need(dn, "w_down", {H, I}, x.scalar_type(), x.device());
  input(a[3], "gate", {T}, at::kFloat, x.device());
  Ffn f;
  f.d = {T, H, I, 1, 1, k, integer(c[0]), integer(c[1]), (float)number(c[2]), (float)number(c[3]), grad < 0 ? k : grad};
  check(moe_ffn_workspace_size(&f.d, &f.fwd, &f.bwd, &f.saved), "moe_ffn_workspace_size");
  return f;
}
const float* gate_of(PyObject* o) { return o == Py_None ? nullptr : (const float*)data(THPVariable_Unpack(o)); }

// ffn_fwd(x, w_gate_up, w_down, gate, act, layout, limit, alpha, add, save, ws, out, saved) -> (out, saved, ws)
PyObject* ffn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const int save = PyObject_IsTrue(a[9]);
    if (save < 0) throw PythonError{};
    if (!save && a[12] != Py_None) refuse("saved is where save=True puts the gate and up values, without it nothing is saved");
    const Ffn f = ffn(a, a + 4, -1);
    const Tensor &x = THPVariable_Unpack(a[0]), &gu = THPVariable_Unpack(a[1]), &dn = THPVariable_Unpack(a[2]);
    const auto dev = x.device();
    const void* add = input(a[8], "add", x.sizes(), x.scalar_type(), dev);
    const Tensor ws = workspace(a[10], f.fwd, dev), out = output(a[11], "out", x.sizes(), x.scalar_type(), dev);
    std::optional<Tensor> saved;
    if (save) saved = workspace(a[12], f.saved, dev);
    launch(dev, "moe_ffn_fwd", [&](hipStream_t s) {
      return moe_ffn_fwd(&f.d, data(x), data(gu), data(dn), gate_of(a[3]), add, data(out), saved ? data(*saved) : nullptr,
                         saved ? saved->nbytes() : 0, data(ws), ws.nbytes(), s);
    });
    return tuple({wrap(out), wrap(saved), wrap(ws)});
  });
}

// ffn_bwd(x, w_gate_up, w_down, gate, act, layout, limit, alpha, d_out, saved, grad_dtype or -1, ws, d_x, d_gate, d_gu, d_dn)
//   -> (d_x, d_gate, d_gu, d_dn, ws)
PyObject* ffn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    const Ffn f = ffn(a, a + 4, integer(a[10]));
    const Tensor &x = THPVariable_Unpack(a[0]), &gu = THPVariable_Unpack(a[1]), &dn = THPVariable_Unpack(a[2]);
    const auto dev = x.device();
    const Tensor& dout = tensor(a[8], "d_out");
    need(dout, "d_out", x.sizes(), x.scalar_type(), dev);
    std::optional<Tensor> saved;
    if (a[9] != Py_None) saved = workspace(a[9], f.saved, dev);
    const auto gt = scalar(f.d.grad_dtype);
    const Tensor ws = workspace(a[11], f.bwd, dev), dx = output(a[12], "d_x", x.sizes(), x.scalar_type(), dev),
                 dgu = output(a[14], "d_w_gate_up", gu.sizes(), gt, dev), ddn = output(a[15], "d_w_down", dn.sizes(), gt, dev);
    std::optional<Tensor> dg;
    if (a[3] != Py_None) dg = output(a[13], "d_gate", {x.size(0)}, at::kFloat, dev);
    launch(dev, "moe_ffn_bwd", [&](hipStream_t s) {
      return moe_ffn_bwd(&f.d, data(x), data(gu), data(dn), gate_of(a[3]), data(dout), saved ? data(*saved) : nullptr,
                         saved ? saved->nbytes() : 0, data(dx), dg ? (float*)data(*dg) : nullptr, data(dgu), data(ddn), data(ws),
                         ws.nbytes(), s);
    });
    return tuple({wrap(dx), wrap(dg), wrap(dgu), wrap(ddn), wrap(ws)});
  });
}

// init(check, raw_stream)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject* {
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    Py_XSETREF(g_check, a[0]);
    Py_XSETREF(g_stream, a[1]);
    Py_RETURN_NONE;
  });
}

#define METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(init),         METHOD(norm_fwd), METHOD(norm_bwd), METHOD(residual_fwd),
                         METHOD(residual_bwd), METHOD(ffn_fwd),  METHOD(ffn_bwd),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
