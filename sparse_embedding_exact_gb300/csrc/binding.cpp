// The dense operators' calls on torch tensors: checks of what the C ABI cannot
// see (devices, types, strides), outputs and scratch from torch's allocator on
// the current stream, one call of the C ABI.  Native, because a short call is
// mostly host time: the norm of four rows takes 3 us on the device, and its
// marshalling in Python took 18 us.
//
// Every function returns its tensors, or the call's status where that is not
// SS_OK.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <string>

#include "sparsecos.h"

namespace {

using at::Tensor;

// A Python error to raise.
struct Refused {
  PyObject *type;
  std::string what;
};

// One that Python has raised already.
struct Raised {};

float number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)v;
}

int32_t code_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return SS_VALUES_F32;
    case at::kBFloat16: return SS_VALUES_BF16;
    case at::kHalf: return SS_VALUES_F16;
    case at::kFloat8_e4m3fn: return SS_VALUES_F8;
    default: return -1;
  }
}
at::ScalarType type_of(int64_t code) {
  switch (code) {
    case SS_VALUES_F32: return at::kFloat;
    case SS_VALUES_BF16: return at::kBFloat16;
    case SS_VALUES_F16: return at::kHalf;
    default: throw Refused{PyExc_TypeError, "not a type of an output"};
  }
}

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

// What every call starts with: the handle, its device and the stream.
struct Call {
  ss_handle *h;
  int64_t device;
  Call(PyObject *handle, PyObject *dev)
      : h(static_cast<ss_handle *>(PyLong_AsVoidPtr(handle))), device(PyLong_AsLongLong(dev)) {}

  void here(const Tensor &t, const char *name) const {
    if (t.is_cuda() && t.get_device() == device) return;
    throw Refused{PyExc_ValueError,
                  std::string(name) + " is on " + t.device().str() + ", the handle's device is cuda:" + std::to_string(device)};
  }
  // A matrix with contiguous rows, or a vector as one row.
  ss_dense matrix(const Tensor &t, const char *name) const {
    here(t, name);
    const int32_t code = code_of(t.scalar_type());
    if (code < 0) throw Refused{PyExc_TypeError, std::string(name) + " has type " + at::toString(t.scalar_type())};
    const int64_t dims = t.dim();
    if (dims != 1 && dims != 2)
      throw Refused{PyExc_ValueError, std::string(name) + " must be a matrix or a vector, got " + std::to_string(dims) + " dimensions"};
    const int64_t rows = dims == 2 ? t.size(0) : 1, cols = t.size(dims - 1);
    if (cols > 1 && t.stride(dims - 1) != 1)
      throw Refused{PyExc_ValueError, std::string(name) + ": the values of a row must be contiguous"};
    return {t.data_ptr(), rows, cols, rows > 1 ? t.stride(0) : cols, code};
  }
  // The address of a contiguous array of the given shape and type, or null.
  void *array(PyObject *o, const char *name, int64_t rows, int64_t cols, at::ScalarType type) const {
    if (o == Py_None) return nullptr;
    const Tensor &t = tensor(o, name);
    here(t, name);
    if (t.scalar_type() != type)
      throw Refused{PyExc_TypeError, std::string(name) + " has type " + at::toString(t.scalar_type()) + ", expected " + at::toString(type)};
    const bool shape = cols < 0 ? t.dim() == 1 && t.size(0) == rows : t.dim() == 2 && t.size(0) == rows && t.size(1) == cols;
    if (!shape || !t.is_contiguous())
      throw Refused{PyExc_ValueError, std::string(name) + ": expected a contiguous array of shape (" + std::to_string(rows) +
                                          (cols < 0 ? ",)" : ", " + std::to_string(cols) + ")")};
    return t.data_ptr();
  }
  float *floats(PyObject *o, const char *name, int64_t rows, int64_t cols = -1) const {
    return static_cast<float *>(array(o, name, rows, cols, at::kFloat));
  }
  Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::empty(size, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device));
  }
  Tensor scratch(int64_t bytes) const { return bytes > 0 ? empty({bytes}, at::kByte) : Tensor(); }
  void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }
};
void *at_of(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
int64_t size_of(const Tensor &t) { return t.defined() ? t.numel() : 0; }

ss_dense dense(const Tensor &t, int64_t rows, int64_t cols, int32_t code) { return {t.data_ptr(), rows, cols, cols, code}; }

PyObject *pack(std::initializer_list<Tensor> out) {
  PyObject *r = PyTuple_New((Py_ssize_t)out.size());
  Py_ssize_t i = 0;
  for (const Tensor &t : out) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// Runs a call's body with its arguments counted and its errors turned into
// Python's.
template <int kArgs, typename Body>
PyObject *guarded(PyObject *const *a, Py_ssize_t n, Body body) {
  HANDLE_TH_ERRORS
  try {
    if (n != kArgs) throw Refused{PyExc_TypeError, "expected " + std::to_string(kArgs) + " arguments"};
    return body(Call(a[0], a[1]));
  } catch (const Refused &r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  } catch (const Raised &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
PyObject *status(ss_status st) { return PyLong_FromLong(st); }

// (handle, device, x, weight, residual or None, eps, 8 bits) -> y, total, factor
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<7>(a, n, [&](Call c) -> PyObject * {
    const Tensor &x = tensor(a[2], "x"), &weight = tensor(a[3], "weight");
    const bool f8 = PyObject_IsTrue(a[6]) == 1, sum = a[4] != Py_None;
    const ss_dense mx = c.matrix(x, "x"), mw = c.matrix(weight, "weight");
    ss_dense mr = {}, mt = {};
    const Tensor y = c.empty(x.sizes(), f8 ? at::kFloat8_e4m3fn : x.scalar_type()), factor = c.empty({mx.n_rows}, at::kFloat);
    Tensor total = x;
    if (sum) {
      mr = c.matrix(tensor(a[4], "residual"), "residual");
      total = c.empty(x.sizes(), x.scalar_type());
      mt = dense(total, mx.n_rows, mx.n_cols, mx.type);
    }
    const ss_dense my = dense(y, mx.n_rows, mx.n_cols, f8 ? SS_VALUES_F8 : mx.type);
    float *f = factor.data_ptr<float>();
    const ss_status st = ss_rms_norm(c.h, &mx, sum ? &mr : nullptr, &mw, number(a[5]), sum ? &mt : nullptr,
                                     &my, f8 ? f : nullptr, f8 ? nullptr : f, c.stream());
    return st ? status(st) : pack({y, total, factor});
  });
}

// (handle, device, grad_y, total, weight, rstd, grad_total or None) -> grad_x, grad_weight
PyObject *norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<7>(a, n, [&](Call c) -> PyObject * {
    const Tensor &total = tensor(a[3], "total"), &weight = tensor(a[4], "weight");
    const ss_dense mg = c.matrix(tensor(a[2], "grad_y"), "grad_y"), mt = c.matrix(total, "total"), mw = c.matrix(weight, "weight");
    const float *rstd = c.floats(a[5], "rstd", mt.n_rows);
    ss_dense mp = {};
    if (a[6] != Py_None) mp = c.matrix(tensor(a[6], "grad_total"), "grad_total");
    const Tensor gx = c.empty(total.sizes(), total.scalar_type()), gw = c.empty(weight.sizes(), weight.scalar_type());
    const Tensor room = c.scratch(ss_rms_norm_backward_scratch(c.h, mt.n_rows, mt.n_cols));
    const ss_dense mx = dense(gx, mt.n_rows, mt.n_cols, mt.type), mv = dense(gw, mw.n_rows, mw.n_cols, mw.type);
    const ss_status st = ss_rms_norm_backward(c.h, &mg, &mt, &mw, rstd, a[6] != Py_None ? &mp : nullptr, &mx, &mv, at_of(room),
                                              size_of(room), c.stream());
    return st ? status(st) : pack({gx, gw});
  });
}

// (handle, device, x, w, bias, activation, residual, x_scale, w_scale, type of y or -1, keep pre) -> y, or y and pre
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<11>(a, n, [&](Call c) -> PyObject * {
    const ss_dense mx = c.matrix(tensor(a[2], "x"), "x"), mw = c.matrix(tensor(a[3], "w"), "w");
    const int64_t M = mx.n_rows, N = mw.n_rows;
    int64_t code = PyLong_AsLongLong(a[9]);
    if (code < 0) code = mx.type == SS_VALUES_F8 ? SS_VALUES_BF16 : mx.type;
    const at::ScalarType out = type_of(code);
    const float *bias = c.floats(a[4], "bias", N), *sx = c.floats(a[7], "x_scale", M), *sw = c.floats(a[8], "w_scale", N);
    const bool sum = a[6] != Py_None, keep = PyObject_IsTrue(a[10]) == 1;
    ss_dense mr = {}, mp = {};
    if (sum) mr = c.matrix(tensor(a[6], "residual"), "residual");
    const Tensor y = c.empty({M, N}, out);
    Tensor pre;
    if (keep) {
      pre = c.empty({M, N}, out);
      mp = dense(pre, M, N, (int32_t)code);
    }
    const ss_dense my = dense(y, M, N, (int32_t)code);
    const Tensor room = c.scratch(ss_linear_scratch(c.h, &mx, &mw));
    const ss_status st = ss_linear(c.h, &mx, sx, &mw, sw, bias, (int32_t)PyLong_AsLong(a[5]), sum ? &mr : nullptr,
                                   keep ? &mp : nullptr, &my, at_of(room), size_of(room), c.stream());
    if (st) return status(st);
    return keep ? pack({y, pre}) : THPVariable_Wrap(y);
  });
}

// (handle, device, grad_y, x, w, pre or None, activation, type of the gradients or -1) -> grad_x, grad_w, grad_bias
PyObject *linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<8>(a, n, [&](Call c) -> PyObject * {
    const Tensor &x = tensor(a[3], "x"), &w = tensor(a[4], "w");
    const ss_dense mg = c.matrix(tensor(a[2], "grad_y"), "grad_y"), mx = c.matrix(x, "x"), mw = c.matrix(w, "w");
    ss_dense mp = {};
    if (a[5] != Py_None) mp = c.matrix(tensor(a[5], "pre"), "pre");
    const int32_t act = (int32_t)PyLong_AsLong(a[6]);
    int64_t code = PyLong_AsLongLong(a[7]);
    if (code < 0) code = mx.type;
    const at::ScalarType type = type_of(code);
    const Tensor gx = c.empty(x.sizes(), type), gw = c.empty(w.sizes(), type), gb = c.empty({mw.n_rows}, at::kFloat);
    const Tensor room = c.scratch(ss_linear_backward_scratch(c.h, &mg, &mx, &mw, act));
    const ss_dense mgx = dense(gx, mx.n_rows, mx.n_cols, (int32_t)code), mgw = dense(gw, mw.n_rows, mw.n_cols, (int32_t)code);
    const ss_status st = ss_linear_backward(c.h, &mg, &mx, &mw, a[5] != Py_None ? &mp : nullptr, act, &mgx, &mgw,
                                            gb.data_ptr<float>(), at_of(room), size_of(room), c.stream());
    return st ? status(st) : pack({gx, gw, gb});
  });
}

// A distillation's common arguments: logits, scores, items, weight or None, T, U.
struct Lists {
  ss_dense logits;
  const float *scores, *weight;
  const int64_t *items;
  int32_t k;
  float t, u;
  Lists(const Call &c, PyObject *const *a) {
    logits = c.matrix(tensor(a[0], "logits"), "logits");
    const Tensor &s = tensor(a[1], "scores");
    if (s.dim() != 2) throw Refused{PyExc_ValueError, "scores must be (rows, k)"};
    const int64_t wide = s.size(1);
    scores = c.floats(a[1], "scores", logits.n_rows, wide);
    items = static_cast<const int64_t *>(c.array(a[2], "items", logits.n_rows, wide, at::kLong));
    weight = c.floats(a[3], "weight", logits.n_rows);
    k = (int32_t)std::min<int64_t>(wide, INT32_MAX);
    t = number(a[4]);
    u = number(a[5]);
  }
};

// (handle, device, lists) -> loss, stats
PyObject *distill(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<8>(a, n, [&](Call c) -> PyObject * {
    const Lists l(c, a + 2);
    const Tensor loss = c.empty({l.logits.n_rows}, at::kFloat), stats = c.empty({l.logits.n_rows, 2}, at::kFloat);
    const ss_status st = ss_distill(c.h, &l.logits, l.scores, l.items, l.k, l.t, l.u, l.weight, loss.data_ptr<float>(),
                                    stats.data_ptr<float>(), c.stream());
    return st ? status(st) : pack({loss, stats});
  });
}

// (handle, device, lists, grad_loss or None, stats) -> grad_logits
PyObject *distill_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<10>(a, n, [&](Call c) -> PyObject * {
    const Lists l(c, a + 2);
    const Tensor &z = tensor(a[2], "logits");
    const float *gl = c.floats(a[8], "grad_loss", l.logits.n_rows), *stats = c.floats(a[9], "stats", l.logits.n_rows, 2);
    const Tensor g = c.empty(z.sizes(), z.scalar_type());
    const ss_dense mg = dense(g, l.logits.n_rows, l.logits.n_cols, l.logits.type);
    const ss_status st = ss_distill_backward(c.h, gl, &l.logits, l.scores, l.items, l.k, l.t, l.u, l.weight, stats, &mg, c.stream());
    return st ? status(st) : THPVariable_Wrap(g);
  });
}

// (handle, device, lists, grad_loss or None, in place) -> loss, grad_logits
PyObject *distill_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded<10>(a, n, [&](Call c) -> PyObject * {
    const Lists l(c, a + 2);
    const Tensor &z = tensor(a[2], "logits");
    const float *gl = c.floats(a[8], "grad_loss", l.logits.n_rows);
    const bool in_place = PyObject_IsTrue(a[9]) == 1;
    const Tensor loss = c.empty({l.logits.n_rows}, at::kFloat), g = in_place ? z : c.empty(z.sizes(), z.scalar_type());
    const ss_dense mg = in_place ? l.logits : dense(g, l.logits.n_rows, l.logits.n_cols, l.logits.type);
    const ss_status st = ss_distill_step(c.h, gl, &l.logits, l.scores, l.items, l.k, l.t, l.u, l.weight, loss.data_ptr<float>(),
                                         &mg, c.stream());
    // torch's record that the logits changed (tensors of its inference mode have none)
    if (!st && in_place && !z.is_inference()) z.unsafeGetTensorImpl()->bump_version();
    return st ? status(st) : pack({loss, g});
  });
}

#define SS_CALL(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SS_CALL(norm),    SS_CALL(norm_backward),    SS_CALL(linear),       SS_CALL(linear_backward),
                         SS_CALL(distill), SS_CALL(distill_backward), SS_CALL(distill_step), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__dense_binding(void) { return PyModule_Create(&module); }
