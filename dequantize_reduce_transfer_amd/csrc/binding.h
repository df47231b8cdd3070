// binding.h -- what the CPython modules over the HIP libraries share: a call's
// arguments checked and unpacked, its outputs allocated, C++ exceptions turned
// into Python ones.  Each module is one source file that includes this.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "fp8q.h"

namespace {

// A Python exception that is to be raised.
struct Refusal {
  PyObject *type;
  std::string text;
};

[[noreturn]] void refuse_type(const std::string &text) { throw Refusal{PyExc_TypeError, text}; }
[[noreturn]] void refuse(const std::string &text) { throw Refusal{PyExc_ValueError, text}; }

std::string dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kByte: return "torch.uint8";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return c10::toString(t);
  }
}

std::string shape_name(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// The call's arguments, and the device that its first tensor is on.
class Call {
 public:
  Call(const char *what, PyObject *const *args, Py_ssize_t given, Py_ssize_t wanted)
      : what_(what), args_(args) {
    if (given != wanted)
      refuse_type(std::string(what) + ": " + std::to_string(wanted) + " arguments are wanted");
  }

  bool absent(int i) const { return args_[i] == Py_None; }

  long long integer(int i, const char *name) const {
    const long long v = PyLong_AsLongLong(args_[i]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse_type(std::string(name) + " must be an integer");
    }
    return v;
  }

  double number(int i, const char *name) const {
    const double v = PyFloat_AsDouble(args_[i]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse_type(std::string(name) + " must be a number");
    }
    return v;
  }

  bool truth(int i, const char *name) const {
    const int v = PyObject_IsTrue(args_[i]);
    if (v < 0) {
      PyErr_Clear();
      refuse_type(std::string(name) + " must be true or false");
    }
    return v > 0;
  }

  void *stream(int i) const { return reinterpret_cast<void *>((intptr_t)integer(i, "stream")); }

  PyObject *object(int i) const { return args_[i]; }

  // A tensor as the kernels need it: one of the dtypes, on a GPU (the one of
  // the call's other tensors), contiguous.
  const at::Tensor &tensor(int i, const char *name, std::initializer_list<at::ScalarType> dtypes) {
    return tensor(args_[i], name, dtypes, true);
  }

  // The same of an object; `contiguous` false: strides are the caller's matter.
  const at::Tensor &tensor(PyObject *o, const char *name, std::initializer_list<at::ScalarType> dtypes,
                           bool contiguous) {
    if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a torch.Tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    bool fits = dtypes.size() == 0;
    for (at::ScalarType d : dtypes) fits = fits || t.scalar_type() == d;
    if (!fits) {
      std::string want;
      for (at::ScalarType d : dtypes) want += (want.empty() ? "" : " or ") + dtype_name(d);
      refuse_type(std::string(name) + " must be " + want + ", got " + dtype_name(t.scalar_type()));
    }
    if (!t.is_cuda()) refuse(std::string(name) + " must be on a GPU");
    if (contiguous && !t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    if (!placed_) {
      device_ = t.device();
      placed_ = true;
    } else if (t.device() != device_) {
      refuse(std::string(what_) + ": all tensors must be on " + device_.str() + ", got one on " +
             t.device().str());
    }
    return t;
  }

  const at::Tensor &shaped(int i, const char *name, at::ScalarType dtype, at::IntArrayRef shape) {
    const at::Tensor &t = tensor(i, name, {dtype});
    if (t.sizes() != shape)
      refuse(std::string(name) + " must be of shape " + shape_name(shape) + ", got " + shape_name(t.sizes()));
    return t;
  }

  // The caller's output, or a new tensor.
  at::Tensor output(int i, const char *name, at::ScalarType dtype, at::IntArrayRef shape) {
    if (!absent(i)) return shaped(i, name, dtype, shape);
    return at::empty(shape, at::TensorOptions(device_).dtype(dtype));
  }

  // A workspace of at least `bytes` (undefined where none is needed or given).
  at::Tensor workspace(int i, size_t bytes) {
    if (!absent(i)) {
      const at::Tensor &t = tensor(i, "workspace", {at::kByte});
      if ((size_t)t.numel() < bytes) refuse("workspace must hold " + std::to_string(bytes) + " bytes");
      return t;
    }
    if (!bytes) return at::Tensor();
    return at::empty({(int64_t)bytes}, at::TensorOptions(device_).dtype(at::kByte));
  }

  c10::Device device() const { return device_; }

 private:
  const char *what_;
  PyObject *const *args_;
  c10::Device device_{c10::kCPU};
  bool placed_ = false;
};

void *ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
float *f32(const at::Tensor &t) { return static_cast<float *>(ptr(t)); }
int *i32(const at::Tensor &t) { return static_cast<int *>(ptr(t)); }

PyObject *result(fp8q_status status, std::initializer_list<at::Tensor> outputs) {
  PyObject *r = PyTuple_New(1 + (Py_ssize_t)outputs.size());
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong((long)status));
  Py_ssize_t i = 1;
  for (const at::Tensor &t : outputs) {
    PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// What torch raises where GPU memory runs out: a RuntimeError of its own, which
// programs catch by that name.
PyObject *out_of_memory_type() {
  PyObject *torch = PyImport_ImportModule("torch");
  PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
  Py_XDECREF(torch);
  if (type) return type;
  PyErr_Clear();
  return Py_NewRef(PyExc_RuntimeError);
}

// Turns a refusal, and any C++ exception (an allocation that failed), into a
// Python exception.
template <typename Body>
PyObject *guarded(Body &&body) {
  try {
    return body();
  } catch (const Refusal &r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const c10::OutOfMemoryError &e) {
    PyObject *type = out_of_memory_type();
    PyErr_SetString(type, e.what_without_backtrace());
    Py_DECREF(type);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

fp8q_format format_code(const Call &c, int i) {
  const long long f = c.integer(i, "fmt");
  if (f != FP8Q_E4M3 && f != FP8Q_E5M2) refuse("fmt must be E4M3 (0) or E5M2 (1)");
  return (fp8q_format)f;
}

// A method that takes its arguments as an array.
#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}

}  // namespace
