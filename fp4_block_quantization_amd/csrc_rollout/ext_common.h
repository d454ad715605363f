// ext_common.h -- what the native halves of the Python binding share: checks
// of tensors, the stream and device of a call, errors, and entry points that
// let no exception pass.  Each half is one translation unit with its own copy.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <stdexcept>
#include <string>

#include "fp4q.h"

namespace {

PyObject* error_type = nullptr;   // Fp4qError
PyObject* check_status = nullptr; // raises for a status other than success
PyObject* raw_stream = nullptr;   // device index -> the current stream's handle

// A Python error is set (Raised), or is to be set (Refused).
struct Raised {};
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

std::string text_of(at::IntArrayRef sizes) {
  std::string s = "[";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
    refuse(std::string(name) + " must be a GPU tensor");
  return THPVariable_Unpack(o);
}

const at::Tensor& typed(PyObject* o, const char* name, at::ScalarType type) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    refuse(std::string(name) + " must be " + at::toString(type) + ", got " +
           at::toString(t.scalar_type()));
  return t;
}

const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType type) {
  const at::Tensor& t = typed(o, name, type);
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t;
}

const at::Tensor& sized(PyObject* o, const char* name, at::ScalarType type, int64_t numel) {
  const at::Tensor& t = dense(o, name, type);
  if (t.numel() != numel)
    refuse(std::string(name) + " must hold " + std::to_string(numel) + " elements, got " +
           std::to_string(t.numel()));
  return t;
}

const at::Tensor& shaped(PyObject* o, const char* name, at::ScalarType type,
                         at::IntArrayRef sizes) {
  const at::Tensor& t = dense(o, name, type);
  if (t.sizes() != sizes)
    refuse(std::string(name) + " must be " + text_of(sizes) + ", got " + text_of(t.sizes()));
  return t;
}

// There is no backward pass: a result without history is no answer to an input that asks for one.
void no_gradient(const at::Tensor& t, const char* name) {
  if (t.requires_grad() && at::GradMode::is_enabled())
    refuse(std::string(name) + " requires a gradient, which this call does not have: detach it, "
                               "or call under torch.no_grad()");
}

// The device that every tensor of a call is on.  It is the current one while this lives: the
// default stream's handle is the same on every device.
struct Device {
  c10::Device device;
  c10::DeviceGuard guard;
  explicit Device(const at::Tensor& t) : device(t.device()), guard(t.device()) {}
  void same(const at::Tensor& t) const {
    if (t.device() != device)
      refuse("all tensors must be on " + device.str() + ", got one on " + t.device().str());
  }
  void* stream() const {
    PyObject* index = PyLong_FromLong(device.index());
    PyObject* r = index ? PyObject_CallOneArg(raw_stream, index) : nullptr;
    Py_XDECREF(index);
    if (!r) throw Raised();
    void* handle = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    if (PyErr_Occurred()) throw Raised();
    return handle;
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(device));
  }
};

// Outputs of a call, each in memory of its own, which costs the host a microsecond apiece: in one
// storage, one that is resized in place, or by torch as an out=, grows over the next without a word.
template <size_t N>
void allocate(const Device& device, const at::IntArrayRef (&shapes)[N],
              const at::ScalarType (&types)[N], at::Tensor* out) {
  for (size_t i = 0; i < N; ++i) out[i] = device.empty(shapes[i], types[i]);
}

struct Workspace {
  at::Tensor held;
  void* data = nullptr;
  int64_t bytes = 0;
  Workspace(PyObject* given, int64_t need, const Device& d) {
    if (given != Py_None) {
      const at::Tensor& t = dense(given, "workspace", at::kByte);
      if (t.numel() < need)
        refuse("workspace must hold at least " + std::to_string(need) + " bytes, got " +
               std::to_string(t.numel()));
      d.same(t);
      data = t.data_ptr();
      bytes = t.numel();
    } else if (need > 0) {
      held = d.empty({need}, at::kByte);
      data = held.data_ptr();
      bytes = need;
    }
  }
};

void check(fp4q_status st, const char* name) {
  if (st == FP4Q_SUCCESS) return;
  PyObject* r = PyObject_CallFunction(check_status, "is", (int)st, name);
  Py_XDECREF(r);
  throw Raised();
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

// Elements from token to token of a BF16 [..., heads, dim] tensor whose
// leading dimensions step evenly and whose last two are dense.
int64_t token_stride(const at::Tensor& t, const char* name, int64_t heads, int64_t dim) {
  if (t.dim() < 3 || t.size(-2) != heads || t.size(-1) != dim)
    refuse(std::string(name) + " must be [..., " + std::to_string(heads) + ", " +
           std::to_string(dim) + "], got " + text_of(t.sizes()));
  if (t.is_contiguous()) return heads * dim;
  if ((dim > 1 && t.stride(-1) != 1) || (heads > 1 && t.stride(-2) != dim))
    refuse(std::string(name) + " must be dense over its last two dimensions");
  int64_t step = 0, tokens = 1;
  for (int64_t i = t.dim() - 3; i >= 0; --i) {
    if (t.size(i) > 1) {
      if (tokens == 1)
        step = t.stride(i);
      else if (t.stride(i) != step * tokens)
        refuse(std::string(name) + " must step evenly from token to token");
    }
    tokens *= t.size(i);
  }
  return tokens > 1 ? step : heads * dim;
}

// An entry point: the argument count, and no exception past it.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count) {
  if (count != ARGS) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  if (!raw_stream) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
  } catch (const Refused& e) {
    PyErr_SetString(error_type, e.what());
  } catch (const std::exception& e) {  // torch's own, such as running out of memory
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// The addresses of a library's calls, after an error type, a status check and a getter of raw
// streams: bind(..) of a native half.
template <size_t N>
bool bind_calls(PyObject* const* args, Py_ssize_t count, void* (&at)[N]) {
  if (count != (Py_ssize_t)N + 3) {
    PyErr_Format(PyExc_TypeError, "bind takes %d arguments", (int)N + 3);
    return false;
  }
  for (size_t i = 0; i < N; ++i) {
    at[i] = PyLong_AsVoidPtr(args[3 + i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return false;
    }
  }
  for (int i = 0; i < 3; ++i) Py_INCREF(args[i]);
  Py_XSETREF(error_type, args[0]);
  Py_XSETREF(check_status, args[1]);
  Py_XSETREF(raw_stream, args[2]);
  return true;
}

#define FP4Q_METHOD(name, f) {name, (PyCFunction)(void*)(f), METH_FASTCALL, nullptr}

}  // namespace
