// What the calls of the compiled binding share: checks of tensors, allocation of
// results and workspaces, the current stream of the tensors' device, errors and
// the method table's entries.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <utility>

#include "../../include/nf4.h"

PyMethodDef* nf4_expert_methods();       // nf4_torch_experts.cpp

namespace {

using at::Tensor;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused(s.str());
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
  return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }

long long integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, " must be an integer");
  }
  return v;
}
bool truth(PyObject* o, const char* name) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) {
    PyErr_Clear();
    refuse(name, " must be true or false");
  }
  return t == 1;
}

// No call has a forward derivative: a tangent would be lost without a word.
using Named = std::initializer_list<std::pair<const char*, PyObject*>>;
void no_tangents(const Named& inputs) {
  for (const auto& [name, o] : inputs)
    if (given(o) && tensor(o, name)._fw_grad(0).defined())
      refuse(name, " carries a forward-mode tangent, and this call has no forward derivative");
}

// Rotation and cache have no gradient either: an input that wants one is refused
// while gradients are recorded, not returned without its history.
void no_derivatives(const Named& inputs) {
  no_tangents(inputs);
  if (!at::GradMode::is_enabled()) return;
  for (const auto& [name, o] : inputs)
    if (given(o) && tensor(o, name).requires_grad())
      refuse(name, " requires a gradient, which this call does not carry: detach it, or call under torch.no_grad()");
}

void need(const Tensor& t, const char* name, at::ScalarType dtype, int64_t numel, const c10::Device* device) {
  if (!t.is_cuda()) refuse(name, " must be a device tensor");
  if (!t.is_contiguous()) refuse(name, " must be contiguous");
  if (t.scalar_type() != dtype) refuse(name, " must be ", dtype, ", got ", t.scalar_type());
  if (numel >= 0 && t.numel() != numel) refuse(name, " must have ", numel, " elements, got ", t.numel());
  if (device && t.device() != *device) refuse(name, " is on ", t.device(), ", expected ", *device);
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const c10::Device& dev) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(dev));
}
Tensor new_workspace(size_t bytes, const c10::Device& dev) {
  if (bytes == SIZE_MAX) bytes = 0;                            // the call itself says why
  return bytes ? fresh({static_cast<int64_t>(bytes)}, at::kByte, dev) : Tensor();
}
Tensor given_workspace(PyObject* o, const c10::Device& dev) {
  const Tensor& t = tensor(o, "ws");
  if (!t.is_cuda()) refuse("ws must be a device tensor");
  if (!t.is_contiguous()) refuse("ws must be contiguous");
  if (t.device() != dev) refuse("ws is on ", t.device(), ", expected ", dev);
  return t;
}
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The tensors' device is made current, its current stream takes the work.
struct On {
  c10::DeviceGuard guard;
  void* stream;
  explicit On(const c10::Device& dev) : guard(dev), stream(c10::hip::getCurrentHIPStream(dev.index()).stream()) {}
};

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <typename... T>
PyObject* several(const T&... t) {
  PyObject* out = PyTuple_New(sizeof...(t));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* x : {&t...}) {
    PyObject* w = wrap(*x);
    if (!w) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, w);
  }
  return out;
}

// Raises a failed C call as the package does (NF4Error with its status), from
// autograd's thread too.
void ok(int status, const char* name) {
  if (!status) return;
  const PyGILState_STATE gil = PyGILState_Ensure();
  PyObject* lib = PyImport_ImportModule("nf4_bit_weight_amd._lib");
  PyObject* none = lib ? PyObject_CallMethod(lib, "check", "si", name, status) : nullptr;
  Py_XDECREF(none);
  Py_XDECREF(lib);
  python_error e;
  e.persist();
  PyGILState_Release(gil);
  throw e;
}

// While a graph is being captured, the gradients of leaves go through their
// accumulators.  One that a living eager graph made belongs to the eager stream,
// and autograd would make that stream wait inside the capture, which ends it,
// and the process with it.  So such a leaf is refused here, in the forward call.
void check_capture(std::initializer_list<std::pair<const char*, const Tensor*>> inputs, const c10::Device& dev) {
  const auto now = c10::hip::getCurrentHIPStream(dev.index());
  hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(now.stream(), &status) != hipSuccess || status != hipStreamCaptureStatusActive) return;
  for (const auto& [name, t] : inputs) {
    if (!t->requires_grad() || !t->is_leaf()) continue;
    const auto acc = torch::autograd::impl::try_get_grad_accumulator(*t);
    const auto stream = acc ? acc->stream() : std::nullopt;
    if (stream && stream->id() != now.id())
      refuse(name, " is captured while an eager graph of the same leaf lives: drop that graph first, or pass a detached leaf");
  }
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  HANDLE_TH_ERRORS                                             // torch's own: out of memory, no device
  try {
    return F(args);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>)), METH_FASTCALL, nullptr};
}

}  // namespace
