// What the package's compiled bindings share: checks of torch arguments, results and
// workspaces, the current stream, and errors on their way to Python.
//
// Only host code: the library's C ABI and torch's C++ interface.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>

#include <cstring>
#include <string>

#include "../../include/fp4gemm.h"

namespace {

// A refused argument, on its way to the entry point that turns it into a Python error.
struct Refused {
  PyObject* type;
  std::string what;
};
// A Python error that is already set.
struct Raised {};

[[noreturn]] void type_error(const std::string& what) { throw Refused{PyExc_TypeError, what}; }
[[noreturn]] void value_error(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

// Forward-mode derivatives: a tensor that carries one does not say so in requires_grad, and read by its
// pointer it would lose it without a word.  The error is torch's own for a function that has none.
[[maybe_unused]] void no_tangents(const char* fn, std::initializer_list<const at::Tensor*> ts) {
  if (!c10::AutogradState::get_tls_state().get_fw_grad_mode()) return;
  for (const at::Tensor* t : ts)
    if (t->defined() && t->_fw_grad(0).defined())
      throw Refused{PyExc_NotImplementedError, std::string(fn) + " has no forward-mode derivative"};
}

std::string dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kChar: return "torch.int8";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    default: return std::string("torch.") + c10::toString(t);
  }
}
std::string shape_name(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

// A contiguous matrix on a GPU, of one of two types.
const at::Tensor& matrix(PyObject* o, const char* name, at::ScalarType a, at::ScalarType b) {
  const at::Tensor& t = tensor(o, name);
  const at::ScalarType got = t.scalar_type();
  if (got != a && got != b)
    type_error(std::string(name) + " must have dtype " + dtype_name(a) + (a == b ? "" : " or " + dtype_name(b)) +
               ", got " + dtype_name(got));
  if (!t.is_cuda()) value_error("tensors must be on a GPU, got " + t.device().str());
  if (t.dim() != 2) value_error(std::string(name) + " must be 2-D");
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t;
}

// A contiguous tensor of this type and shape on this device.
const at::Tensor& need(PyObject* o, const char* name, at::ScalarType dtype, at::IntArrayRef shape, at::Device device) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != dtype)
    type_error(std::string(name) + " must have dtype " + dtype_name(dtype) + ", got " + dtype_name(t.scalar_type()));
  if (t.sizes() != shape)
    value_error(std::string(name) + " must have shape " + shape_name(shape) + ", got " + shape_name(t.sizes()));
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  if (t.device() != device)
    value_error(std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
  return t;
}

// The interpreter lock is not held while memory is taken or kernels are launched.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, at::Device device) {
  const Unlocked u;
  return at::Tensor(at::detail::empty_cuda(shape, dtype, device, std::nullopt));   // what at::empty ends in
}
at::Tensor result(PyObject* out, const char* name, at::ScalarType dtype, at::IntArrayRef shape, at::Device device) {
  return out == Py_None ? empty(shape, dtype, device) : need(out, name, dtype, shape, device);
}

void* ptr(const at::Tensor& t) { return t.data_ptr(); }
float* floats(const at::Tensor& t) { return static_cast<float*>(t.data_ptr()); }

// The current stream of a GPU, as torch.cuda.current_stream(device).cuda_stream.
void* stream_of(at::Device device) {
  static PyObject* const query = [] {
    PyObject* m = PyImport_ImportModule("torch._C");
    PyObject* f = m ? PyObject_GetAttrString(m, "_cuda_getCurrentRawStream") : nullptr;
    Py_XDECREF(m);
    return f;
  }();
  if (!query) throw Raised{};
  PyObject* index = PyLong_FromLong(device.index());
  if (!index) throw Raised{};
  PyObject* r = PyObject_CallFunctionObjArgs(query, index, nullptr);
  Py_DECREF(index);
  if (!r) throw Raised{};
  void* s = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  if (PyErr_Occurred()) throw Raised{};
  return s;
}

// The package's error for a status (its _raise_on).
void check_status(const char* fn, fp4g_status st) {
  if (st == FP4G_OK) return;
  PyObject* m = PyImport_ImportModule("block_scaled_precision_e2m1_amd");
  PyObject* r = m ? PyObject_CallMethod(m, "_raise_on", "si", fn, (int)st) : nullptr;
  Py_XDECREF(m);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", fn, (int)st);
  throw Raised{};
}

template <class F>
void launch(const char* fn, at::Device device, F&& call) {
  void* const stream = stream_of(device);
  fp4g_status st;
  {
    const Unlocked u;
    st = call(stream);
  }
  check_status(fn, st);
}

// The caller's workspace (uint8, any length) or a new one of `bytes`.
struct Space {
  at::Tensor t;
  void* p = nullptr;
  size_t bytes = 0;
};
template <class Size>
Space space(PyObject* given, at::Device device, Size&& size) {
  Space s;
  if (given == Py_None) {
    const int64_t bytes = (int64_t)size();
    if (bytes == 0) return s;
    s.t = empty({bytes}, at::kByte, device);
  } else {
    s.t = need(given, "workspace", at::kByte, {tensor(given, "workspace").numel()}, device);
  }
  s.bytes = (size_t)s.t.numel();
  s.p = s.bytes ? ptr(s.t) : nullptr;
  return s;
}

// The result of a product: `out`, or a new tensor of out_dtype.
[[maybe_unused]] at::Tensor output(PyObject* out, PyObject* out_dtype, int64_t M, int64_t N, at::Device device, int* d_type) {
  at::ScalarType t;
  if (out != Py_None) t = tensor(out, "out").scalar_type();
  else if (THPDtype_Check(out_dtype)) t = reinterpret_cast<THPDtype*>(out_dtype)->scalar_type;
  else type_error("out_dtype must be a torch.dtype");
  if (t != at::kBFloat16 && t != at::kFloat) type_error("out must be float32 or bfloat16");
  *d_type = t == at::kBFloat16 ? FP4G_OUT_BF16 : FP4G_OUT_F32;
  return result(out, "out", t, {M, N}, device);
}

[[maybe_unused]] void multiple_of(int64_t K, int64_t step) {
  if (K % step) value_error("K=" + std::to_string(K) + " must be a multiple of " + std::to_string(step));
}

// Runs f with errors turned into Python's; f returns a new reference.
template <class F>
PyObject* entry(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    at::AutoDispatchBelowADInplaceOrView below;   // results carry no gradient
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const Raised&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = r ? THPVariable_Wrap(t) : nullptr;
    if (!o) {
      Py_XDECREF(r);
      throw Raised{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

#define FASTCALL(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}

}  // namespace
