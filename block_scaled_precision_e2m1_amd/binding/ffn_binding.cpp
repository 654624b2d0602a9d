// The Python binding of the feed-forward operators (include/fp4g_ffn.h) over torch tensors.
//
// The kernels of a decode step take 2 to 10 us, as long as a binding written in Python takes
// to check its arguments and allocate its results (int8_quantize of one token: 9.9 us a
// call, of which the launch is 2.7).  So these operators are bound in C++: every function
// takes its arguments by position from the Python function of the same name in ffn.py,
// checks them, allocates what the caller did not give and calls the C ABI on the current
// stream of their GPU (5.4 us a call of int8_quantize, 3.6 with its outputs given).
//
// Only host code: the library's C ABI and torch's C++ interface.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>

#include <cstring>
#include <string>

#include "../../include/fp4g_ffn.h"

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

std::string dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kChar: return "torch.int8";
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

int activation(PyObject* o) {
  const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  if (s) {
    if (!std::strcmp(s, "silu")) return FP4G_ACT_SILU;
    if (!std::strcmp(s, "gelu")) return FP4G_ACT_GELU;
    if (!std::strcmp(s, "gelu_tanh")) return FP4G_ACT_GELU_TANH;
  }
  PyErr_Clear();
  PyObject* r = PyObject_Repr(o);
  const char* text = r ? PyUnicode_AsUTF8(r) : nullptr;
  std::string what = std::string("act must be one of silu, gelu, gelu_tanh, got ") + (text ? text : "?");
  Py_XDECREF(r);
  PyErr_Clear();
  value_error(what);
}

// The result of a product: `out`, or a new tensor of out_dtype.
at::Tensor output(PyObject* out, PyObject* out_dtype, int64_t M, int64_t N, at::Device device, int* d_type) {
  at::ScalarType t;
  if (out != Py_None) t = tensor(out, "out").scalar_type();
  else if (THPDtype_Check(out_dtype)) t = reinterpret_cast<THPDtype*>(out_dtype)->scalar_type;
  else type_error("out_dtype must be a torch.dtype");
  if (t != at::kBFloat16 && t != at::kFloat) type_error("out must be float32 or bfloat16");
  *d_type = t == at::kBFloat16 ? FP4G_OUT_BF16 : FP4G_OUT_F32;
  return result(out, "out", t, {M, N}, device);
}

void multiple_of(int64_t K, int64_t step) {
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

// X, codes, scales
PyObject* py_int8_quantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 3, [&] {
    const at::Tensor& X = matrix(v[0], "X", at::kFloat, at::kBFloat16);
    const int64_t rows = X.size(0), K = X.size(1);
    const at::Device device = X.device();
    const c10::DeviceGuard guard(device);
    multiple_of(K, 16);
    const at::Tensor codes = result(v[1], "codes", at::kChar, {rows, K}, device);
    const at::Tensor scales = result(v[2], "scales", at::kFloat, {rows}, device);
    launch("int8_quantize", device, [&](void* stream) {
      return int8_quantize(rows, K, ptr(X), X.scalar_type() == at::kBFloat16 ? FP4G_IN_BF16 : FP4G_IN_F32,
                           ptr(codes), floats(scales), stream);
    });
    return tuple({codes, scales});
  });
}

// A, sa, B, sb, out, out_dtype, workspace
PyObject* py_w8a8_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 7, [&] {
    const at::Tensor& A = matrix(v[0], "A", at::kChar, at::kChar);
    const int64_t M = A.size(0), K = A.size(1);
    const at::Device device = A.device();
    const c10::DeviceGuard guard(device);
    multiple_of(K, 16);
    const int64_t N = matrix(v[2], "B", at::kChar, at::kChar).size(0);
    const at::Tensor& B = need(v[2], "B", at::kChar, {N, K}, device);
    const at::Tensor& sb = need(v[3], "sb", at::kFloat, {N}, device);
    const at::Tensor& sa = need(v[1], "sa", at::kFloat, {M}, device);
    int d_type;
    const at::Tensor D = output(v[4], v[5], M, N, device, &d_type);
    const Space w = space(v[6], device, [&] {
      size_t bytes = 0;
      check_status("w8a8_gemm_workspace_size", w8a8_gemm_workspace_size(M, N, K, &bytes));
      return bytes;
    });
    launch("w8a8_gemm", device, [&](void* stream) {
      return w8a8_gemm(M, N, K, ptr(A), floats(sa), ptr(B), floats(sb), ptr(D), d_type, w.p, w.bytes, stream);
    });
    return THPVariable_Wrap(D);
  });
}

// A, sa, Bg, sg, Bu, su, act, out, out_dtype, workspace
PyObject* py_w8a8_gated_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 10, [&] {
    const at::Tensor& A = matrix(v[0], "A", at::kChar, at::kChar);
    const int64_t M = A.size(0), K = A.size(1);
    const at::Device device = A.device();
    const c10::DeviceGuard guard(device);
    multiple_of(K, 16);
    const int64_t N = matrix(v[2], "Bg", at::kChar, at::kChar).size(0);
    const at::Tensor& Bg = need(v[2], "Bg", at::kChar, {N, K}, device);
    const at::Tensor& sg = need(v[3], "sg", at::kFloat, {N}, device);
    const at::Tensor& Bu = need(v[4], "Bu", at::kChar, {N, K}, device);
    const at::Tensor& su = need(v[5], "su", at::kFloat, {N}, device);
    const at::Tensor& sa = need(v[1], "sa", at::kFloat, {M}, device);
    const int act = activation(v[6]);
    int d_type;
    const at::Tensor D = output(v[7], v[8], M, N, device, &d_type);
    const Space w = space(v[9], device, [&] {
      size_t bytes = 0;
      check_status("w8a8_gated_gemm_workspace_size", w8a8_gated_gemm_workspace_size(M, N, K, &bytes));
      return bytes;
    });
    launch("w8a8_gated_gemm", device, [&](void* stream) {
      return w8a8_gated_gemm(M, N, K, ptr(A), floats(sa), ptr(Bg), floats(sg), ptr(Bu), floats(su), act, ptr(D),
                             d_type, w.p, w.bytes, stream);
    });
    return THPVariable_Wrap(D);
  });
}

// X, Wg, Wu, act, save, out, workspace.  None where autograd has to record the call: ffn.py makes
// it again from its autograd function.
PyObject* py_gated_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 7, [&] {
    const at::Tensor& X = matrix(v[0], "X", at::kBFloat16, at::kBFloat16);
    const int64_t M = X.size(0), K = X.size(1);
    const at::Device device = X.device();
    const c10::DeviceGuard guard(device);
    const int64_t N = matrix(v[1], "Wg", at::kBFloat16, at::kBFloat16).size(0);
    multiple_of(K, 8);
    const at::Tensor& Wg = need(v[1], "Wg", at::kBFloat16, {N, K}, device);
    const at::Tensor& Wu = need(v[2], "Wu", at::kBFloat16, {N, K}, device);
    const int act = activation(v[3]);
    const int save = PyObject_IsTrue(v[4]);
    if (save < 0) throw Raised{};
    if (c10::GradMode::is_enabled() && (X.requires_grad() || Wg.requires_grad() || Wu.requires_grad())) Py_RETURN_NONE;
    const at::Tensor H = result(v[5], "out", at::kBFloat16, {M, N}, device);
    at::Tensor G, U;
    if (save) {
      G = empty({M, N}, at::kFloat, device);
      U = empty({M, N}, at::kFloat, device);
    }
    const Space w = space(v[6], device, [&] {
      size_t bytes = 0;
      check_status("gated_gemm_workspace_size", gated_gemm_workspace_size(M, N, K, &bytes));
      return bytes;
    });
    launch("gated_gemm", device, [&](void* stream) {
      return gated_gemm(M, N, K, ptr(X), ptr(Wg), ptr(Wu), act, ptr(H), save ? floats(G) : nullptr, save ?
                        floats(U) : nullptr, w.p, w.bytes, stream);
    });
    return save ? tuple({H, G, U}) : THPVariable_Wrap(H);
  });
}

// dH, X, Wg, Wu, G, U, act, workspace
PyObject* py_gated_gemm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 8, [&] {
    const at::Tensor& X = matrix(v[1], "X", at::kBFloat16, at::kBFloat16);
    const int64_t M = X.size(0), K = X.size(1);
    const at::Device device = X.device();
    const c10::DeviceGuard guard(device);
    const int64_t N = matrix(v[2], "Wg", at::kBFloat16, at::kBFloat16).size(0);
    multiple_of(K, 8);
    const at::Tensor& Wg = need(v[2], "Wg", at::kBFloat16, {N, K}, device);
    const at::Tensor& Wu = need(v[3], "Wu", at::kBFloat16, {N, K}, device);
    const int act = activation(v[6]);
    const at::Tensor& dH = need(v[0], "dH", at::kBFloat16, {M, N}, device);
    const at::Tensor& G = need(v[4], "G", at::kFloat, {M, N}, device);
    const at::Tensor& U = need(v[5], "U", at::kFloat, {M, N}, device);
    const at::Tensor dX = empty({M, K}, at::kBFloat16, device);
    const at::Tensor dWg = empty({N, K}, at::kBFloat16, device);
    const at::Tensor dWu = empty({N, K}, at::kBFloat16, device);
    const Space w = space(v[7], device, [&] {
      size_t bytes = 0, least = 0;
      check_status("gated_gemm_backward_workspace_size", gated_gemm_backward_workspace_size(M, N, K, &bytes, &least));
      return bytes;
    });
    launch("gated_gemm_backward", device, [&](void* stream) {
      return gated_gemm_backward(M, N, K, ptr(dH), ptr(X), ptr(Wg), ptr(Wu), floats(G), floats(U), act, ptr(dX),
                                 ptr(dWg), ptr(dWu), w.p, w.bytes, stream);
    });
    return tuple({dX, dWg, dWu});
  });
}

#define FASTCALL(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FASTCALL(int8_quantize), FASTCALL(w8a8_gemm), FASTCALL(w8a8_gated_gemm), FASTCALL(gated_gemm),
                         FASTCALL(gated_gemm_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ffn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__ffn_binding() { return PyModule_Create(&module); }
