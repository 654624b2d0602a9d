// The Python binding of the operators around a language model's products
// (include/fp4g_lm.h) over torch tensors, in the manner of ffn_binding.cpp: every function takes
// its arguments by position from the Python function of the same name in lm.py, checks them,
// allocates what the caller did not give and calls the C ABI on the current stream of their
// GPU.  Functions that autograd may have to record return None where it has to.
#include "common.hpp"

#include "../../include/fp4g_lm.h"

namespace {

int type_of(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? FP4G_IN_BF16 : FP4G_IN_F32; }

bool recorded(std::initializer_list<const at::Tensor*> ts) {
  if (!c10::GradMode::is_enabled()) return false;
  for (const at::Tensor* t : ts)
    if (t && t->defined() && t->requires_grad()) return true;
  return false;
}

// A tensor of the caller's that is written: autograd learns of it where it is kept for a
// backward pass, and it may not itself be waiting for a gradient or carry a tangent.
at::Tensor written(const char* fn, PyObject* given, const char* name, at::ScalarType dtype, at::IntArrayRef shape, at::Device device) {
  const at::Tensor t = result(given, name, dtype, shape, device);
  if (given != Py_None) {
    no_tangents(fn, {&t});
    if (recorded({&t})) value_error(std::string(name) + " requires a gradient");
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
  return t;
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be a number");
  }
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

// What every norm takes: X, weight, eps, and the residual with its sum.
struct Norm {
  at::Tensor X, W, R, H;
  int64_t rows, K;
  double eps;
  int w_type;
  const void* w() const { return W.defined() ? ptr(W) : nullptr; }
  const void* r() const { return R.defined() ? ptr(R) : nullptr; }
  void* h() const { return H.defined() ? ptr(H) : nullptr; }
};
Norm norm_of(PyObject* x, PyObject* weight, PyObject* eps, PyObject* residual) {
  Norm n;
  n.X = matrix(x, "X", at::kFloat, at::kBFloat16);
  n.rows = n.X.size(0), n.K = n.X.size(1);
  if (weight != Py_None) {
    const at::ScalarType t = tensor(weight, "weight").scalar_type();
    if (t != at::kFloat && t != at::kBFloat16)
      type_error("weight must have dtype torch.float32 or torch.bfloat16, got " + dtype_name(t));
    n.W = need(weight, "weight", t, {n.K}, n.X.device());
  }
  n.w_type = n.W.defined() ? type_of(n.W) : FP4G_IN_F32;
  n.eps = number(eps, "eps");
  if (residual != Py_None) n.R = need(residual, "residual", n.X.scalar_type(), {n.rows, n.K}, n.X.device());
  return n;
}

// X, weight, eps, residual, out, sum_out
PyObject* py_rms_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 6, [&] {
    Norm a = norm_of(v[0], v[1], v[2], v[3]);
    const at::Device device = a.X.device();
    const c10::DeviceGuard guard(device);
    if (v[3] == Py_None && v[5] != Py_None) value_error("sum_out without a residual");
    no_tangents("rms_norm", {&a.X, &a.W, &a.R});
    if (recorded({&a.X, &a.W, &a.R})) {
      if (v[4] != Py_None || v[5] != Py_None) value_error("out and sum_out are not taken where a gradient is recorded");
      Py_RETURN_NONE;
    }
    const at::Tensor Y = written("rms_norm", v[4], "out", a.X.scalar_type(), {a.rows, a.K}, device);
    if (a.R.defined()) a.H = written("rms_norm", v[5], "sum_out", a.X.scalar_type(), {a.rows, a.K}, device);
    launch("rms_norm", device, [&](void* stream) {
      return rms_norm(a.rows, a.K, ptr(a.X), type_of(a.X), a.r(), a.w(), a.w_type, a.eps, a.h(), ptr(Y), stream);
    });
    return a.R.defined() ? tuple({Y, a.H}) : THPVariable_Wrap(Y);
  });
}

// X, weight, eps, residual, codes, keep, sum_out
PyObject* py_rms_norm_quantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 7, [&] {
    Norm a = norm_of(v[0], v[1], v[2], v[3]);
    const at::Device device = a.X.device();
    const c10::DeviceGuard guard(device);
    const char* name = PyUnicode_Check(v[4]) ? PyUnicode_AsUTF8(v[4]) : nullptr;
    PyErr_Clear();
    const bool int8 = name && !std::strcmp(name, "int8");
    if (!int8 && !(name && !std::strcmp(name, "e4m3")))
      value_error(std::string("codes must be \"int8\" or \"e4m3\"") + (name ? std::string(", got ") + name : ""));
    const bool keep = truth(v[5]);
    if (v[3] == Py_None && v[6] != Py_None) value_error("sum_out without a residual");
    no_tangents("rms_norm_quantize", {&a.X, &a.W, &a.R});
    if (recorded({&a.X, &a.W, &a.R})) value_error("rms_norm_quantize has no gradient: call it under torch.no_grad()");
    const at::Tensor codes = empty({a.rows, a.K}, int8 ? at::kChar : at::kByte, device);
    const at::Tensor scales = empty({a.rows}, at::kFloat, device);
    at::Tensor Y;
    if (a.R.defined()) a.H = written("rms_norm_quantize", v[6], "sum_out", a.X.scalar_type(), {a.rows, a.K}, device);
    if (keep) Y = empty({a.rows, a.K}, a.X.scalar_type(), device);
    launch("rms_norm_quantize", device, [&](void* stream) {
      return rms_norm_quantize(a.rows, a.K, ptr(a.X), type_of(a.X), a.r(), a.w(), a.w_type, a.eps, a.h(),
                               keep ? ptr(Y) : nullptr, ptr(codes), int8 ? FP4G_CODE_INT8 : FP4G_CODE_E4M3,
                               floats(scales), stream);
    });
    if (a.R.defined()) return keep ? tuple({codes, scales, a.H, Y}) : tuple({codes, scales, a.H});
    return keep ? tuple({codes, scales, Y}) : tuple({codes, scales});
  });
}

// dY, X, weight, eps, dH, want_dw, workspace
PyObject* py_rms_norm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 7, [&] {
    const Norm a = norm_of(v[1], v[2], v[3], Py_None);
    const at::Device device = a.X.device();
    const c10::DeviceGuard guard(device);
    const at::ScalarType t = a.X.scalar_type();
    const at::Tensor& dY = need(v[0], "dY", t, {a.rows, a.K}, device);
    at::Tensor dH, dW;
    if (v[4] != Py_None) dH = need(v[4], "dH", t, {a.rows, a.K}, device);
    if (a.W.defined() && truth(v[5])) dW = empty({a.K}, a.W.scalar_type(), device);
    const at::Tensor dX = empty({a.rows, a.K}, t, device);
    const Space w = space(v[6], device, [&] {
      size_t bytes = 0;
      check_status("rms_norm_backward_workspace_size", rms_norm_backward_workspace_size(a.rows, a.K, type_of(a.X), &bytes));
      return bytes;
    });
    launch("rms_norm_backward", device, [&](void* stream) {
      return rms_norm_backward(a.rows, a.K, ptr(dY), ptr(a.X), type_of(a.X), a.w(), a.w_type, a.eps,
                               dH.defined() ? ptr(dH) : nullptr, ptr(dX), dW.defined() ? ptr(dW) : nullptr, w.p,
                               w.bytes, stream);
    });
    return tuple({dX, dW});   // None for an undefined tensor
  });
}

// What both passes of the loss take: X, W, target and ignore_index.
struct Loss {
  at::Tensor X, W, target;
  int64_t M, V, K, ignore;
};
Loss loss_of(PyObject* x, PyObject* w, PyObject* target, PyObject* ignore) {
  Loss a;
  a.X = matrix(x, "X", at::kBFloat16, at::kBFloat16);
  a.M = a.X.size(0), a.K = a.X.size(1);
  a.V = matrix(w, "W", at::kBFloat16, at::kBFloat16).size(0);
  multiple_of(a.K, 8);
  a.W = need(w, "W", at::kBFloat16, {a.V, a.K}, a.X.device());
  a.target = need(target, "target", at::kLong, {a.M}, a.X.device());
  a.ignore = PyLong_AsLongLong(ignore);
  if (a.ignore == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("ignore_index must be an integer of 64 bits");
  }
  return a;
}

// X, W, target, ignore_index, save, workspace
PyObject* py_cross_entropy_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 6, [&] {
    const Loss a = loss_of(v[0], v[1], v[2], v[3]);
    const at::Device device = a.X.device();
    const c10::DeviceGuard guard(device);
    const bool save = truth(v[4]);
    no_tangents("cross_entropy_gemm", {&a.X, &a.W});
    if (recorded({&a.X, &a.W})) Py_RETURN_NONE;
    const at::Tensor loss = empty({a.M}, at::kFloat, device);
    at::Tensor lse;
    if (save) lse = empty({a.M}, at::kFloat, device);
    const Space w = space(v[5], device, [&] {
      size_t bytes = 0;
      check_status("cross_entropy_gemm_workspace_size", cross_entropy_gemm_workspace_size(a.M, a.V, a.K, &bytes));
      return bytes;
    });
    launch("cross_entropy_gemm", device, [&](void* stream) {
      return cross_entropy_gemm(a.M, a.V, a.K, ptr(a.X), ptr(a.W), static_cast<const int64_t*>(ptr(a.target)), a.ignore,
                                floats(loss), save ? floats(lse) : nullptr, w.p, w.bytes, stream);
    });
    return save ? tuple({loss, lse}) : THPVariable_Wrap(loss);
  });
}

// dL, X, W, target, lse, ignore_index, want_dx, want_dw, workspace
PyObject* py_cross_entropy_gemm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 9, [&] {
    const Loss a = loss_of(v[1], v[2], v[3], v[5]);
    const at::Device device = a.X.device();
    const c10::DeviceGuard guard(device);
    const at::Tensor& dL = need(v[0], "dL", at::kFloat, {a.M}, device);
    const at::Tensor& lse = need(v[4], "lse", at::kFloat, {a.M}, device);
    at::Tensor dX, dW;
    if (truth(v[6])) dX = empty({a.M, a.K}, at::kBFloat16, device);
    if (truth(v[7])) dW = empty({a.V, a.K}, at::kBFloat16, device);
    const Space w = space(v[8], device, [&] {
      size_t bytes = 0, least = 0;
      check_status("cross_entropy_gemm_backward_workspace_size",
                   cross_entropy_gemm_backward_workspace_size(a.M, a.V, a.K, &bytes, &least));
      return bytes;
    });
    launch("cross_entropy_gemm_backward", device, [&](void* stream) {
      return cross_entropy_gemm_backward(a.M, a.V, a.K, floats(dL), ptr(a.X), ptr(a.W),
                                         static_cast<const int64_t*>(ptr(a.target)), a.ignore, floats(lse),
                                         dX.defined() ? ptr(dX) : nullptr, dW.defined() ? ptr(dW) : nullptr, w.p,
                                         w.bytes, stream);
    });
    return tuple({dX, dW});   // None for an undefined tensor
  });
}

// base, X, A, B, index, scales, out, workspace
PyObject* py_adapter_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return entry(n, 8, [&] {
    const at::Tensor& base = matrix(v[0], "base", at::kBFloat16, at::kFloat);
    const int64_t M = base.size(0), N = base.size(1);
    const at::Device device = base.device();
    const c10::DeviceGuard guard(device);
    const int64_t K = matrix(v[1], "X", at::kBFloat16, at::kBFloat16).size(1);
    const at::Tensor& X = need(v[1], "X", at::kBFloat16, {M, K}, device);
    const at::Tensor& first = tensor(v[2], "A");
    if (first.dim() != 3) value_error("A must be 3-D");
    const int64_t L = first.size(0), R = first.size(1);
    const at::Tensor& A = need(v[2], "A", at::kBFloat16, {L, R, K}, device);
    const at::Tensor& B = need(v[3], "B", at::kBFloat16, {L, N, R}, device);
    const at::Tensor& index = need(v[4], "index", at::kInt, {M}, device);
    at::Tensor scales;
    if (v[5] != Py_None) scales = need(v[5], "scales", at::kFloat, {L}, device);
    multiple_of(K, 8);
    if (R % 8) value_error("R=" + std::to_string(R) + " must be a multiple of 8");
    no_tangents("adapter_gemm", {&base, &X, &A, &B, &scales});
    if (recorded({&base, &X, &A, &B, &scales})) value_error("adapter_gemm has no gradient: call it under torch.no_grad()");
    const at::Tensor D = written("adapter_gemm", v[6], "out", base.scalar_type(), {M, N}, device);
    const Space w = space(v[7], device, [&] {
      size_t bytes = 0;
      check_status("adapter_gemm_workspace_size", adapter_gemm_workspace_size(M, N, K, R, L, &bytes));
      return bytes;
    });
    launch("adapter_gemm", device, [&](void* stream) {
      return adapter_gemm(M, N, K, R, L, ptr(base), ptr(X), ptr(A), ptr(B), scales.defined() ? floats(scales) : nullptr,
                          static_cast<const int32_t*>(ptr(index)), ptr(D),
                          base.scalar_type() == at::kBFloat16 ? FP4G_OUT_BF16 : FP4G_OUT_F32, w.p, w.bytes, stream);
    });
    return THPVariable_Wrap(D);
  });
}

PyMethodDef methods[] = {FASTCALL(rms_norm), FASTCALL(rms_norm_quantize), FASTCALL(rms_norm_backward),
                         FASTCALL(cross_entropy_gemm), FASTCALL(cross_entropy_gemm_backward), FASTCALL(adapter_gemm),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lm_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__lm_binding() { return PyModule_Create(&module); }
