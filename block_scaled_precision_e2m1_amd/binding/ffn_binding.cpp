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
#include "common.hpp"

#include "../../include/fp4g_ffn.h"

namespace {

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
    no_tangents("gated_gemm", {&X, &Wg, &Wu});
    if (c10::GradMode::is_enabled() && (X.requires_grad() || Wg.requires_grad() || Wu.requires_grad())) Py_RETURN_NONE;
    const at::Tensor H = result(v[5], "out", at::kBFloat16, {M, N}, device);
    no_tangents("gated_gemm", {&H});
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

PyMethodDef methods[] = {FASTCALL(int8_quantize), FASTCALL(w8a8_gemm), FASTCALL(w8a8_gated_gemm), FASTCALL(gated_gemm),
                         FASTCALL(gated_gemm_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ffn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__ffn_binding() { return PyModule_Create(&module); }
