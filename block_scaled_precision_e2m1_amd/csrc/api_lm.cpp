// C-ABI entry points of the operators around a language model's products: validate on the
// host, pick a kernel, launch on the caller's stream.  Validation runs before any HIP call,
// so an invalid call returns its status without touching the device.
#include "lm_internal.h"

#include <algorithm>
#include <cmath>

#include "api_checks.hpp"

namespace {

using fp4g::buf;
using fp4g::Buffer;
using fp4g::check_buffers;

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxElems = (int64_t)1 << 50;

bool sizes_fit(std::initializer_list<int64_t> dims) {
  for (int64_t d : dims)
    if (d < 0 || d >= kMaxDim) return false;
  return true;
}
// Whether a buffer of a x b (x c) elements is within the limit; each is below 2^31.
bool holds(int64_t a, int64_t b, int64_t c = 1) {
  if (a == 0 || b == 0 || c == 0) return true;
  return a <= kMaxElems / b && a * b <= kMaxElems / c;
}

bool known_type(int t) { return t == FP4G_IN_F32 || t == FP4G_IN_BF16; }
int64_t size_of(int t) { return t == FP4G_IN_BF16 ? 2 : 4; }

fp4g_status finish(hipError_t e) { return e == hipSuccess ? FP4G_OK : FP4G_EHIP; }

hipError_t zero(void* p, int64_t count, bool bf16, hipStream_t s) {
  return count > 0 ? fp4g::launch_zero_fill(p, count, bf16, s) : hipSuccess;
}

// An input that an output may stand in place of: the two are one buffer then, which the
// output is checked for.
Buffer unless(const Buffer& in, std::initializer_list<const void*> outs) {
  for (const void* o : outs)
    if (o && o == in.p) return buf(nullptr, 0);
  return in;
}

// The arguments of a norm; `codes` true where it is quantized.
fp4g_status check_norm(int64_t rows, int64_t K, const void* X, int x_type, const void* R, const void* W, int w_type,
                       double eps, const void* H, const void* Y, bool quantized, const void* codes, int code_type,
                       const float* scales) {
  if (!sizes_fit({rows, K}) || !holds(rows, K)) return FP4G_EINVAL;
  if (!known_type(x_type) || (W && !known_type(w_type))) return FP4G_EINVAL;
  if (quantized && code_type != FP4G_CODE_INT8 && code_type != FP4G_CODE_E4M3) return FP4G_EINVAL;
  if (!std::isfinite(eps) || eps < 0.0 || !R != !H) return FP4G_EINVAL;
  const int64_t e = size_of(x_type), bytes = rows * K * e, we = size_of(w_type);
  const Buffer x = buf(X, bytes, e), r = buf(R, R ? bytes : 0, e), w = buf(W, W && rows ? K * we : 0, we);
  const Buffer h = buf(H, H ? bytes : 0, e), y = buf(Y, Y || !quantized ? bytes : 0, e);
  const Buffer c = buf(codes, quantized ? rows * K : 0, 1), s = buf(scales, quantized ? rows * 4 : 0, 4);
  const fp4g_status st = check_buffers({x, r, w}, {});
  if (st != FP4G_OK) return st;
  return check_buffers({unless(x, {H, Y}), unless(r, {H, Y}), w}, {h, y, c, s});
}

// Sizes of a loss's products: rows of X and W are operands of the tiles.
fp4g_status check_loss_sizes(int64_t M, int64_t V, int64_t K) {
  if (!sizes_fit({M, V, K}) || !holds(M, K) || !holds(V, K) || !holds(M, V) || (M > 0 && V == 0)) return FP4G_EINVAL;
  return K % 8 != 0 || K > (1 << 21) || M > (1 << 25) ? FP4G_EUNSUPPORTED : FP4G_OK;
}

// The columns of a piece for a workspace of `room` bytes: the choice without a limit, or as many
// as fit; 0 if none do.
int64_t piece_cols(int64_t M, int64_t V, int64_t K, size_t room) {
  for (int64_t cols = fp4g::loss_grad_cols(M, V, K);; cols = std::max<int64_t>(64, cols / 2 / 64 * 64)) {
    if ((size_t)fp4g::loss_grad_bytes(M, V, K, cols) <= room) return cols;
    if (cols == 64) return 0;
  }
}

fp4g_status check_adapter_sizes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L) {
  if (!sizes_fit({M, N, K, R, L}) || !holds(M, N) || !holds(M, K) || !holds(L, R, K) || !holds(L, N, R)) return FP4G_EINVAL;
  return K % 8 != 0 || R % 8 != 0 || R > 256 || K > (1 << 21) || L > fp4g::kMaxAdapters || M > (1 << 25) || N > (1 << 30)
             ? FP4G_EUNSUPPORTED
             : FP4G_OK;
}

}  // namespace

extern "C" {

fp4g_status rms_norm(int64_t rows, int64_t K, const void* X, int x_type, const void* R, const void* W, int w_type,
                     double eps, void* H, void* Y, void* stream) {
  const fp4g_status st = check_norm(rows, K, X, x_type, R, W, w_type, eps, H, Y, false, nullptr, 0, nullptr);
  if (st != FP4G_OK || rows == 0 || K == 0) return st;
  fp4g::NormArgs a{rows, K, X, R, W, H, Y, x_type == FP4G_IN_BF16, w_type == FP4G_IN_BF16, eps};
  return finish(fp4g::launch_rms_norm(a, reinterpret_cast<hipStream_t>(stream)));
}

fp4g_status rms_norm_quantize(int64_t rows, int64_t K, const void* X, int x_type, const void* R, const void* W,
                              int w_type, double eps, void* H, void* Y, void* codes, int code_type, float* scales,
                              void* stream) {
  const fp4g_status st = check_norm(rows, K, X, x_type, R, W, w_type, eps, H, Y, true, codes, code_type, scales);
  if (st != FP4G_OK || rows == 0) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (K == 0) return finish(zero(scales, rows, false, s));
  fp4g::NormArgs a{rows, K, X, R, W, H, Y, x_type == FP4G_IN_BF16, w_type == FP4G_IN_BF16, eps};
  a.codes = codes, a.scales = scales, a.e4m3 = code_type == FP4G_CODE_E4M3;
  return finish(fp4g::launch_rms_norm(a, s));
}

fp4g_status rms_norm_backward_workspace_size(int64_t rows, int64_t K, int x_type, size_t* bytes) {
  if (!sizes_fit({rows, K}) || !holds(rows, K) || !known_type(x_type) || !bytes) return FP4G_EINVAL;
  *bytes = rows == 0 || K == 0 ? 0 : (size_t)fp4g::rms_norm_grad_bytes(rows, K, x_type == FP4G_IN_BF16);
  return FP4G_OK;
}

fp4g_status rms_norm_backward(int64_t rows, int64_t K, const void* dY, const void* X, int x_type, const void* W,
                              int w_type, double eps, const void* dH, void* dX, void* dW, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (!sizes_fit({rows, K}) || !holds(rows, K)) return FP4G_EINVAL;
  if (!known_type(x_type) || (W && !known_type(w_type))) return FP4G_EINVAL;
  if (!std::isfinite(eps) || eps < 0.0 || (dW && !W)) return FP4G_EINVAL;
  const int64_t e = size_of(x_type), bytes = rows * K * e, we = size_of(w_type);
  const Buffer dy = buf(dY, bytes, e), x = buf(X, bytes, e), w = buf(W, W && rows ? K * we : 0, we);
  const Buffer dh = buf(dH, dH ? bytes : 0, e);
  fp4g_status st = check_buffers({dy, x, w, dh}, {});
  if (st != FP4G_OK) return st;
  const bool some = rows > 0 && K > 0, bf16 = x_type == FP4G_IN_BF16;
  st = check_buffers({unless(dy, {dX}), x, w, unless(dh, {dX})},
                     {buf(dX, bytes, e), buf(dW, dW ? K * we : 0, we), buf(workspace, some ? workspace_bytes : 0)});
  if (st != FP4G_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (!some) return finish(dW ? zero(dW, K, w_type == FP4G_IN_BF16, s) : hipSuccess);
  if (workspace_bytes < (size_t)fp4g::rms_norm_grad_bytes(rows, K, bf16)) return FP4G_EINVAL;
  const fp4g::NormGradArgs a{rows, K, dY, X, W, dH, dX, dW, bf16, w_type == FP4G_IN_BF16, eps, workspace};
  return finish(fp4g::launch_rms_norm_grad(a, s));
}

fp4g_status cross_entropy_gemm_workspace_size(int64_t M, int64_t V, int64_t K, size_t* bytes) {
  const fp4g_status st = check_loss_sizes(M, V, K);
  if (st != FP4G_OK) return st;
  if (!bytes) return FP4G_EINVAL;
  *bytes = M == 0 ? 0 : (size_t)fp4g::loss_bytes(M, V, K);
  return FP4G_OK;
}

fp4g_status cross_entropy_gemm(int64_t M, int64_t V, int64_t K, const void* X, const void* W, const int64_t* target,
                               int64_t ignore_index, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                               void* stream) {
  fp4g_status st = check_loss_sizes(M, V, K);
  if (st != FP4G_OK || M == 0) return st;
  st = check_buffers({buf(X, M * K * 2), buf(W, V * K * 2), buf(target, M * 8, 8)},
                     {buf(loss, M * 4, 4), buf(lse, lse ? M * 4 : 0, 4), buf(workspace, workspace_bytes)});
  if (st != FP4G_OK) return st;
  if (workspace_bytes < (size_t)fp4g::loss_bytes(M, V, K)) return FP4G_EINVAL;
  fp4g::LossCall c{M, V, K, X, W, target, ignore_index};
  c.loss = loss, c.lse = lse, c.space = static_cast<uint8_t*>(workspace);
  return finish(fp4g::launch_loss(c, reinterpret_cast<hipStream_t>(stream)));
}

fp4g_status cross_entropy_gemm_backward_workspace_size(int64_t M, int64_t V, int64_t K, size_t* bytes, size_t* least) {
  const fp4g_status st = check_loss_sizes(M, V, K);
  if (st != FP4G_OK) return st;
  if (!bytes || !least) return FP4G_EINVAL;
  *bytes = *least = 0;
  if (M == 0 || K == 0) return FP4G_OK;
  *bytes = (size_t)fp4g::loss_grad_bytes(M, V, K, fp4g::loss_grad_cols(M, V, K));
  *least = std::min(*bytes, (size_t)fp4g::loss_grad_bytes(M, V, K, 64));
  return FP4G_OK;
}

fp4g_status cross_entropy_gemm_backward(int64_t M, int64_t V, int64_t K, const float* dL, const void* X, const void* W,
                                        const int64_t* target, int64_t ignore_index, const float* lse, void* dX,
                                        void* dW, void* workspace, size_t workspace_bytes, void* stream) {
  fp4g_status st = check_loss_sizes(M, V, K);
  if (st != FP4G_OK || K == 0) return st;
  const bool some = M > 0;
  st = check_buffers({buf(dL, M * 4, 4), buf(X, M * K * 2), buf(W, some ? V * K * 2 : 0), buf(target, M * 8, 8),
                      buf(lse, M * 4, 4)},
                     {buf(dX, dX ? M * K * 2 : 0), buf(dW, dW ? V * K * 2 : 0), buf(workspace, some ? workspace_bytes : 0)});
  if (st != FP4G_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (!some) return finish(dW ? zero(dW, V * K, true, s) : hipSuccess);
  const int64_t cols = piece_cols(M, V, K, workspace_bytes);
  if (cols == 0) return FP4G_EINVAL;
  if (!dX && !dW) return FP4G_OK;
  fp4g::LossCall c{M, V, K, X, W, target, ignore_index};
  c.lse = const_cast<float*>(lse), c.dL = dL, c.dX = dX, c.dW = dW;
  c.space = static_cast<uint8_t*>(workspace), c.cols = cols;
  return finish(fp4g::launch_loss_grad(c, s));
}

fp4g_status adapter_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, size_t* bytes) {
  const fp4g_status st = check_adapter_sizes(M, N, K, R, L);
  if (st != FP4G_OK) return st;
  if (!bytes) return FP4G_EINVAL;
  *bytes = M == 0 || N == 0 ? 0 : (size_t)fp4g::adapter_bytes(M, N, K, R, L);
  return FP4G_OK;
}

fp4g_status adapter_gemm(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, const void* base, const void* X,
                         const void* A, const void* B, const float* scales, const int32_t* index, void* D, int d_type,
                         void* workspace, size_t workspace_bytes, void* stream) {
  fp4g_status st = check_adapter_sizes(M, N, K, R, L);
  if (st != FP4G_OK) return st;
  if (d_type != FP4G_OUT_F32 && d_type != FP4G_OUT_BF16) return FP4G_EINVAL;
  if (M == 0 || N == 0) return FP4G_OK;
  const int64_t e = d_type == FP4G_OUT_BF16 ? 2 : 4;
  const Buffer b = buf(base, M * N * e, e);
  const Buffer x = buf(X, M * K * 2), wa = buf(A, L * R * K * 2), wb = buf(B, L * N * R * 2);
  const Buffer s = buf(scales, scales ? L * 4 : 0, 4), i = buf(index, M * 4, 4);
  st = check_buffers({b, x, wa, wb, s, i}, {});
  if (st != FP4G_OK) return st;
  st = check_buffers({unless(b, {D}), x, wa, wb, s, i}, {buf(D, M * N * e, e), buf(workspace, workspace_bytes)});
  if (st != FP4G_OK) return st;
  if (workspace_bytes < (size_t)fp4g::adapter_bytes(M, N, K, R, L)) return FP4G_EINVAL;
  const fp4g::AdapterCall c{M, N, K, R, L, base, X, A, B, scales, index, D, e == 2, static_cast<uint8_t*>(workspace)};
  return finish(fp4g::launch_adapter_gemm(c, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
