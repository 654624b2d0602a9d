// C-ABI entry points of the feed-forward operators: validate on the host, pick a kernel,
// launch on the caller's stream.  Validation runs before any HIP call, so an invalid call
// returns its status without touching the device.
#include "ffn_internal.h"

#include <algorithm>

#include "api_checks.hpp"

namespace {

using fp4g::buf;
using fp4g::check_buffers;
using fp4g::DenseArgs;
using fp4g::DensePlan;

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxElems = (int64_t)1 << 50;
// Row pitches below 2^22 bytes keep a tile of 256 rows inside a 31-bit buffer size.
constexpr int64_t kMaxPitch = (int64_t)1 << 22;
// int8 sums: K * 128 * 128 must stay below 2^31.
constexpr int64_t kMaxInt8K = ((int64_t)1 << 17) - 16;

// Sizes of a product whose operand rows hold K elements of `elem` bytes.
fp4g_status check_sizes(int64_t M, int64_t N, int64_t K, int elem) {
  for (int64_t d : {M, N, K})
    if (d < 0 || d >= kMaxDim) return FP4G_EINVAL;
  for (int64_t d : {M, N})
    if (K > 0 && d > kMaxElems / K) return FP4G_EINVAL;
  if (N > 0 && M > kMaxElems / N) return FP4G_EINVAL;
  if (K % (16 / elem) != 0 || K * elem > kMaxPitch) return FP4G_EUNSUPPORTED;
  if (elem == 1 && K > kMaxInt8K) return FP4G_EUNSUPPORTED;
  return FP4G_OK;
}

bool known_act(int act) { return act == FP4G_ACT_SILU || act == FP4G_ACT_GELU || act == FP4G_ACT_GELU_TANH; }
bool known_out(int t) { return t == FP4G_OUT_F32 || t == FP4G_OUT_BF16; }

fp4g_status finish(hipError_t e) { return e == hipSuccess ? FP4G_OK : FP4G_EHIP; }

// How many slices of partial sums of L products with `gates` weights each fit into `room` bytes.
int64_t slices(int64_t M, int64_t N, int64_t gates, int64_t L, size_t room) {
  const int64_t per = L * gates * M * fp4g::partial_pitch(N) * 4;
  const int64_t cap = per > 0 ? (int64_t)(room / (size_t)per) : 1;
  return cap > 1 ? cap : 1;
}
constexpr size_t kAnyRoom = ~(size_t)0 >> 1;
size_t partial_bytes(int64_t M, int64_t N, int64_t gates, int64_t L, const DensePlan& p) {
  return p.S > 1 ? (size_t)(L * p.S * gates * M * fp4g::partial_pitch(N) * 4) : 0;
}
int64_t stages(int64_t K, int elem) { return (K * elem + 127) / 128; }

// The last plan of this thread, by the sizes and the GPU's compute units: a call follows its
// workspace query, and choosing among tiles and splits anew takes it from 0.33 to 0.54 us at
// 4 x 160 x 160 and from 0.31 to 1.29 us at 4096 x 2048 x 1024 (the backward products' query).
template <class Plan>
struct LastPlan {
  int64_t key[6] = {-1, -1, -1, -1, -1, -1};
  Plan plan{};
  template <class F>
  const Plan& get(int64_t a, int64_t b, int64_t c, int64_t d, int64_t e, F&& choose) {
    const int64_t now[6] = {a, b, c, d, e, fp4g::device_cus()};
    if (!std::equal(now, now + 6, key)) {
      plan = choose();
      std::copy(now, now + 6, key);
    }
    return plan;
  }
};

// The plan of a scaled or gated product, given room for its partial sums: the best of all
// where they fit, else the best with fewer slices.
DensePlan product_plan(int64_t M, int64_t N, int64_t K, int elem, int64_t gates, size_t room) {
  static thread_local LastPlan<DensePlan> last;
  auto choose = [&](int64_t cap) {
    if (fp4g::gemv_takes(M, N, K * elem, gates))
      return DensePlan{fp4g::kGemv, fp4g::gemv_splits(M, N, K * elem, gates, cap), 0.0};
    return fp4g::dense_plan(M, gates * N, 1, stages(K, elem), cap);
  };
  const DensePlan& p = last.get(M, N, K, elem, gates, [&] { return choose(fp4g::kMaxSplits); });
  const int64_t cap = slices(M, N, gates, 1, room);
  return p.S <= cap ? p : choose(cap);
}
// dX (one product over both gradients' K) and dWg and dWu; their partial sums share the room.
fp4g::GradPlan grad_plan(int64_t M, int64_t N, int64_t K, size_t room) {
  static thread_local LastPlan<fp4g::GradPlan> last;
  const fp4g::GradPlan& p =
      last.get(M, N, K, 0, 0, [&] { return fp4g::grad_plan(M, N, K, fp4g::kMaxSplits, fp4g::kMaxSplits); });
  const int64_t cap_x = slices(M, K, 1, 1, room), cap_w = slices(N, K, 1, 2, room);
  return p.x.S <= cap_x && p.w.S <= cap_w ? p : fp4g::grad_plan(M, N, K, cap_x, cap_w);
}

fp4g_status product_workspace(int64_t M, int64_t N, int64_t K, int elem, int64_t gates, size_t* bytes) {
  const fp4g_status st = check_sizes(M, N, K, elem);
  if (st != FP4G_OK) return st;
  if (!bytes) return FP4G_EINVAL;
  *bytes = M == 0 || N == 0 || K == 0 ? 0 : partial_bytes(M, N, gates, 1, product_plan(M, N, K, elem, gates, kAnyRoom));
  return FP4G_OK;
}

// Rows of dG and dU: whole 128-byte K stages of dX.
int64_t grad_pitch(int64_t N) { return (N + 63) / 64 * 64; }

hipError_t zero(void* p, int64_t count, bool bf16, hipStream_t s) {
  return count > 0 ? fp4g::launch_zero_fill(p, count, bf16, s) : hipSuccess;
}

}  // namespace

extern "C" {

fp4g_status int8_quantize(int64_t rows, int64_t K, const void* X, int x_type, void* codes, float* scales,
                          void* stream) {
  const fp4g_status st = check_sizes(rows, 1, K, 1);
  // The row length limits of the products' operands do not bind here.
  if (st == FP4G_EINVAL) return st;
  if (x_type != FP4G_IN_F32 && x_type != FP4G_IN_BF16) return FP4G_EINVAL;
  if (K % 16 != 0) return FP4G_EUNSUPPORTED;
  if (rows == 0) return FP4G_OK;
  const bool bf16 = x_type == FP4G_IN_BF16;
  const fp4g_status sb = check_buffers({buf(X, rows * K * (bf16 ? 2 : 4))},
                                       {buf(codes, rows * K), buf(scales, rows * 4, 4)});
  if (sb != FP4G_OK) return sb;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (K == 0) return finish(zero(scales, rows, false, s));
  return finish(fp4g::launch_int8_quantize(rows, K, X, bf16, codes, scales, s));
}

fp4g_status w8a8_gemm_workspace_size(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  return product_workspace(M, N, K, 1, 1, bytes);
}

fp4g_status w8a8_gemm(int64_t M, int64_t N, int64_t K, const void* A, const float* sa, const void* B, const float* sb,
                      void* D, int d_type, void* workspace, size_t workspace_bytes, void* stream) {
  fp4g_status st = check_sizes(M, N, K, 1);
  if (st != FP4G_OK) return st;
  if (!known_out(d_type)) return FP4G_EINVAL;
  if (M == 0 || N == 0) return FP4G_OK;
  const bool bf16 = d_type == FP4G_OUT_BF16, some = K > 0;
  st = check_buffers({buf(A, M * K), buf(sa, some ? M * 4 : 0, 4), buf(B, N * K), buf(sb, some ? N * 4 : 0, 4)},
                     {buf(D, M * N * (bf16 ? 2 : 4)), buf(workspace, workspace_bytes)});
  if (st != FP4G_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (!some) return finish(zero(D, M * N, bf16, s));
  const DensePlan p = product_plan(M, N, K, 1, 1, workspace_bytes);
  DenseArgs a;
  a.M = (int)M, a.N = (int)N, a.K = (int)K, a.S = p.S;
  a.A[0] = static_cast<const uint8_t*>(A), a.B[0] = static_cast<const uint8_t*>(B);
  a.lda = a.ldb = K, a.sa = sa, a.sb[0] = sb, a.D[0] = D, a.P = workspace, a.bf16_out = bf16;
  return finish(fp4g::launch_w8a8(a, p.tile, s));
}

fp4g_status w8a8_gated_gemm_workspace_size(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  return product_workspace(M, N, K, 1, 2, bytes);
}

fp4g_status w8a8_gated_gemm(int64_t M, int64_t N, int64_t K, const void* A, const float* sa, const void* Bg,
                            const float* sg, const void* Bu, const float* su, int act, void* D, int d_type,
                            void* workspace, size_t workspace_bytes, void* stream) {
  fp4g_status st = check_sizes(M, N, K, 1);
  if (st != FP4G_OK) return st;
  if (!known_out(d_type) || !known_act(act)) return FP4G_EINVAL;
  if (M == 0 || N == 0) return FP4G_OK;
  const bool bf16 = d_type == FP4G_OUT_BF16, some = K > 0;
  st = check_buffers({buf(A, M * K), buf(sa, some ? M * 4 : 0, 4), buf(Bg, N * K), buf(sg, some ? N * 4 : 0, 4),
                      buf(Bu, N * K), buf(su, some ? N * 4 : 0, 4)},
                     {buf(D, M * N * (bf16 ? 2 : 4)), buf(workspace, workspace_bytes)});
  if (st != FP4G_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (!some) return finish(zero(D, M * N, bf16, s));
  const DensePlan p = product_plan(M, N, K, 1, 2, workspace_bytes);
  DenseArgs a;
  a.M = (int)M, a.N = (int)N, a.K = (int)K, a.S = p.S, a.act = act;
  a.A[0] = static_cast<const uint8_t*>(A);
  a.B[0] = static_cast<const uint8_t*>(Bg), a.B[1] = static_cast<const uint8_t*>(Bu);
  a.lda = a.ldb = K, a.sa = sa, a.sb[0] = sg, a.sb[1] = su, a.D[0] = D, a.P = workspace, a.bf16_out = bf16;
  return finish(fp4g::launch_w8a8_gated(a, p.tile, s));
}

fp4g_status gated_gemm_workspace_size(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  return product_workspace(M, N, K, 2, 2, bytes);
}

fp4g_status gated_gemm(int64_t M, int64_t N, int64_t K, const void* X, const void* Wg, const void* Wu, int act, void* H,
                       float* G, float* U, void* workspace, size_t workspace_bytes, void* stream) {
  fp4g_status st = check_sizes(M, N, K, 2);
  if (st != FP4G_OK) return st;
  if (!known_act(act) || !G != !U) return FP4G_EINVAL;
  if (M == 0 || N == 0) return FP4G_OK;
  const int64_t kept = G ? M * N * 4 : 0;
  st = check_buffers({buf(X, M * K * 2), buf(Wg, N * K * 2), buf(Wu, N * K * 2)},
                     {buf(H, M * N * 2), buf(G, kept), buf(U, kept), buf(workspace, workspace_bytes)});
  if (st != FP4G_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (K == 0) {
    hipError_t e = zero(H, M * N, true, s);
    if (e == hipSuccess && G) e = zero(G, M * N, false, s);
    if (e == hipSuccess && G) e = zero(U, M * N, false, s);
    return finish(e);
  }
  const DensePlan p = product_plan(M, N, K, 2, 2, workspace_bytes);
  DenseArgs a;
  a.M = (int)M, a.N = (int)N, a.K = (int)K, a.S = p.S, a.act = act;
  a.A[0] = static_cast<const uint8_t*>(X);
  a.B[0] = static_cast<const uint8_t*>(Wg), a.B[1] = static_cast<const uint8_t*>(Wu);
  a.lda = a.ldb = K * 2, a.D[0] = H, a.G = G, a.U = U, a.P = workspace;
  return finish(fp4g::launch_gated(a, p.tile, s));
}

fp4g_status gated_gemm_backward_workspace_size(int64_t M, int64_t N, int64_t K, size_t* bytes, size_t* least) {
  const fp4g_status st = check_sizes(M, N, K, 2);
  if (st != FP4G_OK) return st;
  if (!bytes || !least) return FP4G_EINVAL;
  const int64_t pitch = grad_pitch(N);
  if (pitch * 2 > kMaxPitch) return FP4G_EUNSUPPORTED;
  *bytes = *least = 0;
  if (M == 0 || N == 0 || K == 0) return FP4G_OK;
  *least = (size_t)(4 * M * pitch);
  const fp4g::GradPlan p = grad_plan(M, N, K, kAnyRoom);
  const size_t x = partial_bytes(M, K, 1, 1, p.x), w = partial_bytes(N, K, 1, 2, p.w);
  *bytes = *least + (x > w ? x : w);
  return FP4G_OK;
}

fp4g_status gated_gemm_backward(int64_t M, int64_t N, int64_t K, const void* dH, const void* X, const void* Wg,
                                const void* Wu, const float* G, const float* U, int act, void* dX, void* dWg,
                                void* dWu, void* workspace, size_t workspace_bytes, void* stream) {
  fp4g_status st = check_sizes(M, N, K, 2);
  if (st != FP4G_OK) return st;
  if (!known_act(act)) return FP4G_EINVAL;
  const int64_t pitch = grad_pitch(N);
  if (pitch * 2 > kMaxPitch) return FP4G_EUNSUPPORTED;
  if (K == 0 || (M == 0 && N == 0)) return FP4G_OK;
  const bool some = M > 0 && N > 0;
  st = check_buffers({buf(dH, M * N * 2, 2), buf(X, some ? M * K * 2 : 0), buf(Wg, some ? N * K * 2 : 0),
                      buf(Wu, some ? N * K * 2 : 0), buf(G, M * N * 4, 4), buf(U, M * N * 4, 4)},
                     {buf(dX, M * K * 2), buf(dWg, N * K * 2), buf(dWu, N * K * 2),
                      buf(workspace, some ? workspace_bytes : 0)});
  if (st != FP4G_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (!some) {
    hipError_t e = zero(dX, M * K, true, s);
    if (e == hipSuccess) e = zero(dWg, N * K, true, s);
    if (e == hipSuccess) e = zero(dWu, N * K, true, s);
    return finish(e);
  }
  const size_t least = (size_t)(4 * M * pitch);
  if (workspace_bytes < least) return FP4G_EINVAL;
  uint8_t* dG = static_cast<uint8_t*>(workspace);
  uint8_t* dU = dG + 2 * M * pitch;
  void* P = dG + least;
  const size_t room = workspace_bytes - least;
  hipError_t e = fp4g::launch_gate_grad(M, N, pitch, dH, G, U, act, dG, dU, s);
  if (e != hipSuccess) return FP4G_EHIP;
  const fp4g::GradPlan p = grad_plan(M, N, K, room);
  DenseArgs x, w;
  x.M = (int)M, x.N = (int)K, x.K = (int)N, x.S = p.x.S;
  x.A[0] = dG, x.A[1] = dU, x.lda = pitch * 2;
  x.B[0] = static_cast<const uint8_t*>(Wg), x.B[1] = static_cast<const uint8_t*>(Wu), x.ldb = K * 2;
  x.D[0] = dX, x.P = P;
  w.M = (int)N, w.N = (int)K, w.K = (int)M, w.L = 2, w.S = p.w.S;
  w.A[0] = dG, w.A[1] = dU, w.lda = pitch * 2;
  w.B[0] = static_cast<const uint8_t*>(X), w.ldb = K * 2;
  w.D[0] = dWg, w.D[1] = dWu, w.P = P;
  return finish(fp4g::launch_grads(x, w, p, s));
}

}  // extern "C"
