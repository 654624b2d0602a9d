/*
 * fp4g_lm.h -- C ABI of the operators that stand around a language model's products in
 * libfp4gemm.so for AMD Instinct MI355X (gfx950): the root-mean-square norm with its 8-bit
 * outputs and its backward pass, the cross entropy over a vocabulary with its backward pass,
 * and low-rank adapters beside a shared projection.
 *
 * Conventions are those of fp4gemm.h: plain device pointers owned by the caller, row-major
 * buffers without padding, calls asynchronous on `stream` (a hipStream_t; NULL is the
 * default stream), no allocation, arguments validated on the host before anything is
 * launched, statuses of fp4g_status.  Only kernels are enqueued, so calls may be captured.
 * Results repeat bit for bit: every sum has a fixed order.
 *
 * Sizes (all entry points): each dimension >= 0 and below 2^31 and each buffer of at most
 * 2^50 elements (FP4G_EINVAL otherwise).  Workspaces are 16-byte aligned, need no clearing
 * and hold nothing between calls; the *_workspace_size queries give their sizes on the
 * current device.  Two calls that may run at once need a workspace each.  Outputs overlap
 * neither an input nor each other, but for the cases named below.
 */
#ifndef FP4G_LM_H
#define FP4G_LM_H

#include "fp4gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The codes of rms_norm_quantize, taken as `int code_type` and validated (FP4G_EINVAL):
 * what w8a8_gemm and w4a8_gemm take as activations. */
typedef enum {
    FP4G_CODE_INT8 = 0,
    FP4G_CODE_E4M3 = 1
} fp4g_code_type;

/* The root-mean-square norm of each row:
 *   h = x, or x + r rounded to their type where R is given,
 *   Y = (h * s) * w,  s = 1 / sqrt(mean(h^2) + eps),
 * with the mean in 64 bits, s rounded to fp32, both products in fp32 and one rounding to Y's
 * type.  X, R, H and Y [rows][K] are all fp32 or all bf16 by x_type; W [K] is fp32 or bf16
 * by w_type, or NULL (w = 1).  H is written where R is given (both or neither,
 * FP4G_EINVAL).  eps is finite and not negative (FP4G_EINVAL); with eps == 0 a row of zeros
 * gives NaN, as the formula does.  Any K; K == 0 is a no-op.  Buffers are aligned to their
 * elements (FP4G_EALIGN).  H may be X or R itself, and Y may be X or R itself, but not both
 * the same one. */
fp4g_status rms_norm(int64_t rows, int64_t K, const void *X, int x_type, const void *R,
                     const void *W, int w_type, double eps, void *H, void *Y, void *stream);

/* The same norm quantized by rows: with y the fp32 products above, before any rounding to
 * Y's type, and T = 127 (int8) or 448 (E4M3), every step in IEEE fp32:
 *   scale = max|y| / T,  inv = min(1 / scale, FLT_MAX),
 *   code  = y * inv rounded to the nearest code, ties to even, clamped to +-T.
 * A row of zeros has scale 0 and zero codes; a row whose y hold an infinity or NaN has a NaN
 * scale and zero codes.  codes [rows][K] are int8 or E4M3 bytes by code_type, scales [rows]
 * fp32.  Y may be NULL: it is not written then.  K == 0 writes scales 0. */
fp4g_status rms_norm_quantize(int64_t rows, int64_t K, const void *X, int x_type, const void *R,
                              const void *W, int w_type, double eps, void *H, void *Y,
                              void *codes, int code_type, float *scales, void *stream);

/* The gradients of rms_norm in X (and in R, which has the same) and in W, from the incoming
 * dY and, where it is not NULL, dH [rows][K], with X the rows that were normed (rms_norm's H
 * where it added a residual), g = dY * w and n = x * s, in fp32 with one rounding each:
 *   dX = s * (g - n * mean(g * n)) + dH,   dW = sum over rows of dY * n.
 * mean(g * n) is s times the mean of g * x, whose sum has to be an fp32 number: it is for rows
 * of up to about 1e33.  dY, dH and dX have X's type, dW has W's.  dW may be NULL and has to be
 * where W is (FP4G_EINVAL).  dX may be dY or dH itself.  The workspace is required (fewer
 * bytes than the query's are FP4G_EINVAL): it holds dW's partial sums.  rows == 0 zeroes dW. */
fp4g_status rms_norm_backward_workspace_size(int64_t rows, int64_t K, int x_type, size_t *bytes);
fp4g_status rms_norm_backward(int64_t rows, int64_t K, const void *dY, const void *X, int x_type,
                              const void *W, int w_type, double eps, const void *dH,
                              void *dX, void *dW, void *workspace, size_t workspace_bytes,
                              void *stream);

/* The softmax cross entropy of bf16 X[M][K] against the vocabulary's bf16 W[V][K], a target
 * token for each row, without the logits z = X W^T in memory:
 *   lse[m] = log sum_v e^z[m][v],   loss[m] = lse[m] - z[m][target[m]],
 * logits with fp32 sums, exponentials of their differences from a row's largest and the sums
 * of these in fp32: no loss is negative.  loss and lse are fp32 [M]; lse may be NULL.  Rows
 * whose target is ignore_index take no part: their loss and lse are 0, and what their X holds
 * reaches no result, though it may be read.  Any other target outside 0 .. V-1 gives a NaN loss.  target is
 * int64 [M].  V >= 1 where M > 0 (FP4G_EINVAL); K a multiple of 8 and at most 2^21, M at most
 * 2^25 (FP4G_EUNSUPPORTED).  X and W are 16-byte aligned, the others aligned to their elements
 * (FP4G_EALIGN).  The workspace is required (fewer bytes than the query's are FP4G_EINVAL). */
fp4g_status cross_entropy_gemm_workspace_size(int64_t M, int64_t V, int64_t K, size_t *bytes);
fp4g_status cross_entropy_gemm(int64_t M, int64_t V, int64_t K, const void *X, const void *W,
                               const int64_t *target, int64_t ignore_index,
                               float *loss, float *lse,
                               void *workspace, size_t workspace_bytes, void *stream);

/* The gradients of cross_entropy_gemm from the incoming fp32 dL[M] and the lse it gave, both
 * bf16:  P = (e^(z - lse) - [v == target]) * dL in fp32, rounded to bf16 once (where at most 128
 * rows take part to two bf16 terms, which keep 16 bits; for that the dL of all rows are
 * divided by one number of 1 to 2, and the products multiplied by it),
 *   dX[M][K] = P W,   dW[V][K] = P^T X   with fp32 sums.
 * P is formed for a piece of the vocabulary at a time, in the workspace: the query gives
 * `bytes`, with which pieces are large enough to fill the GPU, and `least`, the least a call
 * takes (fewer is FP4G_EINVAL).  Rows whose target is ignore_index have dX = 0 and give dW
 * nothing, whatever their X and dL hold; a row with another target outside 0 .. V-1 makes its
 * dX, and dW, NaN.  dX or dW may be NULL where it is not wanted: its product is left out.
 * M == 0 zeroes dW. */
fp4g_status cross_entropy_gemm_backward_workspace_size(int64_t M, int64_t V, int64_t K,
                                                       size_t *bytes, size_t *least);
fp4g_status cross_entropy_gemm_backward(int64_t M, int64_t V, int64_t K, const float *dL,
                                        const void *X, const void *W, const int64_t *target,
                                        int64_t ignore_index, const float *lse,
                                        void *dX, void *dW,
                                        void *workspace, size_t workspace_bytes, void *stream);

/* Low-rank adapters of many requests, beside a projection that they share and that has given
 * base[M][N]: with i = index[m],
 *   D[m] = base[m] + scales[i] * B[i] (A[i] X[m])
 * for bf16 X[M][K], A[L][R][K], B[L][N][R] and fp32 scales[L] (NULL: 1).  Sums and the R
 * values between the products are fp32 (these enter the second product as bf16 terms that add
 * up to them: two, which keep 16 bits, for bf16 results, and three, which keep all, for
 * fp32); base and D are fp32 or bf16 by d_type, rounded once.  A row
 * whose index is outside 0 .. L-1 has no adapter: D[m] = base[m], and its X is not looked at.
 * D may be base itself.  K and R are multiples of 8, R at most 256, K at most 2^21, L at most
 * 8192, M at most 2^25, N at most 2^30 (FP4G_EUNSUPPORTED).  X, A and B are 16-byte aligned,
 * the others aligned to their elements (FP4G_EALIGN).  The workspace is required (fewer
 * bytes than the query's are FP4G_EINVAL). */
fp4g_status adapter_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L,
                                        size_t *bytes);
fp4g_status adapter_gemm(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L,
                         const void *base, const void *X, const void *A, const void *B,
                         const float *scales, const int32_t *index, void *D, int d_type,
                         void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP4G_LM_H */
