/*
 * fp4g_ffn.h -- C ABI of the feed-forward operators of libfp4gemm.so for AMD Instinct
 * MI355X (gfx950): int8 quantization of activations, int8 products, and the gated product
 * of a transformer's feed-forward block in int8 and bf16, with its backward pass.
 *
 * Conventions are those of fp4gemm.h: plain device pointers owned by the caller, row-major
 * buffers without padding, calls asynchronous on `stream` (a hipStream_t; NULL is the
 * default stream), no allocation, arguments validated on the host before anything is
 * launched, statuses of fp4g_status.  Only kernels are enqueued, so calls may be captured.
 *
 * Sizes (all entry points): each dimension >= 0 and below 2^31 and each buffer of at most
 * 2^50 elements (FP4G_EINVAL otherwise).  Operand rows are read 16 bytes at a time: int8
 * rows hold a multiple of 16 elements, bf16 rows a multiple of 8 (FP4G_EUNSUPPORTED
 * otherwise), at most 2^22 bytes.  Operands, the quantizer's input and outputs are 16-byte
 * aligned; scales, and the backward pass's dH, G and U, are aligned to their elements
 * (FP4G_EALIGN otherwise).  Outputs overlap neither an input nor each other.
 *
 * Workspaces: the products split K when their tiles cannot fill the GPU and `workspace`
 * (16-byte aligned, workspace_bytes long) has room for the partial sums.  The
 * *_workspace_size queries give what a call can use on the current device; NULL with 0
 * bytes, or fewer bytes, means a smaller split or none.  Workspaces need no clearing and
 * hold nothing between calls.
 */
#ifndef FP4G_FFN_H
#define FP4G_FFN_H

#include "fp4gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The activation of a gated product, taken as `int act` and validated (FP4G_EINVAL):
 *   FP4G_ACT_SILU       x / (1 + e^-x)
 *   FP4G_ACT_GELU       x (1 + erf(x / sqrt 2)) / 2
 *   FP4G_ACT_GELU_TANH  x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) / 2 */
typedef enum {
    FP4G_ACT_SILU = 0,
    FP4G_ACT_GELU = 1,
    FP4G_ACT_GELU_TANH = 2
} fp4g_act;

/* Row quantizer: X[rows][K] (fp32 or bf16 by x_type, fp4gemm.h) -> int8 codes[rows][K] and
 * fp32 scales[rows], every step in IEEE fp32:
 *   scale = max|x| / 127,  inv = min(1 / scale, FLT_MAX),
 *   code  = x * inv rounded to the nearest integer, ties to even, clamped to +-127.
 * A row of zeros has scale 0 and zero codes; a row holding an infinity or NaN has a NaN
 * scale and zero codes.  K a multiple of 16.  rows == 0 is a no-op; K == 0 writes scales 0. */
fp4g_status int8_quantize(int64_t rows, int64_t K, const void *X, int x_type,
                          void *codes, float *scales, void *stream);

/* D[m][n] = (sum_k A[m][k] B[n][k]) * sa[m] * sb[n] for int8 A[M][K], B[N][K] and fp32
 * scales; D fp32 or bf16 by d_type.  The sums are exact (32-bit integers: K at most
 * 131056, FP4G_EUNSUPPORTED otherwise), and each result is the sum rounded to fp32, two
 * fp32 products and, for bf16, one more rounding.  K a multiple of 16; K == 0 zeroes D. */
fp4g_status w8a8_gemm_workspace_size(int64_t M, int64_t N, int64_t K, size_t *bytes);
fp4g_status w8a8_gemm(int64_t M, int64_t N, int64_t K,
                      const void *A, const float *sa, const void *B, const float *sb,
                      void *D, int d_type, void *workspace, size_t workspace_bytes, void *stream);

/* D[m][n] = act(g) * u with g and u the scaled products (as above) of A with the gate's
 * weights Bg[N][K], sg[N] and with the factor's Bu[N][K], su[N]. */
fp4g_status w8a8_gated_gemm_workspace_size(int64_t M, int64_t N, int64_t K, size_t *bytes);
fp4g_status w8a8_gated_gemm(int64_t M, int64_t N, int64_t K,
                            const void *A, const float *sa,
                            const void *Bg, const float *sg, const void *Bu, const float *su,
                            int act, void *D, int d_type,
                            void *workspace, size_t workspace_bytes, void *stream);

/* The gated product of bf16 X[M][K], Wg[N][K], Wu[N][K]: G = X Wg^T and U = X Wu^T with
 * fp32 sums, H[M][N] = act(G) * U in fp32, rounded once to bf16.  G and U (fp32 [M][N]) are
 * written too where both pointers are given, for gated_gemm_backward; one of the two alone
 * is FP4G_EINVAL.  K a multiple of 8; K == 0 zeroes the outputs. */
fp4g_status gated_gemm_workspace_size(int64_t M, int64_t N, int64_t K, size_t *bytes);
fp4g_status gated_gemm(int64_t M, int64_t N, int64_t K,
                       const void *X, const void *Wg, const void *Wu, int act,
                       void *H, float *G, float *U,
                       void *workspace, size_t workspace_bytes, void *stream);

/* The gradients of gated_gemm, from the incoming bf16 dH[M][N], its inputs and its kept G
 * and U, all outputs bf16:
 *   dG = dH U act'(G),  dU = dH act(G)      computed in fp32, rounded to bf16 once
 *   dX[M][K] = dG Wg + dU Wu,  dWg[N][K] = dG^T X,  dWu[N][K] = dU^T X   with fp32 sums
 * The workspace is required: gated_gemm_backward_workspace_size gives `bytes`, which lets
 * the products split, and `least`, what dG and dU take (fewer is FP4G_EINVAL).  Where M
 * (for dWg, dWu) or N (for dX) is 0 those gradients are zeroed.  N is at most 2^21: rows of dG
 * and dU are operands too (FP4G_EUNSUPPORTED otherwise, from the query as well; gated_gemm
 * itself takes any N). */
fp4g_status gated_gemm_backward_workspace_size(int64_t M, int64_t N, int64_t K, size_t *bytes, size_t *least);
fp4g_status gated_gemm_backward(int64_t M, int64_t N, int64_t K,
                                const void *dH, const void *X, const void *Wg, const void *Wu,
                                const float *G, const float *U, int act,
                                void *dX, void *dWg, void *dWu,
                                void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP4G_FFN_H */
