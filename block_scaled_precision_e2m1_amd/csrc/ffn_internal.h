// Internal interface between the feed-forward entry points (api_ffn.cpp) and their kernel
// launchers.  Arguments reach a launcher only after validation; every launcher enqueues on
// the given stream and returns hipGetLastError().
#pragma once

#include "../../include/fp4g_ffn.h"
#include "internal.h"

namespace fp4g {

// One product of the tile kernels (dense_gemm.hip).
struct DenseArgs {
  int M = 0, N = 0;            // rows and columns of each output
  int K = 0;                   // contraction length of one segment, in elements
  int L = 1;                   // products that share B: A[l] and D[l] are their own
  int S = 1;                   // K slices (partial sums go to P when S > 1)
  const uint8_t* A[2] = {nullptr, nullptr};   // dX: one for each segment; dW: one for each product
  const uint8_t* B[2] = {nullptr, nullptr};   // gated: the gate's and the factor's weights; dX: segments
  int64_t lda = 0, ldb = 0;                   // bytes between rows
  const float* sa = nullptr;                  // int8: a scale for each row of A and of B
  const float* sb[2] = {nullptr, nullptr};
  void* D[2] = {nullptr, nullptr};
  float* G = nullptr;                         // gated: both products, where they are kept
  float* U = nullptr;
  void* P = nullptr;                          // [L][S][gates][M][partial_pitch(N)] 32-bit partial sums
  int act = 0;
  bool bf16_out = true;                       // the type of D
};

// Rows of partial sums are whole groups of 4.
inline
#if defined(__HIPCC__)
__host__ __device__
#endif
int64_t partial_pitch(int64_t N) { return (N + 3) / 4 * 4; }

enum DenseTile {
  kTile256, kTile128, kTile128Deep, kTile64x128, kTile64Deep, kTile64, kTile64x128Long, kTile64Long, kGemv
};
struct DensePlan { DenseTile tile; int S; double us; };   // us: the modelled time
struct GradPlan { DensePlan x, w; bool merged; };         // dX; dWg and dWu; in one launch

// Tile and K split for L products of rows x cols sums (gated: cols counts both weights'
// columns) over KT stages of 128 bytes of K; at most `cap` slices.
DensePlan dense_plan(int64_t rows, int64_t cols, int64_t L, int64_t KT, int64_t cap);

// Whether a product of M tokens with `gates` weights of N rows of KB bytes goes to the kernels
// for few tokens (dense_gemv.hip), and its K split there, of at most `cap` slices.
bool gemv_takes(int64_t M, int64_t N, int64_t KB, int64_t gates);
int gemv_splits(int64_t M, int64_t N, int64_t KB, int64_t gates, int64_t cap);

hipError_t launch_w8a8(const DenseArgs& a, DenseTile tile, hipStream_t s);
hipError_t launch_w8a8_gated(const DenseArgs& a, DenseTile tile, hipStream_t s);
hipError_t launch_gated(const DenseArgs& a, DenseTile tile, hipStream_t s);
hipError_t launch_gemv_w8a8(const DenseArgs& a, hipStream_t s);
hipError_t launch_gemv_w8a8_gated(const DenseArgs& a, hipStream_t s);
hipError_t launch_gemv_gated(const DenseArgs& a, hipStream_t s);
// Adds the slices of a.P and finishes the product.
hipError_t launch_partial_sums(const DenseArgs& a, bool int8, bool gated, hipStream_t s);
// The backward products of an M x N gated product of K inputs, at most cap_x and cap_w slices.
GradPlan grad_plan(int64_t M, int64_t N, int64_t K, int64_t cap_x, int64_t cap_w);
hipError_t launch_grads(const DenseArgs& x, const DenseArgs& w, const GradPlan& p, hipStream_t s);

// dG = dH U act'(G), dU = dH act(G) as bf16 rows of `pitch` elements, zero past N.
hipError_t launch_gate_grad(int64_t M, int64_t N, int64_t pitch, const void* dH, const float* G, const float* U, int act,
                            void* dG, void* dU, hipStream_t s);

hipError_t launch_int8_quantize(int64_t rows, int64_t K, const void* X, bool bf16_in, void* codes, float* scales,
                                hipStream_t s);

}  // namespace fp4g
