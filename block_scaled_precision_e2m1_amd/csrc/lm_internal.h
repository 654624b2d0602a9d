// Internal interface between the entry points of fp4g_lm.h (api_lm.cpp) and their kernel
// launchers.  Arguments reach a launcher only after validation; every launcher enqueues on
// the given stream and returns hipGetLastError().
#pragma once

#include "../../include/fp4g_lm.h"
#include "ffn_internal.h"
#include "internal.h"

namespace fp4g {

struct NormArgs {
  int64_t rows, K;
  const void* X;                  // the type of X, R, H, Y: bf16
  const void* R;                  // null: no residual
  const void* W;                  // null: 1
  void* H;
  void* Y;                        // quantized: may be null
  bool bf16, w_bf16;
  double eps;
  void* codes = nullptr;          // quantized
  float* scales = nullptr;
  bool e4m3 = false;
};
// How many of the rows one launch takes.
int64_t rms_norm_launch_rows(int64_t rows, int64_t K, bool bf16);
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  int64_t rows, K;
  const void* dY;
  const void* X;
  const void* W;                  // null: 1
  const void* dH;                 // null: 0
  void* dX;
  void* dW;                       // null: not wanted
  bool bf16, w_bf16;
  double eps;
  void* P;                        // partial sums of dW
};
// The bytes of P (rows > 0, K > 0).
int64_t rms_norm_grad_bytes(int64_t rows, int64_t K, bool bf16);
hipError_t launch_rms_norm_grad(const NormGradArgs& a, hipStream_t s);

struct LossCall {
  int64_t M, V, K;
  const void *X, *W;
  const int64_t* target;
  int64_t ignore;
  float *loss, *lse;              // lse: may be null; backward: what the forward pass gave
  const float* dL;                // backward
  void *dX, *dW;
  uint8_t* space;
  int64_t cols;                   // backward: columns of a piece
};
// Workspace bytes of the two passes (M, V > 0); backward: with pieces of `cols` columns, and how
// many columns a piece has by choice.
int64_t loss_bytes(int64_t M, int64_t V, int64_t K);
int64_t loss_grad_bytes(int64_t M, int64_t V, int64_t K, int64_t cols);
int64_t loss_grad_cols(int64_t M, int64_t V, int64_t K);
// Whether the forward pass gathers the rows that take part; else its product takes every row.
bool loss_gathers(int64_t M, int64_t V, int64_t K);
// dX's product over a piece of `cols` columns of the vocabulary: its tile and K slices with all M
// rows, and how many slices it may have where fewer rows take part (splits_of).  Never fewer than
// planned: a plan's time is that of its slices, and its partial sums are paid for with any number.
// More only of 8 stages or longer.
struct LossInputPlan { DensePlan plan; int most; };
LossInputPlan loss_input_plan(int64_t M, int64_t K, int64_t cols);
hipError_t launch_loss(const LossCall& a, hipStream_t s);
hipError_t launch_loss_grad(const LossCall& a, hipStream_t s);

struct AdapterCall {
  int64_t M, N, K, R, L;          // M, N > 0; K and R multiples of 8, R <= 256, L <= kMaxAdapters
  const void *base, *X, *A, *B;
  const float* scales;            // null: 1
  const int* index;
  void* D;
  bool bf16;                      // the type of base and D
  uint8_t* space;
};
constexpr int64_t kMaxAdapters = 8192;   // counted in a workgroup's LDS
int64_t adapter_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L);
hipError_t launch_adapter_gemm(const AdapterCall& c, hipStream_t s);

}  // namespace fp4g
