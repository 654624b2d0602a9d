// Internal interface between the entry points of fp4g_lm.h (api_lm.cpp) and their kernel
// launchers.  Arguments reach a launcher only after validation; every launcher enqueues on
// the given stream and returns hipGetLastError().
#pragma once

#include "../../include/fp4g_lm.h"
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

}  // namespace fp4g
