// The elementwise step of the gated block's backward pass for gfx950: from dH (bf16) and the
// kept fp32 products G and U,
//   dG = dH * U * act'(G),   dU = dH * act(G),
// rounded once to bf16, the operands of the gradients' products.  Rows are `pitch` elements
// apart (a multiple of 64) with zeros past N, so the products' K stages of dX are whole and
// every operand row is 16-byte aligned whatever N is.
//
// The rounding is a choice.  fp32 matrix instructions run at a sixteenth of bf16's rate, and
// two bf16 numbers for each of dG and dU would double both products, 3 of the 5 ms of a
// training step of 8192 x 14336 x 4096.  It adds as much error as the rounding of the results
// does: dX, dWg and dWu are off by 0.00235 of their norm, with dG and dU left in fp32 by
// 0.00166 (301 x 1003 x 520 gelu and 1024 x 4096 x 1024 silu, all six gradients).
//
// HBM-bound: 14 bytes an element (2 + 4 + 4 read, 2 + 2 written); 8192 x 14336 takes 310 us,
// 5.3 TB/s.  A lane takes 8 columns of a row: one 16-byte load of dH, two each of G and U
// (past the caches: nothing reads them again; 345 us with plain loads), two 16-byte stores.  With
// 4 columns a lane it takes 335 us, and 301 x 1003 the same 5.4 us.  The loads take
// rows of any length, whose groups start at any element (the hardware takes unaligned vector
// loads); only the group that holds a row's end is read element by element.
#include <algorithm>

#include "dense.hpp"
#include "launch.hpp"

namespace fp4g {
namespace {

__global__ void __launch_bounds__(256)
gate_grad_kernel(int64_t M, int N, int pitch, const uint16_t* __restrict__ dH, const float* __restrict__ G,
                 const float* __restrict__ U, int act, uint8_t* __restrict__ dG, uint8_t* __restrict__ dU) {
  typedef v4i v4i_any __attribute__((aligned(2)));
  typedef v4f v4f_any __attribute__((aligned(4)));
  const int groups = pitch / 8;
  const int64_t total = M * groups;
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < total; x += (int64_t)gridDim.x * 256) {
    // 32-bit division where it will do: the 64-bit one is a hundred instructions.
    const int64_t m = total <= UINT32_MAX ? (uint32_t)x / (uint32_t)groups : x / groups;
    const int n = (int)(x - m * groups) * 8;
    const int64_t at = m * N + n;
    float h[8], g[8], u[8];
    if (n + 8 <= N) {
      const v4i w = __builtin_nontemporal_load(reinterpret_cast<const v4i_any*>(dH + at));
      const v4f_any *gp = reinterpret_cast<const v4f_any*>(G + at), *up = reinterpret_cast<const v4f_any*>(U + at);
      const v4f g0 = __builtin_nontemporal_load(gp), g1 = __builtin_nontemporal_load(gp + 1);
      const v4f u0 = __builtin_nontemporal_load(up), u1 = __builtin_nontemporal_load(up + 1);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[e] = __builtin_bit_cast(float, e & 1 ? (uint32_t)w[e / 2] & 0xffff0000u : (uint32_t)w[e / 2] << 16);
        g[e] = e < 4 ? g0[e & 3] : g1[e & 3];
        u[e] = e < 4 ? u0[e & 3] : u1[e & 3];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool in = n + e < N;
        h[e] = in ? __builtin_bit_cast(float, (uint32_t)dH[at + e] << 16) : 0.0f;
        g[e] = in ? G[at + e] : 0.0f;
        u[e] = in ? U[at + e] : 0.0f;
      }
    }
    uint32_t wg[4], wu[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      float a0, d0, a1, d1;
      act_grad(act, g[e], &a0, &d0);
      act_grad(act, g[e + 1], &a1, &d1);
      wg[e / 2] = pack_bf16x2(h[e] * u[e] * d0, h[e + 1] * u[e + 1] * d1);
      wu[e / 2] = pack_bf16x2(h[e] * a0, h[e + 1] * a1);
    }
    const int64_t to = (m * pitch + n) * 2;
    *reinterpret_cast<v4i*>(dG + to) = v4i{(int)wg[0], (int)wg[1], (int)wg[2], (int)wg[3]};
    *reinterpret_cast<v4i*>(dU + to) = v4i{(int)wu[0], (int)wu[1], (int)wu[2], (int)wu[3]};
  }
}

}  // namespace

hipError_t launch_gate_grad(int64_t M, int64_t N, int64_t pitch, const void* dH, const float* G, const float* U, int act,
                            void* dG, void* dU, hipStream_t s) {
  const int64_t units = ceil_div(M * (pitch / 8), 256);
  const unsigned grid = (unsigned)std::min<int64_t>(units, device_cus() * 16);
  return launch(gate_grad_kernel, grid, 256, s, M, (int)N, (int)pitch, static_cast<const uint16_t*>(dH), G, U, act,
                static_cast<uint8_t*>(dG), static_cast<uint8_t*>(dU));
}

}  // namespace fp4g
