// Pieces shared by the unscaled-operand kernels (int8 and bf16 products, gated feed-forward
// products and their gradients).
//
// Operand tiles reach LDS by buffer_load_dwordx4 ... lds through a raw buffer resource
// whose size ends at the last valid byte of the tile: a lane past it (rows past M, K past
// the end of a row, stages past the end of a slice) moves nothing from memory and writes
// zeros to LDS, so ragged sizes need no masks in the product and no copy can leave its
// operand.  A lane that must not load (the K tail of a row whose next bytes belong to the
// next row) is given the offset kNoLoad, past the end of every resource.
#pragma once

#include "common.hpp"
#include "ffn_internal.h"

namespace fp4g {

typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));

constexpr uint32_t kNoLoad = 0x80000000u;   // resources hold less than 2^31 bytes

// The element types of the operands.
struct I8 { static constexpr int BYTES = 1; typedef v16i acc32; typedef v4i acc16; };
struct BF { static constexpr int BYTES = 2; typedef v16f acc32; typedef v4f acc16; };

// A raw buffer of `bytes` bytes at p (clamped to be non-negative); p and bytes must be
// wave-uniform.  LDS copies of 16 bytes per lane from it: lane i of the wave fetches
// p + off and writes 16 bytes at l + 16 * i.
#if defined(__HIP_DEVICE_COMPILE__)
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes > 0 ? bytes : 0, 0x00020000);
}
__device__ __forceinline__ void lds_buffer16(rsrc_t r, lds_void* l, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, off, 0, 0, 0);
}
// As lds_buffer16, with the nontemporal policy, for data read once.
__device__ __forceinline__ void lds_buffer16_nt(rsrc_t r, lds_void* l, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, l, 16, off, 0, 0, 2);
}
// 16 bytes a lane into registers, zeros past the end.
__device__ __forceinline__ v4i load_buffer16(rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
// __restrict__ matters: the alias scope it leaves on the inlined read is what tells the compiler
// that the read needs no wait of its own for the copies in flight.  Without one it puts
// vmcnt(0) before every read of this kind, which drains the ring: the two products of the
// backward pass at 8192 x 14336 x 4096 took 4317 and 6238 us with those waits, 1440 and
// 1540 us without.  The waits that the ring needs are the kernel's own.
__device__ __forceinline__ v2i lds_read_tr16(const uint8_t* __restrict__ p) {
  return __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                     (__attribute__((address_space(3))) v4s*)p));
}
#else
struct rsrc_t {};
__device__ __forceinline__ rsrc_t make_rsrc(const void*, int) { return {}; }
__device__ __forceinline__ void lds_buffer16(rsrc_t, lds_void*, uint32_t) {}
__device__ __forceinline__ void lds_buffer16_nt(rsrc_t, lds_void*, uint32_t) {}
__device__ __forceinline__ v4i load_buffer16(rsrc_t, uint32_t) { return {}; }
__device__ __forceinline__ v2i lds_read_tr16(const uint8_t*) { return {}; }
#endif

// 32x32 products of 16 bytes of K per lane (32 int8 or 16 bf16 K elements per instruction),
// and 16x16 products of 16 bytes per lane (64 or 32 K elements).  Lane l holds row l % R of
// its operand in K slot l / R; equal slots of the two operands meet.
__device__ __forceinline__ v16i mfma32(v4i a, v4i b, v16i c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
#else
  return c;
#endif
}
__device__ __forceinline__ v16f mfma32(v4i a, v4i b, v16f c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
#else
  return c;
#endif
}
__device__ __forceinline__ v4i mfma16(v4i a, v4i b, v4i c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
#else
  return c;
#endif
}
__device__ __forceinline__ v4f mfma16(v4i a, v4i b, v4f c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
#else
  return c;
#endif
}

// The activations of a gated block, in fp32.  With s(z) = 1 / (1 + e^-z):
//   silu       x s(x)
//   gelu       x erfc(-x / sqrt 2) / 2, which is x (1 + erf(x / sqrt 2)) / 2
//   gelu_tanh  x s(2 sqrt(2/pi) (x + 0.044715 x^3)), which is x (1 + tanh(..)) / 2
// With e = e^-|z|, s(z) is 1 / (1 + e) for z >= 0 and e / (1 + e) below.  e is taken as the
// square of e^(-|z|/2), whose two factors stay normal where e does not, and multiplies x in two
// steps: x s(z) is a normal number down to z = -92, s itself only down to -87.
// e^(-|z|/2) is one hardware 2^x of an fp32 product and the quotient one hardware reciprocal, so
// the relative error of s and of x s is a few fp32 half steps (2^-24) for |z| < 2 and grows like
// |z| from the rounding of the exponent: silu is off by 59 half steps at most in -60 .. -30 and
// 111 at -92; gelu_tanh, whose z is rounded four times more, by 208 at x = -9 (z = -69).  That
// is 2e-5 at worst, far below a bf16 half step of 4e-3.
// gelu's left tail is erfc's, where 1 + erf would cancel (4% off at x = -5, zero from -5.5 on);
// the rounding of erfc's argument makes its error grow like x^2: 18 half steps at most in -4 ..
// -2, 48 in -6 .. -5, 211 at -13.  The derivative's e^(-x^2/2) is a square as well.
// The cubic is evaluated at |x| <= 32, where s has long been 0 or 1: a larger x would overflow
// it and make 0 * inf of the derivative.
struct Sigmoid { float h, r, q; };    // s(z) = h h r, 1 - s(z) = q
__device__ __forceinline__ Sigmoid sigmoid(float z) {
  const float f = __builtin_amdgcn_exp2f(__builtin_fabsf(z) * -0.72134752044448170f);   // log2(e) / 2
  const float e = f * f, r = __builtin_amdgcn_rcpf(1.0f + e);
  return Sigmoid{z < 0.0f ? f : 1.0f, r, z < 0.0f ? r : e * r};
}
__device__ __forceinline__ float cubic_arg(float x, float* slope) {
  constexpr float c = 1.5957691216057308f, q = 0.044715f;       // 2 sqrt(2/pi)
  const float t = __builtin_amdgcn_fmed3f(x, -32.0f, 32.0f), t2 = t * t;
  *slope = c * (1.0f + 3.0f * q * t2);
  return c * t * (1.0f + q * t2);
}
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(x * -0.70710678118654752f); }
__device__ __forceinline__ float act_of(int act, float x) {
  if (act == FP4G_ACT_GELU) return x * normal_cdf(x);
  float z = x, slope;
  if (act == FP4G_ACT_GELU_TANH) z = cubic_arg(x, &slope);
  const Sigmoid s = sigmoid(z);
  return x * s.h * s.r * s.h;
}
// act(x) and its derivative.
__device__ __forceinline__ void act_grad(int act, float x, float* a, float* da) {
  if (act == FP4G_ACT_GELU) {
    const float cdf = normal_cdf(x);
    const float t = __builtin_amdgcn_fmed3f(x, -32.0f, 32.0f);
    const float f = __builtin_amdgcn_exp2f(t * t * -0.36067376022224085f);   // e^(-t^2/4): log2(e) / 4
    *a = x * cdf;
    *da = cdf + t * 0.3989422804014327f * f * f;
    return;
  }
  float z = x, slope = 1.0f;
  if (act == FP4G_ACT_GELU_TANH) z = cubic_arg(x, &slope);
  const Sigmoid s = sigmoid(z);
  const float xh = x * s.h;
  *a = xh * s.r * s.h;
  *da = (s.h + xh * s.q * slope) * s.r * s.h;   // s + x s (1 - s) z'
}

// y = act(y) * u; the activation is uniform, so one of the three loops runs.
template <int V>
__device__ __forceinline__ void gate(int act, float (&y)[V], const float (&u)[V]) {
  if (act == FP4G_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = act_of(FP4G_ACT_SILU, y[e]) * u[e];
  } else if (act == FP4G_ACT_GELU) {
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = act_of(FP4G_ACT_GELU, y[e]) * u[e];
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = act_of(FP4G_ACT_GELU_TANH, y[e]) * u[e];
  }
}

// V results to D[at ..], of which the first `left` exist.  A whole group is one vector store
// at any alignment: rows of an odd length start anywhere, and the hardware splits only the
// stores that cross a line.
// NT (fp32): past the caches.
template <bool BF16, bool NT = false, int V>
__device__ __forceinline__ void store_cols(void* D, int64_t at, int left, const float (&y)[V]) {
  static_assert(V == 4 || (V == 8 && BF16), "16 bytes at most");
  typedef v4i v4i_any __attribute__((aligned(2)));
  typedef v2i v2i_any __attribute__((aligned(2)));
  typedef v4f v4f_any __attribute__((aligned(4)));
  if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(D) + at;
    uint32_t w[V / 2];
#pragma unroll
    for (int e = 0; e < V; e += 2) w[e / 2] = pack_bf16x2(y[e], y[e + 1]);
    if (left >= V) {
      if constexpr (V == 8) *reinterpret_cast<v4i_any*>(p) = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
      else *reinterpret_cast<v2i_any*>(p) = v2i{(int)w[0], (int)w[1]};
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < left) p[e] = (uint16_t)(e & 1 ? w[e / 2] >> 16 : w[e / 2]);
    }
  } else {
    float* p = static_cast<float*>(D) + at;
    if (left >= V) {
      const v4f v{y[0], y[1], y[2], y[3]};
      if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<v4f_any*>(p));
      else *reinterpret_cast<v4f_any*>(p) = v;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < left) p[e] = y[e];
    }
  }
}

}  // namespace fp4g
