// Rows in registers: what the norm's kernels share.
//
// A row of K elements is walked in units of 16 bytes, L lanes a row and C units a lane, unit
// u = lane + c * L.  Rows start at any element (odd K), so units are read and written as
// unaligned vectors, which cost nothing where they happen to be aligned; the last unit of a
// row may be short and goes element by element.
#pragma once

#include "common.hpp"
#include "lm_internal.h"

namespace fp4g {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));

typedef v4u v4u_at2 __attribute__((aligned(2)));
typedef v4u v4u_at4 __attribute__((aligned(4)));

template <bool BF16> struct Unit {
  typedef typename std::conditional<BF16, v4u_at2, v4u_at4>::type any;
  static constexpr int EPU = BF16 ? 8 : 4, ELEM = BF16 ? 2 : 4;
  __device__ static __forceinline__ float at(const v4u& w, int e) {
    if constexpr (BF16) return __builtin_bit_cast(float, e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    const uint32_t bits = w[e];   // a value: the cast of the element itself reads element 0
    return __builtin_bit_cast(float, bits);
  }
  __device__ static __forceinline__ v4u pack(const float (&y)[EPU]) {
    v4u r;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if constexpr (BF16) r[w] = pack_bf16x2(y[2 * w], y[2 * w + 1]);
      else r[w] = __builtin_bit_cast(uint32_t, y[w]);
    }
    return r;
  }
  // Elements first .. first + EPU - 1 of a row of K at p; zeros past its end.
  template <bool NT = false>
  __device__ static __forceinline__ v4u load(const void* p, int64_t first, int64_t K) {
    const uint8_t* q = static_cast<const uint8_t*>(p) + first * ELEM;
    if (first + EPU <= K) {
      if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const any*>(q));
      return *reinterpret_cast<const any*>(q);
    }
    v4u r{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < EPU; ++e)
      if (first + e < K) {
        if constexpr (BF16) r[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(q)[e] << (e & 1 ? 16 : 0);
        else r[e] = reinterpret_cast<const uint32_t*>(q)[e];
      }
    return r;
  }
  __device__ static __forceinline__ void store(void* p, int64_t first, int64_t K, const v4u& v) {
    uint8_t* q = static_cast<uint8_t*>(p) + first * ELEM;
    if (first + EPU <= K) {
      *reinterpret_cast<any*>(q) = v;
    } else {
#pragma unroll
      for (int e = 0; e < EPU; ++e)
        if (first + e < K) {
          if constexpr (BF16) reinterpret_cast<uint16_t*>(q)[e] = (uint16_t)(e & 1 ? v[e / 2] >> 16 : v[e / 2]);
          else reinterpret_cast<uint32_t*>(q)[e] = v[e];
        }
    }
  }
};

// N elements of the weight from `first`, 1 where there is none and 0 past the end.
template <bool BF16, int N>
__device__ __forceinline__ void load_weight(const void* W, int64_t first, int64_t K, float (&w)[N]) {
  constexpr int EPU = Unit<BF16>::EPU;
  if (!W) {
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = 1.0f;
  } else if constexpr (EPU <= N) {
#pragma unroll
    for (int c = 0; c < N / EPU; ++c) {
      const v4u v = Unit<BF16>::load(W, first + c * EPU, K);
#pragma unroll
      for (int e = 0; e < EPU; ++e) w[c * EPU + e] = Unit<BF16>::at(v, e);
    }
  } else {   // four bf16 weights for four fp32 elements
    typedef v2u any __attribute__((aligned(2)));
    const uint16_t* q = static_cast<const uint16_t*>(W) + first;
    v2u v{0, 0};
    if (first + N <= K) {
      v = *reinterpret_cast<const any*>(q);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (first + e < K) v[e / 2] |= (uint32_t)q[e] << (e & 1 ? 16 : 0);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = __builtin_bit_cast(float, e & 1 ? v[e / 2] & 0xffff0000u : v[e / 2] << 16);
  }
}

struct Add {
  template <class T> __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
__device__ __forceinline__ double lane_xor(double v, int d) { return __shfl_xor(v, d); }
__device__ __forceinline__ float lane_xor(float v, int d) { return __shfl_xor(v, d); }
__device__ __forceinline__ uint32_t lane_xor(uint32_t v, int d) { return (uint32_t)__shfl_xor((int)v, d); }

// The combination of v over the L lanes of a row, the same in each: within a wave by
// exchanges, across the waves of a row (L > 64) through `part`, one value a wave of the
// workgroup, which no wave may still be reading from an earlier use.
template <int L, class T, class F>
__device__ __forceinline__ T over_row(T v, F f, T* part) {
#pragma unroll
  for (int d = 1; d < (L < 64 ? L : 64); d *= 2) v = f(v, lane_xor(v, d));
  if constexpr (L > 64) {
    constexpr int W = L / 64;
    const int wave = threadIdx.x >> 6, first = wave / W * W;
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    v = part[first];
#pragma unroll
    for (int w = 1; w < W; ++w) v = f(v, part[first + w]);
  }
  return v;
}

// 1 / sqrt(x) of x >= 0 to a few units in the last place of 64 bits, rounded to fp32: the
// hardware's value and one step of Newton's method, which has nothing to add to 0 and
// infinity.
__device__ __forceinline__ float inv_sqrt(double x) {
  const double r = __builtin_amdgcn_rsq(x);
  const double better = r + 0.5 * r * __builtin_fma(-x * r, r, 1.0);
  return (float)(x > 0.0 && x < __builtin_inf() ? better : r);
}

// Lanes and units a lane for rows of `units` units: the first shape that holds the row.
#define FP4G_NORM_SHAPES(F) \
  F(16, 16, 1) F(32, 32, 1) F(64, 64, 1) F(128, 64, 2) F(256, 64, 4) F(512, 256, 2) F(1024, 256, 4) F(2048, 512, 4) \
  F(4096, 1024, 4)

}  // namespace fp4g
