// Rows in registers: what the norm's kernels share.
//
// A row of K elements is walked in units of 16 bytes, L lanes a row and C units a lane, unit
// u = lane + c * L.  L is 8 to 64, four waves a workgroup, or 0: the whole workgroup, of any
// number of waves, so that a row leaves at most 63 lanes idle.  Rows start at any element (odd
// K), so units are read and written as unaligned vectors, which cost nothing where they
// happen to be aligned.  The last unit of a row may be short: it is read whole, into the next
// row, and what is past its end cleared once all loads are on their way (element by element
// a short unit's own wait would come before the next load); only at the buffer's end it is
// read by elements.
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
  // Elements first .. first + EPU - 1 of a row of K at p.  TAIL: whether the last unit of a row may
  // be short; `more`: whether as many elements as a unit has follow the row.
  template <bool TAIL = true, bool NT = false>
  __device__ static __forceinline__ v4u load(const void* p, int64_t first, int64_t K, bool more) {
    const uint8_t* q = static_cast<const uint8_t*>(p) + first * ELEM;
    if (!TAIL || more || first + EPU <= K) {
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
  // Zeros past the row's end.
  template <bool TAIL = true>
  __device__ static __forceinline__ void clear(v4u& v, int64_t first, int64_t K) {
    if (TAIL && first + EPU > K) {
#pragma unroll
      for (int e = 0; e < EPU; ++e)
        if (first + e >= K) v[BF16 ? e / 2 : e] &= BF16 ? (e & 1 ? 0xffffu : 0u) : 0u;
    }
  }
  template <bool TAIL = true>
  __device__ static __forceinline__ void store(void* p, int64_t first, int64_t K, const v4u& v) {
    uint8_t* q = static_cast<uint8_t*>(p) + first * ELEM;
    if (!TAIL || first + EPU <= K) {
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

// The weights of N elements as they lie in memory, 1 where there are none: loaded before they
// are needed, and four or eight registers until then.
template <bool BF16, int N>
struct Weights {
  static constexpr int EPU = Unit<BF16>::EPU, U = N > EPU ? N / EPU : 1;
  v4u v[U];
  template <bool TAIL = true>
  __device__ __forceinline__ void load(const void* W, int64_t first, int64_t K) {
    if (!W) {
#pragma unroll
      for (int c = 0; c < U; ++c) v[c] = BF16 ? v4u(0x3f803f80u) : v4u(0x3f800000u);
    } else if constexpr (EPU <= N) {
#pragma unroll
      for (int c = 0; c < U; ++c) v[c] = Unit<BF16>::template load<TAIL>(W, first + c * EPU, K, false);
    } else {   // four bf16 weights for four fp32 elements
      typedef v2u any __attribute__((aligned(2)));
      const uint16_t* q = static_cast<const uint16_t*>(W) + first;
      v2u w{0, 0};
      if (!TAIL || first + N <= K) {
        w = *reinterpret_cast<const any*>(q);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (first + e < K) w[e / 2] |= (uint32_t)q[e] << (e & 1 ? 16 : 0);
      }
      v[0] = v4u{w[0], w[1], 0, 0};
    }
  }
  __device__ __forceinline__ float at(int e) const { return Unit<BF16>::at(v[e / EPU], e % EPU); }
};

struct Add {
  template <class T> __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
// Steps of a combination over a wave, of values of one or more 32-bit words: step D pairs lanes D
// apart or, within 16, lanes that already hold the same as those.  No step goes through LDS.
template <int D>
__device__ __forceinline__ void pair_words(uint32_t v, uint32_t* a, uint32_t* b) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (D == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);   // both halves' own half, in every lane
    *a = r[0], *b = r[1];
  } else if constexpr (D == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    *a = r[0], *b = r[1];
  } else {
    // quad_perm [1,0,3,2], [2,3,0,1], row_half_mirror, row_mirror
    constexpr int ctrl = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;
    *a = v, *b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, ctrl, 0xf, 0xf, true);
  }
#else
  *a = *b = v;
#endif
}
template <int D, class T, class F>
__device__ __forceinline__ T pair_step(const T& v, F f) {
  constexpr int W = sizeof(T) / 4;
  struct Words { uint32_t w[W]; };
  const Words in = __builtin_bit_cast(Words, v);
  Words a, b;
#pragma unroll
  for (int i = 0; i < W; ++i) pair_words<D>(in.w[i], &a.w[i], &b.w[i]);
  return f(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
}

// The combination of v over the lanes of a row (L as above), the same in each: within a wave in
// steps, across the waves of a workgroup through `part`, one value a wave, which no wave may
// still be reading from an earlier use; T{} changes nothing.
template <int L, class T, class F>
__device__ __forceinline__ T over_row(T v, F f, T* part) {
  v = pair_step<1>(v, f);
  v = pair_step<2>(v, f);
  v = pair_step<4>(v, f);
  if constexpr (L == 0 || L >= 16) v = pair_step<8>(v, f);
  if constexpr (L == 0 || L >= 32) v = pair_step<16>(v, f);
  if constexpr (L == 0 || L >= 64) v = pair_step<32>(v, f);
  if constexpr (L == 0) {
    const int lane = threadIdx.x & 15, waves = blockDim.x >> 6;
    if (waves > 1) {
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
      __syncthreads();
      v = lane < waves ? part[lane] : T{};
      v = pair_step<1>(v, f);
      v = pair_step<2>(v, f);
      v = pair_step<4>(v, f);
      v = pair_step<8>(v, f);
    }
  }
  return v;
}
template <int L> __device__ __forceinline__ int lanes_of() { return L ? L : (int)blockDim.x; }

// 1 / sqrt(x) of x >= 0 to a few units in the last place of 64 bits, rounded to fp32: the
// hardware's value and one step of Newton's method, which has nothing to add to 0 and
// infinity.
__device__ __forceinline__ float inv_sqrt(double x) {
  const double r = __builtin_amdgcn_rsq(x);
  const double better = r + 0.5 * r * __builtin_fma(-x * r, r, 1.0);
  return (float)(x > 0.0 && x < __builtin_inf() ? better : r);
}

}  // namespace fp4g
