// Row quantizer for gfx950: fp32 or bf16 X[rows][K] -> int8 codes [rows][K] and one fp32
// scale a row, every step in IEEE fp32:
//   scale = max|x| / 127,  inv = min(1 / scale, FLT_MAX),
//   code  = clamp(round to even(x * inv), -127, 127);
// a row of zeros gets scale 0 and zero codes, a row holding an infinity or NaN a NaN scale
// and zero codes (nothing finite stands for it, and the NaN reaches every product of it).
//
// HBM-bound: 5 (fp32) or 3 (bf16) bytes an element; 8192 x 8192 fp32 takes 53 us, 6.4 TB/s.
// The row stays in registers between the maximum and the codes, so X is read once: W waves
// own a row, C 16-byte loads a lane, all issued before the first is used.  Rows longer than
// 16 waves x 8 loads hold (32768 fp32, 65536 bf16) are read twice by the last kernel below.
#include <algorithm>

#include "common.hpp"
#include "ffn_internal.h"
#include "launch.hpp"

namespace fp4g {
namespace {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));

// 16 bytes of X as EPU fp32 values.
template <bool BF16> struct Unit;
template <> struct Unit<false> {
  static constexpr int EPU = 4;
  __device__ static __forceinline__ float at(const v4u& w, int e) {
    const uint32_t bits = w[e];   // a value: the cast of the element itself reads element 0
    return __builtin_bit_cast(float, bits);
  }
};
template <> struct Unit<true> {
  static constexpr int EPU = 8;
  __device__ static __forceinline__ float at(const v4u& w, int e) {
    return __builtin_bit_cast(float, e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
};

// max|x| as bits: magnitudes order like integers, infinities and NaN past every finite one.
template <bool BF16>
__device__ __forceinline__ uint32_t max_bits(const v4u& w, uint32_t most) {
#pragma unroll
  for (int e = 0; e < Unit<BF16>::EPU; ++e)
    most = max(most, __builtin_bit_cast(uint32_t, Unit<BF16>::at(w, e)) & 0x7fffffffu);
  return most;
}

template <bool BF16>
__device__ __forceinline__ void store_codes(uint8_t* q, const v4u& w, float inv) {
  constexpr int EPU = Unit<BF16>::EPU;
  uint32_t word[EPU / 4];
#pragma unroll
  for (int k = 0; k < EPU / 4; ++k) {
    uint32_t c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float y = __builtin_amdgcn_fmed3f(__builtin_rintf(Unit<BF16>::at(w, 4 * k + e) * inv), -127.0f, 127.0f);
      c |= ((uint32_t)(int)y & 255u) << (8 * e);
    }
    word[k] = c;
  }
  if constexpr (BF16) *reinterpret_cast<v2u*>(q) = v2u{word[0], word[1]};
  else *reinterpret_cast<uint32_t*>(q) = word[0];
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}

// The scale and the inverse of a row whose largest magnitude has these bits.
__device__ __forceinline__ float inverse_of(uint32_t most, float* scale) {
  if (most >= 0x7f800000u) {
    *scale = __builtin_nanf("");
    return 0.0f;
  }
  *scale = __builtin_bit_cast(float, most) / 127.0f;
  return fminf(1.0f / *scale, 3.402823466e+38f);
}

// W waves a row, C loads a lane; a workgroup of 4 waves (W when that is more) holds several rows
// when W < 4.  The code of a non-finite row is x * 0 = 0 or NaN: written as zeros below.
template <bool BF16, int W, int C>
__global__ void __launch_bounds__((W < 4 ? 4 : W) * 64)
int8_quantize_kernel(int64_t rows, int K, const uint8_t* __restrict__ X, uint8_t* __restrict__ codes,
                     float* __restrict__ scales) {
  constexpr int EPU = Unit<BF16>::EPU, NW = W < 4 ? 4 : W, RPW = NW / W;
  __shared__ uint32_t part[NW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * RPW + wave / W;
  const int units = K / EPU, first = (wave % W) * 64 + lane;
  const uint8_t* x = X + min(row, rows - 1) * K * (BF16 ? 2 : 4);
  v4u v[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int u = first + c * W * 64;
    v[c] = u < units ? __builtin_nontemporal_load(reinterpret_cast<const v4u*>(x) + u) : v4u{0, 0, 0, 0};
  }
  uint32_t most = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) most = max_bits<BF16>(v[c], most);
  most = wave_max(most);
  if constexpr (W > 1) {
    if (lane == 0) part[wave] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) most = max(most, part[wave / W * W + w]);
  }
  if (row >= rows) return;
  float scale;
  const float inv = inverse_of(most, &scale);
  if (first == 0) scales[row] = scale;
  const bool finite = most < 0x7f800000u;
  uint8_t* q = codes + row * K;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int u = first + c * W * 64;
    if (u < units) store_codes<BF16>(q + u * EPU, finite ? v[c] : v4u{0, 0, 0, 0}, inv);
  }
}

// Longer rows: 16 waves a row, read twice (the second time from the caches if they hold it).
template <bool BF16>
__global__ void __launch_bounds__(1024)
int8_quantize_long_kernel(int K, const uint8_t* __restrict__ X, uint8_t* __restrict__ codes,
                          float* __restrict__ scales) {
  constexpr int EPU = Unit<BF16>::EPU;
  __shared__ uint32_t part[16];
  const int64_t row = blockIdx.x;
  const int units = K / EPU;
  const v4u* x = reinterpret_cast<const v4u*>(X + row * K * (BF16 ? 2 : 4));
  uint32_t most = 0;
  for (int u = threadIdx.x; u < units; u += 1024) most = max_bits<BF16>(x[u], most);
  most = wave_max(most);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) most = max(most, part[w]);
  float scale;
  const float inv = inverse_of(most, &scale);
  if (threadIdx.x == 0) scales[row] = scale;
  const bool finite = most < 0x7f800000u;
  uint8_t* q = codes + row * K;
  for (int u = threadIdx.x; u < units; u += 1024)
    store_codes<BF16>(q + (int64_t)u * EPU, finite ? x[u] : v4u{0, 0, 0, 0}, inv);
}

template <bool BF16, int W, int C>
hipError_t launch_rows(int64_t rows, int64_t K, const void* X, void* codes, float* scales, hipStream_t s) {
  constexpr int NW = W < 4 ? 4 : W;
  // A launch holds fewer than 2^32 threads, so very many short rows take several.
  const int64_t most = ((int64_t)1 << 31) / (NW * 64) * (NW / W);
  for (int64_t first = 0; first < rows; first += most) {
    const int64_t n = std::min(rows - first, most);
    const hipError_t e = launch(int8_quantize_kernel<BF16, W, C>, ceil_div(n, NW / W), NW * 64, s, n, (int)K,
                                static_cast<const uint8_t*>(X) + first * K * (BF16 ? 2 : 4),
                                static_cast<uint8_t*>(codes) + first * K, scales + first);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool BF16>
hipError_t launch_type(int64_t rows, int64_t K, const void* X, void* codes, float* scales, hipStream_t s) {
  // 1 KB loads a row.  Few waves a row keep many rows in flight, many shorten the row: of the
  // shapes that hold a row, these took the least time or within 4% of it at 1 .. 8192 rows.
  // In us, waves x loads: 8192 x 8192 fp32 8x4 56.3, 4x8 58.8, 16x2 61.1; 333 x 14336 bf16
  // 8x4 6.5, 4x8 6.9, 16x4 7.0; 8192 x 1024 fp32 1x4 9.3, 2x2 10.0, 4x1 11.2; 1000 x 4096
  // bf16 4x2 5.4, 2x4 5.6, 8x2 5.7, 16x1 6.6.
  const int64_t loads = ceil_div(K / Unit<BF16>::EPU, 64);
  if (loads <= 1) return launch_rows<BF16, 1, 1>(rows, K, X, codes, scales, s);
  if (loads <= 2) return launch_rows<BF16, 1, 2>(rows, K, X, codes, scales, s);
  if (loads <= 4) return launch_rows<BF16, 1, 4>(rows, K, X, codes, scales, s);
  if (loads <= 8) return launch_rows<BF16, 4, 2>(rows, K, X, codes, scales, s);
  if (loads <= 16) return launch_rows<BF16, 4, 4>(rows, K, X, codes, scales, s);
  if (loads <= 32) return launch_rows<BF16, 8, 4>(rows, K, X, codes, scales, s);
  if (loads <= 64) return launch_rows<BF16, 16, 4>(rows, K, X, codes, scales, s);
  if (loads <= 128) return launch_rows<BF16, 16, 8>(rows, K, X, codes, scales, s);
  return launch(int8_quantize_long_kernel<BF16>, rows, 1024, s, (int)K, static_cast<const uint8_t*>(X),
                static_cast<uint8_t*>(codes), scales);
}

}  // namespace

hipError_t launch_int8_quantize(int64_t rows, int64_t K, const void* X, bool bf16_in, void* codes, float* scales,
                                hipStream_t s) {
  return bf16_in ? launch_type<true>(rows, K, X, codes, scales, s) : launch_type<false>(rows, K, X, codes, scales, s);
}

}  // namespace fp4g
