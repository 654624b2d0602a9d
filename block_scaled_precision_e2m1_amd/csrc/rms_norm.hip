// The root-mean-square norm of rows for gfx950, with the residual's addition and 8-bit
// outputs:
//   h = round(x + r),  s = fp32(1 / sqrt(mean(h^2) + eps)),  y = (h * s) * w
// and, quantized, scale = max|y| / T, code = round(y * min(1 / scale, FLT_MAX)).
//
// HBM-bound: x and r are read once, h and y (or codes) written once.  The row stays in
// registers from the load to the last store: L lanes own a row, C 16-byte units a lane, all
// loaded before the first is used; short rows (heads) share a wave.  Rows longer than the
// largest shape holds are read again by the last kernel below, from h where it was written.
//
// The mean is formed in 64 bits: s is then the same whatever the order of the sum, so that a
// row has the same codes in any shape (a code next to a rounding border turns on s's last
// bit), and no square overflows.  The multiply-adds it takes in 64 bits hide under the loads.
#include <algorithm>

#include "launch.hpp"
#include "norm_rows.hpp"

namespace fp4g {
namespace {

// h of one unit: x, or x + r rounded to their type.
template <bool BF16>
__device__ __forceinline__ v4u add_units(const v4u& x, const v4u& r) {
  typedef Unit<BF16> U;
  float h[U::EPU];
#pragma unroll
  for (int e = 0; e < U::EPU; ++e) h[e] = U::at(x, e) + U::at(r, e);
  return U::pack(h);
}

template <bool BF16>
__device__ __forceinline__ double squares(const v4u& h, double sum) {
#pragma unroll
  for (int e = 0; e < Unit<BF16>::EPU; ++e) {
    const double v = Unit<BF16>::at(h, e);
    sum = __builtin_fma(v, v, sum);
  }
  return sum;
}

// y = (h * s) * w of a unit.
template <bool BF16, class WEIGHTS>
__device__ __forceinline__ void normed(const v4u& h, float s, const WEIGHTS& w, float (&y)[Unit<BF16>::EPU]) {
#pragma unroll
  for (int e = 0; e < Unit<BF16>::EPU; ++e) y[e] = Unit<BF16>::at(h, e) * s * w.at(e);
}

// max|y| as bits: magnitudes order like integers, infinities and NaN past every finite one.
template <int N>
__device__ __forceinline__ uint32_t max_bits(const float (&y)[N], int64_t left, uint32_t most) {
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (e < left) most = max(most, __builtin_bit_cast(uint32_t, y[e]) & 0x7fffffffu);
  return most;
}

// The scale and the inverse of a row whose largest magnitude has these bits.
__device__ __forceinline__ float inverse_of(uint32_t most, float top, float* scale) {
  if (most >= 0x7f800000u) {
    *scale = __builtin_nanf("");
    return 0.0f;
  }
  *scale = __builtin_bit_cast(float, most) / top;
  return fminf(1.0f / *scale, 3.402823466e+38f);
}

// A row of zeros has zero codes (not E4M3's -0), as one that holds an infinity or NaN.
__device__ __forceinline__ bool has_codes(uint32_t most) { return most - 1 < 0x7f800000u - 1; }

// Codes of EPU values at q, of which the first `left` exist.
template <int EPU>
__device__ __forceinline__ void store_codes(uint8_t* q, int64_t left, const float (&y)[EPU], float inv, bool e4m3,
                                            bool some) {
  uint32_t word[EPU / 4];
#pragma unroll
  for (int k = 0; k < EPU / 4; ++k) {
    uint32_t c = 0;
    if (e4m3) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_amdgcn_fmed3f(y[4 * k + e] * inv, -448.0f, 448.0f);
      int p = 0;
      p = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], p, false);
      p = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], p, true);
      c = (uint32_t)p;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = __builtin_amdgcn_fmed3f(__builtin_rintf(y[4 * k + e] * inv), -127.0f, 127.0f);
        c |= ((uint32_t)(int)v & 255u) << (8 * e);
      }
    }
    word[k] = some ? c : 0u;
  }
  if (left >= EPU) {
    typedef uint32_t u32_any __attribute__((aligned(1)));
    typedef v2u v2u_any __attribute__((aligned(1)));
    if constexpr (EPU == 8) *reinterpret_cast<v2u_any*>(q) = v2u{word[0], word[1]};
    else *reinterpret_cast<u32_any*>(q) = word[0];
  } else {
#pragma unroll
    for (int e = 0; e < EPU; ++e)
      if (e < left) q[e] = (uint8_t)(word[e / 4] >> (8 * (e % 4)));
  }
}

// The rows of one launch; a launch holds fewer than 2^32 threads.
struct Rows {
  int64_t rows;
  int K;
  const uint8_t *X, *R;
  const void* W;
  uint8_t *H, *Y, *codes;
  float* scales;
  double eps;
  bool e4m3;
};

// H may be X or R, Y may be X or R: a row's units are stored by the lanes that read them, and
// after every load of theirs.  The weights are asked for before the row's sum is known, so that
// one latency covers both.
template <bool BF16, bool WBF16, bool QUANT, bool TAIL, int L, int C>
__global__ void __launch_bounds__(L ? 256 : 1024) rms_norm_kernel(const Rows a) {
  typedef Unit<BF16> U;
  constexpr int RPW = L ? 256 / L : 1;
  __shared__ double sums[16];
  __shared__ uint32_t mosts[16];
  const int lanes = lanes_of<L>(), lane = threadIdx.x % lanes;
  const int64_t mine = (int64_t)blockIdx.x * RPW + threadIdx.x / lanes;
  const bool there = mine < a.rows;
  const int64_t row = there ? mine : a.rows - 1;
  const int units = ((uint32_t)a.K + U::EPU - 1) / U::EPU;
  const int64_t at = row * a.K * U::ELEM;
  const bool more = (a.rows - 1 - row) * a.K >= U::EPU;
  v4u h[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int u = lane + c * lanes;
    h[c] = u < units ? U::template load<TAIL, true>(a.X + at, (int64_t)u * U::EPU, a.K, more) : v4u{0, 0, 0, 0};
  }
  Weights<WBF16, U::EPU> w[C];
  auto weights = [&]() {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int u = lane + c * lanes;
      if (u < units) w[c].template load<TAIL>(a.W, (int64_t)u * U::EPU, a.K);
    }
  };
  if (a.R) {
    v4u r[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int u = lane + c * lanes;
      r[c] = u < units ? U::template load<TAIL, true>(a.R + at, (int64_t)u * U::EPU, a.K, more) : v4u{0, 0, 0, 0};
    }
    weights();
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int u = lane + c * lanes;
      h[c] = add_units<BF16>(h[c], r[c]);
      U::template clear<TAIL>(h[c], (int64_t)u * U::EPU, a.K);
      if (there && u < units) U::template store<TAIL>(a.H + at, (int64_t)u * U::EPU, a.K, h[c]);
    }
  } else {
    weights();
#pragma unroll
    for (int c = 0; c < C; ++c) U::template clear<TAIL>(h[c], (int64_t)(lane + c * lanes) * U::EPU, a.K);
  }
  double sum = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) sum = squares<BF16>(h[c], sum);
  sum = over_row<L>(sum, Add{}, sums);
  const float s = inv_sqrt(sum / (double)a.K + a.eps);
  float y[QUANT ? C : 1][U::EPU];
  uint32_t most = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int u = lane + c * lanes;
    const int64_t first = (int64_t)u * U::EPU;
    float(&v)[U::EPU] = y[QUANT ? c : 0];
    if (u < units) {
      normed<BF16>(h[c], s, w[c], v);
      if constexpr (QUANT) most = max_bits(v, TAIL ? a.K - first : U::EPU, most);
      if (there && (!QUANT || a.Y)) U::template store<TAIL>(a.Y + at, first, a.K, U::pack(v));
    }
  }
  if constexpr (QUANT) {
    most = over_row<L>(most, Max{}, mosts);
    if (!there) return;
    float scale;
    const float inv = inverse_of(most, a.e4m3 ? 448.0f : 127.0f, &scale);
    if (lane == 0) a.scales[row] = scale;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int u = lane + c * lanes;
      const int64_t first = (int64_t)u * U::EPU;
      if (u < units)
        store_codes(a.codes + row * a.K + first, TAIL ? a.K - first : U::EPU, y[c], inv, a.e4m3, has_codes(most));
    }
  }
}

// Longer rows: 16 waves a row; h is read again for y, and for the codes.
template <bool BF16, bool WBF16, bool QUANT>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(const Rows a) {
  typedef Unit<BF16> U;
  __shared__ double sums[16];
  __shared__ uint32_t mosts[16];
  const int64_t row = blockIdx.x, at = row * a.K * U::ELEM;
  const int units = ((uint32_t)a.K + U::EPU - 1) / U::EPU;
  double sum = 0.0;
  for (int u = threadIdx.x; u < units; u += 1024) {
    const int64_t first = (int64_t)u * U::EPU;
    v4u h = U::load(a.X + at, first, a.K, false);
    if (a.R) {
      h = add_units<BF16>(h, U::load(a.R + at, first, a.K, false));
      U::store(a.H + at, first, a.K, h);
    }
    sum = squares<BF16>(h, sum);
  }
  sum = over_row<0>(sum, Add{}, sums);
  const float s = inv_sqrt(sum / (double)a.K + a.eps);
  const uint8_t* src = (a.R ? a.H : a.X) + at;   // a thread reads what it wrote itself
  uint32_t most = 0;
  for (int u = threadIdx.x; u < units; u += 1024) {
    const int64_t first = (int64_t)u * U::EPU;
    float y[U::EPU];
    Weights<WBF16, U::EPU> w;
    w.load(a.W, first, a.K);
    normed<BF16>(U::load(src, first, a.K, false), s, w, y);
    if constexpr (QUANT) most = max_bits(y, a.K - first, most);
    else U::store(a.Y + at, first, a.K, U::pack(y));
  }
  if constexpr (QUANT) {
    most = over_row<0>(most, Max{}, mosts);
    float scale;
    const float inv = inverse_of(most, a.e4m3 ? 448.0f : 127.0f, &scale);
    if (threadIdx.x == 0) a.scales[row] = scale;
    for (int u = threadIdx.x; u < units; u += 1024) {
      const int64_t first = (int64_t)u * U::EPU;
      float y[U::EPU];
      Weights<WBF16, U::EPU> w;
      w.load(a.W, first, a.K);
      normed<BF16>(U::load(src, first, a.K, false), s, w, y);
      if (a.Y) U::store(a.Y + at, first, a.K, U::pack(y));   // over X, if at all, once it is no longer read
      store_codes(a.codes + row * a.K + first, a.K - first, y, inv, a.e4m3, has_codes(most));
    }
  }
}

// Lanes a row (0: a workgroup) and units a lane; units 0: the rows are too long for any shape.
struct Shape { int lanes, units; };
// Two units a lane: in us, (lanes, units), 131072 x 128 bf16 (8, 2) 12.4, (16, 1) 13.4, (4, 4) 15.5;
// 8192 x 8192 bf16 with a residual (512, 2) 78.6, (256, 4) 80.1.  Of rows longer than a wave, those that
// the chip's 2048 lanes a CU hold all at once with one unit a lane (below 8 MB on 256 CUs) are bound by
// latency and take one; the others need the second unit's loads in flight.  One and two, with a
// residual:
//   below  512 x 2048 bf16 3.3 3.7, 1003 x 1117 fp32 4.9 5.6, 2048 x 1117 bf16 7.0 7.4
//   at it  2048 x 2048 bf16 6.8 6.9 (without 4.9 4.5), 2048 x 1040 fp32 7.9 6.8
//   above  1500 x 2048 fp32 10.3 9.3, 2048 x 4096 bf16 14.2 14.0 (without 8.2 7.4)
// Past 512 units the two are within 4% where few rows are there (512 x 6144 bf16 5.8 6.1, 256 x 8192
// 4.5 4.5).
Shape shape_of(int64_t rows, int64_t units) {
  if (units <= 16) return {8, 2};
  if (units <= 32) return {16, 2};
  if (units <= 64) return {32, 2};
  if (units <= 128) return {64, 2};
  if (units <= 512 && rows * units < 2048 * device_cus()) return {0, 1};
  if (units <= 2048) return {0, 2};
  if (units <= 4096) return {0, 4};
  return {0, 0};
}
struct Launch { int block, per; int64_t most; };   // threads and rows of a workgroup, rows of a launch
Launch launch_of(Shape h, int64_t units) {
  Launch l{1024, 1, 0};
  if (h.lanes) l.block = 256, l.per = 256 / h.lanes;
  else if (h.units) l.block = (int)(ceil_div(units, 64 * h.units) * 64);
  l.most = ((int64_t)1 << 31) / l.block * l.per;
  return l;
}

template <bool BF16, bool WBF16, bool QUANT>
hipError_t launch_rows(const NormArgs& a, hipStream_t s) {
  const int64_t units = ceil_div(a.K, Unit<BF16>::EPU), elem = Unit<BF16>::ELEM;
  const Shape shape = shape_of(a.rows, units);
  const Launch l = launch_of(shape, units);
  void (*kernel)(Rows) = rms_norm_long_kernel<BF16, WBF16, QUANT>;
#define SHAPE(L, C)                                                                                       \
  if (shape.lanes == L && shape.units == C)                                                               \
    kernel = a.K % Unit<BF16>::EPU ? rms_norm_kernel<BF16, WBF16, QUANT, true, L, C>                      \
                                   : rms_norm_kernel<BF16, WBF16, QUANT, false, L, C>
  SHAPE(8, 2);
  SHAPE(16, 2);
  SHAPE(32, 2);
  SHAPE(64, 2);
  SHAPE(0, 1);
  SHAPE(0, 2);
  SHAPE(0, 4);
#undef SHAPE
  for (int64_t first = 0; first < a.rows; first += l.most) {
    const int64_t n = std::min(a.rows - first, l.most), at = first * a.K;
    auto past = [&](const void* p, int64_t bytes) {
      return p ? const_cast<uint8_t*>(static_cast<const uint8_t*>(p)) + bytes : nullptr;
    };
    const Rows r{n, (int)a.K, past(a.X, at * elem), past(a.R, at * elem), a.W, past(a.H, at * elem),
                 past(a.Y, at * elem), past(a.codes, at), a.scales ? a.scales + first : nullptr, a.eps, a.e4m3};
    const hipError_t e = launch(kernel, ceil_div(n, l.per), l.block, s, r);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool BF16, bool WBF16>
hipError_t launch_out(const NormArgs& a, hipStream_t s) {
  return a.codes ? launch_rows<BF16, WBF16, true>(a, s) : launch_rows<BF16, WBF16, false>(a, s);
}

}  // namespace

int64_t rms_norm_launch_rows(int64_t rows, int64_t K, bool bf16) {
  const int64_t units = ceil_div(K, bf16 ? 8 : 4);
  return launch_of(shape_of(rows, units), units).most;
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  if (a.bf16) return a.w_bf16 ? launch_out<true, true>(a, s) : launch_out<true, false>(a, s);
  return a.w_bf16 ? launch_out<false, true>(a, s) : launch_out<false, false>(a, s);
}

}  // namespace fp4g
