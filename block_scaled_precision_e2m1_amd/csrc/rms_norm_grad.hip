// The gradients of the root-mean-square norm for gfx950.  With n = x * s, s as in the norm,
// and g = dy * w:
//   dX = s (g - n mean(g n)) + dH,   dW = sum over rows of dy n.
//
// HBM-bound: dy, x and dH are read once, dX written once.  The workgroups are persistent: a
// lane keeps the same columns of every row it takes, so the weight and dW's sums stay in its
// registers, and the next row's loads are in flight while this row's two sums (of x^2 and of
// g x, from which s and mean(g n) = s mean(g x) follow) go around the row's lanes.  Each
// workgroup then leaves one row of partial sums of dW, and a second kernel adds those in
// order: no atomics, so results repeat bit for bit.
//
// Rows longer than the largest shape holds take three kernels: the two sums of each row, a
// walk down the columns for dX and dW's partial sums, and their sum.
#include <algorithm>

#include "launch.hpp"
#include "norm_rows.hpp"

namespace fp4g {
namespace {

struct Grad {
  int64_t rows;
  int K;
  const uint8_t *dY, *X, *dH;
  const void* W;
  uint8_t* dX;
  float* P;       // [workgroups][K], or null: dW is not wanted
  float* S;       // long rows: s of each row
  double eps;
};

// dX of one unit: s (g - x c) + dH with c = s^2 mean(g x).
template <bool BF16, class WEIGHTS>
__device__ __forceinline__ v4u grad_unit(const v4u& dy, const v4u& x, const WEIGHTS& w, const v4u& dh, float s, float c) {
  typedef Unit<BF16> U;
  float d[U::EPU];
#pragma unroll
  for (int e = 0; e < U::EPU; ++e) d[e] = s * (U::at(dy, e) * w.at(e) - U::at(x, e) * c) + U::at(dh, e);
  return U::pack(d);
}

// c of a row.  s^2 itself leaves fp32's range where rows of about 1e20 or 1e-20 do not.
__device__ __forceinline__ float projection(float s, float gx, int K) { return s * (s * (gx / (float)K)); }

// The two sums of a row, in 64 bits and 32.
struct __attribute__((packed, aligned(4))) Sums {
  double xx;
  float gx;
};
struct AddSums {
  __device__ __forceinline__ Sums operator()(Sums a, Sums b) const { return Sums{a.xx + b.xx, a.gx + b.gx}; }
};

template <bool BF16, class WEIGHTS>
__device__ __forceinline__ void add_unit(const v4u& dy, const v4u& x, const WEIGHTS& w, Sums* t) {
  typedef Unit<BF16> U;
#pragma unroll
  for (int e = 0; e < U::EPU; ++e) {
    const double v = U::at(x, e);
    t->xx = __builtin_fma(v, v, t->xx);
    t->gx += U::at(dy, e) * w.at(e) * U::at(x, e);
  }
}

// dX may be dY or dH: a row's units are stored by the lanes that read them, after their loads.
template <bool BF16, bool WBF16, bool TAIL, int L, int C>
__global__ void __launch_bounds__(L ? 256 : 1024) rms_norm_grad_kernel(const Grad a) {
  typedef Unit<BF16> U;
  constexpr int EPU = U::EPU, RPW = L ? 256 / (L + !L) : 1;
  __shared__ Sums parts[2][16];
  __shared__ float columns[RPW > 1 ? 256 * EPU * C : 1];
  const int lanes = lanes_of<L>(), lane = threadIdx.x % lanes, sub = threadIdx.x / lanes, units = ((uint32_t)a.K + EPU - 1) / EPU;
  Weights<WBF16, EPU> w[C];
  float dw[C][EPU];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (lane + c * lanes < units) w[c].template load<TAIL>(a.W, (int64_t)(lane + c * lanes) * EPU, a.K);
#pragma unroll
    for (int e = 0; e < EPU; ++e) dw[c][e] = 0.0f;
  }
  const v4u none{0, 0, 0, 0};
  auto fetch = [&](const uint8_t* p, int64_t row, v4u(&v)[C]) {
    const bool more = (a.rows - 1 - row) * a.K >= EPU;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int u = lane + c * lanes;
      v[c] = p && u < units && row < a.rows ? U::template load<TAIL, true>(p + row * a.K * U::ELEM, (int64_t)u * EPU, a.K, more)
                                            : none;
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPW;
  // 16 waves of two units a lane have no registers for a second row.
  constexpr bool AHEAD = C == 1;
  v4u x[C], dy[C], dh[C], x1[C], dy1[C], dh1[C];
  auto fetch_row = [&](int64_t row, v4u(&x)[C], v4u(&dy)[C], v4u(&dh)[C]) {
    fetch(a.X, row, x);
    fetch(a.dY, row, dy);
    fetch(a.dH, row, dh);
  };
  if constexpr (AHEAD) fetch_row((int64_t)blockIdx.x * RPW + sub, x, dy, dh);
  int turn = 0;
  // The rows of a workgroup's turn are neighbours; all its waves take the same number of turns.
  for (int64_t first = (int64_t)blockIdx.x * RPW; first < a.rows; first += step, turn ^= 1) {
    const int64_t row = first + sub;
    if constexpr (AHEAD) fetch_row(row + step, x1, dy1, dh1);
    else fetch_row(row, x, dy, dh);
    Sums t{0.0, 0.0f};
    if constexpr (TAIL) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        U::template clear<TAIL>(x[c], (int64_t)(lane + c * lanes) * EPU, a.K);
        U::template clear<TAIL>(dy[c], (int64_t)(lane + c * lanes) * EPU, a.K);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (lane + c * lanes < units) add_unit<BF16>(dy[c], x[c], w[c], &t);
    // Two sets of parts in turn: a wave is at most one row ahead of another's reads.
    t = over_row<L>(t, AddSums{}, parts[turn]);
    const float s = inv_sqrt(t.xx / (double)a.K + a.eps), k = projection(s, t.gx, a.K);
    const int64_t at = row * a.K * U::ELEM;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int u = lane + c * lanes;
      if (u < units && row < a.rows) {
        U::template store<TAIL>(a.dX + at, (int64_t)u * EPU, a.K, grad_unit<BF16>(dy[c], x[c], w[c], dh[c], s, k));
#pragma unroll
        for (int e = 0; e < EPU; ++e) dw[c][e] += U::at(dy[c], e) * (U::at(x[c], e) * s);
      }
      if constexpr (AHEAD) x[c] = x1[c], dy[c] = dy1[c], dh[c] = dh1[c];
    }
  }
  if (!a.P) return;
  float* P = a.P + (int64_t)blockIdx.x * a.K;
  if constexpr (RPW > 1) {   // the rows of a turn, in order
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < EPU; ++e) columns[(sub * C + c) * L * EPU + lane * EPU + e] = dw[c][e];
    __syncthreads();
    for (int k = threadIdx.x; k < a.K; k += 256) {
      const int u = k / EPU, c = u / L, in = c * L * EPU + (u - c * L) * EPU + k % EPU;
      float sum = 0.0f;
      for (int r = 0; r < RPW; ++r) sum += columns[r * C * L * EPU + in];
      P[k] = sum;
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < EPU; ++e) {
        const int64_t k = (int64_t)(lane + c * lanes) * EPU + e;
        if (k < a.K) P[k] = dw[c][e];
      }
  }
}

// Longer rows, first: the sums of each row, as s and k.
template <bool BF16, bool WBF16>
__global__ void __launch_bounds__(1024) rms_norm_grad_sums_kernel(const Grad a) {
  typedef Unit<BF16> U;
  __shared__ Sums parts[2][16];
  const int units = ((uint32_t)a.K + U::EPU - 1) / U::EPU;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const int64_t at = row * a.K * U::ELEM;
    Sums t{0.0, 0.0f};
    for (int u = threadIdx.x; u < units; u += 1024) {
      const int64_t first = (int64_t)u * U::EPU;
      Weights<WBF16, U::EPU> w;
      w.load(a.W, first, a.K);
      add_unit<BF16>(U::load(a.dY + at, first, a.K, false), U::load(a.X + at, first, a.K, false), w, &t);
    }
    t = over_row<0>(t, AddSums{}, parts[turn]);
    if (threadIdx.x == 0) {
      const float s = inv_sqrt(t.xx / (double)a.K + a.eps);
      a.S[2 * row] = s;
      a.S[2 * row + 1] = projection(s, t.gx, a.K);
    }
  }
}

// Then dX and dW's partial sums: a unit of columns a lane, down a share of the rows.
template <bool BF16, bool WBF16>
__global__ void __launch_bounds__(256) rms_norm_grad_columns_kernel(const Grad a, int blocks, int shares) {
  typedef Unit<BF16> U;
  constexpr int EPU = U::EPU;
  const int share = blockIdx.x / blocks;
  const int64_t first = ((int64_t)(blockIdx.x - share * blocks) * 256 + threadIdx.x) * EPU;
  if (first >= a.K) return;
  float dw[EPU] = {};
  Weights<WBF16, EPU> w;
  w.load(a.W, first, a.K);
  const int64_t end = a.rows * (share + 1) / shares;
  for (int64_t row = a.rows * share / shares; row < end; ++row) {
    const int64_t at = row * a.K * U::ELEM;
    const v4u dy = U::load(a.dY + at, first, a.K, false), x = U::load(a.X + at, first, a.K, false);
    const v4u dh = a.dH ? U::load(a.dH + at, first, a.K, false) : v4u{0, 0, 0, 0};
    const float s = a.S[2 * row], k = a.S[2 * row + 1];
    U::store(a.dX + at, first, a.K, grad_unit<BF16>(dy, x, w, dh, s, k));
#pragma unroll
    for (int e = 0; e < EPU; ++e) dw[e] += U::at(dy, e) * (U::at(x, e) * s);
  }
  if (!a.P) return;
#pragma unroll
  for (int e = 0; e < EPU; ++e)
    if (first + e < a.K) a.P[(int64_t)share * a.K + first + e] = dw[e];
}

// dW of 16 columns a workgroup: the partial sums in 64 runs of rows, added in order.
template <bool BF16>
__global__ void __launch_bounds__(1024) rms_norm_weight_kernel(int shares, int K, const float* __restrict__ P, void* dW) {
  __shared__ float sums[64][17];
  const int c = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int first = (int)((int64_t)shares * run / 64), end = (int)((int64_t)shares * (run + 1) / 64);
  for (int64_t k0 = (int64_t)blockIdx.x * 16; k0 < K; k0 += (int64_t)gridDim.x * 16) {
    const int64_t k = k0 + c;
    float sum = 0.0f;
    if (k < K) {
#pragma unroll 8
      for (int r = first; r < end; ++r) sum += P[(int64_t)r * K + k];
    }
    sums[run][c] = sum;
    __syncthreads();
    // Column c's 64 sums by the 16 lanes of one group, 4 each, then across them.
    const int col = threadIdx.x >> 4, part = threadIdx.x & 15;
    if (col < 16) {
      float t = 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) t += sums[part * 4 + r][col];
      t = over_row<16, float>(t, Add{}, nullptr);
      if (part == 0 && k0 + col < K) store_out<BF16>(dW, k0 + col, t);
    }
    __syncthreads();
  }
}

struct Plan { int lanes, block; int64_t groups; };   // block 0: a long row, of `groups` shares of rows
Plan plan_of(int64_t rows, int64_t K, bool bf16) {
  const int64_t units = ceil_div(K, bf16 ? 8 : 4), cus = device_cus();
  if (units > 2048)
    return {0, 0, std::max<int64_t>(1, std::min<int64_t>({rows, 64, 4 * cus / ceil_div(units, 256) + 1}))};
  const int lanes = units <= 16 ? 16 : units <= 32 ? 32 : units <= 64 ? 64 : 0;
  const int block = lanes ? 256 : (int)(ceil_div(units, units <= 1024 ? 64 : 128) * 64);
  // Enough workgroups for the chip, and no more: each writes a row of partial sums.  In us, 1, 2 and 4
  // workgroups a CU: 8192 x 8192 bf16 182, 187, 200 (with the norm); 8192 x 2048 bf16 53.3, 53.3, 55.6.
  // Few short rows are bound by the latency of one after the other, and take twice as many; of longer
  // ones the partial sums' way through memory takes more than that gains.  1 and 2 a CU, the gradient
  // alone:
  //   512 rows of 1040 bf16 7.7 7.7, of 1117 fp32  8.9  8.7, of 1536 bf16  8.5  9.4, fp32  8.4  8.9
  //   1003             9.2 8.5,             11.2 10.0,             10.0 10.4,       10.8 10.8
  //   512 rows of 2048 bf16 9.2 10.9, of 4096 12.7 17.8, of 8192 21.0 28.1
  const int64_t per = lanes ? 256 / lanes : 1, most = cus * std::max(1, 1024 / block);
  const int64_t many = rows < 4 * cus && K <= 1280 ? 2 * cus : std::max(cus, std::min(most, rows / 16));
  return {lanes, block, std::min(ceil_div(rows, per), many)};
}
int64_t sums_bytes(int64_t rows) { return (rows * 8 + 15) / 16 * 16; }

template <bool BF16, bool WBF16>
hipError_t launch_grad(const NormGradArgs& a, hipStream_t s) {
  const Plan p = plan_of(a.rows, a.K, BF16);
  Grad g{a.rows, (int)a.K, static_cast<const uint8_t*>(a.dY), static_cast<const uint8_t*>(a.X),
         static_cast<const uint8_t*>(a.dH), a.W, static_cast<uint8_t*>(a.dX), nullptr, nullptr, a.eps};
  float* const P = reinterpret_cast<float*>(static_cast<uint8_t*>(a.P) + (p.block ? 0 : sums_bytes(a.rows)));
  if (a.dW) g.P = P;
  hipError_t e = hipSuccess;
  if (p.block == 0) {
    g.S = static_cast<float*>(a.P);
    const int blocks = (int)ceil_div(ceil_div(a.K, Unit<BF16>::EPU), 256);
    e = launch(rms_norm_grad_sums_kernel<BF16, WBF16>, std::min(a.rows, 8 * device_cus()), 1024, s, g);
    if (e == hipSuccess)
      e = launch(rms_norm_grad_columns_kernel<BF16, WBF16>, blocks * p.groups, 256, s, g, blocks, (int)p.groups);
  } else {
    const bool tail = a.K % Unit<BF16>::EPU != 0;
    void (*kernel)(Grad) = nullptr;
#define SHAPE(L, C) kernel = tail ? rms_norm_grad_kernel<BF16, WBF16, true, L, C> : rms_norm_grad_kernel<BF16, WBF16, false, L, C>
    if (p.lanes == 16) SHAPE(16, 1);
    else if (p.lanes == 32) SHAPE(32, 1);
    else if (p.lanes == 64) SHAPE(64, 1);
    else if (ceil_div(a.K, Unit<BF16>::EPU) <= 1024) SHAPE(0, 1);
    else SHAPE(0, 2);
#undef SHAPE
    e = launch(kernel, p.groups, p.block, s, g);
  }
  if (e != hipSuccess || !a.dW) return e;
  return launch(rms_norm_weight_kernel<WBF16>, std::min<int64_t>(ceil_div(a.K, 16), 1 << 16), 1024, s, (int)p.groups, (int)a.K,
                static_cast<const float*>(P), a.dW);
}

}  // namespace

int64_t rms_norm_grad_bytes(int64_t rows, int64_t K, bool bf16) {
  const Plan p = plan_of(rows, K, bf16);
  return (p.block ? 0 : sums_bytes(rows)) + p.groups * K * 4;
}

hipError_t launch_rms_norm_grad(const NormGradArgs& a, hipStream_t s) {
  if (a.bf16) return a.w_bf16 ? launch_grad<true, true>(a, s) : launch_grad<true, false>(a, s);
  return a.w_bf16 ? launch_grad<false, true>(a, s) : launch_grad<false, false>(a, s);
}

}  // namespace fp4g
