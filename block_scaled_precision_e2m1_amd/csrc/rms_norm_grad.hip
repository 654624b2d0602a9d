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
template <bool BF16>
__device__ __forceinline__ v4u grad_unit(const v4u& dy, const v4u& x, const float (&w)[Unit<BF16>::EPU], const v4u& dh,
                                         float s, float c) {
  typedef Unit<BF16> U;
  float d[U::EPU];
#pragma unroll
  for (int e = 0; e < U::EPU; ++e) d[e] = s * (U::at(dy, e) * w[e] - U::at(x, e) * c) + U::at(dh, e);
  return U::pack(d);
}

// The two sums of a row, in 64 bits and 32.
struct Sums {
  double xx;
  float gx;
};
struct AddSums {
  __device__ __forceinline__ Sums operator()(Sums a, Sums b) const { return Sums{a.xx + b.xx, a.gx + b.gx}; }
};
__device__ __forceinline__ Sums lane_xor(Sums v, int d) { return Sums{fp4g::lane_xor(v.xx, d), fp4g::lane_xor(v.gx, d)}; }

template <bool BF16>
__device__ __forceinline__ void add_unit(const v4u& dy, const v4u& x, const float (&w)[Unit<BF16>::EPU], Sums* t) {
  typedef Unit<BF16> U;
#pragma unroll
  for (int e = 0; e < U::EPU; ++e) {
    const double v = U::at(x, e);
    t->xx = __builtin_fma(v, v, t->xx);
    t->gx += U::at(dy, e) * w[e] * U::at(x, e);
  }
}

// dX may be dY or dH: a row's units are stored by the lanes that read them, after their loads.
template <bool BF16, bool WBF16, int L, int C>
__global__ void __launch_bounds__(L < 256 ? 256 : L) rms_norm_grad_kernel(const Grad a) {
  typedef Unit<BF16> U;
  constexpr int EPU = U::EPU, NT = L < 256 ? 256 : L, RPW = NT / L;
  __shared__ Sums parts[2][NT / 64];
  __shared__ float columns[RPW > 1 ? NT * EPU * C : 1];
  const int lane = threadIdx.x % L, sub = threadIdx.x / L, units = ((uint32_t)a.K + EPU - 1) / EPU;
  float w[C][EPU], dw[C][EPU];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_weight<WBF16>(a.W, (int64_t)(lane + c * L) * EPU, a.K, w[c]);
#pragma unroll
    for (int e = 0; e < EPU; ++e) dw[c][e] = 0.0f;
  }
  const v4u none{0, 0, 0, 0};
  auto fetch = [&](const uint8_t* p, int64_t row, v4u(&v)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int u = lane + c * L;
      v[c] = p && u < units && row < a.rows ? U::template load<true>(p + row * a.K * U::ELEM, (int64_t)u * EPU, a.K)
                                            : none;
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPW;
  // 16 waves of two units a lane have no registers for a second row.
  constexpr bool AHEAD = L < 1024 || C == 1;
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
#pragma unroll
    for (int c = 0; c < C; ++c) add_unit<BF16>(dy[c], x[c], w[c], &t);
    // Two sets of parts in turn: a wave is at most one row ahead of another's reads.
    t = over_row<L>(t, AddSums{}, parts[turn]);
    const float s = inv_sqrt(t.xx / (double)a.K + a.eps), k = s * s * (t.gx / (float)a.K);
    const int64_t at = row * a.K * U::ELEM;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int u = lane + c * L;
      if (u < units && row < a.rows) {
        U::store(a.dX + at, (int64_t)u * EPU, a.K, grad_unit<BF16>(dy[c], x[c], w[c], dh[c], s, k));
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
    for (int k = threadIdx.x; k < a.K; k += NT) {
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
        const int64_t k = (int64_t)(lane + c * L) * EPU + e;
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
      float w[U::EPU];
      load_weight<WBF16>(a.W, first, a.K, w);
      add_unit<BF16>(U::load(a.dY + at, first, a.K), U::load(a.X + at, first, a.K), w, &t);
    }
    t = over_row<1024>(t, AddSums{}, parts[turn]);
    if (threadIdx.x == 0) {
      const float s = inv_sqrt(t.xx / (double)a.K + a.eps);
      a.S[2 * row] = s;
      a.S[2 * row + 1] = s * s * (t.gx / (float)a.K);
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
  float w[EPU], dw[EPU] = {};
  load_weight<WBF16>(a.W, first, a.K, w);
  const int64_t end = a.rows * (share + 1) / shares;
  for (int64_t row = a.rows * share / shares; row < end; ++row) {
    const int64_t at = row * a.K * U::ELEM;
    const v4u dy = U::load(a.dY + at, first, a.K), x = U::load(a.X + at, first, a.K);
    const v4u dh = a.dH ? U::load(a.dH + at, first, a.K) : v4u{0, 0, 0, 0};
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

// dW of 32 columns a workgroup: the partial sums in eight runs of rows, added in order.
template <bool BF16>
__global__ void __launch_bounds__(256) rms_norm_weight_kernel(int shares, int K, const float* __restrict__ P, void* dW) {
  __shared__ float sums[8][32];
  const int c = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int first = (int)((int64_t)shares * run / 8), end = (int)((int64_t)shares * (run + 1) / 8);
  for (int64_t k0 = (int64_t)blockIdx.x * 32; k0 < K; k0 += (int64_t)gridDim.x * 32) {
    const int64_t k = k0 + c;
    float sum = 0.0f;
    if (k < K) {
#pragma unroll 8
      for (int r = first; r < end; ++r) sum += P[(int64_t)r * K + k];
    }
    sums[run][c] = sum;
    __syncthreads();
    if (run == 0 && k < K) {
#pragma unroll
      for (int r = 1; r < 8; ++r) sum += sums[r][c];
      store_out<BF16>(dW, k, sum);
    }
    __syncthreads();
  }
}

// Lanes and units a lane: the first shape that holds the row.
#define FP4G_GRAD_SHAPES(F) \
  F(16, 16, 1) F(32, 32, 1) F(64, 64, 1) F(128, 128, 1) F(256, 256, 1) F(512, 512, 1) F(1024, 1024, 1) F(2048, 1024, 2)

struct Plan { int lanes; int64_t groups; };   // lanes 0: a long row, of `groups` shares of rows
Plan plan_of(int64_t rows, int64_t K, bool bf16) {
  const int64_t units = ceil_div(K, bf16 ? 8 : 4), cus = device_cus();
  int lanes = 0;
#define PICK(U, L, C) else if (units <= U) lanes = L;
  if (false) {}
  FP4G_GRAD_SHAPES(PICK)
#undef PICK
  // Enough workgroups for the chip, more only where their partial sums (8 bytes a column, for
  // 6 and more of each row) stay a small part.
  if (lanes == 0) return {0, std::max<int64_t>(1, std::min<int64_t>({rows, 64, 4 * cus / ceil_div(units, 256) + 1}))};
  const int64_t per = lanes < 256 ? 256 / lanes : 1, most = lanes > 512 ? cus : lanes > 256 ? 2 * cus : 4 * cus;
  return {lanes, std::max<int64_t>(1, std::min(ceil_div(rows, per), std::max(cus, std::min(most, rows / 16))))};
}
int64_t sums_bytes(int64_t rows) { return (rows * 8 + 15) / 16 * 16; }

template <bool BF16, bool WBF16>
hipError_t launch_grad(const NormGradArgs& a, hipStream_t s) {
  const Plan p = plan_of(a.rows, a.K, BF16);
  Grad g{a.rows, (int)a.K, static_cast<const uint8_t*>(a.dY), static_cast<const uint8_t*>(a.X),
         static_cast<const uint8_t*>(a.dH), a.W, static_cast<uint8_t*>(a.dX), nullptr, nullptr, a.eps};
  float* const P = reinterpret_cast<float*>(static_cast<uint8_t*>(a.P) + (p.lanes ? 0 : sums_bytes(a.rows)));
  if (a.dW) g.P = P;
  hipError_t e = hipSuccess;
  if (p.lanes == 0) {
    g.S = static_cast<float*>(a.P);
    const int blocks = (int)ceil_div(ceil_div(a.K, Unit<BF16>::EPU), 256);
    e = launch(rms_norm_grad_sums_kernel<BF16, WBF16>, std::min(a.rows, 8 * device_cus()), 1024, s, g);
    if (e == hipSuccess)
      e = launch(rms_norm_grad_columns_kernel<BF16, WBF16>, blocks * p.groups, 256, s, g, blocks, (int)p.groups);
  }
#define RUN(U, L, C) else if (p.lanes == L && ceil_div(a.K, Unit<BF16>::EPU) <= U) \
    e = launch(rms_norm_grad_kernel<BF16, WBF16, L, C>, p.groups, L < 256 ? 256 : L, s, g);
  FP4G_GRAD_SHAPES(RUN)
#undef RUN
  if (e != hipSuccess || !a.dW) return e;
  return launch(rms_norm_weight_kernel<WBF16>, std::min<int64_t>(ceil_div(a.K, 32), 1 << 16), 256, s, (int)p.groups, (int)a.K,
                static_cast<const float*>(P), a.dW);
}

}  // namespace

int64_t rms_norm_grad_bytes(int64_t rows, int64_t K, bool bf16) {
  const Plan p = plan_of(rows, K, bf16);
  return (p.lanes ? 0 : sums_bytes(rows)) + p.groups * K * 4;
}

hipError_t launch_rms_norm_grad(const NormGradArgs& a, hipStream_t s) {
  if (a.bf16) return a.w_bf16 ? launch_grad<true, true>(a, s) : launch_grad<true, false>(a, s);
  return a.w_bf16 ? launch_grad<false, true>(a, s) : launch_grad<false, false>(a, s);
}

}  // namespace fp4g
