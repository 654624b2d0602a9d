// The products of int8 and bf16 operands that a feed-forward block takes, on the tiles of
// dense_tile.hpp: which tile and K split a product gets, the launches, and the end of a split
// product.
#include <algorithm>

#include "dense_tile.hpp"
#include "launch.hpp"

namespace fp4g {
namespace {

template <class C, bool BF16, bool SAVE, bool SPLIT>
__global__ void __launch_bounds__(C::NW * 64, C::NW * C::OCC / 4) dense_gemm_kernel(const DenseArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  dense_gemm<C, BF16, SAVE, SPLIT>(a, blockIdx.x, gridDim.x, smem);
}

// Both backward products in one launch: workgroups 0 .. split-1 take the items of x (dX), the
// others those of w (dWg and dWu).  They need the same operands and neither fills the GPU
// where they are small.
template <class CX, class CW, bool SPLITX>
__global__ void __launch_bounds__(CX::NW * 64, CX::NW * CX::OCC / 4)
dense_grads_kernel(const DenseArgs x, const DenseArgs w, int split) {
  static_assert(CX::NW == CW::NW && CX::LDS == CW::LDS && CX::OCC == CW::OCC, "one launch shape");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[CX::LDS];
  const int b = blockIdx.x;
  if (b < split) dense_gemm<CX, true, false, SPLITX>(x, b, split, smem);
  else dense_gemm<CW, true, false, false>(w, b - split, gridDim.x - split, smem);
}

// The end of a split product: sums of the S slices in slice order, then what the unsplit
// kernel does with its sums.  HBM-bound: S (times 2 when gated) 32-bit values in, one out.
// Rows of partial sums are padded to whole groups of 4, one group a lane.
template <class T, bool GATED, bool BF16, bool SAVE>
__global__ void __launch_bounds__(256) dense_reduce_kernel(const DenseArgs a) {
  typedef typename std::conditional<std::is_same<T, I8>::value, v4i, v4f>::type sum4;
  constexpr int W = GATED ? 2 : 1;
  const uint32_t groups = (uint32_t)(partial_pitch(a.N) / 4), per = (uint32_t)a.M * groups;
  for (uint32_t x = blockIdx.x * 256 + threadIdx.x; x < per * a.L; x += gridDim.x * 256) {
    const uint32_t l = x / per, in = x - l * per, m = in / groups, n = (in - m * groups) * 4;
    const sum4* p = static_cast<const sum4*>(a.P) + (int64_t)l * a.S * W * per + in;
    sum4 s[W];
#pragma unroll
    for (int w = 0; w < W; ++w) s[w] = p[(int64_t)w * per];
#pragma unroll 4
    for (int k = 1; k < a.S; ++k)
#pragma unroll
      for (int w = 0; w < W; ++w) s[w] += p[((int64_t)k * W + w) * per];
    float y[4], u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e] = (float)s[0][e];
      u[e] = (float)s[W - 1][e];
      if constexpr (std::is_same<T, I8>::value) {
        const int c = min((int)n + e, a.N - 1);
        y[e] = y[e] * a.sa[m] * a.sb[0][c];
        if constexpr (GATED) u[e] = u[e] * a.sa[m] * a.sb[1][c];
      }
    }
    const int64_t at = (int64_t)m * a.N + n;
    const int left = a.N - (int)n;
    if constexpr (GATED) {
      if constexpr (SAVE) {
        store_cols<false>(a.G, at, left, y);
        store_cols<false>(a.U, at, left, u);
      }
      gate(a.act, y, u);
    }
    store_cols<BF16>(a.D[l], at, left, y);
  }
}

template <class T, bool GATED, bool BF16, bool SAVE>
hipError_t launch_reduce(const DenseArgs& a, hipStream_t s) {
  const int64_t units = ceil_div(a.L * a.M * (partial_pitch(a.N) / 4), 256);
  const unsigned grid = (unsigned)std::min<int64_t>(units, device_cus() * 8);
  return launch(dense_reduce_kernel<T, GATED, BF16, SAVE>, grid, 256, s, a);
}

template <class C, bool BF16, bool SAVE>
hipError_t launch_tiles(const DenseArgs& a, hipStream_t s) {
  const int64_t items = a.L * ceil_div(a.M, C::BM) * ceil_div(a.N, C::OUTN) * a.S;
  if (items > INT32_MAX / 2) return hipErrorInvalidConfiguration;
  const unsigned grid = (unsigned)std::min<int64_t>(items, device_cus() * C::OCC);
  if (a.S > 1) {
    const hipError_t e = launch(dense_gemm_kernel<C, false, false, true>, grid, C::NW * 64, s, a);
    if (e != hipSuccess) return e;
    return launch_reduce<typename C::T, C::GATED, BF16, SAVE>(a, s);
  }
  return launch(dense_gemm_kernel<C, BF16, SAVE, false>, grid, C::NW * 64, s, a);
}

typedef Tiles<BF, kPlain, false, true, 2> GradInput;    // dX = [dG dU] [Wg; Wu]: A rows hold K, B rows are K
typedef Tiles<BF, kPlain, true, true, 1> GradWeights;   // dWg = dG^T X, dWu = dU^T X: both operands' rows are K

template <class S, bool BF16, bool SAVE>
hipError_t launch_cfg(const DenseArgs& a, DenseTile tile, hipStream_t s) {
  switch (tile) {
    case kTile256: return launch_tiles<typename S::t256, BF16, SAVE>(a, s);
    case kTile128: return launch_tiles<typename S::t128, BF16, SAVE>(a, s);
    case kTile128Deep: return launch_tiles<typename S::t128_deep, BF16, SAVE>(a, s);
    case kTile64x128: return launch_tiles<typename S::t64x128, BF16, SAVE>(a, s);
    case kTile64Deep: return launch_tiles<typename S::t64_deep, BF16, SAVE>(a, s);
    case kTile64: return launch_tiles<typename S::t64, BF16, SAVE>(a, s);
    case kTile64x128Long: return launch_tiles<typename S::t64x128_long, BF16, SAVE>(a, s);
    case kTile64Long: return launch_tiles<typename S::t64_long, BF16, SAVE>(a, s);
    case kGemv: break;
  }
  return hipErrorInvalidConfiguration;
}

template <class CX, class CW>
hipError_t launch_both(const DenseArgs& x, const DenseArgs& w, hipStream_t s) {
  const int64_t slots = device_cus() * CX::OCC;
  const int64_t nx = x.S * ceil_div(x.M, CX::BM) * ceil_div(x.N, CX::OUTN);
  const int64_t nw = w.L * ceil_div(w.M, CW::BM) * ceil_div(w.N, CW::OUTN);
  if (nx > INT32_MAX / 2 || nw > INT32_MAX / 2) return hipErrorInvalidConfiguration;
  // A multiple of 8 workgroups for x, so that the others' ids keep their XCDs.
  const int split = (int)(ceil_div(std::min(nx, slots), 8) * 8);
  const unsigned grid = (unsigned)(split + std::min(nw, slots));
  if (x.S == 1) return launch(dense_grads_kernel<CX, CW, false>, grid, CX::NW * 64, s, x, w, split);
  const hipError_t e = launch(dense_grads_kernel<CX, CW, true>, grid, CX::NW * 64, s, x, w, split);
  return e != hipSuccess ? e : launch_reduce<BF, false, true, false>(x, s);
}

struct Tile { DenseTile t; int64_t bm, bn, occ; double us[3], item; };
const Tile kTiles[] = {{kTile256, 256, 256, 1, {1.84}, 5.1},
                       {kTile128, 128, 128, 2, {0.86, 1.20}, 2.0},
                       {kTile128Deep, 128, 128, 1, {0.56}, 3.7},
                       {kTile64x128, 64, 128, 2, {0.36, 0.73}, 2.5},
                       {kTile64Deep, 64, 64, 2, {0.24, 0.50}, 2.4},
                       {kTile64, 64, 64, 3, {0.275, 0.51, 0.68}, 2.1},
                       {kTile64x128Long, 64, 128, 1, {0.326}, 3.2},
                       {kTile64Long, 64, 64, 1, {0.211}, 2.9}};

int64_t items_of(const Tile& c, int64_t rows, int64_t cols, int64_t L) {
  return L * ceil_div(rows, c.bm) * ceil_div(cols, c.bn);
}
double split_us(int64_t rows, int64_t cols, int64_t L, int64_t S) {
  return S > 1 ? 2.7 + (double)(L * rows * cols) * (double)(2 * S + 1) * 4.0 / 6.7e6 : 0.0;
}
// A slice holds at least 4 stages; the reduction's indexes are 32 bits.
bool can_split(int64_t rows, int64_t cols, int64_t L, int64_t KT, int64_t S, int64_t cap) {
  return S == 1 || (S <= std::min<int64_t>(cap, kMaxSplits) && KT / S >= 4 && L * rows * (cols + 8) < (int64_t)1 << 31);
}

}  // namespace

// Tile and K split of a product with `rows` x `cols` sums (gated: cols = 2 N), L of them,
// each a sum of KT stages of 128 bytes: the pair with the least modelled time.  A round of
// items, n to a CU, takes us[n-1] for each stage and `item` for its start and end; a split
// adds a launch and the partial sums' way through memory.  The figures are fitted to the
// measured times of 33 sizes of all five products, M = 20 .. 8192 (every tile, S = 1, 2, 4,
// 8); on those the pair it picks is the fastest measured or within 3% of it.  What the tiles
// are for, in us:
//   int8 8192^3: 256^2 477, 128^2 593, 64 x 128 731, 64^2 907
//   int8 2048 x 4096 x 4096: 128^2 44.2, 256^2 58.8, 64 x 128 53.0
//   int8 200 x 14336 x 4096: 128^2 of two groups 26.8, 128^2 38.0, 64 x 128 30.6
//   int8 1003 x 1117 x 1040: 64 x 128 9.1, 128^2 13.7, 64^2 9.8
//   int8 256 x 8192 x 8192: 64 x 128 with 256-byte stages 32.9, with 128-byte stages 37.1
//   int8 128 x 4096 x 4096: 64^2 with 256-byte stages 11.0, with 5 of 128 bytes 12.7, 64 x 128 16.7
//   int8 100 x 1000 x 1024: 64^2 of 3 stages 6.2, of 5 stages 6.6, 64 x 128 7.3
//   bf16 gated 128 x 4096 x 2048: 64^2 of 5 stages 15.5, of 3 stages 18.3
DensePlan dense_plan_among(uint32_t tiles, int64_t rows, int64_t cols, int64_t L, int64_t KT, int64_t cap) {
  const int64_t cus = device_cus();
  DensePlan best{kTile64, 1, 1e30};
  for (const Tile& c : kTiles)
    for (int64_t S : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (!(tiles >> c.t & 1) || !can_split(rows, cols, L, KT, S, cap)) break;
      const int64_t items = items_of(c, rows, cols, L) * S, full = items / (cus * c.occ), rest = items % (cus * c.occ);
      const double stages = (double)ceil_div(KT, S);
      double t = split_us(rows, cols, L, S) + (double)full * (stages * c.us[c.occ - 1] + c.item);
      if (rest) t += stages * c.us[ceil_div(rest, cus) - 1] + c.item;
      if (t < best.us) best = DensePlan{c.t, (int)S, t};
    }
  return best;
}

DensePlan dense_plan(int64_t rows, int64_t cols, int64_t L, int64_t KT, int64_t cap) {
  return dense_plan_among(~0u, rows, cols, L, KT, cap);
}

// Both backward products in one launch, dX with S slices: the chip's throughput over all their
// items, or the longest item, whichever is more.  Taken where that beats the two launches
// and the microsecond or two between them.
GradPlan grad_plan(int64_t M, int64_t N, int64_t K, int64_t cap_x, int64_t cap_w) {
  const int64_t cus = device_cus(), KX = 2 * ceil_div(N, 64), KW = ceil_div(M, 64);
  GradPlan best{dense_plan(M, K, 1, KX, cap_x), dense_plan(N, K, 2, KW, cap_w), false};
  double best_t = best.x.us + best.w.us + 1.5;
  for (const Tile& c : kTiles) {
    if (c.t != kTile64 && c.t != kTile64Deep && c.t != kTile64x128) continue;
    for (int64_t S = 1; can_split(M, K, 1, KX, S, cap_x); S *= 2) {
      const int64_t nx = items_of(c, M, K, 1) * S, nw = items_of(c, N, K, 2);
      const double sx = (double)ceil_div(KX, S), sw = (double)KW, us = c.us[c.occ - 1];
      const double all = ((double)nx * (sx * us + c.item) + (double)nw * (sw * us + c.item)) / (double)(cus * c.occ);
      const double one = std::max(sx, sw) * c.us[std::min<int64_t>(c.occ, ceil_div(nx + nw, cus)) - 1] + c.item;
      const double t = std::max(all, one) + split_us(M, K, 1, S);
      if (t < best_t) {
        best_t = t;
        best = GradPlan{{c.t, (int)S, t}, {c.t, 1, t}, true};
      }
    }
  }
  return best;
}

hipError_t launch_partial_sums(const DenseArgs& a, bool int8, bool gated, hipStream_t s) {
  if (!int8) return a.G ? launch_reduce<BF, true, true, true>(a, s) : launch_reduce<BF, true, true, false>(a, s);
  if (gated)
    return a.bf16_out ? launch_reduce<I8, true, true, false>(a, s) : launch_reduce<I8, true, false, false>(a, s);
  return a.bf16_out ? launch_reduce<I8, false, true, false>(a, s) : launch_reduce<I8, false, false, false>(a, s);
}

hipError_t launch_w8a8(const DenseArgs& a, DenseTile tile, hipStream_t s) {
  if (tile == kGemv) return launch_gemv_w8a8(a, s);
  return a.bf16_out ? launch_cfg<Tiles<I8, kScaled, false, false, 1>, true, false>(a, tile, s)
                    : launch_cfg<Tiles<I8, kScaled, false, false, 1>, false, false>(a, tile, s);
}

hipError_t launch_w8a8_gated(const DenseArgs& a, DenseTile tile, hipStream_t s) {
  if (tile == kGemv) return launch_gemv_w8a8_gated(a, s);
  return a.bf16_out ? launch_cfg<Tiles<I8, kGated, false, false, 1>, true, false>(a, tile, s)
                    : launch_cfg<Tiles<I8, kGated, false, false, 1>, false, false>(a, tile, s);
}

hipError_t launch_gated(const DenseArgs& a, DenseTile tile, hipStream_t s) {
  if (tile == kGemv) return launch_gemv_gated(a, s);
  return a.G ? launch_cfg<Tiles<BF, kGated, false, false, 1>, true, true>(a, tile, s)
             : launch_cfg<Tiles<BF, kGated, false, false, 1>, true, false>(a, tile, s);
}

hipError_t launch_grads(const DenseArgs& x, const DenseArgs& w, const GradPlan& p, hipStream_t s) {
  if (!p.merged) {
    const hipError_t e = launch_cfg<GradInput, true, false>(x, p.x.tile, s);
    return e != hipSuccess ? e : launch_cfg<GradWeights, true, false>(w, p.w.tile, s);
  }
  switch (p.x.tile) {
    case kTile64x128: return launch_both<GradInput::t64x128, GradWeights::t64x128>(x, w, s);
    case kTile64Deep: return launch_both<GradInput::t64_deep, GradWeights::t64_deep>(x, w, s);
    case kTile64: return launch_both<GradInput::t64, GradWeights::t64>(x, w, s);
    default: return hipErrorInvalidConfiguration;
  }
}

}  // namespace fp4g
