// The softmax cross entropy over a vocabulary for gfx950, without the logits in memory, and its
// gradients:
//   z = X W^T,  lse[m] = log sum_v e^z[m][v],  loss[m] = lse[m] - z[m][target[m]]
//   P = (e^(z - lse) - [v == target]) dL,  dX = P W,  dW = P^T X
//
// Bound by the matrix instructions: 2 M V K operations forward and 6 M V K for the gradients, of
// which 2 form the logits again; M counts the rows that take part.  The products are those of
// dense_tile.hpp:
//
//   * Forward, a tile's end leaves the maximum and the sum of the exponentials of each row over
//     a wave's columns (8 bytes for 64 or 128 logits), and a last kernel joins them.
//   * Backward, the vocabulary is taken in pieces.  A piece's logits are formed again and leave
//     their tiles as P in bf16, the operand of both gradients' products; dW's rows of the piece are
//     then whole, and dX is summed over the pieces in fp32.  For up to kFewRows rows P has two
//     terms, and the gradients' products twice the length: 10 M V K.
//   * Rows without a loss (a prompt's tokens, padding): the rows that have one are gathered first,
//     their number stays on the GPU, and the tiles read it there.  Half of the rows ignored is
//     half of the products.  The gathering copy moves 4 M K bytes.  A small forward product
//     (loss_gathers) takes every row as it is, and what an ignored row gives is left out of
//     the results.  Either way what it holds reaches nothing.
#include <algorithm>

#include "dense_tile.hpp"
#include "launch.hpp"
#include "lm_internal.h"

namespace fp4g {
namespace {

// ---- the rows that take part ----

struct Pick {
  int64_t M, K;                   // K: a multiple of 8
  int64_t V, ignore;
  const int64_t* target;
  const v4i* X;
  const int* counts;              // rows that take part among each 1024, or null: count them here
  v4i* rows;                      // [M][K] those rows, in order
  int *map, *wanted, *count;      // which row each was, its target or -1, and their number
  float *loss, *lse;              // forward: 0 for the rows that take no part
  float* z;                       // forward: the wanted logit, NaN until it is found
  const float* tops;              // backward: with counts, the largest |dL| among each 1024
  float* unscale;                 // backward: what the gradients' products are multiplied by
  const float *dL, *lse_in;       // backward: taken to the rows that take part
  float *g, *lse_out;
  v4i* dX;                        // backward: 0 for the rows that take no part
};
constexpr int kChunk = 1024;

// The sum of n and the maximum of top over a workgroup of 4 waves.
struct Seen { int n; float top; };
__device__ __forceinline__ Seen over_block(Seen v, Seen* part) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    v.n += __shfl_xor(v.n, d);
    v.top = fmaxf(v.top, __shfl_xor(v.top, d));
  }
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) v.n += part[w].n, v.top = fmaxf(v.top, part[w].top);
  return v;
}

// P is rounded to bf16 once dL is in it, and is mostly p - 1 times dL at the wanted tokens.  A mean
// gives one dL to all rows: where they know little, p near 0, all of their roundings would be
// that of dL itself, and the gradients off by up to 0.004 of their norm (1 / 1020, 1 / 4095), where their
// own rounding is 0.0017.  So all dL are divided by one number of 1 .. 2 that takes the largest of them
// down to a power of two, and the products multiplied by it at the end: no sum is larger for it.
__device__ __forceinline__ float unscale_of(float top) {
  if (top < 0x1p-126f) return 1.0f;   // nothing to scale, or nothing to scale it by
  return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, top) & 0x7fffffu) | 0x3f800000u);
}
__device__ __forceinline__ float top_of(float dl) {
  const float m = __builtin_fabsf(dl);
  return m < __builtin_inff() ? m : 0.0f;
}

template <bool GRAD>
__global__ void __launch_bounds__(256) loss_count_kernel(int64_t M, int64_t ignore, const int64_t* __restrict__ target,
                                                         const float* __restrict__ dL, int* __restrict__ counts,
                                                         float* __restrict__ tops) {
  __shared__ Seen part[4];
  const int64_t first = (int64_t)blockIdx.x * kChunk;
  Seen v{0, 0.0f};
#pragma unroll
  for (int i = 0; i < kChunk / 256; ++i) {
    const int64_t m = first + i * 256 + threadIdx.x;
    const bool in = m < M && target[m] != ignore;
    v.n += in;
    if constexpr (GRAD)
      if (in) v.top = fmaxf(v.top, top_of(dL[m]));
  }
  v = over_block(v, part);
  if (threadIdx.x == 0) {
    counts[blockIdx.x] = v.n;
    if constexpr (GRAD) tops[blockIdx.x] = v.top;
  }
}

// A wave for each of 4 rows, or (ROWS == 1) the workgroup for one: how many before take part is
// counted by the whole workgroup, in the rows' chunk alone where the chunks before it are
// counted already.  A row's copy is under way before the count is known.
template <bool GRAD, int ROWS>
__global__ void __launch_bounds__(256) loss_pick_kernel(const Pick a) {
  constexpr int LANES = 256 / ROWS, AHEAD = 4;
  __shared__ Seen part[4];
  const int lane = threadIdx.x % LANES, mine = threadIdx.x / LANES;
  const int64_t row0 = (int64_t)blockIdx.x * ROWS, m = row0 + mine, units = a.K / 8;
  bool in[ROWS], here = false;
#pragma unroll
  for (int w = 0; w < ROWS; ++w) {
    in[w] = row0 + w < a.M && a.target[row0 + w] != a.ignore;
    here |= w == mine && in[w];
  }
  const v4i* x = a.X + m * units;
  v4i held[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (here && lane + i * LANES < units) held[i] = x[lane + i * LANES];
  Seen seen{0, 0.0f};
  int64_t from = 0;
  if (a.counts) {
    from = row0 / kChunk * kChunk;
    for (int64_t c = threadIdx.x; c < row0 / kChunk; c += 256) seen.n += a.counts[c];
    if constexpr (GRAD)
      for (int64_t c = threadIdx.x; c * kChunk < a.M; c += 256) seen.top = fmaxf(seen.top, a.tops[c]);
  }
  // With the largest |dL| of all rows to be found, all of their targets are looked at.
  const int64_t to_row = GRAD && !a.counts ? a.M : row0;
#pragma unroll 4
  for (int64_t i = from + threadIdx.x; i < to_row; i += 256) {
    const bool in = a.target[i] != a.ignore;
    seen.n += in && i < row0;
    if constexpr (GRAD)
      if (in && !a.counts) seen.top = fmaxf(seen.top, top_of(a.dL[i]));
  }
  seen = over_block(seen, part);
  int slot = seen.n, last = seen.n;
#pragma unroll
  for (int w = 0; w < ROWS; ++w) {
    slot += w < mine && in[w];
    last += in[w];
  }
  if (row0 + ROWS >= a.M && threadIdx.x == 0) {
    *a.count = last;
    if constexpr (GRAD) *a.unscale = unscale_of(seen.top);
  }
  if (m >= a.M) return;
  if (!here) {
    if constexpr (GRAD) {
      if (a.dX)
        for (int64_t u = lane; u < units; u += LANES) a.dX[m * units + u] = v4i{0, 0, 0, 0};
    } else if (lane == 0) {
      a.loss[m] = 0.0f;
      if (a.lse) a.lse[m] = 0.0f;
    }
    return;
  }
  v4i* to = a.rows + slot * units;
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (lane + i * LANES < units) to[lane + i * LANES] = held[i];
#pragma unroll 4
  for (int64_t u = lane + AHEAD * LANES; u < units; u += LANES) to[u] = x[u];
  if (lane == 0) {
    const int64_t t = a.target[m];
    const bool known = t >= 0 && t < a.V;
    a.map[slot] = (int)m;
    a.wanted[slot] = known ? (int)t : -1;
    if constexpr (GRAD) {
      a.g[slot] = known ? a.dL[m] * (1.0f / unscale_of(seen.top)) : __builtin_nanf("");
      a.lse_out[slot] = a.lse_in[m];
    } else {
      a.z[slot] = __builtin_nanf("");
    }
  }
}

hipError_t launch_pick(Pick p, int* counts, float* tops, bool grad, hipStream_t s) {
  // Up to 4096 targets (32 KB) are counted by every workgroup for itself.  Backward passes over 128
  // tokens, in us, so and in chunks: 2048 x 256 20.0 22.2, 4096 x 256 29.4 30.2, 4096 x 4096 68.4 66.1,
  // 6000 x 256 38.7 36.4, 8192 x 256 53.4 44.7; forward passes differ by less.
  if (p.M > 4096) {
    const hipError_t e = launch(grad ? loss_count_kernel<true> : loss_count_kernel<false>, ceil_div(p.M, kChunk), 256, s, p.M,
                                p.ignore, p.target, p.dL, counts, tops);
    if (e != hipSuccess) return e;
    p.counts = counts, p.tops = tops;
  }
  // Few rows are spread over the chip: 16 x 4096 take 3 us a row to a workgroup, 7 four to one.  Whole
  // backward passes over 128 tokens: 1024 x 4096 38.7 39.7, 2048 x 4096 51.1 48.5, 2048 x 512 26.1 23.1.
  if (p.M <= 1024) return launch(grad ? loss_pick_kernel<true, 1> : loss_pick_kernel<false, 1>, p.M, 256, s, p);
  return launch(grad ? loss_pick_kernel<true, 4> : loss_pick_kernel<false, 4>, ceil_div(p.M, 4), 256, s, p);
}

// ---- forward ----

// e^(a - b) of a part and its share of a row: of two parts at -infinity 0, their sums are 0 too.
__device__ __forceinline__ float2 join(float2 x, float2 y) {
  const float most = fmaxf(x.x, y.x), from = most == -__builtin_inff() ? 0.0f : most;
  return make_float2(most, x.y * __builtin_amdgcn_exp2f((x.x - from) * kLog2e) +
                               y.y * __builtin_amdgcn_exp2f((y.x - from) * kLog2e));
}

// The parts of a row joined, ROWS rows a workgroup: every 256 / ROWS th part a thread, then the
// threads of a row in pairs.
struct Join {
  int64_t M;
  int parts;
  const float2* part;             // [parts][M]
  const float* z;                 // [M] the wanted logits
  const int *count, *map;         // rows that were gathered and where they were, or null: every row is there,
  const int64_t* target;          // and its target says what becomes of it
  int64_t V, ignore;
  float *loss, *lse;
};
template <int ROWS>
__global__ void __launch_bounds__(256) loss_join_kernel(const Join a) {
  constexpr int Q = 256 / ROWS;
  __shared__ float2 held[Q][ROWS + 1];
  const int r = threadIdx.x % ROWS, q = threadIdx.x / ROWS;
  const int64_t m = (int64_t)blockIdx.x * ROWS + r, rows = a.count ? *a.count : a.M;
  if ((int64_t)blockIdx.x * ROWS >= rows) return;
  const bool there = m < rows;
  float2 all = make_float2(-__builtin_inff(), 0.0f);
  if (there) {
    for (int p = q; p < a.parts; p += 8 * Q) {
      float2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = p + i * Q < a.parts ? a.part[(int64_t)(p + i * Q) * a.M + m] : make_float2(-__builtin_inff(), 0.0f);
#pragma unroll
      for (int d = 4; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < d; ++i) v[i] = join(v[i], v[i + d]);
      all = join(all, v[0]);
    }
  }
  held[q][r] = all;
#pragma unroll
  for (int d = Q / 2; d > 0; d /= 2) {
    __syncthreads();
    if (q < d) held[q][r] = join(held[q][r], held[q + d][r]);
  }
  if (q == 0 && there) {
    all = held[0][r];
    const float l = logf(all.y);
    // (maximum - z) first: it is small where the loss is.
    float loss, lse = all.x + l;
    int64_t row = m;
    if (a.count) {
      row = a.map[m];
      loss = (all.x - a.z[m]) + l;
    } else {
      const int64_t t = a.target[m];
      loss = t >= 0 && t < a.V ? (all.x - a.z[m]) + l : __builtin_nanf("");
      if (t == a.ignore) loss = lse = 0.0f;
    }
    a.loss[row] = loss;
    if (a.lse) a.lse[row] = lse;
  }
}

template <class C, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(C::NW * 64, C::NW * C::OCC / 4) loss_gemm_kernel(const LossArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  dense_gemm<C, BF16, false, SPLIT>(a, blockIdx.x, gridDim.x, smem);
}

// Both gradients' products over all of a small vocabulary in one launch: workgroups 0 .. split-1
// take dX's items, the others dW's.  They need the same operands, and neither fills the GPU.
template <class CX, class CW, bool SPLIT>
__global__ void __launch_bounds__(CX::NW * 64, CX::NW * CX::OCC / 4)
loss_grads_kernel(const LossArgs x, const LossArgs w, int split) {
  static_assert(CX::NW == CW::NW && CX::LDS == CW::LDS && CX::OCC == CW::OCC, "one launch shape");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[CX::LDS];
  const int b = blockIdx.x;
  if (b < split) dense_gemm<CX, !SPLIT, false, SPLIT>(x, b, split, smem);
  else dense_gemm<CW, true, false, false>(w, b - split, gridDim.x - split, smem);
}

template <class C, bool BF16, bool SPLIT>
hipError_t launch_tiles(const LossArgs& a, hipStream_t s) {
  const int64_t items = ceil_div(a.M, C::BM) * ceil_div(a.N, C::OUTN) * a.S;
  if (items > INT32_MAX / 2) return hipErrorInvalidConfiguration;
  return launch(loss_gemm_kernel<C, BF16, SPLIT>, std::min<int64_t>(items, device_cus() * C::OCC), C::NW * 64, s, a);
}

// The tiles whose waves have whole sums (one group of waves): the loss's end joins a row's columns
// in registers.
constexpr uint32_t kOneGroup = 1u << kTile256 | 1u << kTile128 | 1u << kTile64x128 | 1u << kTile64x128Long;

template <class S, bool BF16, bool SPLIT>
hipError_t launch_one_group(const LossArgs& a, DenseTile tile, hipStream_t s) {
  switch (tile) {
    case kTile256: return launch_tiles<typename S::t256, BF16, SPLIT>(a, s);
    case kTile128: return launch_tiles<typename S::t128, BF16, SPLIT>(a, s);
    case kTile64x128: return launch_tiles<typename S::t64x128, BF16, SPLIT>(a, s);
    case kTile64x128Long: return launch_tiles<typename S::t64x128_long, BF16, SPLIT>(a, s);
    default: return hipErrorInvalidConfiguration;
  }
}
template <class S, bool BF16, bool SPLIT>
hipError_t launch_any(const LossArgs& a, DenseTile tile, hipStream_t s) {
  switch (tile) {
    case kTile128Deep: return launch_tiles<typename S::t128_deep, BF16, SPLIT>(a, s);
    case kTile64Deep: return launch_tiles<typename S::t64_deep, BF16, SPLIT>(a, s);
    case kTile64: return launch_tiles<typename S::t64, BF16, SPLIT>(a, s);
    case kTile64Long: return launch_tiles<typename S::t64_long, BF16, SPLIT>(a, s);
    default: return launch_one_group<S, BF16, SPLIT>(a, tile, s);
  }
}
typedef Tiles<BF, kLoss, false, false, 1> Forward;       // X W^T: both operands' rows hold K
typedef Tiles<BF, kProb, false, false, 1> Probabilities; // the same
// Of P in one or two bf16 terms, by the rows that take part.
typedef Tiles<BF, kAccum, false, true, 2> GradInput;     // P W: W's rows are the contraction's
typedef Tiles<BF, kCounted, true, true, 2> GradWeights;  // P^T X: both operands' rows are
int terms_of(int64_t M) { return M <= kFewRows ? 2 : 1; }   // with all rows, as products are planned

// The plans of this thread's last products, by their sizes and the GPU's compute units: a call and
// its workspace query ask for the same few several times, and each is chosen in 0.3 to 0.5 us.
DensePlan plan_among(uint32_t tiles, int64_t rows, int64_t cols, int64_t KT, int64_t cap) {
  struct Kept { int64_t key[6]; DensePlan plan; };
  static thread_local Kept kept[8] = {};
  static thread_local unsigned turn = 0;
  const int64_t key[6] = {tiles, rows, cols, KT, cap, device_cus()};
  for (const Kept& k : kept)
    if (std::equal(key, key + 6, k.key)) return k.plan;
  Kept& k = kept[turn++ % 8];
  k.plan = dense_plan_among(tiles, rows, cols, 1, KT, cap);
  std::copy(key, key + 6, k.key);
  return k.plan;
}
DensePlan plan_of(int64_t rows, int64_t cols, int64_t KT, int64_t cap) { return plan_among(~0u, rows, cols, KT, cap); }

DensePlan forward_plan(int64_t M, int64_t V, int64_t K) { return plan_among(kOneGroup, M, V, ceil_div(K, 64), 1); }
int wave_cols(DenseTile t) { return t == kTile256 ? 128 : 64; }

// Parts of a workspace, each on a line of its own.
struct Space {
  uint8_t* p;
  int64_t used = 0;
  template <class T>
  T* take(int64_t count) {
    T* r = reinterpret_cast<T*>(p + used);
    used += (count * (int64_t)sizeof(T) + 255) / 256 * 256;
    return r;
  }
};
struct Picked {
  uint8_t* rows;
  int *map, *wanted, *count, *counts;
  Picked(Space& s, int64_t M, int64_t K)
      : rows(s.take<uint8_t>(M * K * 2)), map(s.take<int>(M)), wanted(s.take<int>(M)), count(s.take<int>(1)),
        counts(s.take<int>(ceil_div(M, kChunk))) {}
};
struct ForwardSpace {
  Space s;
  Picked picked;
  int64_t parts;
  float* z;
  float2* part;
  ForwardSpace(uint8_t* p, int64_t M, int64_t V, int64_t K)
      : s{p}, picked(s, M, K), parts(ceil_div(V, wave_cols(forward_plan(M, V, K).tile))), z(s.take<float>(M)),
        part(s.take<float2>(parts * M)) {}
};

Pick pick_of(const LossCall& a, const Picked& p) {
  Pick k{};
  k.M = a.M, k.K = a.K, k.V = a.V, k.ignore = a.ignore, k.target = a.target;
  k.X = static_cast<const v4i*>(a.X), k.rows = reinterpret_cast<v4i*>(p.rows);
  k.map = p.map, k.wanted = p.wanted, k.count = p.count;
  return k;
}

// ---- backward ----

// The end of dX's split product: the slices in order, what the pieces before gave, and to the
// rows' places at the last piece.
template <bool BF16>
__global__ void __launch_bounds__(256) loss_reduce_kernel(const LossArgs a) {
  const int rows = *a.count, S = splits_of(a, rows);
  const uint32_t groups = (uint32_t)(a.N / 4), total = (uint32_t)rows * groups;
  const int64_t plane = total;
  for (uint32_t x = blockIdx.x * 256 + threadIdx.x; x < total; x += gridDim.x * 256) {
    const uint32_t m = x / groups, n = (x - m * groups) * 4;
    const v4f* p = static_cast<const v4f*>(a.P) + x;
    v4f t = p[0];
#pragma unroll 4
    for (int k = 1; k < S; ++k) t += p[k * plane];
    if (a.add) t += *reinterpret_cast<const v4f*>(a.add + (int64_t)m * a.N + n);
    if constexpr (BF16) t *= *a.unscale;
    const float y[4] = {t[0], t[1], t[2], t[3]};
    store_cols<BF16>(a.D[0], (int64_t)(BF16 ? a.map[m] : (int)m) * a.N + n, 4, y);
  }
}

int64_t tile_rows(DenseTile t) { return t == kTile256 ? 256 : t == kTile128 || t == kTile128Deep ? 128 : 64; }

// Whether one launch on 64 x 64 tiles holds both gradients' items at once: each is then as long as
// its longest item, and the two run side by side.
bool merges(const DensePlan& x, const DensePlan& w, int64_t M, int64_t cols, int64_t K) {
  const int64_t items = (ceil_div(M, 64) * x.S + ceil_div(cols, 64)) * ceil_div(K, 64);
  return tile_rows(x.tile) == 64 && tile_rows(w.tile) == 64 && items + 8 <= device_cus() * GradInput::t64_deep::OCC;
}
hipError_t launch_both(const LossArgs& x, const LossArgs& w, hipStream_t s) {
  typedef GradInput::t64_deep X;
  typedef GradWeights::t64_deep W;
  // A multiple of 8 workgroups for x, so that the others' ids keep their XCDs.
  const int split = (int)(ceil_div(ceil_div(x.M, 64) * ceil_div(x.N, 64) * x.S, 8) * 8);
  const int64_t grid = split + ceil_div(w.M, 64) * ceil_div(w.N, 64);
  return launch(x.S > 1 ? loss_grads_kernel<X, W, true> : loss_grads_kernel<X, W, false>, grid, X::NW * 64, s, x, w, split);
}
// dX's and dW's products over a piece of the vocabulary, where they are wanted; a split dX is left in
// its slices.
hipError_t launch_products(const LossArgs& x, const DensePlan& px, bool last, const LossArgs& w, const DensePlan& pw,
                           bool both, hipStream_t s) {
  if (both) return launch_both(x, w, s);
  hipError_t e = hipSuccess;
  if (x.D[0]) {
    if (px.S > 1) e = launch_any<GradInput, false, true>(x, px.tile, s);
    else if (last) e = launch_any<GradInput, true, false>(x, px.tile, s);
    else e = launch_any<GradInput, false, false>(x, px.tile, s);
  }
  return e == hipSuccess && w.D[0] ? launch_any<GradWeights, true, false>(w, pw.tile, s) : e;
}


}  // namespace

LossInputPlan loss_input_plan(int64_t M, int64_t K, int64_t cols) {
  const int64_t KT = terms_of(M) * ceil_div(cols, 64);
  const DensePlan plan = plan_of(M, K, KT, kMaxSplits);
  return {plan, (int)std::min<int64_t>(kMaxSplits, std::max<int64_t>(plan.S, KT / 8))};
}

namespace {

struct GradSpace {
  Space s;
  Picked picked;
  float *g, *lse, *tops, *unscale, *kept, *P;
  int64_t ldp;
  uint8_t *prob, *low;
  GradSpace(uint8_t* p, int64_t M, int64_t V, int64_t K, int64_t cols)
      : s{p}, picked(s, M, K), g(s.take<float>(M)), lse(s.take<float>(M)),
        tops(s.take<float>(ceil_div(M, kChunk))), unscale(s.take<float>(1)),
        kept(s.take<float>(cols < V ? M * K : 0)), P(nullptr), ldp(ceil_div(cols, 64) * 64),
        prob(s.take<uint8_t>(M * ldp * 2)), low(s.take<uint8_t>(std::min<int64_t>(M, kFewRows) * ldp * 2)) {
    // Pieces differ by their last one, which may split further.
    int64_t splits = 0;
    for (int64_t c : {std::min(cols, V), V % cols ? V % cols : cols}) {
      const int64_t S = loss_input_plan(M, K, std::min(c, V)).plan.S;
      if (S > 1) splits = std::max(splits, S);
    }
    P = s.take<float>(splits * ceil_div(M, 256) * 256 * K);   // whole tiles: splits_of
  }
};

}  // namespace

int64_t loss_bytes(int64_t M, int64_t V, int64_t K) { return ForwardSpace(nullptr, M, V, K).s.used; }

// Gathering takes 4 us or more.  One tile's rows cost the same whether they take part or not, and
// a product of 2^34 operations takes about 12 us with all of them: those take every row as it
// is, and the join leaves out what takes no part.  Forward, in us, without and with a gathering, none and
// half of the rows ignored: 301 x 1003 x 520 10.9 14.9 and 10.9 14.9, 1000 x 8192 x 1024 (at the border)
// 25.9 31.3 and 25.8 25.2, 2000 x 8192 x 1024 41.7 47.9 and 42.4 41.9, 4096 x 8192 x 1024 76.0 82.2
// and 74.7 47.5.
bool loss_gathers(int64_t M, int64_t V, int64_t K) { return M > 64 && (double)M * (double)V * (double)K > 8.6e9; }

hipError_t launch_loss(const LossCall& c, hipStream_t s) {
  const ForwardSpace w(c.space, c.M, c.V, c.K);
  LossArgs a;
  a.M = (int)c.M, a.N = (int)c.V, a.K = (int)c.K;
  a.B[0] = static_cast<const uint8_t*>(c.W), a.lda = a.ldb = c.K * 2, a.parts = w.part, a.wanted = w.z;
  Join j{c.M, (int)w.parts, w.part, w.z, nullptr, nullptr, c.target, c.V, c.ignore, c.loss, c.lse};
  if (!loss_gathers(c.M, c.V, c.K)) {
    a.A[0] = static_cast<const uint8_t*>(c.X), a.every = c.target;
  } else {
    Pick k = pick_of(c, w.picked);
    k.loss = c.loss, k.lse = c.lse, k.z = w.z;
    const hipError_t e = launch_pick(k, w.picked.counts, nullptr, false, s);
    if (e != hipSuccess) return e;
    a.A[0] = w.picked.rows, a.count = j.count = w.picked.count, a.target = w.picked.wanted, j.map = w.picked.map;
  }
  const hipError_t e = launch_one_group<Forward, true, false>(a, forward_plan(c.M, c.V, c.K).tile, s);
  if (e != hipSuccess) return e;
  // 16 rows side by side are whole lines of parts; few rows of many parts need the threads.  Forward, in
  // us, 1 and 16 rows a workgroup: 301 x 1003 x 128 8.6 7.9, 128 x 4000 (63 parts) 8.3 7.8, 64 x 32000
  // (500 parts) 9.1 10.2, 301 x 32000 15.1 14.9, 301 x 131072 37.2 41.2, 512 x 131072 56.6 55.5,
  // 1024 x 32000 31.6 29.3, 2048 x 32000 56.9 50.2.
  const int rows = c.M >= 512 || w.parts <= 128 ? 16 : 1;
  return launch(rows == 16 ? loss_join_kernel<16> : loss_join_kernel<1>, ceil_div(c.M, rows), 256, s, j);
}

int64_t loss_grad_bytes(int64_t M, int64_t V, int64_t K, int64_t cols) {
  return GradSpace(nullptr, M, V, K, cols).s.used;
}

// Pieces of about 256 MB of P, of equal length but for whole tiles: enough columns to fill the
// chip with each product, few enough that P stays in the last-level cache on its way.
int64_t loss_grad_cols(int64_t M, int64_t V, int64_t K) {
  const int64_t fill = ((int64_t)256 << 20) / (2 * M) / 256 * 256, most = std::min<int64_t>(std::max<int64_t>(fill, 1024), 1 << 20);
  if (V <= most) return ceil_div(V, 64) * 64;
  return ceil_div(ceil_div(V, ceil_div(V, most)), 256) * 256;
}

hipError_t launch_loss_grad(const LossCall& c, hipStream_t s) {
  const GradSpace w(c.space, c.M, c.V, c.K, c.cols);
  Pick k = pick_of(c, w.picked);
  k.dL = c.dL, k.lse_in = c.lse, k.g = w.g, k.lse_out = w.lse, k.unscale = w.unscale, k.dX = static_cast<v4i*>(c.dX);
  hipError_t e = launch_pick(k, w.picked.counts, w.tops, true, s);
  if (e != hipSuccess) return e;
  for (int64_t v = 0; v < c.V; v += c.cols) {
    const int64_t n = std::min(c.cols, c.V - v);
    const uint8_t* W = static_cast<const uint8_t*>(c.W) + v * c.K * 2;
    LossArgs p;
    p.M = (int)c.M, p.N = (int)n, p.K = (int)c.K;
    p.A[0] = w.picked.rows, p.B[0] = W, p.lda = p.ldb = c.K * 2, p.D[0] = w.prob, p.ldp = w.ldp;
    p.count = w.picked.count, p.target = w.picked.wanted, p.col0 = (int)v, p.lse = w.lse, p.g = w.g;
    p.low = w.low;
    e = launch_any<Probabilities, true, false>(p, plan_of(c.M, n, ceil_div(c.K, 64), 1).tile, s);
    if (e != hipSuccess) return e;

    const LossInputPlan input = loss_input_plan(c.M, c.K, n);
    const DensePlan& plan = input.plan;
    const bool last = v + n == c.V;
    LossArgs x, d;
    x.M = (int)c.M, x.N = (int)c.K, x.K = (int)n, x.S = plan.S;
    x.A[0] = w.prob, x.A[1] = w.low, x.lda = w.ldp * 2, x.B[0] = x.B[1] = W, x.ldb = c.K * 2, x.P = w.P;
    x.count = w.picked.count, x.unscale = d.unscale = w.unscale, x.map = w.picked.map, x.add = v > 0 ? w.kept : nullptr;
    x.D[0] = !c.dX ? nullptr : last ? c.dX : w.kept;
    x.bm = (int)tile_rows(plan.tile), x.most = input.most;
    d.M = (int)n, d.N = (int)c.K, d.K = (int)c.M;
    d.A[0] = w.prob, d.A[1] = w.low, d.lda = w.ldp * 2, d.B[0] = d.B[1] = w.picked.rows, d.ldb = c.K * 2;
    if (c.dW) d.D[0] = static_cast<uint8_t*>(c.dW) + v * c.K * 2;
    d.count = w.picked.count;
    const DensePlan weights = plan_of(n, c.K, terms_of(c.M) * ceil_div(c.M, 64), 1);
    const bool both = c.dX && c.dW && n == c.V && merges(plan, weights, c.M, n, c.K);
    e = launch_products(x, plan, last, d, weights, both, s);
    if (e != hipSuccess) return e;
    if (c.dX && plan.S > 1) {
      const int64_t grid = std::min<int64_t>(ceil_div(c.M * (c.K / 4), 256), device_cus() * 8);
      e = launch(last ? loss_reduce_kernel<true> : loss_reduce_kernel<false>, grid, 256, s, x);
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace fp4g
