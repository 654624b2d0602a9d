// Low-rank adapters of many requests beside a shared projection, for gfx950:
//   D[m] = base[m] + s_i B_i (A_i X[m]),  i = index[m];  A_i [R][K], B_i [N][R]
//
// HBM-bound: X and base are read and D written once, and the adapters that are used read once
// where the tokens of each lie in one tile.  Two kernels, both on tiles of up to TM tokens of
// ONE adapter:
//
//   * down   V = X A_i^T.  A wave multiplies 16-row fragments straight from memory (nothing is
//     used twice but by the tokens of its tile) and the four waves of a workgroup, and S
//     workgroups, share K; V's S partial sums are kept in fp32, 4 R bytes a token each.
//   * up     D = base + V B_i^T.  V's sums are added, scaled and split into bf16 terms that all
//     meet the same fragment of B: two for bf16 results (V to 2^-17 of each value, where one
//     alone, 2^-9, would show in them), three for fp32 (all of V's bits).  B's rows are dealt to
//     the instruction's so that a lane ends up with whole 16-byte vectors of a token's columns,
//     and the four lanes of a token with 64 bytes side by side.
//
// The tokens of an adapter are found on the GPU.  Up to 256 tokens every workgroup finds its tile
// by itself, in LDS, from the indexes; more are put in the adapters' order by one
// workgroup first.  The order of a tile's tokens is of no consequence for any of them.
// Tokens without an adapter form tiles too, which `up` copies where D is not base.
#include <algorithm>

#include "dense.hpp"
#include "launch.hpp"
#include "lm_internal.h"

namespace fp4g {
namespace {

constexpr int kDirect = 256;      // tokens whose tiles need no order made beforehand
constexpr float kBf16Max = 0x1.fep127f;

struct Tile { int adapter, first, count, pad; };   // adapter -1: none

struct Args {
  int M, N, K, R, L, S;
  const uint8_t *X, *A, *B;
  const float* scales;
  const int* index;
  const void* base;
  void* D;
  float* V;               // [S][M][R]
  const Tile* tiles;      // ordered tokens: [tiles]
  const int* order;       // [M] tokens by adapter
  const int* count;       // how many tiles there are
  int steps;              // up: steps of 256 columns a workgroup takes
};

__device__ __forceinline__ int adapter_of(int i, int L) { return i >= 0 && i < L ? i : -1; }

// The tile `t` of at most kDirect tokens: its adapter and count (0: there is no such tile), the
// tokens in tok.  The tiles of an adapter hold its tokens in order, TM each; they are
// numbered by their first token.
struct alignas(16) FindSpace { int ids[kDirect], waves[4], lead[2], n; };
template <int TM>
__device__ __forceinline__ Tile find_tile(const Args& a, int t, FindSpace& f, int* tok) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool there = tid < a.M;
  const int id = there ? adapter_of(a.index[tid], a.L) : -2;
  f.ids[tid] = id;
  if (tid == 0) f.lead[0] = -2, f.n = 0;
  __syncthreads();
  int rank = 0;
  if (there) {
#pragma unroll 8
    for (int j = 0; j < tid; j += 4) {
      const v4i o = *reinterpret_cast<const v4i*>(f.ids + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) rank += j + e < tid && o[e] == id;
    }
  }
  const bool leads = there && rank % TM == 0;
  const uint64_t mask = __ballot(leads);
  if (lane == 0) f.waves[wave] = __popcll(mask);
  __syncthreads();
  int number = __popcll(mask & ((1ull << lane) - 1));
  for (int w = 0; w < wave; ++w) number += f.waves[w];
  if (leads && number == t) f.lead[0] = id, f.lead[1] = rank / TM;
  __syncthreads();
  const int adapter = f.lead[0];
  if (there && id == adapter && rank / TM == f.lead[1]) {
    tok[rank % TM] = tid;
    atomicAdd(&f.n, 1);
  }
  __syncthreads();
  return Tile{adapter, 0, f.n, 0};
}
template <int TM, bool DIRECT>
__device__ __forceinline__ Tile tile_of(const Args& a, int t, FindSpace& f, int* tok) {
  if constexpr (DIRECT) {
    return find_tile<TM>(a, t, f, tok);
  } else {
    if (t >= *a.count) return Tile{-2, 0, 0, 0};
    const Tile r = a.tiles[t];
    if ((int)threadIdx.x < r.count) tok[threadIdx.x] = a.order[r.first + threadIdx.x];
    __syncthreads();
    return r;
  }
}

// ---- down ----

// FR blocks of 16 rows of A_i at once.
template <int TM, int FR, bool DIRECT>
__global__ void __launch_bounds__(256) adapter_down_kernel(const Args a) {
  constexpr int FT = TM / 16, RC = FR * 16;
  __shared__ int tok[TM];
  __shared__ FindSpace find;
  __shared__ __attribute__((aligned(16))) float sums[4][TM][RC + 4];
  const int chunks = (a.R + RC - 1) / RC;
  const int slice = blockIdx.x % a.S, rest = blockIdx.x / a.S, r0 = rest % chunks * RC;
  const Tile t = tile_of<TM, DIRECT>(a, rest / chunks, find, tok);
  if (t.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, slot = lane >> 4, rows = min(a.R - r0, RC);
  // Rows past the tile's tokens, or past R, repeat the last one: what they give is not kept.
  const uint8_t* x[FT];
#pragma unroll
  for (int i = 0; i < FT; ++i) x[i] = a.X + (int64_t)tok[min(i * 16 + row, t.count - 1)] * a.K * 2 + slot * 16;
  const uint8_t* w[FR];
#pragma unroll
  for (int j = 0; j < FR; ++j)
    w[j] = a.A + ((int64_t)t.adapter * a.R + r0 + min(j * 16 + row, rows - 1)) * a.K * 2 + slot * 16;
  v4f acc[FT][FR] = {};
  const int units = a.K / 64;
  const int begin = (int)((int64_t)units * slice / a.S), end = (int)((int64_t)units * (slice + 1) / a.S);
  // A unit is a line of 128 bytes of every row: slot h of an instruction takes chunk h, then h + 4.
  // Nothing in it branches (at the end of a branch the compiler waits for the loads within), and
  // the order is pinned: left to itself the compiler puts each load before its use.
  struct Unit { v4i x[2][FT], w[2][FR]; };
  auto fetch = [&](int u, Unit& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < FT; ++i) f.x[h][i] = *reinterpret_cast<const v4i*>(x[i] + (int64_t)u * 128 + h * 64);
#pragma unroll
      for (int j = 0; j < FR; ++j) f.w[h][j] = *reinterpret_cast<const v4i*>(w[j] + (int64_t)u * 128 + h * 64);
    }
  };
  auto multiply = [&](const Unit& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < FR; ++j)
#pragma unroll
        for (int i = 0; i < FT; ++i) acc[i][j] = mfma16(f.w[h][j], f.x[h][i], acc[i][j]);
  };
  // The next unit's loads are on their way while this one is multiplied; past the last the last
  // is read again.
  int u = begin + wave;
  if (u < end) {
    Unit f0, f1;
    fetch(u, f0);
    while (true) {
      fetch(min(u + 4, end - 1), f1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(f0);
      __builtin_amdgcn_sched_barrier(0);
      if ((u += 4) >= end) break;
      fetch(min(u + 4, end - 1), f0);
      __builtin_amdgcn_sched_barrier(0);
      multiply(f1);
      __builtin_amdgcn_sched_barrier(0);
      if ((u += 4) >= end) break;
    }
  }
  if (a.K % 64 != 0 && slice == a.S - 1 && wave == 3) {   // the last line is short
    Unit f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = units * 64 + (h * 4 + slot) * 8 < a.K;
#pragma unroll
      for (int i = 0; i < FT; ++i)
        f.x[h][i] = in ? *reinterpret_cast<const v4i*>(x[i] + (int64_t)units * 128 + h * 64) : v4i{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < FR; ++j)
        f.w[h][j] = in ? *reinterpret_cast<const v4i*>(w[j] + (int64_t)units * 128 + h * 64) : v4i{0, 0, 0, 0};
    }
    multiply(f);
  }
  // A lane holds rows 4 slot .. + 3 of each block of A_i for token `row` of each 16.
#pragma unroll
  for (int i = 0; i < FT; ++i)
#pragma unroll
    for (int j = 0; j < FR; ++j) *reinterpret_cast<v4f*>(&sums[wave][i * 16 + row][j * 16 + 4 * slot]) = acc[i][j];
  __syncthreads();
  for (int e = threadIdx.x; e < TM * RC / 4; e += 256) {
    const int m = e / (RC / 4), r = e % (RC / 4) * 4;
    if (m >= t.count || r >= rows) continue;
    v4f v = *reinterpret_cast<const v4f*>(&sums[0][m][r]);
#pragma unroll
    for (int k = 1; k < 4; ++k) v += *reinterpret_cast<const v4f*>(&sums[k][m][r]);
    *reinterpret_cast<v4f*>(a.V + ((int64_t)slice * a.M + tok[m]) * a.R + r0 + r) = v;
  }
}

// ---- up ----

// The 16 columns of a row that a lane has, as Q vectors of 16 bytes: vector q's columns follow
// those of the row's other three lanes, so that each load and store of a wave covers whole
// 64-byte pieces.  FULL: all of them are there; the code for those that are not stays out of
// the way of the rest.
typedef v4i v4i_at2 __attribute__((aligned(2)));
typedef v4i v4i_at4 __attribute__((aligned(4)));
template <bool BF16>
struct Cols {
  static constexpr int Q = BF16 ? 2 : 4, V = 16 / Q;
  typedef typename std::conditional<BF16, v4i_at2, v4i_at4>::type any;
  v4i v[Q];
  template <bool FULL>
  __device__ __forceinline__ void load(const void* base, int64_t row, int n, int N) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int c = n + q * 4 * V, left = N - c;
      const uint8_t* p = static_cast<const uint8_t*>(base) + (row + c) * (16 / V);
      if (FULL || left >= V) {
        v[q] = *reinterpret_cast<const any*>(p);
      } else {
        v[q] = v4i{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (e < left) {
            if constexpr (BF16) v[q][e / 2] |= (int)((uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (e & 1 ? 16 : 0));
            else v[q][e] = reinterpret_cast<const int*>(p)[e];
          }
      }
    }
  }
  __device__ __forceinline__ float at(int q, int e) const {
    if constexpr (BF16) {
      const uint32_t w = (uint32_t)v[q][e / 2];
      return __builtin_bit_cast(float, e & 1 ? w & 0xffff0000u : w << 16);
    } else {
      const int w = v[q][e];
      return __builtin_bit_cast(float, w);
    }
  }
  // base + acc, block b = q V / 4 + e / 4 holding element e of vector q.
  template <bool FULL>
  __device__ __forceinline__ void add_store(void* D, int64_t row, int n, int N, const v4f (&acc)[4]) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int c = n + q * 4 * V;
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = at(q, e) + acc[q * V / 4 + e / 4][e % 4];
      if (FULL || c < N) store_cols<BF16>(D, row + c, FULL ? V : N - c, y);
    }
  }
};

template <int TM, int RMAX, bool DIRECT, bool BF16>
__global__ void __launch_bounds__(256, TM * RMAX < 64 * 256 || BF16 ? 2 : 1) adapter_up_kernel(const Args a, int shares) {
  constexpr int FT = TM / 16, V = Cols<BF16>::V;
  __shared__ int tok[TM];
  __shared__ FindSpace find;
  constexpr int pitch = RMAX * 2 + 16, TERMS = BF16 ? 2 : 3;
  __shared__ __attribute__((aligned(16))) uint8_t terms[TERMS * TM * pitch];
  const int share = blockIdx.x % shares;
  const Tile t = tile_of<TM, DIRECT>(a, blockIdx.x / shares, find, tok);
  if (t.count == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row = lane & 15, slot = lane >> 4;
  const int first = share * a.steps * 256;
  if (t.adapter < 0) {
    if (a.D == a.base) return;
    const v4f none[4] = {};
    for (int s = 0; s < a.steps; ++s) {
      const int n0 = first + s * 256 + wave * 64, n = n0 + slot * V;
      if (n0 >= a.N) break;
      if (n0 + 64 <= a.N) {
        Cols<BF16> c[FT];
#pragma unroll
        for (int i = 0; i < FT; ++i) c[i].template load<true>(a.base, (int64_t)tok[min(i * 16 + row, t.count - 1)] * a.N, n, a.N);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < FT; ++i)
          if (i * 16 + row < t.count) c[i].template add_store<true>(a.D, (int64_t)tok[i * 16 + row] * a.N, n, a.N, none);
      } else {
        for (int m = row; m < t.count; m += 16) {
          Cols<BF16> c;
          c.template load<false>(a.base, (int64_t)tok[m] * a.N, n, a.N);
          c.template add_store<false>(a.D, (int64_t)tok[m] * a.N, n, a.N, none);
        }
      }
    }
    return;
  }
  // What a step needs of base, and of B for the first 32 of R, is asked for before V is needed.
  // Addresses only advance from step to step: formed anew, in 64 bits, they took as many
  // instructions as the product.
  const int end = min((int64_t)first + a.steps * 256, (int64_t)a.N);
  int n0 = first + wave * 64;
  const uint8_t* B = a.B + (int64_t)t.adapter * a.N * a.R * 2;
  uint32_t of_b[4];
  int64_t at[FT];
#pragma unroll
  for (int i = 0; i < FT; ++i) at[i] = (int64_t)tok[min(i * 16 + row, t.count - 1)] * a.N;
  // Row 4 g + e of block b is the column that element 4 b + e of slot g's 16 stands for.
  auto col_of = [&](int b) { return b * 4 / V * 4 * V + (row >> 2) * V + b * 4 % V + (row & 3); };
#pragma unroll
  for (int b = 0; b < 4; ++b) of_b[b] = (uint32_t)(col_of(b) * a.R + slot * 8) * 2;
  // Rows of B past the last column lie past the buffer's end and read as zeros, as do chunks past R.
  struct Base { Cols<BF16> c[FT]; };
  auto fetch_base = [&](int n, Base& f) {   // tokens past the tile's repeat the last one and are not stored
#pragma unroll
    for (int i = 0; i < FT; ++i) f.c[i].template load<true>(a.base, at[i], n + slot * V, a.N);
  };
  struct Rows { v4i v[4]; };
  auto fetch_b = [&](int n, int kb, Rows& f) {
    const rsrc_t buffer = make_rsrc(B + (int64_t)n * a.R * 2, min(a.N - n, 64) * a.R * 2);
    const bool in = kb + slot * 8 < a.R;
#pragma unroll
    for (int b = 0; b < 4; ++b) f.v[b] = load_buffer16(buffer, in ? of_b[b] + kb * 2 : kNoLoad);
  };
  // Whole steps: 64 columns that all exist.  The last one, short, goes by itself below.
  const int whole = min(end, a.N / 64 * 64);
  // Two sets of four times 16 fp32 columns would not leave two waves a SIMD.
  constexpr bool AHEAD = BF16 || TM == 16;
  Base f0, f1;
  Rows b0, b1;
  if (n0 < whole) {
    if constexpr (AHEAD) fetch_base(n0, f0);
    fetch_b(n0, 0, b0);
    __builtin_amdgcn_sched_barrier(0);
  }
  // V's sums as bf16 terms, zeros past R and past the tile's tokens.
  const int RP = (a.R + 31) / 32 * 32;
  const float scale = a.scales ? a.scales[t.adapter] : 1.0f;
  for (int e = threadIdx.x; e < TM * (RP / 4); e += 256) {
    const int m = e / (RP / 4), r = (e - m * (RP / 4)) * 4;
    v4f v{0.0f, 0.0f, 0.0f, 0.0f};
    if (m < t.count && r < a.R) {
      const float* p = a.V + (int64_t)tok[m] * a.R + r;
      v = *reinterpret_cast<const v4f*>(p);
#pragma unroll 4
      for (int s = 1; s < a.S; ++s) v += *reinterpret_cast<const v4f*>(p + (int64_t)s * a.M * a.R);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] *= scale;
    float c[4];
    // Each term is what the ones before it leave, rounded to bf16.  The first is held to bf16's
    // range, past which the end of fp32's would round to infinity; an infinity or NaN is then in
    // what it leaves, and in the second term alone.
#pragma unroll
    for (int n = 0; n < TERMS; ++n) {
      if (n == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = __builtin_amdgcn_fmed3f(v[k], -kBf16Max, kBf16Max);
      }
      const uint32_t w[2] = {pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3])};
      *reinterpret_cast<v2i*>(terms + (n * TM + m) * pitch + r * 2) = v2i{(int)w[0], (int)w[1]};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] -= __builtin_bit_cast(float, k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
        if (n > 0 && !(__builtin_fabsf(v[k]) < __builtin_inff())) v[k] = 0.0f;
        c[k] = v[k];
      }
    }
  }
  __syncthreads();
  // acc += B's rows f with V's terms kb .. kb + 31, for 16 tokens from `first16`.
  auto multiply = [&](const Rows& f, int kb, int first16, v4f(&acc)[4]) {
    const uint8_t* p = terms + (first16 + row) * pitch + (kb + slot * 8) * 2;
#pragma unroll
    for (int n = 0; n < TERMS; ++n) {
      const v4i t = *reinterpret_cast<const v4i*>(p + n * TM * pitch);
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[b] = mfma16(f.v[b], t, acc[b]);
    }
  };
  // A step's product, with the next step's base and the next rows of B asked for before it.  As
  // compiled b0 = b1 waits for all of them, base's loads among them, which are older: with more than 32
  // of R base is on its way for the first 32 alone.  The choices of an offset, and of the rows that
  // come next, become branches around the loads of B.
  auto step = [&](int n, Base& now, Base& ahead) {
    v4f acc[FT][4] = {};
    const int next = n + 256 < whole ? n + 256 : n;
    if constexpr (AHEAD) fetch_base(next, ahead);
    else fetch_base(n, now);
    __builtin_amdgcn_sched_barrier(0);
    for (int kb = 0; kb < RP; kb += 32) {
      if (kb + 32 < RP) fetch_b(n, kb + 32, b1);
      else fetch_b(next, 0, b1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < FT; ++i) multiply(b0, kb, i * 16, acc[i]);
      __builtin_amdgcn_sched_barrier(0);
      b0 = b1;
    }
#pragma unroll
    for (int i = 0; i < FT; ++i)
      if (i * 16 + row < t.count) now.c[i].template add_store<true>(a.D, at[i], n + slot * V, a.N, acc[i]);
    __builtin_amdgcn_sched_barrier(0);
  };
  while (n0 < whole) {
    step(n0, f0, f1);
    if ((n0 += 256) >= whole) break;
    if constexpr (AHEAD) {
      step(n0, f1, f0);
      n0 += 256;
    }
  }
  if (n0 < end) {
#pragma unroll 1
    for (int i = 0; i < t.count; i += 16) {
      v4f acc[4] = {};
      for (int kb = 0; kb < RP; kb += 32) {
        fetch_b(n0, kb, b0);
        multiply(b0, kb, i, acc);
      }
      if (i + row < t.count) {
        const int64_t mine = (int64_t)tok[i + row] * a.N;
        Cols<BF16> c;
        c.template load<false>(a.base, mine, n0 + slot * V, a.N);
        c.template add_store<false>(a.D, mine, n0 + slot * V, a.N, acc);
      }
    }
  }
}

// ---- the tokens in the adapters' order ----

constexpr int kOrderThreads = 1024;
// The last of the L + 1 buckets is for tokens without an adapter.
template <int TM>
__global__ void __launch_bounds__(kOrderThreads) adapter_order_kernel(int M, int L, const int* __restrict__ index,
                                                                      int* __restrict__ rank, int* __restrict__ order,
                                                                      Tile* __restrict__ tiles, int* __restrict__ count) {
  __shared__ int counts[kMaxAdapters + 1];
  __shared__ int2 waves[kOrderThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, buckets = L + 1;
  for (int b = tid; b < buckets; b += kOrderThreads) counts[b] = 0;
  __syncthreads();
  // The first tokens' buckets and ranks stay in registers, their indexes are all asked for at once.
  constexpr int KEEP = 4;
  int kept[KEEP], ranks[KEEP];
#pragma unroll
  for (int i = 0; i < KEEP; ++i) kept[i] = i * kOrderThreads + tid < M ? index[i * kOrderThreads + tid] : 0;
  auto ranked = [&](int i, bool there) {
    const int id = adapter_of(i, L), bucket = id < 0 ? L : id;
    bool left = there;
    int at = 0;
    // Neighbours mostly share an adapter: two of a wave's adapters are counted at once, the
    // others one by one.
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
      const uint64_t open = __ballot(left);
      if (open == 0) break;
      const int leader = __ffsll((unsigned long long)open) - 1, its = __shfl(bucket, leader);
      const uint64_t same = __ballot(left && bucket == its);
      int old = 0;
      if (lane == leader) old = atomicAdd(&counts[its], __popcll(same));
      old = __shfl(old, leader);
      if (left && bucket == its) {
        at = old + __popcll(same & ((1ull << lane) - 1));
        left = false;
      }
    }
    if (left) at = atomicAdd(&counts[bucket], 1);
    return at;
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    ranks[i] = 0;
    if (i * kOrderThreads < M) ranks[i] = ranked(kept[i], i * kOrderThreads + tid < M);
  }
  for (int64_t m0 = KEEP * kOrderThreads; m0 < M; m0 += kOrderThreads) {
    const int64_t m = m0 + tid;
    const int at = ranked(m < M ? index[m] : 0, m < M);
    if (m < M) rank[m] = at;
  }
  __syncthreads();
  // Where each bucket's tokens and tiles start: a run of buckets a thread.
  const int per = (buckets + kOrderThreads - 1) / kOrderThreads, b0 = min(tid * per, buckets), b1 = min(b0 + per, buckets);
  int2 mine = make_int2(0, 0);
  for (int b = b0; b < b1; ++b) mine.x += counts[b], mine.y += (counts[b] + TM - 1) / TM;
  int2 upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int x = __shfl_up(upto.x, d), y = __shfl_up(upto.y, d);
    if (lane >= d) upto.x += x, upto.y += y;
  }
  if (lane == 63) waves[wave] = upto;
  __syncthreads();
  int2 start = make_int2(upto.x - mine.x, upto.y - mine.y);
  for (int w = 0; w < wave; ++w) start.x += waves[w].x, start.y += waves[w].y;
  for (int b = b0; b < b1; ++b) {
    const int n = counts[b];
    counts[b] = start.x;
    for (int i = 0; i < n; i += TM) tiles[start.y++] = Tile{b < L ? b : -1, start.x + i, min(n - i, TM), 0};
    start.x += n;
  }
  if (tid == kOrderThreads - 1) *count = start.y;
  __syncthreads();
  auto place = [&](int64_t m, int i, int at) {
    const int id = adapter_of(i, L);
    order[counts[id < 0 ? L : id] + at] = (int)m;
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i)
    if (i * kOrderThreads + tid < M) place(i * kOrderThreads + tid, kept[i], ranks[i]);
  for (int64_t m = KEEP * kOrderThreads + tid; m < M; m += kOrderThreads) place(m, index[m], rank[m]);
}

// How a call is cut up: tokens a tile, tiles at most, K slices, columns' shares.
struct Plan {
  bool direct;
  int tm;
  int64_t tiles, S;
};
Plan plan_of(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L) {
  Plan p;
  p.direct = M <= kDirect;
  // 64 tokens share an adapter's reads, 16 leave more tiles.  In us, 16 and 64: 642 x 795 x 5648
  // rank 24 16.4, 25.2; 4000 x 2000 x 2048 rank 128 66.6, 73.9; 1000 x 14336 x 4096 rank 16 26.4, 28.2;
  // about the border, 4 and 64 adapters: 2000 x 16384 x 2048 rank 32 40.2, 45.3 and 54.8, 51.9; 2500 x
  // 16384 x 2048 rank 32 53.8, 51.1 and 70.8, 58.6; past it 4096 x 14336 x 4096 rank 64 135, 91 and 149,
  // 107.  The rule does not look at the rank, which moves the border: 4096 x 4096 x 4096 takes 34.6, 37.2 at
  // rank 16 and 58.4, 49.9 at rank 64.
  p.tm = p.direct || M * N < (int64_t)1 << 25 ? 16 : 64;
  p.tiles = std::min(M, ceil_div(M, p.tm) + L);   // an adapter's last tile may be short; so may that of none
  // Two units of 128 bytes of K a wave at least, and workgroups for the chip: of 64 tokens as many as
  // it holds at once (4096 x 14336 x 4096 rank 64: 17 us with 3 slices, 25 with 4).
  const int64_t units = ceil_div(K, 64), work = p.tiles * std::max<int64_t>(1, ceil_div(R, 64));
  const int64_t room = p.tm == 64 ? device_cus() : 4 * device_cus();
  p.S = std::max<int64_t>(1, std::min({units / 8, room / work, (int64_t)(p.tiles < 64 ? 16 : 4)}));
  return p;
}

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
struct AdapterSpace {
  Space s;
  float* V;
  int *rank, *order, *count;
  Tile* tiles;
  AdapterSpace(uint8_t* p, int64_t M, int64_t R, const Plan& plan)
      : s{p}, V(s.take<float>(plan.S * M * R)), rank(s.take<int>(plan.direct ? 0 : M)),
        order(s.take<int>(plan.direct ? 0 : M)), count(s.take<int>(1)), tiles(s.take<Tile>(plan.direct ? 0 : plan.tiles)) {}
};

template <int TM, bool DIRECT>
hipError_t launch_down(int64_t grid, hipStream_t s, const Args& a) {
  if (a.R <= 16) return launch(adapter_down_kernel<TM, 1, DIRECT>, grid, 256, s, a);
  if (a.R <= 32) return launch(adapter_down_kernel<TM, 2, DIRECT>, grid, 256, s, a);
  return launch(adapter_down_kernel<TM, 4, DIRECT>, grid, 256, s, a);
}

template <int TM, bool DIRECT, bool BF16>
hipError_t launch_up(int64_t grid, hipStream_t s, const Args& a, int shares) {
  if (a.R <= 64) return launch(adapter_up_kernel<TM, 64, DIRECT, BF16>, grid, 256, s, a, shares);
  if (a.R <= 128) return launch(adapter_up_kernel<TM, 128, DIRECT, BF16>, grid, 256, s, a, shares);
  return launch(adapter_up_kernel<TM, 256, DIRECT, BF16>, grid, 256, s, a, shares);
}

}  // namespace

int64_t adapter_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L) {
  return AdapterSpace(nullptr, M, R, plan_of(M, N, K, R, L)).s.used;
}

hipError_t launch_adapter_gemm(const AdapterCall& c, hipStream_t s) {
  // Without adapters, rows of them or columns every token is one without.
  const int64_t L = c.K > 0 && c.R > 0 ? c.L : 0;
  if (L == 0 && c.D == c.base) return hipSuccess;
  const Plan p = plan_of(c.M, c.N, c.K, c.R, c.L);
  const AdapterSpace w(c.space, c.M, c.R, p);
  Args a{(int)c.M, (int)c.N, (int)c.K, (int)c.R, (int)L, (int)p.S, static_cast<const uint8_t*>(c.X),
         static_cast<const uint8_t*>(c.A), static_cast<const uint8_t*>(c.B), c.scales, c.index, c.base, c.D, w.V,
         w.tiles, w.order, w.count, 1};
  hipError_t e = hipSuccess;
  if (!p.direct)
    e = launch(p.tm == 16 ? adapter_order_kernel<16> : adapter_order_kernel<64>, 1, kOrderThreads, s, a.M, a.L, c.index,
               w.rank, w.order, w.tiles, w.count);
  if (e == hipSuccess && L > 0) {
    const int64_t grid = p.tiles * ceil_div(c.R, 64) * p.S;
    if (p.direct) e = launch_down<16, true>(grid, s, a);
    else e = p.tm == 16 ? launch_down<16, false>(grid, s, a) : launch_down<64, false>(grid, s, a);
  }
  if (e != hipSuccess) return e;
  const int64_t steps = ceil_div(c.N, 256), most = std::min(steps, ceil_div(4 * device_cus(), p.tiles));
  a.steps = (int)ceil_div(steps, most);
  const int shares = (int)ceil_div(steps, a.steps);
  const int64_t grid = p.tiles * shares;
  if (p.direct) return c.bf16 ? launch_up<16, true, true>(grid, s, a, shares) : launch_up<16, true, false>(grid, s, a, shares);
  if (p.tm == 16)
    return c.bf16 ? launch_up<16, false, true>(grid, s, a, shares) : launch_up<16, false, false>(grid, s, a, shares);
  return c.bf16 ? launch_up<64, false, true>(grid, s, a, shares) : launch_up<64, false, false>(grid, s, a, shares);
}

}  // namespace fp4g
