// Products of few tokens (1 to 64) for gfx950: the scaled and gated products of
// dense_gemm.hip (the same formulas and the same sums) where the weights are the traffic and
// 64-row tiles would be mostly empty.
//
//   * A workgroup owns RG groups of 16 weight rows (of each weight when gated): they fill
//     the 16-row operand of a 16x16 matrix instruction, the tokens the other.
//   * The waves take K in turn, chunks of SW bytes of every row: wave w chunks w, w + NW, ...
//     Each wave has an LDS ring of its own of D chunks, filled by buffer copies (whole
//     256-byte pieces of a row), and needs no barrier until the end.  The tokens' fragments
//     of a chunk are loaded into registers with its copies.
//   * Few tokens are packed: a load of 16 rows x 64 bytes takes P steps of 16 / P tokens, and
//     the P steps multiply it into sums of their own, of which only the columns of their
//     own step mean anything; the end picks those.  So 1 to 4 tokens cost a quarter of the
//     loads, 5 to 8 half (14336 x 4096 int8, 8 tokens: 16.7 -> 15.1 us).
//   * The 16-byte unit u of row r sits at unit u ^ r of its LDS row: rows are a multiple of
//     256 bytes apart, so 16 rows of one unit would share four banks.
//   * Ragged sizes: rows past N, K past a row's end and chunks past the last are zeros from
//     the buffer resources (dense.hpp); tokens past M repeat the last one and are not stored.
//   * The waves' partial tiles meet in LDS and are added in wave order (results repeat bit
//     for bit); a lane then owns 4 consecutive columns of one token.
//   * HBM-bound for large weights (14336 x 4096 int8, 8 tokens: 12.3 us, 4.8 TB/s; gated bf16,
//     16 tokens: 46-49 us, 4.9 TB/s).  Where N gives few workgroups, bound by what one CU can
//     pull, about 50 KB a us with the tokens' reads: then K is cut into slices too, added by
//     the reduction of dense_gemm.hip.
//
// What was measured for the shape (cold weights, us).  The ring's bytes per workgroup matter
// most: short rings let more workgroups share a CU, and their starts and ends overlap.
//   14336 x 4096 int8, 8 tokens, waves x depth x chunk: 4 x 4 x 256: 17.5, 4 x 2 x 256: 15.6,
//     2 x 2 x 256: 15.1, 4 x 2 x 512: 18.7, 8 x 1 x 512: 17.1; nontemporal copies 13.8
//   gated bf16 14336 x 4096 (235 MB), 16 tokens: 4 x 2 x 256: 49.4, nontemporal 45.0;
//     2 x 2 x 256 with two row groups, nontemporal 46.3
#include <algorithm>

#include "dense.hpp"
#include "launch.hpp"

namespace fp4g {
namespace {

template <class T_, int GATES_, int RG_, int NW_, int SW_, int D_, int TT_, int P_, bool NT_>
struct GemvCfg {
  typedef T_ T;
  static constexpr int GATES = GATES_, RG = RG_, NB = GATES * RG;              // blocks of 16 weight rows
  static constexpr int NW = NW_, SW = SW_, D = D_, TT = TT_, P = P_;           // TT tiles of 16 / P tokens
  static constexpr bool NT = NT_;
  static constexpr int TOK = 16 / P, STEPS = SW / 64;
  static constexpr int UNITS = SW / 16, CHUNK = 16 * SW, SLOT = NB * CHUNK;
  static constexpr int XL = STEPS / P * TT, WL = NB * CHUNK / 1024;            // loads and copies a chunk
  static constexpr int RING = NW * D * SLOT, PART = NW * NB * TT * P * 1024;
  static constexpr int LDS = RING > PART ? RING : PART;
  static_assert(SW >= 256 && SW <= 1024, "swizzle");
  static_assert((D - 1) * (XL + WL) < 64, "vmcnt range");
  static_assert(LDS <= 160 * 1024, "LDS");
  static_assert(P == 1 || TT == 1, "packed steps");
};

template <class C>
__global__ void __launch_bounds__(C::NW * 64) dense_gemv_kernel(const DenseArgs a) {
  typedef typename C::T T;
  typedef typename T::acc16 acc_t;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  const int lane = threadIdx.x & 63, r = lane & 15, s = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slice = a.S > 1 ? blockIdx.x % (uint32_t)a.S : 0, group = a.S > 1 ? blockIdx.x / (uint32_t)a.S : blockIdx.x;
  const int n0 = group * (16 * C::RG);
  const int KB = a.K * T::BYTES, ld = (int)a.ldb;
  const int rounds = ((KB + C::SW - 1) / C::SW + C::NW - 1) / C::NW;
  // A slice of the K split: rounds first .. last - 1 of NW chunks (S <= 16, rounds < 2^14).
  int first = 0, last = rounds;
  if (a.S > 1) {
    first = (uint32_t)(slice * rounds) / (uint32_t)a.S;
    last = (uint32_t)((slice + 1) * rounds) / (uint32_t)a.S;
  }

  // Block b: rows n0 + 16 * (b / GATES) .. of weight b % GATES.
  rsrc_t rw[C::NB];
#pragma unroll
  for (int b = 0; b < C::NB; ++b) {
    const int row = n0 + b / C::GATES * 16, rows = max(min(16, a.N - row), 0);
    rw[b] = make_rsrc(a.B[b % C::GATES] + (int64_t)(rows ? row : 0) * ld, rows * ld);
  }
  const rsrc_t rx = make_rsrc(a.A[0], a.M * (int)a.lda);

  // Copy q of a chunk: units 64q .. 64q+63 of the 16 rows.
  constexpr int WQ = C::CHUNK / 1024;
  uint32_t vw[WQ];
  int kw[WQ];
#pragma unroll
  for (int q = 0; q < WQ; ++q) {
    const int p = q * 64 + lane, row = p / C::UNITS;
    kw[q] = ((p % C::UNITS) ^ row) * 16;
    vw[q] = (uint32_t)row * ld + kw[q];
  }
  // Load k of a chunk: lane (r, s) takes unit s of step k * P + r / TOK of token r % TOK.
  const int kx = r / C::TOK * 64 + s * 16;
  uint32_t vx[C::TT];
#pragma unroll
  for (int t = 0; t < C::TT; ++t)
    vx[t] = (uint32_t)min(r % C::TOK + C::TOK * t, a.M - 1) * (uint32_t)a.lda + kx;

  uint8_t* ring = smem + wave * (C::D * C::SLOT);
  v4i x[C::D][C::STEPS / C::P][C::TT];
  auto issue = [&](int i, auto d_c) {
    constexpr int d = decltype(d_c)::value;
    const int kb = (i * C::NW + wave) * C::SW;
    const int left = i < last ? KB - kb : 0;
#pragma unroll
    for (int k = 0; k < C::STEPS / C::P; ++k)
#pragma unroll
      for (int t = 0; t < C::TT; ++t)
        x[d][k][t] = load_buffer16(rx, k * (64 * C::P) + kx < left ? vx[t] + kb + k * (64 * C::P) : kNoLoad);
#pragma unroll
    for (int b = 0; b < C::NB; ++b)
#pragma unroll
      for (int q = 0; q < WQ; ++q) {
        lds_void* to = (lds_void*)(ring + d * C::SLOT + b * C::CHUNK + q * 1024);
        if constexpr (C::NT) lds_buffer16_nt(rw[b], to, kw[q] < left ? vw[q] + kb : kNoLoad);
        else lds_buffer16(rw[b], to, kw[q] < left ? vw[q] + kb : kNoLoad);
      }
    __builtin_amdgcn_sched_barrier(0);
  };

  acc_t acc[C::NB][C::TT][C::P];
#pragma unroll
  for (int b = 0; b < C::NB; ++b)
#pragma unroll
    for (int t = 0; t < C::TT; ++t)
#pragma unroll
      for (int j = 0; j < C::P; ++j) acc[b][t][j] = acc_t{};

  // The output items of this wave (token tile, row group) and the scales of its lanes there,
  // fetched here so that the end does not wait for them.
  constexpr int OUT = C::TT * C::RG, MY = (OUT + C::NW - 1) / C::NW;
  float sm[MY], sc[MY][C::GATES][4];
  if constexpr (std::is_same<T, I8>::value) {
#pragma unroll
    for (int x = 0; x < MY; ++x) {
      const int item = min(wave + x * C::NW, OUT - 1);
      sm[x] = a.sa[min(C::TOK * (item % C::TT) + r, a.M - 1)];
#pragma unroll
      for (int g = 0; g < C::GATES; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[x][g][e] = a.sb[g][min(n0 + 16 * (item / C::TT) + 4 * s + e, a.N - 1)];
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  static_for<0, C::D>([&](auto d) { issue(first + decltype(d)::value, d); });
  for (int i = first; i < last; i += C::D) {
    static_for<0, C::D>([&](auto d_c) {
      constexpr int d = decltype(d_c)::value;
      // Chunk i + d has landed once only the D - 1 after it are in flight.
      wait_vmcnt<(C::D - 1) * (C::XL + C::WL)>();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < C::STEPS; ++k)
#pragma unroll
        for (int b = 0; b < C::NB; ++b) {
          const v4i w = *reinterpret_cast<const v4i*>(ring + d * C::SLOT + b * C::CHUNK + r * C::SW +
                                                      (((4 * k + s) ^ r) << 4));
#pragma unroll
          for (int t = 0; t < C::TT; ++t) acc[b][t][k % C::P] = mfma16(w, x[d][k / C::P][t], acc[b][t][k % C::P]);
        }
      // The fragments are in registers (the instructions above waited for them): the slot is free.
      __builtin_amdgcn_sched_barrier(0);
      issue(i + C::D + d, d_c);
    });
  }

  // ---- the end ----
  wait_vmcnt<0>();
  barrier_lds();
  acc_t* part = reinterpret_cast<acc_t*>(smem);
#pragma unroll
  for (int b = 0; b < C::NB; ++b)
#pragma unroll
    for (int t = 0; t < C::TT; ++t)
#pragma unroll
      for (int j = 0; j < C::P; ++j)
        part[(((wave * C::NB + b) * C::TT + t) * C::P + j) * 64 + lane] = acc[b][t][j];
  barrier_lds();
#pragma unroll
  for (int x = 0; x < MY; ++x) {
    const int item = wave + x * C::NW;
    if (item >= OUT) break;
    const int tile = item % C::TT, rg = item / C::TT;
    const int m = C::TOK * tile + r, n = n0 + 16 * rg + 4 * s, left = a.N - n;
    if (r >= C::TOK || m >= a.M || n >= a.N) continue;
    acc_t sum[C::GATES];
#pragma unroll
    for (int g = 0; g < C::GATES; ++g) {
      sum[g] = acc_t{};
#pragma unroll
      for (int w = 0; w < C::NW; ++w)
#pragma unroll
        for (int j = 0; j < C::P; ++j)
          sum[g] += part[(((w * C::NB + rg * C::GATES + g) * C::TT + tile) * C::P + j) * 64 + lane + j * C::TOK];
    }
    if (a.S > 1) {
      const int64_t pitch = partial_pitch(a.N);
#pragma unroll
      for (int g = 0; g < C::GATES; ++g)
        static_cast<acc_t*>(a.P)[((((int64_t)slice * C::GATES + g) * a.M + m) * pitch + n) / 4] = sum[g];
      continue;
    }
    float y[C::GATES][4];
#pragma unroll
    for (int g = 0; g < C::GATES; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[g][e] = (float)sum[g][e];
        if constexpr (std::is_same<T, I8>::value) y[g][e] = y[g][e] * sm[x] * sc[x][g][e];
      }
    const int64_t at = (int64_t)m * a.N + n;
    if constexpr (C::GATES == 2) {
      if (a.G) {
        store_cols<false>(a.G, at, left, y[0]);
        store_cols<false>(a.U, at, left, y[1]);
      }
      gate(a.act, y[0], y[1]);
    }
    if (a.bf16_out) store_cols<true>(a.D[0], at, left, y[0]);
    else store_cols<false>(a.D[0], at, left, y[0]);
  }
}

template <class C>
hipError_t launch_gemv(const DenseArgs& a, hipStream_t s) {
  return launch(dense_gemv_kernel<C>, ceil_div(a.N, 16 * C::RG) * a.S, C::NW * 64, s, a);
}

// Weights of 32 MB and more stream past the caches (the eight L2s hold that much together).
// With enough rows for two CUs in three they take nontemporal copies, two row groups a
// workgroup, which halves the tokens' reads, and two waves.  Against one group: 14336 x 4096
// int8, 16 and 32 tokens, 16.8 -> 14.4 and 23.7 -> 18.4 us; bf16 gated, 16 and 32 tokens,
// 45.8 -> 46.3 and 57.9 -> 52.3 us; 6000 x 2000 bf16 gated, 30 tokens, 18.8 -> 16.3 us; but
// with fewer rows (4096 x 8192 int8 gated, 16 tokens) 16.2 -> 20.1 us.  Smaller weights may
// stay in the caches and need the workgroups too: one row group, and four waves where the
// tokens leave LDS and registers for them (gated bf16 1024 x 1024, 1 token: 5.2 against 5.8
// us with two; 64 tokens, int8 1000 x 1024: 6.9 against 5.4 us).
constexpr int64_t kStreamBytes = (int64_t)32 << 20;
bool streams(int64_t N, int64_t KB, int64_t gates) { return gates * N * KB >= kStreamBytes; }
bool wide(int64_t N, int64_t KB, int64_t gates) {
  return streams(N, KB, gates) && ceil_div(N, 32) * 3 >= device_cus() * 2;
}

template <class T, int GATES, int TT, int P>
hipError_t launch_tokens(const DenseArgs& a, hipStream_t s) {
  if (wide(a.N, a.ldb, GATES)) {
    if constexpr (TT <= 2) return launch_gemv<GemvCfg<T, GATES, 2, 2, 256, 2, TT, P, true>>(a, s);
    return hipErrorInvalidConfiguration;   // gemv_takes refuses these
  }
  return launch_gemv<GemvCfg<T, GATES, 1, TT == 1 ? 4 : 2, 256, 2, TT, P, false>>(a, s);
}

template <class T, int GATES>
hipError_t launch_form(const DenseArgs& a, hipStream_t s) {
  hipError_t e;
  if (a.M <= 4) e = launch_tokens<T, GATES, 1, 4>(a, s);
  else if (a.M <= 8) e = launch_tokens<T, GATES, 1, 2>(a, s);
  else if (a.M <= 16) e = launch_tokens<T, GATES, 1, 1>(a, s);
  else if (a.M <= 32) e = launch_tokens<T, GATES, 2, 1>(a, s);
  else e = launch_tokens<T, GATES, 4, 1>(a, s);
  if (e != hipSuccess || a.S == 1) return e;
  return launch_partial_sums(a, std::is_same<T, I8>::value, GATES == 2, s);
}

}  // namespace

// Up to 32 tokens, and up to 64 of weights that do not stream: with 64 tokens and 14336 x 4096
// int8 gated weights the tiles take 32.4 us and this 37.1, with 1000 x 1024 8.5 and 8.5, and
// ungated 64 x 1000 x 1024 8.3 and 5.4.
// N below 2^27 is at most 2^23 groups of 256 threads, half of the 2^32 threads that a launch
// holds fewer than; gemv_splits keeps their slices below it too.
bool gemv_takes(int64_t M, int64_t N, int64_t KB, int64_t gates) {
  return N < (int64_t)1 << 27 && M <= (streams(N, KB, gates) ? 32 : 64);
}

// The K split: a workgroup reads its weights and all the tokens at about 50 KB a us, the chip
// 4.8 MB a us; a split adds a launch and the partial sums.
int gemv_splits(int64_t M, int64_t N, int64_t KB, int64_t gates, int64_t cap) {
  const double rows = wide(N, KB, gates) ? 32.0 : 16.0, cus = (double)device_cus();
  const double groups = (double)ceil_div(N, (int64_t)rows), own = (gates * rows + (double)M) * (double)KB;
  const int64_t rounds = ceil_div(KB, M <= 16 ? 1024 : 512);
  cap = std::min(cap, (((int64_t)1 << 32) - 1) / ((int64_t)groups * 256));
  int best = 1;
  double best_t = 1e30;
  for (int64_t S = 1; S <= std::min<int64_t>({cap, rounds / 2, kMaxSplits}) || S == 1; S *= 2) {
    const double per_cu = (double)ceil_div((int64_t)groups * S, (int64_t)cus);
    double t = std::max((double)(gates * N * KB) / 4.8e6, per_cu * own / (double)S / 5.0e4);
    if (S > 1) t += 3.5 + (double)(S * gates * M * N) * 8.0 / 4.0e6;
    if (t < best_t) {
      best_t = t;
      best = (int)S;
    }
  }
  return best;
}

hipError_t launch_gemv_w8a8(const DenseArgs& a, hipStream_t s) { return launch_form<I8, 1>(a, s); }
hipError_t launch_gemv_w8a8_gated(const DenseArgs& a, hipStream_t s) { return launch_form<I8, 2>(a, s); }
hipError_t launch_gemv_gated(const DenseArgs& a, hipStream_t s) { return launch_form<BF, 2>(a, s); }

}  // namespace fp4g
