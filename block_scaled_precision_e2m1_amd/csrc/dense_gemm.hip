// Tile products of int8 and bf16 operands for gfx950, with the ends that a feed-forward
// block gives them:
//
//   scaled   D[m][n] = (sum_k A[m][k] B[n][k]) * sa[m] * sb[n]               int8
//   gated    D[m][n] = act(g) * u,  g, u the products of A with B[0] and B[1] int8, bf16
//   plain    D[m][n] = sum_k A[m][k] B[k][n]  over one or two (A, B) pairs    bf16
//
// The loop works on bytes.  A 32x32 matrix instruction of either type takes 16 bytes of K
// per lane and the same 32 cycles, so one tile, one ring and one schedule serve both.
//
//   * One workgroup of 4 waves (2 x 2) per BM x BN tile; a wave owns WM x WN.  At 256 x 256
//     a wave's 128 x 128 sums fill 256 AGPRs and each fragment read from LDS feeds four
//     matrix instructions, which halves the LDS traffic of a 64 x 64 wave tile.
//   * A K stage is 128 bytes of every row of A and of B (a cache line; 128 int8 or 64 bf16
//     elements).  Stages live in a ring of STAGES slots, filled by buffer copies straight
//     to LDS whose resources end with the operand's tile (dense.hpp): every ragged edge
//     reads zeros.
//   * Operand forms.  A "row" operand has K contiguous: 16-byte chunk c of row r sits at
//     chunk c ^ swz(r), so ds_read_b128 of 32 rows is free of bank conflicts.  A "column"
//     operand (bf16; the gradients' products sum over rows of their operands) has K
//     strided: the stage is 64 K rows of the tile's columns, and ds_read_b64_tr_b16 turns
//     4 K rows x 16 columns into the fragment's order.  Its 64-byte units are XORed with
//     the K row's low bits, so that the four rows one read touches lie in different banks.
//   * K slots.  In quarter q of a stage, slot h (lane / 32) holds chunk 4h + q of a row, which
//     is K elements 32h + 8q .. +7 for bf16: column operands read exactly those K rows.
//   * The schedule is the one measured for the MXFP4 tiles (mxfp4_gemm.hip): the next
//     quarter's fragments are read under this quarter's 16 matrix instructions, and the
//     copies of a later stage are issued between them, in a pinned order; one barrier a
//     stage sits before the last quarter.
//   * Gated tiles take BN/2 columns of each weight: in every wave half of the 32-column
//     blocks are g and the other half u of the same outputs, so the gate is applied in the
//     wave's own registers' worth of sums and g and u never travel.
//   * The end goes through the wave's share of the (then idle) ring in strips of 32 rows:
//     sums are written as the instruction leaves them (a lane owns 4 consecutive columns)
//     and read back along rows, so results leave as 16 bytes a lane, whole lines a row,
//     whatever the row's alignment (the hardware takes unaligned vector stores).  The
//     activation is applied on that way back, in a rolled loop: with three activations in
//     line for each of a wave's sums the code would not fit the instruction cache.
//   * Work items are numbered so that the tiles one XCD runs at once share A and B panels in
//     its L2.  With too few tiles to fill the chip, K is cut into S slices, whose sums are
//     added in slice order by a second kernel (no atomics: results repeat bit for bit).
#include <algorithm>

#include "dense.hpp"

namespace fp4g {
namespace {

__device__ __forceinline__ int swz(int r) { return ((r >> 1) & 7) ^ ((r & 1) << 2); }

// Column operands: the 64-byte unit u of K row k sits at unit u ^ unit_swz(k) of its LDS row, so
// the four rows k .. k+3 (k % 4 == 0) of one unit lie in different banks: rows of 256 and 512
// bytes all start in bank 0, rows of 128 bytes in alternate halves of the banks.
template <int PITCH>
__device__ __forceinline__ int unit_swz(int k) { return PITCH >= 256 ? k & 3 : (k >> 1) & 1; }

enum Form { kScaled, kGated, kPlain };

template <class T_, int FORM_, int BM_, int BN_, int WM_, int WN_, int STAGES_, bool ACOL_, bool BCOL_, int NSEG_>
struct TileCfg {
  typedef T_ T;
  static constexpr int FORM = FORM_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_, NSEG = NSEG_;
  static constexpr bool ACOL = ACOL_, BCOL = BCOL_, GATED = FORM_ == kGated;
  static constexpr int NW = (BM / WM) * (BN / WN), NWN = BN / WN;
  static constexpr int ROWB = 128, KE = ROWB / T::BYTES;      // bytes and elements of K per stage
  static constexpr int A_BYTES = BM * ROWB, STAGE = (BM + BN) * ROWB, LDS = STAGE * STAGES;
  static constexpr int IA = BM / 8 / NW, IB = BN / 8 / NW, LOADS = IA + IB;   // 1 KB copies per wave per stage
  static constexpr int FI = WM / 32, FJ = WN / 32;
  static constexpr int OUTN = GATED ? BN / 2 : BN, WOUT = GATED ? WN / 2 : WN;   // output columns: tile, wave
  static constexpr int STRIP = WN * 4 + 16;                   // LDS pitch of a row of a wave's sums
  static_assert(!(ACOL || BCOL) || T::BYTES == 2, "column operands are bf16");
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "copies per wave");
  static_assert(!GATED || BN / NW <= WN / 2, "each wave copies rows of one weight");
  static_assert(NW * 32 * STRIP <= LDS && LDS <= 160 * 1024, "LDS");
  static_assert(STAGES >= 2 && (STAGES - 1) * LOADS < 64, "vmcnt range");
};

struct Item { int l, s, tm, tn; };

// Work item `wg` of `total`: consecutive ids go to the 8 XCDs in turn, so they are regrouped
// to give each XCD a contiguous run, in which the slices of one tile are neighbours and the
// tiles go in groups of 8 tile rows, column by column.
__device__ __forceinline__ Item item_of(int wg, int total, int S, int tiles_m, int tiles_n) {
  // Runs of equal length; the first total % 8 of them take one more item.
  const int q = total >> 3, rem = total & 7, x = wg & 7;
  int lin = x * q + min(x, rem) + (wg >> 3);
  Item it;
  it.s = lin % S;
  lin /= S;
  const int T = tiles_m * tiles_n;
  it.l = lin / T;
  const int t = lin - it.l * T;
  constexpr int G = 8;
  const int group = t / (G * tiles_n), first = group * G, size = min(G, tiles_m - first);
  const int in = t - group * G * tiles_n;
  it.tm = first + in % size;
  it.tn = in / size;
  return it;
}

template <class C, bool BF16, bool SAVE, bool SPLIT>
__global__ void __launch_bounds__(C::NW * 64) dense_gemm_kernel(const DenseArgs a) {
  typedef typename C::T T;
  constexpr int FI = C::FI, FJ = C::FJ;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::NWN, wn = wave % C::NWN;
  const int hi = lane >> 5, r32 = lane & 31;
  const int tiles_m = (a.M + C::BM - 1) / C::BM, tiles_n = (a.N + C::OUTN - 1) / C::OUTN;
  const int total = a.L * tiles_m * tiles_n * a.S;
  const int KT1 = (a.K + C::KE - 1) / C::KE, KT = C::NSEG * KT1;
  const int lda = (int)a.lda, ldb = (int)a.ldb;

  // ---- this lane's part of a copy: offsets from the tile's first byte ----
  // Row operand, copy q of the wave: rows 8q' .. 8q'+7 (q' = wave * I + q), 8 lanes a row.
  // Column operand: 1 KB of the stage's 64 K rows of BM (BN) columns.
  uint32_t va[C::IA], vb[C::IB];
  int ca[2], cb[2];          // row operands: the byte of K within the stage, even and odd copies
#pragma unroll
  for (int q = 0; q < C::IA; ++q) {
    const int n = wave * C::IA + q;
    if constexpr (C::ACOL) {
      constexpr int PITCH = C::BM * 2;
      const int p = 1024 * n + 16 * lane, k = p / PITCH, w = p % PITCH;
      va[q] = (uint32_t)k * lda + (((w >> 6) ^ unit_swz<PITCH>(k)) << 6 | (w & 63));
    } else {
      const int row = 8 * n + (lane >> 3), c = ((lane & 7) ^ swz(row)) * 16;
      va[q] = (uint32_t)row * lda + c;
      ca[n & 1] = c;
    }
  }
  // Gated: the rows this wave copies belong to one of the weights; within the tile, row r
  // of LDS is output column (r / WN) * WN/2 + r % (WN/2) of weight (r % WN) / (WN/2).
  const int bwhich = C::GATED ? (wave * C::IB * 8) % C::WN / (C::WN / 2) : 0;
#pragma unroll
  for (int q = 0; q < C::IB; ++q) {
    const int n = wave * C::IB + q;
    if constexpr (C::BCOL) {
      constexpr int PITCH = C::BN * 2;
      const int p = 1024 * n + 16 * lane, k = p / PITCH, w = p % PITCH;
      vb[q] = (uint32_t)k * ldb + (((w >> 6) ^ unit_swz<PITCH>(k)) << 6 | (w & 63));
    } else {
      const int row = 8 * n + (lane >> 3), c = ((lane & 7) ^ swz(row)) * 16;
      const int src = C::GATED ? row / C::WN * (C::WN / 2) + row % (C::WN / 2) : row;
      vb[q] = (uint32_t)src * ldb + c;
      cb[n & 1] = c;
    }
  }

  // ---- the current item ----
  Item it;
  int m0 = 0, n0 = 0, ks0 = 0, KS = 0;
  auto setup = [&](int work) {
    it = item_of(work, total, a.S, tiles_m, tiles_n);
    m0 = it.tm * C::BM;
    n0 = it.tn * C::OUTN;
    ks0 = (int)((int64_t)it.s * KT / a.S);
    KS = (int)((int64_t)(it.s + 1) * KT / a.S) - ks0;
  };
  // Copy q (A's, then B's) of stage ks of the item into slot ks % STAGES.  A stage past the
  // end of the slice has an empty resource: no traffic, zeros in a slot that is not used.
  auto issue_one = [&](int ks, int q) {
    uint8_t* base = smem + (ks % C::STAGES) * C::STAGE;
    const int g = ks0 + ks;
    const int seg = C::NSEG == 2 && g >= KT1 ? 1 : 0;
    const int kk = g - seg * KT1;
    const bool live = ks < KS;
    if (q < C::IA) {
      const uint8_t* src = a.A[C::NSEG == 2 ? seg : it.l];
      if constexpr (C::ACOL) {
        const int rows = min(a.K - kk * C::KE, C::KE);
        const rsrc_t r = make_rsrc(src + (int64_t)kk * C::KE * lda + m0 * 2, live ? rows * lda - m0 * 2 : 0);
        lds_buffer16(r, (lds_void*)(base + 1024 * (wave * C::IA + q)), va[q]);
      } else {
        const int rows = min(a.M - m0, C::BM), left = a.K * T::BYTES - kk * C::ROWB;
        const rsrc_t r = make_rsrc(src + (int64_t)m0 * lda + kk * C::ROWB, live ? rows * lda - kk * C::ROWB : 0);
        lds_buffer16(r, (lds_void*)(base + 1024 * (wave * C::IA + q)),
                     ca[(wave * C::IA + q) & 1] < left ? va[q] : kNoLoad);
      }
    } else {
      const int i = q - C::IA;
      const uint8_t* src = a.B[C::NSEG == 2 ? seg : bwhich];
      if constexpr (C::BCOL) {
        const int rows = min(a.K - kk * C::KE, C::KE);
        const rsrc_t r = make_rsrc(src + (int64_t)kk * C::KE * ldb + n0 * 2, live ? rows * ldb - n0 * 2 : 0);
        lds_buffer16(r, (lds_void*)(base + C::A_BYTES + 1024 * (wave * C::IB + i)), vb[i]);
      } else {
        const int rows = min(a.N - n0, C::OUTN), left = a.K * T::BYTES - kk * C::ROWB;
        const rsrc_t r = make_rsrc(src + (int64_t)n0 * ldb + kk * C::ROWB, live ? rows * ldb - kk * C::ROWB : 0);
        lds_buffer16(r, (lds_void*)(base + C::A_BYTES + 1024 * (wave * C::IB + i)),
                     cb[(wave * C::IB + i) & 1] < left ? vb[i] : kNoLoad);
      }
    }
  };

  // ---- fragments ----
  v4i fa[2][FI], fb[2][FJ];
  // Column operand: the 16 lanes of a group read K rows k, k+1, k+2, k+3 (lane / 4) of 16
  // columns; lane i of the group receives column i of all four.
  const int ti = lane & 15, tq = ti >> 2, tb = ((lane >> 4) & 1) * 32 + (ti & 3) * 8;
  auto read_col = [&](const uint8_t* tile, auto pitch_c, int blk, int kq) {
    constexpr int PITCH = decltype(pitch_c)::value;
    const uint8_t* p = tile + (32 * hi + 8 * kq + tq) * PITCH + ((blk ^ unit_swz<PITCH>(tq)) << 6) + tb;
    const v2i lo = lds_read_tr16(p), up = lds_read_tr16(p + 4 * PITCH);
    return v4i{lo[0], lo[1], up[0], up[1]};
  };
  auto read_frag = [&](int ks, int kq, int set, int r) {
    const uint8_t* base = smem + (ks % C::STAGES) * C::STAGE;
    const int c = 4 * hi + kq;
    if (r < FI) {
      if constexpr (C::ACOL) {
        fa[set][r] = read_col(base, std::integral_constant<int, C::BM * 2>{}, wm * FI + r, kq);
      } else {
        const int row = wm * C::WM + r * 32 + r32;
        fa[set][r] = *reinterpret_cast<const v4i*>(base + row * C::ROWB + ((c ^ swz(row)) << 4));
      }
    } else {
      const int j = r - FI;
      if constexpr (C::BCOL) {
        fb[set][j] = read_col(base + C::A_BYTES, std::integral_constant<int, C::BN * 2>{}, wn * FJ + j, kq);
      } else {
        const int row = wn * C::WN + j * 32 + r32;
        fb[set][j] = *reinterpret_cast<const v4i*>(base + C::A_BYTES + row * C::ROWB + ((c ^ swz(row)) << 4));
      }
    }
  };

  typename T::acc32 acc[FI][FJ];
  // The matrix instructions of a quarter on register set SET; extra(q) issues that slot's
  // memory instructions (the scheduling barriers keep the order as written).
  auto quarter = [&](auto set_c, auto&& extra) {
    constexpr int SET = decltype(set_c)::value;
#pragma unroll
    for (int q = 0; q < FI * FJ; ++q) {
      const int i = q / FJ, j = q % FJ;
      // B first: the sums are D^T, so a lane owns 4 consecutive columns of a row.
      acc[i][j] = mfma32(fb[SET][j], fa[SET][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      extra(q);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Copies 0 .. LH-1 of a stage go out under the last quarter of the stage STAGES before it
  // (right after the barrier that frees its slot), the rest under the following quarter 0.
  constexpr int LH = (C::LOADS + 1) / 2, FR = FI + FJ, NQ = FI * FJ;
  auto mid_quarter = [&](int ks, auto kq_c) {
    constexpr int KQ = decltype(kq_c)::value;
    quarter(std::integral_constant<int, (KQ & 1)>{}, [&](int q) {
#pragma unroll
      for (int r = q; r < FR; r += NQ) read_frag(ks, KQ + 1, (KQ + 1) & 1, r);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (KQ == 0) {
#pragma unroll
        for (int r = LH + q; r < C::LOADS; r += NQ) issue_one(ks + C::STAGES - 1, r);
      }
    });
  };
  auto prologue = [&]() {
#pragma unroll
    for (int p = 0; p < C::STAGES - 1; ++p)
#pragma unroll
      for (int q = 0; q < C::LOADS; ++q) issue_one(p, q);
#pragma unroll
    for (int q = 0; q < LH; ++q) issue_one(C::STAGES - 1, q);
  };

  // Persistent: at most one workgroup per CU (times its occupancy) walks the items.
  for (int work = blockIdx.x; work < total; work += gridDim.x) {
    setup(work);
    prologue();
    // Stage 0 has landed once only the copies issued after it are in flight.
    wait_vmcnt<(C::STAGES - 2) * C::LOADS + LH>();
    barrier_lds();
#pragma unroll
    for (int r = 0; r < FR; ++r) read_frag(0, 0, 0, r);
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j) acc[i][j] = typename T::acc32{};

    for (int ks = 0; ks < KS; ++ks) {
      mid_quarter(ks, std::integral_constant<int, 0>{});
      mid_quarter(ks, std::integral_constant<int, 1>{});
      mid_quarter(ks, std::integral_constant<int, 2>{});
      // Stage ks+1 has landed once at most the STAGES-2 stages after it are in flight; the
      // barrier publishes it and says that every wave has read slot ks % STAGES to its end
      // (the last quarter's fragments are in registers: barrier_lds waits for LDS reads).
      wait_vmcnt<(C::STAGES - 2) * C::LOADS>();
      barrier_lds();
      quarter(std::integral_constant<int, 1>{}, [&](int q) {
#pragma unroll
        for (int r = q; r < LH; r += NQ) issue_one(ks + C::STAGES, r);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = q; r < FR; r += NQ) read_frag(ks + 1, 0, 0, r);
      });
    }
    // ---- the end ----
    const int mw = m0 + wm * C::WM, nw = n0 + wn * C::WOUT;
    // A lane writes row r32 of every strip and reads column group `col` of it: the scales of
    // both are fetched here once, under the wait for the ring.
    constexpr int ELEM = SPLIT || !BF16 || SAVE ? 4 : 2, V = 16 / ELEM, LPR = C::WOUT / V;
    static_assert(64 % LPR == 0, "a lane keeps its columns");
    constexpr bool SCALED = !SPLIT && std::is_same<T, I8>::value;
    typedef typename std::conditional<std::is_same<T, I8>::value, int, float>::type sum_t;
    const int col = lane % LPR * V, n = nw + col;
    float sm[FI], sc[C::GATED ? 2 : 1][V];
    if constexpr (SCALED) {
#pragma unroll
      for (int i = 0; i < FI; ++i) sm[i] = a.sa[min(mw + i * 32 + r32, a.M - 1)];
#pragma unroll
      for (int w = 0; w < (C::GATED ? 2 : 1); ++w)
#pragma unroll
        for (int e = 0; e < V; ++e) sc[w][e] = a.sb[w][min(n + e, a.N - 1)];
    }
    // No copy may still be landing when the ring is reused, and no wave may still read it.
    wait_vmcnt<0>();
    barrier_lds();
    uint8_t* strip = smem + wave * (32 * C::STRIP);
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      // In: lane (hi, r32) holds row r32, columns j*32 + 8*g + 4*hi + 0..3 of block row i.
      // The row's scale goes into the 16 bytes past its sums.
#pragma unroll
      for (int j = 0; j < FJ; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          typedef decltype(acc[i][j][0] + acc[i][j][0]) e_t;
          typedef e_t e4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<e4*>(strip + r32 * C::STRIP + (j * 32 + 8 * g + 4 * hi) * 4) =
              e4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
        }
      if constexpr (SCALED) *reinterpret_cast<float*>(strip + r32 * C::STRIP + C::WN * 4) = sm[i];
      // Out: V columns a lane, along rows.
      const int rows = min(a.M - (mw + i * 32), 32);
#pragma unroll 1
      for (int row = lane / LPR; row < rows; row += 64 / LPR) {
        const sum_t* g = reinterpret_cast<const sum_t*>(strip + row * C::STRIP) + col;
        const int64_t m = mw + i * 32 + row;
        if constexpr (SPLIT) {
          const int64_t pitch = partial_pitch(a.N);
          if (n < pitch) {
#pragma unroll
            for (int w = 0; w < (C::GATED ? 2 : 1); ++w) {
              const int64_t plane = ((int64_t)it.l * a.S + it.s) * (C::GATED ? 2 : 1) + w;
              *reinterpret_cast<v4i*>(static_cast<int*>(a.P) + (plane * a.M + m) * pitch + n) =
                  *reinterpret_cast<const v4i*>(g + w * C::WOUT);
            }
          }
        } else if (n < a.N) {
          // int8 sums are exact in 32 bits and are rounded to fp32 here.
          float y[V], u[V], rs = 1.0f;
          if constexpr (SCALED) rs = *reinterpret_cast<const float*>(strip + row * C::STRIP + C::WN * 4);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            y[e] = (float)g[e];
            if constexpr (SCALED) y[e] = y[e] * rs * sc[0][e];
          }
          const int64_t at = m * a.N + n;
          const int left = a.N - n;
          if constexpr (C::GATED) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              u[e] = (float)g[C::WOUT + e];
              if constexpr (SCALED) u[e] = u[e] * rs * sc[1][e];
            }
            if constexpr (SAVE) {
              store_cols<false>(a.G, at, left, y);
              store_cols<false>(a.U, at, left, u);
            }
            gate(a.act, y, u);
          }
          store_cols<BF16>(a.D[it.l], at, left, y);
        }
      }
    }
    // No wave may start the next item's copies while another still reads its strips.
    barrier_lds();
  }
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
  hipLaunchKernelGGL((dense_reduce_kernel<T, GATED, BF16, SAVE>), dim3(grid), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <class C, bool BF16, bool SAVE>
hipError_t launch_tiles(const DenseArgs& a, int per_cu, hipStream_t s) {
  const int64_t items = a.L * ceil_div(a.M, C::BM) * ceil_div(a.N, C::OUTN) * a.S;
  if (items > INT32_MAX) return hipErrorInvalidConfiguration;
  const unsigned grid = (unsigned)std::min<int64_t>(items, device_cus() * per_cu);
  if (a.S > 1) {
    hipLaunchKernelGGL((dense_gemm_kernel<C, false, false, true>), dim3(grid), dim3(C::NW * 64), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_reduce<typename C::T, C::GATED, BF16, SAVE>(a, s);
  }
  hipLaunchKernelGGL((dense_gemm_kernel<C, BF16, SAVE, false>), dim3(grid), dim3(C::NW * 64), 0, s, a);
  return hipGetLastError();
}

template <class T, int FORM, bool ACOL, bool BCOL, int NSEG, bool BF16, bool SAVE>
hipError_t launch_cfg(const DenseArgs& a, DenseTile tile, hipStream_t s) {
  switch (tile) {
    case kTile256: return launch_tiles<TileCfg<T, FORM, 256, 256, 128, 128, 2, ACOL, BCOL, NSEG>, BF16, SAVE>(a, 1, s);
    case kTile128: return launch_tiles<TileCfg<T, FORM, 128, 128, 64, 64, 2, ACOL, BCOL, NSEG>, BF16, SAVE>(a, 2, s);
    default: return launch_tiles<TileCfg<T, FORM, 64, 128, 32, 64, 3, ACOL, BCOL, NSEG>, BF16, SAVE>(a, 2, s);
  }
}

}  // namespace

// Tile and K split of a product with `rows` x `cols` sums (gated: cols = 2 N), L of them,
// each a sum of KT stages.
DensePlan dense_plan(int64_t rows, int64_t cols, int64_t L, int64_t KT, int64_t cap) {
  const int64_t cus = device_cus();
  struct { DenseTile t; int64_t bm, bn, per_cu; double stage_us; } const tiles[] = {
      {kTile256, 256, 256, 1, 1.4}, {kTile128, 128, 128, 2, 0.75}, {kTile64, 64, 128, 2, 0.5}};
  DensePlan best{kTile64, 1};
  double best_t = 1e30;
  for (const auto& c : tiles) {
    const int64_t items = L * ceil_div(rows, c.bm) * ceil_div(cols, c.bn);
    for (int64_t S = 1; S <= std::min<int64_t>({cap, KT, kMaxSplits}); ++S) {
      if (S > 1 && (KT / S < 4 || L * rows * (cols + 8) >= (int64_t)1 << 31)) break;   // 32-bit sums' indexes
      const int64_t slots = cus * c.per_cu;
      double t = (double)ceil_div(items * S, slots) * (ceil_div(KT, S) * c.stage_us + 2.0);
      if (S > 1) t += 3.0 + (double)(L * rows * cols) * 4.0 * (S + 1) / 4.0e6;
      if (t < best_t) {
        best_t = t;
        best = DensePlan{c.t, (int)S};
      }
    }
  }
  return best;
}

hipError_t launch_partial_sums(const DenseArgs& a, bool int8, bool gated, hipStream_t s) {
  if (!int8) return a.G ? launch_reduce<BF, true, true, true>(a, s) : launch_reduce<BF, true, true, false>(a, s);
  if (gated) return a.bf16_out ? launch_reduce<I8, true, true, false>(a, s) : launch_reduce<I8, true, false, false>(a, s);
  return a.bf16_out ? launch_reduce<I8, false, true, false>(a, s) : launch_reduce<I8, false, false, false>(a, s);
}

hipError_t launch_w8a8(const DenseArgs& a, DenseTile tile, hipStream_t s) {
  if (tile == kGemv) return launch_gemv_w8a8(a, s);
  return a.bf16_out ? launch_cfg<I8, kScaled, false, false, 1, true, false>(a, tile, s)
              : launch_cfg<I8, kScaled, false, false, 1, false, false>(a, tile, s);
}

hipError_t launch_w8a8_gated(const DenseArgs& a, DenseTile tile, hipStream_t s) {
  if (tile == kGemv) return launch_gemv_w8a8_gated(a, s);
  return a.bf16_out ? launch_cfg<I8, kGated, false, false, 1, true, false>(a, tile, s)
              : launch_cfg<I8, kGated, false, false, 1, false, false>(a, tile, s);
}

hipError_t launch_gated(const DenseArgs& a, DenseTile tile, hipStream_t s) {
  if (tile == kGemv) return launch_gemv_gated(a, s);
  return a.G ? launch_cfg<BF, kGated, false, false, 1, true, true>(a, tile, s)
             : launch_cfg<BF, kGated, false, false, 1, true, false>(a, tile, s);
}

// dX = [dG dU] [Wg; Wu]: A rows hold K, B rows are K.
hipError_t launch_grad_input(const DenseArgs& a, DenseTile tile, hipStream_t s) {
  return launch_cfg<BF, kPlain, false, true, 2, true, false>(a, tile, s);
}

// dWg = dG^T X and dWu = dU^T X: the rows of both operands are K.
hipError_t launch_grad_weights(const DenseArgs& a, DenseTile tile, hipStream_t s) {
  return launch_cfg<BF, kPlain, true, true, 1, true, false>(a, tile, s);
}

}  // namespace fp4g
