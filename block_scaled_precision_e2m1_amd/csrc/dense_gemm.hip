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
//   * Small products have a CU or so to a tile and few matrix instructions a stage, and are
//     bound by the latency of one wave's instructions.  Their tiles get two groups of waves
//     (KG = 2), each multiplying half of every stage's quarters into sums of its own, which
//     the end adds: twice the waves to hide latency behind, at the same LDS reads a product.
//   * A K stage is 128 bytes of every row of A and of B (a cache line; 128 int8 or 64 bf16
//     elements), or 256 for the two "long" tiles, which halves the barriers where few tiles
//     walk a long K with a CU to themselves.  Stages live in a ring of STAGES slots, filled by buffer copies straight
//     to LDS whose resources end with the operand's tile (dense.hpp): every ragged edge
//     reads zeros.
//   * Operand forms.  A "row" operand has K contiguous: 16-byte chunk c of row r sits at
//     chunk c ^ swz(r), so ds_read_b128 of 32 rows is free of bank conflicts.  A "column"
//     operand (bf16; the gradients' products sum over rows of their operands) has K
//     strided: the stage is 64 K rows of the tile's columns, and ds_read_b64_tr_b16 turns
//     4 K rows x 16 columns into the fragment's order.  Its 64-byte units are XORed with
//     the K row's low bits, so that the four rows one read touches lie in different banks.
//   * K slots.  In quarter q of a stage ("quarters" are 32 bytes of K: 4 in a stage of 128
//     bytes), slot h (lane / 32) holds chunk 4h + q of a row, which is K elements
//     32h + 8q .. +7 for bf16: column operands read exactly those K rows.
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
#include "launch.hpp"

namespace fp4g {
namespace {

template <int ROWB>
__device__ __forceinline__ int swz(int r) { return ROWB == 128 ? ((r >> 1) & 7) ^ ((r & 1) << 2) : r & 15; }

// Column operands: the 64-byte unit u of K row k sits at unit u ^ unit_swz(k) of its LDS row, so
// the four rows k .. k+3 (k % 4 == 0) of one unit lie in different banks: rows of 256 and 512
// bytes all start in bank 0, rows of 128 bytes in alternate halves of the banks.
template <int PITCH>
__device__ __forceinline__ int unit_swz(int k) { return PITCH >= 256 ? k & 3 : (k >> 1) & 1; }

enum Form { kScaled, kGated, kPlain };

// KG groups of waves share a tile: group g multiplies quarters QN g .. of every stage, which
// is ROWB bytes of K.  OCC workgroups share a CU.
template <class T_, int FORM_, int BM_, int BN_, int WM_, int WN_, int KG_, int ROWB_, int STAGES_, int OCC_,
          bool ACOL_, bool BCOL_, int NSEG_>
struct TileCfg {
  typedef T_ T;
  static constexpr int FORM = FORM_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, KG = KG_, STAGES = STAGES_, OCC = OCC_;
  static constexpr int NSEG = NSEG_;
  static constexpr bool ACOL = ACOL_, BCOL = BCOL_, GATED = FORM_ == kGated;
  static constexpr int NWN = BN / WN, NWT = (BM / WM) * NWN, NW = NWT * KG;    // waves: of a group, of the workgroup
  static constexpr int QN = ROWB_ / 32 / KG;                  // quarters of a stage a wave multiplies
  static constexpr int ROWB = ROWB_, KE = ROWB / T::BYTES;      // bytes and elements of K per stage
  static constexpr int RPC = 1024 / ROWB, CPR = ROWB / 16;    // rows a copy, chunks a row
  static constexpr int A_BYTES = BM * ROWB, STAGE = (BM + BN) * ROWB, LDS = STAGE * STAGES;
  // 1 KB copies of a wave in a stage.
  static constexpr int IA = BM * ROWB / 1024 / NW, IB = BN * ROWB / 1024 / NW, LOADS = IA + IB;
  static constexpr int FI = WM / 32, FJ = WN / 32;
  static constexpr int OUTN = GATED ? BN / 2 : BN, WOUT = GATED ? WN / 2 : WN;   // output columns: tile, wave
  static constexpr int STRIP = WN * 4 + 16;                   // LDS pitch of a row of a wave's sums
  static_assert(!(ACOL || BCOL) || T::BYTES == 2, "column operands are bf16");
  static_assert(IA * NW * 1024 == A_BYTES && IB * NW * 1024 == BN * ROWB, "copies per wave");
  static_assert(!GATED || (IB * RPC <= WN / 2 && WN / 2 % (IB * RPC) == 0), "each wave copies rows of one weight");
  static_assert(NW * 32 * STRIP <= LDS && LDS * OCC <= 160 * 1024, "LDS");
  static_assert(STAGES >= 2 && (STAGES - 1) * LOADS < 64, "vmcnt range");
  static_assert(KG == 1 || KG == 2, "two quarters a wave at least");
};

struct Item { int l, s, tm, tn; };

// Work item `wg` of `total`: consecutive ids go to the 8 XCDs in turn, so they are regrouped
// to give each XCD a contiguous run, in which the slices of one tile are neighbours and the
// tiles go in groups of 8 tile rows, column by column.  Divisions take hundreds of cycles
// before a workgroup's first copy, so those that a small product does not need are skipped.
__device__ __forceinline__ Item item_of(int wg, int total, int S, int L, int tiles_m, int tiles_n) {
  // Runs of equal length; the first total % 8 of them take one more item.
  const int q = total >> 3, rem = total & 7, x = wg & 7;
  uint32_t lin = x * q + min(x, rem) + (wg >> 3);
  Item it{0, 0, 0, 0};
  if (S > 1) {
    it.s = lin % (uint32_t)S;
    lin /= (uint32_t)S;
  }
  if (L > 1) {
    const uint32_t T = tiles_m * tiles_n;
    it.l = lin / T;
    lin -= it.l * T;
  }
  constexpr int G = 8;
  int first = 0, size = tiles_m;
  if (tiles_m > G) {
    const uint32_t group = lin / (uint32_t)(G * tiles_n);
    first = group * G;
    size = min(G, tiles_m - first);
    lin -= first * tiles_n;
  }
  if (size == G) {
    it.tm = first + lin % G;
    it.tn = lin / G;
  } else {
    it.tn = lin / (uint32_t)size;
    it.tm = first + lin - it.tn * size;
  }
  return it;
}

// The items `block`, `block` + `grid`, .. of a product, by one workgroup.
template <class C, bool BF16, bool SAVE, bool SPLIT>
__device__ __forceinline__ void dense_gemm(const DenseArgs& a, int block, int grid, uint8_t* smem) {
  typedef typename C::T T;
  constexpr int FI = C::FI, FJ = C::FJ, QN = C::QN;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = wave / C::NWT, wt = wave % C::NWT, wm = wt / C::NWN, wn = wt % C::NWN;
  const int hi = lane >> 5, r32 = lane & 31;
  // Sizes reach 2^31 - 1: what passes them by part of a tile is formed unsigned.
  const int tiles_m = ((uint32_t)a.M + C::BM - 1) / C::BM, tiles_n = ((uint32_t)a.N + C::OUTN - 1) / C::OUTN;
  const int total = a.L * tiles_m * tiles_n * a.S;
  const int KT1 = ((uint32_t)a.K + C::KE - 1) / C::KE, KT = C::NSEG * KT1;
  const int lda = (int)a.lda, ldb = (int)a.ldb;

  // ---- the current item ----
  Item it;
  int m0 = 0, n0 = 0, ks0 = 0, KS = 0;
  auto setup = [&](int work) {
    it = item_of(work, total, a.S, a.L, tiles_m, tiles_n);
    m0 = it.tm * C::BM;
    n0 = it.tn * C::OUTN;
    ks0 = 0;
    KS = KT;
    if (SPLIT) {   // S slices; S <= 16 and KT <= 2^25 (the rows of a weight gradient), so 32 bits hold S * KT
      ks0 = (uint32_t)(it.s * KT) / (uint32_t)a.S;
      KS = (uint32_t)((it.s + 1) * KT) / (uint32_t)a.S - ks0;
    }
  };

  // ---- copies ----
  // The stage being copied, `ist` of the item's KS: where its rows start, how many bytes of the
  // operand lie from there to the tile's end, this lane's offsets, its slot.  From one
  // stage to the next only the starts move; stages before `plain` need no more than that,
  // so that the scalar work of a stage stays small (it was half of a small tile's
  // instructions when every copy formed its resource anew).
  //   Row operand, copy q of the wave: rows 8n .. 8n+7 (n = wave * I + q), 8 lanes a row.
  //   Column operand: 1 KB of the stage's 64 K rows of BM (BN) columns.
  const uint8_t *pa = nullptr, *pb = nullptr;
  int na = 0, nb = 0, ist = 0, plain = 0, wr = 0;
  uint32_t va[C::IA], vb[C::IB];
  // Gated: the rows this wave copies belong to one of the weights; within the tile, row r
  // of LDS is output column (r / WN) * WN/2 + r % (WN/2) of weight (r % WN) / (WN/2).
  const int bwhich = C::GATED ? (wave * C::IB * C::RPC) % C::WN / (C::WN / 2) : 0;
  // This lane's offset from the stage's start in copy n of a column operand of PITCH bytes a row.
  auto col_offset = [&](auto pitch_c, int n, int ld) {
    constexpr int PITCH = decltype(pitch_c)::value;
    const int p = 1024 * n + 16 * lane, k = p / PITCH, w = p % PITCH;
    return (uint32_t)k * ld + (((w >> 6) ^ unit_swz<PITCH>(k)) << 6 | (w & 63));
  };
  auto new_stage = [&]() {
    if (ist >= KS) {   // past the slice: no traffic, zeros in a slot that is not used
      na = nb = 0;
      return;
    }
    const int g = ks0 + ist, seg = C::NSEG == 2 && g >= KT1 ? 1 : 0, kk = g - seg * KT1;
    const int left = a.K - kk * C::KE;
    // The last stage of a segment may end inside a row, and the next segment starts afresh.
    plain = kk + 1 >= KT1 ? ist + 1 : min(KS, ist + KT1 - 1 - kk);
    const uint8_t* A = a.A[C::NSEG == 2 ? seg : it.l];
    const uint8_t* B = a.B[C::NSEG == 2 ? seg : bwhich];
    if constexpr (C::ACOL) {
      pa = A + (int64_t)kk * C::KE * lda + m0 * 2;
      na = min(left, C::KE) * lda - m0 * 2;
    } else {
      pa = A + (int64_t)m0 * lda + kk * C::ROWB;
      na = min(a.M - m0, C::BM) * lda - kk * C::ROWB;
    }
#pragma unroll
    for (int q = 0; q < C::IA; ++q) {
      const int n = wave * C::IA + q, row = n * C::RPC + lane / C::CPR, c = ((lane % C::CPR) ^ swz<C::ROWB>(row)) * 16;
      if constexpr (C::ACOL) va[q] = col_offset(std::integral_constant<int, C::BM * 2>{}, n, lda);
      else va[q] = c < left * T::BYTES ? (uint32_t)row * lda + c : kNoLoad;
    }
    if constexpr (C::BCOL) {
      pb = B + (int64_t)kk * C::KE * ldb + n0 * 2;
      nb = min(left, C::KE) * ldb - n0 * 2;
    } else {
      pb = B + (int64_t)n0 * ldb + kk * C::ROWB;
      nb = min(a.N - n0, C::OUTN) * ldb - kk * C::ROWB;
    }
#pragma unroll
    for (int q = 0; q < C::IB; ++q) {
      const int n = wave * C::IB + q, row = n * C::RPC + lane / C::CPR, c = ((lane % C::CPR) ^ swz<C::ROWB>(row)) * 16;
      const int src = C::GATED ? row / C::WN * (C::WN / 2) + row % (C::WN / 2) : row;
      if constexpr (C::BCOL) vb[q] = col_offset(std::integral_constant<int, C::BN * 2>{}, n, ldb);
      else vb[q] = c < left * T::BYTES ? (uint32_t)src * ldb + c : kNoLoad;
    }
  };
  auto next_stage = [&]() {
    ++ist;
    wr = wr + C::STAGE == C::LDS ? 0 : wr + C::STAGE;
    if (ist < plain) {
      pa += C::ACOL ? (int64_t)C::KE * lda : C::ROWB;
      pb += C::BCOL ? (int64_t)C::KE * ldb : C::ROWB;
      if constexpr (!C::ACOL) na -= C::ROWB;
      if constexpr (!C::BCOL) nb -= C::ROWB;
    } else {
      new_stage();
    }
  };
  // Copy q (A's, then B's) of the stage.
  auto issue_one = [&](int q) {
    if (q < C::IA) lds_buffer16(make_rsrc(pa, na), (lds_void*)(smem + wr + 1024 * (wave * C::IA + q)), va[q]);
    else
      lds_buffer16(make_rsrc(pb, nb), (lds_void*)(smem + wr + C::A_BYTES + 1024 * (wave * C::IB + q - C::IA)),
                   vb[q - C::IA]);
  };

  // ---- fragments ----
  // Of a row operand: block r's fragment of quarter j is at fo[j] + r * 32 rows.  Of a column
  // operand: at fo[r] + j * 8 K rows; the 16 lanes of a group read K rows k, k+1, k+2, k+3
  // (lane / 4) of 16 columns, and lane i of the group receives column i of all four.
  v4i fa[2][FI], fb[2][FJ];
  constexpr int NFA = C::ACOL ? FI : QN, NFB = C::BCOL ? FJ : QN;
  const int ti = lane & 15, tq = ti >> 2, tb = ((lane >> 4) & 1) * 32 + (ti & 3) * 8;
  auto row_frag = [&](int row, int j) {
    return row * C::ROWB + (((C::CPR / 2 * hi + kg * QN + j) ^ swz<C::ROWB>(r32)) << 4);
  };
  auto col_frag = [&](auto pitch_c, int blk) {
    constexpr int PITCH = decltype(pitch_c)::value;
    return (C::KE / 2 * hi + 8 * kg * QN + tq) * PITCH + ((blk ^ unit_swz<PITCH>(tq)) << 6) + tb;
  };
  int foa[NFA], fob[NFB], ca[NFA], cb[NFB];   // offsets within a slot, and with the slot's start
#pragma unroll
  for (int i = 0; i < NFA; ++i) {
    if constexpr (C::ACOL) foa[i] = col_frag(std::integral_constant<int, C::BM * 2>{}, wm * FI + i);
    else foa[i] = row_frag(wm * C::WM + r32, i);
  }
#pragma unroll
  for (int i = 0; i < NFB; ++i) {
    if constexpr (C::BCOL) fob[i] = C::A_BYTES + col_frag(std::integral_constant<int, C::BN * 2>{}, wn * FJ + i);
    else fob[i] = C::A_BYTES + row_frag(wn * C::WN + r32, i);
  }
  int rd = 0;   // the slot being read
  auto read_slot = [&]() {
#pragma unroll
    for (int i = 0; i < NFA; ++i) ca[i] = foa[i] + rd;
#pragma unroll
    for (int i = 0; i < NFB; ++i) cb[i] = fob[i] + rd;
  };
  auto read_col = [&](auto pitch_c, int at) {
    constexpr int PITCH = decltype(pitch_c)::value;
    const v2i lo = lds_read_tr16(smem + at), up = lds_read_tr16(smem + at + 4 * PITCH);
    return v4i{lo[0], lo[1], up[0], up[1]};
  };
  // Fragment x of quarter j of this wave, in the order the matrix instructions want them: the
  // first of B and of A, then the rest of B's, then of A's.
  auto read_frag = [&](int j, int x) {
    const int r = x == 1 ? 0 : x > FJ ? x - FJ : x == 0 ? FI : FI + x - 1;
    if (r < FI) {
      if constexpr (C::ACOL)
        fa[j & 1][r] = read_col(std::integral_constant<int, C::BM * 2>{}, ca[r] + j * (16 * C::BM));
      else fa[j & 1][r] = *reinterpret_cast<const v4i*>(smem + ca[j] + r * (32 * C::ROWB));
    } else {
      const int b = r - FI;
      if constexpr (C::BCOL)
        fb[j & 1][b] = read_col(std::integral_constant<int, C::BN * 2>{}, cb[b] + j * (16 * C::BN));
      else fb[j & 1][b] = *reinterpret_cast<const v4i*>(smem + cb[j] + b * (32 * C::ROWB));
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
  // When the memory instructions of a stage go out.  The fragments of the next quarter are
  // read evenly over a quarter's NQ matrix instructions, and a stage's copies evenly over
  // two quarters: the last one of the stage STAGES before it (after the barrier that frees
  // its slot) and the next stage's first.  Bursts of either stall the waves that issue them:
  // at 8192 x 14336 x 4096 the backward products take 1508 and 1585 us with one of each after
  // every matrix instruction until they are out, 1458 and 1541 us spread.  Copies spread
  // over three quarters land too late (1550 and 1555 us), in one they crowd (1604, 1681).
  constexpr int FR = FI + FJ, NQ = FI * FJ, SPAN = QN > 4 ? QN / 2 : 2;
  constexpr int LH = (C::LOADS + SPAN - 1) / SPAN;   // copies in the last quarter
  auto copies = [&](int part, int q) {   // part 0: the last quarter, 1 ..: quarters 0 ..
#pragma unroll
    for (int c = 0; c < C::LOADS; ++c)
      if (SPAN * c * NQ / C::LOADS == part * NQ + q) issue_one(c);
  };
  auto reads = [&](int j, int q) {
#pragma unroll
    for (int r = 0; r < FR; ++r)
      if (r * NQ / FR == q) read_frag(j, r);
  };
  auto mid_quarter = [&](auto j_c) {
    constexpr int J = decltype(j_c)::value;
    quarter(std::integral_constant<int, (J & 1)>{}, [&](int q) {
      reads(J + 1, q);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (J + 1 < SPAN) copies(J + 1, q);
    });
  };
  auto prologue = [&]() {
    ist = wr = rd = 0;
    new_stage();
#pragma unroll
    for (int p = 0; p < C::STAGES - 1; ++p) {
#pragma unroll
      for (int q = 0; q < C::LOADS; ++q) issue_one(q);
      next_stage();
    }
#pragma unroll
    for (int q = 0; q < LH; ++q) issue_one(q);
  };

  // Persistent: at most OCC workgroups per CU walk the items.
  for (int work = block; work < total; work += grid) {
    setup(work);
    // A lane writes row r32 of every strip of the wave's sums and reads column group `col` of it:
    // it fetches the scales of both here, so that the end does not wait for them.
    const uint32_t mw = m0 + wm * C::WM, nw = n0 + wn * C::WOUT;
    constexpr int ELEM = SPLIT || !BF16 || SAVE ? 4 : 2, V = 16 / ELEM, LPR = C::WOUT / V;
    static_assert(64 % LPR == 0 && C::STRIP % 16 == 0, "a lane keeps its columns");
    constexpr bool SCALED = !SPLIT && std::is_same<T, I8>::value;
    typedef typename std::conditional<std::is_same<T, I8>::value, int, float>::type sum_t;
    const int col = lane % LPR * V;
    const uint32_t n = nw + col;
    float sm[FI], sc[C::GATED ? 2 : 1][V];
    if constexpr (SCALED) {
#pragma unroll
      for (int i = 0; i < FI; ++i) sm[i] = a.sa[min(mw + i * 32 + r32, a.M - 1u)];
#pragma unroll
      for (int w = 0; w < (C::GATED ? 2 : 1); ++w)
#pragma unroll
        for (int e = 0; e < V; ++e) sc[w][e] = a.sb[w][min(n + e, a.N - 1u)];
    }
    __builtin_amdgcn_sched_barrier(0);   // before the copies: the counted waits below skip none of those
    prologue();
    // Stage 0 has landed once only the copies issued after it are in flight.
    wait_vmcnt<(C::STAGES - 2) * C::LOADS + LH>();
    barrier_lds();
    read_slot();
#pragma unroll
    for (int r = 0; r < FR; ++r) read_frag(0, r);
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j) acc[i][j] = typename T::acc32{};

    for (int ks = 0; ks < KS; ++ks) {
      static_for<0, QN - 1>([&](auto j) { mid_quarter(j); });
      // Stage ks+1 has landed once at most the STAGES-2 stages after it are in flight; the
      // barrier publishes it and says that every wave has read slot ks % STAGES to its end
      // (the last quarter's fragments are in registers: barrier_lds waits for LDS reads).
      wait_vmcnt<(C::STAGES - 2) * C::LOADS>();
      barrier_lds();
      next_stage();
      rd = rd + C::STAGE == C::LDS ? 0 : rd + C::STAGE;
      read_slot();
      quarter(std::integral_constant<int, (QN - 1) & 1>{}, [&](int q) {
        copies(0, q);
        __builtin_amdgcn_sched_barrier(0);
        reads(0, q);
      });
    }
    // ---- the end ----
    // No copy may still be landing when the ring is reused, and no wave may still read it.
    wait_vmcnt<0>();
    barrier_lds();
    uint8_t* strip = smem + wave * (32 * C::STRIP);
    const uint8_t* strips = smem + wt * (32 * C::STRIP);   // group 0's; the other group's is GROUP further
    constexpr int GROUP = C::NWT * 32 * C::STRIP, ROWS = 32 / C::KG;
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      if (C::KG > 1 && i > 0) barrier_lds();
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
      if constexpr (C::KG > 1) barrier_lds();
      // Out: V columns a lane, along rows; with two groups each takes half of the rows and adds
      // both groups' sums.  A batch of rows is read before the first is used: one wave a SIMD
      // would wait for LDS at every row (int8 8192^3 475.9 -> 469.2 us, dX at 8192 x 14336 x
      // 4096 1461 -> 1447 us).
      constexpr int RPI = 64 / LPR, ITERS = RPI < ROWS ? ROWS / RPI : 1;
      constexpr int MOST = C::GATED ? 2 : 4, BATCH = ITERS < MOST ? ITERS : MOST;
      static_assert(ITERS % BATCH == 0, "whole batches");
      typedef sum_t sumv __attribute__((ext_vector_type(4)));
      constexpr int W = C::GATED ? 2 : 1;
#pragma unroll 1
      for (int b = 0; b < ITERS; b += BATCH) {
        sum_t g[BATCH][W * V];
        float rs[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int row = ROWS * kg + min((b + k) * RPI + lane / LPR, ROWS - 1);
#pragma unroll
          for (int x = 0; x < W * V; x += 4) {
            const uint8_t* at = strips + row * C::STRIP + (x / V * C::WOUT + col + x % V) * 4;
            const sumv* p = reinterpret_cast<const sumv*>(at);
            sumv v = *p;
            if constexpr (C::KG > 1) v += p[GROUP / 16];
#pragma unroll
            for (int e = 0; e < 4; ++e) g[k][x + e] = v[e];
          }
          if constexpr (SCALED) rs[k] = *reinterpret_cast<const float*>(strips + row * C::STRIP + C::WN * 4);
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int r = (b + k) * RPI + lane / LPR;
          const int64_t m = (int64_t)mw + i * 32 + ROWS * kg + r;
          if (RPI > ROWS && r >= ROWS) continue;   // more lanes than rows
          if constexpr (SPLIT) {
            const int64_t pitch = partial_pitch(a.N);
            if (m < a.M && n < pitch) {
#pragma unroll
              for (int w = 0; w < W; ++w) {
                const int64_t plane = ((int64_t)it.l * a.S + it.s) * W + w;
                *reinterpret_cast<sumv*>(static_cast<sum_t*>(a.P) + (plane * a.M + m) * pitch + n) =
                    sumv{g[k][w * V], g[k][w * V + 1], g[k][w * V + 2], g[k][w * V + 3]};
              }
            }
          } else if (m < a.M && n < (uint32_t)a.N) {
            // int8 sums are exact in 32 bits and are rounded to fp32 here.
            float y[V], u[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
              y[e] = (float)g[k][e];
              if constexpr (SCALED) y[e] = y[e] * rs[k] * sc[0][e];
            }
            const int64_t at = m * a.N + n;
            const int left = a.N - (int)n;
            if constexpr (C::GATED) {
#pragma unroll
              for (int e = 0; e < V; ++e) {
                u[e] = (float)g[k][V + e];
                if constexpr (SCALED) u[e] = u[e] * rs[k] * sc[1][e];
              }
              if constexpr (SAVE) {
                // Large products' G and U would push the operands' panels out of the L2s. Forward:
                // 4096 x 2048 x 1024 43.4 -> 41.0 us, 4096^3 231.7 -> 230.6 us, 8192 x 14336 x
                // 4096 1591 -> 1603 us; with the backward pass 144.0 -> 138.5, 705 -> 700 and no
                // change (4951 and 4953 us).
                store_cols<false, C::BM == 256>(a.G, at, left, y);
                store_cols<false, C::BM == 256>(a.U, at, left, u);
              }
              gate(a.act, y, u);
            }
            store_cols<BF16>(a.D[it.l], at, left, y);
          }
        }
      }
    }
    // No wave may start the next item's copies while another still reads its strips.
    barrier_lds();
  }
}

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

// The tiles by name, for one form of product.
template <class T, int FORM, bool ACOL, bool BCOL, int NSEG>
struct Tiles {
  template <int BM, int BN, int WM, int WN, int KG, int STAGES, int OCC, int ROWB = 128>
  using Cfg = TileCfg<T, FORM, BM, BN, WM, WN, KG, ROWB, STAGES, OCC, ACOL, BCOL, NSEG>;
  typedef Cfg<256, 256, 128, 128, 1, 2, 1> t256;
  typedef Cfg<128, 128, 64, 64, 1, 2, 2> t128;
  typedef Cfg<128, 128, 64, 64, 2, 4, 1> t128_deep;
  typedef Cfg<64, 128, 32, 64, 1, 3, 2> t64x128;
  typedef Cfg<64, 64, 32, 32, 2, 5, 2> t64_deep;
  typedef Cfg<64, 64, 32, 64, 2, 3, 3> t64;
  typedef Cfg<64, 128, 32, 64, 1, 3, 1, 256> t64x128_long;
  typedef Cfg<64, 64, 32, 32, 2, 4, 1, 256> t64_long;
};
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
DensePlan dense_plan(int64_t rows, int64_t cols, int64_t L, int64_t KT, int64_t cap) {
  const int64_t cus = device_cus();
  DensePlan best{kTile64, 1, 1e30};
  for (const Tile& c : kTiles)
    for (int64_t S : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (!can_split(rows, cols, L, KT, S, cap)) break;
      const int64_t items = items_of(c, rows, cols, L) * S, full = items / (cus * c.occ), rest = items % (cus * c.occ);
      const double stages = (double)ceil_div(KT, S);
      double t = split_us(rows, cols, L, S) + (double)full * (stages * c.us[c.occ - 1] + c.item);
      if (rest) t += stages * c.us[ceil_div(rest, cus) - 1] + c.item;
      if (t < best.us) best = DensePlan{c.t, (int)S, t};
    }
  return best;
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
