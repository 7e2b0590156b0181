// Newton-Schulz orthogonalisation of weight gradients on gfx950 (the Muon
// optimiser's direction of an update), next to the gradients that wgrad and
// reduce_grad leave in grad_home [E,H,H'].
//
//   X = G / (|G| + eps), then per step  X = a X + (b A + c A A) X,  A = X X^T.
//
// Every step multiplies X from the left by a polynomial in A, and all of these
// commute, so X stays (polynomial in the first A) X_0.  The kernels therefore
// iterate on m x m matrices (m the shorter side, n the longer) and touch the
// long side twice:
//   A = X_0 X_0^T                                (first product, K = n)
//   R = I + (b A + c A A) / a                    per step
//   T = R A,  P = R P                            (P = R in the first)
//   A = a^2 R T
//   out = (prod a) P X_0                         (last product)
// All m x m matrices are symmetric, so only the tiles on and above the diagonal are
// computed, and every element above it is written twice: to the bit, for an antisymmetric
// part, however small at first, would grow to 1e-2 of the result.  Five steps are 17 such
// products, m^3 / 2 multiply-adds each, and the long side's n m^2 / 2 and n m^2; taken on X
// itself each step would have n m^2 / 2 + m^3 / 2 + n m^2.  At n = 3.5 m that is 13.75 m^3
// against 28.75 m^3.
//
// Rounding: P amplifies what is lost in A by up to prod a (485 for the usual
// five steps) in the directions of small singular values, and the gradient of
// an expert with few tokens has almost only those.  bf16 (2^-9) or fp16
// (2^-12) operands would leave nothing there, so every matrix is held as a
// pair of fp16, v = hi + lo (22 bits), and a product is hi hi + hi lo + lo hi
// on the matrix units, summed in fp32.  Before its rounding to bf16 (1.7e-3 of its norm) the
// result is then off by 1e-5 of its norm at full rank, at rank one and m up to 2048 by 3e-4 (all
// rows share its norm) to 1e-3 (two rows hold it; 4.4e-3 the worst of 40000), half of which the
// 22 bits leave even if all sums were exact.
// Values are scaled by 2^14, so entries up to 4 are held, and down to 2^-28
// with 11 or more bits.
//
// Layout: a row of k values is stored as blocks of 128 bytes, 32 hi then 32
// lo, zero behind the last value; a GEMM operand is then a 256-row tile of 128-byte
// rows, as in gemm_core.h, whose loads, swizzle and ring are used as they are.  All
// products are C = U V^T with both operands contiguous along K: the
// m x m matrices are symmetric, and G / |G| is written in both orientations (X_0 is that times
// |G| / (|G| + eps), which the first product's scale and the last one's take in).
#include <cmath>

#include "gemm_core.h"

namespace moonep {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr float kScale = 16384.0f;            // stored = value * 2^14
// Doubles per matrix in front of the workspace: partial sums of the squared norm, then |G| / (|G| +
// eps), which is kept apart from the pairs (X_0 is held as G / |G|), for a gradient far below eps
// would leave nothing in them.
constexpr int kParts = 255, kNormLd = 256;
constexpr int kK = 32;                        // values of K per step (a 64-element block)

// ------------------------------------------------------------- K loop
// A workgroup's tile is 64 MI x 64 NJ: four waves in a 2 x 2 grid, each MI x NJ
// blocks of 32 x 32.  One step = 32 values of K = two 16-deep halves, hi in
// fragment columns kk = 0, 1 and lo in kk = 2, 3: per half three groups of MI
// NJ MFMAs, h.a h.b, h.a l.b and l.a h.b.  The operand bytes of a step are
// those of 64 values in 16 bits and its MFMAs 1.5 times theirs, so the loads
// and LDS reads hide more easily than in the expert GEMMs.  The groups run
// B-fragment by B-fragment: in the third one h.b[j] is free after its MI MFMAs
// and takes the next half's, so two fragment sets suffice.
//
// The ring: kSlots = 5 slots shared by A and B as in gemm_core.h (A one step
// ahead, B two), or, kDeep, 5 slots for each (both four steps ahead), which a
// launch of few workgroups needs: its operands were just written by other XCDs,
// a load takes as long as several steps, and no second workgroup fills the gap
// (five steps on four 1024 x 2048 matrices: 537 us without, 492 us with; one of 2048 x
// 7168: 1064 and 927 us).
template <int MI, int NJ, bool kDeep>
struct Tile3 {
  static constexpr int kRows = 64 * MI, kCols = 64 * NJ;
  static constexpr int kNA = 2 * MI, kNB = 2 * NJ;                      // loads per wave and step
  static constexpr int kSlot = 128 * (kRows > kCols ? kRows : kCols);   // bytes of a ring slot
  static constexpr int kLds = (kDeep ? 2 : 1) * kSlots * kSlot;
  static constexpr int kWaveLds = kLds / 4;                             // a wave's share of the ring
  static constexpr int kAheadA = kDeep ? kSlots - 1 : 1, kAheadB = kDeep ? kSlots - 1 : 2;
  // loads that may be outstanding when the next step's tiles have to be there
  static constexpr int kLater = kDeep ? (kSlots - 2) * (kNA + kNB) : kNB;
  // a workgroup takes a CU (160 KiB of LDS), or two share one
  static constexpr int kWavesPerSimd = kLds > 81920 ? 1 : 2;
  lds_t* base;
  template <int J>
  __device__ __forceinline__ lds_t* a() const {
    return base + (kDeep ? J % kSlots : (2 * J + 1) % kSlots) * kSlot;
  }
  template <int J>
  __device__ __forceinline__ lds_t* b() const {
    return base + (kDeep ? kSlots + J % kSlots : (2 * J) % kSlots) * kSlot;
  }
};

template <int MI, int NJ>
struct Frag3 {
  bf16x8 a[MI], b[NJ];
};

template <int MI, int NJ>
__device__ __forceinline__ void mma3(f32x16 acc[MI][NJ], const bf16x8& a, const bf16x8& b, int i,
                                     int j) {
  acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, b),
                                                     __builtin_bit_cast(f16x8, a), acc[i][j], 0, 0,
                                                     0);
}

__device__ __forceinline__ bf16x8 read3(const lds_t* tile, int row0, int kk) {
  const int lane = threadIdx.x & 63;
  return RowTile::frag(tile, row0 + (lane & 31), kk, lane >> 5);
}

// at most N LDS-DMA loads of this wave outstanding
template <int N>
__device__ __forceinline__ void wait_dma() {
  static_assert(N == 4 || N == 8 || N == 12 || N == 24, "outstanding loads");
  if constexpr (N == 12) asm volatile("s_waitcnt vmcnt(12)" ::: "memory");
  else if constexpr (N == 4) asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
  else if constexpr (N == 8) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
  else asm volatile("s_waitcnt vmcnt(24)" ::: "memory");
}

// Half HALF of step j (J = j mod 5).  The loads of the A and B tiles some
// steps ahead go out between the step's first MFMAs, into slots that step j -
// 1 read; before the first fragment of step j + 1 is read comes the wait for
// that step's tiles and the barrier.  h.b[NJ-1] of a half is read at its own start.
template <int J, int HALF, int MI, int NJ, bool kDeep>
__device__ __forceinline__ void khalf3(const RowTileT<2 * MI>& la, const RowTileT<2 * NJ>& lb,
                                       const Tile3<MI, NJ, kDeep>& ring, uint32_t koa,
                                       uint32_t kob, Frag3<MI, NJ>& h, Frag3<MI, NJ>& l,
                                       f32x16 acc[MI][NJ], int arow0, int bcol0) {
  typedef Tile3<MI, NJ, kDeep> TL;
  constexpr int J1 = J + 1, JA = J + TL::kAheadA, JB = J + TL::kAheadB;
  constexpr int GRP = MI * NJ, N = 3 * GRP, NA = TL::kNA, NB = TL::kNB;
  constexpr int F = 2 * GRP + MI;                        // h.b[0] is free from here, h.a MI before
  constexpr int HA = NJ == 4 ? F + 1 : 2 * GRP;          // reads of the next h.a
  constexpr int BAR = N + (HA < F ? HA : F) - 1;
  constexpr int B0 = 3 * NA, BS = (BAR - B0) / NB;
  static_assert(BS >= 1 && B0 + (NB - 1) * BS <= BAR, "loads must precede the barrier");
  const lds_t* A = ring.template a<J>();
  const lds_t* Bt = ring.template b<J>();
  const lds_t* nA = HALF ? ring.template a<J1>() : A;    // the next half's hi fragments
  const lds_t* nB = HALF ? ring.template b<J1>() : Bt;
  constexpr int nkk = HALF ? 0 : 1;
#pragma unroll
  for (int o = 0; o < N; ++o) {
    const int p = N * HALF + o, mi = o % MI, mj = o / MI % NJ;
    if (o < GRP) mma3<MI, NJ>(acc, h.a[mi], h.b[mj], mi, mj);
    else if (o < 2 * GRP) mma3<MI, NJ>(acc, h.a[mi], l.b[mj], mi, mj);
    else mma3<MI, NJ>(acc, l.a[mi], h.b[mj], mi, mj);
    if (o == 0) h.b[NJ - 1] = read3(Bt, bcol0 + 32 * (NJ - 1), HALF);
    if (o >= 1 && o < 1 + NJ) l.b[o - 1] = read3(Bt, bcol0 + 32 * (o - 1), 2 + HALF);
    if (o >= 1 + NJ && o < 1 + NJ + MI)
      l.a[o - 1 - NJ] = read3(A, arow0 + 32 * (o - 1 - NJ), 2 + HALF);
    if (p % 3 == 1 && p / 3 < NA) la.issue1(ring.template a<JA>(), p / 3, koa);
    if (p >= B0 && (p - B0) % BS == 0 && (p - B0) / BS < NB)
      lb.issue1(ring.template b<JB>(), (p - B0) / BS, kob);
    if (p == BAR) {
      MOONEP_PIN();
      wait_dma<TL::kLater>();
      barrier_reads_done();
    }
    if (o >= HA && o < HA + MI) h.a[o - HA] = read3(nA, arow0 + 32 * (o - HA), nkk);
    if (o == F) h.b[0] = read3(nB, bcol0, nkk);
    if constexpr (NJ == 4) {
      if (o == F + MI + 1) h.b[1] = read3(nB, bcol0 + 32, nkk);
      if (o == F + 2 * MI) h.b[2] = read3(nB, bcol0 + 64, nkk);
    }
    MOONEP_PIN();
  }
}

template <int J, int MI, int NJ, bool kDeep>
__device__ __forceinline__ void kstep3(const RowTileT<2 * MI>& la, const RowTileT<2 * NJ>& lb,
                                       const Tile3<MI, NJ, kDeep>& ring, int j, int nk,
                                       Frag3<MI, NJ>& h, Frag3<MI, NJ>& l, f32x16 acc[MI][NJ],
                                       int arow0, int bcol0) {
  typedef Tile3<MI, NJ, kDeep> TL;
  const int ja = j + TL::kAheadA, jb = j + TL::kAheadB;
  const uint32_t koa = ja < nk ? la.koff((int64_t)ja * BK) : kOob;
  const uint32_t kob = jb < nk ? lb.koff((int64_t)jb * BK) : kOob;
  MOONEP_PIN();
  khalf3<J, 0, MI, NJ, kDeep>(la, lb, ring, koa, kob, h, l, acc, arow0, bcol0);
  khalf3<J, 1, MI, NJ, kDeep>(la, lb, ring, koa, kob, h, l, acc, arow0, bcol0);
}

// One step of a wave whose part of the tile is not wanted: its loads and barrier only.
template <int J, int MI, int NJ, bool kDeep>
__device__ __forceinline__ void kstep3_loads(const RowTileT<2 * MI>& la,
                                             const RowTileT<2 * NJ>& lb,
                                             const Tile3<MI, NJ, kDeep>& ring, int j, int nk) {
  typedef Tile3<MI, NJ, kDeep> TL;
  const int ja = j + TL::kAheadA, jb = j + TL::kAheadB;
  la.issue(ring.template a<J + TL::kAheadA>(), (int64_t)ja * BK, ja < nk);
  lb.issue(ring.template b<J + TL::kAheadB>(), (int64_t)jb * BK, jb < nk);
  wait_dma<TL::kLater>();
  barrier_reads_done();
}

// acc = U V^T of the tile.  kTwoSums: the sum of every five steps (160 values
// of K) starts at zero and is added to `sum` after them, in place of one chain
// over all of K.  idle: see kstep3_loads (acc is then not set).
template <int MI, int NJ, bool kDeep, bool kTwoSums>
__device__ __forceinline__ void gemm3_loop(const RowTileT<2 * MI>& la, const RowTileT<2 * NJ>& lb,
                                           const Tile3<MI, NJ, kDeep>& ring, int nk,
                                           f32x16 acc[MI][NJ], int arow0, int bcol0, bool idle) {
  typedef Tile3<MI, NJ, kDeep> TL;
  lb.issue(ring.template b<0>(), 0, true);
  la.issue(ring.template a<0>(), 0, true);
  lb.issue(ring.template b<1>(), BK, 1 < nk);
  if constexpr (kDeep) {
    la.issue(ring.template a<1>(), BK, 1 < nk);
    lb.issue(ring.template b<2>(), 2 * BK, 2 < nk);
    la.issue(ring.template a<2>(), 2 * BK, 2 < nk);
    lb.issue(ring.template b<3>(), 3 * BK, 3 < nk);
    la.issue(ring.template a<3>(), 3 * BK, 3 < nk);
  }
  if (idle) {
    wait_dma<TL::kLater>();
    barrier_reads_done();
    for (int j = 0; j < nk; j += kSlots) {
      kstep3_loads<0>(la, lb, ring, j, nk);
      if (j + 1 < nk) kstep3_loads<1>(la, lb, ring, j + 1, nk);
      if (j + 2 < nk) kstep3_loads<2>(la, lb, ring, j + 2, nk);
      if (j + 3 < nk) kstep3_loads<3>(la, lb, ring, j + 3, nk);
      if (j + 4 < nk) kstep3_loads<4>(la, lb, ring, j + 4, nk);
    }
    wait_loads<0>();
    barrier_reads_done();
    return;
  }
  f32x16 sum[kTwoSums ? MI : 1][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        acc[i][j][v] = 0.0f;
        if constexpr (kTwoSums) sum[i][j][v] = 0.0f;
      }
      // cleared here, while the first tiles are in flight
      if constexpr (kTwoSums) asm volatile("" : "+a"(sum[i][j]));
      else asm volatile("" : "+a"(acc[i][j]));
    }
  wait_dma<TL::kLater>();
  barrier_reads_done();
  Frag3<MI, NJ> h, l;
#pragma unroll
  for (int q = 0; q < NJ - 1; ++q) h.b[q] = read3(ring.template b<0>(), bcol0 + 32 * q, 0);
#pragma unroll
  for (int q = 0; q < MI; ++q) h.a[q] = read3(ring.template a<0>(), arow0 + 32 * q, 0);
  for (int j = 0; j < nk; j += kSlots) {
    kstep3<0>(la, lb, ring, j, nk, h, l, acc, arow0, bcol0);
    if (j + 1 < nk) kstep3<1>(la, lb, ring, j + 1, nk, h, l, acc, arow0, bcol0);
    if (j + 2 < nk) kstep3<2>(la, lb, ring, j + 2, nk, h, l, acc, arow0, bcol0);
    if (j + 3 < nk) kstep3<3>(la, lb, ring, j + 3, nk, h, l, acc, arow0, bcol0);
    if (j + 4 < nk) kstep3<4>(la, lb, ring, j + 4, nk, h, l, acc, arow0, bcol0);
    if constexpr (kTwoSums) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int jj = 0; jj < NJ; ++jj) {
          sum[i][jj] += acc[i][jj];
          asm volatile("" : "+a"(sum[i][jj]));
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][jj][v] = 0.0f;
        }
    }
  }
  if constexpr (kTwoSums) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj) acc[i][jj] = sum[i][jj];
  }
  wait_loads<0>();
  barrier_reads_done();
}

// The loop of the 64 x 64 tile: a wave has one block and six MFMAs a step, too
// few to slot the rest between, so the step is kept short instead.  A step's
// fragments are read while the step before is multiplied; hi hi and the two
// cross terms go to accumulators of their own (with two accumulators, chains of
// four dependent MFMAs: 18% slower for one of 1024 x 2048), which are
// added to the result every ten steps.
struct Frag1 {
  bf16x8 a[4], b[4];                                     // columns kk
};
typedef Tile3<1, 1, true> Tile1;

__device__ __forceinline__ void read1(Frag1& f, const lds_t* A, const lds_t* Bt, int arow0,
                                      int bcol0) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    f.a[kk] = read3(A, arow0, kk);
    f.b[kk] = read3(Bt, bcol0, kk);
  }
}

template <int J>
__device__ __forceinline__ void kstep1(const RowTileT<2>& la, const RowTileT<2>& lb,
                                       const Tile1& ring, int j, int nk, const Frag1& f,
                                       Frag1& next, f32x16 acc[3], int arow0, int bcol0,
                                       bool idle) {
  wait_dma<8>();                                         // step j + 1's tiles, in every wave,
  barrier_reads_done();                                  // and step j's fragments
  la.issue(ring.a<J + 4>(), (int64_t)(j + 4) * BK, j + 4 < nk);
  lb.issue(ring.b<J + 4>(), (int64_t)(j + 4) * BK, j + 4 < nk);
  if (idle) return;
  read1(next, ring.a<J + 1>(), ring.b<J + 1>(), arow0, bcol0);
  const auto mma = [&](int x, int i, int k) {
    acc[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, f.b[k]),
                                                    __builtin_bit_cast(f16x8, f.a[i]), acc[x], 0,
                                                    0, 0);
  };
  mma(1, 0, 2); mma(0, 0, 0); mma(2, 2, 0); mma(1, 1, 3); mma(0, 1, 1); mma(2, 3, 1);
}

__device__ __forceinline__ void gemm1_loop(const RowTileT<2>& la, const RowTileT<2>& lb,
                                           const Tile1& ring, int nk, f32x16& sum, int arow0,
                                           int bcol0, bool idle) {
  la.issue(ring.a<0>(), 0, true);
  lb.issue(ring.b<0>(), 0, true);
  la.issue(ring.a<1>(), BK, 1 < nk);
  lb.issue(ring.b<1>(), BK, 1 < nk);
  la.issue(ring.a<2>(), 2 * BK, 2 < nk);
  lb.issue(ring.b<2>(), 2 * BK, 2 < nk);
  la.issue(ring.a<3>(), 3 * BK, 3 < nk);
  lb.issue(ring.b<3>(), 3 * BK, 3 < nk);
  f32x16 acc[3];
#pragma unroll
  for (int v = 0; v < 16; ++v) sum[v] = acc[0][v] = acc[1][v] = acc[2][v] = 0.0f;
  wait_dma<12>();
  barrier_reads_done();
  Frag1 f, g;
  if (!idle) read1(f, ring.a<0>(), ring.b<0>(), arow0, bcol0);
  for (int j = 0; j < nk; j += 10) {
    kstep1<0>(la, lb, ring, j, nk, f, g, acc, arow0, bcol0, idle);
    if (j + 1 < nk) kstep1<1>(la, lb, ring, j + 1, nk, g, f, acc, arow0, bcol0, idle);
    if (j + 2 < nk) kstep1<2>(la, lb, ring, j + 2, nk, f, g, acc, arow0, bcol0, idle);
    if (j + 3 < nk) kstep1<3>(la, lb, ring, j + 3, nk, g, f, acc, arow0, bcol0, idle);
    if (j + 4 < nk) kstep1<4>(la, lb, ring, j + 4, nk, f, g, acc, arow0, bcol0, idle);
    if (j + 5 < nk) kstep1<0>(la, lb, ring, j + 5, nk, g, f, acc, arow0, bcol0, idle);
    if (j + 6 < nk) kstep1<1>(la, lb, ring, j + 6, nk, f, g, acc, arow0, bcol0, idle);
    if (j + 7 < nk) kstep1<2>(la, lb, ring, j + 7, nk, g, f, acc, arow0, bcol0, idle);
    if (j + 8 < nk) kstep1<3>(la, lb, ring, j + 8, nk, f, g, acc, arow0, bcol0, idle);
    if (j + 9 < nk) kstep1<4>(la, lb, ring, j + 9, nk, g, f, acc, arow0, bcol0, idle);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      sum[v] += acc[0][v] + (acc[1][v] + acc[2][v]);
      acc[0][v] = acc[1][v] = acc[2][v] = 0.0f;
    }
  }
  wait_loads<0>();
  barrier_reads_done();
}

// ---------------------------------------------------------- epilogue pieces
// A 32 x 32 block of a pair matrix is 32 rows of 128 bytes.  In LDS the
// 16-byte chunk c of row r sits at c ^ ((r >> 1) & 7), which spreads a
// column of chunks over the banks.
constexpr int kBlockBytes = 32 * 128;
__device__ __forceinline__ int blk_off(int r, int byte) {
  return r * 128 + (((byte >> 4) ^ ((r >> 1) & 7)) << 4) + (byte & 15);
}

// v is made before it is split: where hi is rounded from the unrounded product that v comes
// from (one mixed instruction), and lo from v and another hi, the two are a whole unit of hi
// apart near a tie, which a low-rank result shows 400-fold.
__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
  asm volatile("" : "+v"(v));
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

// four values of row r, columns c .. c + 3 (c % 4 == 0)
__device__ __forceinline__ void put_row4(lds_t* blk, int r, int c, const f16x4& hi,
                                         const f16x4& lo) {
  *(__attribute__((address_space(3))) u32x2*)(blk + blk_off(r, 2 * c)) =
      __builtin_bit_cast(u32x2, hi);
  *(__attribute__((address_space(3))) u32x2*)(blk + blk_off(r, 64 + 2 * c)) =
      __builtin_bit_cast(u32x2, lo);
}
// 16 bytes of the staged block's transpose: its row n0 + lane % 16, its columns 8 g .. 8 g + 7 (g
// = lane / 16), hi or lo, by the transposing LDS read (lane q of 16 points at row k0 + q / 4,
// columns n0 + 4 (q % 4) .. + 3 and gets column n0 + q, rows k0 .. k0 + 3)
__device__ __forceinline__ u32x4 read_transposed(const lds_t* blk, int n0, int lo) {
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
  i16x4 h[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int off = blk_off(8 * g + 4 * t + (q >> 2), 64 * lo + 2 * (n0 + 4 * (q & 3)));
    h[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) i16x4*)(blk + off));
  }
  return __builtin_bit_cast(u32x4, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
}
// a staged block to rows row0 .. row0 + 31 (those below `rows`) of a pair matrix, block column cb
__device__ __forceinline__ void flush_block(const lds_t* blk, uint16_t* dst, int64_t ld, int row0,
                                            int rows, int cb) {
  const int lane = threadIdx.x & 63, ch = lane & 7;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int r = t * 8 + (lane >> 3);
    const u32x4 v = *(const __attribute__((address_space(3))) u32x4*)(blk + blk_off(r, ch * 16));
    if (row0 + r < rows) *(u32x4*)(dst + (int64_t)(row0 + r) * ld + cb * 64 + ch * 8) = v;
  }
}
// its transpose likewise
__device__ __forceinline__ void flush_transposed(const lds_t* blk, uint16_t* dst, int64_t ld,
                                                 int row0, int rows, int cb) {
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int lo = t & 1, r = 16 * (t >> 1) + q;
    const u32x4 v = read_transposed(blk, 16 * (t >> 1), lo);
    if (row0 + r < rows) *(u32x4*)(dst + (int64_t)(row0 + r) * ld + cb * 64 + 32 * lo + 8 * g) = v;
  }
}
// a block on the diagonal: the part below it from the transpose, so that the
// matrix is symmetric to the bit
__device__ __forceinline__ void flush_diagonal(const lds_t* blk, uint16_t* dst, int64_t ld,
                                               int row0, int rows, int cb) {
  const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int lo = t & 1, r = 16 * (t >> 1) + q;
    const i16x8 m = __builtin_bit_cast(i16x8, read_transposed(blk, 16 * (t >> 1), lo));
    i16x8 v = *(const __attribute__((address_space(3))) i16x8*)(blk + blk_off(r, 64 * lo + 16 * g));
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * g + e < r) v[e] = m[e];
    if (row0 + r < rows)
      *(i16x8*)(dst + (int64_t)(row0 + r) * ld + cb * 64 + 32 * lo + 8 * g) = v;
  }
}

// The lane's elements of a 32 x 32 block of a pair matrix, in the layout of the accumulators
// (row lane % 32; v = 4 q + e holds column 8 q + 4 (lane / 32) + e): 16-byte loads of whole
// chunks, whose halves the two lanes of a row then trade.
struct PairBlock {
  u32x4 c[2][2];                                      // [hi, lo][chunk pair]
  __device__ __forceinline__ void load(const uint16_t* rowp, int cb) {
    const int lh = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int p = 0; p < 2; ++p) c[t][p] = *(const u32x4*)(rowp + cb * 64 + 32 * t + 8 * (2 * p + lh));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int p = 0; p < 2; ++p) c[t][p] = u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void trade() {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const auto r = __builtin_amdgcn_permlane32_swap(c[t][p][d], c[t][p][2 + d], false, false);
          c[t][p][d] = r[0];                          // q = 2 p, dword d
          c[t][p][2 + d] = r[1];                      // q = 2 p + 1
        }
  }
  __device__ __forceinline__ float value(int v) const {
    const int q = v >> 2, e = v & 3;
    const unsigned hw = c[0][q >> 1][2 * (q & 1) + (e >> 1)];
    const unsigned lw = c[1][q >> 1][2 * (q & 1) + (e >> 1)];
    const uint16_t hb = (uint16_t)(e & 1 ? hw >> 16 : hw), lb = (uint16_t)(e & 1 ? lw >> 16 : lw);
    return (float)__builtin_bit_cast(_Float16, hb) + (float)__builtin_bit_cast(_Float16, lb);
  }
};

// ------------------------------------------------------------ m x m products
// One tile of out = alpha U V^T, or I + alpha U V^T + beta in (kIn), a symmetric m x m matrix of
// which the tile's part on and above the diagonal is computed and written twice.
struct SymTile {
  const uint16_t* u;
  const uint16_t* v;
  const uint16_t* in;
  uint16_t* out;
  float alpha, beta;
  int m, uld, ld, nk;        // rows; row strides of u, v and of in, out; K steps
  int m0, n0;                // the tile's first row and column
};

template <int MI, int NJ, bool kDeep, bool kTwoSums, bool kIn>
__device__ __forceinline__ void sym_tile(const SymTile& a, const Tile3<MI, NJ, kDeep>& ring) {
  typedef Tile3<MI, NJ, kDeep> TL;
  const int m0 = a.m0, n0 = a.n0;
  const int wave = wave_id(), wm = wave >> 1, wn = wave & 1;
  const int arow0 = wm * 32 * MI, bcol0 = wn * 32 * NJ;
  // a wave wholly below the diagonal or outside the matrix
  const bool idle = n0 + bcol0 + 32 * NJ <= m0 + arow0 || m0 + arow0 >= a.m || n0 + bcol0 >= a.m;

  RowTileT<2 * MI> la;
  RowTileT<2 * NJ> lb;
  la.init(a.u + (int64_t)m0 * a.uld, a.uld, a.m - m0 < TL::kRows ? a.m - m0 : TL::kRows);
  lb.init(a.v + (int64_t)n0 * a.uld, a.uld, a.m - n0 < TL::kCols ? a.m - n0 : TL::kCols);
  f32x16 acc[MI][NJ];
  if constexpr (MI == 1 && NJ == 1)
    gemm1_loop(la, lb, ring, a.nk, acc[0][0], arow0, bcol0, idle);
  else
    gemm3_loop<MI, NJ, kDeep, kTwoSums>(la, lb, ring, a.nk, acc, arow0, bcol0, idle);
  if (idle) return;

  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  lds_t* stage = ring.base + wave * TL::kWaveLds;
  static_assert(NJ * kBlockBytes <= TL::kWaveLds, "a row of blocks is staged");
  const int ncb = a.ld / 64;                             // blocks along a row
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int row0 = m0 + arow0 + 32 * i, row = row0 + lr;
    PairBlock in[kIn ? NJ : 1];
    if constexpr (kIn) {
      const uint16_t* rowp = a.in + (int64_t)row * a.ld;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        in[j].zero();
        if (row < a.m && (n0 + bcol0) / 32 + j < ncb) in[j].load(rowp, (n0 + bcol0) / 32 + j);
      }
      MOONEP_PIN();
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int col0 = n0 + bcol0 + 32 * j;
      if (col0 < row0 || col0 / 32 >= ncb) continue;     // below the diagonal its mirror is written
      if constexpr (kIn) in[j].trade();
#pragma unroll
      for (int qd = 0; qd < 4; ++qd) {
        const int c = acc_col(qd, lh);
        f16x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = a.alpha * acc[i][j][4 * qd + e];
          if constexpr (kIn) {
            v = __builtin_fmaf(a.beta, in[j].value(4 * qd + e), v);
            if (row == col0 + c + e && row < a.m) v += kScale;
          }
          _Float16 h, l;
          split(v, h, l);
          hi[e] = h;
          lo[e] = l;
        }
        put_row4(stage + j * kBlockBytes, lr, c, hi, lo);
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int col0 = n0 + bcol0 + 32 * j;
      if (col0 < row0 || col0 / 32 >= ncb) continue;
      if (col0 == row0) {
        flush_diagonal(stage + j * kBlockBytes, a.out, a.ld, row0, a.m, col0 / 32);
      } else {
        flush_block(stage + j * kBlockBytes, a.out, a.ld, row0, a.m, col0 / 32);
        if (row0 / 32 < ncb)
          flush_transposed(stage + j * kBlockBytes, a.out, a.ld, col0, a.m, row0 / 32);
      }
    }
    MOONEP_PIN();
  }
}

// One product for nmat matrices, one or two problems (operand and result sets) per launch.
struct SymArgs {
  const uint16_t* u[2];
  const uint16_t* v[2];
  uint16_t* out[2];
  const uint16_t* in;        // (kIn, one problem)
  int64_t ustride;           // elements between matrices of u and v
  int64_t ostride;           // of in and out
  const double* factor;      // null, or a factor of each matrix's u and v, kNormLd apart
  float alpha, beta;
  int m, uld, ld, nk;        // as in SymTile
  int nt, tiles, nmat;       // square tiles along a side, of a matrix; matrices
  int64_t total;             // tiles in all
  int64_t whole;             // (ortho_sym_rounds) those not computed in four parts
};

__device__ __forceinline__ int64_t xcd_tile(int64_t total) {
  // XCD x takes the x-th eighth of the tiles: neighbouring tiles of a matrix share its L2
  const int64_t per = (total + kXcds - 1) / kXcds;
  const int64_t c = blockIdx.x / kXcds, t = (int64_t)(blockIdx.x % kXcds) * per + c;
  return c < per && t < total ? t : -1;
}

// Square tile t, `side` wide: those of a matrix cover the part on and above the diagonal, row
// by row.
__device__ __forceinline__ void sym_tile_at(const SymArgs& a, SymTile& s, int64_t t, int side) {
  const int64_t mat = t / a.tiles;
  int q = (int)(t - mat * a.tiles), ti = 0;
  for (; q >= a.nt - ti; ++ti) q -= a.nt - ti;
  const int pr = mat >= a.nmat ? 1 : 0;
  const int64_t mi = mat - (pr ? a.nmat : 0);
  s.u = a.u[pr] + mi * a.ustride;
  s.v = a.v[pr] + mi * a.ustride;
  s.in = a.in + mi * a.ostride;
  s.out = a.out[pr] + mi * a.ostride;
  s.alpha = a.alpha; s.beta = a.beta;
  s.m = a.m; s.uld = a.uld; s.ld = a.ld; s.nk = a.nk;
  s.m0 = ti * side;
  s.n0 = (ti + q) * side;
}

// One workgroup per tile; a square tile is NJ / MI of them.
template <int MI, int NJ, bool kDeep, bool kTwoSums, bool kIn>
__global__ __attribute__((amdgpu_flat_work_group_size(kThreads, kThreads),
                          amdgpu_waves_per_eu(Tile3<MI, NJ, kDeep>::kWavesPerSimd,
                                              Tile3<MI, NJ, kDeep>::kWavesPerSimd)))
void ortho_sym(SymArgs a) {
  typedef Tile3<MI, NJ, kDeep> TL;
  __shared__ __attribute__((aligned(16))) char lds_mem[TL::kLds];
  const TL ring = {(lds_t*)lds_mem};
  const int64_t t = xcd_tile(a.total);
  if (t < 0) return;
  SymTile s;
  const int part = (int)(t % (NJ / MI));
  sym_tile_at(a, s, t / (NJ / MI), TL::kCols);
  s.m0 += part * TL::kRows;
  if (a.factor) {
    const double f = a.factor[(t / (NJ / MI) / a.tiles % a.nmat) * kNormLd];
    s.alpha = (float)(s.alpha * f * f);
  }
  if (s.m0 < a.m) sym_tile<MI, NJ, kDeep, kTwoSums, kIn>(s, ring);
}

// The same with 256-wide tiles of which the last ones, those that would not fill a round of the
// CUs, are computed as four 128-wide ones each.
template <bool kIn>
__global__ __attribute__((amdgpu_flat_work_group_size(kThreads, kThreads), amdgpu_waves_per_eu(1, 1)))
void ortho_sym_rounds(SymArgs a) {
  typedef Tile3<4, 4, false> TL;
  typedef Tile3<2, 2, true> TS;
  static_assert(TL::kLds == TS::kLds, "one ring for both");
  __shared__ __attribute__((aligned(16))) char lds_mem[TL::kLds];
  const int64_t parts0 = (a.whole + kXcds - 1) / kXcds * kXcds;      // the first of the parts
  const bool whole = blockIdx.x < parts0;
  const int64_t b = whole ? blockIdx.x : blockIdx.x - parts0;
  const int64_t count = whole ? a.whole : 4 * (a.total - a.whole);
  const int64_t per = (count + kXcds - 1) / kXcds, c = b / kXcds, q = (int64_t)(b % kXcds) * per + c;
  if (c >= per || q >= count) return;
  SymTile s;
  sym_tile_at(a, s, whole ? q : a.whole + q / 4, TL::kCols);
  if (whole) {
    sym_tile<4, 4, false, false, kIn>(s, TL{(lds_t*)lds_mem});
  } else {
    s.m0 += q & 2 ? TS::kRows : 0;
    s.n0 += q & 1 ? TS::kCols : 0;
    if (s.m0 < a.m && s.n0 < a.m && s.m0 <= s.n0)
      sym_tile<2, 2, true, false, kIn>(s, TS{(lds_t*)lds_mem});
  }
}

// --------------------------------------------------------------- last product
// out = alpha U V^T as bf16 [mu][mv], dense.
struct OutArgs {
  const uint16_t* u;         // [nmat][mu][ld]
  const uint16_t* v;         // [nmat][mv][ld]
  uint16_t* out;             // [nmat][mu][mv]
  int64_t ustride, vstride;
  const double* factor;      // of each matrix, kNormLd apart
  float alpha;
  int mu, mv, ld, nk, ntm, ntn, nmat, wide;   // wide: 16-byte stores are aligned
  int64_t total;
};

template <int MI, int NJ, bool kDeep>
__global__ __attribute__((amdgpu_flat_work_group_size(kThreads, kThreads),
                          amdgpu_waves_per_eu(Tile3<MI, NJ, kDeep>::kWavesPerSimd,
                                              Tile3<MI, NJ, kDeep>::kWavesPerSimd)))
void ortho_out(OutArgs a) {
  typedef Tile3<MI, NJ, kDeep> TL;
  __shared__ __attribute__((aligned(16))) char lds_mem[TL::kLds];
  const TL ring = {(lds_t*)lds_mem};
  const int64_t t = xcd_tile(a.total);
  if (t < 0) return;
  const int per = a.ntm * a.ntn;
  const int64_t mi = t / per;
  const int q = (int)(t - mi * per), tm = q / a.ntn, tn = q % a.ntn;
  const int m0 = tm * TL::kRows, n0 = tn * TL::kCols;
  const int wave = wave_id(), wm = wave >> 1, wn = wave & 1;
  const int arow0 = wm * 32 * MI, bcol0 = wn * 32 * NJ;
  const int rows_valid = a.mu - m0 < TL::kRows ? a.mu - m0 : TL::kRows;
  const int cols_valid = a.mv - n0 < TL::kCols ? a.mv - n0 : TL::kCols;
  const bool idle = arow0 >= rows_valid || bcol0 >= cols_valid;

  RowTileT<2 * MI> la;
  RowTileT<2 * NJ> lb;
  la.init(a.u + mi * a.ustride + (int64_t)m0 * a.ld, a.ld, rows_valid);
  lb.init(a.v + mi * a.vstride + (int64_t)n0 * a.ld, a.ld, cols_valid);
  f32x16 acc[MI][NJ];
  if constexpr (MI == 1 && NJ == 1)
    gemm1_loop(la, lb, ring, a.nk, acc[0][0], arow0, bcol0, idle);
  else
    gemm3_loop<MI, NJ, kDeep, false>(la, lb, ring, a.nk, acc, arow0, bcol0, idle);
  if (idle) return;

  uint16_t* out = a.out + (mi * a.mu + m0) * (int64_t)a.mv + n0;
  const float factor = (float)a.factor[mi * kNormLd];
  const auto value = [&](float v) { return factor * (a.alpha * v); };
  typedef Stage<32 * MI, 32 * NJ> St;
  static_assert(St::kBytes <= TL::kWaveLds, "a wave's sub-tile is staged in its share of the ring");
  lds_t* reg = ring.base + wave * TL::kWaveLds;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int qd = 0; qd < 4; ++qd)
        St::put(reg, i, j, qd,
                pack_bf16x2(value(acc[i][j][4 * qd]), value(acc[i][j][4 * qd + 1])),
                pack_bf16x2(value(acc[i][j][4 * qd + 2]), value(acc[i][j][4 * qd + 3])));
  if (a.wide) {
    St::flush(reg, make_rsrc(out, (int64_t)rows_valid * a.mv * 2), arow0, a.mv, bcol0, cols_valid);
    return;
  }
  // rows that do not start on 16 bytes: one column per lane
  const int lane = threadIdx.x & 63;
  constexpr int kPer = 64 / (32 * NJ) > 0 ? 64 / (32 * NJ) : 1;      // rows per store
  for (int r0 = 0; r0 < 32 * MI; r0 += kPer)
#pragma unroll
    for (int c0 = 0; c0 < 32 * NJ; c0 += 64) {
      const int r = r0 + lane / (64 / kPer), c = c0 + lane % (64 / kPer);
      const int off = r * St::kRowBytes + (c >> 3) * 16 + 8 * (((c >> 2) & 1) ^ ((r >> 4) & 1)) +
                      2 * (c & 3);
      const uint16_t v = *(const __attribute__((address_space(3))) uint16_t*)(reg + off);
      if (arow0 + r < rows_valid && bcol0 + c < cols_valid)
        out[(int64_t)(arow0 + r) * a.mv + bcol0 + c] = v;
    }
}

// --------------------------------------------------------------- first passes
template <class T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(uint16_t v) {
  return __uint_as_float((uint32_t)v << 16);
}

// Partial sums of squares of each matrix, in 64 bits (a square in 32 bits
// would vanish for gradients below 1e-19 and overflow above 1e19).
template <class T>
__global__ __launch_bounds__(kThreads) void ortho_norm(const T* g, int64_t elems, int64_t vecs,
                                                       double* part) {
  __shared__ double sh[kThreads / 64];
  constexpr int N = 16 / (int)sizeof(T);
  const T* p = g + (int64_t)blockIdx.y * elems;
  double s = 0.0;
  struct __attribute__((aligned(16))) Vec {
    T v[N];
  };
  const int64_t step = (int64_t)kParts * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < vecs; i += step) {
    const Vec x = ((const Vec*)p)[i];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const double d = (double)to_f32<T>(x.v[e]);
      s += d * d;
    }
  }
  for (int64_t i = vecs * N + (int64_t)blockIdx.x * kThreads + threadIdx.x; i < elems; i += step) {
    const double d = (double)to_f32<T>(p[i]);
    s += d * d;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * kNormLd + blockIdx.x] = sh[0] + sh[1] + sh[2] + sh[3];
}

// G / |G| in both orientations as pairs: a 64 x 64 piece of G per workgroup.  A lane
// stores 16 bytes, hi or lo of eight values, so that eight lanes write a whole
// 128-byte block row.
template <class T>
__global__ __launch_bounds__(kThreads) void ortho_load(const T* g, int rows, int cols, float eps,
                                                       int wide, double* part, uint16_t* nat,
                                                       uint16_t* tr, int64_t nat_stride,
                                                       int64_t tr_stride) {
  __shared__ float tile[64][65];
  __shared__ double sh[kThreads / 64];
  const int64_t mi = blockIdx.z;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64, tid = threadIdx.x;
  double s = tid < kParts ? part[mi * kNormLd + tid] : 0.0;
  const T* p = g + mi * rows * (int64_t)cols;
  float x[4][4];
  struct __attribute__((aligned(4 * sizeof(T)))) Four {
    T v[4];
  };
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = r0 + (tid >> 4) + 16 * u, c = c0 + 4 * (tid & 15);
    const T* q = p + (int64_t)r * cols + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[u][e] = 0.0f;
    if (r < rows) {
      if (wide) {
        if (c < cols) {
          const Four v = *(const Four*)q;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[u][e] = to_f32<T>(v.v[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < cols) x[u][e] = to_f32<T>(q[e]);
      }
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((tid & 63) == 0) sh[tid >> 6] = s;
  __syncthreads();
  const double norm = sqrt(sh[0] + sh[1] + sh[2] + sh[3]);
  const double f = norm > 0.0 ? (double)kScale / norm : norm;         // (a NaN stays one)
  if (r0 == 0 && c0 == 0 && tid == 0) part[mi * kNormLd + kParts] = norm / (norm + (double)eps);
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      tile[(tid >> 4) + 16 * u][4 * (tid & 15) + e] = (float)((double)x[u][e] * f);
  __syncthreads();
  const int nld = (cols + kK - 1) / kK * 64, tld = (rows + kK - 1) / kK * 64;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const bool t = u >= 4;                          // then the transposed copy
    const int unit = tid + kThreads * (u & 3);      // 64 rows x 2 blocks x 8 pieces
    const int r = unit >> 4, kb = unit >> 3 & 1, piece = unit & 7, c = 32 * kb + 8 * (piece & 3);
    const int row = (t ? c0 : r0) + r, blk = (t ? r0 : c0) / 32 + kb;
    if (row >= (t ? cols : rows) || blk * 64 >= (t ? tld : nld)) continue;
    f16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      _Float16 h, l;
      split(t ? tile[c + e][r] : tile[r][c + e], h, l);
      v[e] = piece < 4 ? h : l;
    }
    uint16_t* d = t ? tr + mi * tr_stride + (int64_t)row * tld : nat + mi * nat_stride + (int64_t)row * nld;
    *(f16x8*)(d + blk * 64 + piece * 8) = v;
  }
}

// --------------------------------------------------------------------- host
int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int ceil_div(int v, int m) { return (v + m - 1) / m; }

struct OrthoLayout {
  int m, n;                       // shorter and longer side
  int sld, xld;                   // row strides (elements): m x m matrices and X_0^T; X_0
  int64_t x, xt, sq;              // elements per matrix: X_0, X_0^T, one m x m matrix
  int64_t bytes;                  // per matrix
  int group;                      // matrices taken at a time
};

OrthoLayout ortho_layout(int n, int rows, int cols) {
  OrthoLayout o;
  o.m = rows < cols ? rows : cols;
  o.n = rows < cols ? cols : rows;
  o.sld = (int)up(o.m, kK) * 2;
  o.xld = (int)up(o.n, kK) * 2;
  o.x = up((int64_t)o.m * o.xld, 128);
  o.xt = up((int64_t)o.n * o.sld, 128);
  o.sq = up((int64_t)o.m * o.sld, 128);
  o.bytes = 2 * (o.x + o.xt + 5 * o.sq) + kNormLd * (int64_t)sizeof(double);
  // Matrices per launch: enough for 8 rounds of 256-wide tiles on the 256 CUs (the last round
  // is then at most an eighth of the work); more would only take more memory.
  const int64_t nt = ceil_div(o.m, 256), tiles = nt * (nt + 1) / 2;
  const int64_t cap = (2048 + tiles - 1) / tiles;
  const int64_t groups = n < 1 ? 1 : (n + cap - 1) / cap;
  o.group = n < 1 ? 1 : (int)((n + groups - 1) / groups);
  return o;
}

// Which tiles a product takes, by how many there are (MOONEP_ORTHO_TILE_*).
//
// 256-wide ones bring half the operand bytes per multiply-add into LDS, and at the board's power
// limit bytes are time.  They are taken from one per CU on, where they cover at most 1/8 more
// than 128-wide ones do (diagonal tiles and the last row and column).  Up to 192 of them that
// would start another round are done in quarters.  Five steps, without and with quarters, and in
// 128-wide tiles: 32 of 1024 x 2048 (320 tiles) 3.19, 2.93, 3.08 ms; 8 of 2048 x 4096 (288)
// 5.43, 4.73, 5.04 ms; 16 of them (576) 9.72, 9.52, 9.77 ms.  Where they cover more, with them and
// by the rule: 40 of 896 x 1000 2.59 and 2.37 ms, 16 of 1400 x 1500 3.37 and 3.25 ms, 200 of 509 x
// 600 3.16 and 2.94 ms.
//
// 128-wide ones: from one per CU on two of their workgroups share a CU and hide each other's
// prologue and epilogue.
//
// 64-wide ones where the 128-wide ones would leave half the CUs idle (a step of theirs takes a
// third of the time), where up to two per CU of them would be a quarter or more empty, and where a
// matrix is one of either.  One of 1024 x 2048 (36 tiles of 128): 227 us against 380 us; five of
// 509 x 1283 (50): 183 and 291 us; one of 290 x 700 (6): 112 and 199 us; 24 of 290 x 700 (144, 5/8
// of them filled) 218 and 280 us; 1000 of 50 x 100 401 and 476 us; but four of 1024 x 2048 (144)
// 532 and 492 us.
//
// The last product has 256-wide tiles from half a round on: it is dense, and its
// epilogue is short (1 to 3% at 128 .. 512 tiles).
constexpr int kCus = 256, kQuarters = 192, kSmall = 128;

template <int MI, int NJ, bool kDeep, bool kTwoSums, bool kIn>
void run_sym(SymArgs& a, int problems, hipStream_t s) {
  a.nt = ceil_div(a.m, 64 * NJ);
  a.tiles = a.nt * (a.nt + 1) / 2;
  a.total = (int64_t)problems * a.nmat * a.tiles * (NJ / MI);
  ortho_sym<MI, NJ, kDeep, kTwoSums, kIn><<<(unsigned)pad_grid(a.total), kThreads, 0, s>>>(a);
}

template <bool kIn>
void run_sym_rounds(SymArgs& a, int problems, hipStream_t s) {
  a.nt = ceil_div(a.m, 256);
  a.tiles = a.nt * (a.nt + 1) / 2;
  a.total = (int64_t)problems * a.nmat * a.tiles;
  const int64_t rest = a.total % kCus;
  a.whole = rest <= kQuarters ? a.total - rest : a.total;
  const int64_t blocks = pad_grid(a.whole) + pad_grid(4 * (a.total - a.whole));
  ortho_sym_rounds<kIn><<<(unsigned)blocks, kThreads, 0, s>>>(a);
}

template <int MI, int NJ, bool kDeep>
void run_out(OutArgs& r, hipStream_t s) {
  r.ntm = ceil_div(r.mu, 64 * MI);
  r.ntn = ceil_div(r.mv, 64 * NJ);
  r.total = (int64_t)r.nmat * r.ntm * r.ntn;
  ortho_out<MI, NJ, kDeep><<<(unsigned)pad_grid(r.total), kThreads, 0, s>>>(r);
}

// The tile of a launch over n symmetric m x m products (two_sums: the one over the long side and
// the first step's, whose larger tile is 128 x 256).
int sym_tile_of(int m, int64_t n, bool two_sums) {
  const int64_t n256 = ceil_div(m, 256), n128 = ceil_div(m, 128), n64 = ceil_div(m, 64);
  const int64_t t256 = n * (n256 * (n256 + 1) / 2), t128 = n * (n128 * (n128 + 1) / 2);
  const int64_t t64 = n * (n64 * (n64 + 1) / 2);
  const bool small = t128 <= kSmall || t64 <= t128 || (t128 <= 2 * kCus && t64 <= 3 * t128);
  if (t256 >= (two_sums ? 2 * kCus : kCus) && 32 * t256 <= 9 * t128)
    return two_sums ? MOONEP_ORTHO_TILE_128X256 : MOONEP_ORTHO_TILE_256;
  if (small) return MOONEP_ORTHO_TILE_64;
  return t128 > kCus ? MOONEP_ORTHO_TILE_128 : MOONEP_ORTHO_TILE_128_DEEP;
}

int last_tile_of(int mu, int mv, int64_t n) {
  const int64_t t256 = n * ceil_div(mu, 256) * ceil_div(mv, 256);
  const int64_t t128 = n * ceil_div(mu, 128) * ceil_div(mv, 128);
  if (t256 >= kSmall) return MOONEP_ORTHO_TILE_256;
  return t128 > kSmall ? MOONEP_ORTHO_TILE_128_DEEP : MOONEP_ORTHO_TILE_64;
}

// The product of one launch (kIn: the one that adds to its operand).
template <bool kTwoSums, bool kIn>
void run_product(SymArgs& a, int problems, hipStream_t s) {
  switch (sym_tile_of(a.m, (int64_t)problems * a.nmat, kTwoSums)) {
    case MOONEP_ORTHO_TILE_64: run_sym<1, 1, true, false, kIn>(a, problems, s); break;
    case MOONEP_ORTHO_TILE_128_DEEP: run_sym<2, 2, true, kTwoSums, kIn>(a, problems, s); break;
    case MOONEP_ORTHO_TILE_128: run_sym<2, 2, false, kTwoSums, kIn>(a, problems, s); break;
    default:
      if constexpr (kTwoSums) run_sym<2, 4, false, true, kIn>(a, problems, s);
      else run_sym_rounds<kIn>(a, problems, s);
  }
}

void run_last(OutArgs& r, hipStream_t s) {
  switch (last_tile_of(r.mu, r.mv, r.nmat)) {
    case MOONEP_ORTHO_TILE_64: run_out<1, 1, true>(r, s); break;
    case MOONEP_ORTHO_TILE_128_DEEP: run_out<2, 2, true>(r, s); break;
    default: run_out<4, 4, false>(r, s);
  }
}

template <class T>
hipError_t orthogonalize(const T* g, int n, int rows, int cols, const float* co, int steps,
                         float eps, uint16_t* out, char* ws, hipStream_t s) {
  const OrthoLayout o = ortho_layout(n, rows, cols);
  const int64_t elems = (int64_t)rows * cols;
  double* part = (double*)ws;
  uint16_t* x = (uint16_t*)(ws + (int64_t)o.group * kNormLd * sizeof(double));
  uint16_t* xt = x + o.group * o.x;
  uint16_t* sq[5];
  for (int i = 0; i < 5; ++i) sq[i] = xt + o.group * o.xt + i * (o.group * o.sq);
  const bool tall = rows > cols;
  constexpr int N = 16 / (int)sizeof(T);

  for (int i0 = 0; i0 < n; i0 += o.group) {
    const int nm = n - i0 < o.group ? n - i0 : o.group;
    const T* gi = g + i0 * elems;
    const bool al = (uintptr_t)gi % 16 == 0 && elems % N == 0;
    const int wide = (uintptr_t)gi % (4 * sizeof(T)) == 0 && cols % 4 == 0;
    ortho_norm<T><<<dim3(kParts, nm), kThreads, 0, s>>>(gi, elems, al ? elems / N : 0, part);
    ortho_load<T><<<dim3(ceil_div(cols, 64), ceil_div(rows, 64), nm), kThreads, 0, s>>>(
        gi, rows, cols, eps, wide, part, tall ? xt : x, tall ? x : xt, tall ? o.xt : o.x,
        tall ? o.x : o.xt);

    SymArgs a;
    a.m = o.m;
    a.ld = o.sld;
    a.ostride = o.sq;
    a.nmat = nm;
    auto set = [&](int i, const uint16_t* u, const uint16_t* v, uint16_t* to) {
      a.u[i] = u; a.v[i] = v; a.out[i] = to;
    };
    uint16_t *A = sq[0], *R = sq[1], *Tm = sq[2], *P = sq[3], *P2 = sq[4];
    // The first product with two sums: a chain of fp32 additions over all of n would round by
    // 2e-7 .. 7e-7 of the sum, which a low-rank result shows thousands of times larger.  So it does
    // what the first step's products lose: T = R A is a fifth of its terms where a singular value
    // is one, and its rounding reaches the result 6800 times larger, that of the second step's
    // 1700 times and the third's 400 times.  Rank one, most of the norm in few rows, worst of 32 of
    // 2048 x 7168: 4.1e-3 with one chain, 2.0e-3 with two sums here, 1.8e-3 in the second step too,
    // 1.3e-3 in all (21.2, 21.6, 22.2 and 23.7 ms).
    set(0, x, x, A);
    set(1, x, x, A);
    a.in = A;
    a.ustride = o.x; a.uld = o.xld; a.nk = o.xld / BK;
    a.factor = part + kParts;
    a.alpha = 1.0f / kScale; a.beta = 0.0f;
    run_product<true, false>(a, 1, s);
    a.ustride = o.sq; a.uld = o.sld; a.nk = o.sld / BK;
    a.factor = nullptr;
    double gain = 1.0;
    for (int i = 0; i < steps; ++i) {
      const float ca = co[3 * i], cb = co[3 * i + 1], cc = co[3 * i + 2];
      const bool more = i + 1 < steps;
      gain *= ca;
      if (i > 0) {
        uint16_t* t = P;
        P = P2;
        P2 = t;
      }
      uint16_t* Ri = i == 0 ? P : R;                     // P of the first step is its R
      set(0, A, A, Ri);
      a.alpha = cc / ca / kScale; a.beta = cb / ca;
      if (i == 0) run_product<true, true>(a, 1, s);
      else run_product<false, true>(a, 1, s);
      a.alpha = 1.0f / kScale;
      int k = 0;
      if (more) set(k++, Ri, A, Tm);
      if (i > 0) set(k++, Ri, P2, P);
      if (k && i == 0) run_product<true, false>(a, k, s);
      else if (k) run_product<false, false>(a, k, s);
      if (more) {
        set(0, Ri, Tm, A);
        a.alpha = ca * ca / kScale;
        if (i == 0) run_product<true, false>(a, 1, s);
        else run_product<false, false>(a, 1, s);
      }
    }
    OutArgs r;
    r.u = tall ? xt : P;
    r.v = tall ? P : xt;
    r.ustride = tall ? o.xt : o.sq;
    r.vstride = tall ? o.sq : o.xt;
    r.out = out + i0 * elems;
    r.factor = part + kParts;
    r.alpha = (float)(gain / ((double)kScale * kScale));
    r.mu = rows; r.mv = cols; r.ld = o.sld; r.nk = o.sld / BK;
    r.nmat = nm;
    r.wide = cols % 8 == 0 && (uintptr_t)out % 16 == 0;
    run_last(r, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

bool ortho_shape_ok(int32_t n, int32_t rows, int32_t cols) {
  return n >= 0 && rows >= 1 && cols >= 1 && rows <= 65536 && cols <= 65536 &&
         (int64_t)rows * cols < (int64_t(1) << 29);
}

// Whether every matrix stays within what a pair holds, whatever the input.  The eigenvalues of
// A, R, T and P are functions of X's singular values, which start in [0, 1]; with x the largest
// they can be before a step, and l = x^2 that of A, the step's
//   r(l) = 1 + (b l + c l^2) / a  and  x' = max a x r(x^2)
// have their extremes at the ends, at the vertex of r and where a + 3 b l + 5 c l^2 = 0.
bool ortho_coeffs_ok(const float* coeffs, int32_t steps) {
  constexpr double kMax = 3.99;                          // of 65504 / 2^14
  double gain = 1.0, x = 1.0, p = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double a = coeffs[3 * i], b = coeffs[3 * i + 1], c = coeffs[3 * i + 2];
    if (!(a > 0.0) || !std::isfinite(b) || !std::isfinite(c)) return false;
    gain *= a;
    if (!(gain <= MOONEP_ORTHO_MAX_GAIN)) return false;
    const double top = x * x;
    const auto r = [&](double l) { return std::fabs(1.0 + (b * l + c * l * l) / a); };
    double most = std::fmax(1.0, r(top)), next = a * x * r(top);
    const auto at = [&](double l) {
      if (!(l > 0.0 && l < top)) return;                 // (a NaN or infinity: no such point)
      most = std::fmax(most, r(l));
      next = std::fmax(next, a * std::sqrt(l) * r(l));
    };
    at(-b / (2.0 * c));
    const double root = std::sqrt(9.0 * b * b - 20.0 * a * c);
    at((-3.0 * b + root) / (10.0 * c));
    at((-3.0 * b - root) / (10.0 * c));
    at(-a / (3.0 * b));                                  // c = 0
    p *= most;
    // R, P and T = R A; the last step's result is not held as a pair
    if (!(most <= kMax && p <= kMax && most * top <= kMax)) return false;
    x = next;
    if (i + 1 < steps && !(x * x <= kMax)) return false;
  }
  return true;
}

int64_t ortho_ws_bytes(int32_t n, int32_t rows, int32_t cols) {
  if (n == 0) return 0;
  const OrthoLayout o = ortho_layout(n, rows, cols);
  return o.group * o.bytes;
}

int32_t ortho_tile(int32_t n, int32_t rows, int32_t cols, int32_t product) {
  const OrthoLayout o = ortho_layout(n, rows, cols);
  switch (product) {
    case MOONEP_ORTHO_FIRST: return sym_tile_of(o.m, o.group, true);
    case MOONEP_ORTHO_R: case MOONEP_ORTHO_A: return sym_tile_of(o.m, o.group, false);
    case MOONEP_ORTHO_TP: return sym_tile_of(o.m, 2 * (int64_t)o.group, false);
    case MOONEP_ORTHO_LAST: return last_tile_of(rows, cols, o.group);
    default: return -1;
  }
}

hipError_t launch_orthogonalize(const void* g, int32_t dtype, int32_t n, int32_t rows,
                                int32_t cols, const float* coeffs, int32_t steps, float eps,
                                uint16_t* out, void* ws, hipStream_t s) {
  return dtype == MOONEP_F32
             ? orthogonalize((const float*)g, n, rows, cols, coeffs, steps, eps, out, (char*)ws, s)
             : orthogonalize((const uint16_t*)g, n, rows, cols, coeffs, steps, eps, out,
                             (char*)ws, s);
}

}  // namespace moonep
