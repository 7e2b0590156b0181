// The shared expert on gfx950: a gated feed-forward block that every token
// passes, dense and in token order, beside the routed experts of the MoonEP
// path (MoonEP README, "Usage > Integration": the projections are stored
// [H,H'] like theirs), and its gradients.
//
//   Z = bf16(f(X Wg) * (X Wu)),   Y = bf16(Z Wd^T + add),   f(g) = g sigma(c(g))
//   silu:      c = g
//   gelu_tanh: c = 2 sqrt(2/pi) (g + 0.044715 g^3)
// backward, with G = X Wg and U = X Wu taken again:
//   dZ = dY Wd (kept in fp32),  dU = bf16(dZ f(G)),  dG = bf16(dZ U f'(G)),
//   f'(g) = s (1 + g (1 - s) c'(g)), s = sigma(c(g))
//   dX = dG Wg^T + dU Wu^T,  dWg = X^T dG,  dWu = X^T dU,  dWd = dY^T Z
// Products are summed in fp32 on bf16 operands; Z, dG and dU are rounded once,
// to be operands.
//
// Design for CDNA4.  Two kinds of tiles:
//  - large: 256 rows by gemm_core.h's four waves and K loop, or 128 rows by eight
//    waves, by 256 columns, one workgroup per CU, where they fill the GPU;
//  - small: 128, 64 or 32 rows by 128 columns with a plain ring of LDS-DMA
//    stages, where they do not.
// Where tiles alone leave CUs idle, K is cut into splits, so that a few tokens
// still stream the weights through every CU; the splits' sums go to the workspace
// in fp32 and an elementwise kernel adds them in order (no atomics: results
// repeat) and finishes.  Bound by the matrix units at the power limit with many
// tokens (32768 of 7168 x 2048: 2.25 to 2.31 ms from card to card, 1250 to 1280
// TFLOP/s; backward 5.95 to 6.09 ms, 1260 to 1290), by
// the delivery of tiles to the CUs with a few hundred (1024: 108 us), by the
// weights' bytes with few (8: 24 us, of which the two products 20 us at 4.4 TB/s).
#include "gemm_core.h"

namespace moonep {
namespace {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------- activation
struct Act {
  float f, df;       // f(g), f'(g)
};
template <int KIND>
__device__ __forceinline__ Act activate(float g) {
  float c, dc;
  if constexpr (KIND == MOONEP_ACT_SILU) {
    c = g;
    dc = 1.0f;
  } else {
    constexpr float k = 1.5957691216057308f;      // 2 sqrt(2 / pi)
    // c(g) is far past where sigma is 0 or 1: no overflow of its cube (a NaN
    // stays in the g outside)
    const float t = fminf(fmaxf(g, -1e4f), 1e4f);
    c = k * t * (1.0f + 0.044715f * t * t);
    dc = k * (1.0f + 3 * 0.044715f * t * t);
  }
  // the hardware's reciprocal and exponential: off by about (1 + |c|) 1e-7, far
  // below the rounding to bf16 that follows; 0 below c of -87, where f(g) is below 1e-35
  const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-c));
  // s first: where it is 0, g dc may be past fp32
  const float f = g * s;
  return {f, s + f * ((1.0f - s) * dc)};
}
__device__ __forceinline__ Act activate(int kind, float g) {
  return kind == MOONEP_ACT_SILU ? activate<MOONEP_ACT_SILU>(g)
                                 : activate<MOONEP_ACT_GELU_TANH>(g);
}

__device__ __forceinline__ float bf16_of(unsigned pair, int hi) {
  return __uint_as_float(hi ? pair & 0xFFFF0000u : pair << 16);
}

// ------------------------------------------------------------- small tiles
// Column tile of 128 columns as two regions of 64 (gate and up, or two halves
// of one matrix): 64 k rows of 128 B each, whole cache lines.
typedef ColTileT<64, 2> ColTile64;
template <class T> struct TileBytes;
template <int NL> struct TileBytes<RowTileT<NL>> { static constexpr int value = NL * 4096; };
template <int NL> struct TileBytes<RowTile2<NL>> { static constexpr int value = NL * 4096; };
template <> struct TileBytes<ColTile64> { static constexpr int value = ColTile64::kBytes; };

template <class T>
__device__ __forceinline__ bf16x8 frag_of(const lds_t* tile, int base, int kk) {
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  if constexpr (T::kRows) return T::frag(tile, base + lr, kk, lh);
  else return T::frag(tile, base, kk, lh);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// The K loop of the small tiles: DEPTH stages of A and B, loads DEPTH - 1 steps
// ahead (out-of-range ones past the end keep the wait counts), one barrier a
// step: it orders the arrival of step j's stage before its reads, and all reads
// of step j - 1 before the loads into its slot.
template <int MI, int NJ, int DEPTH, class TA, class TB>
__device__ __forceinline__ void small_loop(const TA& la, const TB& lb, lds_t* lds, int j0, int j1,
                                           f32x16 (&acc)[MI][NJ], int arow0, const int (&nrow)[NJ]) {
  constexpr int kA = TileBytes<TA>::value, kStage = kA + TileBytes<TB>::value;
  constexpr int kPer = TA::kLoads + TB::kLoads;
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d) {
    const bool v = j0 + d < j1;
    la.issue(lds + d * kStage, (int64_t)(j0 + d) * BK, v);
    lb.issue(lds + d * kStage + kA, (int64_t)(j0 + d) * BK, v);
  }
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  int slot = 0;
  for (int j = j0; j < j1; ++j) {
    wait_vm<(DEPTH - 2) * kPer>();
    barrier_reads_done();
    {
      const int jn = j + DEPTH - 1;
      lds_t* to = lds + (slot == 0 ? DEPTH - 1 : slot - 1) * kStage;
      la.issue(to, (int64_t)jn * BK, jn < j1);
      lb.issue(to + kA, (int64_t)jn * BK, jn < j1);
    }
    const lds_t* A = lds + slot * kStage;
    const lds_t* Bt = A + kA;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      bf16x8 fa[MI], fb[NJ];
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[i] = frag_of<TA>(A, arow0 + 32 * i, kk);
#pragma unroll
      for (int i = 0; i < NJ; ++i) fb[i] = frag_of<TB>(Bt, nrow[i], kk);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int n = 0; n < NJ; ++n)
          acc[i][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[n], fa[i], acc[i][n], 0, 0, 0);
    }
    slot = slot == DEPTH - 1 ? 0 : slot + 1;
  }
  wait_vm<0>();                 // nothing in flight when the workgroup ends
}

// Rows of a small tile by template: waves 2 x 2 with (BM / 64) x 2 blocks each,
// or, at 32 rows, one block of 32 columns each.  DEEP: twice the stages, for
// launches that leave a CU one workgroup.
template <int BM, bool DEEP>
struct Small {
  static constexpr int MI = BM == 128 ? 2 : 1, NJ = BM == 32 ? 1 : 2;
  static constexpr int DEPTH = (BM == 128 ? 2 : BM == 64 ? 3 : 4) * (DEEP ? 2 : 1);
  static constexpr int kLds = DEPTH * (BM * 128 + 16384);
  int arow0;
  int nrow[NJ];          // the first 32 columns of a pair lie in region 0, the second in region 1
  __device__ __forceinline__ Small() {
    const int w = threadIdx.x >> 6;
    if constexpr (BM == 32) {
      arow0 = 0;
      nrow[0] = 32 * w;
    } else {
      arow0 = (w >> 1) * 32 * MI;
      nrow[0] = (w & 1) * 32;
      nrow[1] = 64 + (w & 1) * 32;
    }
  }
};

struct SmallArgs {
  // sub-problem p < 3: A [M][K] rows (or [K][M] columns), B; see small_kernel
  const uint16_t* a[3];
  const uint16_t* b[3];
  void* out[3];
  const uint16_t* add;
  float* part;
  int M, N, K;           // of every sub-problem
  int ntm, ntn, S;       // tiles of all sub-problems together: ntm x ntn, each cut into S splits
  int act, f32;
};

enum SmallOp {
  OP_GATEUP,             // rows X, columns Wg and Wu: 64 of each a tile
  OP_GRAD,               // the same, then tiles of dZ: rows dY, columns of Wd
  OP_ROWS,               // rows A, rows B: Z Wd^T
  OP_ROWS2,              // rows [dG|dU], rows [Wg|Wu]: K = 2 H'
  OP_WGRAD               // columns A, columns B: three products over the tokens
};
template <int OP, int BM> struct SmallTiles { typedef RowTileT<BM / 32> A; typedef ColTile64 B; };
template <int BM> struct SmallTiles<OP_ROWS, BM> {
  typedef RowTileT<BM / 32> A; typedef RowTileT<4> B;
};
template <int BM> struct SmallTiles<OP_ROWS2, BM> {
  typedef RowTile2<BM / 32> A; typedef RowTile2<4> B;
};
template <int BM> struct SmallTiles<OP_WGRAD, BM> { typedef ColTile64 A; typedef ColTile64 B; };

// One tile, one split.  PART: the sums go to part [S][M][all columns] in fp32
// (columns: G, U and dZ side by side for OP_GATEUP and OP_GRAD; OP_WGRAD has
// [S][3][M][N]).  Otherwise the tile is finished here: OP_GATEUP writes Z,
// OP_ROWS and OP_ROWS2 bf16 (+ add), OP_WGRAD bf16 or adds to fp32.
template <int OP, int BM, bool PART, bool DEEP>
__device__ __forceinline__ void small_tile(const SmallArgs& a, unsigned block, char* smem) {
  typedef Small<BM, DEEP> G;
  typedef typename SmallTiles<OP, BM>::A TA;
  typedef typename SmallTiles<OP, BM>::B TB;
  constexpr int MI = G::MI, NJ = G::NJ;
  const G g;
  // each XCD takes a run of tiles: M fastest (they share the weights), then N, then the split
  const int64_t total = (int64_t)a.ntm * a.ntn * a.S, per = (total + kXcds - 1) / kXcds;
  const int64_t l = (int64_t)(block % kXcds) * per + block / kXcds;
  if (block / kXcds >= per || l >= total) return;
  const int tm = (int)(l % a.ntm);
  int tn = (int)(l / a.ntm % a.ntn);
  const int sp = (int)(l / ((int64_t)a.ntm * a.ntn));
  const int m0 = tm * BM;
  const int mv = a.M - m0 < BM ? a.M - m0 : BM;
  const int nk = (a.K + BK - 1) / BK;
  const int j0 = (int)((int64_t)nk * sp / a.S), j1 = (int)((int64_t)nk * (sp + 1) / a.S);
  int p = 0;                     // sub-problem
  if constexpr (OP == OP_GRAD) {
    const int gu = a.N / 64;
    if (tn >= gu) {
      p = 2;
      tn -= gu;
    }
  }
  if constexpr (OP == OP_WGRAD) {
    const int each = a.ntn / 3;
    p = tn / each;
    tn -= p * each;
  }
  const bool pair = (OP == OP_GATEUP || OP == OP_GRAD) && p == 0;
  const int n0 = tn * (pair ? 64 : 128);
  const int nv = a.N - n0 < (pair ? 64 : 128) ? a.N - n0 : (pair ? 64 : 128);
  TA la;
  TB lb;
  const uint16_t *pa = a.a[p], *pb = a.b[p];
  if constexpr (OP == OP_GATEUP || OP == OP_GRAD) {
    la.init(pa + (int64_t)m0 * a.K, a.K, mv);
    if (pair) lb.init(pb + n0, a.b[1] + n0, a.N, a.K, nv, nv);
    else lb.init(pb + n0, pb + n0 + 64, a.N, a.K, nv < 64 ? nv : 64, nv < 64 ? 0 : nv - 64);
  } else if constexpr (OP == OP_ROWS) {
    la.init(pa + (int64_t)m0 * a.K, a.K, mv);
    lb.init(pb + (int64_t)n0 * a.K, a.K, nv);
  } else if constexpr (OP == OP_ROWS2) {
    const int k1 = a.K / 2;
    la.init(pa + (int64_t)m0 * k1, a.a[1] + (int64_t)m0 * k1, k1, mv, k1);
    lb.init(pb + (int64_t)n0 * k1, a.b[1] + (int64_t)n0 * k1, k1, nv, k1);
  } else {
    la.init(pa + m0, pa + m0 + 64, a.M, a.K, mv < 64 ? mv : 64, mv < 64 ? 0 : mv - 64);
    lb.init(pb + n0, pb + n0 + 64, a.N, a.K, nv < 64 ? nv : 64, nv < 64 ? 0 : nv - 64);
  }
  f32x16 acc[MI][NJ];
  small_loop<MI, NJ, G::DEPTH>(la, lb, (lds_t*)smem, j0, j1, acc, g.arow0, g.nrow);

  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  if constexpr (PART) {
    const int64_t cols = OP == OP_GATEUP ? 2LL * a.N : OP == OP_GRAD ? 3LL * a.N : a.N;
    float* out = a.part + (OP == OP_WGRAD ? (int64_t)sp * 3 + p : sp) * a.M * cols;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int m = g.arow0 + 32 * i + lr;
      if (m >= mv) continue;
      float* row = out + (int64_t)(m0 + m) * cols;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          int c = g.nrow[j] + acc_col(q, lh);
          int64_t col;
          if (pair) {
            const int up = c >> 6;
            c &= 63;
            col = (int64_t)up * a.N + n0 + c;
          } else {
            col = (int64_t)p * (OP == OP_GRAD ? a.N : 0) + n0 + c;
          }
          if (c < nv)
            *(f32x4*)(row + col) = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                         acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        }
    }
  } else if constexpr (OP == OP_GATEUP && BM == 32) {
    // waves 0, 1 hold the gate's columns, 2, 3 the up's: these go by way of LDS
    typedef __attribute__((address_space(3))) f32x4 lds_f4;
    constexpr int kRow = 36;                       // floats
    const int w = threadIdx.x >> 6;
    lds_t* at = (lds_t*)smem + ((w & 1) * 32 + lr) * kRow * 4;
    __syncthreads();                               // every wave has read its last stage
    if (w >= 2) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(lds_f4*)(at + acc_col(q, lh) * 4) = f32x4{acc[0][0][4 * q], acc[0][0][4 * q + 1],
                                                    acc[0][0][4 * q + 2], acc[0][0][4 * q + 3]};
    }
    __syncthreads();
    if (w >= 2 || lr >= mv) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = 32 * w + acc_col(q, lh);
      if (c >= nv) continue;
      const f32x4 u = *(const lds_f4*)(at + acc_col(q, lh) * 4);
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = activate(a.act, acc[0][0][4 * q + e]).f * u[e];
      *(u32x2*)((uint16_t*)a.out[0] + (int64_t)(m0 + lr) * a.N + n0 + c) =
          u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
  } else {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int m = g.arow0 + 32 * i + lr;
      if (m >= mv) continue;
#pragma unroll
      for (int j = 0; j < (OP == OP_GATEUP ? 1 : NJ); ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = g.nrow[j] + acc_col(q, lh);
          if (c >= nv) continue;
          const int64_t at = (int64_t)(m0 + m) * a.N + n0 + c;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
          if constexpr (OP == OP_GATEUP) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = activate(a.act, v[e]).f * acc[i][1][4 * q + e];
          }
          if constexpr (OP == OP_ROWS) {
            if (a.add) {
              const u32x2 d = *(const u32x2*)(a.add + at);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] += bf16_of(d[e >> 1], e & 1);
            }
          }
          if (OP == OP_WGRAD && a.f32) {
            f32x4* w = (f32x4*)((float*)a.out[p] + at);
            f32x4 o = *w;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] += v[e];
            *w = o;
          } else {
            *(u32x2*)((uint16_t*)a.out[p] + at) = u32x2{pack_bf16x2(v[0], v[1]),
                                                        pack_bf16x2(v[2], v[3])};
          }
        }
    }
  }
}

template <int OP, int BM, bool PART, bool DEEP>
__global__ __launch_bounds__(kThreads, DEEP ? 1 : 2) void small_kernel(SmallArgs a) {
  __shared__ __attribute__((aligned(16))) char smem[Small<BM, DEEP>::kLds];
  small_tile<OP, BM, PART, DEEP>(a, blockIdx.x, smem);
}

// dX and the weight gradients, which both need dG and dU and not each other, in
// one launch: the first nx workgroups are dX's.
template <int BM, bool DEEP>
__global__ __launch_bounds__(kThreads, DEEP ? 1 : 2) void small_last(SmallArgs x, SmallArgs w,
                                                                     unsigned nx) {
  constexpr int kX = Small<BM, DEEP>::kLds, kW = Small<128, DEEP>::kLds;
  __shared__ __attribute__((aligned(16))) char smem[kX > kW ? kX : kW];
  if (blockIdx.x < nx) small_tile<OP_ROWS2, BM, false, DEEP>(x, blockIdx.x, smem);
  else small_tile<OP_WGRAD, 128, false, DEEP>(w, blockIdx.x - nx, smem);
}

// Z Wd^T (+ add) of up to 32 tokens without splits between workgroups: a
// workgroup takes 32 rows of Wd and its four waves every fourth 64 values of K,
// each with stages of its own, so that nothing but its own loads holds a wave up
// until the four sums are added in LDS.
struct Wave32 {
  static constexpr int kDepth = 4, kStage = 4 * 8192;        // A and B of each wave
  static constexpr int kLds = kDepth * kStage;
};
__global__ __launch_bounds__(kThreads, 1) void few_rows(SmallArgs a) {
  __shared__ __attribute__((aligned(16))) char smem[Wave32::kLds];
  const int w = wave_id(), lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  const int n0 = blockIdx.x * 32, blocks = a.K / BK, steps = (blocks + 3) / 4;
  const DmaRsrc ra = make_dma_rsrc(a.a[0], (int64_t)a.M * a.K * 2);
  const DmaRsrc rb = make_dma_rsrc(a.b[0] + (int64_t)n0 * a.K, 32LL * a.K * 2);
  // as RowTileT: load i holds rows 8 i .. 8 i + 7
  const int r = lane >> 3, c = (lane & 7) ^ RowTile::swz(r);
  const uint32_t voff[2] = {(uint32_t)(r * a.K * 2 + c * 16), (uint32_t)(r * a.K * 2 + (c ^ 4) * 16)};
  lds_t* mine = (lds_t*)smem + w * 8192;
  auto issue = [&](int j) {
    const int b = 4 * j + w;
    const uint32_t ko = b < blocks ? (uint32_t)(b * BK * 2) : kOob;
    lds_t* to = mine + (j % Wave32::kDepth) * Wave32::kStage;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = voff[i & 1] + (ko + (uint32_t)(16 * i * a.K));
      load_lds(ra, to + i * 1024, at);
      load_lds(rb, to + 4096 + i * 1024, at);
    }
  };
#pragma unroll
  for (int j = 0; j < Wave32::kDepth - 1; ++j) issue(j);
  f32x16 acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
  for (int j = 0; j < steps; ++j) {
    wait_vm<(Wave32::kDepth - 2) * 8>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // step j - 1 is read
    issue(j + Wave32::kDepth - 1);
    const lds_t* A = mine + (j % Wave32::kDepth) * Wave32::kStage;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(RowTile::frag(A + 4096, lr, kk, lh),
                                                    RowTile::frag(A, lr, kk, lh), acc, 0, 0, 0);
  }
  wait_vm<0>();
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  // rows of 32 sums and a gap: 36 words
  __attribute__((address_space(3))) float* sums = (__attribute__((address_space(3))) float*)mine;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *(__attribute__((address_space(3))) f32x4*)(sums + lr * 36 + acc_col(q, lh)) =
        f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
  __syncthreads();
  const int m = threadIdx.x >> 3, col = 4 * (threadIdx.x & 7);
  if (m >= a.M) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const f32x4 t = *(const __attribute__((address_space(3))) f32x4*)(
        (const __attribute__((address_space(3))) float*)((lds_t*)smem + s * 8192) + m * 36 + col);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += t[e];
  }
  const int64_t at = (int64_t)m * a.N + n0 + col;
  if (a.add) {
    const u32x2 d = *(const u32x2*)(a.add + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += bf16_of(d[e >> 1], e & 1);
  }
  *(u32x2*)((uint16_t*)a.out[0] + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// ------------------------------------------------------------- joins
// Four neighbouring elements of every split of NP products (at p + i step),
// added in the splits' order; eight splits' loads are in flight together (one
// at a time 16 of them took 9 us for 8 tokens).
template <int NP>
__device__ __forceinline__ void add_splits(f32x4 (&v)[NP], const float* p, int64_t step, int S,
                                           int64_t slab) {
#pragma unroll
  for (int i = 0; i < NP; ++i) v[i] = f32x4{0, 0, 0, 0};
  for (int s0 = 0; s0 < S; s0 += 8) {
    f32x4 t[8][NP];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k == 0 || s0 + k < S) {
#pragma unroll
        for (int i = 0; i < NP; ++i) t[k][i] = *(const f32x4*)(p + (s0 + k) * slab + i * step);
      }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k == 0 || s0 + k < S) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][e] += t[k][i][e];
      }
  }
}
constexpr int kJoin = 64;      // threads of a joining workgroup
__device__ __forceinline__ u32x2 pack4(const float v[4]) {
  return u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// z [M,N] from part [S][M][2N]; with dZ (part [S][M][3N]) dg, du and z.
template <bool GRAD>
__global__ __launch_bounds__(kJoin) void join_gate(const float* part, int S, int M, int N, int act,
                                                 uint16_t* z, uint16_t* dg, uint16_t* du) {
  const int64_t i = ((int64_t)blockIdx.x * kJoin + threadIdx.x) * 4;
  if (i >= (int64_t)M * N) return;
  const int64_t m = i / N, n = i % N, cols = (GRAD ? 3LL : 2LL) * N, slab = (int64_t)M * cols;
  f32x4 v[GRAD ? 3 : 2];
  add_splits(v, part + m * cols + n, N, S, slab);
  const f32x4 g = v[0], u = v[1], dz = v[GRAD ? 2 : 0];
  float zv[4], dgv[4], duv[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const Act t = activate(act, g[e]);
    zv[e] = t.f * u[e];
    dgv[e] = dz[e] * u[e] * t.df;
    duv[e] = dz[e] * t.f;
  }
  *(u32x2*)(z + i) = pack4(zv);
  if constexpr (GRAD) {
    *(u32x2*)(dg + i) = pack4(dgv);
    *(u32x2*)(du + i) = pack4(duv);
  }
}

// out [n] bf16 from part [S][n] (+ add)
__global__ __launch_bounds__(kJoin) void join_rows(const float* part, int S, int64_t n,
                                                 const uint16_t* add, uint16_t* out) {
  const int64_t i = ((int64_t)blockIdx.x * kJoin + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4 s[1];
  add_splits(s, part + i, 0, S, n);
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = s[0][e];
  if (add) {
    const u32x2 d = *(const u32x2*)(add + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += bf16_of(d[e >> 1], e & 1);
  }
  *(u32x2*)(out + i) = pack4(v);
}

// dw_p [n] from part [S][3][n]: bf16, or added to fp32
struct JoinW {
  void* out[3];
};
__global__ __launch_bounds__(kJoin) void join_wgrad(const float* part, int S, int64_t n, int f32,
                                                  JoinW w) {
  const int64_t i = ((int64_t)blockIdx.x * kJoin + threadIdx.x) * 4;
  if (i >= n) return;
  const int p = blockIdx.y;
  f32x4 s[1];
  add_splits(s, part + p * n + i, 0, S, 3 * n);
  if (f32) {
    f32x4* o = (f32x4*)((float*)w.out[p] + i);
    f32x4 t = *o;
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] += s[0][e];
    *o = t;
  } else {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = s[0][e];
    *(u32x2*)((uint16_t*)w.out[p] + i) = pack4(v);
  }
}

// ------------------------------------------------------------- large tiles
// A 256-row tile is four waves of 128 x 128 on gemm_core.h's loop.  A 128-row
// one (128 x 256) is eight waves of 64 x 64, two to a SIMD: a step has half the
// MFMAs, and one wave's waits for the barrier and for LDS are then filled by the
// other (against four waves of 64 x 128 in as many stages: 4000 tokens of 512 x
// 768 26.5 -> 24.3 us; the same at 1024 tokens of 7168 x 2048, where either way
// the tiles' bytes, 48 KiB a step and CU, arrive at 27 bytes a clock, like the 64
// KiB of the 256-row tiles).
struct Four {
  static constexpr int kWaves = 4, NJ = 4;
  template <int MI> struct Tiles {
    typedef RowTileT<2 * MI> A;
    typedef RowTile2<2 * MI> A2;
    typedef RowTile B;
    typedef RowTile2<8> B2;
    typedef ColTile Col;
  };
};

typedef ColTileT<128, 4> ColTile8;     // gemm_core.h's column tile loaded by eight waves
struct Eight {
  static constexpr int kWaves = 8, NJ = 2;
  template <int MI> struct Tiles {
    typedef RowTileT<2> A;
    typedef RowTile2<2> A2;
    typedef RowTileT<4> B;
    typedef RowTile2<4> B2;
    typedef ColTile8 Col;
  };
};

// K loop of eight waves: three whole stages of 48 KiB (A 16, B 32), all loads
// two steps ahead.  Step j = 16 MFMAs a wave in four sub-steps; a sub-step reads
// the next one's four fragments, the loads go out after every second MFMA, and
// the barrier comes when the step's last fragments are read: it orders the
// arrival of step j + 1's stage before its reads, and all reads of step j before
// the loads of step j + 3 into its stage.
constexpr int kMidA = 16384, kMidStage = kMidA + kSlotBytes;
struct Frags8 {
  bf16x8 a[2], b[2];
};
template <class TA, class TB>
__device__ __forceinline__ void read_frag8(Frags8& f, int q, const lds_t* A, int kk, int arow0,
                                           const int (&nrow)[2]) {
  if (q == 0 || q == 3) f.a[q / 3] = frag_of<TA>(A, arow0 + 32 * (q / 3), kk);
  else f.b[q - 1] = frag_of<TB>(A + kMidA, nrow[q - 1], kk);
}
template <int J, class TA, class TB>
__device__ __forceinline__ void eight_step(const TA& la, const TB& lb, lds_t* base, int j, int nk,
                                           Frags8& f0, Frags8& f1, f32x16 (&acc)[2][2], int arow0,
                                           const int (&nrow)[2]) {
  static_assert(TA::kLoads == 2 && TB::kLoads == 4, "the wait counts a stage's loads");
  constexpr int P = 16, BAR = 11;
  const lds_t* A = base + J * kMidStage;
  const lds_t* An = base + (J + 1) % 3 * kMidStage;
  lds_t* to = base + (J + 2) % 3 * kMidStage;
  const uint32_t koa = j + 2 < nk ? la.koff((int64_t)(j + 2) * BK) : kOob;
  const uint32_t kob = j + 2 < nk ? lb.koff((int64_t)(j + 2) * BK) : kOob;
  MOONEP_PIN();
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int sub = p / 4, idx = p % 4;
    Frags8& f = (sub & 1) ? f1 : f0;
    acc[idx >> 1][idx & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
        f.b[idx & 1], f.a[idx >> 1], acc[idx >> 1][idx & 1], 0, 0, 0);
    if (sub < 3) read_frag8<TA, TB>((sub & 1) ? f0 : f1, idx, A, sub + 1, arow0, nrow);
    if (p & 1) {
      if (p / 2 < 2) la.issue1(to, p / 2, koa);
      else if (p / 2 < 6) lb.issue1(to + kMidA, p / 2 - 2, kob);
    }
    if (p == BAR) {
      MOONEP_PIN();
      wait_vm<6>();
      barrier_reads_done();
    }
    if (p > BAR) read_frag8<TA, TB>(f0, p - BAR - 1, An, 0, arow0, nrow);
    MOONEP_PIN();
  }
}

template <class G, int MI, class TA, class TB>
__device__ __forceinline__ void product(const TA& la, const TB& lb, const Ring& ring, int nk,
                                        f32x16 (&acc)[MI][G::NJ], int arow0,
                                        const int (&nrow)[G::NJ]) {
  if constexpr (G::kWaves == 4) {
    gemm_loop<MI>(la, lb, ring, nk, acc, arow0, nrow);
  } else {
    lds_t* base = ring.base;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      la.issue(base + d * kMidStage, d * BK, d < nk);
      lb.issue(base + d * kMidStage + kMidA, d * BK, d < nk);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    wait_vm<6>();
    barrier_reads_done();
    Frags8 f0, f1;
#pragma unroll
    for (int q = 0; q < 4; ++q) read_frag8<TA, TB>(f0, q, base, 0, arow0, nrow);
    for (int j = 0; j < nk; j += 3) {
      eight_step<0>(la, lb, base, j, nk, f0, f1, acc, arow0, nrow);
      if (j + 1 < nk) eight_step<1>(la, lb, base, j + 1, nk, f0, f1, acc, arow0, nrow);
      if (j + 2 < nk) eight_step<2>(la, lb, base, j + 2, nk, f0, f1, acc, arow0, nrow);
    }
    wait_vm<0>();
    __syncthreads();               // the stages may be reused
  }
}

struct LargeArgs {
  const uint16_t* x;
  const uint16_t* dy;
  const uint16_t* w[3];
  const uint16_t* add;
  uint16_t* z;
  uint16_t* y;
  float* dz;
  uint16_t* dg;
  uint16_t* du;
  uint16_t* dx;
  void* dw[3];
  float* part;           // sums of the splits, fp32
  int T, H, Hp, act, f32;
  int ntm, ntn, S;
};

struct LargeTile {
  int m0, rows, nt, sp;
};
// M-tiles of `height` rows in groups of eight, each group swept over the
// N-tiles, as in gemm_core.h: what runs together on an XCD shares weight slabs.
__device__ __forceinline__ bool large_tile(const LargeArgs& a, int height, LargeTile* t,
                                           unsigned block) {
  const int64_t each = (int64_t)a.ntm * a.ntn, total = each * a.S, per = (total + kXcds - 1) / kXcds;
  int64_t l = (int64_t)(block % kXcds) * per + block / kXcds;
  if (block / kXcds >= per || l >= total) return false;
  t->sp = (int)(l / each);
  l -= t->sp * each;
  const int group = (int)(l / (8LL * a.ntn));
  const int gm = a.ntm - 8 * group < 8 ? a.ntm - 8 * group : 8;
  const int rem = (int)(l - 8LL * group * a.ntn);
  t->nt = rem / gm;
  t->m0 = (8 * group + rem % gm) * height;
  t->rows = a.T - t->m0 < height ? a.T - t->m0 : height;
  return true;
}

// Where a wave's blocks lie in a tile: rows m0 + 32 i; columns of block j at
// col(j), or, of a pair of 128-column regions (gate and up), with the first half
// of its blocks in the one and the other half at the same columns of the other.
template <class G, int MI>
struct Waves {
  static constexpr int NJ = G::NJ, kHalf = NJ / 2, kAcross = G::kWaves / 2;
  int w, m0, n;                            // wave, its first row, its place along N
  int nrow[NJ], pair[NJ];
  __device__ __forceinline__ Waves() {
    w = threadIdx.x >> 6;
    n = w % kAcross;
    m0 = w / kAcross * 32 * MI;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      nrow[j] = 32 * (NJ * n + j);
      pair[j] = 128 * (j / kHalf) + 32 * (kHalf * n + j % kHalf);
    }
  }
};

// 256 rows in tiles of four waves (a last one of up to 128 rows with half the
// blocks), 128 rows in tiles of eight.
#define MOONEP_LARGE(name, body)                                                           \
  __global__ __attribute__((amdgpu_flat_work_group_size(256, 256),                         \
                            amdgpu_waves_per_eu(1, 1))) void name##_256(LargeArgs a) {     \
    MOONEP_RING(smem);                                                                     \
    LargeTile t;                                                                           \
    if (!large_tile(a, 256, &t, blockIdx.x)) return;                                       \
    if (t.rows <= kHalfTileM) body<Four, 2, false>(a, smem, t);                            \
    else body<Four, 4, false>(a, smem, t);                                                 \
  }                                                                                        \
  MOONEP_LARGE_128(name##_128, body, false)
// PART: one of S splits of K, whose sums go to a.part [S][T][columns] in fp32.
#define MOONEP_LARGE_128(name, body, PART)                                                 \
  __global__ __attribute__((amdgpu_flat_work_group_size(512, 512),                         \
                            amdgpu_waves_per_eu(2, 2))) void name(LargeArgs a) {           \
    MOONEP_RING(smem);                                                                     \
    LargeTile t;                                                                           \
    if (!large_tile(a, 128, &t, blockIdx.x)) return;                                       \
    body<Eight, 2, PART>(a, smem, t);                                                      \
  }

// Steps [j0, j0 + n) of K of a split.
struct Steps {
  int j0, n;
};
template <bool PART>
__device__ __forceinline__ Steps steps_of(const LargeArgs& a, const LargeTile& t, int nk) {
  if constexpr (!PART) return {0, nk};
  const int j0 = (int)((int64_t)nk * t.sp / a.S);
  return {j0, (int)((int64_t)nk * (t.sp + 1) / a.S) - j0};
}

// The accumulators to fp32 rows: block j of this lane's row lies at row + col[j].
template <class G, int MI>
__device__ __forceinline__ void store_f32(const f32x16 (&acc)[MI][G::NJ], const Waves<G, MI>& at,
                                          float* out, int64_t ld, int rows,
                                          const int64_t (&col)[G::NJ], const int (&left)[G::NJ]) {
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = at.m0 + 32 * i + lr;
    if (m >= rows) continue;
    float* row = out + (int64_t)m * ld;
#pragma unroll
    for (int j = 0; j < G::NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = acc_col(q, lh);
        if (c < left[j])
          *(f32x4*)(row + col[j] + c) = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                              acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      }
  }
}

// 128 gate and 128 up columns, K = H.
template <class G, int MI, bool PART>
__device__ __forceinline__ void gateup_product(const LargeArgs& a, const Ring& smem,
                                               const LargeTile& t, f32x16 (&acc)[MI][G::NJ],
                                               const Waves<G, MI>& at) {
  const int n0 = t.nt * 128, nv = a.Hp - n0 < 128 ? a.Hp - n0 : 128;
  const Steps k = steps_of<PART>(a, t, a.H / BK);
  const int64_t k0 = (int64_t)k.j0 * BK;
  typename G::template Tiles<MI>::A la;
  typename G::template Tiles<MI>::Col lb;
  la.init(a.x + (int64_t)t.m0 * a.H + k0, a.H, t.rows);
  lb.init(a.w[0] + k0 * a.Hp + n0, a.w[1] + k0 * a.Hp + n0, a.Hp, a.H - k0, nv, nv);
  product<G, MI>(la, lb, smem, k.n, acc, at.m0, at.pair);
}

template <class G, int MI, bool PART>
__device__ __forceinline__ void large_gateup_tile(const LargeArgs& a, const Ring& smem,
                                                  const LargeTile& t) {
  typedef Waves<G, MI> Wv;
  const Wv at;
  const int n0 = t.nt * 128, nv = a.Hp - n0 < 128 ? a.Hp - n0 : 128;
  f32x16 acc[MI][G::NJ];
  gateup_product<G, MI, PART>(a, smem, t, acc, at);
  if constexpr (PART) {
    int64_t col[G::NJ];
    int left[G::NJ];
#pragma unroll
    for (int j = 0; j < G::NJ; ++j) {
      const int c = at.pair[j] & 127;
      col[j] = (at.pair[j] >> 7) * (int64_t)a.Hp + n0 + c;
      left[j] = nv - c;
    }
    store_f32<G, MI>(acc, at, a.part + ((int64_t)t.sp * a.T + t.m0) * 2 * a.Hp, 2LL * a.Hp, t.rows,
                     col, left);
    return;
  }
  // 32 rows at a time through LDS, to be stored as whole rows
  typedef Stage<32, 32 * Wv::kHalf> St;
  lds_t* reg = smem.base + at.w * St::kBytes;
  const Rsrc zs = make_rsrc(a.z + (int64_t)t.m0 * a.Hp + n0, (int64_t)t.rows * a.Hp * 2);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
#pragma unroll
    for (int j = 0; j < Wv::kHalf; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          z[e] = activate(a.act, acc[i][j][4 * q + e]).f * acc[i][j + Wv::kHalf][4 * q + e];
        St::put(reg, 0, j, q, pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
      }
    St::flush(reg, zs, at.m0 + 32 * i, a.Hp, at.pair[0], nv);
  }
}

// What is added to 32 rows of a wave's 32 NJ columns, as it is stored: lane l has
// eight columns of one of an access's 64 / kLanes rows.  Places past the tile's
// rows or columns read one inside it, for loads under a condition would each
// wait behind a branch; what they give is never stored.
template <int NJ>
struct Added {
  static constexpr int kLanes = 4 * NJ, kRows = 64 / kLanes, kPieces = 32 / kRows;
  u32x4 v[kPieces];
  __device__ __forceinline__ void load(const uint16_t* add, int64_t ld, int m0, int rows, int c0,
                                       int cols) {
    const int lane = threadIdx.x & 63, c = c0 + 8 * (lane % kLanes);
    if (!add) {
#pragma unroll
      for (int t = 0; t < kPieces; ++t) v[t] = u32x4{0, 0, 0, 0};
      return;
    }
#pragma unroll
    for (int t = 0; t < kPieces; ++t) {
      const int m = m0 + kRows * t + lane / kLanes;
      v[t] = *(const u32x4*)(add + (int64_t)(m < rows ? m : rows - 1) * ld + (c < cols ? c : 0));
    }
  }
};

// A tile of 256 bf16 columns from the accumulators (+ add).  What is added is
// read along whole rows, so the sums go through LDS in fp32, 32 rows at a time,
// to meet it and to be stored as whole rows; each 32 rows' loads are issued
// before the 32 rows in front are finished.  (Read at the accumulators' places, 8
// bytes a lane and row, it cost 150 us of 32768 tokens' 990.  Without anything
// added too: all of a wave's rows staged in bf16 before the first is stored took
// 2271 us for the whole forward there, this 2226 us.)
template <class G, int MI>
__device__ __forceinline__ void store_rows(const Ring& smem, const f32x16 (&acc)[MI][G::NJ],
                                           const Waves<G, MI>& wv, const uint16_t* add,
                                           uint16_t* out, int64_t ld, int rows, int cols) {
  constexpr int NJ = G::NJ;
  typedef __attribute__((address_space(3))) float lds_f;
  typedef Added<NJ> Ad;
  constexpr int kRow = 32 * NJ + 4;               // floats: 32 rows' pieces on distinct banks
  lds_f* reg = (lds_f*)(smem.base + wv.w * (32 * kRow * 4));
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5, c0 = wv.nrow[0];
  const Rsrc to = make_rsrc(out, (int64_t)rows * ld * 2);
  Ad next;
  next.load(add, ld, wv.m0, rows, c0, cols);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    MOONEP_PIN();                 // else every block's loads move up here, and their registers spill
    const Ad now = next;
    if (i + 1 < MI) next.load(add, ld, wv.m0 + 32 * (i + 1), rows, c0, cols);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(__attribute__((address_space(3))) f32x4*)(reg + lr * kRow + 32 * j + acc_col(q, lh)) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                  acc[i][j][4 * q + 3]};
    const int c = 8 * (lane % Ad::kLanes);
#pragma unroll
    for (int p = 0; p < Ad::kPieces; ++p) {
      const int r = Ad::kRows * p + lane / Ad::kLanes;
      const lds_f* from = reg + r * kRow + c;
      const f32x4 s0 = *(const __attribute__((address_space(3))) f32x4*)from;
      const f32x4 s1 = *(const __attribute__((address_space(3))) f32x4*)(from + 4);
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = e < 2 ? s0[2 * (e & 1)] : s1[2 * (e & 1)];
        const float hi = e < 2 ? s0[2 * (e & 1) + 1] : s1[2 * (e & 1) + 1];
        o[e] = pack_bf16x2(lo + bf16_of(now.v[p][e], 0), hi + bf16_of(now.v[p][e], 1));
      }
      const int m = wv.m0 + 32 * i + r;
      const uint32_t off = c0 + c < cols ? (uint32_t)(((int64_t)m * ld + c0 + c) * 2) : kOob;
      __builtin_amdgcn_raw_buffer_store_b128(o, to, off, 0, 0);
    }
  }
}

// Y: 256 columns, K = H'.
template <class G, int MI, bool PART>
__device__ __forceinline__ void large_down_tile(const LargeArgs& a, const Ring& smem,
                                                const LargeTile& t) {
  constexpr int NJ = G::NJ;
  const Waves<G, MI> wv;
  const int n0 = t.nt * BN, cols = a.H - n0 < BN ? a.H - n0 : BN;
  const Steps k = steps_of<PART>(a, t, a.Hp / BK);
  const int64_t k0 = (int64_t)k.j0 * BK, at = (int64_t)t.m0 * a.H + n0;
  typename G::template Tiles<MI>::A la;
  typename G::template Tiles<MI>::B lb;
  la.init(a.z + (int64_t)t.m0 * a.Hp + k0, a.Hp, t.rows);
  lb.init(a.w[2] + (int64_t)n0 * a.Hp + k0, a.Hp, cols);
  f32x16 acc[MI][NJ];
  product<G, MI>(la, lb, smem, k.n, acc, wv.m0, wv.nrow);
  if constexpr (PART) {
    int64_t col[NJ];
    int left[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      col[j] = n0 + wv.nrow[j];
      left[j] = cols - wv.nrow[j];
    }
    store_f32<G, MI>(acc, wv, a.part + ((int64_t)t.sp * a.T + t.m0) * a.H, a.H, t.rows, col, left);
    return;
  }
  store_rows<G, MI>(smem, acc, wv, a.add ? a.add + at : nullptr, a.y + at, a.H, t.rows, cols);
}

// dZ in fp32: 256 columns of H', K = H.
template <class G, int MI, bool PART>
__device__ __forceinline__ void large_dz_tile(const LargeArgs& a, const Ring& smem,
                                              const LargeTile& t) {
  static_assert(!PART, "K is not cut");
  const Waves<G, MI> at;
  const int n0 = t.nt * BN, cols = a.Hp - n0 < BN ? a.Hp - n0 : BN;
  const int nv0 = cols < 128 ? cols : 128;
  typename G::template Tiles<MI>::A la;
  typename G::template Tiles<MI>::Col lb;
  la.init(a.dy + (int64_t)t.m0 * a.H, a.H, t.rows);
  lb.init(a.w[2] + n0, a.w[2] + n0 + 128, a.Hp, a.H, nv0, cols - nv0);
  f32x16 acc[MI][G::NJ];
  product<G, MI>(la, lb, smem, a.H / BK, acc, at.m0, at.nrow);
  int64_t col[G::NJ];
  int left[G::NJ];
#pragma unroll
  for (int j = 0; j < G::NJ; ++j) {
    col[j] = n0 + at.nrow[j];
    left[j] = cols - at.nrow[j];
  }
  store_f32<G, MI>(acc, at, a.dz + (int64_t)t.m0 * a.Hp, a.Hp, t.rows, col, left);
}

// dG, dU and Z from the gate/up product and dZ.
template <class G, int MI, bool PART>
__device__ __forceinline__ void large_gu_tile(const LargeArgs& a, const Ring& smem,
                                              const LargeTile& t) {
  static_assert(!PART, "K is not cut");
  typedef Waves<G, MI> Wv;
  constexpr int kHalf = Wv::kHalf;
  const Wv wv;
  const int n0 = t.nt * 128, nv = a.Hp - n0 < 128 ? a.Hp - n0 : 128;
  f32x16 acc[MI][G::NJ];
  gateup_product<G, MI, false>(a, smem, t, acc, wv);
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  typedef Stage<32 * MI, 32 * kHalf> St;
  lds_t* reg_g = smem.base + wv.w * (2 * St::kBytes);
  lds_t* reg_u = reg_g + St::kBytes;
  const int64_t at = (int64_t)t.m0 * a.Hp + n0, range = (int64_t)t.rows * a.Hp * 2;
  // Z is kept in the accumulators of U until dG and dU are stored (all three stored 32 rows at a
  // time: 24948 tokens of 256 x 2368 457 -> 479 us)
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    MOONEP_PIN();
    f32x4 dzv[kHalf][4];
#pragma unroll
    for (int j = 0; j < kHalf; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // places past the edge read one inside it, as in Added
        const int m = wv.m0 + i * 32 + lr, n = wv.pair[j] + acc_col(q, lh);
        dzv[j][q] = *(const f32x4*)(a.dz + at + (int64_t)(m < t.rows ? m : t.rows - 1) * a.Hp +
                                    (n < nv ? n : 0));
      }
#pragma unroll
    for (int j = 0; j < kHalf; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float dg[4], du[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = acc[i][j + kHalf][4 * q + e], d = dzv[j][q][e];
          const Act f = activate(a.act, acc[i][j][4 * q + e]);
          du[e] = d * f.f;
          dg[e] = d * u * f.df;
          acc[i][j + kHalf][4 * q + e] = f.f * u;
        }
        St::put(reg_g, i, j, q, pack_bf16x2(dg[0], dg[1]), pack_bf16x2(dg[2], dg[3]));
        St::put(reg_u, i, j, q, pack_bf16x2(du[0], du[1]), pack_bf16x2(du[2], du[3]));
      }
  }
  St::flush(reg_g, make_rsrc(a.dg + at, range), wv.m0, a.Hp, wv.pair[0], nv);
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < kHalf; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        St::put(reg_g, i, j, q,
                pack_bf16x2(acc[i][j + kHalf][4 * q], acc[i][j + kHalf][4 * q + 1]),
                pack_bf16x2(acc[i][j + kHalf][4 * q + 2], acc[i][j + kHalf][4 * q + 3]));
  St::flush(reg_u, make_rsrc(a.du + at, range), wv.m0, a.Hp, wv.pair[0], nv);
  St::flush(reg_g, make_rsrc(a.z + at, range), wv.m0, a.Hp, wv.pair[0], nv);
}

// A tile whose K range starts at k0 of another's (for splits of two matrices one after the other,
// whose base cannot be moved).
template <class T>
struct From {
  static constexpr bool kRows = T::kRows;
  static constexpr int kLoads = T::kLoads;
  T t;
  int64_t k0;
  __device__ __forceinline__ uint32_t koff(int64_t k) const { return t.koff(k0 + k); }
  __device__ __forceinline__ void issue1(lds_t* tile, int i, uint32_t ko) const {
    t.issue1(tile, i, ko);
  }
  __device__ __forceinline__ void issue(lds_t* tile, int64_t k, bool valid) const {
    t.issue(tile, k0 + k, valid);
  }
  __device__ __forceinline__ static bf16x8 frag(const lds_t* tile, int row, int kk, int lh) {
    return T::frag(tile, row, kk, lh);
  }
};

// dX: 256 columns of H, K = 2 H' over [dG | dU] and [Wg | Wu].
template <class G, int MI, bool PART>
__device__ __forceinline__ void large_dx_tile(const LargeArgs& a, const Ring& smem,
                                              const LargeTile& t) {
  const Waves<G, MI> at;
  const int n0 = t.nt * BN, cols = a.H - n0 < BN ? a.H - n0 : BN;
  const int64_t ab = (int64_t)t.m0 * a.Hp, bb = (int64_t)n0 * a.Hp;
  f32x16 acc[MI][G::NJ];
  if constexpr (PART) {
    const Steps k = steps_of<PART>(a, t, 2 * a.Hp / BK);
    From<typename G::template Tiles<MI>::A2> la;
    From<typename G::template Tiles<MI>::B2> lb;
    la.k0 = lb.k0 = (int64_t)k.j0 * BK;
    la.t.init(a.dg + ab, a.du + ab, a.Hp, t.rows, a.Hp);
    lb.t.init(a.w[0] + bb, a.w[1] + bb, a.Hp, cols, a.Hp);
    product<G, MI>(la, lb, smem, k.n, acc, at.m0, at.nrow);
    int64_t col[G::NJ];
    int left[G::NJ];
#pragma unroll
    for (int j = 0; j < G::NJ; ++j) {
      col[j] = n0 + at.nrow[j];
      left[j] = cols - at.nrow[j];
    }
    store_f32<G, MI>(acc, at, a.part + ((int64_t)t.sp * a.T + t.m0) * a.H, a.H, t.rows, col, left);
    return;
  }
  typename G::template Tiles<MI>::A2 la;
  typename G::template Tiles<MI>::B2 lb;
  la.init(a.dg + ab, a.du + ab, a.Hp, t.rows, a.Hp);
  lb.init(a.w[0] + bb, a.w[1] + bb, a.Hp, cols, a.Hp);
  product<G, MI>(la, lb, smem, 2 * a.Hp / BK, acc, at.m0, at.nrow);
  store_rows<G, MI>(smem, acc, at, nullptr, a.dx + (int64_t)t.m0 * a.H + n0, a.H, t.rows, cols);
}

// G, U and dZ of a middling number of tokens in one launch, in splits: tiles of
// gate and up columns, then tiles of 256 columns of dZ, as two regions of 128
// like the others.
template <class G, int MI, bool PART>
__device__ __forceinline__ void large_grad_tile(const LargeArgs& a, const Ring& smem,
                                                const LargeTile& t) {
  static_assert(PART, "K is always cut");
  const Waves<G, MI> wv;
  const int gu = (a.Hp + 127) / 128;
  const bool dz = t.nt >= gu;
  const int n0 = dz ? (t.nt - gu) * 256 : t.nt * 128, rest = a.Hp - n0;
  const int nv0 = rest < 128 ? rest : 128;
  const int nv1 = !dz ? nv0 : rest < 256 ? rest - nv0 : 128;
  const Steps k = steps_of<PART>(a, t, a.H / BK);
  const int64_t k0 = (int64_t)k.j0 * BK, at = k0 * a.Hp + n0;
  typename G::template Tiles<MI>::A la;
  typename G::template Tiles<MI>::Col lb;
  la.init((dz ? a.dy : a.x) + (int64_t)t.m0 * a.H + k0, a.H, t.rows);
  lb.init(a.w[dz ? 2 : 0] + at, dz ? a.w[2] + at + 128 : a.w[1] + at, a.Hp, a.H - k0, nv0, nv1);
  f32x16 acc[MI][G::NJ];
  product<G, MI>(la, lb, smem, k.n, acc, wv.m0, wv.pair);
  int64_t col[G::NJ];
  int left[G::NJ];
#pragma unroll
  for (int j = 0; j < G::NJ; ++j) {
    const int region = wv.pair[j] >> 7, c = wv.pair[j] & 127;
    col[j] = (dz ? 2LL * a.Hp + region * 128 : region * (int64_t)a.Hp) + n0 + c;
    left[j] = (region ? nv1 : nv0) - c;
  }
  store_f32<G, MI>(acc, wv, a.part + ((int64_t)t.sp * a.T + t.m0) * 3 * a.Hp, 3LL * a.Hp, t.rows,
                   col, left);
}

MOONEP_LARGE(large_gateup, large_gateup_tile)
MOONEP_LARGE_128(large_gateup_splits, large_gateup_tile, true)
MOONEP_LARGE(large_down, large_down_tile)
MOONEP_LARGE_128(large_down_splits, large_down_tile, true)
MOONEP_LARGE(large_dz, large_dz_tile)
MOONEP_LARGE(large_gu, large_gu_tile)
MOONEP_LARGE(large_dx, large_dx_tile)
MOONEP_LARGE_128(large_dx_splits, large_dx_tile, true)
MOONEP_LARGE_128(large_grad_splits, large_grad_tile, true)

// dW of the three projections, the sum over the tokens: tiles of 256 columns of
// H' and 256 rows of H by four waves, or 128 by eight.
typedef ColTileT<128, 8> ColTileA8;    // one region loaded by eight waves

// F32: added to fp32 (both ends in one kernel would keep the sums twice, and spill).
template <class G, int MI, bool PART, bool F32>
__device__ __forceinline__ void wgrad_tile(const LargeArgs& a, const Ring& smem, unsigned block) {
  constexpr int kM = G::kWaves == 4 ? 256 : 128, NJ = G::NJ;
  const int64_t each = (int64_t)a.ntm * a.ntn, total = 3 * each * a.S;
  const int64_t per = (total + kXcds - 1) / kXcds;
  int64_t l = (int64_t)(block % kXcds) * per + block / kXcds;
  if (block / kXcds >= per || l >= total) return;
  LargeTile t;
  t.sp = (int)(l / (3 * each));
  l -= t.sp * 3 * each;
  const int p = (int)(l / each), rem = (int)(l % each);
  const int m0 = rem / a.ntn * kM, n0 = rem % a.ntn * BN;
  const int mv = a.H - m0 < kM ? a.H - m0 : kM, nv = a.Hp - n0 < BN ? a.Hp - n0 : BN;
  const int nv0 = nv < 128 ? nv : 128;
  const Steps k = steps_of<PART>(a, t, (a.T + BK - 1) / BK);
  const int64_t k0 = (int64_t)k.j0 * BK;
  const uint16_t* A = (p == 2 ? a.dy : a.x) + k0 * a.H + m0;
  const uint16_t* Bm = (p == 0 ? a.dg : p == 1 ? a.du : a.z) + k0 * a.Hp + n0;
  const Waves<G, MI> wv;
  typename G::template Tiles<MI>::Col lb;
  lb.init(Bm, Bm + 128, a.Hp, a.T - k0, nv0, nv - nv0);
  f32x16 acc[MI][NJ];
  if constexpr (G::kWaves == 4) {
    const int mv0 = mv < 128 ? mv : 128;
    ColTile la;
    la.init(A, A + 128, a.H, a.T - k0, mv0, mv - mv0);
    product<G, MI>(la, lb, smem, k.n, acc, wv.m0, wv.nrow);
  } else {
    ColTileA8 la;
    la.init(A, a.H, a.T - k0, mv);
    product<G, MI>(la, lb, smem, k.n, acc, wv.m0, wv.nrow);
  }
  const int64_t at = (int64_t)m0 * a.Hp + n0;
  if constexpr (PART) {
    int64_t col[NJ];
    int left[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      col[j] = wv.nrow[j];
      left[j] = nv - wv.nrow[j];
    }
    float* out = a.part + ((int64_t)t.sp * 3 + p) * a.H * a.Hp + at;
    store_f32<G, MI>(acc, wv, out, a.Hp, mv, col, left);
    return;
  }
  void* out = p == 0 ? a.dw[0] : p == 1 ? a.dw[1] : a.dw[2];
  if constexpr (!F32) {
    store_rows<G, MI>(smem, acc, wv, nullptr, (uint16_t*)out + at, a.Hp, mv, nv);
    return;
  }
  // read-modify-write, the reads of a block row before its writes
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = wv.m0 + i * 32 + lr;
    float* row = (float*)out + at + (int64_t)m * a.Hp;
    f32x4 v[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = wv.nrow[j] + acc_col(q, lh);
        if (m < mv && n < nv) v[j][q] = *(const f32x4*)(row + n);
      }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = wv.nrow[j] + acc_col(q, lh);
        if (m < mv && n < nv) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][q][e] += acc[i][j][4 * q + e];
          *(f32x4*)(row + n) = v[j][q];
        }
      }
  }
}
template <bool F32>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256),
                          amdgpu_waves_per_eu(1, 1))) void large_wgrad_256(LargeArgs a) {
  MOONEP_RING(smem);
  wgrad_tile<Four, 4, false, F32>(a, smem, blockIdx.x);
}
template <bool F32>
__global__ __attribute__((amdgpu_flat_work_group_size(512, 512),
                          amdgpu_waves_per_eu(2, 2))) void large_wgrad_128(LargeArgs a) {
  MOONEP_RING(smem);
  wgrad_tile<Eight, 2, false, F32>(a, smem, blockIdx.x);
}
__global__ __attribute__((amdgpu_flat_work_group_size(512, 512),
                          amdgpu_waves_per_eu(2, 2))) void large_wgrad_splits(LargeArgs a) {
  MOONEP_RING(smem);
  wgrad_tile<Eight, 2, true, false>(a, smem, blockIdx.x);
}

// The weight gradients and dX, which both need dG and dU and not each other, in
// one launch where their tiles are alike: dX's shorter tiles fill what the last
// round of the others leaves idle (a multiple of the XCDs, nw workgroups, is the
// weight gradients').
template <bool F32>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256),
                          amdgpu_waves_per_eu(1, 1))) void large_last_256(LargeArgs w, LargeArgs x,
                                                                          unsigned nw) {
  MOONEP_RING(smem);
  if (blockIdx.x < nw) {
    wgrad_tile<Four, 4, false, F32>(w, smem, blockIdx.x);
    return;
  }
  LargeTile t;
  if (!large_tile(x, 256, &t, blockIdx.x - nw)) return;
  if (t.rows <= kHalfTileM) large_dx_tile<Four, 2, false>(x, smem, t);
  else large_dx_tile<Four, 4, false>(x, smem, t);
}
template <bool F32>
__global__ __attribute__((amdgpu_flat_work_group_size(512, 512),
                          amdgpu_waves_per_eu(2, 2))) void large_last_128(LargeArgs w, LargeArgs x,
                                                                          unsigned nw) {
  MOONEP_RING(smem);
  LargeTile t;
  if (blockIdx.x < nw) wgrad_tile<Eight, 2, false, F32>(w, smem, blockIdx.x);
  else if (large_tile(x, 128, &t, blockIdx.x - nw)) large_dx_tile<Eight, 2, false>(x, smem, t);
}

// ------------------------------------------------------------- choice
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How one product runs: `rows` of a tile (256 and 128 with large = true), its tiles and splits.
struct Shape {
  bool large;
  int rows, ntm, ntn, S;
};

// Splits of nk steps for so many small tiles: a workgroup per CU (with deep rings), or two where
// one would leave a quarter of them idle; at least four steps each.  Twelve steps are done before
// another launch could have joined them.  (Two workgroups per CU throughout: 64 tokens of 7168 x
// 2048 39.8 us, 256 tokens 72 us; this 34.5 and 53 us: half the splits leave half the sums.)
int splits(int64_t tiles, int nk) {
  int64_t S = 256 / tiles;
  if (tiles * S < 192) S = 512 / tiles;
  if (S > nk / 4) S = nk / 4;
  return (int)(S < 1 || nk <= 12 ? 1 : S);
}

// Splits of 128-row large tiles that fill the GPU with at least 16 steps each, or 0.
int large_splits(int64_t tiles, int nk) {
  if (tiles < 1 || tiles > 256) return 0;
  const int64_t S = 256 / tiles;
  return tiles * S >= 192 && nk / S >= 16 ? (int)S : 0;
}

// Microseconds of so many large tiles, a round of one per CU after the other: about what the two
// kinds took for 20000 tokens of H or H' 64 to 2560 and 2560, and for 32768 of 7168 x 2048.  A
// 128-row tile's start and end cost less, and its rounds are finer; many steps favour 256 rows.
double cost256(int64_t tiles, int nk) { return ceil_div(tiles, 256) * (12.0 + 1.45 * nk); }
double cost128(int64_t tiles, int nk) { return ceil_div(tiles, 256) * (5.0 + 0.85 * nk); }

// A product of M rows in tiles of so many columns, K in nk steps of 64.  `half`: 128-row large
// tiles may be cut into splits.
Shape pick(int64_t M, int64_t cols_small, int64_t cols_large, int nk, bool half) {
  Shape s;
  s.S = 1;
  // large tiles where they fill the GPU (one workgroup per CU)
  const int64_t n256 = ceil_div(M, 256) * cols_large, n128 = ceil_div(M, 128) * cols_large;
  const int S = half && n128 < 192 ? large_splits(n128, nk) : 0;
  s.large = n128 >= 192 || S > 0;
  if (s.large) {
    s.rows = S == 0 && cost256(n256, nk) < cost128(n128, nk) ? 256 : 128;
    s.ntn = (int)cols_large;
    if (S > 0) s.S = S;
  } else {
    s.rows = M <= 32 ? 32 : M <= 64 ? 64 : 128;
    s.ntn = (int)cols_small;
  }
  s.ntm = (int)ceil_div(M, s.rows);
  if (!s.large) s.S = splits((int64_t)s.ntm * s.ntn, nk);
  return s;
}
Shape gateup_shape(int64_t T, int H, int Hp) {
  return pick(T, Hp / 64, ceil_div(Hp, 128), H / BK, true);
}
Shape down_shape(int64_t T, int H, int Hp) {
  return pick(T, ceil_div(H, 128), ceil_div(H, 256), Hp / BK, true);
}
Shape dx_shape(int64_t T, int H, int Hp) {
  return pick(T, ceil_div(H, 128), ceil_div(H, 256), 2 * Hp / BK, true);
}
// dG, dU, Z: tiles of gate and up; small ones, and 128-row large ones in splits (`parts`), with
// those of dZ in the same launch.
struct GradShape {
  Shape s;
  bool parts;
};
GradShape grad_shape(int64_t T, int H, int Hp) {
  GradShape g;
  const int64_t gu = ceil_div(Hp, 128), all = gu + ceil_div(Hp, 256), m = ceil_div(T, 128);
  const int S = m * gu < 192 ? large_splits(m * all, H / BK) : 0;
  g.s = pick(T, Hp / 64 + gu, gu, H / BK, false);
  g.parts = S > 0 || !g.s.large;
  if (S > 0) g.s = {true, 128, (int)m, (int)all, S};
  return g;
}
Shape wgrad_shape(int64_t T, int H, int Hp) {
  const int nk = (int)ceil_div(T, BK);
  const int cols = (int)ceil_div(Hp, 256), m256 = (int)ceil_div(H, 256), m128 = (int)ceil_div(H, 128);
  const int64_t n256 = 3LL * m256 * cols, n128 = 3LL * m128 * cols;
  const int S = n128 < 192 ? large_splits(n128, nk) : 1;
  if (S > 0) {
    // near a tie the larger tiles' whole rows store faster (512 tokens of 7168 x 2048: the whole
    // backward 179 us, with 128-row ones 185 us)
    if (S == 1 && cost256(n256, nk) < 1.05 * cost128(n128, nk)) return {true, 256, m256, cols, 1};
    return {true, 128, m128, cols, S};
  }
  Shape s = {false, 128, m128, 3 * (int)ceil_div(Hp, 128), 1};
  s.S = splits((int64_t)s.ntm * s.ntn, nk);
  return s;
}

// Whether few_rows takes the down product: with 32 rows of Wd a workgroup either fills the CUs or is
// done in 16 steps.
bool few(int64_t T, int H, int Hp) { return T <= 32 && (H / 32 >= 128 || Hp <= 4096); }

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

// Workspace: what lies where, in bytes.
struct FwdWs {
  int64_t z, part, total;
};
FwdWs fwd_ws(int64_t T, int H, int Hp) {
  FwdWs w;
  w.z = 0;
  w.part = round256(T * Hp * 2);
  const Shape g = gateup_shape(T, H, Hp), d = down_shape(T, H, Hp);
  int64_t p = 0;
  if (g.S > 1) p = (int64_t)g.S * T * 2 * Hp * 4;
  if (d.S > 1 && !few(T, H, Hp) && (int64_t)d.S * T * H * 4 > p) p = (int64_t)d.S * T * H * 4;
  w.total = w.part + round256(p);
  return w;
}
struct BwdWs {
  int64_t z, dg, du, dz, part, total;
};
BwdWs bwd_ws(int64_t T, int H, int Hp) {
  BwdWs w;
  const int64_t one = round256(T * Hp * 2);
  w.z = 0;
  w.dg = one;
  w.du = 2 * one;
  w.dz = w.part = 3 * one;
  const GradShape g = grad_shape(T, H, Hp);
  const Shape x = dx_shape(T, H, Hp), d = wgrad_shape(T, H, Hp);
  int64_t p = g.parts ? (int64_t)g.s.S * T * 3 * Hp * 4 : T * Hp * 4;
  if (x.S > 1 && (int64_t)x.S * T * H * 4 > p) p = (int64_t)x.S * T * H * 4;
  if (d.S > 1 && (int64_t)d.S * 3 * H * Hp * 4 > p) p = (int64_t)d.S * 3 * H * Hp * 4;
  w.total = w.part + round256(p);
  return w;
}

unsigned blocks_of(const Shape& s) {
  return (unsigned)(ceil_div((int64_t)s.ntm * s.ntn * s.S, kXcds) * kXcds);
}
unsigned joins(int64_t n) { return (unsigned)ceil_div(n, 4 * kJoin); }

SmallArgs with_shape(SmallArgs a, const Shape& s) {
  a.ntm = s.ntm;
  a.ntn = s.ntn;
  a.S = s.S;
  return a;
}

// One workgroup per CU at most: deep rings.
bool deep(const Shape& s) { return (int64_t)s.ntm * s.ntn * s.S <= 256; }

// Whether dX and the weight gradients, asked for together, are one launch, and whether its small
// tiles' rings are deep: by the workgroups of both.
bool joined(const Shape& x, const Shape& w) {
  return x.S == 1 && w.S == 1 && x.large == w.large && (!x.large || x.rows == w.rows);
}
bool joined_deep(const Shape& x, const Shape& w) { return blocks_of(x) + blocks_of(w) <= 256; }

int32_t tile_of(const Shape& s, bool deep_rings) {
  if (s.large) return s.rows == 256 ? MOONEP_FFN_TILE_256X256 : MOONEP_FFN_TILE_128X256;
  const int32_t t = s.rows == 32 ? MOONEP_FFN_TILE_32 : s.rows == 64 ? MOONEP_FFN_TILE_64
                                                                     : MOONEP_FFN_TILE_128;
  return t + (deep_rings ? MOONEP_FFN_TILE_DEEP : 0);
}

template <int OP, int BM, bool PART>
void run_small_as(const Shape& s, const SmallArgs& a, hipStream_t st) {
  if (deep(s)) small_kernel<OP, BM, PART, true><<<blocks_of(s), kThreads, 0, st>>>(a);
  else small_kernel<OP, BM, PART, false><<<blocks_of(s), kThreads, 0, st>>>(a);
}
template <int OP>
void run_small(const Shape& s, bool part, const SmallArgs& in, hipStream_t st) {
  const SmallArgs a = with_shape(in, s);
  constexpr bool kPart = OP == OP_GRAD;            // always in parts
  if constexpr (OP == OP_WGRAD) {
    if (part) run_small_as<OP, 128, true>(s, a, st);
    else run_small_as<OP, 128, false>(s, a, st);
  } else if (s.rows == 128) {
    if (part || kPart) run_small_as<OP, 128, true>(s, a, st);
    else run_small_as<OP, 128, kPart>(s, a, st);
  } else if (s.rows == 64) {
    if (part || kPart) run_small_as<OP, 64, true>(s, a, st);
    else run_small_as<OP, 64, kPart>(s, a, st);
  } else if constexpr (OP == OP_ROWS) {            // what few() leaves: long sums, few columns
    small_kernel<OP, 32, true, true><<<blocks_of(s), kThreads, 0, st>>>(a);
  } else {
    if (part || kPart) run_small_as<OP, 32, true>(s, a, st);
    else run_small_as<OP, 32, kPart>(s, a, st);
  }
}

template <int BM>
void run_last(const Shape& xs, const Shape& ws, const SmallArgs& x, const SmallArgs& w,
              hipStream_t st) {
  const unsigned nx = blocks_of(xs), n = nx + blocks_of(ws);
  if (joined_deep(xs, ws)) small_last<BM, true><<<n, kThreads, 0, st>>>(x, w, nx);
  else small_last<BM, false><<<n, kThreads, 0, st>>>(x, w, nx);
}

LargeArgs with_shape(LargeArgs a, const Shape& s) {
  a.ntm = s.ntm;
  a.ntn = s.ntn;
  a.S = s.S;
  return a;
}
#define MOONEP_RUN_LARGE(kernel, shape, args)                                              \
  do {                                                                                     \
    const LargeArgs la_ = with_shape(args, shape);                                         \
    if ((shape).rows == 256) kernel##_256<<<blocks_of(shape), 256, 0, s>>>(la_);           \
    else kernel##_128<<<blocks_of(shape), 512, 0, s>>>(la_);                               \
  } while (0)
// the same, or splits of 128-row tiles
#define MOONEP_RUN_LARGE_SPLITS(kernel, shape, args)                                       \
  do {                                                                                     \
    if ((shape).S == 1) MOONEP_RUN_LARGE(kernel, shape, args);                             \
    else kernel##_splits<<<blocks_of(shape), 512, 0, s>>>(with_shape(args, shape));        \
  } while (0)

}  // namespace

bool shared_ffn_shape_ok(int64_t T, int32_t H, int32_t Hp) {
  return T >= 0 && T < (int64_t(1) << 31) && H >= 64 && H % 64 == 0 && H <= 65536 && Hp >= 64 &&
         Hp % 64 == 0 && Hp <= 65536 && (int64_t)H * Hp < (int64_t(1) << 30);
}
bool shared_ffn_bwd_shape_ok(int64_t T, int32_t H, int32_t Hp) {
  return shared_ffn_shape_ok(T, H, Hp) && T * (H > Hp ? H : Hp) < (int64_t(1) << 30);
}
int64_t shared_ffn_ws_bytes(int64_t T, int32_t H, int32_t Hp) {
  return T == 0 ? 0 : fwd_ws(T, H, Hp).total;
}
int64_t shared_ffn_bwd_ws_bytes(int64_t T, int32_t H, int32_t Hp) {
  return T == 0 ? 0 : bwd_ws(T, H, Hp).total;
}

int32_t shared_ffn_tile(int64_t T, int32_t H, int32_t Hp, int32_t product, int32_t* splits) {
  Shape s;
  switch (product) {
    case MOONEP_FFN_GATEUP: s = gateup_shape(T, H, Hp); break;
    case MOONEP_FFN_DOWN: s = down_shape(T, H, Hp); break;
    case MOONEP_FFN_GRAD: s = grad_shape(T, H, Hp).s; break;
    case MOONEP_FFN_DX: s = dx_shape(T, H, Hp); break;
    case MOONEP_FFN_WGRAD: s = wgrad_shape(T, H, Hp); break;
    default: return -1;
  }
  *splits = s.S;
  if (product == MOONEP_FFN_DOWN && few(T, H, Hp)) {
    *splits = 1;
    return MOONEP_FFN_TILE_FEW;
  }
  return tile_of(s, deep(s));
}

int32_t shared_ffn_last_tile(int64_t T, int32_t H, int32_t Hp) {
  const Shape x = dx_shape(T, H, Hp), w = wgrad_shape(T, H, Hp);
  return joined(x, w) ? tile_of(x, joined_deep(x, w)) : -1;
}

hipError_t launch_shared_ffn(const uint16_t* x, const uint16_t* const w[3], int32_t act,
                             const uint16_t* add, int64_t T, int32_t H, int32_t Hp, uint16_t* y,
                             char* ws, hipStream_t s) {
  const FwdWs at = fwd_ws(T, H, Hp);
  const Shape g = gateup_shape(T, H, Hp), d = down_shape(T, H, Hp);
  uint16_t* z = (uint16_t*)(ws + at.z);
  float* part = (float*)(ws + at.part);
  LargeArgs big = {};
  big.x = x; big.add = add; big.z = z; big.y = y;
  for (int i = 0; i < 3; ++i) big.w[i] = w[i];
  big.part = part; big.T = (int)T; big.H = H; big.Hp = Hp; big.act = act;
  if (g.large) {
    MOONEP_RUN_LARGE_SPLITS(large_gateup, g, big);
  } else {
    SmallArgs a = {};
    a.a[0] = x; a.b[0] = w[0]; a.b[1] = w[1]; a.out[0] = z;
    a.part = part; a.M = (int)T; a.N = Hp; a.K = H; a.act = act;
    run_small<OP_GATEUP>(g, g.S > 1, a, s);
  }
  if (g.S > 1)
    join_gate<false><<<joins(T * Hp), kJoin, 0, s>>>(part, g.S, (int)T, Hp, act, z, nullptr,
                                                     nullptr);
  if (few(T, H, Hp)) {
    SmallArgs a = {};
    a.a[0] = z; a.b[0] = w[2]; a.out[0] = y; a.add = add;
    a.M = (int)T; a.N = H; a.K = Hp;
    few_rows<<<H / 32, kThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  if (d.large) {
    MOONEP_RUN_LARGE_SPLITS(large_down, d, big);
  } else {
    SmallArgs a = {};
    a.a[0] = z; a.b[0] = w[2]; a.out[0] = y; a.add = add;
    a.part = part; a.M = (int)T; a.N = H; a.K = Hp;
    run_small<OP_ROWS>(d, d.S > 1, a, s);
  }
  if (d.S > 1) join_rows<<<joins(T * H), kJoin, 0, s>>>(part, d.S, T * H, add, y);
  return hipGetLastError();
}

hipError_t launch_shared_ffn_bwd(const uint16_t* x, const uint16_t* dy,
                                 const uint16_t* const w[3], int32_t act, int64_t T, int32_t H,
                                 int32_t Hp, uint16_t* dx, void* const dw[3], int32_t dw_type,
                                 char* ws, hipStream_t s) {
  if (T == 0) {                  // sums over no tokens
    if (dw) {
      SmallArgs a = {};
      for (int i = 0; i < 3; ++i) a.out[i] = dw[i];
      a.M = H; a.N = Hp; a.f32 = dw_type == MOONEP_F32;
      const Shape z = {false, 128, (int)ceil_div(H, 128), 3 * (int)ceil_div(Hp, 128), 1};
      run_small<OP_WGRAD>(z, false, a, s);
    }
    return hipGetLastError();
  }
  const BwdWs at = bwd_ws(T, H, Hp);
  const GradShape g = grad_shape(T, H, Hp);
  const Shape dxs = dx_shape(T, H, Hp), ws_ = wgrad_shape(T, H, Hp);
  LargeArgs big = {};
  big.x = x; big.dy = dy; big.dx = dx;
  big.z = (uint16_t*)(ws + at.z); big.dg = (uint16_t*)(ws + at.dg); big.du = (uint16_t*)(ws + at.du);
  big.dz = (float*)(ws + at.dz);
  for (int i = 0; i < 3; ++i) {
    big.w[i] = w[i];
    big.dw[i] = dw ? dw[i] : nullptr;
  }
  big.T = (int)T; big.H = H; big.Hp = Hp; big.act = act; big.f32 = dw_type == MOONEP_F32;
  float* part = (float*)(ws + at.part);
  big.part = part;
  if (!g.parts) {
    Shape z = g.s;
    z.ntn = (int)ceil_div(Hp, BN);
    MOONEP_RUN_LARGE(large_dz, z, big);
    MOONEP_RUN_LARGE(large_gu, g.s, big);
  } else if (g.s.large) {
    large_grad_splits<<<blocks_of(g.s), 512, 0, s>>>(with_shape(big, g.s));
  } else {
    SmallArgs a = {};
    a.a[0] = x; a.a[2] = dy; a.b[0] = w[0]; a.b[1] = w[1]; a.b[2] = w[2];
    a.part = part; a.M = (int)T; a.N = Hp; a.K = H; a.act = act;
    run_small<OP_GRAD>(g.s, true, a, s);
  }
  if (g.parts)
    join_gate<true><<<joins(T * Hp), kJoin, 0, s>>>(part, g.s.S, (int)T, Hp, act, big.z, big.dg,
                                                    big.du);
  SmallArgs xa = {}, wa = {};
  xa.a[0] = big.dg; xa.a[1] = big.du; xa.b[0] = w[0]; xa.b[1] = w[1]; xa.out[0] = dx;
  xa.part = part; xa.M = (int)T; xa.N = H; xa.K = 2 * Hp;
  wa.a[0] = wa.a[1] = x; wa.a[2] = dy;
  wa.b[0] = big.dg; wa.b[1] = big.du; wa.b[2] = big.z;
  wa.part = part; wa.M = H; wa.N = Hp; wa.K = (int)T; wa.f32 = big.f32;
  JoinW j;
  for (int i = 0; i < 3; ++i) wa.out[i] = j.out[i] = big.dw[i];
  const bool one = dx && dw && joined(dxs, ws_);
  if (one && !dxs.large) {
    const SmallArgs ax = with_shape(xa, dxs), aw = with_shape(wa, ws_);
    if (dxs.rows == 128) run_last<128>(dxs, ws_, ax, aw, s);
    else if (dxs.rows == 64) run_last<64>(dxs, ws_, ax, aw, s);
    else run_last<32>(dxs, ws_, ax, aw, s);
    return hipGetLastError();
  }
  if (one) {
    const LargeArgs ax = with_shape(big, dxs), aw = with_shape(big, ws_);
    const unsigned nw = (unsigned)(ceil_div(3LL * ws_.ntm * ws_.ntn, kXcds) * kXcds);
    const unsigned n = nw + blocks_of(dxs);
    if (ws_.rows == 256) (big.f32 ? large_last_256<true> : large_last_256<false>)
        <<<n, 256, 0, s>>>(aw, ax, nw);
    else (big.f32 ? large_last_128<true> : large_last_128<false>)<<<n, 512, 0, s>>>(aw, ax, nw);
    return hipGetLastError();
  }
  if (dx) {
    if (dxs.large) {
      MOONEP_RUN_LARGE_SPLITS(large_dx, dxs, big);
    } else {
      run_small<OP_ROWS2>(dxs, dxs.S > 1, xa, s);
    }
    if (dxs.S > 1) join_rows<<<joins(T * H), kJoin, 0, s>>>(part, dxs.S, T * H, nullptr, dx);
  }
  if (dw) {
    if (ws_.large) {
      const LargeArgs a = with_shape(big, ws_);
      const unsigned n = (unsigned)(ceil_div(3LL * a.ntm * a.ntn * a.S, kXcds) * kXcds);
      if (ws_.rows == 256) (big.f32 ? large_wgrad_256<true> : large_wgrad_256<false>)
          <<<n, 256, 0, s>>>(a);
      else if (ws_.S == 1) (big.f32 ? large_wgrad_128<true> : large_wgrad_128<false>)
          <<<n, 512, 0, s>>>(a);
      else large_wgrad_splits<<<n, 512, 0, s>>>(a);
    } else {
      run_small<OP_WGRAD>(ws_, ws_.S > 1, wa, s);
    }
    const int64_t n = (int64_t)H * Hp;
    if (ws_.S > 1) join_wgrad<<<dim3(joins(n), 3), kJoin, 0, s>>>(part, ws_.S, n, big.f32, j);
  }
  return hipGetLastError();
}

}  // namespace moonep
