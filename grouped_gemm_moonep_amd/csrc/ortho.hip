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
//   S = A A,  B = (b A + c S) / a                per step
//   T = A + B A,  P = P + B P                    (P = I + B in the first)
//   A = a^2 (T + B T)
//   out = (prod a) P X_0                         (last product)
// All m x m matrices are symmetric, so only the tiles on and above the
// diagonal are computed and every element above it is written twice: to the bit, for an
// antisymmetric part, however small at first, would grow to 1e-2 of the result.  Per step 3.5 m^3 ..
// 4 m^3 multiply-adds of which half are done, against (2 n/m + 1) m^3 (1.5 n/m + 0.5
// done) for the steps taken on X itself: at n = 3.5 m 26 m^3 in all against 57 m^3.
//
// Rounding: P amplifies what is lost in A by up to prod a (485 for the usual
// five steps) in the directions of small singular values, and the gradient of
// an expert with few tokens has almost only those.  bf16 (2^-9) or fp16
// (2^-12) operands would leave nothing there, so every matrix is held as a
// pair of fp16, v = hi + lo (22 bits), and a product is hi hi + hi lo + lo hi
// on the matrix units, summed in fp32: 1e-5 .. 1e-3 of the result's norm is
// left for full rank .. rank one, below the 2e-3 of rounding it to bf16.
// Values are scaled by 2^14, so entries up to 4 are held, and down to 2^-28
// with 11 or more bits.
//
// Layout: a row of k values is stored as blocks of 128 bytes, 32 hi then 32
// lo, zero behind the last value; a GEMM operand is then a 256-row tile of 128-byte
// rows, as in gemm_core.h, whose loads, swizzle and ring are used as they are.  All
// products are C = U V^T with both operands contiguous along K: the
// m x m matrices are symmetric, and X_0 is written in both orientations.
#include "gemm_core.h"

namespace moonep {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr float kScale = 16384.0f;            // stored = value * 2^14
constexpr int kParts = 256;                   // partial sums of a matrix's norm
constexpr int kK = 32;                        // values of K per step (a 64-element block)

// ------------------------------------------------------------- K loop
// One step = 32 values of K = two 16-deep halves, hi in fragment columns kk =
// 0, 1 and lo in kk = 2, 3: per half three groups of 16 MFMAs, h.a h.b, h.a l.b
// and l.a h.b.  The operand bytes of a step are those of 64 values in 16 bits
// and its MFMAs 1.5 times theirs, so the loads and LDS reads hide more easily
// than in the expert GEMMs.  The groups run B-fragment by B-fragment: in the third
// one h.b[j] is free after its four MFMAs and takes the next half's, so two
// fragment sets (64 registers) suffice.
template <int MI>
struct Frag3 {
  bf16x8 a[MI], b[4];
};

template <int MI>
__device__ __forceinline__ void mma3(f32x16 acc[MI][4], const bf16x8& a, const bf16x8& b, int i,
                                     int j) {
  acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, b),
                                                     __builtin_bit_cast(f16x8, a), acc[i][j], 0, 0,
                                                     0);
}

__device__ __forceinline__ bf16x8 read3(const lds_t* tile, int row0, int kk) {
  const int lane = threadIdx.x & 63;
  return RowTile::frag(tile, row0 + (lane & 31), kk, lane >> 5);
}

// Half HALF of step j (J = j mod 5): three groups of 4 MI MFMAs.  The loads of
// A(j+1), then of B(j+2), go out between the step's first MFMAs; when the
// first B fragment of the last group is free comes the wait for step j + 1's
// tiles and the barrier, then the reads of step j + 1's first fragments (all
// but h.b[3], which that step reads first).
template <int J, int HALF, int MI>
__device__ __forceinline__ void khalf3(const RowTileT<2 * MI>& la, const RowTile& lb,
                                       const Ring& ring, uint32_t koa, uint32_t kob, Frag3<MI>& h,
                                       Frag3<MI>& l, f32x16 acc[MI][4], int arow0,
                                       const int nrow[4]) {
  constexpr int J1 = (J + 1) % kSlots, J2 = (J + 2) % kSlots;
  constexpr int GRP = 4 * MI, N = 3 * GRP, BAR = 21 * MI - 1, B0 = 6 * MI, BS = (BAR - B0) / 8;
  static_assert(B0 >= 3 * 2 * MI && B0 + 7 * BS <= BAR, "loads must precede the barrier");
  const lds_t* A = ring.a<J>();
  const lds_t* Bt = ring.b<J>();
  const lds_t* nA = HALF ? ring.a<J1>() : A;             // the next half's hi fragments
  const lds_t* nB = HALF ? ring.b<J1>() : Bt;
  constexpr int nkk = HALF ? 0 : 1;
#pragma unroll
  for (int o = 0; o < N; ++o) {
    const int p = N * HALF + o, mi = o % MI, mj = o / MI % 4;
    if (o < GRP) mma3<MI>(acc, h.a[mi], h.b[mj], mi, mj);
    else if (o < 2 * GRP) mma3<MI>(acc, h.a[mi], l.b[mj], mi, mj);
    else mma3<MI>(acc, l.a[mi], h.b[mj], mi, mj);
    if (o == 0) h.b[3] = read3(Bt, nrow[3], HALF);
    if (o >= 1 && o < 5) l.b[o - 1] = read3(Bt, nrow[o - 1], 2 + HALF);
    if (o >= 5 && o < 5 + MI) l.a[o - 5] = read3(A, arow0 + 32 * (o - 5), 2 + HALF);
    if (p % 3 == 1 && p / 3 < 2 * MI) la.issue1(ring.a<J1>(), p / 3, koa);
    if (p >= B0 && (p - B0) % BS == 0 && (p - B0) / BS < 8)
      lb.issue1(ring.b<J2>(), (p - B0) / BS, kob);
    if (p == BAR) {
      MOONEP_PIN();
      wait_loads<kLoadsPerStep>();
      barrier_reads_done();
    }
    constexpr int F = 9 * MI;                            // h.b[0] and h.a are free
    if (o == F) h.b[0] = read3(nB, nrow[0], nkk);
    if (o > F && o <= F + MI) h.a[o - F - 1] = read3(nA, arow0 + 32 * (o - F - 1), nkk);
    if (o == F + MI + 1) h.b[1] = read3(nB, nrow[1], nkk);
    if (o == F + 2 * MI) h.b[2] = read3(nB, nrow[2], nkk);
    MOONEP_PIN();
  }
}

template <int J, int MI>
__device__ __forceinline__ void kstep3(const RowTileT<2 * MI>& la, const RowTile& lb,
                                       const Ring& ring, int j, int nk, Frag3<MI>& h, Frag3<MI>& l,
                                       f32x16 acc[MI][4], int arow0, const int nrow[4]) {
  const uint32_t koa = j + 1 < nk ? la.koff((int64_t)(j + 1) * BK) : kOob;
  const uint32_t kob = j + 2 < nk ? lb.koff((int64_t)(j + 2) * BK) : kOob;
  MOONEP_PIN();
  khalf3<J, 0, MI>(la, lb, ring, koa, kob, h, l, acc, arow0, nrow);
  khalf3<J, 1, MI>(la, lb, ring, koa, kob, h, l, acc, arow0, nrow);
}

// kTwoSums: the sum of every five steps (160 values of K) starts at zero and is added to `sum`
// after them, in place of one chain over all of K.
template <int MI, bool kTwoSums>
__device__ __forceinline__ void gemm3_loop(const RowTileT<2 * MI>& la, const RowTile& lb,
                                           const Ring& ring, int nk, f32x16 acc[MI][4], int arow0,
                                           const int nrow[4]) {
  lb.issue(ring.b<0>(), 0, true);
  la.issue(ring.a<0>(), 0, true);
  lb.issue(ring.b<1>(), BK, 1 < nk);
  f32x16 sum[kTwoSums ? MI : 1][4];
  if constexpr (kTwoSums) zero_acc<MI>(sum);
  zero_acc<MI>(acc);
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kTwoSums) asm volatile("" : "+a"(sum[i][j]));
      else asm volatile("" : "+a"(acc[i][j]));
    }
  wait_loads<kLoadsPerStep>();
  barrier_reads_done();
  Frag3<MI> h, l;
#pragma unroll
  for (int q = 0; q < 3; ++q) h.b[q] = read3(ring.b<0>(), nrow[q], 0);
#pragma unroll
  for (int q = 0; q < MI; ++q) h.a[q] = read3(ring.a<0>(), arow0 + 32 * q, 0);
  for (int j = 0; j < nk; j += kSlots) {
    kstep3<0, MI>(la, lb, ring, j, nk, h, l, acc, arow0, nrow);
    if (j + 1 < nk) kstep3<1, MI>(la, lb, ring, j + 1, nk, h, l, acc, arow0, nrow);
    if (j + 2 < nk) kstep3<2, MI>(la, lb, ring, j + 2, nk, h, l, acc, arow0, nrow);
    if (j + 3 < nk) kstep3<3, MI>(la, lb, ring, j + 3, nk, h, l, acc, arow0, nrow);
    if (j + 4 < nk) kstep3<4, MI>(la, lb, ring, j + 4, nk, h, l, acc, arow0, nrow);
    if constexpr (kTwoSums) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
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
      for (int jj = 0; jj < 4; ++jj) acc[i][jj] = sum[i][jj];
  }
  wait_loads<0>();
  __syncthreads();
}

// ---------------------------------------------------------- epilogue pieces
// A 32 x 32 block of a pair matrix is 32 rows of 128 bytes.  In LDS the
// 16-byte chunk c of row r sits at c ^ ((r >> 1) & 7), which spreads a
// column of chunks over the banks.
constexpr int kBlockBytes = 32 * 128;
__device__ __forceinline__ int blk_off(int r, int byte) {
  return r * 128 + (((byte >> 4) ^ ((r >> 1) & 7)) << 4) + (byte & 15);
}

__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
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
// the same four values as column r, rows c .. c + 3
__device__ __forceinline__ void put_col4(lds_t* blk, int r, int c, const f16x4& hi,
                                         const f16x4& lo) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    *(__attribute__((address_space(3))) _Float16*)(blk + blk_off(c + e, 2 * r)) = hi[e];
    *(__attribute__((address_space(3))) _Float16*)(blk + blk_off(c + e, 64 + 2 * r)) = lo[e];
  }
}
// the part on and above the diagonal of a diagonal block, and its mirror image
__device__ __forceinline__ void put_diag4(lds_t* blk, int r, int c, const f16x4& hi,
                                          const f16x4& lo) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (c + e < r) continue;
    *(__attribute__((address_space(3))) _Float16*)(blk + blk_off(r, 2 * (c + e))) = hi[e];
    *(__attribute__((address_space(3))) _Float16*)(blk + blk_off(r, 64 + 2 * (c + e))) = lo[e];
    *(__attribute__((address_space(3))) _Float16*)(blk + blk_off(c + e, 2 * r)) = hi[e];
    *(__attribute__((address_space(3))) _Float16*)(blk + blk_off(c + e, 64 + 2 * r)) = lo[e];
  }
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

// ------------------------------------------------------------ m x m products
// out = alpha U V^T + beta in, symmetric, for nmat matrices and one or two
// problems (operand and result sets) in one launch.
struct SymArgs {
  const uint16_t* u[2];
  const uint16_t* v[2];
  const uint16_t* in[2];     // null: no second term
  uint16_t* out[2];
  uint16_t* out_id;          // null, or where out + I goes (first problem)
  int64_t ustride;           // elements between matrices of u and v
  int64_t ostride;           // of in, out and out_id
  float alpha, beta;
  int m, uld, ld, nk;        // rows; row strides of u, v and of in, out; K steps
  int nt, tiles, nmat;       // tiles per side, upper tiles per matrix, matrices
  int64_t total;             // workgroups in use
};

__device__ __forceinline__ int64_t xcd_tile(int64_t total) {
  // XCD x takes the x-th eighth of the tiles: neighbouring tiles of a matrix share its L2
  const int64_t per = (total + kXcds - 1) / kXcds;
  const int64_t c = blockIdx.x / kXcds, t = (int64_t)(blockIdx.x % kXcds) * per + c;
  return c < per && t < total ? t : -1;
}

// MI = 4: tiles of 256 x 256; MI = 2 (the first product, with two sums): the
// upper and the lower half of such a tile are a workgroup each.
template <int MI>
__global__ __attribute__((amdgpu_flat_work_group_size(kThreads, kThreads),
                          amdgpu_waves_per_eu(1, 1))) void ortho_sym(SymArgs a) {
  MOONEP_RING(smem);
  constexpr int kRows = 64 * MI;
  const int64_t t = xcd_tile(a.total);
  if (t < 0) return;
  const int64_t mat = t / a.tiles;
  int q = (int)(t - mat * a.tiles), ti = 0;
  const int part = q % (4 / MI);
  q /= 4 / MI;
  for (; q >= a.nt - ti; ++ti) q -= a.nt - ti;
  const int tj = ti + q;
  const int pr = mat >= a.nmat ? 1 : 0;
  const int64_t mi = mat - (pr ? a.nmat : 0);
  const uint16_t* U = a.u[pr] + mi * a.ustride;
  const uint16_t* V = a.v[pr] + mi * a.ustride;
  const uint16_t* in = a.in[pr] ? a.in[pr] + mi * a.ostride : nullptr;
  uint16_t* out = a.out[pr] + mi * a.ostride;
  uint16_t* out_id = a.out_id && !pr ? a.out_id + mi * a.ostride : nullptr;
  const int m0 = ti * BM + part * kRows, n0 = tj * BN;
  if (m0 >= a.m) return;
  const int wave = wave_id(), wm = wave >> 1, wn = wave & 1;
  const int nrow[4] = {wn * 128, wn * 128 + 32, wn * 128 + 64, wn * 128 + 96};

  RowTileT<2 * MI> la;
  RowTile lb;
  la.init(U + (int64_t)m0 * a.uld, a.uld, a.m - m0 < kRows ? a.m - m0 : kRows);
  lb.init(V + (int64_t)n0 * a.uld, a.uld, a.m - n0 < BN ? a.m - n0 : BN);
  f32x16 acc[MI][4];
  gemm3_loop<MI, MI == 2>(la, lb, smem, a.nk, acc, wm * 32 * MI, nrow);

  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
  lds_t* direct = smem.base + wave * (8 * kBlockBytes);
  lds_t* mirror = direct + 4 * kBlockBytes;
  const int ncb = a.ld / 64;                                // blocks along a row
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int row0 = m0 + wm * 32 * MI + 32 * i, row = row0 + lr;
    // one row of blocks: 4 blocks of this wave; with out_id, a second round for out + I
    f16x4 ih[4][4], il[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int qd = 0; qd < 4; ++qd) {
        const int cb = (n0 + nrow[j]) / 32;
        ih[j][qd] = f16x4{0, 0, 0, 0};
        il[j][qd] = f16x4{0, 0, 0, 0};
        if (in && row < a.m && cb < ncb) {
          const uint16_t* s = in + (int64_t)row * a.ld + cb * 64 + acc_col(qd, lh);
          ih[j][qd] = *(const f16x4*)s;
          il[j][qd] = *(const f16x4*)(s + 32);
        }
      }
    MOONEP_PIN();
    const int rounds = out_id ? 2 : 1;
    for (int rd = 0; rd < rounds; ++rd) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col0 = n0 + nrow[j];
        if (col0 < row0) continue;                       // below the diagonal: its mirror is written
#pragma unroll
        for (int qd = 0; qd < 4; ++qd) {
          const int c = acc_col(qd, lh);
          f16x4 hi, lo;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = a.alpha * acc[i][j][4 * qd + e];
            v += a.beta * ((float)ih[j][qd][e] + (float)il[j][qd][e]);
            if (rd && row == col0 + c + e && row < a.m) v += kScale;
            _Float16 h, l;
            split(v, h, l);
            hi[e] = h;
            lo[e] = l;
          }
          if (col0 == row0) {
            put_diag4(direct + j * kBlockBytes, lr, c, hi, lo);
          } else {
            put_row4(direct + j * kBlockBytes, lr, c, hi, lo);
            put_col4(mirror + j * kBlockBytes, lr, c, hi, lo);
          }
        }
      }
      uint16_t* dst = rd ? out_id : out;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col0 = n0 + nrow[j];
        if (col0 < row0) continue;
        if (col0 / 32 < ncb) flush_block(direct + j * kBlockBytes, dst, a.ld, row0, a.m, col0 / 32);
        if (col0 != row0 && row0 / 32 < ncb)
          flush_block(mirror + j * kBlockBytes, dst, a.ld, col0, a.m, row0 / 32);
      }
    }
    MOONEP_PIN();
  }
}

// --------------------------------------------------------------- last product
// out = alpha U V^T as bf16 [mu][mv], dense.
struct OutArgs {
  const uint16_t* u;         // [nmat][mu][ld]
  const uint16_t* v;         // [nmat][mv][ld]
  uint16_t* out;             // [nmat][mu][mv]
  int64_t ustride, vstride;
  float alpha;
  int mu, mv, ld, nk, ntm, ntn, nmat, wide;   // wide: 16-byte stores are aligned
  int64_t total;
};

__global__ __attribute__((amdgpu_flat_work_group_size(kThreads, kThreads),
                          amdgpu_waves_per_eu(1, 1))) void ortho_out(OutArgs a) {
  MOONEP_RING(smem);
  const int64_t t = xcd_tile(a.total);
  if (t < 0) return;
  const int per = a.ntm * a.ntn;
  const int64_t mi = t / per;
  const int q = (int)(t - mi * per), tm = q / a.ntn, tn = q % a.ntn;
  const int m0 = tm * BM, n0 = tn * BN;
  const int wave = wave_id(), wm = wave >> 1, wn = wave & 1;
  const int nrow[4] = {wn * 128, wn * 128 + 32, wn * 128 + 64, wn * 128 + 96};
  const int rows_valid = a.mu - m0 < BM ? a.mu - m0 : BM;
  const int cols_valid = a.mv - n0 < BN ? a.mv - n0 : BN;

  RowTile la, lb;
  la.init(a.u + mi * a.ustride + (int64_t)m0 * a.ld, a.ld, rows_valid);
  lb.init(a.v + mi * a.vstride + (int64_t)n0 * a.ld, a.ld, cols_valid);
  f32x16 acc[4][4];
  gemm3_loop<4, false>(la, lb, smem, a.nk, acc, wm * 128, nrow);

  uint16_t* out = a.out + (mi * a.mu + m0) * (int64_t)a.mv + n0;
  if (a.wide) {
    typedef Stage<128, 128> St;
    lds_t* reg = smem.base + wave * St::kBytes;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int qd = 0; qd < 4; ++qd)
          St::put(reg, i, j, qd,
                  pack_bf16x2(a.alpha * acc[i][j][4 * qd], a.alpha * acc[i][j][4 * qd + 1]),
                  pack_bf16x2(a.alpha * acc[i][j][4 * qd + 2], a.alpha * acc[i][j][4 * qd + 3]));
    St::flush(reg, make_rsrc(out, (int64_t)rows_valid * a.mv * 2), wm * 128, a.mv, wn * 128,
              cols_valid);
    return;
  }
  const int lane = threadIdx.x & 63, lr = lane & 31, lh = lane >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int qd = 0; qd < 4; ++qd)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = wm * 128 + 32 * i + lr, c = nrow[j] + acc_col(qd, lh) + e;
          if (r < rows_valid && c < cols_valid)
            out[(int64_t)r * a.mv + c] =
                __builtin_bit_cast(uint16_t, (__bf16)(a.alpha * acc[i][j][4 * qd + e]));
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
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * kParts + blockIdx.x] = sh[0] + sh[1] + sh[2] + sh[3];
}

// X_0 in both orientations as pairs: a 64 x 64 piece of G per workgroup.
template <class T>
__global__ __launch_bounds__(kThreads) void ortho_load(const T* g, int rows, int cols, float eps,
                                                       const double* part, uint16_t* nat,
                                                       uint16_t* tr, int64_t nat_stride,
                                                       int64_t tr_stride) {
  __shared__ float tile[64][65];
  __shared__ double sh[kThreads / 64];
  const int64_t mi = blockIdx.z;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64, tid = threadIdx.x;
  double s = part[mi * kParts + tid];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((tid & 63) == 0) sh[tid >> 6] = s;
  const T* p = g + mi * rows * (int64_t)cols;
  float x[16];
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int r = r0 + (tid >> 6) + 4 * u, c = c0 + (tid & 63);
    x[u] = r < rows && c < cols ? to_f32<T>(p[(int64_t)r * cols + c]) : 0.0f;
  }
  __syncthreads();
  const double f = (double)kScale / (sqrt(sh[0] + sh[1] + sh[2] + sh[3]) + (double)eps);
#pragma unroll
  for (int u = 0; u < 16; ++u)
    tile[(tid >> 6) + 4 * u][tid & 63] = (float)((double)x[u] * f);
  __syncthreads();
  const int nld = (cols + kK - 1) / kK * 64, tld = (rows + kK - 1) / kK * 64;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int unit = tid + kThreads * (u & 1);      // 64 rows x 8 groups of 8 columns
    const int r = unit >> 3, c = (unit & 7) * 8;
    const bool t = u >= 2;                          // then the transposed copy
    const int row = (t ? c0 : r0) + r, col = (t ? r0 : c0) + c;
    const int nrows = t ? cols : rows, ld = t ? tld : nld;
    if (row >= nrows || col / 32 * 64 >= ld) continue;
    f16x8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      _Float16 h, l;
      split(t ? tile[c + e][r] : tile[r][c + e], h, l);
      hi[e] = h;
      lo[e] = l;
    }
    uint16_t* d = (t ? tr + mi * tr_stride : nat + mi * nat_stride) + (int64_t)row * ld +
                  col / 32 * 64 + (col & 31);
    *(f16x8*)d = hi;
    *(f16x8*)(d + 32) = lo;
  }
}

// --------------------------------------------------------------------- host
int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

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
  o.bytes = 2 * (o.x + o.xt + 5 * o.sq) + kParts * (int64_t)sizeof(double);
  // Matrices per launch: enough for 8 rounds of tiles on the 256 CUs (the last round is then
  // at most an eighth of the work); more would only take more memory.
  const int64_t nt = (o.m + BM - 1) / BM, tiles = nt * (nt + 1) / 2;
  const int64_t cap = (2048 + tiles - 1) / tiles;
  const int64_t groups = n < 1 ? 1 : (n + cap - 1) / cap;
  o.group = n < 1 ? 1 : (int)((n + groups - 1) / groups);
  return o;
}

template <class T>
hipError_t orthogonalize(const T* g, int n, int rows, int cols, const float* co, int steps,
                         float eps, uint16_t* out, char* ws, hipStream_t s) {
  const OrthoLayout o = ortho_layout(n, rows, cols);
  const int64_t elems = (int64_t)rows * cols;
  double* part = (double*)ws;
  uint16_t* x = (uint16_t*)(ws + (int64_t)o.group * kParts * sizeof(double));
  uint16_t* xt = x + o.group * o.x;
  uint16_t* sq[5];
  for (int i = 0; i < 5; ++i) sq[i] = xt + o.group * o.xt + i * (o.group * o.sq);
  const bool tall = rows > cols;
  constexpr int N = 16 / (int)sizeof(T);

  for (int i0 = 0; i0 < n; i0 += o.group) {
    const int nm = n - i0 < o.group ? n - i0 : o.group;
    const T* gi = g + i0 * elems;
    const bool al = (uintptr_t)gi % 16 == 0 && elems % N == 0;
    ortho_norm<T><<<dim3(kParts, nm), kThreads, 0, s>>>(gi, elems, al ? elems / N : 0, part);
    ortho_load<T><<<dim3((cols + 63) / 64, (rows + 63) / 64, nm), kThreads, 0, s>>>(
        gi, rows, cols, eps, part, tall ? xt : x, tall ? x : xt, tall ? o.xt : o.x,
        tall ? o.x : o.xt);

    SymArgs a;
    a.m = o.m;
    a.ld = o.sld;
    a.ostride = o.sq;
    a.nt = (o.m + BM - 1) / BM;
    a.tiles = a.nt * (a.nt + 1) / 2;
    a.nmat = nm;
    auto sym = [&](int problems) {
      a.total = (int64_t)problems * nm * a.tiles;
      ortho_sym<4><<<(unsigned)pad_grid(a.total), kThreads, 0, s>>>(a);
    };
    auto set = [&](int i, const uint16_t* u, const uint16_t* v, const uint16_t* in, uint16_t* to) {
      a.u[i] = u; a.v[i] = v; a.in[i] = in; a.out[i] = to;
    };
    uint16_t *A = sq[0], *B = sq[1], *Tm = sq[2], *P = sq[3], *P2 = sq[4];
    // The first product: a chain of fp32 additions over all of K would round by 2e-7 .. 7e-7
    // of the sum, which a low-rank result shows thousands of times larger.
    set(0, x, x, nullptr, A);
    set(1, nullptr, nullptr, nullptr, nullptr);
    a.out_id = nullptr;
    a.ustride = o.x; a.uld = o.xld; a.nk = o.xld / BK;
    a.alpha = 1.0f / kScale; a.beta = 0.0f;
    a.tiles = 2 * (a.nt * (a.nt + 1) / 2);
    a.total = (int64_t)nm * a.tiles;
    ortho_sym<2><<<(unsigned)pad_grid(a.total), kThreads, 0, s>>>(a);
    a.tiles /= 2;
    a.ustride = o.sq; a.uld = o.sld; a.nk = o.sld / BK;
    double gain = 1.0;
    for (int i = 0; i < steps; ++i) {
      const float ca = co[3 * i], cb = co[3 * i + 1], cc = co[3 * i + 2];
      gain *= ca;
      set(0, A, A, A, B);
      a.alpha = cc / ca / kScale; a.beta = cb / ca;
      a.out_id = i == 0 ? P : nullptr;
      sym(1);
      a.out_id = nullptr;
      a.alpha = 1.0f / kScale; a.beta = 1.0f;
      const bool more = i + 1 < steps;
      int k = 0;
      if (more) set(k++, B, A, A, Tm);
      if (i > 0) {
        set(k++, B, P, P, P2);
        uint16_t* t = P;
        P = P2;
        P2 = t;
      }
      if (k) sym(k);
      if (more) {
        set(0, B, Tm, Tm, A);
        a.alpha = ca * ca / kScale; a.beta = ca * ca;
        sym(1);
      }
    }
    OutArgs r;
    r.u = tall ? xt : P;
    r.v = tall ? P : xt;
    r.ustride = tall ? o.xt : o.sq;
    r.vstride = tall ? o.sq : o.xt;
    r.out = out + i0 * elems;
    r.alpha = (float)(gain / ((double)kScale * kScale));
    r.mu = rows; r.mv = cols; r.ld = o.sld; r.nk = o.sld / BK;
    r.ntm = (rows + BM - 1) / BM;
    r.ntn = (cols + BN - 1) / BN;
    r.nmat = nm;
    r.wide = cols % 8 == 0 && (uintptr_t)out % 16 == 0;
    r.total = (int64_t)nm * r.ntm * r.ntn;
    ortho_out<<<(unsigned)pad_grid(r.total), kThreads, 0, s>>>(r);
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

int64_t ortho_ws_bytes(int32_t n, int32_t rows, int32_t cols) {
  if (n == 0) return 0;
  const OrthoLayout o = ortho_layout(n, rows, cols);
  return o.group * o.bytes;
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
