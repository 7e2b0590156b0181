// A block's end and the next one's start on gfx950: the block's outputs are
// summed, normalised, gated, scaled and added to the residual stream, and the
// stream is normalised for what comes next, in one pass; and its gradients.
// In a block with experts y is combine's output (MoonEP README, "API guide >
// combine fwd": output_sh) and y2 the shared expert's.
//
//   a  = y (+ y2)
//   n  = a rstd(a) w_post          rstd(v) = (mean(v^2) + eps)^(-1/2); n = a without w_post
//   h' = h + scale gate n          gate: one, [W], [T] or [T,W]
//   u  = h' rstd(h') w_pre
// and backward, with dh the gradient of h', du that of u, s = rstd(h'), r = rstd(a):
//   v  = du w_pre,  D = dh + s (v - h' s^2 mean(v h'))     the stream's gradient
//   dw_pre = sum_t du h' s
//   dn = scale gate D,  dgate = scale D n  (summed over what the gate is shared by)
//   v  = dn w_post,  dy = r (v - a r^2 mean(v a)),  dw_post = sum_t dn a r
//
// Design for CDNA4: every operand is read once and every result written once,
// so a row stays in registers between its sums.  A row of up to 1024 elements
// belongs to a wave, whose sums need no barrier; a longer one to a workgroup of
// as few waves as hold it with one 8-element vector a lane (up to 4096) or two, in
// the backward beyond 8192 four.
// Bound by bytes: 32768 rows of 7168 in bf16 with two outputs and both norms take
// 450 us (2.35 GB, 5.2 TB/s; a copy reaches 4.9 to 5.4), backward 705 us (3.29 GB
// and the shares below; 664 us without its sums).
#include "internal.h"

namespace moonep {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kVals = 3;           // sums taken together

__device__ __forceinline__ unsigned pack2(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
}

// Eight elements of a row as they lie in memory.
template <class T> struct Raw;
template <> struct Raw<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *(const u32x4*)p; }
  __device__ __forceinline__ void zero() { v = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int i) const {
    const unsigned w = v[i >> 1];
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
};
template <> struct Raw<float> {
  f32x4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = *(const f32x4*)p;
    v[1] = *(const f32x4*)(p + 4);
  }
  __device__ __forceinline__ void zero() { v[0] = v[1] = f32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int i) const { return v[i >> 2][i & 3]; }
};
__device__ __forceinline__ void put8(uint16_t* p, const float f[8], bool past) {
  const u32x4 v = {pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
  if (past) __builtin_nontemporal_store(v, (u32x4*)p);
  else *(u32x4*)p = v;
}
__device__ __forceinline__ void put8(float* p, const float f[8], bool past) {
  const f32x4 v[2] = {{f[0], f[1], f[2], f[3]}, {f[4], f[5], f[6], f[7]}};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (past) __builtin_nontemporal_store(v[i], (f32x4*)p + i);
    else *((f32x4*)p + i) = v[i];
  }
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float f[8]) {
  put8(p, f, false);
}

// Sum of 16 lanes, the same in each of them.
__device__ __forceinline__ float sum16(float v) {
#define MOONEP_STEP(ctrl) \
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), ctrl, 0xF, 0xF, true))
  MOONEP_STEP(0xB1);    // quad 1,0,3,2
  MOONEP_STEP(0x4E);    // quad 2,3,0,1
  MOONEP_STEP(0x141);   // half-row mirror
  MOONEP_STEP(0x140);   // row mirror
#undef MOONEP_STEP
  return v;
}
__device__ __forceinline__ float lane_of(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

// Sums of N values over the lanes of a row: a wave's, or a workgroup's through
// LDS, where two buffers take turns, so that one barrier a sum is enough (a
// buffer is written again only behind the barrier of the sum in between).
template <bool kWave>
struct RowSum {
  float (*buf)[kVals][16];
  int turn;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    static_assert(N <= kVals, "one row of 16 lanes a value");
    float t[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float s = sum16(v[i]);
      t[i] = (lane_of(s, 0) + lane_of(s, 16)) + (lane_of(s, 32) + lane_of(s, 48));
    }
    if constexpr (!kWave) {
      const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
      float (*b)[16] = buf[turn];
      turn ^= 1;
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) b[i][wave] = t[i];
      }
      __syncthreads();
      const int row = lane >> 4, col = lane & 15;
      const float s = sum16(row < N && col < (int)(blockDim.x >> 6) ? b[row < N ? row : 0][col] : 0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = lane_of(s, 16 * i);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = t[i];
  }
};

// The lanes of a row and the rows of a workgroup.
template <bool kWave>
struct Place {
  int lane, lanes;           // of the row
  int64_t row, step;         // first row and distance to the next
  __device__ __forceinline__ Place() {
    if constexpr (kWave) {
      lane = threadIdx.x & 63;
      lanes = 64;
      row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
      step = (int64_t)gridDim.x * 4;
    } else {
      lane = threadIdx.x;
      lanes = blockDim.x;
      row = blockIdx.x;
      step = gridDim.x;
    }
  }
};

__device__ __forceinline__ float rstd(float ss, float inv_w, float eps) {
  return 1.0f / sqrtf(ss * inv_w + eps);
}

// A row as it is loaded.
template <class TS, int VPT>
struct RowIn {
  Raw<TS> h[VPT];
  Raw<uint16_t> y[VPT], y2[VPT], g[VPT];
  float gt;
  template <bool kWave>
  __device__ __forceinline__ void load(const NormArgs& a, const Place<kWave>& at, int64_t r) {
    gt = a.gate_kind == MOONEP_GATE_TOKEN ? ((const float*)a.gate)[r] : 1.0f;
    const int64_t base = r * a.W;
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int c = 8 * (at.lane + p * at.lanes);
      h[p].zero();
      y[p].zero();
      y2[p].zero();
      g[p].zero();
      if (c < a.W) {
        h[p].load((const TS*)a.h + base + c);
        if (a.y) y[p].load(a.y + base + c);
        if (a.y2) y2[p].load(a.y2 + base + c);
        if (a.gate_kind == MOONEP_GATE_FULL) g[p].load((const uint16_t*)a.gate + base + c);
      }
    }
  }
};

template <class TS, int VPT, bool kWave, int kMost>
__global__ __launch_bounds__(kMost) void norm_kernel(NormArgs a) {
  __shared__ float red[2][kVals][16];
  RowSum<kWave> sum{red, 0};
  const Place<kWave> at;
  const int W = a.W;
  const float inv_w = 1.0f / (float)W;
  // Results that the caches cannot hold are stored past them (32768 rows of 7168 in bf16: 454 ->
  // 442 us; the backward, stored so, 704 -> 743 us).
  const bool past = a.T * W > (int64_t(1) << 25);
  for (int64_t r = at.row; r < a.T; r += at.step) {
    const int64_t base = r * W;
    RowIn<TS, VPT> cur;
    cur.load(a, at, r);
    float h[VPT][8];
    float ss[1] = {0.0f};
#pragma unroll
    for (int p = 0; p < VPT; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[p][i] = cur.y[p].get(i) + cur.y2[p].get(i);
        ss[0] += h[p][i] * h[p][i];
      }
    float ra = 1.0f;
    if (a.w_post) {
      sum(ss);
      ra = rstd(ss[0], inv_w, a.eps);
    }
    const float f = a.scale * cur.gt;
    ss[0] = 0.0f;
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int c = 8 * (at.lane + p * at.lanes);
      if (c < W) {
        if (a.y) {
          Raw<float> w, g;
          if (a.w_post) w.load(a.w_post + c);
          if (a.gate_kind == MOONEP_GATE_CHANNEL) g.load((const float*)a.gate + c);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float n = h[p][i];
            if (a.w_post) n *= ra * w.get(i);
            if (a.gate_kind == MOONEP_GATE_CHANNEL) n *= g.get(i);
            if (a.gate_kind == MOONEP_GATE_FULL) n *= cur.g[p].get(i);
            h[p][i] = cur.h[p].get(i) + f * n;
          }
          put8((TS*)a.h_out + base + c, h[p], past);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) h[p][i] = cur.h[p].get(i);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] += h[p][i] * h[p][i];
      }
    }
    if (a.w_pre) {
      sum(ss);
      const float rh = rstd(ss[0], inv_w, a.eps);
#pragma unroll
      for (int p = 0; p < VPT; ++p) {
        const int c = 8 * (at.lane + p * at.lanes);
        if (c < W) {
          Raw<float> w;
          w.load(a.w_pre + c);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[p][i] *= rh * w.get(i);
          put8(a.u + base + c, h[p], past);
        }
      }
    }
  }
}

template <class TS, int VPT>
struct RowBwdIn {
  Raw<TS> h[VPT], dh[VPT];
  Raw<uint16_t> du[VPT], y[VPT], y2[VPT], g[VPT];
  float gt;
  template <bool kWave>
  __device__ __forceinline__ void load(const NormBwdArgs& a, const Place<kWave>& at, int64_t r,
                                       bool need_a) {
    gt = a.gate_kind == MOONEP_GATE_TOKEN ? ((const float*)a.gate)[r] : 1.0f;
    const int64_t base = r * a.W;
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int c = 8 * (at.lane + p * at.lanes);
      h[p].zero();
      dh[p].zero();
      du[p].zero();
      y[p].zero();
      y2[p].zero();
      g[p].zero();
      if (c < a.W) {
        if (a.w_pre) {
          h[p].load((const TS*)a.h + base + c);
          du[p].load(a.du + base + c);
        }
        if (a.dh) dh[p].load((const TS*)a.dh + base + c);
        if (need_a) {
          y[p].load(a.y + base + c);
          if (a.y2) y2[p].load(a.y2 + base + c);
        }
        if (a.gate_kind == MOONEP_GATE_FULL) g[p].load((const uint16_t*)a.gate + base + c);
      }
    }
  }
};

// A lane's sums over tokens for its columns, in registers or, where these do not
// hold all three, in LDS, whose places no other lane touches.
template <int VPT, bool kLds>
struct Sums {
  float v[VPT][8];
  __device__ __forceinline__ Sums(void*) {
#pragma unroll
    for (int p = 0; p < VPT; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
  }
  __device__ __forceinline__ void add(int p, const float (&t)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[p][i] += t[i];
  }
  __device__ __forceinline__ void store(int p, float* to) const { store8(to, v[p]); }
};
template <int VPT>
struct Sums<VPT, true> {
  typedef __attribute__((address_space(3))) f32x4 lds_f4;
  static constexpr int kBytes = 512 * VPT * 32;
  lds_f4* at;                          // the next four of a lane's sums lie 512 places on
  __device__ __forceinline__ Sums(void* lds) : at((lds_f4*)lds + threadIdx.x) {
#pragma unroll
    for (int q = 0; q < 2 * VPT; ++q) at[512 * q] = f32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void add(int p, const float (&t)[8]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f32x4 o = at[512 * (2 * p + q)];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += t[4 * q + e];
      at[512 * (2 * p + q)] = o;
    }
  }
  __device__ __forceinline__ void store(int p, float* to) const {
#pragma unroll
    for (int q = 0; q < 2; ++q) *((f32x4*)to + q) = at[512 * (2 * p + q)];
  }
};

// A workgroup's share of one sum; the sums of four waves with rows of their own
// leave as one.
template <int VPT, bool kWave, class S>
__device__ __forceinline__ void put_share(const S& s, const Place<kWave>& at, int W, float* q) {
  if constexpr (kWave) {
    __shared__ __attribute__((aligned(16))) float four[4][64 * 8 * VPT];
    __syncthreads();
#pragma unroll
    for (int p = 0; p < VPT; ++p) s.store(p, &four[threadIdx.x >> 6][8 * (at.lane + 64 * p)]);
    __syncthreads();
    for (int c = 4 * threadIdx.x; c < W; c += 1024) {
      f32x4 t = *(const f32x4*)&four[0][c];
#pragma unroll
      for (int w = 1; w < 4; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] += four[w][c + e];
      *(f32x4*)(q + c) = t;
    }
  } else {
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int c = 8 * (at.lane + p * at.lanes);
      if (c < W) s.store(p, q + c);
    }
  }
}

// Sums over tokens stay with a lane, for its columns, over all rows of its
// wave or workgroup; each workgroup then writes its share to part [3][shares][W]
// and norm_bwd_sum adds the shares, in an order that T and W fix.  With four
// vectors a lane two of the three sums lie in LDS (8192 rows of 16384 in bf16 with
// two outputs 443 us, 4.2 TB/s; two vectors in 1024 lanes, whose 128 registers
// spill, 1394 us).  Up to 8192
// elements registers hold all (32768 rows of 7168 707 us, in LDS 742 us).
template <class TS, int VPT, bool kWave, int kMost>
__global__ __launch_bounds__(kMost) void norm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[2][kVals][16];
  RowSum<kWave> sum{red, 0};
  const Place<kWave> at;
  const int W = a.W;
  const float inv_w = 1.0f / (float)W;
  const bool channel = a.gate_kind == MOONEP_GATE_CHANNEL && a.dgate;
  const bool need_a = a.y && (a.w_post || a.gate_kind != MOONEP_GATE_NONE);
  constexpr bool kLds = VPT == 4;
  __shared__ __attribute__((aligned(16))) char held[2][kLds ? Sums<VPT, true>::kBytes : 16];
  Sums<VPT, false> s_pre(nullptr);
  Sums<VPT, kLds> s_post(held[0]), s_gate(held[1]);
  for (int64_t r = at.row; r < a.T; r += at.step) {
    const int64_t base = r * W;
    Place<kWave> in = at;
    // the addresses are taken anew for each row: kept, they would make the widest rows spill
    if constexpr (kLds) asm volatile("" : "+v"(in.lane));
    RowBwdIn<TS, VPT> cur;
    cur.load(a, in, r, need_a);
    float d[VPT][8], av[VPT][8];
    float s3[3] = {0.0f, 0.0f, 0.0f};       // h'^2, v h', a^2: each vector's, then theirs
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int c = 8 * (in.lane + p * in.lanes);
      Raw<float> w;
      w.zero();
      if (a.w_pre && c < W) w.load(a.w_pre + c);
      float t[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = cur.h[p].get(i);
        av[p][i] = cur.y[p].get(i) + cur.y2[p].get(i);
        d[p][i] = cur.du[p].get(i) * w.get(i);
        t[0] += h * h;
        t[1] += d[p][i] * h;
        t[2] += av[p][i] * av[p][i];
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) s3[k] += t[k];
    }
    if (a.w_pre || a.w_post) sum(s3);
    const float rh = a.w_pre ? rstd(s3[0], inv_w, a.eps) : 0.0f;
    const float ra = a.w_post ? rstd(s3[2], inv_w, a.eps) : 1.0f;
    const float mh = s3[1] * inv_w * rh * rh;
    float s2[2] = {0.0f, 0.0f};             // D n, w_post dn a
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      const int c = 8 * (in.lane + p * in.lanes);
      if (c < W) {
        Raw<float> w, g;
        if (a.w_post) w.load(a.w_post + c);
        if (a.gate_kind == MOONEP_GATE_CHANNEL) g.load((const float*)a.gate + c);
        float dg[8], dw[8], t[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float h = cur.h[p].get(i);
          dw[i] = cur.du[p].get(i) * (h * rh);
          d[p][i] = cur.dh[p].get(i) + rh * (d[p][i] - h * mh);
        }
        s_pre.add(p, dw);
        store8((TS*)a.dres + base + c, d[p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float hat = av[p][i] * ra;
          const float n = a.w_post ? hat * w.get(i) : hat;
          const float sd = a.scale * d[p][i];
          dg[i] = sd * n;
          t[0] += dg[i];
          float dn = sd * cur.gt;
          if (a.gate_kind == MOONEP_GATE_CHANNEL) dn *= g.get(i);
          if (a.gate_kind == MOONEP_GATE_FULL) dn *= cur.g[p].get(i);
          dw[i] = dn * hat;
          d[p][i] = a.w_post ? dn * w.get(i) : dn;
          t[1] += d[p][i] * av[p][i];
        }
        s2[0] += t[0];
        s2[1] += t[1];
        if (!kLds || a.dw_post) s_post.add(p, dw);
        if (!kLds || channel) s_gate.add(p, dg);
        if (a.gate_kind == MOONEP_GATE_FULL && a.dgate) store8((uint16_t*)a.dgate + base + c, dg);
      }
    }
    const bool token = a.gate_kind == MOONEP_GATE_TOKEN && a.dgate;
    if (token || (a.dy && a.w_post)) sum(s2);
    if (token && in.lane == 0) ((float*)a.dgate)[r] = s2[0];
    if (a.dy) {
      const float ma = a.w_post ? s2[1] * inv_w * ra * ra : 0.0f;
#pragma unroll
      for (int p = 0; p < VPT; ++p) {
        const int c = 8 * (in.lane + p * in.lanes);
        if (c < W) {
#pragma unroll
          for (int i = 0; i < 8; ++i)         // without a norm a is no part of it, infinite or not
            d[p][i] = a.w_post ? ra * (d[p][i] - av[p][i] * ma) : d[p][i];
          store8(a.dy + base + c, d[p]);
        }
      }
    }
  }
  if (!a.part) return;
  float* q = a.part + (int64_t)blockIdx.x * W;
  const int64_t each = (int64_t)a.shares * W;
  if (a.dw_pre) put_share<VPT, kWave>(s_pre, at, W, q);
  if (a.dw_post) put_share<VPT, kWave>(s_post, at, W, q + each);
  if (channel) put_share<VPT, kWave>(s_gate, at, W, q + 2 * each);
}

// out_k [W] = the sum of the shares of part[k]: a workgroup takes 64 columns,
// each of its 16 waves every 16th share.
__global__ __launch_bounds__(1024) void norm_bwd_sum(const float* part, int shares, int W,
                                                     float* dw_pre, float* dw_post, float* dgate) {
  float* out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dgate;
  if (!out) return;
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const float* p = part + (int64_t)blockIdx.y * shares * W + c;
  float v = 0.0f;
  if (c < W) {
#pragma unroll 8
    for (int i = wave; i < shares; i += 16) v += p[(int64_t)i * W];
  }
  s[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && c < W) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][lane];
    out[c] = t;
  }
}

// Workgroups of a launch and the lanes of each: up to 1024 elements a wave, up to 4096 a workgroup
// with a vector a lane, beyond two, in the backward past 8192 four.  Workgroups per CU: as many as
// have `waves` waves, one at least.
// Forward: many more than run at once, so that a workgroup has few rows: of 7168 elements up to 18688
// workgroups, of 16384 up to 8192 (32768 rows of 7168 in bf16, one or two each: 448 us, with nine
// workgroups per CU 485 us; the next row's loads ahead of a row's sums 480 to 490 us).  Backward: as few
// workgroups as keep the CUs busy, for each leaves a share of the sums over tokens (702 us with one
// per CU, 728 us with three; 16384 rows of 4096 208 us with two per CU, 235 us with one).
struct NormGrid {
  int vpt, threads;
  bool wave;
  int64_t blocks;
};
NormGrid norm_grid(int64_t T, int W, bool bwd) {
  NormGrid g;
  const int vecs = W / 8;
  g.wave = vecs <= 128;
  g.vpt = vecs <= 64 || (vecs > 128 && vecs <= 512) ? 1 : bwd && vecs > 1024 ? 4 : 2;
  g.threads = g.wave ? 256 : (vecs + 64 * g.vpt - 1) / (64 * g.vpt) * 64;
  const int64_t need = g.wave ? (T + 3) / 4 : T;
  const int waves = !bwd ? 512 : g.vpt == 1 ? 16 : g.vpt == 2 ? 12 : 8;
  const int per_cu = waves * 64 / g.threads;
  const int64_t most = 256LL * (per_cu > 1 ? per_cu : 1);
  g.blocks = need < most ? need : most;
  return g;
}
}  // namespace

bool norm_shape_ok(int64_t T, int32_t W) {
  return T >= 0 && T < (int64_t(1) << 31) && W >= 8 && W % 8 == 0 && W <= MOONEP_NORM_MAX_W;
}

int32_t norm_shares(int64_t T, int32_t W) {
  return (int32_t)norm_grid(T, W, true).blocks;
}

int64_t norm_ws_bytes(int64_t T, int32_t W) { return 3LL * norm_shares(T, W) * W * 4; }

template <class TS>
static hipError_t norm_as(const NormArgs& a, hipStream_t s) {
  const NormGrid g = norm_grid(a.T, a.W, false);
  if (g.wave && g.vpt == 1) norm_kernel<TS, 1, true, 256><<<(unsigned)g.blocks, g.threads, 0, s>>>(a);
  else if (g.wave) norm_kernel<TS, 2, true, 256><<<(unsigned)g.blocks, g.threads, 0, s>>>(a);
  else if (g.vpt == 1) norm_kernel<TS, 1, false, 512><<<(unsigned)g.blocks, g.threads, 0, s>>>(a);
  else if (g.threads <= 512) norm_kernel<TS, 2, false, 512><<<(unsigned)g.blocks, g.threads, 0, s>>>(a);
  else norm_kernel<TS, 2, false, 1024><<<(unsigned)g.blocks, g.threads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_norm(const NormArgs& a, int32_t dtype, hipStream_t s) {
  return dtype == MOONEP_F32 ? norm_as<float>(a, s) : norm_as<uint16_t>(a, s);
}

template <class TS>
static hipError_t norm_bwd_as(const NormBwdArgs& a, hipStream_t s) {
  const NormGrid g = norm_grid(a.T, a.W, true);
  if (g.blocks == 0) {}                              // no tokens: the sums below are zeros
  else if (g.wave && g.vpt == 1) norm_bwd_kernel<TS, 1, true, 256><<<(unsigned)g.blocks, g.threads, 0, s>>>(a);
  else if (g.wave) norm_bwd_kernel<TS, 2, true, 256><<<(unsigned)g.blocks, g.threads, 0, s>>>(a);
  else if (g.vpt == 1) norm_bwd_kernel<TS, 1, false, 512><<<(unsigned)g.blocks, g.threads, 0, s>>>(a);
  else if (g.vpt == 2) norm_bwd_kernel<TS, 2, false, 512><<<(unsigned)g.blocks, g.threads, 0, s>>>(a);
  else norm_bwd_kernel<TS, 4, false, 512><<<(unsigned)g.blocks, g.threads, 0, s>>>(a);
  float* dgate = a.gate_kind == MOONEP_GATE_CHANNEL ? (float*)a.dgate : nullptr;
  if (a.dw_pre || a.dw_post || dgate) {
    norm_bwd_sum<<<dim3((unsigned)((a.W + 63) / 64), 3), 1024, 0, s>>>(a.part, a.shares, a.W,
                                                                      a.dw_pre, a.dw_post, dgate);
  }
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, int32_t dtype, hipStream_t s) {
  return dtype == MOONEP_F32 ? norm_bwd_as<float>(a, s) : norm_bwd_as<uint16_t>(a, s);
}

}  // namespace moonep
