// Router of the MoonEP path on gfx950: the top-K choice and the route weights
// that planning and dispatch take (MoonEP README, "API guide > dispatch fwd":
// topk_experts_sk, route_weights_sk come from the framework's router), and
// their gradient with respect to the logits.
//
//   score_e = softmax(l)_e or sigma(l_e)
//   choice: the K largest of l_e, or of score_e + bias_e when a bias is given,
//           in descending order, equal ones by ascending expert
//   w_k    = scale * score_k, divided by the sum of the K scores if normalized
// and backward, with q = score of the chosen, g = scale * dw, t = sum_k q_k:
//   normalized: dq_k = (g_k - sum_j g_j q_j / t) / t, else dq_k = g_k
//   softmax:    dl_e = q_e (dq_e [chosen] - sum_j dq_j q_j); normalized this
//               is q_k (g_k - sum_j g_j q_j) with q the softmax over the chosen
//   sigmoid:    dl_k = dq_k sigma(l_k) sigma(-l_k), 0 elsewhere
// A logit of -inf closes its expert: it comes after every open one and its
// weight and gradient are 0; a token without an open expert has weights and
// gradients of 0.  A NaN comes first, so it shows in the weights; whatever the
// logits, the K ids of a token are distinct and in range.
//
// A token's row is read once by G lanes (a power of two), VPL consecutive
// logits each, and the kernel is bound by instructions rather than by its
// bytes, so the choice is kept short: each lane sorts its VPL keys once, and
// each of the K extractions is a maximum over the lanes' heads (a DPP
// butterfly on 32-bit keys that order like the floats), the lowest lane that
// has it (a ballot) and a shift in that lane's list.
#include "internal.h"

namespace moonep {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kNone = INT32_MIN;             // below every key

// float -> int32 of the same order; -0 like +0, NaN above +inf
__device__ __forceinline__ int key_of(float x) {
  x = x + 0.0f;
  const int b = __float_as_int(x);
  const int k = b ^ ((b >> 31) & 0x7FFFFFFF);
  return x != x ? 0x7FC00000 : k;
}
__device__ __forceinline__ float key_value(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF));
}

// Butterfly step over lanes 1, 2, 4, ... apart, of a value that is already
// equal within each aligned run of 1 << STEP lanes: the mirrored row patterns
// then do for an exchange.
template <int STEP>
__device__ __forceinline__ int swap_lanes(int v) {
  if constexpr (STEP == 0) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);   // quad 1,0,3,2
  if constexpr (STEP == 1) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);   // quad 2,3,0,1
  if constexpr (STEP == 2) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);  // half-row mirror
  if constexpr (STEP == 3) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);  // row mirror
  if constexpr (STEP == 4) return __shfl_xor(v, 16, 64);
  if constexpr (STEP == 5) return __shfl_xor(v, 32, 64);
}
template <int G, int STEP = 0>
__device__ __forceinline__ int group_max(int v) {
  if constexpr ((1 << STEP) >= G) return v;
  else {
    const int o = swap_lanes<STEP>(v);
    return group_max<G, STEP + 1>(o > v ? o : v);
  }
}
template <int G, int STEP = 0>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr ((1 << STEP) >= G) return v;
  else return group_sum<G, STEP + 1>(v + __int_as_float(swap_lanes<STEP>(__float_as_int(v))));
}
template <int G>
__device__ __forceinline__ float group_maxf(float v) {   // NaN and -inf kept, as the keys order them
  return key_value(group_max<G>(key_of(v)));
}
template <int G>
__device__ __forceinline__ double group_sum64(double v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// The lowest lane (within its group of G) for which `hit` holds; one does.
template <int G>
__device__ __forceinline__ int first_lane(bool hit) {
  const uint64_t m = __ballot(hit);
  if constexpr (G == 64) {
    return __builtin_ctzll(m);
  } else {
    const int lane = threadIdx.x & 63;
    const uint32_t half = lane & 32 ? (uint32_t)(m >> 32) : (uint32_t)m;
    return __builtin_ctz(half >> (lane & 31 & ~(G - 1)));
  }
}

template <class T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float(float v) { return v; }
template <> __device__ __forceinline__ float to_float(uint16_t v) {
  return __uint_as_float((uint32_t)v << 16);
}
template <class T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float(float v) { return v; }
template <> __device__ __forceinline__ uint16_t from_float(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// VPL consecutive elements starting at p + e0 as a vector of the widest
// aligned pieces; vec: E % VPL == 0 and a 16-byte aligned array.
template <class T, int VPL>
struct Pack {
  static constexpr int kBytes = VPL * (int)sizeof(T);
  static constexpr int kUnit = kBytes % 16 == 0 ? 16 : kBytes % 8 == 0 ? 8 : 4;
  struct __attribute__((aligned(kUnit))) Raw {
    T v[VPL];
  };
};
template <class T, int VPL>
__device__ __forceinline__ void load_row(const T* row, int E, int e0, bool vec, float out[VPL]) {
  if (vec) {
    if (e0 < E) {
      const typename Pack<T, VPL>::Raw r = *(const typename Pack<T, VPL>::Raw*)(row + e0);
#pragma unroll
      for (int j = 0; j < VPL; ++j) out[j] = to_float<T>(r.v[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j < E) out[j] = to_float<T>(row[e0 + j]);
  }
}

struct RouteArgs {
  const void* logits;    // [T][E]
  const float* bias;     // [E] or null
  int32_t* topk;         // [T][K]
  float* rw;             // [T][K]
  const float* drw;      // [T][K] (backward)
  void* dlogits;         // [T][E] (backward)
  float scale;
  int T, E, K, normalize, vec;
};

enum { kLogits = 0, kSigmoidBias, kSoftmaxBias };      // what the choice goes by

// sum that a softmax divides by, and the value it subtracts: a row with no open expert has
// e^(l - 0) = 0 everywhere and a sum of 0, for which its reciprocal is taken as 0
__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float inv_or_zero(float s) { return s == 0.0f ? 0.0f : 1.0f / s; }
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// The choice in 64 bits, for the rows where two of the first K + 1 scores
// stand closer than their rounding in 32: the same extractions on doubles.
template <int G, int VPL, int BY>
__device__ __forceinline__ void choose64(const float* l, const float* bias, int E, int K,
                                                   int e0, int gl, int sel[32 / (G < 32 ? G : 32)]) {
  double key[VPL];
  double top = -INFINITY, sum = 0.0;
  if (BY == kSoftmaxBias) {
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j < E && (double)l[j] > top) top = (double)l[j];
#pragma unroll
    for (int o = 1; o < G; o <<= 1) {
      const double t = __shfl_xor(top, o, 64);
      top = t > top ? t : top;
    }
    if (top == -INFINITY) top = 0.0;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j < E) sum += exp((double)l[j] - top);
    sum = group_sum64<G>(sum);
    if (sum == 0.0) sum = 1.0;
  }
  uint32_t left = 0;                           // elements not taken yet
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const double x = (double)l[j];
    double s = BY == kSoftmaxBias ? exp(x - top) / sum : 1.0 / (1.0 + exp(-x));
    if (e0 + j < E) {
      s += (double)bias[e0 + j];
      left |= 1u << j;
    }
    if (l[j] == -INFINITY) s = -INFINITY;
    key[j] = s != s ? INFINITY : s;            // NaN beside +inf: both come first
  }
  for (int k = 0; k < K; ++k) {
    double best = -INFINITY;
    int at = 1 << 20;                          // expert id; none
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if ((left >> j & 1) && (key[j] > best || at == 1 << 20)) {
        best = key[j];
        at = e0 + j;
      }
#pragma unroll
    for (int o = 1; o < G; o <<= 1) {
      const double b = __shfl_xor(best, o, 64);
      const int i = __shfl_xor(at, o, 64);
      if ((b > best && i != 1 << 20) || (b == best && i < at)) {
        best = b;
        at = i;
      }
    }
    if (at >= e0 && at < e0 + VPL) left &= ~(1u << (at - e0));
#pragma unroll
    for (int q = 0; q < 32 / (G < 32 ? G : 32); ++q)
      if (k == q * G + gl) sel[q] = at;
  }
}

template <class T, int G, int VPL, int BY, bool kSigmoid>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
  constexpr int kSel = 32 / (G < 32 ? G : 32);          // chosen experts a lane keeps
  const int lane = threadIdx.x & 63, gl = lane % G;
  const int64_t row = ((int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6)) * (64 / G) + lane / G;
  if (row >= a.T) return;                               // whole groups
  const T* lrow = (const T*)a.logits + row * a.E;
  const int e0 = gl * VPL;
  float l[VPL];
  load_row<T, VPL>(lrow, a.E, e0, a.vec, l);

  // softmax over all experts: its maximum and the inverse of its sum
  float top = 0.0f, inv = 0.0f;
  if (BY == kSoftmaxBias || (!kSigmoid && !a.normalize)) {
    int m = kNone;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int k = e0 + j < a.E ? key_of(l[j]) : kNone;
      m = k > m ? k : m;
    }
    top = finite_or_zero(key_value(group_max<G>(m)));
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j < a.E) s += expf(l[j] - top);
    inv = inv_or_zero(group_sum<G>(s));
  }

  int key[VPL], id[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    id[j] = e0 + j;
    key[j] = kNone;
    if (e0 + j < a.E) {
      float s = l[j];
      if (BY != kLogits) {
        s = (BY == kSigmoidBias ? sigmoid(l[j]) : expf(l[j] - top) * inv) + a.bias[e0 + j];
        if (l[j] == -INFINITY) s = -INFINITY;
      }
      key[j] = key_of(s);
    }
  }
  // sort the lane's keys, descending; neighbours change places only when
  // strictly out of order, so equal keys keep ascending experts
#pragma unroll
  for (int p = VPL - 1; p > 0; --p)
#pragma unroll
    for (int j = 0; j < p; ++j) {
      const bool less = key[j] < key[j + 1];
      const int hk = less ? key[j + 1] : key[j], lk = less ? key[j] : key[j + 1];
      const int hi = less ? id[j + 1] : id[j], li = less ? id[j] : id[j + 1];
      key[j] = hk; key[j + 1] = lk;
      id[j] = hi; id[j + 1] = li;
    }

  int sel[kSel];
  float val[kSel];                                      // the chosen expert's logit
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    sel[q] = 0;
    val[q] = 0.0f;
  }
  bool close = false;                                   // two neighbours within their rounding
  float prev = INFINITY;
  const int base = lane & ~(G - 1);
  const int rounds = BY != kLogits && a.K < a.E ? a.K + 1 : a.K;
  for (int k = 0; k < rounds; ++k) {
    const int m = group_max<G>(key[0]);
    const int win = first_lane<G>(key[0] == m);
    const int e = G == 64 ? __builtin_amdgcn_readlane(id[0], win) : __shfl(id[0], base + win, 64);
    if (BY != kLogits) {
      // The 32-bit score is within 2^-20 of the exact one (exp, reciprocal and
      // product: a few units of 2^-24 of a value of at most 1) and its sum with
      // the bias is rounded once more.
      const float v = key_value(m);
      if (k > 0 && !(prev - v > 0x1p-19f + 0x1p-22f * (fabsf(v) + fabsf(prev)))) close = true;
      prev = v;
    }
#pragma unroll
    for (int q = 0; q < kSel; ++q)
      if (k < a.K && k == q * G + gl) {
        sel[q] = e;
        if (BY == kLogits) val[q] = key_value(m);
      }
    if (gl == win) {
#pragma unroll
      for (int j = 0; j + 1 < VPL; ++j) {
        key[j] = key[j + 1];
        id[j] = id[j + 1];
      }
      key[VPL - 1] = kNone;
    }
  }
  if (BY != kLogits) {
    // the whole group takes the 64-bit choice (every lane of it saw the same keys)
    if (close) choose64<G, VPL, BY>(l, a.bias, a.E, a.K, e0, gl, sel);
#pragma unroll
    for (int q = 0; q < kSel; ++q) {
      const int k = q * G + gl;
      val[q] = to_float<T>(lrow[k < a.K ? sel[q] : 0]);
    }
  }

  // weights: lane gl holds the chosen experts gl, gl + G, ...
  float w[kSel];
  float mx = 0.0f;
  if (!kSigmoid && a.normalize) {
    int m = kNone;
#pragma unroll
    for (int q = 0; q < kSel; ++q) {
      const int k = q * G + gl < a.K ? key_of(val[q]) : kNone;
      m = k > m ? k : m;
    }
    mx = finite_or_zero(key_value(group_max<G>(m)));
  } else if (!kSigmoid) {
    mx = top;
  }
  float sum = 0.0f;
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    w[q] = kSigmoid ? sigmoid(val[q]) : expf(val[q] - mx);
    if (q * G + gl < a.K) sum += w[q];
  }
  float f = kSigmoid ? 1.0f : inv;
  if (a.normalize) f = inv_or_zero(group_sum<G>(sum));
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    const int k = q * G + gl;
    if (k < a.K) {
      a.topk[row * a.K + k] = sel[q];
      a.rw[row * a.K + k] = w[q] * f * a.scale;
    }
  }
}

// A wave's own LDS operations complete in order; only the compiler must not
// move them across this point.
__device__ __forceinline__ void lds_settled() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Backward: the chosen experts' gradients are scattered into a row of LDS
// (zeros elsewhere), from which the G lanes write the whole row.
template <class T, int G, int VPL, bool kSigmoid>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(RouteArgs a) {
  constexpr int kSel = 32 / (G < 32 ? G : 32);
  __shared__ __attribute__((aligned(16))) float rows[kWaves * 64 * VPL];
  const int lane = threadIdx.x & 63, gl = lane % G, wv = threadIdx.x >> 6;
  const int64_t row = ((int64_t)blockIdx.x * kWaves + wv) * (64 / G) + lane / G;
  if (row >= a.T) return;
  const T* lrow = (const T*)a.logits + row * a.E;
  float* lds = rows + (wv * (64 / G) + lane / G) * (G * VPL);
  const int e0 = gl * VPL;
#pragma unroll
  for (int j = 0; j < VPL; ++j) lds[e0 + j] = 0.0f;
  lds_settled();

  const bool dense = !kSigmoid && !a.normalize;
  float l[VPL];
  float top = 0.0f, inv = 0.0f;
  if (dense) {
    load_row<T, VPL>(lrow, a.E, e0, a.vec, l);
    int m = kNone;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int k = e0 + j < a.E ? key_of(l[j]) : kNone;
      m = k > m ? k : m;
    }
    top = finite_or_zero(key_value(group_max<G>(m)));
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      l[j] = e0 + j < a.E ? expf(l[j] - top) : 0.0f;
      s += l[j];
    }
    inv = inv_or_zero(group_sum<G>(s));
  }

  int id[kSel];
  float x[kSel], g[kSel];
  int m = kNone;
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    const int k = q * G + gl;
    id[q] = k < a.K ? a.topk[row * a.K + k] : -1;
    if ((unsigned)id[q] >= (unsigned)a.E) id[q] = -1;   // never out of the row
    g[q] = id[q] < 0 ? 0.0f : a.drw[row * a.K + k] * a.scale;
    x[q] = id[q] < 0 ? -INFINITY : to_float<T>(lrow[id[q]]);
    const int kx = id[q] < 0 ? kNone : key_of(x[q]);
    m = kx > m ? kx : m;
  }
  if (!kSigmoid && !dense) top = finite_or_zero(key_value(group_max<G>(m)));
  float p[kSel], t = 0.0f;
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    p[q] = id[q] < 0 ? 0.0f : kSigmoid ? sigmoid(x[q]) : expf(x[q] - top);
    t += p[q];
  }
  float gq = 0.0f;
  if (a.normalize) {
    inv = inv_or_zero(group_sum<G>(t));
  } else if (kSigmoid) {
    inv = 1.0f;
  }
#pragma unroll
  for (int q = 0; q < kSel; ++q) gq += g[q] * (p[q] * inv);
  if (a.normalize || dense) gq = group_sum<G>(gq);
  else gq = 0.0f;
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    float d;
    if (dense) d = g[q];
    else if (!kSigmoid) d = p[q] * inv * (g[q] - gq);
    else d = (g[q] - gq) * inv * p[q] * sigmoid(-x[q]);
    if (id[q] >= 0) lds[id[q]] = d;
  }
  lds_settled();
  float d[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    d[j] = lds[e0 + j];
    if (dense) d[j] = l[j] * inv * (d[j] - gq);
  }
  T* out = (T*)a.dlogits + row * a.E;
  if (a.vec) {
    if (e0 < a.E) {
      typename Pack<T, VPL>::Raw r;
#pragma unroll
      for (int j = 0; j < VPL; ++j) r.v[j] = from_float<T>(d[j]);
      *(typename Pack<T, VPL>::Raw*)(out + e0) = r;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (e0 + j < a.E) out[e0 + j] = from_float<T>(d[j]);
  }
}

template <class T, int G, int VPL>
void run_route(RouteArgs a, const RouteForm& f, bool bwd, hipStream_t s) {
  const unsigned per = kWaves * (64 / G);
  const unsigned blocks = (unsigned)(((int64_t)a.T + per - 1) / per);
  a.vec = a.E % VPL == 0 && (uintptr_t)a.logits % 16 == 0 && (uintptr_t)a.dlogits % 16 == 0;
  const bool sig = f.score == MOONEP_SCORE_SIGMOID;
  if (bwd) {
    if (sig) route_bwd_kernel<T, G, VPL, true><<<blocks, kThreads, 0, s>>>(a);
    else route_bwd_kernel<T, G, VPL, false><<<blocks, kThreads, 0, s>>>(a);
  } else if (!a.bias) {
    if (sig) route_kernel<T, G, VPL, kLogits, true><<<blocks, kThreads, 0, s>>>(a);
    else route_kernel<T, G, VPL, kLogits, false><<<blocks, kThreads, 0, s>>>(a);
  } else if (sig) {
    route_kernel<T, G, VPL, kSigmoidBias, true><<<blocks, kThreads, 0, s>>>(a);
  } else {
    route_kernel<T, G, VPL, kSoftmaxBias, false><<<blocks, kThreads, 0, s>>>(a);
  }
}

// Lanes and logits per lane for E experts: four logits per lane while the
// lanes last (a row's 16 bytes per lane in one load), then more logits.
template <class T>
hipError_t route_by_size(const RouteArgs& a, const RouteForm& f, bool bwd, hipStream_t s) {
  if (a.E <= 32) run_route<T, 8, 4>(a, f, bwd, s);
  else if (a.E <= 64) run_route<T, 16, 4>(a, f, bwd, s);
  else if (a.E <= 128) run_route<T, 32, 4>(a, f, bwd, s);
  else if (a.E <= 256) run_route<T, 64, 4>(a, f, bwd, s);
  else if (a.E <= 384) run_route<T, 64, 6>(a, f, bwd, s);
  else if (a.E <= 512) run_route<T, 64, 8>(a, f, bwd, s);
  else run_route<T, 64, 16>(a, f, bwd, s);
  return hipGetLastError();
}

RouteArgs route_args(const Ctx& c, const RouteForm& f) {
  RouteArgs a;
  a.logits = nullptr; a.bias = nullptr; a.topk = nullptr; a.rw = nullptr;
  a.drw = nullptr; a.dlogits = nullptr;
  a.scale = f.scale;
  a.T = c.d.R * c.d.S; a.E = c.d.E; a.K = c.d.K; a.normalize = f.normalize; a.vec = 0;
  return a;
}

}  // namespace

hipError_t launch_route(const Ctx& c, const void* logits, const float* bias, const RouteForm& f,
                        int32_t* topk, float* rw, hipStream_t s) {
  RouteArgs a = route_args(c, f);
  a.logits = logits; a.bias = bias; a.topk = topk; a.rw = rw;
  return f.dtype == MOONEP_F32 ? route_by_size<float>(a, f, false, s)
                               : route_by_size<uint16_t>(a, f, false, s);
}

hipError_t launch_route_bwd(const Ctx& c, const void* logits, const RouteForm& f,
                            const int32_t* topk, const float* drw, void* dlogits, hipStream_t s) {
  RouteArgs a = route_args(c, f);
  a.logits = logits; a.topk = const_cast<int32_t*>(topk); a.drw = drw; a.dlogits = dlogits;
  return f.dtype == MOONEP_F32 ? route_by_size<float>(a, f, true, s)
                               : route_by_size<uint16_t>(a, f, true, s);
}

}  // namespace moonep
