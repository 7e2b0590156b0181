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
// gradients of 0.  A NaN comes first, so it shows in the weights (one in the bias comes
// first too, though no weight shows it); whatever the logits and the bias, the K ids of a
// token are distinct and in range.
//
// Design for CDNA4: the rows are short, so the kernels are bound by
// instructions and by the latency of a row's few dependent steps, not by their
// bytes.  G lanes take a row (four rows to a wave at 256 experts), with 16-byte
// loads dealt out lane by lane.  A logit (or score) and its expert are packed
// into one 64-bit key that orders like a double: the float's bits on top, the
// expert below, inverted where that makes the lower one larger.  A compare and
// exchange is then a v_max_f64 and a v_min_f64, no equal keys exist, and the
// expert comes along.  Every lane sorts its keys eight at a time, keeping the
// best; the K largest of the row are drawn from the heads of its lanes' lists by
// a DPP maximum.  (One row per wave, 32-bit keys with the expert beside them and a
// ballot for the lane: 21.6 us for 32768 rows of 256 fp32 logits, K = 8, and 89 us
// for 65536 rows of 384 bf16 logits with a bias; this form 9.4 us and 33 us under the
// profiler, 9.0 us and 29.6 us a call without it.)  Rows in which two of the first scores with a
// bias are equal or nearly so cost the exact ranking: the second case takes 144 us with a bias
// of zero, where bf16 logits often tie.
#include "internal.h"

namespace moonep {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

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
template <int STEP>
__device__ __forceinline__ double swap_lanes(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)swap_lanes<STEP>((int)(uint32_t)b);
  const uint32_t hi = (uint32_t)swap_lanes<STEP>((int)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// The larger of two keys.  An instruction by hand, since the compiler would
// put each operand through a maximum with itself first, in case it is a signalling
// NaN; the two wait states are those of a value that a DPP instruction reads next.
__device__ __forceinline__ double larger(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2\n\ts_nop 1" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
template <int G, int STEP = 0>
__device__ __forceinline__ double group_max(double v) {
  if constexpr ((1 << STEP) >= G) return v;
  else return group_max<G, STEP + 1>(larger(v, swap_lanes<STEP>(v)));
}
template <int G, int STEP = 0>
__device__ __forceinline__ float group_maxf(float v) {       // a NaN is passed over
  if constexpr ((1 << STEP) >= G) return v;
  else return group_maxf<G, STEP + 1>(
      __builtin_fmaxf(v, __int_as_float(swap_lanes<STEP>(__float_as_int(v)))));
}
template <int G, int STEP = 0>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr ((1 << STEP) >= G) return v;
  else return group_sum<G, STEP + 1>(v + __int_as_float(swap_lanes<STEP>(__float_as_int(v))));
}
template <int G, int STEP = 0>
__device__ __forceinline__ double group_sum(double v) {
  if constexpr ((1 << STEP) >= G) return v;
  else return group_sum<G, STEP + 1>(v + swap_lanes<STEP>(v));
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

// Lane gl of G holds VPL elements of a row: vectors gl, gl + G, ... of N = 16
// bytes each, so local element i is element_of(i).
template <class T, int G>
__device__ __forceinline__ int element_of(int gl, int i) {
  constexpr int N = 16 / (int)sizeof(T);
  return N * (gl + G * (i / N)) + i % N;
}
template <class T>
struct __attribute__((aligned(16))) Vec {
  T v[16 / sizeof(T)];
};
// wide: E is a multiple of N and the rows are 16-byte aligned.  Elements past
// the row are -inf: closed, and behind the row's own closed ones by their number.
template <class T, int G, int VPL>
__device__ __forceinline__ void load_row(const T* row, int E, int gl, bool wide, float out[VPL]) {
  constexpr int N = 16 / (int)sizeof(T);
  if (wide) {
#pragma unroll
    for (int j = 0; j < VPL / N; ++j) {
      const bool in = N * (gl + G * j) < E;
      Vec<T> r = {};
      if (in) r = *(const Vec<T>*)(row + N * (gl + G * j));
#pragma unroll
      for (int i = 0; i < N; ++i) out[N * j + i] = in ? to_float<T>(r.v[i]) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      out[i] = -INFINITY;
      if (element_of<T, G>(gl, i) < E) out[i] = to_float<T>(row[element_of<T, G>(gl, i)]);
    }
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
  int T, E, K, normalize;
  int wide, bias_wide;   // 16-byte loads of the rows, of the bias
};

enum { kLogits = 0, kSigmoidBias, kSoftmaxBias };      // what the choice goes by

// What a softmax subtracts and multiplies with: a row with no open expert has a maximum of -inf
// and a sum of 0, for which 0 and 0 are taken.
__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float inv_or_zero(float s) { return s == 0.0f ? 0.0f : 1.0f / s; }
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Softmax over all experts of a row: its maximum and the inverse of its sum.  The exponentials
// here are the hardware's (their error grows with the distance from the maximum as their
// share of the sum falls: |x| 2^-23 relative at e^x, under 2^-24 of the largest).  A lane adds
// its own in four chains, so that no value passes more than VPL / 4 + 1 + log2 G <= 13 additions,
// each of which may round a sum just above one up by 2^-24 of it.
// kKeep: l becomes the exponentials.
template <int G, int VPL, bool kKeep = false>
__device__ __forceinline__ void softmax_row(float l[VPL], float* top, float* inv) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    m = __builtin_fmaxf(m, l[i]);
  *top = finite_or_zero(group_maxf<G>(m));
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float e = __expf(l[i] - *top);
    s[i % 4] += e;
    if (kKeep) l[i] = e;
  }
  *inv = inv_or_zero(group_sum<G>((s[0] + s[1]) + (s[2] + s[3])));
}

// ------------------------------------------------------------------- keys
// Float x and expert e as a double: x's bits are its upper half (a float's
// exponent field is shorter, so no value, infinity or canonical NaN becomes a
// NaN or infinity of the double), the lower half e for a negative x and its
// complement otherwise: of equal x the lower expert has the larger key.
__device__ __forceinline__ double key_of(float x, int e) {
  const int b = x != x ? 0x7FC00000 : __float_as_int(x);
  const uint32_t lo = (uint32_t)(e ^ ~(b >> 31));
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)b << 32 | lo);
}
__device__ __forceinline__ double no_key() {           // below every key
  return __builtin_bit_cast(double, (uint64_t)0xFFEFFFFF00000000ull);
}
__device__ __forceinline__ float key_value(double k) {
  return __int_as_float((int)(__builtin_bit_cast(uint64_t, k) >> 32));
}
__device__ __forceinline__ int key_low(double k) { return (int)(uint32_t)__builtin_bit_cast(uint64_t, k); }
__device__ __forceinline__ int expert_of(int low) { return low < 0 ? ~low : low; }

__device__ __forceinline__ void order(double& a, double& b) {        // a >= b
  const double x = __builtin_fmax(a, b), y = __builtin_fmin(a, b);
  a = x;
  b = y;
}
// eight keys, descending: Batcher's odd-even merge sort
__device__ __forceinline__ void sort8(double k[8]) {
  order(k[0], k[1]); order(k[2], k[3]); order(k[4], k[5]); order(k[6], k[7]);
  order(k[0], k[2]); order(k[1], k[3]); order(k[4], k[6]); order(k[5], k[7]);
  order(k[1], k[2]); order(k[5], k[6]);
  order(k[0], k[4]); order(k[1], k[5]); order(k[2], k[6]); order(k[3], k[7]);
  order(k[2], k[4]); order(k[3], k[5]);
  order(k[1], k[2]); order(k[3], k[4]); order(k[5], k[6]);
}
__device__ __forceinline__ void bitonic8(double* k) {
#pragma unroll
  for (int s = 4; s > 0; s >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & s)) order(k[i], k[i + s]);
}
// Two sorted eights: the best eight in t, and in `next` the best of all that
// were left out (kNext); or all sixteen in t (DEPTH 16).
template <int DEPTH, bool kNext>
__device__ __forceinline__ void merge(double* t, const double c[8], double* next) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DEPTH == 16) t[15 - i] = __builtin_fmin(t[i], c[7 - i]);
    if constexpr (kNext) *next = __builtin_fmax(*next, __builtin_fmin(t[i], c[7 - i]));
    t[i] = __builtin_fmax(t[i], c[7 - i]);
  }
  bitonic8(t);
  if constexpr (DEPTH == 16) bitonic8(t + 8);
}

// ---------------------------------------------------------- close scores
// Exact scores: what orders two experts whose 32-bit scores lie within their rounding.
template <class T, int G, int BY>
struct Exact {
  const T* row;
  const float* bias;
  double top, sum;
  __device__ __forceinline__ void init(const T* r, const float* b, int E, int gl) {
    row = r;
    bias = b;
    if (BY == kSoftmaxBias) {
      float m = -INFINITY;
      for (int e = gl; e < E; e += G) m = __builtin_fmaxf(m, to_float<T>(row[e]));
      top = (double)finite_or_zero(group_maxf<G>(m));
      double s = 0.0;
      for (int e = gl; e < E; e += G) s += exp((double)to_float<T>(row[e]) - top);
      s = group_sum<G>(s);
      sum = s == 0.0 ? 1.0 : s;
    }
  }
  __device__ __forceinline__ double score(int e) const {
    const float l = to_float<T>(row[e]);
    if (l == -INFINITY) return -INFINITY;
    const double x = (double)l;
    const double b = (double)bias[e];
    const double s = (BY == kSoftmaxBias ? exp(x - top) / sum : 1.0 / (1.0 + exp(-x))) + b;
    if (x != x || b != b) return INFINITY;              // before all finite ones and +inf
    return fmin(s == s ? s : x, 0x1.fffffffffffffp+1023);
  }
};

// Lane gl holds candidate gl of `n` (every expert that can be among the first
// K, in the order of the 32-bit scores); returns the expert of rank gl.
template <class T, int G, int BY>
__device__ __forceinline__ int rank_candidates(const Exact<T, G, BY>& ex, int id, int n, int gl) {
  const int base = (threadIdx.x & 63) - gl;
  const double mine = gl < n ? ex.score(id) : -INFINITY;
  int rank = 0;
  for (int t = 0; t < n; ++t) {
    const double s = __shfl(mine, base + t, 64);
    const int e = __shfl(id, base + t, 64);
    rank += s > mine || (s == mine && e < id) ? 1 : 0;
  }
  if (gl >= n) rank = gl;                              // n .. G - 1: out of the way
  return __builtin_amdgcn_ds_permute((base + rank) * 4, id);
}

// The whole choice by exact scores, for a row with more candidates than lanes.
template <class T, int G, int BY, int kSel>
__device__ __forceinline__ void choose_exact(const Exact<T, G, BY>& ex, int E, int K, int gl,
                                             int sel[kSel]) {
  double last = INFINITY;
  int last_e = -1;                                     // the one taken before
  for (int k = 0; k < K; ++k) {
    double best = -INFINITY;
    int at = E;
    for (int e = gl; e < E; e += G) {
      const double s = ex.score(e);
      const bool open = s < last || (s == last && e > last_e);
      if (open && (s > best || at == E)) {
        best = s;
        at = e;
      }
    }
#pragma unroll
    for (int o = 1; o < G; o <<= 1) {
      const double b = __shfl_xor(best, o, 64);
      const int i = __shfl_xor(at, o, 64);
      if (i < E && (at == E || b > best || (b == best && i < at))) {
        best = b;
        at = i;
      }
    }
    last = best;
    last_e = at;
#pragma unroll
    for (int q = 0; q < kSel; ++q)
      if (k == q * G + gl) sel[q] = at;
  }
}

// ---------------------------------------------------------------- forward
// A lane's list keeps DEPTH keys: all of its own, or 8 >= K of them and, with
// a bias, the next one.
template <class T, int G, int VPL, int DEPTH, int BY, bool kSigmoid>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
  constexpr bool kShort = VPL > DEPTH;                  // K <= 8
  constexpr int kMaxSel = kShort ? 8 : 32;
  constexpr int kSel = G < kMaxSel ? kMaxSel / G : 1;   // chosen experts a lane keeps
  constexpr bool kNext = kShort && BY != kLogits;
  const int lane = threadIdx.x & 63, gl = lane % G;
  const int64_t row = ((int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6)) * (64 / G) + lane / G;
  if (row >= a.T) return;                               // whole groups
  const T* lrow = (const T*)a.logits + row * a.E;
  float l[VPL];
  load_row<T, G, VPL>(lrow, a.E, gl, a.wide, l);
  float top = 0.0f, inv = 0.0f;
  if (BY == kSoftmaxBias || (!kSigmoid && !a.normalize)) softmax_row<G, VPL>(l, &top, &inv);

  // asked of the wave first: one branch past the replacement, which hardly any wave needs, in
  // place of a compare per logit (32768 rows of 256 fp32: 19.3 us, with the compare 20.4 us)
  const bool no_scores = BY == kSoftmaxBias && __any(inv != inv) && inv != inv;

  double t[DEPTH], next = no_key();
#pragma unroll
  for (int c = 0; c < VPL; c += 8) {
    double k[8];
    float b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (BY != kLogits && a.bias_wide) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const int e = element_of<T, G>(gl, c + i);
        if (e < a.E) {
          const Vec<float> v = *(const Vec<float>*)(a.bias + e);
#pragma unroll
          for (int q = 0; q < 4; ++q) b[i + q] = v.v[q];
        }
      }
    } else if (BY != kLogits) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = element_of<T, G>(gl, c + i);
        if (e < a.E) b[i] = a.bias[e];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = l[c + i];
      // The hardware's exponential and reciprocal (their rounding: see below).  A closed expert
      // keeps its -inf.  A NaN in the bias comes first, as one in the logit does.  A softmax with a
      // NaN or +inf has no scores: its logits order instead.
      if (BY == kSigmoidBias) {
        s = __builtin_amdgcn_rcpf(1.0f + __expf(-s)) + b[i];
        s = l[c + i] == -INFINITY ? -INFINITY : s;
      } else if (BY == kSoftmaxBias) {
        s = __expf(s - top) * inv + b[i];
        s = l[c + i] == -INFINITY ? l[c + i] : s;
        if (no_scores && b[i] == b[i]) s = l[c + i];
      }
      k[i] = key_of(s + 0.0f, element_of<T, G>(gl, c + i));          // -0 as +0
    }
    sort8(k);
    if (c == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = k[i];
    } else {
      merge<DEPTH, kNext>(t, k, &next);
    }
  }

  int sel[kSel];
#pragma unroll
  for (int q = 0; q < kSel; ++q) sel[q] = 0;
  // Draw k: the largest head of the group's lists, kept by lane k % G and taken off its list.
  auto draw = [&](int k, int deep) {
    const double m = group_max<G>(t[0]);
#pragma unroll
    for (int q = 0; q < kSel; ++q)
      if (k == q * G + gl) sel[q] = key_low(m);
    if (t[0] == m) {
#pragma unroll
      for (int j = 0; j + 1 < DEPTH; ++j)
        if (j < deep) t[j] = t[j + 1];
      if (deep >= DEPTH) {
        t[DEPTH - 1] = kNext ? next : no_key();
        if (kNext) next = no_key();
      }
    }
    return m;
  };
  if constexpr (BY == kLogits && kShort) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < a.K) draw(k, 7 - k);                      // a list still has 7 - k draws before it
  } else if constexpr (BY == kLogits) {
    for (int k = 0; k < a.K; ++k) draw(k, DEPTH);
  }
  if constexpr (BY != kLogits) {
    // With a bias the draw goes on past K, up to G experts, while the scores
    // stay within their rounding of the K-th, 32 units of 2^-24 for two scores together.
    // A sigmoid is off by 2 units for the hardware's exponential and under 1 for its
    // argument (|x| 2^-23 relative, where x e^-x < 0.4), 1 for the sum and 2 for the
    // reciprocal.  A softmax's score likewise by 2 and 1 and 1 for the product, but two of them
    // are at most 1 together; the sum, which scales both, by 13 for its additions, 2 and under
    // 4 for its exponentials (the mean of |x| times the score is below 1.8 for 1024
    // experts) and 1 for its inverse: 24 in all.  The sum with the bias is rounded once more.
    const int limit = a.K + 1 > a.E ? a.E : a.K < G ? (G < a.E ? G : a.E) : a.K + 1;
    int n = a.K;                                        // candidates
    bool close = false, more = true;
    float prev = INFINITY;
    const auto take = [&](int k, int deep) {            // false: no further draw is needed
      const float v = key_value(draw(k, deep));
      const bool apart = prev - v > 0x1p-19f + 0x1p-22f * fabsf(prev);
      if (k < a.K) {
        if (k > 0 && !apart) close = true;
        prev = v;
        return true;
      }
      more = more && !apart;
      if (more) n = k + 1;
      return (bool)__any(more);
    };
    if constexpr (kShort) {
      // Ten draws at most, so only the 9 - k first keys of a list matter behind draw k.  The
      // first nine find every list whole (next is its ninth key); the tenth, which says whether
      // nine candidates are all, does unless one list gave those nine.
      bool on = true, empty = false;
#pragma unroll
      for (int k = 0; k < 10; ++k)
        if (on) {
          if (k == 9) empty = __ballot(t[0] == no_key()) >> (lane - gl) & ((1ull << G) - 1);
          on = take(k, 9 - k);
        }
      if (more || (empty && n == 9)) n = G + 1;
    } else {
      for (int k = 0; k < limit; ++k)
        if (!take(k, DEPTH)) break;
    }
#pragma unroll
    for (int q = 0; q < kSel; ++q) sel[q] = expert_of(sel[q]);
    if (close || n > a.K) {
      Exact<T, G, BY> ex;
      ex.init(lrow, a.bias, a.E, gl);
      const bool whole = n < G || (n == G && n == a.E);
      if (whole) sel[0] = rank_candidates<T, G, BY>(ex, sel[0], n, gl);
      else choose_exact<T, G, BY, kSel>(ex, a.E, a.K, gl, sel);
    }
  } else {
#pragma unroll
    for (int q = 0; q < kSel; ++q) sel[q] = expert_of(sel[q]);
  }

  // weights: lane gl holds the chosen experts gl, gl + G, ...
  float w[kSel], mx = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    w[q] = q * G + gl < a.K ? to_float<T>(lrow[sel[q]]) : -INFINITY;
    mx = __builtin_fmaxf(mx, w[q]);
  }
  if (!kSigmoid) mx = a.normalize ? finite_or_zero(group_maxf<G>(mx)) : top;
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    w[q] = kSigmoid ? sigmoid(w[q]) : expf(w[q] - mx);
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

// --------------------------------------------------------------- backward
// A wave's own LDS operations complete in order; only the compiler must not
// move them across this point.
__device__ __forceinline__ void lds_settled() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The chosen experts' gradients are scattered into a row of LDS (zeros
// elsewhere), from which the G lanes write the whole row.
template <class T, int G, int VPL, bool kSigmoid>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(RouteArgs a) {
  constexpr int kSel = G < 32 ? 32 / G : 1, N = 16 / (int)sizeof(T);
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  __shared__ __attribute__((aligned(16))) float rows[kWaves * 64 * VPL];
  const int lane = threadIdx.x & 63, gl = lane % G, wv = threadIdx.x >> 6;
  const int64_t row = ((int64_t)blockIdx.x * kWaves + wv) * (64 / G) + lane / G;
  if (row >= a.T) return;
  const T* lrow = (const T*)a.logits + row * a.E;
  float* lds = rows + (wv * (64 / G) + lane / G) * (G * VPL);
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < VPL; i += 4) *(f32x4*)(lds + 4 * (gl + G * (i / 4))) = zero;
  lds_settled();

  const bool dense = !kSigmoid && !a.normalize;
  int id[kSel];
  float x[kSel], g[kSel];
  float mx = -INFINITY;
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    const int k = q * G + gl;
    id[q] = k < a.K ? a.topk[row * a.K + k] : -1;
    if ((unsigned)id[q] >= (unsigned)a.E) id[q] = -1;   // never out of the row
    g[q] = id[q] < 0 ? 0.0f : a.drw[row * a.K + k] * a.scale;
    x[q] = id[q] < 0 ? -INFINITY : to_float<T>(lrow[id[q]]);
    mx = __builtin_fmaxf(mx, x[q]);
  }
  float l[VPL];
  float top = 0.0f, inv = 1.0f;
  if (dense) {
    load_row<T, G, VPL>(lrow, a.E, gl, a.wide, l);
    softmax_row<G, VPL, true>(l, &top, &inv);
  } else if (!kSigmoid) {
    top = finite_or_zero(group_maxf<G>(mx));
  }
  float p[kSel], t = 0.0f;
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    p[q] = id[q] < 0 ? 0.0f : kSigmoid ? sigmoid(x[q]) : expf(x[q] - top);
    t += p[q];
  }
  if (a.normalize) inv = inv_or_zero(group_sum<G>(t));
  float gq = 0.0f;                                      // sum_j g_j q_j / t, or sum_j g_j q_j
  if (a.normalize || dense) {
#pragma unroll
    for (int q = 0; q < kSel; ++q) gq += g[q] * (p[q] * inv);
    gq = group_sum<G>(gq);
  }
#pragma unroll
  for (int q = 0; q < kSel; ++q) {
    float d = g[q];
    // the quotient first: it is at most 1, while the inverse of a sum of low sigmoids nears 2^128
    if (!dense) d = (d - gq) * (p[q] * inv);
    if (kSigmoid) d *= sigmoid(-x[q]);
    if (id[q] >= 0) lds[id[q]] = d;
  }
  lds_settled();
  T* out = (T*)a.dlogits + row * a.E;
  float d[VPL];
#pragma unroll
  for (int i = 0; i < VPL; i += 4) {
    const f32x4 v = *(const f32x4*)(lds + element_of<T, G>(gl, i));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      d[i + e] = v[e];
      if (dense) d[i + e] = l[i + e] * inv * (v[e] - gq);
    }
  }
  if (a.wide) {
#pragma unroll
    for (int j = 0; j < VPL / N; ++j) {
      Vec<T> r;
#pragma unroll
      for (int i = 0; i < N; ++i) r.v[i] = from_float<T>(d[j * N + i]);
      if (N * (gl + G * j) < a.E) *(Vec<T>*)(out + N * (gl + G * j)) = r;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (element_of<T, G>(gl, i) < a.E) out[element_of<T, G>(gl, i)] = from_float<T>(d[i]);
  }
}

// ------------------------------------------------------------------- host
template <class T, int G, int VPL, int DEPTH>
void run_route(const RouteArgs& a, const RouteForm& f, hipStream_t s) {
  const unsigned per = kWaves * (64 / G);
  const unsigned blocks = (unsigned)(((int64_t)a.T + per - 1) / per);
  const bool sig = f.score == MOONEP_SCORE_SIGMOID;
  if (!a.bias) {
    if (sig) route_kernel<T, G, VPL, DEPTH, kLogits, true><<<blocks, kThreads, 0, s>>>(a);
    else route_kernel<T, G, VPL, DEPTH, kLogits, false><<<blocks, kThreads, 0, s>>>(a);
  } else if (sig) {
    route_kernel<T, G, VPL, DEPTH, kSigmoidBias, true><<<blocks, kThreads, 0, s>>>(a);
  } else {
    route_kernel<T, G, VPL, DEPTH, kSoftmaxBias, false><<<blocks, kThreads, 0, s>>>(a);
  }
}

template <class T, int G, int VPL>
void run_route_bwd(const RouteArgs& a, const RouteForm& f, hipStream_t s) {
  const unsigned per = kWaves * (64 / G);
  const unsigned blocks = (unsigned)(((int64_t)a.T + per - 1) / per);
  if (f.score == MOONEP_SCORE_SIGMOID)
    route_bwd_kernel<T, G, VPL, true><<<blocks, kThreads, 0, s>>>(a);
  else
    route_bwd_kernel<T, G, VPL, false><<<blocks, kThreads, 0, s>>>(a);
}

// Lanes and logits per lane for E experts: few lanes with long lists, so that
// a wave's draws serve several rows; a list of eight is enough up to K = 8,
// above that a lane keeps all of its keys.
template <class T>
hipError_t route_by_size(const RouteArgs& a, const RouteForm& f, hipStream_t s) {
  if (a.E <= 64) run_route<T, 8, 8, 8>(a, f, s);
  else if (a.E <= 128) run_route<T, 16, 8, 8>(a, f, s);
  else if (a.K <= 8 && a.E <= 256) run_route<T, 16, 16, 8>(a, f, s);
  else if (a.K <= 8 && a.E <= 384) run_route<T, 16, 24, 8>(a, f, s);
  else if (a.K <= 8 && a.E <= 512) run_route<T, 16, 32, 8>(a, f, s);
  else if (a.E <= 512) run_route<T, 64, 8, 8>(a, f, s);
  else run_route<T, 64, 16, 16>(a, f, s);
  return hipGetLastError();
}

template <class T>
hipError_t route_bwd_by_size(const RouteArgs& a, const RouteForm& f, hipStream_t s) {
  if (a.E <= 64) run_route_bwd<T, 8, 8>(a, f, s);
  else if (a.E <= 128) run_route_bwd<T, 16, 8>(a, f, s);
  else if (a.E <= 256) run_route_bwd<T, 16, 16>(a, f, s);
  else if (a.E <= 384) run_route_bwd<T, 16, 24>(a, f, s);
  else if (a.E <= 512) run_route_bwd<T, 16, 32>(a, f, s);
  else run_route_bwd<T, 64, 16>(a, f, s);
  return hipGetLastError();
}

RouteArgs route_args(const Ctx& c, const RouteForm& f, const void* logits, const void* dlogits) {
  RouteArgs a;
  a.logits = logits; a.bias = nullptr; a.topk = nullptr; a.rw = nullptr;
  a.drw = nullptr; a.dlogits = const_cast<void*>(dlogits);
  a.scale = f.scale;
  a.T = c.d.R * c.d.S; a.E = c.d.E; a.K = c.d.K; a.normalize = f.normalize;
  a.bias_wide = 0;
  a.wide = a.E % (f.dtype == MOONEP_F32 ? 4 : 8) == 0 && (uintptr_t)logits % 16 == 0 &&
           (uintptr_t)dlogits % 16 == 0;
  return a;
}

}  // namespace

hipError_t launch_route(const Ctx& c, const void* logits, const float* bias, const RouteForm& f,
                        int32_t* topk, float* rw, hipStream_t s) {
  RouteArgs a = route_args(c, f, logits, nullptr);
  a.bias = bias; a.topk = topk; a.rw = rw;
  a.bias_wide = a.E % 4 == 0 && (uintptr_t)bias % 16 == 0;
  return f.dtype == MOONEP_F32 ? route_by_size<float>(a, f, s) : route_by_size<uint16_t>(a, f, s);
}

hipError_t launch_route_bwd(const Ctx& c, const void* logits, const RouteForm& f,
                            const int32_t* topk, const float* drw, void* dlogits, hipStream_t s) {
  RouteArgs a = route_args(c, f, logits, dlogits);
  a.topk = const_cast<int32_t*>(topk); a.drw = drw;
  return f.dtype == MOONEP_F32 ? route_bwd_by_size<float>(a, f, s)
                               : route_bwd_by_size<uint16_t>(a, f, s);
}

}  // namespace moonep
