// The gate over experts in groups, from sigmoid or softmax scores, and its
// gradient.
//
// Forward, for a token's logits l [E] (an excluded expert has l = -inf):
//   s_e     = 1 / (1 + exp(-l_e)), or exp(l_e) / sum_m exp(l_m)
//   key_e   = s_e + bias_e, in 64 bits
//   the E experts are `groups` runs of E / groups; a group's score is the sum of
//   its two largest keys, and e_1..e_k are the experts with the largest keys of
//   the topk_groups groups with the largest scores (equal ones by lower index)
//   probs_j = scale * s_{e_j}, or with renorm scale * s_{e_j} / sum_m s_{e_m}
// Gradient, with d_j = scale * grad_probs_j and w_j = probs_j / scale:
//   sigmoid   d_j s_j (1 - s_j), with renorm w_j (1 - s_j) (d_j - sum_m d_m w_m)
//             at the picks
//   softmax   p_e (D_e - sum_j d_j p_{e_j}) with D_e = d_j at the pick e_j = e and
//             0 elsewhere, with renorm w_j (d_j - sum_m d_m w_m) at the picks
//
// A choice made on rounded keys depends on the rounding, as two of a few hundred
// scores lie within 2^-24 of each other in one of some thousand rows.  The keys
// are therefore computed as doubles (fp64 runs at the rate of unpacked fp32
// here), and the low 10 bits of a key (13 for more than 1024 experts) are
// replaced by the expert's index, so that one double orders by key and then by
// index: a comparison is one v_max_f64 and nothing has to travel with it.  Keys
// that agree in the remaining 42 (39) bits count as equal.
//
// A row belongs to 16, 32 or 64 neighbouring lanes, a lane holds EPL successive
// experts.  It sorts them once (63 exchanges of two instructions for 16), after
// which a pick is the maximum over the lanes' first entries, and the lane that
// owned it moves up by one: 30 instructions, against 75 for a search through
// all entries.
//
// Sums and maxima are added in a fixed order.
//
// Measured, 256 experts in 8 groups, 4 groups and 8 experts chosen, sigmoid with
// bias: 16 tokens, bf16, 5.2 us, a chain of dependent steps; 13824 tokens, fp32,
// 14.8 us, 1.05 TB/s, bound by the fp64 instructions of the keys and the sort (the
// library's exp instead of the one here: 18.7).  Gradient, 13824 tokens, bf16: 7 us,
// a launch and 13.8 MB.
#include "pgg_device.h"

namespace pgg {

namespace {

constexpr int kThreads = 256;
constexpr float kNegInf = -__builtin_inff();
constexpr int kMaxGroups = PGG_GATE_MAX_GROUPS;

// Keys outside the scores' range, all finite so that their low bits can hold an index
constexpr double kMostKey = 0x1p1000, kExcluded = -0x1p1000, kMissing = -0x1p1023;

struct GroupedArgs {
  const void* logits;   // [T, E]
  const float* bias;    // [E] or NULL
  int64_t* ids;         // [T, k]
  float* probs;         // [T, k]
  int64_t T;
  int32_t E, k, groups, topk_groups;
  int32_t softmax, renorm;
  float scale;
};

struct GroupedGradArgs {
  const void* logits;        // [T, E]
  const int64_t* ids;        // [T, k]
  const float* grad_probs;   // [T, k]
  void* grad_logits;         // [T, E]
  int64_t T;
  int32_t E, k;
  int32_t softmax, renorm;
  float scale;
};

// inline assembly: the compiler would first canonicalise operands that come from bit operations
__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

template <int N>
__device__ __forceinline__ uint32_t rotate16(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + N, 0xF, 0xF, false));
}

// The values that a lane and its partner N places on hold (N < 16: rotation
// within 16 lanes, the first being the lane's own; otherwise the lane N bits away,
// the lower lane's first).
template <int N>
__device__ __forceinline__ void partners(uint32_t v, uint32_t& a, uint32_t& b) {
  if constexpr (N < 16) {
    a = v;
    b = rotate16<N>(v);
  } else if constexpr (N == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  }
}
template <int N, class Op>
__device__ __forceinline__ float step(float v, Op op) {
  uint32_t a, b;
  partners<N>(__builtin_bit_cast(uint32_t, v), a, b);
  return op(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
template <int N, class Op>
__device__ __forceinline__ double step(double v, Op op) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  uint32_t a[2], b[2];
  partners<N>(static_cast<uint32_t>(u), a[0], b[0]);
  partners<N>(static_cast<uint32_t>(u >> 32), a[1], b[1]);
  return op(__builtin_bit_cast(double, static_cast<uint64_t>(a[1]) << 32 | a[0]),
            __builtin_bit_cast(double, static_cast<uint64_t>(b[1]) << 32 | b[0]));
}

// Reduction over the LPR lanes of a row; every lane gets the result.
template <int LPR, class V, class Op>
__device__ __forceinline__ V reduce(V v, Op op) {
  v = step<8>(v, op);
  v = step<4>(v, op);
  v = step<2>(v, op);
  v = step<1>(v, op);
  if constexpr (LPR >= 32) v = step<16>(v, op);
  if constexpr (LPR >= 64) v = step<32>(v, op);
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  return reduce<LPR>(v, [](float a, float b) { return a + b; });
}
template <int LPR>
__device__ __forceinline__ double row_sum(double v) {
  return reduce<LPR>(v, [](double a, double b) { return a + b; });
}
// Largest value; NaN where any is NaN.
__device__ __forceinline__ float max_nan(float a, float b) { return a != a || a > b ? a : b; }
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
  return reduce<LPR>(v, [](float a, float b) { return max_nan(a, b); });
}

// The largest logit, as softmax subtracts it: 0 for a row of -inf.
__device__ __forceinline__ float pivot(float m) { return m == kNegInf ? 0.0f : m; }

template <class T>
__device__ __forceinline__ void load4(const typename T::elem* row, int e, int E, float (&v)[4]) {
  typename T::elem x[4];
  if (e + 4 <= E) {
    __builtin_memcpy(x, row + e, sizeof(x));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_float<T>(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = e + i < E ? to_float<T>(row[e + i]) : kNegInf;
  }
}

// 1 / v for v >= 1, within an ulp: two Newton steps on the hardware's estimate.
__device__ __forceinline__ double reciprocal(double v) {
  double r = __builtin_amdgcn_rcp(v);
  r = __builtin_fma(__builtin_fma(-v, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-v, r, 1.0), r, r);
}

// exp(v) for v <= 0, to 2^-44 of itself, more than a key keeps (2^-46 down to v = -100):
// v = n ln 2 + r with |r| <= ln 2 / 2, the Taylor polynomial of degree 11 at r (the
// first term left out is 2^-47), times 2^n; ln 2 as one double is off by 2^-55, n
// times.  Below -800 as at -800, which is 0; NaN likewise.
__device__ __forceinline__ double exp_negative(double v) {
  v = max64(v, -800.0);
  const double n = __builtin_rint(v * 1.4426950408889634);
  const double r = __builtin_fma(n, -0.6931471805599453, v);
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, static_cast<int>(n));
}

__device__ __forceinline__ double sigmoid_score(float l) {
  const double x = l, q = exp_negative(-fabs(x));
  return (x >= 0.0 ? 1.0 : q) * reciprocal(1.0 + q);
}

// Key and index in one double; BITS of it are the index's.  A NaN comes out as the
// largest key, and so does a logit above `limit` or a NaN: softmax makes a NaN of +inf.
template <int BITS>
__device__ __forceinline__ double pack_key(double key, float l, float limit, int e) {
  const uint64_t u = __builtin_bit_cast(uint64_t, max64(min64(key, kMostKey), kExcluded));
  constexpr uint32_t mask = (1u << BITS) - 1;
  constexpr uint32_t most = __builtin_bit_cast(uint64_t, kMostKey) >> 32, least = most | 0x80000000u;
  // (the low words of both are only index)
  uint32_t hi = static_cast<uint32_t>(u >> 32), lo = static_cast<uint32_t>(u);
  const bool banned = l == kNegInf, first = !(l <= limit);
  hi = banned ? least : first ? most : hi;
  lo = banned || first ? 0u : lo;
  const uint32_t low = static_cast<uint32_t>(e ^ ~(static_cast<int32_t>(hi) >> 31));   // a lower index is larger
  lo = (lo & ~mask) | (low & mask);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
template <int BITS>
__device__ __forceinline__ int32_t packed_index(double v) {
  constexpr uint32_t mask = (1u << BITS) - 1;
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t low = static_cast<uint32_t>(u) & mask;
  return static_cast<int32_t>(static_cast<int64_t>(u) < 0 ? low : mask - low);
}
template <int BITS>
__device__ __forceinline__ double without_index(double v) {
  constexpr uint64_t mask = (uint64_t(1) << BITS) - 1;
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, v) & ~mask);
}

// A group's score from its two largest packed keys: an excluded expert adds
// nothing, a group of excluded experts comes last.
template <int BITS>
__device__ __forceinline__ double group_score(double first, double second) {
  const double a = without_index<BITS>(first), b = without_index<BITS>(second);
  return a <= kExcluded ? kExcluded : b <= kExcluded ? a : a + b;
}

// The two largest of what (a, b) with a >= b and a further v hold.
__device__ __forceinline__ void keep2(double& a, double& b, double v) {
  b = max64(b, min64(a, v));
  a = max64(a, v);
}

// Sorts descending (odd-even merges).
template <int N>
__device__ __forceinline__ void sort_descending(double (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const double a = v[i + j], b = v[i + j + k];
            v[i + j] = max64(a, b);
            v[i + j + k] = min64(a, b);
          }
}

// Drops the first entry where `own`; the first `DEPTH` entries stay right.
template <int DEPTH, int N>
__device__ __forceinline__ void pop(double (&v)[N], bool own) {
#pragma unroll
  for (int i = 0; i < (DEPTH < N ? DEPTH : N); ++i) {
    const double next = i + 1 < N ? v[i + 1] : kMissing;
    v[i] = own ? next : v[i];
  }
}

// LDS operations of a wave are done in order; only the compiler has to keep it.
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The k picks are kept LPR to a register: pick j by lane j % LPR.
template <int LPR>
constexpr int kPickRegs = (PGG_GATE_MAX_TOPK + LPR - 1) / LPR;

__device__ __forceinline__ float sigmoid_exact(float l) {
  const float q = expf(-fabsf(l));
  return (l >= 0.0f ? 1.0f : q) / (1.0f + q);
}

// Weights before the scale, of k picks with the logits l (-inf: no pick or an
// excluded one, weight 0).  top / total: the row's pivot and sum of exp (softmax
// without renorm).
template <int LPR>
__device__ __forceinline__ void weights(int k, bool softmax, bool renorm, float top, float total,
                                        const float (&l)[kPickRegs<LPR>], float (&w)[kPickRegs<LPR>]) {
  constexpr int R = kPickRegs<LPR>;
  if (!renorm) {
#pragma unroll
    for (int s = 0; s < R; ++s)
      if (s * LPR < k) {
        if (softmax) {
          const float e = expf(l[s] - top);
          w[s] = total == 0.0f ? e : e / total;
        } else {
          w[s] = sigmoid_exact(l[s]);
        }
      }
    return;
  }
  float m = l[0];
#pragma unroll
  for (int s = 1; s < R; ++s) m = max_nan(l[s], m);
  top = pivot(row_max<LPR>(m));
  // sigmoid scores share the factor exp(min(top, 0)), which is left out: they
  // may all be too small for fp32, their ratios are not
  if (!softmax) top = top > 0.0f ? 0.0f : top;
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < R; ++s)
    if (s * LPR < k) {
      if (softmax) w[s] = expf(l[s] - top);
      else w[s] = l[s] >= 0.0f ? 1.0f / (1.0f + expf(-l[s])) : expf(l[s] - top) / (1.0f + expf(l[s]));
      sum += w[s];
    }
  sum = row_sum<LPR>(sum);
#pragma unroll
  for (int s = 0; s < R; ++s)
    if (s * LPR < k) w[s] = sum == 0.0f ? w[s] : w[s] / sum;
}

template <class T, int LPR>
__device__ __forceinline__ void store_picks(const GroupedArgs& a, const typename T::elem* row, int64_t t, int lane,
                                            bool live, const int32_t (&sel)[kPickRegs<LPR>], float top, float total) {
  constexpr int R = kPickRegs<LPR>;
  float l[R], w[R];
#pragma unroll
  for (int s = 0; s < R; ++s) l[s] = s * LPR + lane < a.k ? to_float<T>(row[sel[s]]) : kNegInf;
  weights<LPR>(a.k, a.softmax, a.renorm, top, total, l, w);
#pragma unroll
  for (int s = 0; s < R; ++s) {
    const int j = s * LPR + lane;
    if (live && j < a.k) {
      a.ids[t * a.k + j] = sel[s];
      a.probs[t * a.k + j] = w[s] * a.scale;
    }
  }
}

// E <= LPR * EPL <= 1024: lane c of a row holds the experts from EPL c on.
template <class T, int LPR, int EPL>
__global__ __launch_bounds__(kThreads) void grouped_gate_kernel(GroupedArgs a) {
  using E = typename T::elem;
  constexpr int BITS = 10, kRows = kThreads / LPR;
  extern __shared__ double scratch[];   // groups that end inside a lane: the rows' keys
  __shared__ double s_two[kRows][LPR][2];
  __shared__ double s_score[kRows][kMaxGroups];
  __shared__ uint8_t s_open[kRows][kMaxGroups];
  const int lane = threadIdx.x % LPR, r = threadIdx.x / LPR;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + r;
  // rows past the end repeat the last one (whole waves stay together) and store nothing
  const bool live = t < a.T;
  const int64_t tr = live ? t : a.T - 1;
  const E* __restrict__ row = static_cast<const E*>(a.logits) + tr * a.E;
  const int e0 = lane * EPL;
  float l[EPL];
#pragma unroll
  for (int i = 0; i < EPL; i += 4) load4<T>(row, e0 + i, a.E, *reinterpret_cast<float(*)[4]>(&l[i]));
  float top = 0.0f;
  double total = 1.0, key[EPL];
  const float limit = a.softmax ? 3.402823466e38f : -kNegInf;
  if (a.softmax) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = max_nan(l[i], m);
    top = pivot(row_max<LPR>(m));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      key[i] = exp_negative(static_cast<double>(l[i]) - static_cast<double>(top));
      sum += key[i];
    }
    total = row_sum<LPR>(sum);
    const double norm = reciprocal(max64(total, 1.0));   // at least 1 but for a row of -inf
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] *= norm;
    if (top != top || top == -kNegInf) total = __builtin_nan("");   // a NaN or +inf logit: exp_negative takes neither
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = sigmoid_score(l[i]);
  }
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
      float b[4];
      load4<TF32>(a.bias, e0 + i, a.E, b);
#pragma unroll
      for (int q = 0; q < 4; ++q) key[i + q] += static_cast<double>(b[q]);
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = pack_key<BITS>(key[i], l[i], limit, e0 + i);
  if (e0 + EPL > a.E) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e0 + i >= a.E) key[i] = kMissing;
  }
  const int each = a.E / a.groups;
  const bool whole = each % EPL == 0;   // a lane's experts are of one group
  if (a.groups > 1 && !whole) {
    double* keys = scratch + static_cast<size_t>(r) * a.E;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e0 + i < a.E) keys[e0 + i] = key[i];
    wave_fence();
    for (int g = lane; g < a.groups; g += LPR) {
      double first = kMissing, second = kMissing;
      for (int i = 0; i < each; ++i) keep2(first, second, keys[g * each + i]);
      s_score[r][g] = group_score<BITS>(first, second);
    }
  }
  sort_descending(key);
  if (a.groups > 1) {
    if (whole) {
      s_two[r][lane][0] = key[0];
      s_two[r][lane][1] = key[EPL > 1 ? 1 : 0];
      wave_fence();
      const int span = each / EPL;   // lanes of a group; there are at most LPR groups
      if (lane < a.groups) {
        double first = kMissing, second = kMissing;
        for (int i = 0; i < span; ++i) {
          keep2(first, second, s_two[r][lane * span + i][0]);
          keep2(first, second, s_two[r][lane * span + i][1]);
        }
        s_score[r][lane] = group_score<BITS>(first, second);
      }
    }
    wave_fence();
    for (int g = lane; g < a.groups; g += LPR) {
      const double mine = s_score[r][g];
      int before = 0;
#pragma unroll 4
      for (int o = 0; o < a.groups; ++o) {
        const double other = s_score[r][o];
        before += other > mine || (other == mine && o < g);
      }
      s_open[r][g] = before < a.topk_groups;
    }
    wave_fence();
    if (whole) {
      const int g = min(e0 / each, a.groups - 1);
      if (!s_open[r][g]) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = kMissing;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (key[i] > kMissing && !s_open[r][packed_index<BITS>(key[i]) / each]) key[i] = kMissing;
      sort_descending(key);
    }
  }

  int32_t sel[kPickRegs<LPR>];
#pragma unroll
  for (int s = 0; s < kPickRegs<LPR>; ++s) {
    sel[s] = 0;
    for (int j = 0; j < min(LPR, a.k - s * LPR); ++j) {
      const double best = reduce<LPR>(key[0], [](double x, double y) { return max64(x, y); });
      const bool own = key[0] == best;
      if (EPL > 8 && a.k > 8) pop<EPL>(key, own);
      else pop<8>(key, own);
      if (lane == j) sel[s] = packed_index<BITS>(best);
    }
  }
  store_picks<T, LPR>(a, row, tr, lane, live, sel, top, static_cast<float>(total));
}

// Any E up to 8192: one wave, a workgroup of its own, per row; the keys in LDS.
// Every pick looks through them again.
template <class T>
__global__ __launch_bounds__(64) void grouped_gate_long_kernel(GroupedArgs a) {
  using E = typename T::elem;
  constexpr int LPR = 64, BITS = 13;
  extern __shared__ double scratch[];
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const E* __restrict__ row = static_cast<const E*>(a.logits) + t * a.E;
  float top = 0.0f;
  double total = 1.0;
  const float limit = a.softmax ? 3.402823466e38f : -kNegInf;
  if (a.softmax) {
    float m = kNegInf;
    for (int e = lane; e < a.E; e += LPR) m = max_nan(to_float<T>(row[e]), m);
    top = pivot(row_max<LPR>(m));
    double sum = 0.0;
    for (int e = lane; e < a.E; e += LPR)
      sum += exp_negative(static_cast<double>(to_float<T>(row[e])) - static_cast<double>(top));
    total = row_sum<LPR>(sum);
  }
  const double norm = reciprocal(max64(total, 1.0));
  if (top != top || top == -kNegInf) total = __builtin_nan("");
  for (int e = lane; e < a.E; e += LPR) {
    const float l = to_float<T>(row[e]);
    double v = a.softmax ? exp_negative(static_cast<double>(l) - static_cast<double>(top)) * norm : sigmoid_score(l);
    if (a.bias) v += static_cast<double>(a.bias[e]);
    scratch[e] = pack_key<BITS>(v, l, limit, e);
  }
  wave_fence();
  if (a.groups > 1) {
    const int each = a.E / a.groups;
    double mine = kMissing;   // the score of group `lane`
    for (int g = 0; g < a.groups; ++g) {
      double first = kMissing, second = kMissing;
      for (int i = lane; i < each; i += LPR) keep2(first, second, scratch[g * each + i]);
#pragma unroll
      for (int d = 32; d >= 1; d /= 2) {
        const double f = __shfl_xor(first, d), s = __shfl_xor(second, d);
        keep2(first, second, f);
        keep2(first, second, s);
      }
      const double v = group_score<BITS>(first, second);
      if (lane == g) mine = v;
    }
    int before = 0;
    for (int o = 0; o < a.groups; ++o) {
      const double other = __shfl(mine, o);
      before += other > mine || (other == mine && o < lane);
    }
    const uint64_t open = __ballot(lane < a.groups && before < a.topk_groups);
    for (int g = 0; g < a.groups; ++g)
      if (!(open >> g & 1))
        for (int i = lane; i < each; i += LPR) scratch[g * each + i] = kMissing;
    wave_fence();
  }
  int32_t sel = 0;   // topk <= 64: one pick to a lane
  double last = __builtin_inf();
  for (int j = 0; j < a.k; ++j) {
    double best = kMissing;
    for (int e = lane; e < a.E; e += LPR) {
      const double v = scratch[e];
      best = v < last ? max64(best, v) : best;
    }
    last = reduce<LPR>(best, [](double x, double y) { return max64(x, y); });
    if (lane == j) sel = packed_index<BITS>(last);
  }
  const int32_t one[1] = {sel};
  store_picks<T, LPR>(a, row, t, lane, true, one, top, static_cast<float>(total));
}

// LPR lanes per row, rows of one wave only; E floats of LDS per row, which hold
// the picks' values and kUnpicked elsewhere.
constexpr uint32_t kUnpicked = 0x7FC0DEADu;   // a NaN; a value that is one is stored as another

template <class T, int LPR, int THREADS>
__global__ __launch_bounds__(THREADS) void grouped_gate_grad_kernel(GroupedGradArgs a) {
  using E = typename T::elem;
  constexpr int R = kPickRegs<LPR>;
  extern __shared__ uint32_t picked_rows[];
  const int lane = threadIdx.x % LPR;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (THREADS / LPR) + threadIdx.x / LPR;
  const bool live = t < a.T;
  const int64_t tr = live ? t : a.T - 1;   // whole waves stay together
  const E* __restrict__ row = static_cast<const E*>(a.logits) + tr * a.E;
  uint32_t* picked = picked_rows + threadIdx.x / LPR * a.E;
  // this lane's picks; an id outside the experts selects nothing
  int32_t id[R];
  float d[R], l[R], w[R];
#pragma unroll
  for (int s = 0; s < R; ++s) {
    const int j = s * LPR + lane;
    const int64_t e = j < a.k ? a.ids[tr * a.k + j] : -1;
    id[s] = static_cast<uint64_t>(e) < static_cast<uint64_t>(a.E) ? static_cast<int32_t>(e) : -1;
    d[s] = id[s] >= 0 ? a.grad_probs[tr * a.k + j] * a.scale : 0.0f;
    l[s] = id[s] >= 0 ? to_float<T>(row[id[s]]) : kNegInf;
  }
  for (int e = lane; e < a.E; e += LPR) picked[e] = kUnpicked;
  const bool dense = a.softmax && !a.renorm;   // every expert has a gradient
  float top = 0.0f, total = 1.0f;
  if (dense) {
    float m = kNegInf;
    for (int e = 4 * lane; e < a.E; e += 4 * LPR) {
      float x[4];
      load4<T>(row, e, a.E, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max_nan(x[i], m);
    }
    top = pivot(row_max<LPR>(m));
    float sum = 0.0f;
    for (int e = 4 * lane; e < a.E; e += 4 * LPR) {
      float x[4];
      load4<T>(row, e, a.E, x);
      sum += (expf(x[0] - top) + expf(x[1] - top)) + (expf(x[2] - top) + expf(x[3] - top));
    }
    total = row_sum<LPR>(sum);
  }
  weights<LPR>(a.k, a.softmax, a.renorm, top, total, l, w);
  float mean = 0.0f;   // sum_j d_j w_j
  if (dense || a.renorm) {
#pragma unroll
    for (int s = 0; s < R; ++s)
      if (s * LPR < a.k && id[s] >= 0) mean += d[s] * w[s];
    mean = row_sum<LPR>(mean);
  }
  wave_fence();
#pragma unroll
  for (int s = 0; s < R; ++s)
    if (s * LPR < a.k && id[s] >= 0) {
      float v = d[s];
      if (!dense) {
        v = w[s] * (v - mean);
        if (!a.softmax) v *= sigmoid_exact(-l[s]);
      }
      picked[id[s]] = v == v ? __builtin_bit_cast(uint32_t, v) : 0x7FC00000u;
    }
  wave_fence();
  if (!live) return;
  const float inv = total == 0.0f ? 1.0f : 1.0f / total;
  E* out = static_cast<E*>(a.grad_logits) + t * a.E;
  for (int e0 = 4 * lane; e0 < a.E; e0 += 4 * LPR) {
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (dense) load4<T>(row, e0, a.E, x);
    E g[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = e0 + i < a.E ? picked[e0 + i] : kUnpicked;
      const float v = u != kUnpicked ? __builtin_bit_cast(float, u) : 0.0f;
      g[i] = from_float<T>(dense ? expf(x[i] - top) * inv * (v - mean) : v);
    }
    if (e0 + 4 <= a.E) {
      __builtin_memcpy(out + e0, g, sizeof(g));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i < a.E) out[e0 + i] = g[i];
    }
  }
}

dim3 rows_grid(int64_t T, int per) { return dim3(static_cast<unsigned>((T + per - 1) / per)); }

template <class T, int LPR, int EPL>
hipError_t launch_rows(const GroupedArgs& a, hipStream_t s) {
  constexpr int kRows = kThreads / LPR;
  const bool whole = a.E / a.groups % EPL == 0;
  const size_t lds = a.groups > 1 && !whole ? sizeof(double) * kRows * static_cast<size_t>(a.E) : 0;
  hipLaunchKernelGGL((grouped_gate_kernel<T, LPR, EPL>), rows_grid(a.T, kRows), dim3(kThreads), lds, s, a);
  return hipGetLastError();
}

// Few tokens: more lanes to a row, so that the work and the code of a wave are
// shorter.  Groups of experts that end inside a lane's run of EPL take a way
// through LDS and a second sort, so shorter runs that end with them are taken
// instead.  Measured in us (a launch in a row of launches, bf16, 8 groups, 8
// picks), 64 lanes of 4, 32 of 8 and 16 of 16:
//   256 experts: 1024 tokens 5.5, 5.9, 7.9; 2048 6.3, 5.9, 7.9; 4096 8.3, 7.0, 8.1
//   160 experts (20 to a group): 1024 5.2, 8.0, 12.2; 4096 7.7, 9.1, 12.3; 13824 18.5, 19.0, 20.1
//   512 experts, 64 lanes of 8 and 32 of 16: 2048 7.6, 8.2; 4096 10.9, 10.0; 13824 28.0, 23.3
//   128 experts, 32 lanes of 4 and 16 of 8: 4096 5.9, 6.2; 13824 11.4, 10.8
template <class T>
hipError_t launch_typed(const GroupedArgs& a, hipStream_t s) {
  const int each = a.E / a.groups;
  auto split = [&](int run) { return a.groups > 1 && each % run != 0 && each % (run / 2) == 0; };
  if (a.E <= 64) return launch_rows<T, 16, 4>(a, s);
  if (a.E <= 128) return a.T <= 4096 || split(8) ? launch_rows<T, 32, 4>(a, s) : launch_rows<T, 16, 8>(a, s);
  if (a.E <= 256) return a.T <= 1024 || split(8) ? launch_rows<T, 64, 4>(a, s) : launch_rows<T, 32, 8>(a, s);
  if (a.E <= 512) return a.T <= 2048 || split(16) ? launch_rows<T, 64, 8>(a, s) : launch_rows<T, 32, 16>(a, s);
  if (a.E <= 1024) return launch_rows<T, 64, 16>(a, s);
  hipLaunchKernelGGL((grouped_gate_long_kernel<T>), rows_grid(a.T, 1), dim3(64), sizeof(double) * a.E, s, a);
  return hipGetLastError();
}

template <class T, int LPR, int THREADS>
hipError_t launch_grad_rows(const GroupedGradArgs& a, hipStream_t s) {
  const size_t lds = sizeof(uint32_t) * (THREADS / LPR) * static_cast<size_t>(a.E);
  hipLaunchKernelGGL((grouped_gate_grad_kernel<T, LPR, THREADS>), rows_grid(a.T, THREADS / LPR), dim3(THREADS), lds,
                     s, a);
  return hipGetLastError();
}

// LDS: 32 KiB at most per workgroup, 16 with many rows, but one row always fits.
// Few rows: more lanes to a row.  Measured in us as above, 16, 32 and 64 lanes:
//   256 experts: 2048 tokens 5.3, 4.0, 3.7; 4096 5.4, 4.3, 4.4; 13824 7.4, 6.7, 8.6
//   512 experts: 4096 -, 5.4, 5.1; 13824 -, 8.9, 10.4;  64 experts: 2048 3.9, 3.5, -; 13824 5.4, 5.4, -
template <class T>
hipError_t launch_grad_typed(const GroupedGradArgs& a, hipStream_t s) {
  if (a.E <= 128 || (a.E <= 512 && a.T > 4096)) return launch_grad_rows<T, 32, 256>(a, s);
  if (a.E <= 1024) return launch_grad_rows<T, 64, 256>(a, s);
  return launch_grad_rows<T, 64, 64>(a, s);
}

}  // namespace

hipError_t launch_gate_grouped(const pgg_moe_gate_grouped_desc& d, const void* logits, const float* bias, int64_t* ids,
                               float* probs, hipStream_t s) {
  const GroupedArgs a = {logits, bias, ids, probs, d.tokens, static_cast<int32_t>(d.experts),
                         static_cast<int32_t>(d.topk), static_cast<int32_t>(d.groups),
                         static_cast<int32_t>(d.topk_groups), d.score == PGG_SCORE_SOFTMAX, d.renorm, d.scale};
  if (d.dtype == PGG_F32) return launch_typed<TF32>(a, s);
  return d.dtype == PGG_BF16 ? launch_typed<TBf16>(a, s) : launch_typed<TF16>(a, s);
}

hipError_t launch_gate_grouped_grad(const pgg_moe_gate_grouped_desc& d, const void* logits, const int64_t* ids,
                                    const float* grad_probs, void* grad_logits, hipStream_t s) {
  const GroupedGradArgs a = {logits, ids, grad_probs, grad_logits, d.tokens, static_cast<int32_t>(d.experts),
                             static_cast<int32_t>(d.topk), d.score == PGG_SCORE_SOFTMAX, d.renorm, d.scale};
  if (d.dtype == PGG_F32) return launch_grad_typed<TF32>(a, s);
  return d.dtype == PGG_BF16 ? launch_grad_typed<TBf16>(a, s) : launch_grad_typed<TF16>(a, s);
}

}  // namespace pgg
