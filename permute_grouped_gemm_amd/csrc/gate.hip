// The router's gate and its gradient.
//
// Forward, for a token's logits l [E] (an excluded expert has l = -inf):
//   lse     = log sum_e exp(l_e)
//   e_1..e_k = the experts with the k largest l_e + bias_e, larger first, equal
//             ones by lower index (NaN counts as larger than any number).  The
//             bias is added to the logit, not to the score exp(l_e - lse).
//   probs_j = scale * exp(l_{e_j} - lse), or with renorm
//             scale * exp(l_{e_j}) / sum_m exp(l_{e_m})
// Gradient, with d_j = scale * grad_probs_j and p = softmax(l) = exp(l - lse):
//   grad_l_e = p_e * (D_e - sum_j d_j p_{e_j}) + grad_lse * p_e, with D_e = d_j at
//   the pick e_j = e (a token's picks are distinct) and 0 at the other experts,
//   or with renorm and u = softmax of the chosen logits
//   grad_l_{e_j} = u_j * (d_j - sum_m d_m u_m), plus grad_lse * p_e everywhere.
//
// Both read the logits once; small batches are bound by the launch, large ones
// by the picks (forward) and by reading and writing (gradient).  A row belongs
// to 16, 32 or 64 neighbouring lanes, so one wave takes up to four rows, and a
// lane holds chunks of four successive experts.  The forward keeps the row in
// registers, as the logits and as order-preserving integer keys: picking the
// largest is then an integer maximum over the lanes (row rotations of the
// data-parallel primitives, no LDS), followed by a minimum over the indices
// that hold it, and only the owner's entry is struck out before the next
// pick.  Against one row per wave this shares the fixed cost of a pick, about
// 40 instructions, between four rows.  In the gradient, lane j of a row takes
// pick j and hands its d_j to the expert's lane through LDS.
//
// Sums and maxima are fp32 and are added in a fixed order.
//
// Measured: 13824 tokens, 60 experts, 8 picks, fp32: forward 6.5 us (3.3 MB read,
// 1.4 written: the eight picks that follow one another, not bytes), gradient 5.3 us
// (4.9 MB read, 3.3 written, 1.5 TB/s; in a row of launches 4.4); 16 tokens of 16
// experts 3.4 us, a launch's own time.
#include "pgg_device.h"

namespace pgg {

namespace {

constexpr int kGateThreads = 256;
constexpr float kNegInf = -__builtin_inff();

struct GateArgs {
  const void* logits;   // [T, E]
  const float* bias;    // [E] or NULL
  int64_t* ids;         // [T, k]
  float* probs;         // [T, k]
  float* lse;           // [T] or NULL
  int64_t T;
  int32_t E, k;
  int32_t renorm;
  float scale;
};

struct GateGradArgs {
  const void* logits;        // [T, E]
  const float* lse;          // [T]
  const int64_t* ids;        // [T, k]
  const float* grad_probs;   // [T, k]
  const float* grad_lse;     // [T] or NULL
  void* grad_logits;         // [T, E]
  int64_t T;
  int32_t E, k;
  int32_t renorm;
  float scale;
};

// Unsigned order of the result = order of the floats, -0 equal to +0, NaN
// above +inf.  Every key is above 0, which marks a struck-out or missing entry.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);   // -0 + 0 = +0
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// Value of the lane N places on within its group of 16 lanes.
template <int N>
__device__ __forceinline__ uint32_t rotate16(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + N, 0xF, 0xF, false));
}

// Reductions over the LPR lanes of a row; every lane gets the result.
template <int LPR, class Op>
__device__ __forceinline__ uint32_t reduce_u32(uint32_t v, Op op) {
  v = op(v, rotate16<8>(v));
  v = op(v, rotate16<4>(v));
  v = op(v, rotate16<2>(v));
  v = op(v, rotate16<1>(v));
  if constexpr (LPR >= 32) v = op(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 16)));
  if constexpr (LPR >= 64) v = op(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 32)));
  return v;
}

template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  return reduce_u32<LPR>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}

template <int LPR>
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  return reduce_u32<LPR>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  return __builtin_bit_cast(float, reduce_u32<LPR>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  }));
}

// Largest value of a row; NaN where any is NaN (its key is the largest).
template <int LPR>
__device__ __forceinline__ float row_max_float(float v) {
  const uint32_t k = row_max<LPR>(order_key(v));
  if (k == 0xFFFFFFFFu) return __builtin_nanf("");
  return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The largest logit, as softmax subtracts it: 0 for a row of -inf.
__device__ __forceinline__ float pivot(float m) { return m == kNegInf ? 0.0f : m; }

// Four successive entries from e on; past E: -inf.
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

// The k picks are kept LPR to a register: pick j by lane j % LPR.
template <int LPR>
constexpr int kPickRegs = (PGG_GATE_MAX_TOPK + LPR - 1) / LPR;

// Weights of the picks, and the stores.  sel[s] is the expert of pick
// s * LPR + lane; top / total are the pivot and the sum of exp of the whole row.
template <class T, int LPR>
__device__ __forceinline__ void finish_row(const GateArgs& a, const typename T::elem* row, int64_t t, int lane,
                                           const int32_t (&sel)[kPickRegs<LPR>], float top, float total) {
  float l[kPickRegs<LPR>];
#pragma unroll
  for (int s = 0; s < kPickRegs<LPR>; ++s)
    l[s] = s * LPR + lane < a.k ? to_float<T>(row[sel[s]]) : kNegInf;
  if (a.renorm) {
    float m = l[0];
#pragma unroll
    for (int s = 1; s < kPickRegs<LPR>; ++s) m = (l[s] != l[s] || l[s] > m) ? l[s] : m;
    top = pivot(row_max_float<LPR>(m));
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < kPickRegs<LPR>; ++s) sum += expf(l[s] - top);
    total = row_sum<LPR>(sum);
  }
#pragma unroll
  for (int s = 0; s < kPickRegs<LPR>; ++s) {
    const int j = s * LPR + lane;
    if (j < a.k) {
      const float e = expf(l[s] - top);
      a.ids[t * a.k + j] = sel[s];
      a.probs[t * a.k + j] = (total == 0.0f ? e : e / total) * a.scale;   // NaN stays NaN
    }
  }
}

// E <= LPR * EPL: the row lives in registers, entry i of lane c is expert
// 4 (i / 4 * LPR + c) + i % 4.
template <class T, int LPR, int EPL>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateArgs a) {
  using E = typename T::elem;
  const int lane = threadIdx.x % LPR;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kGateThreads / LPR) + threadIdx.x / LPR;
  // rows past the end repeat the last one (whole waves stay together) and store nothing
  const bool live = t < a.T;
  const int64_t tr = live ? t : a.T - 1;
  const E* __restrict__ row = static_cast<const E*>(a.logits) + tr * a.E;
  auto expert = [&](int i) { return 4 * (i / 4 * LPR + lane) + i % 4; };
  float l[EPL];
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; i += 4) load4<T>(row, expert(i), a.E, *reinterpret_cast<float(*)[4]>(&l[i]));
  float m = l[0];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert(i);
    const float b = a.bias && e < a.E ? a.bias[e] : 0.0f;
    key[i] = e < a.E ? order_key(l[i] + b) : 0u;
    m = (l[i] != l[i] || l[i] > m) ? l[i] : m;
  }
  const float top = pivot(row_max_float<LPR>(m));
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) sum += expf(l[i] - top);
  const float total = row_sum<LPR>(sum);

  int32_t sel[kPickRegs<LPR>];
#pragma unroll
  for (int s = 0; s < kPickRegs<LPR>; ++s) {
    sel[s] = 0;
    for (int j = 0; j < min(LPR, a.k - s * LPR); ++j) {
      uint32_t best = key[0];
      uint32_t at = expert(0);
#pragma unroll
      for (int i = 1; i < EPL; ++i)
        if (key[i] > best) {
          best = key[i];
          at = expert(i);
        }
      const uint32_t top_key = row_max<LPR>(best);
      const uint32_t e = row_min<LPR>(best == top_key ? at : 0xFFFFFFFFu);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (e == static_cast<uint32_t>(expert(i))) key[i] = 0u;
      if (lane == j) sel[s] = static_cast<int32_t>(e);
    }
  }
  if (live) {
    if (a.lse && lane == 0) a.lse[t] = top + logf(total);
    finish_row<T, LPR>(a, row, t, lane, sel, top, total);
  }
}

// Any E: one wave per row, which every pick reads again (from L1/L2): the next
// pick is the largest (key, lower index) below the last one.
template <class T>
__global__ __launch_bounds__(kGateThreads) void gate_long_kernel(GateArgs a) {
  using E = typename T::elem;
  constexpr int LPR = 64;
  const int lane = threadIdx.x % LPR;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kGateThreads / LPR) + threadIdx.x / LPR;
  if (t >= a.T) return;
  const E* __restrict__ row = static_cast<const E*>(a.logits) + t * a.E;
  float m = kNegInf;
  for (int e = lane; e < a.E; e += LPR) {
    const float v = to_float<T>(row[e]);
    m = (v != v || v > m) ? v : m;
  }
  const float top = pivot(row_max_float<LPR>(m));
  float sum = 0.0f;
  for (int e = lane; e < a.E; e += LPR) sum += expf(to_float<T>(row[e]) - top);
  const float total = row_sum<LPR>(sum);

  int32_t sel[kPickRegs<LPR>];
  uint32_t last_key = 0xFFFFFFFFu;
  int64_t last = -1;
#pragma unroll
  for (int s = 0; s < kPickRegs<LPR>; ++s) {
    sel[s] = 0;
    for (int j = 0; j < min(LPR, a.k - s * LPR); ++j) {
      uint32_t best = 0u, at = 0xFFFFFFFFu;
      for (int e = lane; e < a.E; e += LPR) {
        const uint32_t key = order_key(to_float<T>(row[e]) + (a.bias ? a.bias[e] : 0.0f));
        const bool left = key < last_key || (key == last_key && e > last);
        if (left && key > best) {
          best = key;
          at = e;
        }
      }
      last_key = row_max<LPR>(best);
      last = row_min<LPR>(best == last_key ? at : 0xFFFFFFFFu);
      if (lane == j) sel[s] = static_cast<int32_t>(last);
    }
  }
  if (a.lse && lane == 0) a.lse[t] = top + logf(total);
  finish_row<T, LPR>(a, row, t, lane, sel, top, total);
}

// LPR lanes per row, rows of one wave only; E floats of LDS per row, which hold
// d_j at the picks and kUnpicked elsewhere.
constexpr uint32_t kUnpicked = 0x7FC0DEADu;   // a NaN; those among the d_j are stored as another

// Up to this |lse| its fp32 rounding changes exp(l - lse) by 2^-21 of itself at
// most.  Beyond, exp(l - lse) is divided by its sum over the row: in a row of the
// type's lowest value log E is lost in lse, and every expert's exp(l - lse) is 1.
// The sum reads the row once more (13824 x 256, bf16: 8.5 us if it is made for
// every row, 7.7 without).
constexpr float kNearLse = 16.0f;

template <class T, int LPR, int THREADS>
__global__ __launch_bounds__(THREADS) void gate_grad_kernel(GateGradArgs a) {
  using E = typename T::elem;
  extern __shared__ uint32_t picked_rows[];
  const int lane = threadIdx.x % LPR;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (THREADS / LPR) + threadIdx.x / LPR;
  const bool live = t < a.T;
  const int64_t tr = live ? t : a.T - 1;   // whole waves stay together
  const E* __restrict__ row = static_cast<const E*>(a.logits) + tr * a.E;
  uint32_t* picked = picked_rows + threadIdx.x / LPR * a.E;
  const float lse = a.lse[tr];
  const float glse = a.grad_lse ? a.grad_lse[tr] : 0.0f;
  // this lane's picks; an id outside the experts selects nothing
  int32_t id[kPickRegs<LPR>];
  float d[kPickRegs<LPR>], l[kPickRegs<LPR>];
#pragma unroll
  for (int s = 0; s < kPickRegs<LPR>; ++s) {
    const int j = s * LPR + lane;
    const int64_t e = j < a.k ? a.ids[tr * a.k + j] : -1;
    id[s] = static_cast<uint64_t>(e) < static_cast<uint64_t>(a.E) ? static_cast<int32_t>(e) : -1;
    d[s] = id[s] >= 0 ? a.grad_probs[tr * a.k + j] * a.scale : 0.0f;
    l[s] = id[s] >= 0 ? to_float<T>(row[id[s]]) : kNegInf;
  }
  for (int e = lane; e < a.E; e += LPR) picked[e] = kUnpicked;
  auto soft = [&](float x) { return lse == kNegInf ? 0.0f : expf(x - lse); };
  float qnorm = 1.0f;   // softmax = soft * qnorm
  if ((!a.renorm || a.grad_lse) && fabsf(lse) > kNearLse) {
    float total = 0.0f;
    for (int e0 = 4 * lane; e0 < a.E; e0 += 4 * LPR) {
      float x[4];
      load4<T>(row, e0, a.E, x);
      total += (soft(x[0]) + soft(x[1])) + (soft(x[2]) + soft(x[3]));
    }
    total = row_sum<LPR>(total);
    qnorm = total == 0.0f ? 1.0f : 1.0f / total;
  }
  // p = exp(l - top) * inv, the weights the picks come from
  float top = lse, inv = qnorm;
  if (a.renorm) {
    float m = l[0];
#pragma unroll
    for (int s = 1; s < kPickRegs<LPR>; ++s) m = (l[s] != l[s] || l[s] > m) ? l[s] : m;
    top = row_max_float<LPR>(m);
  }
  top = pivot(top);
  float p[kPickRegs<LPR>], sum = 0.0f;
#pragma unroll
  for (int s = 0; s < kPickRegs<LPR>; ++s) {
    p[s] = expf(l[s] - top);
    sum += p[s];
  }
  if (a.renorm) {
    sum = row_sum<LPR>(sum);
    inv = sum == 0.0f ? 1.0f : 1.0f / sum;
  }
  float mean = 0.0f;   // sum_j d_j p_j
#pragma unroll
  for (int s = 0; s < kPickRegs<LPR>; ++s)
    if (id[s] >= 0) mean += d[s] * (p[s] * inv);
  mean = row_sum<LPR>(mean);
  // LDS operations of a wave are done in order; only the compiler has to keep it
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int s = 0; s < kPickRegs<LPR>; ++s)
    if (id[s] >= 0) picked[id[s]] = d[s] == d[s] ? __builtin_bit_cast(uint32_t, d[s]) : 0x7FC00000u;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (!live) return;
  E* out = static_cast<E*>(a.grad_logits) + t * a.E;
  for (int e0 = 4 * lane; e0 < a.E; e0 += 4 * LPR) {
    float x[4];
    load4<T>(row, e0, a.E, x);
    E g[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = e0 + i < a.E ? picked[e0 + i] : kUnpicked;
      const bool hit = u != kUnpicked;
      const float di = hit ? __builtin_bit_cast(float, u) : 0.0f;
      const float q = soft(x[i]) * qnorm;
      float v;
      if (a.renorm) v = hit ? expf(x[i] - top) * inv * (di - mean) : 0.0f;
      else v = q * (di - mean);
      if (a.grad_lse) v += glse * q;
      g[i] = from_float<T>(v);
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

template <int LPR, int THREADS = kGateThreads>
dim3 rows_grid(int64_t T) {
  constexpr int64_t per = THREADS / LPR;
  return dim3(static_cast<unsigned>((T + per - 1) / per));
}

template <class T>
hipError_t launch_gate_typed(const GateArgs& a, hipStream_t s) {
  const dim3 b(kGateThreads);
  if (a.E <= 64) hipLaunchKernelGGL((gate_kernel<T, 16, 4>), rows_grid<16>(a.T), b, 0, s, a);
  else if (a.E <= 128) hipLaunchKernelGGL((gate_kernel<T, 16, 8>), rows_grid<16>(a.T), b, 0, s, a);
  else if (a.E <= 256) hipLaunchKernelGGL((gate_kernel<T, 16, 16>), rows_grid<16>(a.T), b, 0, s, a);
  else if (a.E <= 512) hipLaunchKernelGGL((gate_kernel<T, 32, 16>), rows_grid<32>(a.T), b, 0, s, a);
  else if (a.E <= 1024) hipLaunchKernelGGL((gate_kernel<T, 64, 16>), rows_grid<64>(a.T), b, 0, s, a);
  else hipLaunchKernelGGL((gate_long_kernel<T>), rows_grid<64>(a.T), b, 0, s, a);
  return hipGetLastError();
}

template <class T, int LPR, int THREADS>
hipError_t launch_gate_grad_rows(const GateGradArgs& a, hipStream_t s) {
  const size_t lds = sizeof(uint32_t) * (THREADS / LPR) * static_cast<size_t>(a.E);
  hipLaunchKernelGGL((gate_grad_kernel<T, LPR, THREADS>), (rows_grid<LPR, THREADS>(a.T)), dim3(THREADS), lds, s, a);
  return hipGetLastError();
}

// 16 KiB of LDS at most per workgroup, but one row always fits (32 KiB)
template <class T>
hipError_t launch_gate_grad_typed(const GateGradArgs& a, hipStream_t s) {
  if (a.E <= 64) return launch_gate_grad_rows<T, 16, 256>(a, s);
  if (a.E <= 128) return launch_gate_grad_rows<T, 32, 256>(a, s);
  if (a.E <= 1024) return launch_gate_grad_rows<T, 64, 256>(a, s);
  return launch_gate_grad_rows<T, 64, 64>(a, s);
}

}  // namespace

hipError_t launch_gate(const pgg_moe_gate_desc& d, const void* logits, const float* bias, int64_t* ids,
                       float* probs, float* lse, hipStream_t s) {
  const GateArgs a = {logits, bias, ids, probs, lse, d.tokens, static_cast<int32_t>(d.experts),
                      static_cast<int32_t>(d.topk), d.renorm, d.scale};
  if (d.dtype == PGG_F32) return launch_gate_typed<TF32>(a, s);
  return d.dtype == PGG_BF16 ? launch_gate_typed<TBf16>(a, s) : launch_gate_typed<TF16>(a, s);
}

hipError_t launch_gate_grad(const pgg_moe_gate_desc& d, const void* logits, const float* lse, const int64_t* ids,
                            const float* grad_probs, const float* grad_lse, void* grad_logits, hipStream_t s) {
  const GateGradArgs a = {logits, lse, ids, grad_probs, grad_lse, grad_logits, d.tokens,
                          static_cast<int32_t>(d.experts), static_cast<int32_t>(d.topk), d.renorm, d.scale};
  if (d.dtype == PGG_F32) return launch_gate_grad_typed<TF32>(a, s);
  return d.dtype == PGG_BF16 ? launch_gate_grad_typed<TBf16>(a, s) : launch_gate_grad_typed<TF16>(a, s);
}

}  // namespace pgg
