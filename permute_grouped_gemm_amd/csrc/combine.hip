// The end of a block: the experts' rows summed per token, a norm of the sum, the
// residual stream, and the norm in front of the next block.
//
//   c      = sum_j p_j y_j                 y_j = permuted[row(t, j)], p_j = probs[t, j]
//   a      = c r w_post,  r = 1 / sqrt(mean(c^2) + eps)         (or c)
//   out    = alpha residual + g a
//   normed = out q w_next,  q = 1 / sqrt(mean(out^2) + eps)
//
// Gradient, from go = d/d out and gn = d/d normed, u = gn w_next:
//   go    += q (u - n mean(u n)),  n = out q                    (d/d out in all)
//   residual: alpha go        w_next: sum_t gn out q
//   m      = c r, s = sum_h go w_post m                         (r and w_post 1 without it)
//   gate:  s                  w_post: sum_t g go m
//   gc     = g r (go w_post - m s / H)                          (or g go)
//   y_j:   p_j gc             p_j: sum_h gc y_j
// q and r stay with the rows that they normalise: their cubes leave fp32's range
// for rows of 1e13 and more, and for rows near 0 under a small eps.
//
// Both are bound by reading and writing the rows once.  A workgroup takes a
// token, a thread 8 successive elements of each of its rows (16 in the gradient,
// 32 of rows of more than 8192), so the rows of up to 8 slots are requested at once
// and stay in registers from the first use to the last; only the sums over h go
// through LDS.  The forward's loads and stores carry the non-temporal hint
// (110592 x 7168, f16: 374 us, 5.8 TB/s, and 427 without it; the gradient, bf16,
// takes 822 us without, 4.8 TB/s, and 887 with it).  In the gradient a workgroup goes
// through tokens in steps of the grid and keeps its part of the weights' gradients
// in registers (of long rows in memory); a second kernel adds the workgroups' parts.
//
// The routing index is read as it is where it holds rows (row_idx_type 1);
// otherwise it is searched where it is short, and inverted by a launch before
// where it is long.  It is checked beside the work: in one spare workgroup with a
// bit per row where M is small, else by workgroups of the same launch against the
// tables that the launch before has filled.  Rows outside [0, M) read and write
// row 0.
#include <algorithm>

#include "pgg_nn.h"
#include "pgg_prep.h"

namespace pgg {

namespace {

struct CombineArgs {
  const void* permuted;
  const int64_t* eri;
  const float* probs;
  const void* residual;
  const void* post;
  const float* gate;
  const void* next;
  void* out;            // forward
  void* normed;
  const void* grad_out; // gradient
  const void* grad_normed;
  void* grad_permuted;
  float* grad_probs;
  void* grad_residual;
  float* grad_gate;
  float* part_post;     // [workgroups, H]
  float* part_next;
  const int32_t* inv;   // NULL: eri holds the rows
  int64_t M, batch, H, topk;
  float alpha, eps, inv_h;
  int32_t check;        // workgroups in front that check the index
  int32_t bits;         // 1: one, with a bit per row
  int32_t scan;         // 1: a token's rows are looked for in eri
  PrepArgs prep;
  WsView ws;
};

constexpr int kMaxWaves = 16;
constexpr int kBitRows = 16384;   // rows that the spare workgroup's bits hold

// Slots whose rows are requested together and, where they are all, stay in
// registers: as many as fit 128 registers with one piece of a row to a thread (a
// workgroup of up to 16 waves), 256 with more (up to 8 waves).
template <class T, int NCH>
constexpr int kHeld = NCH == 4 ? (__is_same(T, TF32) ? 1 : 2) : __is_same(T, TF32) && NCH == 2 ? 4 : 8;
template <int NCH>
constexpr int kMaxThreads = NCH > 1 ? 512 : 1024;

// 8 elements as loaded.
template <class T>
struct Eight {
  u32x4_t v[8 / T::kPerChunk];
};

// How rows divide into pieces of 8.  kOverlap: the last piece ends with the row
// and shares its first elements with the piece before, so that all loads are whole;
// the shared elements count in the sums in the piece before only.  With the last
// piece's elements loaded and stored one by one 333 tokens x 2, 2039, bf16, took
// 8.2 us instead of 7.0, and the gradient 22.3 instead of 20.4.
// kShort: fewer than 8 elements.
enum Rows { kEven, kOverlap, kShort };

// One of a thread's pieces of a row: elements h + first .. h + 7 are its own
// (kShort: the first `last`), none if last is 0, when h is a place to read from.
struct Piece {
  uint32_t h;
  int first, last;
};

// A thread without a piece reads as another one, in no branch of its own.
// STREAM: not to be kept in the caches.
typedef unsigned int u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));   // at any address

template <class T, Rows ROWS, bool STREAM = false>
__device__ __forceinline__ Eight<T> load8(const void* base, int64_t row, const Piece& c) {
  using E = typename T::elem;
  const E* p = static_cast<const E*>(base) + row + c.h;
  Eight<T> r;
  if constexpr (ROWS != kShort) {
#pragma unroll
    for (int h = 0; h < 8 / T::kPerChunk; ++h) {
      const u32x4_any_t* q = reinterpret_cast<const u32x4_any_t*>(p + h * T::kPerChunk);
      r.v[h] = STREAM ? __builtin_nontemporal_load(q) : *q;
    }
  } else {
    E e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = k < c.last ? p[k] : E(0);
    __builtin_memcpy(&r, e, sizeof(r));
  }
  return r;
}

template <class T>
__device__ __forceinline__ Eight<T> ones8() {
  constexpr uint32_t one = __is_same(T, TF32) ? 0x3F800000u : __is_same(T, TBf16) ? 0x3F803F80u : 0x3C003C00u;
  Eight<T> r;
#pragma unroll
  for (int h = 0; h < 8 / T::kPerChunk; ++h) r.v[h] = u32x4_t{one, one, one, one};
  return r;
}

template <class T>
__device__ __forceinline__ float get(const Eight<T>& r, int k) {
  if constexpr (T::kPerChunk == 4) {
    const uint32_t u = r.v[k >> 2][k & 3];
    return __builtin_bit_cast(float, u);
  } else {
    const uint32_t u = r.v[0][k >> 1];
    return to_float<T>(static_cast<uint16_t>(k & 1 ? u >> 16 : u & 0xFFFFu));
  }
}

// SHARED: both pieces store the elements they share, which come out alike; not
// where another piece's threads still read what is stored over.
template <class T, Rows ROWS, bool SHARED, bool STREAM = false>
__device__ __forceinline__ void store8(void* base, int64_t row, const Piece& c, const float (&v)[8]) {
  using E = typename T::elem;
  E* p = static_cast<E*>(base) + row + c.h;
  E e[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) e[k] = from_float<T>(v[k]);
  if (ROWS == kEven || (ROWS == kOverlap && (SHARED || c.first == 0))) {
    u32x4_t v[8 / T::kPerChunk];
    __builtin_memcpy(v, e, sizeof(e));
#pragma unroll
    for (int h = 0; h < 8 / T::kPerChunk; ++h) {
      u32x4_any_t* q = reinterpret_cast<u32x4_any_t*>(p + h * T::kPerChunk);
      if constexpr (STREAM) __builtin_nontemporal_store(static_cast<u32x4_any_t>(v[h]), q);
      else *q = v[h];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k >= c.first && k < c.last) p[k] = e[k];
  }
}

// sum += a b, for an element k of this piece (past a short row's end all inputs are 0).
template <Rows ROWS>
__device__ __forceinline__ void add(const Piece& c, int k, float a, float b, float& sum) {
  const bool other = ROWS == kOverlap && k < c.first;
  sum = __builtin_fmaf(other ? 0.0f : a, other ? 0.0f : b, sum);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// Sum of v[0..N) over the workgroup, in wave order; s: N x kMaxWaves words that
// nobody uses until the barrier after next.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*s)[kMaxWaves]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = wave_sum(v[n]);
    if (lane == 0) s[n][wave] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float sum = s[n][0];
    for (int w = 1; w < waves; ++w) sum += s[n][w];
    v[n] = sum;
  }
}

// The workgroups that check the index.
__device__ __forceinline__ void check_index(const CombineArgs& a, int bid, uint32_t* bits) {
  if (a.bits) {
    if (threadIdx.x == 0) {
      a.ws.hdr->err = kNoError;
      a.ws.hdr->n_tiles = 0;
    }
    for (int i = threadIdx.x; i < kBitRows / 32; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    for (int64_t p = threadIdx.x; p < a.M; p += blockDim.x) {
      const int64_t v = a.eri[p];
      if (v < 0 || v >= a.M) {
        set_error(a.ws.hdr, PGG_DEV_INDEX_RANGE, p);
      } else {
        const uint32_t bit = 1u << (v & 31);
        if (atomicOr(&bits[v >> 5], bit) & bit) set_error(a.ws.hdr, PGG_DEV_INDEX_DUP, v);
      }
    }
    return;
  }
  for (int64_t p = static_cast<int64_t>(bid) * blockDim.x + threadIdx.x; p < a.M;
       p += static_cast<int64_t>(a.check) * blockDim.x) {
    const int64_t v = a.eri[p];
    if (v < 0 || v >= a.M) set_error(a.ws.hdr, PGG_DEV_INDEX_RANGE, p);
    else verify_one(a.prep, a.eri, a.ws, p);
  }
}

// Header and index tables (entries outside [0, M) are skipped, and reported by check_index).
__global__ __launch_bounds__(256) void combine_index_kernel(PrepArgs prep, const int64_t* eri, WsView w) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    w.hdr->err = kNoError;
    w.hdr->n_tiles = 0;
  }
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t < prep.M && eri[t] >= 0 && eri[t] < prep.M) index_one(prep, eri, w, t);
}

__device__ __forceinline__ float uniform(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int32_t, v)));
}

// Rows and probabilities of up to 64 slots from position p on, slot q in lane q:
// one load for all of them, after which each comes from a scalar register.
struct Slots {
  int32_t row;
  float prob;

  // found: the token's rows as find_rows leaves them, j the slot of position p
  __device__ __forceinline__ void load(const CombineArgs& a, int64_t p, int n, const int32_t* found, int64_t j) {
    const int lane = threadIdx.x & 63, q = min(lane, n - 1);
    const int64_t at = p + q;
    const int64_t r = a.scan ? found[j + q] : a.inv ? a.inv[at] : a.eri[at];
    row = static_cast<uint64_t>(r) < static_cast<uint64_t>(a.M) ? static_cast<int32_t>(r) : 0;
    prob = a.probs[at];
  }
  __device__ __forceinline__ int64_t row_of(int q) const { return __builtin_amdgcn_readlane(row, q); }
  __device__ __forceinline__ float prob_of(int q) const {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int32_t, prob), q));
  }
};

// Rows of token t's slots where the index holds positions and is short: every
// workgroup looks through all of it.  Ends with a barrier.
constexpr int kScanSlots = 64;
__device__ __forceinline__ void find_rows(const CombineArgs& a, int64_t t, int32_t* found) {
  if (threadIdx.x < kScanSlots) found[threadIdx.x] = 0;
  __syncthreads();
  const int64_t p0 = t * a.topk;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < a.M; i += blockDim.x) {
    const int64_t j = a.eri[i] - p0;
    if (j >= 0 && j < a.topk) found[j] = static_cast<int32_t>(i);
  }
  __syncthreads();
}

// The rows of n <= HELD slots (after the last, the last again).
template <class T, int NCH, Rows ROWS, bool STREAM, int HELD>
__device__ __forceinline__ void load_slots(const CombineArgs& a, const Slots& s, const Piece (&piece)[NCH],
                                           Eight<T> (&y)[HELD][NCH]) {
#pragma unroll
  for (int q = 0; q < HELD; ++q) {
    const int64_t row = s.row_of(q) * a.H;
#pragma unroll
    for (int i = 0; i < NCH; ++i) y[q][i] = load8<T, ROWS, STREAM>(a.permuted, row, piece[i]);
  }
}

// c += p_j y_j, in slot order.
template <class T, int NCH, int HELD>
__device__ __forceinline__ void add_slots(const Slots& s, int n, const Eight<T> (&y)[HELD][NCH], float (&c)[NCH][8]) {
#pragma unroll
  for (int q = 0; q < HELD; ++q)
    if (q < n)
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) c[i][k] = __builtin_fmaf(s.prob_of(q), get<T>(y[q][i], k), c[i][k]);
}

// This thread's pieces of a row.
template <int NCH, Rows ROWS>
__device__ __forceinline__ void pieces(int64_t H, Piece (&c)[NCH]) {
  const int n = static_cast<int>(H);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int at = 8 * static_cast<int>(threadIdx.x + i * blockDim.x);
    c[i].last = max(0, min(8, n - at));
    c[i].first = 0;
    c[i].h = c[i].last == 0 ? 0 : at;
    if (ROWS == kOverlap && c[i].last > 0 && c[i].last < 8) {
      c[i].first = 8 - c[i].last;
      c[i].last = 8;
      c[i].h = n - 8;
    }
  }
}

template <class T, int NCH, Rows ROWS>
__global__ __launch_bounds__(kMaxThreads<NCH>) void combine_kernel(CombineArgs a) {
  constexpr int HELD = kHeld<T, NCH>;
  __shared__ union {
    float sums[2][1][kMaxWaves];
    uint32_t bits[kBitRows / 32];
  } s;
  if (static_cast<int>(blockIdx.x) < a.check) {
    check_index(a, blockIdx.x, s.bits);
    return;
  }
  const int64_t t = static_cast<int64_t>(blockIdx.x) - a.check;
  Piece piece[NCH];
  pieces<NCH, ROWS>(a.H, piece);
  Slots slots;
  __shared__ int32_t s_found[kScanSlots];
  if (a.scan) find_rows(a, t, s_found);
  slots.load(a, t * a.topk, static_cast<int>(min<int64_t>(HELD, a.topk)), s_found, 0);
  Eight<T> res[NCH], post[NCH], next[NCH], y[HELD][NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    res[i] = load8<T, ROWS, true>(a.residual, t * a.H, piece[i]);
    if (a.post) post[i] = load8<T, ROWS>(a.post, 0, piece[i]);
    if (a.next) next[i] = load8<T, ROWS>(a.next, 0, piece[i]);
  }
  const float gate = a.gate ? uniform(a.gate[t]) : 1.0f;
  float c[NCH][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) c[i][k] = 0.0f;
  for (int64_t j0 = 0; j0 < a.topk; j0 += HELD) {
    const int n = static_cast<int>(min<int64_t>(HELD, a.topk - j0));
    if (j0) slots.load(a, t * a.topk + j0, n, s_found, j0);
    load_slots<T, NCH, ROWS, true, HELD>(a, slots, piece, y);
    add_slots<T, NCH, HELD>(slots, n, y, c);
  }

  float r = 1.0f;
  if (a.post) {
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (piece[i].last > 0)
#pragma unroll
        for (int k = 0; k < 8; ++k) add<ROWS>(piece[i], k, c[i][k], c[i][k], sum[0]);
    block_sum<1>(sum, s.sums[0]);
    r = 1.0f / sqrtf(sum[0] * a.inv_h + a.eps);
  }
  float sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NCH; ++i)
    if (piece[i].last > 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = a.post ? c[i][k] * r * get<T>(post[i], k) : c[i][k];
        c[i][k] = __builtin_fmaf(a.alpha, get<T>(res[i], k), gate * v);
        add<ROWS>(piece[i], k, c[i][k], c[i][k], sum[0]);
      }
      store8<T, ROWS, false, true>(a.out, t * a.H, piece[i], c[i]);
    }
  if (!a.next) return;
  block_sum<1>(sum, s.sums[1]);
  const float q = 1.0f / sqrtf(sum[0] * a.inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < NCH; ++i)
    if (piece[i].last > 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) c[i][k] *= q * get<T>(next[i], k);
      store8<T, ROWS, false, true>(a.normed, t * a.H, piece[i], c[i]);
    }
}

// ONCE: topk <= HELD, all rows stay.
template <class T, int NCH, Rows ROWS, bool ONCE>
__global__ __launch_bounds__(kMaxThreads<NCH>) void combine_grad_kernel(CombineArgs a) {
  constexpr int HELD = kHeld<T, NCH>;
  // Long rows leave no registers for the weights' gradients, which then stay in
  // this workgroup's part in memory, nor for inputs that wait for their use.
  constexpr bool kLong = NCH > 2;
  // A missing post_weight is 1 where registers hold it: with fewer branches the
  // compiler spills fewer scalar registers (13824 x 8 x 7168, bf16: 821 us, and 872
  // with branches).  In fp32 it would spill vector registers instead.
  constexpr bool kOnes = !kLong && !__is_same(T, TF32);
  __shared__ union {
    struct {
      float one[1][kMaxWaves], two[2][kMaxWaves], three[1][kMaxWaves], slots[HELD][kMaxWaves];
    } sums;
    uint32_t bits[kBitRows / 32];
  } s;
  if (static_cast<int>(blockIdx.x) < a.check) {
    check_index(a, blockIdx.x, s.bits);
    return;
  }
  __shared__ int32_t s_found[kScanSlots];
  const int64_t first = static_cast<int64_t>(blockIdx.x) - a.check, step = static_cast<int64_t>(gridDim.x) - a.check;
  Piece piece[NCH];
  pieces<NCH, ROWS>(a.H, piece);
  Eight<T> post_reg[NCH], next_reg[NCH];
  float dpost[kLong ? 1 : NCH][8], dnext[kLong ? 1 : NCH][8];
  if constexpr (!kLong) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (a.post) post_reg[i] = load8<T, ROWS>(a.post, 0, piece[i]);
      else if (kOnes) post_reg[i] = ones8<T>();
      if (a.next) next_reg[i] = load8<T, ROWS>(a.next, 0, piece[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) dpost[i][k] = dnext[i][k] = 0.0f;
    }
  }
  auto post = [&](int i) { return kLong ? load8<T, ROWS>(a.post, 0, piece[i]) : post_reg[i]; };
  auto next = [&](int i) { return kLong ? load8<T, ROWS>(a.next, 0, piece[i]) : next_reg[i]; };
  // adds to a weight's gradient
  auto add_weight = [&](float* part, float (&sum)[kLong ? 1 : NCH][8], int64_t t, int i, const float (&v)[8]) {
    if constexpr (kLong) {
      float* p = part + first * a.H + piece[i].h;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k >= piece[i].first && k < piece[i].last) p[k] = t == first ? v[k] : p[k] + v[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[i][k] += v[k];
    }
  };
  for (int64_t t = first; t < a.batch; t += step) {
    Slots slots;
    if (a.scan) find_rows(a, t, s_found);
    slots.load(a, t * a.topk, static_cast<int>(min<int64_t>(HELD, a.topk)), s_found, 0);
    Eight<T> res_reg[NCH], go_reg[NCH], gn_reg[NCH], y[HELD][NCH];
    if constexpr (!kLong) {
      // the weights are widened where they are used: as loop invariants they would take 16 registers, not 8
#pragma unroll
      for (int v = 0; v < 8 / T::kPerChunk; ++v) 
#pragma unroll
        for (int i = 0; i < NCH; ++i) asm volatile("" : "+v"(post_reg[i].v[v]), "+v"(next_reg[i].v[v]));
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        res_reg[i] = load8<T, ROWS>(a.residual, t * a.H, piece[i]);
        go_reg[i] = load8<T, ROWS>(a.grad_out, t * a.H, piece[i]);
        if (a.next) gn_reg[i] = load8<T, ROWS>(a.grad_normed, t * a.H, piece[i]);
      }
    }
    auto input = [&](const void* from, const Eight<T>& reg, int i) {
      return kLong ? load8<T, ROWS>(from, t * a.H, piece[i]) : reg;
    };
    const float gate = a.gate ? uniform(a.gate[t]) : 1.0f;
    float c[NCH][8], go[NCH][8];
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) c[i][k] = 0.0f;
    for (int64_t j0 = 0; j0 < a.topk; j0 += HELD) {
      const int n = static_cast<int>(min<int64_t>(HELD, a.topk - j0));
      if (!ONCE && j0) slots.load(a, t * a.topk + j0, n, s_found, j0);
      load_slots<T, NCH, ROWS, false, HELD>(a, slots, piece, y);
      add_slots<T, NCH, HELD>(slots, n, y, c);
      if (ONCE) break;
    }

    float r = 1.0f;
    if (a.post) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (piece[i].last > 0)
#pragma unroll
          for (int k = 0; k < 8; ++k) add<ROWS>(piece[i], k, c[i][k], c[i][k], sum[0]);
      block_sum<1>(sum, s.sums.one);
      r = 1.0f / sqrtf(sum[0] * a.inv_h + a.eps);
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) c[i][k] *= r;   // c is m from here on
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const Eight<T> raw = input(a.grad_out, go_reg[i], i);
#pragma unroll
      for (int k = 0; k < 8; ++k) go[i][k] = get<T>(raw, k);
    }
    if (a.next) {
      // out, from m
      auto out = [&](int i, float (&v)[8]) {
        const Eight<T> res = input(a.residual, res_reg[i], i);
        if (kOnes || a.post) {
          const Eight<T> w = post(i);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            v[k] = __builtin_fmaf(a.alpha, get<T>(res, k), gate * (c[i][k] * get<T>(w, k)));
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = __builtin_fmaf(a.alpha, get<T>(res, k), gate * c[i][k]);
        }
      };
      float sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (piece[i].last > 0) {
          float v[8];
          out(i, v);
          const Eight<T> gn = input(a.grad_normed, gn_reg[i], i), w = next(i);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            add<ROWS>(piece[i], k, v[k], v[k], sum[0]);
            add<ROWS>(piece[i], k, get<T>(gn, k) * get<T>(w, k), v[k], sum[1]);
          }
        }
      block_sum<2>(sum, s.sums.two);
      const float q = 1.0f / sqrtf(sum[0] * a.inv_h + a.eps);
      const float back = q * (q * (sum[1] * a.inv_h));   // q mean(u n)
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (piece[i].last > 0) {
          float v[8], d[8];
          out(i, v);
          const Eight<T> gn = input(a.grad_normed, gn_reg[i], i), w = next(i);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float n = v[k] * q;
            d[k] = get<T>(gn, k) * n;
            go[i][k] += q * (get<T>(gn, k) * get<T>(w, k)) - n * back;
          }
          add_weight(a.part_next, dnext, t, i, d);
        }
    }
    float dot = 0.0f;   // sum go w_post m
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (piece[i].last > 0) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = a.alpha * go[i][k];
        if (kOnes || a.post) {
          const Eight<T> w = post(i);
#pragma unroll
          for (int k = 0; k < 8; ++k) add<ROWS>(piece[i], k, go[i][k] * get<T>(w, k), c[i][k], dot);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) add<ROWS>(piece[i], k, go[i][k], c[i][k], dot);
        }
        store8<T, ROWS, true>(a.grad_residual, t * a.H, piece[i], v);
      }
    float total[1] = {dot};
    block_sum<1>(total, s.sums.three);   // (its barrier also parts the sums of successive tokens)
    if (a.gate && threadIdx.x == 0) a.grad_gate[t] = total[0];
    const float back = gate * (r * (total[0] * a.inv_h));
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (piece[i].last > 0) {
        if (a.post) {
          const Eight<T> w = post(i);
          float d[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            d[k] = gate * go[i][k] * c[i][k];
            go[i][k] = (gate * r) * (go[i][k] * get<T>(w, k)) - c[i][k] * back;
          }
          add_weight(a.part_post, dpost, t, i, d);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) go[i][k] *= gate;
        }
      }
    // go is the gradient of c now; rows and probabilities are taken from their lanes again
    asm volatile("" : "+v"(slots.row), "+v"(slots.prob));
    for (int64_t j0 = 0; j0 < a.topk; j0 += HELD) {
      const int n = static_cast<int>(min<int64_t>(HELD, a.topk - j0));
      if constexpr (!ONCE) {   // the rows did not stay
        slots.load(a, t * a.topk + j0, n, s_found, j0);
        load_slots<T, NCH, ROWS, false, HELD>(a, slots, piece, y);
        __syncthreads();   // the sums of the slots before have been read
      }
#pragma unroll
      for (int q = 0; q < HELD; ++q)
        if (q < n) {
          const float p = slots.prob_of(q);
          const int64_t row = slots.row_of(q) * a.H;
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < NCH; ++i)
            if (piece[i].last > 0) {
              float v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                add<ROWS>(piece[i], k, go[i][k], get<T>(y[q][i], k), sum);
                v[k] = p * go[i][k];
              }
              store8<T, ROWS, true>(a.grad_permuted, row, piece[i], v);
            }
          sum = wave_sum(sum);
          if ((threadIdx.x & 63) == 0) s.sums.slots[q][threadIdx.x >> 6] = sum;
        }
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < n) {
        float v = s.sums.slots[threadIdx.x][0];
        for (int w = 1; w < static_cast<int>(blockDim.x >> 6); ++w) v += s.sums.slots[threadIdx.x][w];
        a.grad_probs[t * a.topk + j0 + threadIdx.x] = v;
      }
      if (ONCE) break;
    }
  }
  if constexpr (!kLong) {
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (piece[i].last > 0) {
        if (a.post) store8<TF32, ROWS, true>(a.part_post, first * a.H, piece[i], dpost[i]);
        if (a.next) store8<TF32, ROWS, true>(a.part_next, first * a.H, piece[i], dnext[i]);
      }
  }
}

// Sum of the workgroups' parts, in a fixed order: kSumCols columns to a workgroup,
// kSumRows threads to a column; blockIdx.y 1: the second pair.  32 columns are a
// whole line of the cache.  The gradient of 333 tokens x 2 took (2048 elements, and
// 7168, bf16) with 16 x 16 16.2 us and 29.5, 32 x 16 14.7 and 26.0, 32 x 32 13.9 and
// 26.2, 16 x 64 16.0 and 30.1.
constexpr int kSumCols = 32, kSumRows = 32;
__global__ __launch_bounds__(kSumCols * kSumRows) void combine_weights_kernel(const float* part0, const float* part1,
                                                                              float* out0, float* out1, int64_t H,
                                                                              int32_t rows) {
  const float* part = blockIdx.y ? part1 : part0;
  float* out = blockIdx.y ? out1 : out0;
  if (!out) return;
  __shared__ float s[kSumRows][kSumCols + 1];
  const int col = threadIdx.x % kSumCols, r0 = threadIdx.x / kSumCols;
  const int64_t h = static_cast<int64_t>(blockIdx.x) * kSumCols + col;
  float v = 0.0f;
  if (h < H)
#pragma unroll 8
    for (int r = r0; r < rows; r += kSumRows) v += part[r * H + h];
  s[r0][col] = v;
  __syncthreads();
  if (r0 == 0 && h < H) {
#pragma unroll
    for (int q = 1; q < kSumRows; ++q) v += s[q][col];
    out[h] = v;
  }
}

template <class T, Rows ROWS>
hipError_t launch_rows(const CombinePlan& p, const CombineArgs& a, bool grad, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.check + (grad ? p.grad_blocks : p.batch))), block(p.threads(grad));
  if constexpr (ROWS == kShort) {   // (the smaller kernels)
    if (grad) hipLaunchKernelGGL((combine_grad_kernel<T, 4, ROWS, false>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((combine_kernel<T, 1, ROWS>), grid, block, 0, s, a);
  } else if (!grad) {
    if (p.row_long) hipLaunchKernelGGL((combine_kernel<T, 4, ROWS>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((combine_kernel<T, 1, ROWS>), grid, block, 0, s, a);
  } else {
    if (p.row_long) hipLaunchKernelGGL((combine_grad_kernel<T, 4, ROWS, false>), grid, block, 0, s, a);
    else if (a.topk > kHeld<T, 2>) hipLaunchKernelGGL((combine_grad_kernel<T, 2, ROWS, false>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((combine_grad_kernel<T, 2, ROWS, true>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

template <class T>
hipError_t launch_typed(const CombinePlan& p, const CombineArgs& a, bool grad, hipStream_t s) {
  if (p.H % 8 == 0) return launch_rows<T, kEven>(p, a, grad, s);
  return p.H > 8 ? launch_rows<T, kOverlap>(p, a, grad, s) : launch_rows<T, kShort>(p, a, grad, s);
}

hipError_t launch_any(const CombinePlan& p, CombineArgs& a, const int64_t* eri, void* ws, bool grad, hipStream_t s) {
  char* base = static_cast<char*>(ws);
  WsView w{};
  w.hdr = reinterpret_cast<WsHeader*>(base + p.off_header);
  w.inv = reinterpret_cast<int32_t*>(base + p.off_inv);
  w.ori = reinterpret_cast<int32_t*>(base + p.off_ori);
  a.eri = eri;
  a.inv = p.row_idx_type == 0 ? w.inv : nullptr;
  a.M = p.M;
  a.batch = p.batch;
  a.H = p.H;
  a.topk = p.topk;
  a.alpha = p.alpha;
  a.eps = p.eps;
  a.inv_h = 1.0f / static_cast<float>(p.H);
  a.part_post = reinterpret_cast<float*>(base + p.off_part);
  a.part_next = a.part_post + static_cast<int64_t>(p.grad_blocks) * p.H;
  a.ws = w;
  a.prep.M = p.M;
  a.prep.row_idx_type = p.row_idx_type;
  // a spare workgroup with a bit per row, 16 entries to a thread at most
  const int64_t threads = p.threads(grad);
  // Short indexes of positions are searched by every token's workgroup, which saves
  // the launch that inverts them: up to 8 entries to a thread, and batch * M entries
  // in all, 16 MB from the caches (gradient, which reads more beside them, 8).
  // Searched and inverted in us, in a graph, bf16, topk x M, forward and gradient:
  //   H 7168: 1 x 512 10.2 11.8, 26.6 28.0; 1 x 1024 24.7 25.5, 39.4 39.2; 1 x 2048 47.1 45.2, 67.9 62.8;
  //     1 x 7168 170 141, -; 8 x 2048 9.2 10.7, 25.9 26.5; 8 x 4096 16.3 18.5, 43.7 40.4; 8 x 7168 35.6 32.1, -
  //   H 2048: 1 x 512 5.8 7.1, 15.2 16.6; 1 x 1024 7.8 8.8, 22.3 22.7; 2 x 2048 9.5 10.5, 24.9 23.4
  //   H 64: 1 x 512 5.2 5.9, 9.9 10.6; 1 x 1024 6.6 6.1, 12.1 11.7 (8 entries to a thread are 512)
  a.scan = p.row_idx_type == 0 && p.M <= std::min<int64_t>(kBitRows, 8 * threads) && p.topk <= kScanSlots &&
           p.batch * p.M <= (grad ? 1 << 20 : 1 << 21);
  a.bits = a.scan || (p.row_idx_type == 1 && p.M <= std::min<int64_t>(kBitRows, 16 * threads));
  a.check = a.bits ? 1 : static_cast<int32_t>(std::min<int64_t>((p.M + 4 * threads - 1) / (4 * threads), 1024));
  hipError_t e = hipSuccess;
  if (!a.bits) {
    hipLaunchKernelGGL(combine_index_kernel, dim3(static_cast<unsigned>((p.M + 255) / 256)), dim3(256), 0, s, a.prep, eri,
                       w);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  if (p.dtype == PGG_F32) return launch_typed<TF32>(p, a, grad, s);
  return p.dtype == PGG_BF16 ? launch_typed<TBf16>(p, a, grad, s) : launch_typed<TF16>(p, a, grad, s);
}

}  // namespace

hipError_t launch_combine(const CombinePlan& p, const void* permuted, const int64_t* eri, const float* probs,
                          const void* residual, const void* post, const float* gate, const void* next, void* out,
                          void* normed, void* ws, hipStream_t s) {
  CombineArgs a = {};
  a.permuted = permuted;
  a.probs = probs;
  a.residual = residual;
  a.post = post;
  a.gate = gate;
  a.next = next;
  a.out = out;
  a.normed = normed;
  return launch_any(p, a, eri, ws, false, s);
}

hipError_t launch_combine_grad(const CombinePlan& p, const pgg_moe_combine_grad_args& g, void* ws, hipStream_t s) {
  CombineArgs a = {};
  a.permuted = g.permuted;
  a.probs = g.probs;
  a.residual = g.residual;
  a.post = g.post_weight;
  a.gate = g.gate;
  a.next = g.next_weight;
  a.grad_out = g.grad_out;
  a.grad_normed = g.grad_normed;
  a.grad_permuted = g.grad_permuted;
  a.grad_probs = g.grad_probs;
  a.grad_residual = g.grad_residual;
  a.grad_gate = g.grad_gate;
  hipError_t e = launch_any(p, a, g.expanded_row_idx, ws, true, s);
  if (e != hipSuccess || (!g.grad_post_weight && !g.grad_next_weight)) return e;
  hipLaunchKernelGGL(combine_weights_kernel, dim3(static_cast<unsigned>((p.H + kSumCols - 1) / kSumCols), 2),
                     dim3(kSumCols * kSumRows), 0, s,
                     a.part_post, a.part_next, g.grad_post_weight, g.grad_next_weight, p.H,
                     static_cast<int32_t>(p.grad_blocks));
  return hipGetLastError();
}

}  // namespace pgg
