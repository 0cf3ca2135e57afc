// A shared projection with low-rank adapters of many requests beside it:
//
//   y[t, :] = x[t, :] * W + scale[p] * (x[t, :] * A_p^T) * B_p      p = adapter_ids[t]
//
// W [K, N] is the same for every token; A_p and B_p hold one row per rank,
// A [P, R, K] and B [P, R, N]; a token with a negative id has no adapter.
// Tokens may come in any order; requests of many tokens are runs of one id.
//
// The inner product z = scale * x * A_p^T is computed first, in fp32, into the
// workspace ([T, R], a few values per token).  Then the shared product runs on
// the tiles of pgg_nn.h, and the tokens' z * B_p are added to its fp32
// accumulators before the one rounding of the store, so y is written once and
// the projection is never read back.
//
// Which adapter a row has is data.  A wave goes through the adapters found among
// 64 of its rows at a time: it multiplies all 64 with one adapter and keeps the
// rows that have it.  Selecting results, not operands, means that infinities or
// NaN in one request's adapter stay in that request's rows.  Runs of one id make
// that one pass, 64 different ids 64 passes.
//
// z is fp32 and the matrix instructions take 16 bits, so in these tiles z is split
// into two bf16 parts (relative error 2^-16, far below the rounding of a 16-bit y;
// bf16 has the range of fp32, so nothing overflows), and an fp16 B_p into two bf16
// parts exactly; all products of the parts are added.  fp32 inputs use fp32
// matrix instructions, and where splits are added afterwards z keeps its 24 bits.
//
// With few tokens the projection is bound by reading W once and the launches:
// the reduction is split over workgroups, the first launch also computes z,
// token by token, in spare workgroups, and a second one adds the splits in
// split order and the tokens' z * B_p.  Batches too small to fill the chip with
// tiles split the reduction and finish in the same way.  Rows of x or W that are
// not 16-byte aligned are copied to padded rows first where the plan finds that
// it pays.
//
// Measured: 16 tokens, 7168 x 4096, 60 adapters of rank 16, bf16: product and z 14
// us (62 MB, 4.4 TB/s), sums 4.6 us; 13824 tokens, 7168 x 2048, runs of 300, f16: z
// 62-71 us, product 0.39-0.40 ms.  Mixed ids cost the large tiles more, one pass over
// 64 rows per adapter: the same call with 60 adapters in any order takes 1.34 ms in
// f16, whose B is split too, and 0.90 in bf16, against 0.44 and 0.40 in runs.
#include <algorithm>

#include "pgg_few.h"
#include "pgg_prep.h"

namespace pgg {

namespace {

struct LoraArgs {
  const void* A;            // x [T, R]
  const void* W;            // weight [R, C]
  const void* A_end;        // where they end
  const void* W_end;
  const void* a;            // [P, rank, R]
  const void* b;            // [P, rank, C]
  const void* a_end;        // where a ends
  const int64_t* ids;       // [T]
  const float* scales;      // [P]
  float* z;                 // [T, rank]
  void* y;                  // [T, C]
  float* part;              // split partials [ksplit, T, C], or NULL
  WsHeader* hdr;
  int64_t R, C, T, kspan;
  int64_t lda, ldw;         // row strides of A and W
  int64_t P;
  int32_t rank;
  int32_t few;              // few tokens: z comes with the product
  int32_t n_slots, n_col_tiles;
};

// The token's adapter, or -1 where it has none (also for an id past the
// adapters, which the header reports).
__device__ __forceinline__ int32_t adapter_of(const LoraArgs& a, int64_t t) {
  const int64_t p = a.ids[t];
  return p >= 0 && p < a.P ? static_cast<int32_t>(p) : -1;
}

// One workgroup: the header, with the smallest token whose id is past the
// adapters.  The loads are independent, eight at a time.
__device__ void check_ids(const LoraArgs& a) {
  __shared__ unsigned long long bad;
  if (threadIdx.x == 0) bad = ~0ull;
  __syncthreads();
  int64_t mine = a.T;
  const int64_t step = static_cast<int64_t>(blockDim.x) * 8;
  for (int64_t t = threadIdx.x; t < a.T; t += step) {
    int64_t id[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) id[u] = a.ids[min(t + u * static_cast<int64_t>(blockDim.x), a.T - 1)];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (id[u] >= a.P) mine = min(mine, min(t + u * static_cast<int64_t>(blockDim.x), a.T - 1));
  }
  if (mine < a.T) atomicMin(&bad, static_cast<unsigned long long>(mine));
  __syncthreads();
  if (threadIdx.x == 0) {
    reset_header(a.hdr);
    if (bad != ~0ull) set_error(a.hdr, PGG_DEV_ADAPTER_RANGE, static_cast<long long>(bad));
  }
}

// One wave: z of token t, ranks r to r + RW - 1, with its adapter p.  Lanes run
// along the reduction, 2 or 4 loads of every row at a time, and their sums are
// added over a fixed tree.
template <class T, int RW>
__device__ __forceinline__ void shrink_ranks(const LoraArgs& a, int64_t t, int32_t p, int r) {
  using E = typename T::elem;
  constexpr int EPC = T::kPerChunk, kUnroll = RW == 1 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  const E* x = static_cast<const E*>(a.A) + t * a.R;
  const E* ar[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i)
    ar[i] = static_cast<const E*>(a.a) + (static_cast<int64_t>(p) * a.rank + min(r + i, a.rank - 1)) * a.R;
  float sum[RW][kUnroll] = {};
  for (int64_t k = lane * EPC; k < a.R; k += 64 * EPC * kUnroll) {
    u32x4_t vx[kUnroll], vw[RW][kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = k + u * 64 * EPC;
      vx[u] = load16_part<T>(x + at, a.R - at, a.A_end);
#pragma unroll
      for (int i = 0; i < RW; ++i) vw[i][u] = load16_part<T>(ar[i] + at, a.R - at, a.a_end);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      E ex[EPC];
      __builtin_memcpy(ex, &vx[u], 16);
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        E ew[EPC];
        __builtin_memcpy(ew, &vw[i][u], 16);
#pragma unroll
        for (int e = 0; e < EPC; ++e) sum[i][u] = fmaf(to_float<T>(ex[e]), to_float<T>(ew[e]), sum[i][u]);
      }
    }
  }
  const float scale = a.scales[p];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    float total = sum[i][0] + sum[i][1];
    if constexpr (kUnroll == 4) total += sum[i][2] + sum[i][3];
#pragma unroll
    for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d);
    if (lane == 0 && r + i < a.rank) a.z[t * a.rank + r + i] = scale * total;
  }
}

// ---------------------------------------------------------------- z, many tokens

// 32 tokens x 16 NB ranks per workgroup (blockIdx.y: which ranks), the
// reduction split over its eight waves and added in wave order.  Bound by
// reading x once: a load takes 64 bytes of 16 rows, and eight waves with 4 x
// (2 + NB) loads each keep them coming.  Workgroups go to the 8 XCDs in turn, and
// each XCD takes a run of tokens, so that the adapter of a request is fetched by
// one L2 and not by eight (2.2 -> 1.8 million lines from memory at 13824 tokens
// of 7168, 60 adapters of rank 16 in runs of 300: 69 us, 198 MB of x alone take
// about 40).  The last workgroup along x checks the ids.
//
// A pass over x for every adapter among the 32 tokens; where there are more
// than kShrinkPasses of them, every token with its own ranks instead.  One
// pass of rank 16 takes about 60 us at the size above, the tokens one by one 330;
// 32 passes took 1100.
template <int NB>
constexpr int kShrinkPasses = 4 * NB;

template <class T, int NB>
__global__ __launch_bounds__(512) void lora_shrink_kernel(LoraArgs a) {
  using E = typename T::elem;
  constexpr int EPC = T::kPerChunk, kStep = 4 * EPC, kUnroll = NB == 4 ? 2 : 4, kWaves = 8;
  __shared__ float red[kWaves][32][16 * NB + 4];
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) check_ids(a);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, lg = lane >> 4;
  const int per_xcd = (gridDim.x - 1 + 7) / 8;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x % 8) * per_xcd + blockIdx.x / 8) * 32;
  if (t0 >= a.T) return;
  const int rows = static_cast<int>(min<int64_t>(32, a.T - t0));
  const int r0 = blockIdx.y * 16 * NB;
  const int64_t R = a.R;
  const int32_t id = (lane & 31) < rows ? adapter_of(a, t0 + (lane & 31)) : -1;
  // the waves take kUnroll steps of the reduction in turn: together they read
  // 8 x 256 successive bytes of every row
  const int64_t steps = (R + kStep - 1) / kStep, whole = R / kStep;
  const E* x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) x[i] = static_cast<const E*>(a.A) + (t0 + min(16 * i + lr, rows - 1)) * R + lg * EPC;
  uint32_t pending = static_cast<uint32_t>(__ballot(id >= 0));
  int adapters = 0;
  for (uint32_t left = pending; left && adapters <= kShrinkPasses<NB>; ++adapters)
    left &= ~static_cast<uint32_t>(__ballot(id == __shfl(id, __builtin_ctz(left))));
  if (adapters > kShrinkPasses<NB>) {
    for (int i = wave; i < rows * 4 * NB; i += kWaves) {
      const int32_t p = __shfl(id, i / (4 * NB));
      const int r = r0 + i % (4 * NB) * 4;
      if (p >= 0 && r < a.rank) shrink_ranks<T, 4>(a, t0 + i / (4 * NB), p, r);
    }
    return;
  }
  while (pending) {
    const int32_t p = __shfl(id, __builtin_ctz(pending));
    const uint32_t mine = static_cast<uint32_t>(__ballot(id == p));
    pending &= ~mine;
    const E* ar[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      ar[b] = static_cast<const E*>(a.a) +
              (static_cast<int64_t>(p) * a.rank + min(r0 + 16 * b + lr, a.rank - 1)) * R + lg * EPC;
    f32x4_t acc[2][NB];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[i][b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t s = wave * kUnroll; s < steps; s += kWaves * kUnroll) {
      u32x4_t fx[kUnroll][2], fw[kUnroll][NB];
      if (s + kUnroll <= whole) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
          for (int i = 0; i < 2; ++i) fx[u][i] = load16(x[i] + (s + u) * kStep);
#pragma unroll
          for (int b = 0; b < NB; ++b) fw[u][b] = load16(ar[b] + (s + u) * kStep);
        }
      } else {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int64_t left = R - (s + u) * kStep - lg * EPC;
#pragma unroll
          for (int i = 0; i < 2; ++i) fx[u][i] = load16_part<T>(x[i] + (s + u) * kStep, left, a.A_end);
#pragma unroll
          for (int b = 0; b < NB; ++b) fw[u][b] = load16_part<T>(ar[b] + (s + u) * kStep, left, a.a_end);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int b = 0; b < NB; ++b) mma_block<T>(acc[i][b], fw[u][b], fx[u][i]);
    }
    // lane: token 16 i + lr, ranks 16 b + 4 lg ..
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b)
        *reinterpret_cast<f32x4_t*>(&red[wave][16 * i + lr][16 * b + 4 * lg]) = acc[i][b];
    __syncthreads();
    const float scale = a.scales[p];
    for (int e = threadIdx.x; e < 32 * 16 * NB; e += 512) {
      const int m = e / (16 * NB), r = e % (16 * NB);
      if (((mine >> m) & 1) && r0 + r < a.rank) {
        float sum = red[0][m][r];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += red[w][m][r];
        a.z[(t0 + m) * a.rank + r0 + r] = scale * sum;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- z, few tokens

// A workgroup takes a token and 4 RW ranks of it, RW to a wave.  RW = 1 makes the
// most workgroups, for the fewest tokens; RW = 4 reads x a quarter as often.
// Workgroup rank_blocks<RW> checks the ids.
template <int RW>
__host__ __device__ __forceinline__ int rank_blocks(int64_t tokens, int32_t rank) {
  return static_cast<int>(tokens) * ((rank + 4 * RW - 1) / (4 * RW));
}

template <class T, int RW>
__device__ __forceinline__ void shrink_token(const LoraArgs& a, int block) {
  if (block == rank_blocks<RW>(a.T, a.rank)) {
    check_ids(a);
    return;
  }
  const int per = (a.rank + 4 * RW - 1) / (4 * RW);
  const int64_t t = block / per;
  const int r = (block % per * 4 + static_cast<int>(threadIdx.x >> 6)) * RW;
  const int32_t p = adapter_of(a, t);
  if (p >= 0 && r < a.rank) shrink_ranks<T, RW>(a, t, p, r);
}

template <class T, int RW>
__global__ __launch_bounds__(256) void lora_shrink_token_kernel(LoraArgs a) {
  shrink_token<T, RW>(a, blockIdx.x);
}

// ---------------------------------------------------------------- the shared product

// 8 fp32 values as two bf16 parts.  The first is the upper half of the value's
// bits, finite for every finite value (rounding would make infinities of those
// above the largest bf16), the second the rest, rounded.  (A NaN out of
// arithmetic has its quiet bit in the upper half.)  An infinite value has no
// rest, and the other operand's rest may be 0 as well: `fin` is the first part
// with zeros for what is not finite, for products with a rest, where infinity
// times 0 would make a NaN that the values' product is not.
__device__ __forceinline__ void split_bf16(const float (&v)[8], u32x4_t& hi, u32x4_t& lo, u32x4_t& fin) {
  uint16_t h[8], l[8], f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    h[e] = static_cast<uint16_t>(__builtin_bit_cast(uint32_t, v[e]) >> 16);
    const float rest = v[e] - to_float<TBf16>(h[e]);
    l[e] = rest == rest ? from_float<TBf16>(rest) : 0;
    f[e] = rest == rest ? h[e] : 0;
  }
  __builtin_memcpy(&hi, h, 16);
  __builtin_memcpy(&lo, l, 16);
  __builtin_memcpy(&fin, f, 16);
}

// The same for 8 elements of B, which need no rounding: fp16 leaves at most 3 bits
// after the first part's, bf16 none.  `fin` and the rest are those of the value
// clamped to the type's range, finite and with its sign.
template <class T>
__device__ __forceinline__ void split_b(const typename T::elem (&b)[8], u32x4_t& hi, u32x4_t& lo, u32x4_t& fin) {
  constexpr float kMost = __is_same(T, TF16) ? 65504.0f : 0x1.fep127f;
  auto upper = [](float v) { return static_cast<uint16_t>(__builtin_bit_cast(uint32_t, v) >> 16); };
  uint16_t h[8], l[8], f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float v = to_float<T>(b[e]), c = __builtin_amdgcn_fmed3f(v, -kMost, kMost);
    h[e] = upper(v);
    f[e] = upper(c);
    l[e] = upper(c - to_float<TBf16>(f[e]));
  }
  __builtin_memcpy(&hi, h, 16);
  __builtin_memcpy(&lo, l, 16);
  __builtin_memcpy(&fin, f, 16);
}

struct LoraOp {
  using Args = LoraArgs;

  template <int BM>
  static __device__ __forceinline__ bool tile(const Args& a, int slot, MTile& t, void*) {
    const int64_t row0 = static_cast<int64_t>(slot) * BM;
    t.g = 0;
    t.row0 = static_cast<int32_t>(row0);
    t.rows = static_cast<int32_t>(min<int64_t>(BM, a.T - row0));
    t.pad = 0;
    return t.rows > 0;
  }

  static __device__ __forceinline__ int64_t src(const Args&, const MTile& t, int r, const void*) {
    return int64_t(t.row0) + r;
  }
  static __device__ __forceinline__ int64_t weight(const Args&, const MTile&) { return 0; }

  static constexpr bool kPaired = false;
  static __device__ __forceinline__ int64_t src_base(const Args&, const MTile& t) { return t.row0; }
  static __device__ __forceinline__ int64_t first_column(int ct, int bn) { return static_cast<int64_t>(ct) * bn; }

  // past the end: a valid column, not stored
  static __device__ __forceinline__ int64_t half_column(const Args& a, int ct, int j, int n) {
    return min<int64_t>(first_column(ct, 256) + j * 128 + n, a.ldw - 8);
  }

  template <int BN>
  static __device__ __forceinline__ ColumnRun column(const Args& a, int ct, int n) {
    const int64_t c = static_cast<int64_t>(ct) * BN + n;
    return {c, a.C - c};
  }

  static __device__ __forceinline__ int64_t columns(const Args& a) { return a.C; }

  // few tokens: workgroups that compute z, and one that checks the ids
  static __host__ __device__ __forceinline__ int extra(const Args& a) {
    return a.few ? rank_blocks<1>(a.T, a.rank) + 1 : 0;
  }
  template <class T>
  static __device__ __forceinline__ void extra_work(const Args& a, int i, void*) {
    shrink_token<T, 1>(a, i);
  }

  // Adds z * B_p of every adapter p found among the wave's rows, four blocks of
  // rows and kStep ranks at a time: the rows' z first, then the adapters in
  // increasing order.  Lane l has row l % B of every block of rows and column
  // l % B of every block of columns, and place l / B along the ranks.
  template <class T, int B, class Acc, int NI, int NJ, class Column>
  static __device__ __forceinline__ void adjust(const Args& a, const MTile& t, int m0, int lane, Acc (&acc)[NI][NJ],
                                                Column column) {
    using E = typename T::elem;
    constexpr int EPC = T::kPerChunk, kStep = 64 / B * EPC, kNone = 0x7FFFFFFF, kGroup = NI < 4 ? NI : 4;
    if (a.part) return;   // split: lora_finish_kernel does it
#pragma unroll
    for (int g = 0; g < NI; g += kGroup) {
      int32_t id[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int row = m0 + (g + i) * B + lane % B;
        id[i] = row < t.rows ? adapter_of(a, int64_t(t.row0) + row) : -1;
      }
      const float* z0 = a.z + (int64_t(t.row0) + m0 + g * B + lane % B) * a.rank;
      for (int r0 = 0; r0 < a.rank; r0 += kStep) {
        const int r = r0 + EPC * (lane / B);
        u32x4_t zh[kGroup], zl[kGroup], zf[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          const float* z = z0 + static_cast<int64_t>(i) * B * a.rank + r;
          float v[EPC];
          if (id[i] >= 0 && r + EPC <= a.rank) {
            __builtin_memcpy(v, z, sizeof(v));
          } else {
#pragma unroll
            for (int e = 0; e < EPC; ++e) v[e] = id[i] >= 0 && r + e < a.rank ? z[e] : 0.0f;
          }
          if constexpr (EPC == 8) split_bf16(v, zh[i], zl[i], zf[i]);
          else __builtin_memcpy(&zh[i], v, 16);
        }
        for (int32_t last = -1;;) {
          int32_t p = kNone;
#pragma unroll
          for (int i = 0; i < kGroup; ++i) p = id[i] > last ? min(p, id[i]) : p;
#pragma unroll
          for (int d = B / 2; d; d >>= 1) p = min(p, __shfl_xor(p, d));
          p = __builtin_amdgcn_readfirstlane(p);
          if (p == kNone) break;
          last = p;
          const E* b = static_cast<const E*>(a.b) + (static_cast<int64_t>(p) * a.rank + r) * a.C;
          E raw[NJ][EPC];
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int64_t c = column(j) + lane % B;
#pragma unroll
            for (int e = 0; e < EPC; ++e) raw[j][e] = c < a.C && r + e < a.rank ? b[e * a.C + c] : E(0);
          }
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            u32x4_t bh, bl, bf;
            if constexpr (EPC == 8) {
              split_b<T>(raw[j], bh, bl, bf);
            } else {
              __builtin_memcpy(&bh, raw[j], 16);
            }
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
              Acc d;
#pragma unroll
              for (int e = 0; e < B * B / 64; ++e) d[e] = 0.0f;
              if constexpr (EPC == 8) {
                mma_block<TBf16>(d, bh, zh[i]);
                mma_block<TBf16>(d, bf, zl[i]);
                if constexpr (__is_same(T, TF16)) {
                  mma_block<TBf16>(d, bl, zf[i]);
                  mma_block<TBf16>(d, bl, zl[i]);   // up to 2^-14: both parts are truncated, not rounded
                }
              } else {
                mma<T>(d, bh, zh[i]);
              }
#pragma unroll
              for (int e = 0; e < B * B / 64; ++e)
                acc[g + i][j][e] = id[i] == p ? acc[g + i][j][e] + d[e] : acc[g + i][j][e];
            }
            __builtin_amdgcn_sched_barrier(0);   // one block of columns at a time: registers
          }
        }
      }
    }
  }

  template <class T>
  struct Side {};
  template <class T>
  static __device__ __forceinline__ Side<T> fetch(const Args&, const MTile&, int, int64_t, int64_t) {
    return {};
  }

  template <class T>
  static __device__ __forceinline__ void piece(const Args& a, const MTile& t, int m, int64_t c, int64_t left,
                                               const float (&v)[8], const Side<T>&) {
    const int64_t token = int64_t(t.row0) + m;
    if (a.part)
      store8<TF32, false>(a.part + (static_cast<int64_t>(t.pad) * a.T + token) * a.C + c, left, v);
    else
      store8<T>(static_cast<typename T::elem*>(a.y) + token * a.C + c, left, v);
  }
};

// Adds the splits' partial products in split order and the token's z * B_p, for
// V successive columns per thread (V = 4: C is a multiple of 4).
template <class T, int V>
__global__ __launch_bounds__(256) void lora_finish_kernel(LoraArgs a, int32_t ksplit) {
  using E = typename T::elem;
  struct alignas(V * 4) Floats { float v[V]; };
  struct alignas(sizeof(E)) Elems { E v[V]; };
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t n = a.T * a.C;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n / V; i += step) {
    const int64_t e = i * V, t = e / a.C, c = e - t * a.C;
    Floats sum = *reinterpret_cast<const Floats*>(a.part + e);
#pragma unroll 8
    for (int32_t s = 1; s < ksplit; ++s) {
      const Floats f = *reinterpret_cast<const Floats*>(a.part + s * n + e);
#pragma unroll
      for (int k = 0; k < V; ++k) sum.v[k] += f.v[k];
    }
    const int32_t p = adapter_of(a, t);
    if (p >= 0) {
      const E* b = static_cast<const E*>(a.b) + static_cast<int64_t>(p) * a.rank * a.C + c;
      Floats d = {};
#pragma unroll 8
      for (int32_t r = 0; r < a.rank; ++r) {
        Elems x;
        __builtin_memcpy(&x, b + r * a.C, sizeof(x));
        const float z = a.z[t * a.rank + r];
#pragma unroll
        for (int k = 0; k < V; ++k) d.v[k] = fmaf(z, to_float<T>(x.v[k]), d.v[k]);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) sum.v[k] += d.v[k];
    }
    Elems y;
#pragma unroll
    for (int k = 0; k < V; ++k) y.v[k] = from_float<T>(sum.v[k]);
    __builtin_memcpy(static_cast<E*>(a.y) + e, &y, sizeof(y));
  }
}

template <class T, int V>
hipError_t launch_finish(const LoraArgs& a, int32_t ksplit, hipStream_t s) {
  const int64_t blocks = std::min<int64_t>((a.T * a.C / V + 255) / 256, 4096);
  hipLaunchKernelGGL((lora_finish_kernel<T, V>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a, ksplit);
  return hipGetLastError();
}

template <class T, int BM, int BN, int WM, int WN>
hipError_t launch_reg(LoraArgs a, const LoraPlan& p, hipStream_t s) {
  a.n_slots = static_cast<int32_t>((a.T + BM - 1) / BM);
  a.n_col_tiles = static_cast<int32_t>((a.C + BN - 1) / BN);
  return launch_nn_reg<T, LoraOp, BM, BN, WM, WN, 2>(a, p.ksplit, s);
}

template <class T, int NB>
hipError_t launch_shrink(const LoraArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.T + 32 * 8 - 1) / (32 * 8) * 8 + 1),
                  static_cast<unsigned>((a.rank + 16 * NB - 1) / (16 * NB)));
  hipLaunchKernelGGL((lora_shrink_kernel<T, NB>), grid, dim3(512), 0, s, a);
  return hipGetLastError();
}

template <class T, int RW>
hipError_t launch_shrink_token(const LoraArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((lora_shrink_token_kernel<T, RW>), dim3(static_cast<unsigned>(rank_blocks<RW>(a.T, a.rank)) + 1),
                     dim3(256), 0, s, a);
  return hipGetLastError();
}

// Up to this many tokens and ranks z is computed token by token: a token reads
// its whole adapter, but workgroups are many, their reads contiguous, and the
// order of the ids does not matter.  Whole calls in us, bf16, K 4096, N 512, 16
// adapters, token by token and in tiles, runs of 300 ids and mixed ones:
//   2048 tokens, rank 16: 62 and 64, mixed 60 and 145; rank 64: 107 and 93, 107
//     and 398; rank 256: 292 and 122, 294 and 463
//   4096 tokens, rank 16: 82 and 71, mixed 80 and 151
constexpr int64_t kTokenByToken = 2048, kTokenRanks = 2048 * 64;
bool token_by_token(const LoraArgs& a) { return a.T <= kTokenByToken && a.T * a.rank <= kTokenRanks; }

// What the direct-to-LDS kernels need: 16-byte rows, and 32-bit byte offsets
// into 256 rows of x and 64 rows of W.
bool direct_rows(const LoraArgs& a) {
  auto fits = [](const void* ptr, int64_t ld) { return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld % 8 == 0; };
  return fits(a.A, a.lda) && fits(a.W, a.ldw) && a.lda < (int64_t(1) << 23) && a.ldw < (int64_t(1) << 25);
}

template <class T>
hipError_t launch_typed(const LoraPlan& p, LoraArgs a, void* padded_x, void* padded_w, hipStream_t s) {
  const bool direct = T::kPerChunk == 8 && direct_rows(a);
  hipError_t e = hipSuccess;
  // z: beside the product, token by token, or in tiles
  if (!a.few && token_by_token(a)) e = launch_shrink_token<T, 4>(a, s);
  else if (!a.few)
    e = a.rank <= 16 ? launch_shrink<T, 1>(a, s) : a.rank <= 32 ? launch_shrink<T, 2>(a, s) : launch_shrink<T, 4>(a, s);
  if (e != hipSuccess) return e;
  if constexpr (T::kPerChunk == 8) {
    a.n_col_tiles = static_cast<int32_t>((a.C + 255) / 256);
    if (a.few && direct) {
      a.n_slots = static_cast<int32_t>((a.T + 63) / 64);
      e = a.T <= 32 ? launch_few<T, LoraOp, 32>(a, p.ksplit, s) : launch_few<T, LoraOp, 64>(a, p.ksplit, s);
    } else if (a.few) {
      e = launch_reg<T, 32, 256, 1, 4>(a, p, s);
    } else {
      LoraArgs b = a;   // with the operands that the plan lays out anew
      if (p.pad_a) {
        b.A = padded_x;
        b.lda = p.lda;
      }
      if (p.pad_w) {
        b.W = padded_w;
        b.ldw = p.ldw;
      }
      b.n_slots = static_cast<int32_t>((a.T + 255) / 256);
      if (!p.pipe || !direct_rows(b)) {
        e = launch_reg<T, 128, 128, 2, 2>(a, p, s);
      } else {
        if (p.pad_a) e = launch_pad_rows(a.A, padded_x, a.T, a.R, b.lda, s);
        if (e == hipSuccess && p.pad_w) e = launch_pad_rows(a.W, padded_w, a.R, a.C, b.ldw, s);
        if (e == hipSuccess) e = launch_pipe<T, LoraOp, false>(b, p.ksplit, s);
      }
    }
  } else {
    e = a.few ? launch_reg<T, 32, 128, 1, 4>(a, p, s) : launch_reg<T, 128, 128, 2, 2>(a, p, s);
  }
  if (e != hipSuccess || !a.part) return e;
  // four columns per thread once that leaves a thread for every lane of the chip's 1024 SIMDs
  return a.C % 4 == 0 && a.T * a.C >= 4 * 65536 ? launch_finish<T, 4>(a, p.ksplit, s)
                                                : launch_finish<T, 1>(a, p.ksplit, s);
}

}  // namespace

hipError_t launch_lora(const LoraPlan& p, const void* x, const void* weight, const void* a, const void* b,
                       const int64_t* ids, const float* scales, void* y, void* ws, hipStream_t s) {
  char* base = static_cast<char*>(ws);
  LoraArgs g;
  g.A = x;
  g.W = weight;
  g.a = a;
  g.b = b;
  g.ids = ids;
  g.scales = scales;
  g.z = reinterpret_cast<float*>(base + p.off_z);
  g.y = y;
  g.few = p.few;
  g.part = p.few || p.ksplit > 1 ? reinterpret_cast<float*>(base + p.off_part) : nullptr;
  g.hdr = reinterpret_cast<WsHeader*>(base + p.off_header);
  const size_t es = p.dtype == PGG_F32 ? 4 : 2;
  g.A_end = static_cast<const char*>(x) + es * p.T * p.K;
  g.W_end = static_cast<const char*>(weight) + es * p.K * p.N;
  g.a_end = static_cast<const char*>(a) + es * p.P * p.rank * p.K;
  g.R = p.K;
  g.lda = p.K;
  g.ldw = p.N;
  g.C = p.N;
  g.T = p.T;
  g.kspan = p.kspan;
  g.P = p.P;
  g.rank = p.rank;
  void* px = base + p.off_pad_a;
  void* pw = base + p.off_pad_w;
  if (p.dtype == PGG_F32) return launch_typed<TF32>(p, g, px, pw, s);
  return p.dtype == PGG_BF16 ? launch_typed<TBf16>(p, g, px, pw, s) : launch_typed<TF16>(p, g, px, pw, s);
}

}  // namespace pgg
