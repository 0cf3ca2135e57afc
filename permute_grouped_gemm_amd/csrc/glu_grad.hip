// Gradient through the experts' gated product, from the gradient of the
// products that follow it:
//
//   dh[i, f]       = sum_d grad_y[i, d] * W[g(i), f, d]       W[g]: the expert's second matrix, [F, D]
//   grad_gate[i, f] = dh * up[i, f] * act'(gate[i, f])
//   grad_up[i, f]   = dh * act(gate[i, f])
//   h[i, f]         = act(gate[i, f]) * up[i, f]              (recomputed, for the gradient of W)
//
// dh stays in the fp32 accumulators: a tile reads the saved products (gate |
// up)[M, 2F] at its place and stores the three results.
//
// Both operands hold the reduction d contiguously, the layout that MFMA
// operands take, so tiles are staged in LDS as rows of 16-byte chunks, chunk c
// of row r at c ^ ((r >> 1) & 7).  Calls with too few tiles to fill the chip
// split the reduction; the fp32 partial products of the splits go to the
// workspace and a second kernel adds them in split order.
//
// Many rows are bound by the matrix instructions (pgg_pipe.h: 110592 rows x 7168 x
// 2048, f16, 3.0 ms), few by reading the weights: 666 rows in 59 of 64 experts, D
// 2039, F 1403, bf16, 338 MB of them in 94 us (3.6 TB/s, rows at any address through
// registers) and 6.4 us for the sums; 16 experts of 24 rows, D 4096, F 1408, bf16,
// 185 MB in a call of 54 us.  fp32, 8 experts of 1024 rows, D 4096, F 2048: 1.18 ms,
// 116 TFLOP/s.
// grad and h are rounded once, from fp32.
#include <algorithm>

#include "pgg_act.h"
#include "pgg_local.h"
#include "pgg_pipe.h"

namespace pgg {

namespace {

struct GluGradArgs {
  const void* A;            // grad_y [M, R]
  const void* W;            // weight [G, F, R]
  const void* A_end;        // where they end
  const void* W_end;
  const void* gate_up;      // [M, C]
  const WsHeader* hdr;
  const MTile* tiles;
  void* grad;               // [M, C]
  void* h;                  // [M, F] or NULL
  float* part;              // split partials of dh [ksplit, M, F], or NULL
  int64_t M;
  int64_t R, C, F, kspan;
  int64_t lda, ldw;         // row strides of A and W
  int32_t bm;               // rows of a table entry
  int32_t n_slots, n_col_tiles;
  // without tables: group_list itself, and the preparation for the error word
  int32_t local;
  const int64_t* gl;
  PrepArgs prep;
  WsView ws;
};

template <int ACT>
struct GluGradOp {
  using Args = GluGradArgs;
  static constexpr bool kPaired = false;

  template <int BM>
  static __device__ __forceinline__ bool tile(const Args& a, int slot, MTile& t, void* lds) {
    if constexpr (BM <= 64) {
      if (a.local) {
        const bool found = local_tile(a.gl, a.prep.G, a.M, BM, slot, t, static_cast<int32_t*>(lds));
        __syncthreads();   // before LDS is used again
        return found;
      }
    }
    if (a.hdr->err != kNoError) return false;
    const int sub = a.bm / BM;   // tiles to a table entry
    const int entry = slot / sub;
    if (entry >= a.hdr->n_tiles) return false;
    t = a.tiles[entry];
    const int skip = (slot - entry * sub) * BM;
    t.row0 += skip;
    t.rows = min(t.rows - skip, BM);
    return t.rows > 0;
  }

  static __device__ __forceinline__ int64_t src_base(const Args&, const MTile& t) { return t.row0; }
  static __device__ __forceinline__ int64_t src(const Args&, const MTile& t, int r, const void*) {
    return int64_t(t.row0) + r;
  }
  static __device__ __forceinline__ int64_t weight(const Args& a, const MTile& t) { return t.g * a.F * a.ldw; }
  static __device__ __forceinline__ int64_t first_column(int ct, int bn) { return static_cast<int64_t>(ct) * bn; }

  static __device__ __forceinline__ int64_t columns(const Args& a) { return a.F; }

  template <class T, int B, class Acc, class Column>
  static __device__ __forceinline__ void adjust(const Args&, const MTile&, int, int, Acc&, Column) {}

  // 8 gate and 8 up values
  template <class T>
  struct Side {
    Raw8<T> gate, up;
  };

  template <class T>
  static __device__ __forceinline__ Side<T> fetch(const Args& a, const MTile& t, int m, int64_t f, int64_t left) {
    if (a.part) return {};
    const typename T::elem* p = static_cast<const typename T::elem*>(a.gate_up) + int64_t(t.row0 + m) * a.C + f;
    return {load_raw8<T>(p, left), load_raw8<T>(p + a.F, left)};
  }

  template <class T>
  static __device__ __forceinline__ void piece(const Args& a, const MTile& t, int m, int64_t f, int64_t left,
                                               const float (&dh)[8], const Side<T>& side) {
    using E = typename T::elem;
    const int64_t row = t.row0 + m, at = row * a.C + f;
    if (a.part) {
      store8<TF32, false>(a.part + (static_cast<int64_t>(t.pad) * a.M + row) * a.F + f, left, dh);
      return;
    }
    float gate[8], up[8], h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float value, slope;
      activate_grad<ACT>(to_float<T>(side.gate.e[e]), value, slope);
      const float u = to_float<T>(side.up.e[e]);
      gate[e] = dh[e] * u * slope;
      up[e] = dh[e] * value;
      h[e] = value * u;
    }
    store8<T>(static_cast<E*>(a.grad) + at, left, gate);
    store8<T>(static_cast<E*>(a.grad) + at + a.F, left, up);
    if (a.h) store8<T>(static_cast<E*>(a.h) + row * a.F + f, left, h);
  }
};

// Through registers: every type and alignment.  Rows and columns past the
// tile's repeat valid ones and are not stored; elements past the reduction are
// zero in both operands.
template <class T, class Op, int BM, int BN, int WM, int WN, int EU>
__global__ __launch_bounds__(WM * WN * 64) __attribute__((amdgpu_waves_per_eu(EU, EU)))
void glu_grad_reg_kernel(GluGradArgs a) {
  using E = typename T::elem;
  constexpr int NT = WM * WN * 64;
  constexpr int EPC = T::kPerChunk;
  constexpr int kChunks = 8;
  constexpr int BK = kChunks * EPC;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int FM = WTM / 32, FN = WTN / 32;
  constexpr int A_CHUNKS = BM * kChunks, B_CHUNKS = BN * kChunks;
  constexpr int A_PER_T = A_CHUNKS / NT, B_PER_T = B_CHUNKS / NT;
  static_assert(WTM % 32 == 0 && WTN % 32 == 0, "whole 32x32 blocks per wave");
  static_assert(A_CHUNKS % NT == 0 && B_CHUNKS % NT == 0, "a stage splits evenly");
  __shared__ u32x4_t lds[2][A_CHUNKS + B_CHUNKS];

  if (BM <= 64 && a.local && blockIdx.x == gridDim.x - 1) {   // the one workgroup that is no tile's
    if (blockIdx.y == 0) {
      long long* scratch = reinterpret_cast<long long*>(&lds[0][0]);
      reset_header(a.ws.hdr);
      __syncthreads();
      groups_phase(a.prep, a.gl, a.ws, scratch, scratch + blockDim.x);
    }
    return;
  }
  int slot, ct;
  if (!tile_place(a, slot, ct)) return;
  MTile tile;
  if (!Op::template tile<BM>(a, slot, tile, lds)) return;
  tile.pad = blockIdx.y;
  const int64_t col0 = Op::first_column(ct, BN);
  const int64_t kbeg = static_cast<int64_t>(blockIdx.y) * a.kspan;   // this workgroup's split
  const int64_t D = min<int64_t>(a.R - kbeg, a.kspan);

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int wm = wave % WM, wn = wave / WM;
  const int lr = lane & 31, lh = lane >> 5;

  const E* arow[A_PER_T];
  const E* brow[B_PER_T];
#pragma unroll
  for (int s = 0; s < A_PER_T; ++s) {
    const int q = tid + s * NT;
    const int64_t row = Op::src(a, tile, min(q / kChunks, tile.rows - 1), nullptr);
    arow[s] = static_cast<const E*>(a.A) + row * a.lda + kbeg + (q % kChunks) * EPC;
  }
#pragma unroll
  for (int s = 0; s < B_PER_T; ++s) {
    const int q = tid + s * NT;
    const int64_t f = min<int64_t>(col0 + q / kChunks, a.F - 1);
    brow[s] = static_cast<const E*>(a.W) + Op::weight(a, tile) + f * a.ldw + kbeg + (q % kChunks) * EPC;
  }

  u32x4_t ra[A_PER_T], rb[B_PER_T];
  auto load_stage = [&](int kt) {
    const int64_t k0 = static_cast<int64_t>(kt) * BK;
    if (k0 + BK <= D) {
#pragma unroll
      for (int s = 0; s < A_PER_T; ++s) ra[s] = load16(arow[s] + k0);
#pragma unroll
      for (int s = 0; s < B_PER_T; ++s) rb[s] = load16(brow[s] + k0);
    } else {
#pragma unroll
      for (int s = 0; s < A_PER_T; ++s)
        ra[s] = load16_part<T>(arow[s] + k0, D - k0 - (tid + s * NT) % kChunks * EPC, a.A_end);
#pragma unroll
      for (int s = 0; s < B_PER_T; ++s)
        rb[s] = load16_part<T>(brow[s] + k0, D - k0 - (tid + s * NT) % kChunks * EPC, a.W_end);
    }
  };
  auto store_stage = [&](int buf) {
#pragma unroll
    for (int s = 0; s < A_PER_T; ++s) {
      const int q = tid + s * NT;
      lds[buf][q / kChunks * kChunks + a_slot(q / kChunks, q % kChunks)] = ra[s];
    }
#pragma unroll
    for (int s = 0; s < B_PER_T; ++s) {
      const int q = tid + s * NT;
      lds[buf][A_CHUNKS + q / kChunks * kChunks + a_slot(q / kChunks, q % kChunks)] = rb[s];
    }
  };

  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  auto compute = [&](int buf) {
    const u32x4_t* As = lds[buf];
    const u32x4_t* Bs = lds[buf] + A_CHUNKS;
    u32x4_t fa[2][FM], fb[2][FN];
    auto load_frags = [&](int q, u32x4_t (&xa)[FM], u32x4_t (&xb)[FN]) {
      const int sl = a_slot(lr, 2 * q + lh);
#pragma unroll
      for (int i = 0; i < FM; ++i) xa[i] = As[(wm * WTM + i * 32 + lr) * kChunks + sl];
#pragma unroll
      for (int j = 0; j < FN; ++j) xb[j] = Bs[(wn * WTN + j * 32 + lr) * kChunks + sl];
    };
    load_frags(0, fa[0], fb[0]);
#pragma unroll
    for (int q = 0; q < kChunks / 2; ++q) {
      if (q + 1 < kChunks / 2) load_frags(q + 1, fa[(q + 1) & 1], fb[(q + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) mma<T>(acc[i][j], fb[q & 1][j], fa[q & 1][i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  const int nk = static_cast<int>((D + BK - 1) / BK);
  load_stage(0);
  store_stage(0);
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    if (kt + 1 < nk) load_stage(kt + 1);
    compute(kt & 1);
    if (kt + 1 < nk) store_stage((kt & 1) ^ 1);
    __syncthreads();
  }
  store_blocks<T, Op, false, FM, FN>(a, tile, col0 + wn * WTN, wm * WTM, lane, acc);
}

template <class T, int BM, int WM, int EU, int ACT>
hipError_t launch_reg(const Plan& p, GluGradArgs a, hipStream_t s) {
  constexpr int BN = 128;
  a.n_slots = p.max_tiles * (p.bm / BM);
  a.n_col_tiles = static_cast<int32_t>((a.F + BN - 1) / BN);
  const unsigned blocks = tile_blocks(a) + (BM <= 64 && a.local ? 1 : 0);
  hipLaunchKernelGGL((glu_grad_reg_kernel<T, GluGradOp<ACT>, BM, BN, WM, 4 / WM, EU>), dim3(blocks, p.ksplit),
                     dim3(256), 0, s, a);
  return hipGetLastError();
}

// What the direct-to-LDS kernel needs: 16-byte rows, and 32-bit byte offsets
// into 256 rows of either operand.
bool direct(const GluGradArgs& a) {
  auto fits = [](const void* ptr, int64_t ld) { return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld % 8 == 0; };
  return fits(a.A, a.lda) && fits(a.W, a.ldw) && a.lda < (int64_t(1) << 23);
}

template <class T, int ACT>
hipError_t launch_typed(const Plan& p, GluGradArgs a, void* padded_a, void* padded_w, hipStream_t s) {
  if (p.bm == 32) return launch_reg<T, 32, 1, 4, ACT>(p, a, s);
  if (p.bm == 64) return launch_reg<T, 64, 2, 3, ACT>(p, a, s);
  if constexpr (T::kPerChunk == 8) {
    GluGradArgs b = a;   // with the operands that the plan lays out anew
    if (p.pad_a) {
      b.A = padded_a;
      b.W = padded_w;
      b.lda = b.ldw = p.lda;
    }
    if (direct(b)) {
      hipError_t e = hipSuccess;
      if (p.pad_a) {
        e = launch_pad_rows(a.A, padded_a, p.M, a.R, b.lda, s);
        if (e == hipSuccess) e = launch_pad_rows(a.W, padded_w, p.G * a.F, a.R, b.ldw, s);
      }
      b.n_slots = p.max_tiles;
      b.n_col_tiles = static_cast<int32_t>((a.F + 255) / 256);
      return e == hipSuccess ? launch_pipe<T, GluGradOp<ACT>, true>(b, p.ksplit, s) : e;
    }
  }
  return launch_reg<T, 128, 2, 2, ACT>(p, a, s);
}

// Adds the splits' partial products in split order and stores the gradients.
template <class T, int ACT>
__global__ __launch_bounds__(256) void glu_grad_finish_kernel(GluGradArgs a, int32_t ksplit) {
  using E = typename T::elem;
  if (a.hdr->err != kNoError) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t n = a.M * a.F;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < n; e += step) {
    const int64_t row = e / a.F, at = row * a.C + (e - row * a.F);
    float dh = a.part[e];
#pragma unroll 8
    for (int32_t s = 1; s < ksplit; ++s) dh += a.part[s * n + e];
    const E* gu = static_cast<const E*>(a.gate_up);
    const float up = to_float<T>(gu[at + a.F]);
    float value, slope;
    activate_grad<ACT>(to_float<T>(gu[at]), value, slope);
    static_cast<E*>(a.grad)[at] = from_float<T>(dh * up * slope);
    static_cast<E*>(a.grad)[at + a.F] = from_float<T>(dh * value);
    if (a.h) static_cast<E*>(a.h)[e] = from_float<T>(value * up);
  }
}

template <class T, int ACT>
hipError_t launch_all(const Plan& p, const GluGradArgs& a, void* pa, void* pw, hipStream_t s) {
  const hipError_t e = launch_typed<T, ACT>(p, a, pa, pw, s);
  if (e != hipSuccess || p.ksplit == 1) return e;
  const int64_t blocks = std::min<int64_t>((a.M * a.F + 255) / 256, 2048);
  hipLaunchKernelGGL((glu_grad_finish_kernel<T, ACT>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a,
                     p.ksplit);
  return hipGetLastError();
}

template <int ACT>
hipError_t launch_act(const Plan& p, const GluGradArgs& a, void* pa, void* pw, hipStream_t s) {
  if (p.dtype == PGG_F32) return launch_all<TF32, ACT>(p, a, pa, pw, s);
  return p.dtype == PGG_BF16 ? launch_all<TBf16, ACT>(p, a, pa, pw, s) : launch_all<TF16, ACT>(p, a, pa, pw, s);
}

}  // namespace

hipError_t launch_glu_grad(const Plan& p, int32_t act, const void* grad_y, const void* weight, const void* gate_up,
                           const int64_t* group_list, void* grad, void* h, void* ws, hipStream_t s) {
  const WsView w = ws_view(p, ws);
  GluGradArgs a;
  a.A = grad_y;
  a.W = weight;
  a.gate_up = gate_up;
  a.hdr = w.hdr;
  a.tiles = w.tiles;
  a.grad = grad;
  a.h = h;
  const size_t es = p.dtype == PGG_F32 ? 4 : 2;
  a.A_end = static_cast<const char*>(grad_y) + es * p.M * p.N;
  a.W_end = static_cast<const char*>(weight) + es * p.G * p.K * p.N;
  a.R = p.N;          // the plan keeps the reduction in N and the columns in K
  a.F = p.K;
  a.C = 2 * p.K;
  a.kspan = p.kspan;
  a.M = p.M;
  a.part = p.ksplit > 1 ? w.ring : nullptr;
  a.lda = a.ldw = p.N;
  a.bm = p.bm;
  a.local = p.local;
  a.gl = group_list;
  a.prep = prep_args(p);
  a.ws = w;
  void* pa = static_cast<char*>(ws) + p.off_pad_a;
  void* pw = static_cast<char*>(ws) + p.off_pad_w;
  return act == PGG_ACT_SILU ? launch_act<PGG_ACT_SILU>(p, a, pa, pw, s)
                             : launch_act<PGG_ACT_GELU_TANH>(p, a, pa, pw, s);
}

}  // namespace pgg
