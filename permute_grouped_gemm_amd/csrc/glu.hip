// Gated product of the experts, the first half of a gated feed-forward layer:
//
//   (gate | up)[i, :] = x[p(i) / topK, :] * W[g(i)]      W[g] is [K, 2F]: gate columns, then up columns
//   h[i, f]           = act(gate[i, f]) * up[i, f]
//
// for the expanded rows i of the routing index (rows of one expert are
// neighbours, experts hold any number of them).  Neither the permuted copy of
// x nor, unless the caller wants it for the backward pass, the [M, 2F] product
// is stored: a tile of the product holds gate columns in its even blocks of 32
// and the matching up columns in its odd ones, so a wave has both of a pair in
// registers and the activation is part of the store.  h is rounded once, from
// the fp32 accumulators.
//
// Many rows per expert are bound by the matrix instructions, few by reading
// the used experts' weights once.  The tiles and the pipelines are those of
// pgg_nn.h; with few rows per expert the reduction is split over workgroups so
// that enough of them stream weights, the fp32 partial products of the splits
// go to the workspace, and a second kernel adds them in split order and applies
// the activation.  Rows of x or W that are not 16-byte aligned are copied to
// padded rows first where the product is large enough to pay for it (the plan
// says so); otherwise the tiles that load through registers take them.
//
// Measured calls: 16384 rows x 7168 x 4096, bf16, 16 experts, 0.83 ms; 128 rows, 12
// experts used, the same widths, 127 us; 128 rows, K 256, F 64, fp32, two launches
// of 7.6 and 2.0 us.
#include <algorithm>

#include "pgg_act.h"
#include "pgg_few.h"
#include "pgg_local.h"

namespace pgg {

namespace {

struct GluArgs {
  const void* A;            // x [batch, R]
  const void* W;            // weight [G, R, C]
  const void* A_end;        // where they end
  const void* W_end;
  const WsHeader* hdr;
  const MTile* tiles;
  const int32_t* ori;       // expanded row -> original position
  void* h;                  // [M, F]
  void* gate_up;            // [M, C] or NULL
  float* part;              // split partials [ksplit, M, C], or NULL
  int64_t R, C, F, M, kspan;
  int64_t lda, ldw, Fw;     // row strides of A and W; columns from gate to up in a W row
  uint32_t topk;
  int32_t bm;               // rows of a table entry
  int32_t n_slots, n_col_tiles;
  // without tables: group_list and the index themselves, and the preparation for the error word
  int32_t local;
  const int64_t* eri;
  const int64_t* gl;
  PrepArgs prep;
  WsView ws;
};

template <int ACT>
struct GluOp {
  using Args = GluArgs;

  template <int BM>
  static __device__ __forceinline__ bool tile(const Args& a, int slot, MTile& t, void* lds) {
    if constexpr (BM <= 64) {
      if (a.local) {
        int32_t* words = static_cast<int32_t*>(lds);
        if (!local_tile(a.gl, a.prep.G, a.M, BM, slot, t, words)) return false;
        local_rows(a.eri, a.M, a.prep.row_idx_type, t, words + kLocalWords);
        return true;
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

  static __device__ __forceinline__ int64_t src(const Args& a, const MTile& t, int r, const void* lds) {
    const int32_t p = a.local ? static_cast<const int32_t*>(lds)[kLocalWords + r] : a.ori[t.row0 + r];
    return static_cast<uint32_t>(p) / a.topk;
  }

  static __device__ __forceinline__ int64_t weight(const Args& a, const MTile& t) {
    return t.g * a.R * a.ldw;
  }

  static constexpr bool kPaired = true;
  static __device__ __forceinline__ int64_t src_base(const Args&, const MTile&) { return 0; }
  static __device__ __forceinline__ int64_t first_column(int ct, int bn) { return static_cast<int64_t>(ct) * (bn / 2); }

  template <int BN>
  static __device__ __forceinline__ ColumnRun column(const Args& a, int ct, int n) {
    const int64_t f = first_column(ct, BN) + (n >> 6) * 32 + (n & 31);
    return {f + ((n >> 5) & 1) * a.F, a.F - f};
  }

  // run j (0: gate, 1: up), column n; past the end: a valid one, not stored
  static __device__ __forceinline__ int64_t half_column(const Args& a, int ct, int j, int n) {
    return j * a.Fw + min<int64_t>(first_column(ct, 256) + n, a.Fw - 8);
  }

  static __device__ __forceinline__ int64_t columns(const Args& a) { return a.F; }
  static __host__ __device__ __forceinline__ int extra(const Args& a) { return a.local; }
  template <class T>
  static __device__ __forceinline__ void extra_work(const Args& a, int, void* lds) {
    prep_block(a.prep, a.eri, a.gl, a.ws, static_cast<long long*>(lds));
  }

  template <class T, int B, class Acc, class Column>
  static __device__ __forceinline__ void adjust(const Args&, const MTile&, int, int, Acc&, Column) {}

  template <class T>
  static __device__ __forceinline__ void piece(const Args& a, const MTile& t, int m, int64_t f, int64_t left,
                                               const float (&gate)[8], const float (&up)[8]) {
    using E = typename T::elem;
    const int64_t row = t.row0 + m;
    if (a.part) {
      float* p = a.part + (static_cast<int64_t>(t.pad) * a.M + row) * a.C + f;
      store8<TF32, false>(p, left, gate);
      store8<TF32, false>(p + a.F, left, up);
      return;
    }
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = activate<ACT>(gate[e]) * up[e];
    store8<T>(static_cast<E*>(a.h) + row * a.F + f, left, h);
    if (a.gate_up) {
      E* p = static_cast<E*>(a.gate_up) + row * a.C + f;
      store8<T>(p, left, gate);
      store8<T>(p + a.F, left, up);
    }
  }
};

// Adds the splits' partial products in split order and stores h (and the products).
template <class T, int ACT>
__global__ __launch_bounds__(256) void glu_finish_kernel(GluArgs a, int32_t ksplit) {
  using E = typename T::elem;
  if (a.hdr->err != kNoError) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t n = a.M * a.F, plane = a.M * a.C;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < n; e += step) {
    const int64_t row = e / a.F, f = e - row * a.F;
    const float* p = a.part + row * a.C + f;
    float gate = p[0], up = p[a.F];
    for (int32_t s = 1; s < ksplit; ++s) {
      gate += p[s * plane];
      up += p[s * plane + a.F];
    }
    static_cast<E*>(a.h)[e] = from_float<T>(activate<ACT>(gate) * up);
    if (a.gate_up) {
      static_cast<E*>(a.gate_up)[row * a.C + f] = from_float<T>(gate);
      static_cast<E*>(a.gate_up)[row * a.C + a.F + f] = from_float<T>(up);
    }
  }
}

template <class T, int BM, int BN, int WM, int WN, int EU, int ACT>
hipError_t launch_reg(const Plan& p, GluArgs a, hipStream_t s) {
  a.n_slots = p.max_tiles * (p.bm / BM);
  a.n_col_tiles = static_cast<int32_t>((a.F + BN / 2 - 1) / (BN / 2));
  return launch_nn_reg<T, GluOp<ACT>, BM, BN, WM, WN, EU>(a, p.ksplit, s);
}

// What the direct-to-LDS kernels need: 16-byte rows, and 32-bit byte offsets
// into all of x and into 64 rows of W.
bool direct(const Plan& p, const GluArgs& a) {
  auto fits = [](const void* ptr, int64_t ld) { return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld % 8 == 0; };
  return fits(a.A, a.lda) && fits(a.W, a.ldw) && a.Fw % 8 == 0 && p.batch * a.lda < (int64_t(1) << 31) - 64 &&
         a.ldw < (int64_t(1) << 25);
}

template <class T, int ACT>
hipError_t launch_16(const Plan& p, GluArgs a, void* padded_x, void* padded_w, hipStream_t s) {
  a.n_slots = p.max_tiles;
  a.n_col_tiles = static_cast<int32_t>((a.F + 127) / 128);
  if (p.regime == kStream) {
    if (!direct(p, a)) return launch_reg<T, 32, 256, 1, 4, 2, ACT>(p, a, s);
    return p.bm == 32 ? launch_few<T, GluOp<ACT>, 32>(a, p.ksplit, s) : launch_few<T, GluOp<ACT>, 64>(a, p.ksplit, s);
  }
  GluArgs b = a;   // with the operands that the plan lays out anew
  if (p.pad_a) {
    b.A = padded_x;
    b.lda = p.lda;
  }
  if (p.pad_w) {
    b.W = padded_w;
    b.ldw = p.ldw;
    b.Fw = p.ldw / 2;
  }
  if (!direct(p, b)) return launch_reg<T, 128, 128, 2, 2, 2, ACT>(p, a, s);
  hipError_t e = hipSuccess;
  if (p.pad_a) e = launch_pad_rows(a.A, padded_x, p.batch, a.R, b.lda, s);
  if (e == hipSuccess && p.pad_w) e = launch_pad_rows(a.W, padded_w, p.G * a.R * 2, a.F, b.Fw, s);
  return e == hipSuccess ? launch_pipe<T, GluOp<ACT>, false>(b, p.ksplit, s) : e;
}

template <class T, int ACT>
hipError_t finish(const GluArgs& a, int32_t ksplit, hipStream_t s) {
  const int64_t blocks = std::min<int64_t>((a.M * a.F + 255) / 256, 2048);
  hipLaunchKernelGGL((glu_finish_kernel<T, ACT>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a, ksplit);
  return hipGetLastError();
}

template <int ACT>
hipError_t launch_act(const Plan& p, const GluArgs& a, void* px, void* pw, hipStream_t s) {
  hipError_t e;
  if (p.dtype == PGG_F32)
    e = p.regime == kStream ? launch_reg<TF32, 32, 256, 1, 4, 2, ACT>(p, a, s)
                            : launch_reg<TF32, 128, 128, 2, 2, 2, ACT>(p, a, s);
  else
    e = p.dtype == PGG_BF16 ? launch_16<TBf16, ACT>(p, a, px, pw, s) : launch_16<TF16, ACT>(p, a, px, pw, s);
  if (e != hipSuccess || p.ksplit == 1) return e;
  if (p.dtype == PGG_F32) return finish<TF32, ACT>(a, p.ksplit, s);
  return p.dtype == PGG_BF16 ? finish<TBf16, ACT>(a, p.ksplit, s) : finish<TF16, ACT>(a, p.ksplit, s);
}

}  // namespace

hipError_t launch_glu(const Plan& p, int32_t act, const void* x, const void* weight, void* h, void* gate_up,
                      const int64_t* eri, const int64_t* group_list, void* ws, hipStream_t s) {
  const WsView w = ws_view(p, ws);
  GluArgs a;
  a.A = x;
  a.W = weight;
  a.hdr = w.hdr;
  a.tiles = w.tiles;
  a.ori = w.ori;
  a.h = h;
  a.gate_up = gate_up;
  a.part = p.ksplit > 1 ? w.ring : nullptr;
  const size_t es = p.dtype == PGG_F32 ? 4 : 2;
  a.A_end = static_cast<const char*>(x) + es * p.batch * p.N;
  a.W_end = static_cast<const char*>(weight) + es * p.G * p.N * p.K;
  a.R = p.N;          // the plan keeps the reduction in N and the columns in K
  a.C = p.K;
  a.F = a.Fw = p.K / 2;
  a.lda = p.N;
  a.ldw = p.K;
  a.M = p.M;
  a.kspan = p.kspan;
  a.topk = static_cast<uint32_t>(p.topk);
  a.bm = p.bm;
  a.local = p.local;
  a.eri = eri;
  a.gl = group_list;
  a.prep = prep_args(p);
  a.ws = w;
  void* px = static_cast<char*>(ws) + p.off_pad_a;
  void* pw = static_cast<char*>(ws) + p.off_pad_w;
  return act == PGG_ACT_SILU ? launch_act<PGG_ACT_SILU>(p, a, px, pw, s)
                             : launch_act<PGG_ACT_GELU_TANH>(p, a, px, pw, s);
}

}  // namespace pgg
