// Tiles of a product whose weights hold the output columns contiguously:
//
//   acc[r, c] = sum_k A[src(r), k] * W[k, c]           (fp32 accumulate)
//
// for a block of rows that share the [R, C] matrix W.  What differs between
// the operators that use them comes as an Op:
//
//   Op::Args                 kernel arguments, with A, W, where they end (A_end,
//                            W_end) and their row strides (lda, ldw), R (the
//                            reduction), n_slots, n_col_tiles, and kspan
//                            (reduction elements of one split)
//   Op::tile<BM>(args, slot, t, lds)  rows [t.row0, t.row0 + t.rows) of group t.g;
//                            false: no tile.  (The kernels put the split into
//                            t.pad.)  It may leave something in LDS for
//   Op::src(args, t, r, lds) row of A that tile row r reads
//   Op::extra(args), Op::extra_work<T>(args, i, lds)  workgroups in front of those
//                            of tiles of few rows, and what they do
//   Op::weight(args, t)      first element of the tile's W
//   Op::column<BN>(args, ct, n)  column of W at column n (a multiple of 4) of
//                            the tile, and how many of W's columns follow in that run
//   Op::columns(args)        number of output columns
//   Op::first_column(ct, bn) output column of the tile's first one
//   Op::kPaired              blocks of 32 columns belong together two by two and
//                            make 32 output columns
//   Op::adjust<T, B>(args, t, m0, lane, acc, column)
//                            (tiles of more than 64 rows) may change a wave's
//                            accumulators acc[i][j], blocks of B x B at tile row
//                            m0 + B i and output column column(j)
//   Op::piece<T>(args, t, m, c, left, v, w)
//                            takes 8 successive columns from c on of tile row m,
//                            of which `left` exist (0 or less: none); for pairs,
//                            v and w are those of the first and the second
//                            block, otherwise w is what
//   Op::fetch<T>(args, t, m, c, left)  of type Op::Side<T> had loaded for the piece
//
// The matrix instructions get the columns as their first operand, so that a
// lane ends with columns of one row; two lanes of that row exchange every other
// group of four, and rows are stored in pieces of 8 columns.
//
// nn_reg_kernel takes every type and alignment (loads through registers, any
// tile); pgg_pipe.h has the kernel for many rows of aligned 16-bit data,
// pgg_few.h the one for few.  Measured, gated product of 24 rows for each of 16
// experts: bf16, K 4095, F 2047, 536 MB of weights in 126 us (4.3 TB/s; the
// aligned kernel takes 99 us for 4096 and 2048); fp32, K 2048, F 1408, 369 MB in
// 96 us (3.8 TB/s).  fp32, 8 experts of 1024 rows, K 4096, F 2048: 2.17 ms, 127
// TFLOP/s (a library product of 8192^3 runs at 153).  With a load's latency between two stages, fewer bytes are
// under way than in a ring.
//
// Operand layouts in LDS.  An A row is contiguous along k, which is what an
// MFMA operand wants (a lane takes 16 bytes of one row): rows of 8 chunks of
// 16 bytes, chunk c of row r at c ^ ((r >> 1) & 7), so that the 16 rows a read
// serves at a time fall on different banks.  W is contiguous along c, so the
// stage keeps it as loaded, rows of k, and 16-bit operands are read transposed
// with ds_read_b64_tr_b16: in each group of 16 lanes, lane i receives element
// i % 4 of the 8-byte chunks addressed by lanes 4j + i / 4 (j = 0..3); lanes
// that address row k0 + s / 4, columns n0 + 4 (s % 4) give lane i column
// n0 + i at rows k0..k0+3.  fp32 operands take one k per lane and step.
// Segments of 64 bytes of row k sit at s ^ swz(k), which puts the rows of one
// read on different banks.
#pragma once

#include "pgg_device.h"

namespace pgg {

namespace {

typedef __fp16 h16x4_t __attribute__((__vector_size__(4 * sizeof(__fp16))));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

// A run of W's columns: the first, and how many columns from there belong to
// the same run (0 or less: none).
struct ColumnRun {
  int64_t first, left;
};

// 16 bytes from any address (the hardware takes unaligned vector loads).
template <class E>
__device__ __forceinline__ u32x4_t load16(const E* p) {
  u32x4_t v;
  __builtin_memcpy(&v, p, sizeof(v));
  return v;
}

// The same of which only the first `left` elements count: zeros after them.
// Reads up to 16 bytes from p on, but nothing at `end` or past it.
template <class T>
__device__ __forceinline__ u32x4_t load16_part(const typename T::elem* p, int64_t left, const void* end) {
  using E = typename T::elem;
  constexpr int EPC = T::kPerChunk;
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (left <= 0) return v;
  if (p + EPC <= static_cast<const E*>(end)) {
    v = load16(p);
    if (left >= EPC) return v;
#pragma unroll
    for (int w = 0; w < 4; ++w) {   // element w EPC / 4 and, of 16 bits, the one after it
      const int k = w * EPC / 4;
      if (k >= left) v[w] = 0u;
      else if (EPC == 8 && k + 1 >= left) v[w] &= 0xFFFFu;
    }
  } else {
    E e[EPC];
#pragma unroll
    for (int t = 0; t < EPC; ++t) e[t] = t < left && p + t < static_cast<const E*>(end) ? p[t] : E(0);
    __builtin_memcpy(&v, e, sizeof(v));
  }
  return v;
}

// Tile of a workgroup: in the XCD raster where the launch fills the chip, and
// otherwise columns fastest, so that few tiles spread over all XCDs.
template <class Args>
__device__ __forceinline__ bool tile_place(const Args& a, int& slot, int& ct) {
  const int tiles = a.n_slots * a.n_col_tiles;
  if (tiles >= 256) return raster<8, 4>(blockIdx.x, a.n_slots, a.n_col_tiles, slot, ct);
  ct = static_cast<int>(blockIdx.x) % a.n_col_tiles;
  slot = static_cast<int>(blockIdx.x) / a.n_col_tiles;
  return slot < a.n_slots;
}

// Workgroups along x that tile_place needs.
template <class Args>
unsigned tile_blocks(const Args& a) {
  const unsigned tiles = static_cast<unsigned>(a.n_slots) * static_cast<unsigned>(a.n_col_tiles);
  return tiles >= 256 ? (tiles + 255) / 256 * 256 : tiles;   // whole raster rounds
}

__device__ __forceinline__ int a_slot(int r, int c) { return c ^ ((r >> 1) & 7); }

// Byte offset of byte b of W row k in a stage whose W rows are ROW bytes.
template <class T, int ROW>
__device__ __forceinline__ uint32_t w_offset(int k, int b) {
  const int swz = T::kPerChunk == 8 ? (k & 3) : (((k >> 2) & 1) << 1);
  return static_cast<uint32_t>(k * ROW + (((b >> 6) ^ swz) << 6) + (b & 63));
}

// 8 (16-bit) or 4 (fp32) consecutive k from kc * EPC on of one column per lane
// (lane lr of each half: column n + lr; the halves take successive chunks).
template <class T, int ROW>
__device__ __forceinline__ u32x4_t read_w(const char* base, int q, int n, int lane) {
  if constexpr (T::kPerChunk == 8) {
    const int grp = lane >> 4, s = lane & 15;
    const int nb = 2 * (n + 16 * (grp & 1) + 4 * (s & 3));
    const int k = 8 * (2 * q + (grp >> 1)) + (s >> 2);
    u32x2_t part[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      auto p = (__attribute__((address_space(3))) h16x4_t*)(
          (__attribute__((address_space(3))) char*)(base + w_offset<T, ROW>(k + 4 * u, nb)));
      part[u] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4f16(p));
    }
    return u32x4_t{part[0][0], part[0][1], part[1][0], part[1][1]};
  } else {
    const int k = 4 * (2 * q + (lane >> 5));
    u32x4_t v;
#pragma unroll
    for (int t = 0; t < 4; ++t)
      v[t] = *reinterpret_cast<const uint32_t*>(base + w_offset<T, ROW>(k + t, (n + (lane & 31)) * 4));
    return v;
  }
}

template <class T>
__device__ __forceinline__ void mma_block(f32x16_t& acc, u32x4_t a, u32x4_t b) {
  mma<T>(acc, a, b);
}

// Vectors at any address.
typedef u32x4_t __attribute__((aligned(2))) u32x4_any_t;

// 8 stored elements.
template <class T>
struct Raw8 {
  typename T::elem e[8];
};

// From memory that is read once: the non-temporal hint leaves the caches to the
// operands, which many tiles share.
template <class T>
__device__ __forceinline__ Raw8<T> load_raw8(const typename T::elem* p, int64_t left) {
  Raw8<T> r;
  if (left >= 8) {
    u32x4_t x[sizeof(r.e) / 16];
#pragma unroll
    for (unsigned q = 0; q < sizeof(r.e) / 16; ++q)
      x[q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any_t*>(p) + q);
    __builtin_memcpy(r.e, x, sizeof(r.e));
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t) r.e[t] = t < left ? p[t] : typename T::elem(0);
  }
  return r;
}

// 8 values to p, of which the first `left` exist, rounded once; NT: with the
// non-temporal hint, for results that this call does not read again.
template <class T, bool NT = true>
__device__ __forceinline__ void store8(typename T::elem* p, int64_t left, const float (&v)[8]) {
  using E = typename T::elem;
  E e[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) e[t] = from_float<T>(v[t]);
  if (left >= 8) {
    u32x4_t x[sizeof(e) / 16];
    __builtin_memcpy(x, e, sizeof(e));
#pragma unroll
    for (unsigned q = 0; q < sizeof(e) / 16; ++q) {
      if constexpr (NT) __builtin_nontemporal_store(x[q], reinterpret_cast<u32x4_any_t*>(p) + q);
      else reinterpret_cast<u32x4_any_t*>(p)[q] = x[q];
    }
  } else if (left > 0) {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (t < left) p[t] = e[t];
  }
}

// What the upper half of the wave holds in x for what the lower one holds in y.
__device__ __forceinline__ void exchange32(float& x, float& y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y),
                                                  false, false);
  const uint32_t x1 = r[0], y1 = r[1];
  x = __builtin_bit_cast(float, x1);
  y = __builtin_bit_cast(float, y1);
}

// Columns of a 32 x 32 block, 32 rows to its 32 lanes per half: accumulator v
// is column 8 (v / 4) + 4 (lane / 32) + v % 4.  Piece q (0, 1) of this lane
// after the exchange starts at column 16 q + 8 (lane / 32).
__device__ __forceinline__ void piece32(const f32x16_t& acc, int q, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = acc[8 * q + e];
    v[4 + e] = acc[8 * q + 4 + e];
    exchange32(v[e], v[4 + e]);
  }
}

// All of a wave's 32 x 32 blocks: first tile row m0, first output column c0.
template <class T, class Op, bool ADJUST, int FM, int FN>
__device__ __forceinline__ void store_blocks(const typename Op::Args& a, const MTile& t, int64_t c0, int m0, int lane,
                                             f32x16_t (&acc)[FM][FN]) {
  if constexpr (ADJUST) Op::template adjust<T, 32>(a, t, m0, lane, acc, [&](int j) { return c0 + 32 * j; });
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + i * 32 + (lane & 31);
#pragma unroll
    for (int j = 0; j < FN; j += Op::kPaired ? 2 : 1) {
      const int64_t c = c0 + (Op::kPaired ? j / 2 : j) * 32;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float v[8];
        piece32(acc[i][j], q, v);
        const int64_t at = c + 16 * q + 8 * (lane >> 5);
        const int64_t left = m < t.rows ? Op::columns(a) - at : 0;
        if constexpr (Op::kPaired) {
          float w[8];
          piece32(acc[i][j + 1], q, w);
          Op::template piece<T>(a, t, m, at, left, v, w);
        } else {
          Op::template piece<T>(a, t, m, at, left, v, Op::template fetch<T>(a, t, m, at, left));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Through registers: any type, alignment and tile.  The loads of the next
// stage are in flight while the current one is multiplied.  Rows past the
// tile's and columns past the matrix repeat valid ones (they reach only
// accumulators that are never stored); elements past the reduction are zero in
// both operands.
// ---------------------------------------------------------------------------
template <class T, class Op, int BM, int BN, int WM, int WN, int EU>
__global__ __launch_bounds__(WM * WN * 64) __attribute__((amdgpu_waves_per_eu(EU, EU)))
void nn_reg_kernel(typename Op::Args a) {
  using E = typename T::elem;
  constexpr int NT = WM * WN * 64;
  constexpr int EPC = T::kPerChunk;
  constexpr int kChunks = 8;
  constexpr int BK = kChunks * EPC;
  constexpr int ROW = BN * int(sizeof(E));
  constexpr int kRowChunks = ROW / 16;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int FM = WTM / 32, FN = WTN / 32;
  constexpr int A_CHUNKS = BM * kChunks, B_CHUNKS = BK * kRowChunks;
  constexpr int A_PER_T = A_CHUNKS / NT, B_PER_T = B_CHUNKS / NT;
  static_assert(ROW >= 256, "four 64-byte segments to a W row");
  static_assert(WTM % 32 == 0 && WTN % 32 == 0, "whole 32x32 blocks per wave");
  static_assert(A_CHUNKS % NT == 0 && B_CHUNKS % NT == 0, "a stage splits evenly");

  __shared__ u32x4_t lds[2][A_CHUNKS + B_CHUNKS];

  int slot, ct;
  if constexpr (BM <= 64) {   // few rows: columns fastest, whatever the number of tiles
    int bid = blockIdx.x;
    const int extra = Op::extra(a);
    if (bid < extra) {
      if (blockIdx.y == 0) Op::template extra_work<T>(a, bid, lds);
      return;
    }
    bid -= extra;
    ct = bid % a.n_col_tiles;
    slot = bid / a.n_col_tiles;
    if (slot >= a.n_slots) return;
  } else {
    if (!tile_place(a, slot, ct)) return;
  }
  MTile tile;
  if (!Op::template tile<BM>(a, slot, tile, lds)) return;
  tile.pad = blockIdx.y;
  const int rows = tile.rows;
  const int64_t ldw = a.ldw;
  const int64_t kbeg = static_cast<int64_t>(blockIdx.y) * a.kspan;
  const int64_t kend = min<int64_t>(a.R, kbeg + a.kspan);

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int wm = wave % WM, wn = wave / WM;
  const int lr = lane & 31, lh = lane >> 5;

  const E* arow[A_PER_T];
#pragma unroll
  for (int s = 0; s < A_PER_T; ++s) {
    const int q = tid + s * NT;
    const int64_t row = Op::src(a, tile, min(q / kChunks, rows - 1), lds);
    arow[s] = static_cast<const E*>(a.A) + row * a.lda + (q % kChunks) * EPC;
  }
  // Columns past the matrix are not stored, so a chunk may hold anything there:
  // it is read whole, from the row's end on into the next row, and a chunk
  // outside altogether is read from the run's start.
  const E* W = static_cast<const E*>(a.W) + Op::weight(a, tile);
  int64_t col[B_PER_T];
#pragma unroll
  for (int s = 0; s < B_PER_T; ++s) {
    const int q = tid + s * NT;
    const ColumnRun run = Op::template column<BN>(a, ct, (q % kRowChunks) * EPC);
    col[s] = run.left > 0 ? run.first : run.first + run.left - Op::columns(a);
  }

  u32x4_t ra[A_PER_T], rb[B_PER_T];
  auto load_stage = [&](int kt) {
    const int64_t k0 = kbeg + static_cast<int64_t>(kt) * BK;
    const E* wk = W + k0 * ldw;
    // inside the reduction, and a chunk may run past the stage's last row
    if (k0 + BK <= kend && wk + BK * ldw + EPC <= static_cast<const E*>(a.W_end)) {
#pragma unroll
      for (int s = 0; s < A_PER_T; ++s) ra[s] = load16(arow[s] + k0);
#pragma unroll
      for (int s = 0; s < B_PER_T; ++s) rb[s] = load16(wk + (tid + s * NT) / kRowChunks * ldw + col[s]);
    } else {
#pragma unroll
      for (int s = 0; s < A_PER_T; ++s)
        ra[s] = load16_part<T>(arow[s] + k0, kend - k0 - (tid + s * NT) % kChunks * EPC, a.A_end);
#pragma unroll
      for (int s = 0; s < B_PER_T; ++s) {
        const int k = (tid + s * NT) / kRowChunks;
        rb[s] = load16_part<T>(wk + k * ldw + col[s], k0 + k < kend ? EPC : 0, a.W_end);
      }
    }
  };
  if constexpr (BM <= 64) __syncthreads();   // the rows have been read from LDS
  auto store_stage = [&](int buf) {
#pragma unroll
    for (int s = 0; s < A_PER_T; ++s) {
      const int q = tid + s * NT;
      lds[buf][q / kChunks * kChunks + a_slot(q / kChunks, q % kChunks)] = ra[s];
    }
    char* base = reinterpret_cast<char*>(&lds[buf][A_CHUNKS]);
#pragma unroll
    for (int s = 0; s < B_PER_T; ++s) {
      const int q = tid + s * NT;
      *reinterpret_cast<u32x4_t*>(base + w_offset<T, ROW>(q / kRowChunks, q % kRowChunks * 16)) = rb[s];
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
    const char* Bs = reinterpret_cast<const char*>(&lds[buf][A_CHUNKS]);
    u32x4_t fa[2][FM], fb[2][FN];
    auto load_frags = [&](int q, u32x4_t (&xa)[FM], u32x4_t (&xb)[FN]) {
      const int sl = a_slot(lr, 2 * q + lh);   // fragment rows start at multiples of 32
#pragma unroll
      for (int i = 0; i < FM; ++i) xa[i] = As[(wm * WTM + i * 32 + lr) * kChunks + sl];
#pragma unroll
      for (int j = 0; j < FN; ++j) xb[j] = read_w<T, ROW>(Bs, q, wn * WTN + j * 32, lane);
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

  const int nk = static_cast<int>((kend - kbeg + BK - 1) / BK);
  load_stage(0);
  store_stage(0);
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    if (kt + 1 < nk) load_stage(kt + 1);
    compute(kt & 1);
    if (kt + 1 < nk) store_stage((kt & 1) ^ 1);
    __syncthreads();
  }
  const int64_t c0 = Op::first_column(ct, BN) + wn * (Op::kPaired ? WTN / 2 : WTN);
  store_blocks<T, Op, (BM > 64), FM, FN>(a, tile, c0, wm * WTM, lane, acc);
}

template <class T, class Op, int BM, int BN, int WM, int WN, int EU>
hipError_t launch_nn_reg(const typename Op::Args& a, int ksplit, hipStream_t s) {
  unsigned tiles = tile_blocks(a);
  if (BM <= 64) tiles = static_cast<unsigned>(Op::extra(a)) + static_cast<unsigned>(a.n_slots) * a.n_col_tiles;
  hipLaunchKernelGGL((nn_reg_kernel<T, Op, BM, BN, WM, WN, EU>), dim3(tiles, static_cast<unsigned>(ksplit)),
                     dim3(WM * WN * 64), 0, s, a);
  return hipGetLastError();
}

}  // namespace

}  // namespace pgg
