// Tiles of a product whose weights hold the output columns contiguously:
//
//   acc[r, c] = sum_k A[src(r), k] * W[k, c]           (fp32 accumulate)
//
// for a block of rows that share the [R, C] matrix W.  What differs between
// the operators that use them comes as an Op:
//
//   Op::Args                 kernel arguments, with A, W, R (the reduction), C
//                            (the row length of W), n_slots, n_col_tiles, and
//                            kspan (reduction elements of one blockIdx.y)
//   Op::tile(args, slot, t)  rows [t.row0, t.row0 + t.rows) of group t.g; false: no tile
//   Op::src(args, t, r)      row of A that tile row r reads
//   Op::weight(args, t)      first element of the tile's W
//   Op::column<BN>(args, ct, n)  column of W at column n (a multiple of 4) of
//                            the tile, and how many of W's columns follow in that run
//   Op::store<...>(...)      takes the accumulators
//
// Two kernels: nn_dma_kernel (16-bit types, 16-byte aligned rows, 256 x 256
// tiles loaded straight into LDS) and nn_reg_kernel (every type and alignment,
// loads through registers, any tile).
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

// The same with only the first `left` elements read, zeros after them.
template <class T>
__device__ __forceinline__ u32x4_t load16_part(const typename T::elem* p, int64_t left) {
  using E = typename T::elem;
  constexpr int EPC = T::kPerChunk;
  if (left >= EPC) return load16(p);
  E e[EPC];
#pragma unroll
  for (int t = 0; t < EPC; ++t) e[t] = t < left ? p[t] : E(0);
  u32x4_t v;
  __builtin_memcpy(&v, e, sizeof(v));
  return v;
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
  if (!raster<8, 4>(blockIdx.x, a.n_slots, a.n_col_tiles, slot, ct)) return;
  MTile tile;
  if (!Op::template tile<BM>(a, slot, tile)) return;
  const int rows = tile.rows;
  const int64_t C = a.C;
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
    arow[s] = static_cast<const E*>(a.A) + Op::src(a, tile, min(q / kChunks, rows - 1)) * a.R + (q % kChunks) * EPC;
  }
  const E* W = static_cast<const E*>(a.W) + Op::weight(a, tile);
  ColumnRun run[B_PER_T];
  bool whole = true;
#pragma unroll
  for (int s = 0; s < B_PER_T; ++s) {
    const int q = tid + s * NT;
    run[s] = Op::template column<BN>(a, ct, (q % kRowChunks) * EPC);
    whole = whole && run[s].left >= EPC;
  }
  whole = __syncthreads_and(whole);

  u32x4_t ra[A_PER_T], rb[B_PER_T];
  auto load_stage = [&](int kt) {
    const int64_t k0 = kbeg + static_cast<int64_t>(kt) * BK;
    const E* wk = W + k0 * C;
    if (whole && k0 + BK <= kend) {
#pragma unroll
      for (int s = 0; s < A_PER_T; ++s) ra[s] = load16(arow[s] + k0);
#pragma unroll
      for (int s = 0; s < B_PER_T; ++s) rb[s] = load16(wk + (tid + s * NT) / kRowChunks * C + run[s].first);
    } else {
#pragma unroll
      for (int s = 0; s < A_PER_T; ++s)
        ra[s] = load16_part<T>(arow[s] + k0, kend - k0 - (tid + s * NT) % kChunks * EPC);
#pragma unroll
      for (int s = 0; s < B_PER_T; ++s) {
        const int k = (tid + s * NT) / kRowChunks;
        rb[s] = load16_part<T>(wk + k * C + run[s].first, k0 + k < kend ? run[s].left : 0);
      }
    }
  };
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
        for (int j = 0; j < FN; ++j) mma<T>(acc[i][j], fa[q & 1][i], fb[q & 1][j]);
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
  Op::template store<T, BN, FM, FN>(a, tile, ct, wm * WTM, wn * WTN, lane, acc);
}

template <class T, class Op, int BM, int BN, int WM, int WN, int EU>
hipError_t launch_nn_reg(const typename Op::Args& a, int ksplit, hipStream_t s) {
  unsigned tiles = static_cast<unsigned>(a.n_slots) * static_cast<unsigned>(a.n_col_tiles);
  tiles = (tiles + 8 * 32 - 1) / (8 * 32) * (8 * 32);   // whole raster rounds
  hipLaunchKernelGGL((nn_reg_kernel<T, Op, BM, BN, WM, WN, EU>), dim3(tiles, static_cast<unsigned>(ksplit)),
                     dim3(WM * WN * 64), 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Straight into LDS (16-bit types, every row 16-byte aligned): 256 x 256
// tiles, 8 waves (two per SIMD) of 128 x 64 accumulators, two LDS stages of 64
// k (128 bytes of every A row, 512 bytes of 64 W rows; 128 KiB in all), loads
// that write no register and explicit waits on their counter.  The refill of
// a stage is issued by the first wave of each SIMD right after the stage
// barrier and by the second after its last MFMAs, so one of the two always
// feeds the matrix unit.  Lanes with nothing to load read 16 zero bytes.
// ---------------------------------------------------------------------------
template <class T, class Op>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void nn_dma_kernel(typename Op::Args a) {
  using E = typename T::elem;
  constexpr int BM = 256, BN = 256, NT = 512, kWaves = 8, WM = 2;
  constexpr int WTM = 128, WTN = 64, FM = 4, FN = 2;
  constexpr int kChunks = 8, BK = 64, kPairs = kChunks / 2, kStages = 2;
  constexpr int ROW = BN * 2, kRowChunks = ROW / 16;
  constexpr int kSlotsA = BM * kChunks, kStageSlots = kSlotsA + BK * kRowChunks;
  constexpr int kLoadsA = kSlotsA / NT, kLoadsB = BK * kRowChunks / NT;
  __shared__ u32x4_t lds[kStages * kStageSlots];

  int slot, ct;
  if (!raster<8, 4>(blockIdx.x, a.n_slots, a.n_col_tiles, slot, ct)) return;
  MTile tile;
  if (!Op::template tile<BM>(a, slot, tile)) return;
  const int rows = tile.rows;
  const int64_t R = a.R, C = a.C;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int lr = lane & 31, lh = lane >> 5;

  // A: load j of this lane fills row r0 + 64 j, slot lane % 8, which holds
  // chunk dma_c (the same for every j).
  const int r0 = wave * 8 + (lane >> 3);
  const int dma_c = a_slot(r0, lane & 7);
  const E* pa[kLoadsA];
#pragma unroll
  for (int j = 0; j < kLoadsA; ++j)
    pa[j] = static_cast<const E*>(a.A) + Op::src(a, tile, min(r0 + 64 * j, rows - 1)) * R + dma_c * 8;
  // W: load j fills stage row kb_j (two rows to a wave instruction), chunk
  // lane % 32, which holds logical chunk lc_j.
  const E* W = static_cast<const E*>(a.W) + Op::weight(a, tile);
  int64_t boff[kLoadsB];
  uint32_t vb = 0;
#pragma unroll
  for (int j = 0; j < kLoadsB; ++j) {
    const int kb = (j * kWaves + wave) * 2 + lane / kRowChunks;
    const int pc = lane % kRowChunks;
    const int lc = (((pc >> 2) ^ (kb & 3)) << 2) | (pc & 3);
    const ColumnRun run = Op::template column<BN>(a, ct, lc * 8);
    boff[j] = kb * C + run.first;
    vb |= (run.left > 0 ? 1u : 0u) << j;
  }
  const void* zero = &kZero16;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));

  auto issue = [&](int kt) {
    const uint32_t base = lds0 + static_cast<uint32_t>((kt % kStages) * kStageSlots * 16);
    const int64_t k0 = static_cast<int64_t>(kt) * BK;
    const bool in_k = k0 + dma_c * 8 < R;
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j)
      dma16(in_k ? static_cast<const void*>(pa[j] + k0) : zero,
            base + static_cast<uint32_t>((j * kWaves + wave) * 64 * 16));
    const E* wk = W + k0 * C;
#pragma unroll
    for (int j = 0; j < kLoadsB; ++j) {
      const int kb = (j * kWaves + wave) * 2 + lane / kRowChunks;
      dma16(k0 + kb < R && ((vb >> j) & 1) ? static_cast<const void*>(wk + boff[j]) : zero,
            base + static_cast<uint32_t>((kSlotsA + (j * kWaves + wave) * 64) * 16));
    }
  };
  auto load_frags = [&](int kt, int q, u32x4_t (&fa)[FM], u32x4_t (&fb)[FN]) {
    const u32x4_t* st = lds + (kt % kStages) * kStageSlots;
    const int sl = a_slot(lr, 2 * q + lh);
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = st[(wm * WTM + i * 32 + lr) * kChunks + sl];
#pragma unroll
    for (int j = 0; j < FN; ++j)
      fb[j] = read_w<T, ROW>(reinterpret_cast<const char*>(st + kSlotsA), q, wn * WTN + j * 32, lane);
  };
  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  auto mfmas = [&](const u32x4_t (&fa)[FM], const u32x4_t (&fb)[FN]) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) mma<T>(acc[i][j], fa[i], fb[j]);
    __builtin_amdgcn_sched_barrier(0);
  };

  const int nk = static_cast<int>((R + BK - 1) / BK);
#pragma unroll
  for (int s = 0; s < kStages; ++s)
    if (s < nk) issue(s);
  u32x4_t fa0[FM], fb0[FN], fa1[FM], fb1[FN];
  if (nk > 1) wait_then_barrier<kLoadsA + kLoadsB>(); else wait_then_barrier<0>();
  load_frags(0, 0, fa0, fb0);
  int kt = 0;
  for (; kt + kStages < nk; ++kt) {
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      if (q + 1 < kPairs) {
        if (q & 1) load_frags(kt, q + 1, fa0, fb0); else load_frags(kt, q + 1, fa1, fb1);
      } else {
        wait_then_barrier<0>();
        if (wave < kWaves / 2) issue(kt + kStages);
        load_frags(kt + 1, 0, fa0, fb0);
      }
      if (q & 1) mfmas(fa1, fb1); else mfmas(fa0, fb0);
      if (q + 1 == kPairs && wave >= kWaves / 2) issue(kt + kStages);
    }
  }
  for (; kt < nk; ++kt) {
#pragma unroll
    for (int q = 0; q < kPairs; ++q) {
      if (q + 1 < kPairs) {
        if (q & 1) load_frags(kt, q + 1, fa0, fb0); else load_frags(kt, q + 1, fa1, fb1);
      } else if (kt + 1 < nk) {
        wait_then_barrier<0>();
        load_frags(kt + 1, 0, fa0, fb0);
      }
      if (q & 1) mfmas(fa1, fb1); else mfmas(fa0, fb0);
    }
  }
  Op::template store<T, BN, FM, FN>(a, tile, ct, wm * WTM, wn * WTN, lane, acc);
}

template <class T, class Op>
hipError_t launch_nn_dma(const typename Op::Args& a, hipStream_t s) {
  unsigned tiles = static_cast<unsigned>(a.n_slots) * static_cast<unsigned>(a.n_col_tiles);
  tiles = (tiles + 8 * 32 - 1) / (8 * 32) * (8 * 32);
  hipLaunchKernelGGL((nn_dma_kernel<T, Op>), dim3(tiles), dim3(512), 0, s, a);
  return hipGetLastError();
}

// Row of accumulator v in its 32x32 block, for lane half lh (its column is the
// lane's place in the half).
__device__ __forceinline__ int acc_row(int v, int lh) { return 8 * (v >> 2) + 4 * lh + (v & 3); }

}  // namespace

}  // namespace pgg
