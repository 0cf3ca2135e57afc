// 256 x 256 tiles of a 16-bit product with fp32 accumulation, for many rows:
//
//   acc[r, c] = sum_k A[src(r), k] * B[k, c]
//
// with every row 16-byte aligned.  B comes in one of two layouts: NT = false,
// a matrix W [R, C] that holds the output columns contiguously (read from LDS
// with the transposing ds_read_b64_tr_b16, as in pgg_nn.h), or NT = true, rows
// of R contiguous reduction elements, one per output column (read like A).
//
// 8 waves (2 along rows x 4 along columns; the two of a SIMD differ in their
// rows), 128 x 64 accumulators each, in 16 x 16 blocks.  A wave's columns are two
// runs of 32, run j at tile column 128 j + 32 wn, so that all waves' first runs
// make one of 128 and the second runs another.  (A gated product puts gate
// columns in one and up columns in the other.)
//
// A stage is 64 reduction elements: 64 KiB of LDS in four quarters A0 A1 B0 B1
// of 16 KiB, A0 holding the first 64 rows of every wave, B0 the first run of
// columns.  It is multiplied in four phases of 16 matrix instructions per wave,
// A0 B0, A0 B1, A1 B1, A1 B0, and each phase has two halves: fetch (fragments from
// LDS to registers, two direct-to-LDS loads of a later stage) and multiply.  The
// first wave of every SIMD runs one half ahead of the second, with a workgroup
// barrier between halves, so that on each SIMD one wave always multiplies while
// the other fetches, and the loads are spread evenly over time.  The 16 matrix instructions of a half take 256 cycles, the
// fetch of four waves at most 12 reads each, 192 cycles of LDS.
//
// A quarter is refilled, for the stage after next, as soon as both waves of
// every SIMD have read it: A0 and B0 from the second phase on, B1 in the
// fourth, A1 in the first phase of the following stage.  A load so has six or
// seven phases, 1.5 stages, until its data is needed.  In every phase the loads
// that the next phase's fetch needs are the oldest 2 of 12 outstanding ones:
// one wait for "at most 10" covers them, and no phase drains the queue.
//
// Measured, kernel time: gated product of 16384 rows x 7168 x 4096 in 16 experts,
// bf16, products saved, 0.81-0.84 ms (1.15-1.19 PFLOP/s); gradient, NT, 110592 rows x
// 7168 x 2048 in 60 experts, f16, 3.0 ms (1.08); adapters' projection, 13824 x 7168 x
// 2048, f16, 0.40 ms (1.0: 432 tiles are 1.7 rounds of the chip).  Matrix
// instructions fill 52-59 % of the cycles, at a clock that falls to 1.7 GHz; on
// all-zero operands the same calls run at 1.7-1.8 PFLOP/s, so the power limit takes
// a part.  It is not all of it: under the same limit a library product of the first
// size, without activation and with one weight, runs at 1.31, and these kernels read
// 2.8 GB where 1.0 is needed (the gradient 9.8 for 4.3).
#pragma once

#include "pgg_nn.h"

namespace pgg {

namespace {

// Direct global -> LDS load of 16 bytes per lane from base + off (bytes).
__device__ __forceinline__ void dma16_off(const void* base, uint32_t off, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(m0), "v"(off), "s"(base) : "memory", "m0");
}

// This wave's LDS operations done, and at most VM vector memory operations
// outstanding (VM < 0: any number); then the workgroup's barrier.
template <int VM>
__device__ __forceinline__ void fetched_barrier() {
  constexpr int n = VM < 0 ? 63 : VM;
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | ((n >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ void plain_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 16 x 16 blocks: lane l holds 8 reduction elements, from 8 (l / 16) on, of row
// l % 16 of either operand, and of the result column l % 16, rows 4 (l / 16) on.
template <class T>
__device__ __forceinline__ void mma_block(f32x4_t& acc, u32x4_t a, u32x4_t b) {
  if constexpr (__is_same(T, TBf16)) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                  acc, 0, 0, 0);
  } else if constexpr (__is_same(T, TF32)) {   // 4 elements, from 4 (l / 16) on: one instruction each
    const f32x4_t fa = __builtin_bit_cast(f32x4_t, a), fb = __builtin_bit_cast(f32x4_t, b);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[0], fb[0], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[1], fb[1], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[2], fb[2], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[3], fb[3], acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                 acc, 0, 0, 0);
  }
}

// Two neighbouring 16 x 16 blocks, columns first: accumulator v of lane l is
// column 4 (l / 16) + v of row l % 16.  After the exchange between the odd
// groups of 16 lanes of x and the even ones of y, lane l holds 8 successive
// columns from run_column(l) on.
__device__ __forceinline__ int run_column(int lane) { return 16 * ((lane >> 4) & 1) + 8 * (lane >> 5); }

__device__ __forceinline__ void piece16(const f32x4_t& x, const f32x4_t& y, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float xe = x[e], ye = y[e];
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, xe), __builtin_bit_cast(uint32_t, ye),
                                                    false, false);
    const uint32_t x1 = r[0], y1 = r[1];
    v[e] = __builtin_bit_cast(float, x1);
    v[4 + e] = __builtin_bit_cast(float, y1);
  }
}

// 8 consecutive k, from 32 s + 8 (lane / 16) on, of column n + lane % 16 of a
// quarter of 256-byte rows.  As read_w of pgg_nn.h, with the 32-byte halves of
// a segment exchanged in every other 8 rows, since the lanes read together
// cover the same 16 columns of rows k.. and k + 8...
__device__ __forceinline__ uint32_t quarter_offset(int k, int b) {
  return static_cast<uint32_t>(k * 256 + (((b >> 6) ^ (k & 3)) << 6) + ((b & 63) ^ (((k >> 3) & 1) << 5)));
}

__device__ __forceinline__ u32x4_t read_quarter(const char* base, int s, int n, int lane) {
  const int i = lane & 15;
  const int k = 32 * s + 8 * (lane >> 4) + (i >> 2);
  const int b = 2 * (n + 4 * (i & 3));
  u32x2_t part[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    auto p = (__attribute__((address_space(3))) h16x4_t*)(
        (__attribute__((address_space(3))) char*)(base + quarter_offset(k + 4 * u, b)));
    part[u] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4f16(p));
  }
  return u32x4_t{part[0][0], part[0][1], part[1][0], part[1][1]};
}

// A wave's accumulators: NI blocks of 16 rows from tile row m0 on, and two runs
// of 32 columns, the first from output column c0 on.
template <class T, class Op, int NI>
__device__ __forceinline__ void store_runs(const typename Op::Args& a, const MTile& tile, int64_t c0, int m0, int lane,
                                           const f32x4_t (&acc)[NI][4]) {
  auto row = [&](int i) { return m0 + i * 16 + (lane & 15); };
  auto left = [&](int i, int64_t c) { return row(i) < tile.rows ? Op::columns(a) - c : 0; };
  const int64_t c1 = c0 + run_column(lane);
  if constexpr (Op::kPaired) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float v[8], w[8];
      piece16(acc[i][0], acc[i][1], v);
      piece16(acc[i][2], acc[i][3], w);
      Op::template piece<T>(a, tile, row(i), c1, left(i, c1), v, w);
    }
  } else {
    // what the pieces need from memory is loaded kAhead rows of blocks ahead
    constexpr int kAhead = 2;
    typename Op::template Side<T> side[kAhead][2];
    auto fetch = [&](int i) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        side[i % kAhead][j] = Op::template fetch<T>(a, tile, row(i), c1 + 128 * j, left(i, c1 + 128 * j));
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v[8];
        piece16(acc[i][2 * j], acc[i][2 * j + 1], v);
        Op::template piece<T>(a, tile, row(i), c1 + 128 * j, left(i, c1 + 128 * j), v, side[i % kAhead][j]);
      }
      if (i + kAhead < NI) fetch(i + kAhead);
    }
  }
}

template <bool B>
struct Whole {
  static constexpr bool value = B;
};

template <class T, class Op, bool NT>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void pipe_kernel(typename Op::Args a) {
  using E = typename T::elem;
  constexpr int kStageBytes = 65536, kQuarter = 16384;
  constexpr int kA = 0, kB = 2 * kQuarter;    // byte offsets of the operands in a stage
  __shared__ u32x4_t lds[2 * kStageBytes / 16];

  int slot, ct;
  if (!tile_place(a, slot, ct)) return;
  MTile tile;
  if (!Op::template tile<256>(a, slot, tile, lds)) return;
  tile.pad = blockIdx.y;
  // this workgroup's split of the reduction
  const int64_t R = a.R, lda = a.lda, ldw = a.ldw;
  const int64_t kbeg = static_cast<int64_t>(blockIdx.y) * a.kspan;
  const int64_t span = min<int64_t>(R - kbeg, a.kspan);

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  // quarters A_h of this wave that hold rows of the tile: the others are not multiplied
  const bool has0 = tile.rows > wm * 128, has1 = tile.rows > wm * 128 + 64;
  const int lr = lane & 15, lg = lane >> 4;

  // Load u of quarter A_h of this wave: 8 tile rows 128 u + 64 h + 8 wave + ...,
  // 128 bytes each; LDS slot lane % 8 of a row holds chunk `chunk`.
  const int l8 = lane >> 3;
  const int chunk = a_slot(8 * wave + l8, lane & 7);
  const int64_t row_base = Op::src_base(a, tile);
  const char* pa = reinterpret_cast<const char*>(static_cast<const E*>(a.A) + row_base * lda + kbeg);
  uint32_t oa[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = min(128 * u + 64 * h + 8 * wave + l8, tile.rows - 1);
      oa[h][u] = static_cast<uint32_t>((Op::src(a, tile, r, lds) - row_base) * lda * 2) + chunk * 16;
    }
  // Load u of quarter B_j.  NT: 8 columns' rows, as for A.  Otherwise 4 rows of
  // k, 256 bytes each, whose 16-byte chunks sit where quarter_offset puts them.
  const E* W = static_cast<const E*>(a.W) + Op::weight(a, tile) + kbeg * (NT ? 1 : ldw);
  const int kq = lane >> 4;                                     // which of the 4 rows
  const char* pb;
  uint32_t ob[2][2];
  if constexpr (NT) {
    const int64_t c0 = Op::first_column(ct, 256);
    pb = reinterpret_cast<const char*>(W + c0 * ldw);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t c = min<int64_t>(c0 + 128 * j + 64 * u + 8 * wave + l8, a.F - 1);
        ob[j][u] = static_cast<uint32_t>((c - c0) * ldw * 2) + chunk * 16;
      }
  } else {
    pb = reinterpret_cast<const char*>(W);
    const int n = ((((lane & 15) >> 2) ^ kq) << 5) | (((lane & 3) ^ (wave & 2)) << 3);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t c = Op::half_column(a, ct, j, n);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        ob[j][u] = static_cast<uint32_t>(((32 * u + 4 * wave + kq) * ldw + c) * 2);
    }
  }
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));
  const void* zero = &kZero16;

  const int nk = static_cast<int>((span + 63) >> 6);
  const int n_full = static_cast<int>(span >> 6);      // stages without a tail
  // The two loads of a quarter for stage kt.  Whole: the stage lies inside the
  // reduction.  Otherwise elements past it read zeros (also whole stages, as
  // every phase issues its two loads).
  auto load_a = [&](int kt, int h, auto whole) {
    const uint32_t m0 = lds0 + (kt & 1) * kStageBytes + kA + h * kQuarter + wave * 1024;
    const char* p = pa + static_cast<int64_t>(kt) * 128;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if constexpr (decltype(whole)::value) dma16_off(p, oa[h][u], m0 + u * 8192);
      else dma16(kt * 64 + chunk * 8 < span ? static_cast<const void*>(p + oa[h][u]) : zero, m0 + u * 8192);
    }
  };
  auto load_b = [&](int kt, int j, auto whole) {
    const uint32_t m0 = lds0 + (kt & 1) * kStageBytes + kB + j * kQuarter + wave * 1024;
    const char* p = pb + static_cast<int64_t>(kt) * (NT ? 128 : 128 * ldw);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t k = static_cast<int64_t>(kt) * 64 + (NT ? chunk * 8 : 32 * u + 4 * wave + kq);
      if constexpr (decltype(whole)::value) dma16_off(p, ob[j][u], m0 + u * 8192);
      else dma16(k < span ? static_cast<const void*>(p + ob[j][u]) : zero, m0 + u * 8192);
    }
  };
  // fragments of a quarter, [16 rows or columns][32 reduction elements]
  const char* base = reinterpret_cast<const char*>(lds);
  auto read_rows = [&](const char* quarter, int row, int q) {
    return *reinterpret_cast<const u32x4_t*>(quarter + (row + lr) * 128 + a_slot(lr, 4 * q + lg) * 16);
  };
  auto read_a = [&](int kt, int h, u32x4_t (&f)[4][2]) {
    const char* st = base + (kt & 1) * kStageBytes + kA + h * kQuarter;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i][q] = read_rows(st, wm * 64 + i * 16, q);
  };
  auto read_b = [&](int kt, int j, u32x4_t (&f)[2][2]) {
    const char* st = base + (kt & 1) * kStageBytes + kB + j * kQuarter;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if constexpr (NT) f[n][q] = read_rows(st, wn * 32 + n * 16, q);
        else f[n][q] = read_quarter(st, q, wn * 32 + n * 16, lane);
      }
  };

  f32x4_t acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](int h, int j, const u32x4_t (&fa)[4][2], const u32x4_t (&fb)[2][2]) {
    __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n) mma_block<T>(acc[4 * h + i][2 * j + n], fb[n][q], fa[i][q]);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
  };

  u32x4_t fa[4][2], fb0[2][2], fb1[2][2];
  auto stage = [&](int kt, auto whole, auto full) {
    const bool work0 = decltype(full)::value || has0, work1 = decltype(full)::value || has1;
    if (work0) {
      read_a(kt, 0, fa);
      read_b(kt, 0, fb0);
    }
    load_a(kt + 1, 1, whole);
    fetched_barrier<10>();
    if (work0) multiply(0, 0, fa, fb0);
    plain_barrier();

    if (work0) read_b(kt, 1, fb1);
    load_a(kt + 2, 0, whole);
    fetched_barrier<10>();
    if (work0) multiply(0, 1, fa, fb1);
    plain_barrier();

    if (work1) read_a(kt, 1, fa);
    load_b(kt + 2, 0, whole);
    fetched_barrier<-1>();
    if (work1) multiply(1, 1, fa, fb1);
    plain_barrier();

    load_b(kt + 2, 1, whole);
    fetched_barrier<10>();
    if (work1) multiply(1, 0, fa, fb0);
    plain_barrier();
  };
  const Whole<true> yes;
  const Whole<false> no;
  load_a(0, 0, no);
  load_b(0, 0, no);
  load_b(0, 1, no);
  load_a(0, 1, no);
  load_a(1, 0, no);
  load_b(1, 0, no);
  load_b(1, 1, no);
  fetched_barrier<10>();
  if (wave >= 4) plain_barrier();   // the second wave of each SIMD: half a phase behind
  int kt = 0;
  if (tile.rows > 192)
    for (; kt + 2 < n_full; ++kt) stage(kt, yes, yes);
  else
    for (; kt + 2 < n_full; ++kt) stage(kt, yes, no);
  for (; kt < nk; ++kt) stage(kt, no, yes);
  if (wave < 4) plain_barrier();
  fetched_barrier<0>();   // the zeros past the reduction have landed before LDS is released

  const int64_t c0 = Op::first_column(ct, 256) + wn * 32;
  Op::template adjust<T, 16>(a, tile, wm * 128, lane, acc, [&](int j) { return c0 + 128 * (j >> 1) + 16 * (j & 1); });
  store_runs<T, Op, 8>(a, tile, c0, wm * 128, lane, acc);
}

template <class T, class Op, bool NT>
hipError_t launch_pipe(const typename Op::Args& a, int ksplit, hipStream_t s) {
  hipLaunchKernelGGL((pipe_kernel<T, Op, NT>), dim3(tile_blocks(a), static_cast<unsigned>(ksplit)), dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace

}  // namespace pgg
