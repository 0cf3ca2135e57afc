// Tiles of few rows of a 16-bit product whose weights hold the output columns
// contiguously, every row 16-byte aligned: BM (32 or 64) rows x 256 columns of
//
//   acc[r, c] = sum_k A[src(r), k] * W[k, c]           (fp32 accumulate)
//
// over one split of the reduction.  The weights are read once and bound the
// kernel, so it is built to keep reads in flight: stages of 32 k (two runs of
// 128 columns, as in pgg_pipe.h, and 64 bytes of every A row) go straight into
// a ring of kStages LDS slots, two workgroups to a compute unit, so that up to
// 2 (kStages - 1) stages of 18 or 20 KiB are under way per compute unit, and
// one barrier per stage both publishes a stage and frees the slot of the one
// before.  Weight loads carry the non-temporal hint.
//
// Workgroups are numbered with the columns fastest: those that run together
// read whole rows of W.  Four waves, wave w with columns 32 w .. of both runs.
//
// Measured: gated product of 128 rows, 12 experts of 7168 x 4096, bf16, 707 MB in
// 119-126 us, 5.6-5.9 TB/s, the rate of a kernel that only reads (5.2-6.1).
#pragma once

#include "pgg_pipe.h"

namespace pgg {

namespace {

__device__ __forceinline__ void dma16_off_nt(const void* base, uint32_t off, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt"
               :: "s"(m0), "v"(off), "s"(base) : "memory", "m0");
}

template <int BM>
constexpr int kFewStages = BM == 32 ? 4 : 3;

template <class T, class Op, int BM>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2)))
void few_kernel(typename Op::Args a, int32_t ksplit) {
  using E = typename T::elem;
  constexpr int kStages = kFewStages<BM>, kRun = 8192, kStageBytes = 2 * kRun + BM * 64;
  constexpr int kLoads = 5;               // of one wave in a stage
  constexpr int kRowsPerWave = BM / 4;    // A rows that one wave loads
  __shared__ u32x4_t lds[kStages * kStageBytes / 16];

  int bid = blockIdx.x;
  const int extra = Op::extra(a);
  if (bid < extra) {
    Op::template extra_work<T>(a, bid, lds);
    return;
  }
  bid -= extra;
  const int ct = bid % a.n_col_tiles;
  const int split = bid / a.n_col_tiles % ksplit;
  MTile tile;
  if (!Op::template tile<BM>(a, bid / a.n_col_tiles / ksplit, tile, lds)) return;
  tile.pad = split;
  const int64_t R = a.R, lda = a.lda, ldw = a.ldw;
  const int64_t kbeg = static_cast<int64_t>(split) * a.kspan;
  const int64_t span = min<int64_t>(R - kbeg, a.kspan);

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;

  // A: rows of 64 bytes, chunk c of row r at c ^ ((r >> 2) & 3)
  const int ar = wave * kRowsPerWave + (lane >> 2) % kRowsPerWave;
  const int chunk = (lane & 3) ^ ((ar >> 2) & 3);
  const int64_t row_base = Op::src_base(a, tile);
  const char* pa = reinterpret_cast<const char*>(static_cast<const E*>(a.A) + row_base * lda + kbeg);
  const int64_t src = Op::src(a, tile, min(ar, tile.rows - 1), lds);
  const uint32_t oa = static_cast<uint32_t>((src - row_base) * lda * 2) + chunk * 16;
  // W: load u of run j, 4 rows of k
  const char* pb = reinterpret_cast<const char*>(static_cast<const E*>(a.W) + Op::weight(a, tile) + kbeg * ldw);
  const int n = ((((lane & 15) >> 2) ^ lg) << 5) | (((lane & 3) ^ (wave & 2)) << 3);
  uint32_t ob[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      ob[j][u] = static_cast<uint32_t>(((16 * u + 4 * wave + lg) * ldw + Op::half_column(a, ct, j, n)) * 2);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));
  const void* zero = &kZero16;
  __syncthreads();   // the rows have been read from LDS

  auto load = [&](int kt, int slot) {
    const uint32_t m0 = lds0 + slot * kStageBytes;
    const char* p = pb + static_cast<int64_t>(kt) * 64 * ldw;
    const char* q = pa + static_cast<int64_t>(kt) * 64;
    const bool whole = (kt + 1) * 32 <= span;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t at = m0 + j * kRun + u * 4096 + wave * 1024;
        if (whole) dma16_off_nt(p, ob[j][u], at);
        else dma16(kt * 32 + 16 * u + 4 * wave + lg < span ? static_cast<const void*>(p + ob[j][u]) : zero, at);
      }
    if (lane < 4 * kRowsPerWave) {
      const uint32_t at = m0 + 2 * kRun + wave * kRowsPerWave * 64;
      if (whole) dma16_off(q, oa, at);
      else dma16(kt * 32 + chunk * 8 < span ? static_cast<const void*>(q + oa) : zero, at);
    }
  };

  f32x4_t acc[BM / 16][4];
#pragma unroll
  for (int i = 0; i < BM / 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const int nk = static_cast<int>((span + 31) >> 5);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s)
    if (s < nk) load(s, s);
  int slot = 0;
  for (int kt = 0; kt < nk; ++kt) {
    // stage kt has landed; the kStages - 2 after it may still be under way
    if (kt + kStages - 2 < nk) fetched_barrier<(kStages - 2) * kLoads>();
    else fetched_barrier<0>();
    if (kt + kStages - 1 < nk) load(kt + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
    const char* st = reinterpret_cast<const char*>(lds) + slot * kStageBytes;
    u32x4_t fa[BM / 16], fb[4];
#pragma unroll
    for (int i = 0; i < BM / 16; ++i)
      fa[i] = *reinterpret_cast<const u32x4_t*>(st + 2 * kRun + (i * 16 + lr) * 64 + ((lg ^ ((lr >> 2) & 3)) << 4));
#pragma unroll
    for (int j = 0; j < 4; ++j) fb[j] = read_quarter(st + (j >> 1) * kRun, 0, wave * 32 + (j & 1) * 16, lane);
#pragma unroll
    for (int i = 0; i < BM / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_block<T>(acc[i][j], fb[j], fa[i]);
    slot = slot + 1 == kStages ? 0 : slot + 1;
  }
  store_runs<T, Op, BM / 16>(a, tile, Op::first_column(ct, 256) + wave * 32, 0, lane, acc);
}

template <class T, class Op, int BM>
hipError_t launch_few(const typename Op::Args& a, int32_t ksplit, hipStream_t s) {
  const unsigned blocks =
      static_cast<unsigned>(Op::extra(a)) + static_cast<unsigned>(a.n_slots) * a.n_col_tiles * ksplit;
  hipLaunchKernelGGL((few_kernel<T, Op, BM>), dim3(blocks), dim3(256), 0, s, a, ksplit);
  return hipGetLastError();
}

}  // namespace

}  // namespace pgg
