// Experts' products with 4-bit weights, many rows per expert, x in a 16-bit
// type: tiles of 64 rows x 256 columns, bound by the matrix instructions and by
// turning codes into their operands.
//
// Four waves, each with 64 of the columns and all rows, so that no code is
// expanded twice in a tile; two workgroups to a compute unit, of which one
// multiplies while the other expands.  A stage is one packed tile's 128 k: x goes
// straight into LDS (16 KiB, chunk c of row r at c ^ (r & 15), which puts the 16
// rows of a read on different banks), the codes straight into registers, both
// one stage ahead.  The sums of x over the scale groups, by which the zero points
// are multiplied, are computed once per row of x by a kernel before; a group's
// product starts from -zero times that sum as the instruction's third operand.
// x on no 16-byte boundary, which the direct loads need, goes through registers: loaded
// a stage ahead, and stored when the stage before has been multiplied.
//
// Measured: 2048 tokens to 8 of 16 experts each (16384 rows), 7168 x 4096 with gate,
// groups of 128, zero points, bf16: 0.98 to 1.05 ms on several cards, 0.92 to 0.98
// PFLOP/s (a library product of 8192^3: 1.19).  1024 rows to each of 16 experts,
// 7168 x 4096 without gate: 0.99 ms, 1.16 with x at an odd address (6.67 in the tiles
// of few rows).  The matrix instructions are busy 45 % of the time; copies of the kernel without
// its loads took 0.81 ms, without the scales' multiply-adds 0.85.  Not faster: codes
// with the non-temporal hint (1.06, the tiles of an expert share them), reading the
// operands of the next 32 k ahead, tiles of 2 x 16, 4 x 8 or 16 x 4 for the order of
// the workgroups instead of 8 x 4, raised priority around the instructions.
#include <algorithm>

#include "pgg_w4.h"

namespace pgg {

namespace {

constexpr int kTileRows = 64, kTileStage = kTileRows * 256;

template <class T, int SUB, bool ZEROS, bool ALIGNED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2)))
void w4_tile_kernel(W4Args a) {
  using E = typename T::elem;
  constexpr int RB = kTileRows / 16, kStages = 2;
  __shared__ u32x4_t lds[kStages * kTileStage / 16];
  __shared__ float s_sum[kStages][SUB][kTileRows];
  __shared__ int32_t s_rows[kTileRows];

  int slot, ct;
  if (!tile_place(a, slot, ct)) return;
  MTile tile;
  if (!w4_find(a, slot, kTileRows, tile, s_rows)) return;

  // the tile is the same for the whole workgroup: scalar registers
  tile.g = __builtin_amdgcn_readfirstlane(tile.g);
  tile.row0 = __builtin_amdgcn_readfirstlane(tile.row0);
  tile.rows = __builtin_amdgcn_readfirstlane(tile.rows);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int64_t cb = 4 * static_cast<int64_t>(ct) + wave;
  const bool mine = cb < a.CB;   // past the last column block: the last again, not stored
  const W4Planes planes =
      w4_planes<T, SUB>(a, static_cast<int64_t>(tile.g) * a.KB * a.CB + (mine ? cb : a.CB - 1));
  const int kb0 = blockIdx.y * a.kb_span, kb1 = min(kb0 + a.kb_span, a.KB);

  // x: load q of this wave, rows 16 wave + 4 q + lane / 16
  uint32_t ox[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = 16 * wave + 4 * q + lg;
    ox[q] = static_cast<uint32_t>(s_rows[r] * a.lda * 2) + 16 * (lr ^ (r & 15));
  }
  const float* psum = a.sums + static_cast<int64_t>(s_rows[lane]) * (a.KB * SUB);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(lds));
  const uint32_t sum0 = __builtin_amdgcn_readfirstlane(lds_offset(s_sum));
  u32x4_t held[4];   // x on no 16-byte boundary: the same pieces through registers
  auto load_x = [&](int kb) {
    const uint32_t m0 = lds0 + (kb & 1) * kTileStage + wave * 4096;
    const char* p = static_cast<const char*>(a.x) + static_cast<int64_t>(kb) * (2 * kW4K);
    const int64_t left = a.K - static_cast<int64_t>(kb) * kW4K;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (!ALIGNED) {
        const int chunk = lr ^ (4 * q + lg);   // 16 wave is a multiple of 16
        held[q] = load16(8 * chunk < left ? p + ox[q] : reinterpret_cast<const char*>(&kZero16));
      } else if (left >= kW4K) {
        dma16_off(p, ox[q], m0 + q * 1024);
      } else {
        const int chunk = lr ^ (4 * q + lg);
        dma16(8 * chunk < left ? static_cast<const void*>(p + ox[q]) : static_cast<const void*>(&kZero16),
              m0 + q * 1024);
      }
    }
    if (wave == 0) {
#pragma unroll
      for (int u = 0; u < SUB; ++u)
        dma4(psum + kb * SUB + u, sum0 + ((kb & 1) * SUB + u) * kTileRows * 4);
    }
  };

  // these into their stage, which all waves have read before the last barrier
  auto store_x = [&](int kb) {
    if constexpr (!ALIGNED)
#pragma unroll
      for (int q = 0; q < 4; ++q) lds[(kb & 1) * (kTileStage / 16) + wave * 256 + q * 64 + lane] = held[q];
  };

  f32x4_t acc[RB][4];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const char* base = reinterpret_cast<const char*>(lds);
  auto multiply = [&](const W4Weights<T, SUB>& w, int buf) {
    const char* st = base + buf * kTileStage + lr * 256;
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      constexpr int kSteps = 4 / SUB;
      u32x4_t f[kSteps][4];
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) f[s][j] = w4_expand<T>(w.code[j][u * kSteps + s]);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const f32x4_t sum = *reinterpret_cast<const f32x4_t*>(&s_sum[buf][u][16 * i + 4 * lg]);
        u32x4_t x[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
          x[s] = *reinterpret_cast<const u32x4_t*>(st + i * 4096 + (((4 * (u * kSteps + s) + lg) ^ lr) << 4));
        f32x4_t part[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float zero = ZEROS ? -w.zero_of(u, j) : -8.0f;
          part[j] = f32x4_t{zero * sum[0], zero * sum[1], zero * sum[2], zero * sum[3]};
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_block<T>(part[j], x[s], f[s][j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[i][j][v] = __builtin_fmaf(w.scale[u].get(j), part[j][v], acc[i][j][v]);
        // in this place: left alone, the products of several groups move behind the
        // expansion of all their codes, which does not fit the registers
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(acc[i][j]));
      }
    }
  };

  W4Weights<T, SUB> w[2];
  load_x(kb0);
  store_x(kb0);
  w[0].load_there(planes, static_cast<uint32_t>(kb0) * a.CB, lane);
  for (int kb = kb0; kb < kb1; kb += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (kb + h < kb1) {
        // stage kb + h has landed, and the buffer of the next has been read
        fetched_barrier<0>();
        if (kb + h + 1 < kb1) load_x(kb + h + 1);
        w[1 - h].load_there(planes, static_cast<uint32_t>(min(kb + h + 1, kb1 - 1)) * a.CB, lane);   // past the end: unused
        multiply(w[h], (kb + h) & 1);
        if (kb + h + 1 < kb1) store_x(kb + h + 1);
      }
  }
  fetched_barrier<0>();
  if (!mine) return;
  if (w4_not_finite(acc)) {
    const E* row[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) row[i] = static_cast<const E*>(a.x) + s_rows[16 * i + lr] * a.lda + 8 * lg;
    w4_again<T, RB, SUB>(a, planes, kb0, kb1, row, lane, acc);
  }
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = 16 * i + 4 * lg + v;
      if (r >= tile.rows) continue;
      const int64_t row = tile.row0 + r;
      const f32x4_t q = {acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]};
      if (a.part) {
        float* to = a.part + (static_cast<int64_t>(blockIdx.y) * a.M + row) * (64ll * a.CB) + 64ll * cb + 4 * lr;
        *reinterpret_cast<f32x4_t*>(to) = q;
      } else {
        w4_store<T>(a, row, cb, lr, q);
      }
    }
}

// Sums of the rows of x over the scale groups of 128, 64 or 32 columns: a wave
// takes 1024 elements, a lane 16 of them.
template <class T>
__global__ __launch_bounds__(256) void w4_sums_kernel(const void* x, float* sums, int64_t rows, int64_t K, int64_t lda,
                                                      int32_t KB, int32_t sub) {
  using E = typename T::elem;
  const int64_t row = blockIdx.x;
  const E* p = static_cast<const E*>(x) + row * lda;
  const int lanes = 8 / sub;   // of one group
  for (int64_t k = 16ll * threadIdx.x; k < 128ll * KB; k += 16 * 256) {
    float v = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4_t raw = load16(k + 8 * h < K ? p + k + 8 * h : reinterpret_cast<const E*>(&kZero16));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u = raw[i];
        v += to_float<T>(static_cast<uint16_t>(u & 0xFFFFu)) + to_float<T>(static_cast<uint16_t>(u >> 16));
      }
    }
    for (int m = 1; m < lanes; m <<= 1) v += __shfl_xor(v, m);
    if (((threadIdx.x) & (lanes - 1)) == 0) sums[row * KB * sub + k / (16 * lanes)] = v;
  }
}

template <class T, int SUB>
hipError_t launch_sub(const W4Args& a, hipStream_t s) {
  const dim3 grid(tile_blocks(a), static_cast<unsigned>(a.ksplit));
  const bool aligned = reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
  if (a.zeros && aligned) hipLaunchKernelGGL((w4_tile_kernel<T, SUB, true, true>), grid, dim3(256), 0, s, a);
  else if (a.zeros) hipLaunchKernelGGL((w4_tile_kernel<T, SUB, true, false>), grid, dim3(256), 0, s, a);
  else if (aligned) hipLaunchKernelGGL((w4_tile_kernel<T, SUB, false, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((w4_tile_kernel<T, SUB, false, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_typed(const W4Plan& p, const W4Args& a, float* sums, hipStream_t s) {
  hipLaunchKernelGGL((w4_sums_kernel<T>), dim3(static_cast<unsigned>(p.base.batch)), dim3(256), 0, s, a.x, sums,
                     p.base.batch, a.K, a.lda, a.KB, p.sub);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.sub == 1) return launch_sub<T, 1>(a, s);
  return p.sub == 2 ? launch_sub<T, 2>(a, s) : launch_sub<T, 4>(a, s);
}

}  // namespace

hipError_t launch_w4_tile(const W4Plan& p, const W4Args& a, hipStream_t s) {
  float* sums = const_cast<float*>(a.sums);
  return p.layout.dtype == PGG_BF16 ? launch_typed<TBf16>(p, a, sums, s) : launch_typed<TF16>(p, a, sums, s);
}

}  // namespace pgg
