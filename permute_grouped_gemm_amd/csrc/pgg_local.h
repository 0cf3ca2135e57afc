// Tile and rows of a workgroup straight from group_list and the routing index,
// for calls whose few groups one workgroup scans at once: every workgroup finds
// its own tile, which takes no longer than reading a table, and saves the
// launch that would have written it (about 5 us of a small call's 15).  A
// workgroup of the same launch runs the full preparation for the error word.
//
// Nothing here reads or returns an index out of range, whatever the tables hold:
// counts that are negative or do not add up to M give no tile, index values
// outside [0, M) row 0.
#pragma once

#include "pgg_prep.h"

namespace pgg {

namespace {

constexpr int kLocalThreads = 256;   // of the workgroups that do this
constexpr int kLocalWords = 16;      // int32 of scratch that local_tile uses

// The slot-th tile of bm rows, in expert order; false: there is none.  Ends with
// a barrier.
__device__ __forceinline__ bool local_tile(const int64_t* gl, int64_t G, int64_t M, int bm, int slot, MTile& t,
                                           int32_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t count = tid < G ? gl[tid] : 0;
  const bool bad = count < 0 || count > M;
  const int c = bad ? 0 : static_cast<int>(count), n = (c + bm - 1) / bm;
  int rows = c, tiles = n;   // inclusive sums
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int r = __shfl_up(rows, d), k = __shfl_up(tiles, d);
    if (lane >= d) {
      rows += r;
      tiles += k;
    }
  }
  if (lane == 63) {
    scratch[wave] = rows;
    scratch[4 + wave] = tiles;
  }
  // over the waves through the same words: the barrier that reduces a value
  // would take 256 bytes of LDS of its own, and the 32-row tiles of the gradient
  // leave none (4 workgroups to a compute unit take all 160 KiB)
  const bool wave_bad = __ballot(bad) != 0;
  if (lane == 0) scratch[11 + wave] = wave_bad;
  if (tid == 0) scratch[10] = 0;
  __syncthreads();
  bool any_bad = false;
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    any_bad |= scratch[11 + w] != 0;
    total += scratch[w];
    if (w < wave) {
      rows += scratch[w];
      tiles += scratch[4 + w];
    }
  }
  if (any_bad || total != M) return false;
  const int skip = (slot - (tiles - n)) * bm;   // rows of the group before the tile
  if (slot >= tiles - n && slot < tiles) {
    scratch[8] = tid;
    scratch[9] = rows - c + skip;
    scratch[10] = min(bm, c - skip);
  }
  __syncthreads();
  t.g = scratch[8];
  t.row0 = scratch[9];
  t.rows = scratch[10];
  t.pad = 0;
  return t.rows > 0;
}

// original[r] = original position of the tile's row r.  Ends with a barrier.
__device__ __forceinline__ void local_rows(const int64_t* eri, int64_t M, int row_idx_type, const MTile& t,
                                           int32_t* original) {
  const int tid = threadIdx.x;
  if (row_idx_type == 0) {
    if (tid < t.rows) {
      const int64_t p = eri[t.row0 + tid];
      original[tid] = p >= 0 && p < M ? static_cast<int32_t>(p) : 0;
    }
  } else {   // the positions whose row is one of the tile's
    if (tid < t.rows) original[tid] = 0;
    __syncthreads();
    for (int64_t p = tid; p < M; p += kLocalThreads) {
      const int64_t r = eri[p] - t.row0;
      if (r >= 0 && r < t.rows) original[r] = static_cast<int32_t>(p);
    }
  }
  __syncthreads();
}

}  // namespace

}  // namespace pgg
