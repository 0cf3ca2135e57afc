// Experts' products with 4-bit weights: what the kernels share.
//
//   y[i, n] = sum_k x[src(i), k] * (code[g, k, n] - zero[g, u, n]) * scale[g, u, n],   u = k / group_size
//
// Arithmetic.  Codes 0..15 are exact in both 16-bit types, so the matrix
// instructions multiply the codes themselves, and zero point and scale follow in
// fp32 on the sum over one group:
//
//   acc += scale * (sum_k code x  -  zero * sum_k x)
//
// sum_k x comes from the same instructions with a matrix of ones.  Nothing is
// rounded but the fp32 sums.  As the fp8 format e4m3 holds 0..15 times 2^-9 in
// its 16 lowest bytes (8 subnormal, 8 of the first exponent), a byte that holds a
// code converts to either 16-bit type in one instruction for two codes, with 2^9
// as the conversion's scale: with the masks 7 instructions for 8 codes.
// A result that is not finite (an infinity or NaN in x or in a scale, or an
// overflow) is computed again with code - zero multiplied directly, so that an
// infinity times a weight of one sign stays an infinity.
// x in fp32 is cut into three bf16 parts, 8 bits of the 24 each, which are exact but
// for bits below 2^-133, bf16's smallest number (|x| below 2^-110 has such).
//
// Layout.  Tiles of 128 k x 64 columns, [G][KB][CB][4 blocks][64 lanes][16 bytes]:
// lane l of block j holds column column_of(l % 16, j) of the tile, and its word s
// the 8 codes of k = 32 s + 8 (l / 16) + i, i < 4 in the low and i >= 4 in the
// high half of byte i % 4: what the 16 x 16 x 32 instruction wants in step s.  A
// wave reads 4 KiB in a row.  Scales and zero points follow in planes of their
// own, [G][KB][CB][SUB][64 columns in the order 4 (l % 16) + j], SUB groups of a
// tile of 128 k (1, 2 or 4), so a lane's four come in one load.  A lane so has
// four neighbouring columns of every row it holds.  Gated weights have gate
// columns in blocks 0 and 1 and the matching up columns in 2 and 3.
// Codes past the last row or column are 0; x is read as 0 past its last column.
#pragma once

#include "pgg_act.h"
#include "pgg_local.h"
#include "pgg_pipe.h"

namespace pgg {

constexpr int kW4K = 128, kW4Cols = 64;          // a packed tile
constexpr int kW4TileBytes = kW4K * kW4Cols / 2;

struct W4Args {
  const void* x;
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;     // NULL: 8
  void* out;                // [M, cols] or, gated, [M, F]
  float* part;              // [ksplit, M, 64 CB], or NULL
  const float* sums;        // (tiles) sums of x over the groups, [batch, KB SUB]
  const WsHeader* hdr;
  const MTile* tiles;
  const int32_t* ori;
  int64_t M, K, cols;       // K: of x, a multiple of 8 (fp32: 4); cols: output columns (gated: F)
  int64_t lda;
  int32_t KB, CB, kb_span, ksplit;
  int32_t n_slots, n_col_tiles;
  int32_t beside;           // column blocks of a workgroup
  uint32_t topk;
  int32_t gated, act;
  // without tables
  int32_t local;
  const int64_t* eri;       // NULL: row i reads row i of x
  const int64_t* gl;
  PrepArgs prep;
  WsView ws;
};

// Many rows per expert (w4_tile.hip).
hipError_t launch_w4_tile(const W4Plan& p, const W4Args& a, hipStream_t s);

namespace {

// Column of the product (gated: gate columns, then up) in tile column block cb.
__host__ __device__ __forceinline__ int64_t w4_column(int64_t cb, int i, int j, bool gated, int64_t F) {
  if (!gated) return cb * 64 + 4 * i + j;
  return cb * 32 + 2 * i + (j & 1) + (j >> 1) * F;
}

template <class T>
struct W4Type {
  static constexpr int kParts = 1, kVec = 1;   // bf16 / f16 parts of x; 16-byte loads of 8 elements
  using Mma = T;
};
template <>
struct W4Type<TF32> {
  static constexpr int kParts = 3, kVec = 2;
  using Mma = TBf16;
};

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// 8 codes of a word as the matrix instruction's operand.
template <class Mma>
__device__ __forceinline__ u32x4_t w4_expand(uint32_t w) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  if constexpr (__is_same(Mma, TBf16)) {
    return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true))};
  } else {
    return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, true)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, true))};
  }
}

// The same of code - zero, any whole zero point (exact: at most 4 bits).
template <class Mma>
__device__ __forceinline__ u32x4_t w4_expand_difference(uint32_t w, float zero) {
  uint16_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    e[i] = from_float<Mma>(static_cast<float>((w >> (8 * (i & 3) + 4 * (i >> 2))) & 15u) - zero);
  u32x4_t v;
  __builtin_memcpy(&v, e, sizeof(v));
  return v;
}

template <class Mma>
__device__ __forceinline__ u32x4_t ones() {
  const uint32_t one = __is_same(Mma, TBf16) ? 0x3F803F80u : 0x3C003C00u;
  return u32x4_t{one, one, one, one};
}

// 8 elements of x as operands: themselves, or the three parts of fp32.
// SAFE: a part after an infinity or NaN is 0 (otherwise NaN, which makes the
// result one that is computed again).
template <class T, bool SAFE>
__device__ __forceinline__ void w4_parts(const u32x4_t (&x)[W4Type<T>::kVec], u32x4_t (&p)[W4Type<T>::kParts]) {
  if constexpr (W4Type<T>::kParts == 1) {
    p[0] = x[0];
  } else {
    uint32_t h[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = x[i >> 2][i & 3];
      const float v = __builtin_bit_cast(float, u);
      h[0][i] = SAFE && v != v ? 0x7FC00000u : u;
      const float r = v - __builtin_bit_cast(float, u & 0xFFFF0000u);
      h[1][i] = SAFE && r != r ? 0u : __builtin_bit_cast(uint32_t, r);
      const float q = r - __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, r) & 0xFFFF0000u);
      h[2][i] = SAFE && q != q ? 0u : __builtin_bit_cast(uint32_t, q);
    }
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) p[s][i] = (h[s][2 * i] >> 16) | (h[s][2 * i + 1] & 0xFFFF0000u);
  }
}

// Four scales as loaded, and one of them widened.
template <class T>
struct W4Scales {
  u32x2_t v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t p, uint32_t off, uint32_t base = 0) {
    v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(p, off, base, 0));
  }
  __device__ __forceinline__ float get(int j) const {
    return to_float<T>(static_cast<uint16_t>(v[j >> 1] >> (16 * (j & 1))));
  }
};
template <>
struct W4Scales<TF32> {
  f32x4_t v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t p, uint32_t off, uint32_t base = 0) {
    v = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(p, off, base, 0));
  }
  __device__ __forceinline__ float get(int j) const { return v[j]; }
};

// The packed weights of a wave's column block, as buffers: a tile past the wave's
// last is asked for at an offset outside and reads zeros without an access, so
// that every load is issued in every round and none waits for a branch.
struct W4Planes {
  __amdgpu_buffer_rsrc_t codes, scales, zeros;
  int32_t have_zeros;
};

template <class T, int SUB>
__device__ __forceinline__ W4Planes w4_planes(const W4Args& a, int64_t tile0) {
  constexpr int kFlags = 0x00027000;   // raw 32-bit elements
  constexpr int64_t kScaleBytes = SUB * 64 * sizeof(typename T::elem);
  const int64_t span = (a.KB - 1) * static_cast<int64_t>(a.CB) + 1;   // tiles from the first to the last
  W4Planes p;
  p.codes = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.codes + tile0 * kW4TileBytes), 0,
                                              static_cast<int>(span * kW4TileBytes), kFlags);
  p.scales = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char*>(static_cast<const char*>(a.scales) + tile0 * kScaleBytes), 0,
      static_cast<int>(span * kScaleBytes), kFlags);
  p.have_zeros = a.zeros != nullptr;
  p.zeros = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.zeros + (a.zeros ? tile0 * SUB * 64 : 0)), 0,
                                              a.zeros ? static_cast<int>(span * SUB * 64) : 0, kFlags);
  return p;
}

// What a wave holds of one tile of 128 k x 64 columns.
template <class T, int SUB>
struct W4Weights {
  u32x4_t code[4];
  W4Scales<T> scale[SUB];
  uint32_t zero[SUB];

  // tile: its number from the wave's first on, or any if `there` is false
  __device__ __forceinline__ void load(const W4Planes& p, uint32_t tile, bool there, int lane) {
    constexpr int kNonTemporal = 2;
    const uint32_t c = there ? tile * kW4TileBytes + lane * 16 : kOutside;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      code[j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(p.codes, c + 1024 * j, 0, kNonTemporal));
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const uint32_t at = (tile * SUB + u) * 64 + 4 * (lane & 15);
      scale[u].load(p.scales, there ? at * static_cast<uint32_t>(sizeof(typename T::elem)) : kOutside);
      zero[u] = p.have_zeros ? __builtin_amdgcn_raw_buffer_load_b32(p.zeros, there ? at : kOutside, 0, 0) : 0x08080808u;
    }
  }
  // The same for a tile that is there, its number in a scalar register, and that
  // other workgroups read again.
  __device__ __forceinline__ void load_there(const W4Planes& p, uint32_t tile, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      code[j] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(p.codes, lane * 16 + 1024 * j, tile * kW4TileBytes, 0));
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      constexpr uint32_t kElem = sizeof(typename T::elem);
      const uint32_t at = 4 * (lane & 15), from = (tile * SUB + u) * 64;
      scale[u].load(p.scales, at * kElem, from * kElem);
      zero[u] = p.have_zeros ? __builtin_amdgcn_raw_buffer_load_b32(p.zeros, at, from, 0) : 0x08080808u;
    }
  }
  __device__ __forceinline__ float zero_of(int u, int j) const {
    return static_cast<float>((zero[u] >> (8 * j)) & 255u);
  }
};

// Row r of the tile -> row of x.
__device__ __forceinline__ int64_t w4_source(const W4Args& a, const MTile& t, int r, const int32_t* rows) {
  if (rows) return rows[r];
  const int64_t i = t.row0 + r;
  return a.eri ? static_cast<uint32_t>(a.ori[i]) / a.topk : i;
}

// 8 elements of a row from p on, of which `left` exist, a multiple of a chunk of
// 16 bytes; zeros after them.
template <class T>
__device__ __forceinline__ void w4_load_x(u32x4_t (&v)[W4Type<T>::kVec], const typename T::elem* p, int64_t left) {
  using E = typename T::elem;
  const E* zero = reinterpret_cast<const E*>(&kZero16);
#pragma unroll
  for (int h = 0; h < W4Type<T>::kVec; ++h) v[h] = load16(h * T::kPerChunk < left ? p + h * T::kPerChunk : zero);
}

// A wave's result once more for [kb0, kb1), with code - zero multiplied
// directly, x and weights straight from memory.
template <class T, int RB, int SUB>
__device__ __forceinline__ void w4_again(const W4Args& a, const W4Planes& planes, int kb0, int kb1,
                                         const typename T::elem* const (&px)[RB], int lane, f32x4_t (&acc)[RB][4]) {
  using Mma = typename W4Type<T>::Mma;
  constexpr int P = W4Type<T>::kParts;
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = kb0; kb < kb1; ++kb) {
    W4Weights<T, SUB> w;
    w.load(planes, static_cast<uint32_t>(kb) * a.CB, true, lane);
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      f32x4_t part[RB][4];
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = u * 4 / SUB; s < (u + 1) * 4 / SUB; ++s) {
        const int64_t k = static_cast<int64_t>(kb) * kW4K + 32 * s;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          __builtin_amdgcn_sched_barrier(0);   // one operand at a time: registers, not time, count here
          const u32x4_t f = w4_expand_difference<Mma>(w.code[j][s], w.zero_of(u, j));
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            u32x4_t raw[W4Type<T>::kVec], p[P];
            w4_load_x<T>(raw, px[i] + k, a.K - k - 8 * (lane >> 4));
            w4_parts<T, true>(raw, p);
#pragma unroll
            for (int q = 0; q < P; ++q) mma_block<Mma>(part[i][j], p[q], f);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(w.scale[u].get(j), part[i][j][v], acc[i][j][v]);
    }
  }
}

template <int RB>
__device__ __forceinline__ bool w4_not_finite(const f32x4_t (&acc)[RB][4]) {
  float m = 0.0f;   // 0 times a finite value is 0, otherwise NaN
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) m = __builtin_fmaf(0.0f, acc[i][j][v], m);
  return __ballot(m != m) != 0;
}

// The tile of 4 columns (blocks 0..3 of lane position i) of one row: the
// activation, and the store.
template <class T>
__device__ __forceinline__ void w4_store(const W4Args& a, int64_t row, int64_t cb, int i, const f32x4_t& v) {
  using E = typename T::elem;
  E* out = static_cast<E*>(a.out) + row * a.cols;
  if (a.gated) {
    const int64_t f = cb * 32 + 2 * i;
    float h[2];
    if (a.act == PGG_ACT_SILU) {
      h[0] = activate<PGG_ACT_SILU>(v[0]) * v[2];
      h[1] = activate<PGG_ACT_SILU>(v[1]) * v[3];
    } else {
      h[0] = activate<PGG_ACT_GELU_TANH>(v[0]) * v[2];
      h[1] = activate<PGG_ACT_GELU_TANH>(v[1]) * v[3];
    }
    const E e[2] = {from_float<T>(h[0]), from_float<T>(h[1])};
    if (f + 2 <= a.cols) __builtin_memcpy(out + f, e, sizeof(e));
    else if (f < a.cols) out[f] = e[0];
    return;
  }
  const int64_t c = cb * 64 + 4 * i;
  const E e[4] = {from_float<T>(v[0]), from_float<T>(v[1]), from_float<T>(v[2]), from_float<T>(v[3])};
  if (c + 4 <= a.cols) {
    __builtin_memcpy(out + c, e, sizeof(e));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < a.cols) out[c + j] = e[j];
  }
}

// The slot-th tile of bm rows in expert order, found by every wave for itself
// from at most 256 counts; false: there is none, or the counts are not M rows.
__device__ __forceinline__ bool w4_local_tile(const int64_t* gl, int64_t G, int64_t M, int bm, int slot, MTile& t) {
  const int lane = threadIdx.x & 63;
  int c[4], rows = 0, tiles = 0;
  int64_t total = 0;
  bool bad = false;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int g = 4 * lane + q;
    const int64_t count = g < G ? gl[g] : 0;
    bad |= count < 0 || count > M;
    c[q] = count < 0 || count > M ? 0 : static_cast<int>(count);
    total += c[q];
    rows += c[q];
    tiles += (c[q] + bm - 1) / bm;
  }
  if (__ballot(bad)) return false;
  int before_rows = rows, before_tiles = tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int r = __shfl_up(before_rows, d), k = __shfl_up(before_tiles, d);
    const int64_t s = __shfl_xor(total, d);
    if (lane >= d) {
      before_rows += r;
      before_tiles += k;
    }
    total += s;
  }
  if (total != M) return false;
  before_rows -= rows;
  before_tiles -= tiles;
  int g = -1, row0 = 0, n = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int mine = (c[q] + bm - 1) / bm, skip = slot - before_tiles;
    if (skip >= 0 && skip < mine) {
      g = 4 * lane + q;
      row0 = before_rows + skip * bm;
      n = min(bm, c[q] - skip * bm);
    }
    before_rows += c[q];
    before_tiles += mine;
  }
  const uint64_t owner = __ballot(g >= 0);
  if (!owner) return false;
  const int from = __builtin_ctzll(owner);
  t.g = __shfl(g, from);
  t.row0 = __shfl(row0, from);
  t.rows = __shfl(n, from);
  t.pad = 0;
  return true;
}

// Rows of x that the tile's rows read, for calls without tables.  Ends with a barrier.
__device__ __forceinline__ void w4_local_rows(const W4Args& a, const MTile& t, int bm, int32_t* rows) {
  const int tid = threadIdx.x;
  if (!a.eri) {
    if (tid < bm) rows[tid] = t.row0 + min(tid, t.rows - 1);
  } else if (a.prep.row_idx_type == 0) {
    if (tid < bm) {
      const int64_t p = a.eri[t.row0 + min(tid, t.rows - 1)];
      rows[tid] = p >= 0 && p < a.M ? static_cast<int32_t>(static_cast<uint32_t>(p) / a.topk) : 0;
    }
  } else {   // the positions whose row is one of the tile's
    if (tid < bm) rows[tid] = 0;
    __syncthreads();
    for (int64_t p = tid; p < a.M; p += blockDim.x) {
      const int64_t r = a.eri[p] - t.row0;
      if (r >= 0 && r < t.rows) rows[r] = static_cast<int32_t>(static_cast<uint32_t>(p) / a.topk);
    }
  }
  __syncthreads();
}

// The tile of a workgroup, and where its rows come from (rows: bm words of LDS).
__device__ __forceinline__ bool w4_find(const W4Args& a, int slot, int bm, MTile& t, int32_t* rows) {
  if (a.local) {
    if (!w4_local_tile(a.gl, a.prep.G, a.M, bm, slot, t)) return false;
    w4_local_rows(a, t, bm, rows);
    return true;
  }
  if (a.hdr->err != kNoError || slot >= a.hdr->n_tiles) return false;
  t = a.tiles[slot];
  if (t.rows <= 0) return false;
  if (static_cast<int>(threadIdx.x) < bm)
    rows[threadIdx.x] = static_cast<int32_t>(w4_source(a, t, min(static_cast<int>(threadIdx.x), t.rows - 1), nullptr));
  __syncthreads();
  return true;
}

// The error word of a call without tables, by one workgroup: the counts by its
// first wave, the index with a bit per row.
__device__ __forceinline__ void w4_check(const W4Args& a, uint32_t* bits) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    a.ws.hdr->err = kNoError;
    a.ws.hdr->n_tiles = 0;
  }
  if (a.eri)
    for (int64_t i = tid; i < (a.M + 31) / 32; i += blockDim.x) bits[i] = 0;
  __syncthreads();
  if (tid < 64) {
    int64_t total = 0;
    int first_bad = kLocalGroups;
    for (int g = tid; g < a.prep.G; g += 64) {
      const int64_t c = a.gl[g];
      if (c < 0) first_bad = min(first_bad, g);
      else total += min<int64_t>(c, a.M + 1);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      total += __shfl_xor(total, d);
      first_bad = min(first_bad, __shfl_xor(first_bad, d));
    }
    if (tid == 0) {
      if (first_bad < kLocalGroups) set_error(a.ws.hdr, PGG_DEV_GROUP_NEGATIVE, first_bad);
      else if (total != a.M) set_error(a.ws.hdr, PGG_DEV_GROUP_SUM, total);
    }
  }
  if (a.eri)
    for (int64_t p = tid; p < a.M; p += blockDim.x) {
      const int64_t v = a.eri[p];
      if (v < 0 || v >= a.M) {
        set_error(a.ws.hdr, PGG_DEV_INDEX_RANGE, p);
      } else {
        const uint32_t bit = 1u << (v & 31);
        if (atomicOr(&bits[v >> 5], bit) & bit) set_error(a.ws.hdr, PGG_DEV_INDEX_DUP, v);
      }
    }
}

}  // namespace

}  // namespace pgg
