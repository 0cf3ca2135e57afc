// Experts' products with 4-bit weights, few rows per expert: bound by reading
// the used experts' weights once.
//
// A wave takes BM rows x 64 columns and a part of the reduction, and walks its
// tiles of 128 k on its own, without a barrier: 4 KiB of codes a tile go straight
// into registers, two tiles ahead, and so does x (its rows are read by every
// column block, from L1 and L2).  A workgroup's waves share column blocks and parts
// as the plan says; the sums of one block meet in LDS at the end.  Where that makes
// too few workgroups, the reduction is split over workgroups too, and a second
// kernel adds the partial results in order.
//
// Measured: 128 rows, 12 experts of 7168 x 4096 in groups of 128, bf16, 182 MB in
// 37 us, 4.9 TB/s (a large copy on this card: 4.9); one row for each of 64 experts
// of that size 152 us, 6.4 TB/s of codes and scales.  The codes carry the
// non-temporal hint: with 8 layers' weights in turn the 12 experts take 38.9 us with
// it and 41.7 without (one layer again and again, which a model does not do, 38.7 and
// 34.1: it fits the last cache).  Where few experts have all rows, whose codes several
// tiles read, it costs instead: 4 layers in turn, 16 experts, rows on all of them 46.4
// and 50.2, on 2 26.6 and 24.1; 64 experts of 2048 x 2816, 37.4 and 41.3, 30.6 and 26.7.
#include <algorithm>

#include "pgg_w4.h"

namespace pgg {

namespace {

// What a wave holds of x for one tile.
template <class T, int RB>
struct W4Rows {
  u32x4_t x[RB][4][W4Type<T>::kVec];

  // kb past the last: the last again
  __device__ __forceinline__ void load(const W4Args& a, int kb, const typename T::elem* const (&px)[RB], int lane) {
    const int64_t k0 = static_cast<int64_t>(min(kb, a.KB - 1)) * kW4K;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s) w4_load_x<T>(x[i][s], px[i] + k0 + 32 * s, a.K - k0 - 32 * s - 8 * (lane >> 4));
  }
};

template <class T, int RB, int SUB>
__device__ __forceinline__ void w4_multiply(const W4Weights<T, SUB>& w, const W4Rows<T, RB>& rows, f32x4_t (&acc)[RB][4]) {
  using Mma = typename W4Type<T>::Mma;
  constexpr int P = W4Type<T>::kParts;
#pragma unroll
  for (int u = 0; u < SUB; ++u) {
    f32x4_t part[RB][4], sum[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      sum[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 4; ++j) part[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int s = u * 4 / SUB; s < (u + 1) * 4 / SUB; ++s) {
      __builtin_amdgcn_sched_barrier(0);   // the operands of one step at a time
      u32x4_t f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = w4_expand<Mma>(w.code[j][s]);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        u32x4_t p[P];
        w4_parts<T, false>(rows.x[i][s], p);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          mma_block<Mma>(sum[i], p[q], ones<Mma>());
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_block<Mma>(part[i][j], p[q], f[j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float scale = w.scale[u].get(j), zero = w.zero_of(u, j);
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[i][j][v] = __builtin_fmaf(scale, __builtin_fmaf(-zero, sum[i][v], part[i][j][v]), acc[i][j][v]);
      }
  }
}

// Tiles of 128 k that are loaded ahead, and waves to a SIMD.  More tiles cost
// registers and so waves: 3 tiles, of codes alone or of both, took 40 to 44 us
// where 2 take 37 (128 rows x 7168 x 4096, 12 experts, bf16).
constexpr int kAhead = 2;
template <class T, int RB>
constexpr int kW4Waves = __is_same(T, TF32) || RB == 2 ? 2 : 3;

constexpr int kW4MaxWaves = 8;

template <class T, int RB, int SUB>
__global__ __launch_bounds__(kW4MaxWaves * 64) __attribute__((amdgpu_waves_per_eu(kW4Waves<T, RB>)))
void w4_rows_kernel(W4Args a) {
  using E = typename T::elem;
  constexpr int BM = 16 * RB, kPitch = kW4Cols + 4;
  __shared__ float lds[kW4MaxWaves * BM * kPitch];
  __shared__ int32_t s_rows[BM];
  static_assert(sizeof(lds) * 8 >= kLocalRows, "a bit per row for the check of the index");

  int bid = blockIdx.x;
  if (a.local) {
    if (bid == 0) {
      w4_check(a, reinterpret_cast<uint32_t*>(lds));
      return;
    }
    --bid;
  }
  const int ct = bid % a.n_col_tiles;
  const int split = bid / a.n_col_tiles % a.ksplit;
  MTile tile;
  if (!w4_find(a, bid / a.n_col_tiles / a.ksplit, BM, tile, s_rows)) return;

  // waves: `beside` with column blocks side by side, and these times `waves`
  // parts of the reduction
  const int lane = threadIdx.x & 63, beside = a.beside, waves = (blockDim.x >> 6) / beside;
  const int id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = id / beside;
  const int cb = ct * beside + id % beside;
  const bool there = cb < a.CB;   // the last workgroup of a row may have waves too many
  const E* px[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
    px[i] = static_cast<const E*>(a.x) + s_rows[16 * i + (lane & 15)] * a.lda + 8 * (lane >> 4);
  const W4Planes planes =
      w4_planes<T, SUB>(a, static_cast<int64_t>(__builtin_amdgcn_readfirstlane(tile.g)) * a.KB * a.CB + (there ? cb : 0));
  // this wave's tiles of the workgroup's [first, first + count)
  const int first = split * a.kb_span, count = there ? min(a.kb_span, a.KB - first) : 0;
  const int kb0 = first + count * wave / waves, kb1 = first + count * (wave + 1) / waves;

  f32x4_t acc[RB][4];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  W4Weights<T, SUB> w[kAhead];
  W4Rows<T, RB> rows[kAhead];
  auto load = [&](int kb, int to) {
    rows[to].load(a, kb, px, lane);
    __builtin_amdgcn_sched_barrier(0);
    w[to].load(planes, static_cast<uint32_t>(kb) * a.CB, kb < kb1, lane);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) load(kb0 + d, d);
  for (int kb = kb0; kb < kb1; kb += kAhead) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      if (kb + d < kb1) w4_multiply<T, RB, SUB>(w[d], rows[d], acc);
      __builtin_amdgcn_sched_barrier(0);
      load(kb + d + kAhead, d);
    }
  }
  if (w4_not_finite(acc)) w4_again<T, RB, SUB>(a, planes, kb0, kb1, px, lane, acc);

  // the waves' sums, in wave order
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const f32x4_t q = {acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]};
      *reinterpret_cast<f32x4_t*>(lds + (id * BM + 16 * i + 4 * (lane >> 4) + v) * kPitch + 4 * (lane & 15)) = q;
    }
  __syncthreads();
  for (int p = threadIdx.x; p < tile.rows * 16 * beside; p += blockDim.x) {
    const int c = p & 15, b = (p >> 4) % beside, r = (p >> 4) / beside;
    const int block = ct * beside + b;
    if (block >= a.CB) continue;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(lds + (b * BM + r) * kPitch + 4 * c);
    for (int w = 1; w < waves; ++w)
      v += *reinterpret_cast<const f32x4_t*>(lds + ((w * beside + b) * BM + r) * kPitch + 4 * c);
    const int64_t row = tile.row0 + r;
    if (a.part) {
      float* to = a.part + (static_cast<int64_t>(split) * a.M + row) * (64ll * a.CB) + 64ll * block + 4 * c;
      *reinterpret_cast<f32x4_t*>(to) = v;
    } else {
      w4_store<T>(a, row, block, c, v);
    }
  }
}

// Adds the splits' partial results in split order and stores the result.
template <class T>
__global__ __launch_bounds__(256) void w4_finish_kernel(W4Args a) {
  if (a.hdr->err != kNoError) return;
  const int64_t pieces = 16ll * a.CB, n = a.M * pieces, plane = a.M * 64ll * a.CB;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < n; e += step) {
    const int64_t row = e / pieces, p = e - row * pieces;
    const float* from = a.part + e * 4;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(from);
    for (int32_t s = 1; s < a.ksplit; ++s) v += *reinterpret_cast<const f32x4_t*>(from + s * plane);
    w4_store<T>(a, row, p >> 4, static_cast<int>(p & 15), v);
  }
}

// The layout: a thread makes the 16 bytes of one lane in all four blocks, from 4
// codes (gated: 2 gate and 2 up) of 32 rows.
__global__ __launch_bounds__(256) void w4_pack_codes_kernel(const uint8_t* codes, uint8_t* packed, int64_t K, int64_t N,
                                                            int32_t KB, int32_t CB, int32_t gated, int64_t total) {
  const int64_t F = N / 2, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; id < total; id += step) {
    const int lane = static_cast<int>(id & 63), i16 = lane & 15;
    const int64_t tile = id >> 6, cb = tile % CB, kb = tile / CB % KB, g = tile / CB / KB;
    const int64_t n0 = w4_column(cb, i16, 0, gated, F), n2 = w4_column(cb, i16, 2, gated, F);
    const int64_t left = (gated ? F : N) - n0;   // columns from n0 on
    const int64_t k0 = kb * kW4K + 8 * (lane >> 4);
    const uint8_t* from = codes + (g * K + k0) * N;
    u32x4_t v[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (k0 + 32 * s + i >= K) continue;
        const uint8_t* row = from + (32 * s + i) * N;
        uint8_t c[4] = {0, 0, 0, 0};
        if (left >= (gated ? 2 : 4)) {
          __builtin_memcpy(c, row + n0, 2);
          __builtin_memcpy(c + 2, row + n2, 2);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((gated ? j & 1 : j) < left) c[j] = row[w4_column(cb, i16, j, gated, F)];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] |= (c[j] & 15u) << (8 * (i & 3) + 4 * (i >> 2));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j][s] = w[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<u32x4_t*>(packed)[tile * 256 + 64 * j + lane] = v[j];
  }
}

// Scales and zero points: a thread makes one of each.
template <class E>
__global__ __launch_bounds__(256) void w4_pack_scales_kernel(const E* scales, const uint8_t* zeros, E* out_s,
                                                             uint8_t* out_z, int64_t rows, int64_t N, int64_t group_size,
                                                             int32_t KB, int32_t CB, int32_t sub, int32_t gated,
                                                             int64_t total) {
  const int64_t F = N / 2, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; id < total; id += step) {
    const int i = static_cast<int>(id & 63) >> 2, j = static_cast<int>(id & 3);
    const int64_t u = (id >> 6) % sub, tile = (id >> 6) / sub;
    const int64_t cb = tile % CB, kb = tile / CB % KB, g = tile / CB / KB;
    const int64_t n = w4_column(cb, i, j, gated, F);
    const bool inside = gated ? cb * 32 + 2 * i + (j & 1) < F : n < N;
    const int64_t r = (kb * kW4K + u * (kW4K / sub)) / group_size;
    const bool have = inside && r < rows;
    const int64_t at = (g * rows + r) * N + n;
    out_s[id] = have ? scales[at] : E(0);
    if (out_z) out_z[id] = have ? zeros[at] & 15 : 0;
  }
}

unsigned blocks_for(int64_t n) { return static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 1 << 20)); }

template <class T, int RB, int SUB>
hipError_t launch_rows(const W4Plan& p, const W4Args& a, hipStream_t s) {
  const unsigned blocks = (a.local ? 1u : 0u) + static_cast<unsigned>(a.n_slots) * a.n_col_tiles * a.ksplit;
  hipLaunchKernelGGL((w4_rows_kernel<T, RB, SUB>), dim3(blocks), dim3(64u * p.waves * a.beside), 0, s, a);
  return hipGetLastError();
}

template <class T, int RB>
hipError_t launch_sub(const W4Plan& p, const W4Args& a, hipStream_t s) {
  if (p.sub == 1) return launch_rows<T, RB, 1>(p, a, s);
  return p.sub == 2 ? launch_rows<T, RB, 2>(p, a, s) : launch_rows<T, RB, 4>(p, a, s);
}

template <class T>
hipError_t launch_typed(const W4Plan& p, const W4Args& a, hipStream_t s) {
  hipError_t e;
  if (p.tiles) e = launch_w4_tile(p, a, s);
  else if constexpr (__is_same(T, TF32)) e = launch_sub<T, 1>(p, a, s);
  else e = p.base.bm == 16 ? launch_sub<T, 1>(p, a, s) : launch_sub<T, 2>(p, a, s);
  if (e != hipSuccess || a.ksplit == 1) return e;
  hipLaunchKernelGGL((w4_finish_kernel<T>), dim3(std::min(blocks_for(a.M * 16 * a.CB), 2048u)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_pack(const W4Layout& l, const uint8_t* codes, const void* scales, const uint8_t* zeros,
                          void* packed, hipStream_t s) {
  char* base = static_cast<char*>(packed);
  const int64_t lanes = l.tiles * 64, entries = l.tiles * l.sub * 64;
  hipLaunchKernelGGL(w4_pack_codes_kernel, dim3(blocks_for(lanes)), dim3(256), 0, s, codes,
                     reinterpret_cast<uint8_t*>(base), l.K, l.N, l.KB, l.CB, l.gated, lanes);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  uint8_t* z = l.zeros ? reinterpret_cast<uint8_t*>(base + l.off_zeros) : nullptr;
  const int64_t rows = (l.K + l.group_size - 1) / l.group_size;
  if (l.dtype == PGG_F32)
    hipLaunchKernelGGL((w4_pack_scales_kernel<uint32_t>), dim3(blocks_for(entries)), dim3(256), 0, s,
                       static_cast<const uint32_t*>(scales), zeros, reinterpret_cast<uint32_t*>(base + l.off_scales), z,
                       rows, l.N, l.group_size, l.KB, l.CB, l.sub, l.gated, entries);
  else
    hipLaunchKernelGGL((w4_pack_scales_kernel<uint16_t>), dim3(blocks_for(entries)), dim3(256), 0, s,
                       static_cast<const uint16_t*>(scales), zeros, reinterpret_cast<uint16_t*>(base + l.off_scales), z,
                       rows, l.N, l.group_size, l.KB, l.CB, l.sub, l.gated, entries);
  return hipGetLastError();
}

hipError_t launch_w4(const W4Plan& p, int32_t act, const void* x, const void* packed, const int64_t* eri,
                     const int64_t* group_list, void* out, void* ws, hipStream_t s) {
  const WsView w = ws_view(p.base, ws);
  const W4Layout& l = p.layout;
  const char* base = static_cast<const char*>(packed);
  W4Args a = {};
  a.x = x;
  if (p.base.pad_a) {   // rows of whole chunks of 16 bytes; fp32 as pairs of 16-bit elements
    const int64_t halves = l.dtype == PGG_F32 ? 2 : 1;
    void* padded = static_cast<char*>(ws) + p.base.off_pad_a;
    const hipError_t e = launch_pad_rows(x, padded, p.base.batch, l.K * halves, p.base.lda * halves, s);
    if (e != hipSuccess) return e;
    a.x = padded;
  }
  a.codes = reinterpret_cast<const uint8_t*>(base);
  a.scales = base + l.off_scales;
  a.zeros = l.zeros ? reinterpret_cast<const uint8_t*>(base + l.off_zeros) : nullptr;
  a.out = out;
  a.part = p.ksplit > 1 ? w.ring : nullptr;
  a.hdr = w.hdr;
  a.tiles = w.tiles;
  a.ori = w.ori;
  a.M = p.base.M;
  a.K = p.base.pad_a ? p.base.lda : l.K;
  a.cols = l.gated ? l.N / 2 : l.N;
  a.lda = p.base.lda;
  a.KB = l.KB;
  a.CB = l.CB;
  a.kb_span = p.kb_span;
  a.ksplit = p.ksplit;
  a.sums = reinterpret_cast<const float*>(static_cast<const char*>(ws) + p.off_sums);
  a.n_slots = p.base.max_tiles;
  a.beside = p.tiles ? 4 : p.beside;
  a.n_col_tiles = (l.CB + a.beside - 1) / a.beside;
  a.topk = static_cast<uint32_t>(p.base.topk);
  a.gated = l.gated;
  a.act = act;
  a.local = p.base.local;
  a.eri = eri;
  a.gl = group_list;
  a.prep = prep_args(p.base);
  a.ws = w;
  if (l.dtype == PGG_F32) return launch_typed<TF32>(p, a, s);
  return l.dtype == PGG_BF16 ? launch_typed<TBf16>(p, a, s) : launch_typed<TF16>(p, a, s);
}

}  // namespace pgg
