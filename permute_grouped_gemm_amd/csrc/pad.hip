// Rows of 16-bit elements copied to padded rows, so that each starts on a
// 16-byte boundary: bound by reading and writing them once.  A power of two of
// lanes takes a row (or a few rows share a workgroup), each lane 16 bytes at a
// time; the source is read from any address.
#include <algorithm>

#include "pgg_nn.h"

namespace pgg {

namespace {

__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* src, uint16_t* dst, int64_t rows, int64_t len,
                                                       int64_t pitch, int32_t shift) {
  const int lanes = 1 << shift;
  const int64_t step = static_cast<int64_t>(gridDim.x) << (8 - shift);
  const uint16_t* end = src + rows * len;
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) << (8 - shift)) + (threadIdx.x >> shift); r < rows; r += step)
    for (int64_t c = (threadIdx.x & (lanes - 1)) * 8; c < pitch; c += lanes * 8)
      *reinterpret_cast<u32x4_t*>(dst + r * pitch + c) = load16_part<TBf16>(src + r * len + c, len - c, end);
}

}  // namespace

hipError_t launch_pad_rows(const void* src, void* dst, int64_t rows, int64_t len, int64_t pitch, hipStream_t s) {
  int32_t shift = 3;
  while (shift < 8 && (8 << shift) < pitch) ++shift;
  const int64_t blocks = std::min<int64_t>((rows + (256 >> shift) - 1) / (256 >> shift), 4096);
  hipLaunchKernelGGL(pad_rows_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s,
                     static_cast<const uint16_t*>(src), static_cast<uint16_t*>(dst), rows, len, pitch, shift);
  return hipGetLastError();
}

}  // namespace pgg
