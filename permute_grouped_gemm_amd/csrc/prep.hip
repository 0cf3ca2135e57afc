// Kernels of the index preparation; the device code is in pgg_prep.h (the
// weight-sweep producer runs the same preparation in a spare workgroup).
#include "pgg_prep.h"

namespace pgg {

namespace {

__global__ __launch_bounds__(kPrepThreads) void prep_fused_kernel(PrepArgs a, const int64_t* eri,
                                                                  const int64_t* gl, WsView w) {
  __shared__ long long scratch[2 * kPrepThreads];
  prep_block(a, eri, gl, w, scratch);
}

__global__ __launch_bounds__(kPrepThreads) void prep_groups_kernel(PrepArgs a, const int64_t* gl,
                                                                   WsView w) {
  __shared__ long long scratch[2 * kPrepThreads];
  reset_header(w.hdr);
  __syncthreads();
  groups_phase(a, gl, w, scratch, scratch + blockDim.x);
}

__global__ __launch_bounds__(256) void prep_index_kernel(PrepArgs a, const int64_t* eri, WsView w) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t < a.M) index_one(a, eri, w, t);
}

__global__ __launch_bounds__(256) void prep_verify_kernel(PrepArgs a, const int64_t* eri, WsView w) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t < a.M) verify_one(a, eri, w, t);
}

// Workgroup 0: header and group tables.  The others: the index entries, without
// the header (which workgroup 0 may not have reset yet); prep_check_kernel
// reports what they skip.
__global__ __launch_bounds__(kPrepThreads) void prep_tables_kernel(PrepArgs a, const int64_t* eri,
                                                                   const int64_t* gl, WsView w) {
  __shared__ long long scratch[2 * kPrepThreads];
  if (blockIdx.x == 0) {
    reset_header(w.hdr);
    __syncthreads();
    groups_phase(a, gl, w, scratch, scratch + kPrepThreads);
    return;
  }
  const int64_t t = static_cast<int64_t>(blockIdx.x - 1) * blockDim.x + threadIdx.x;
  if (t < a.M && eri[t] >= 0 && eri[t] < a.M) index_one(a, eri, w, t);
}

__global__ __launch_bounds__(256) void prep_check_kernel(PrepArgs a, const int64_t* eri, WsView w) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t >= a.M) return;
  if (eri[t] < 0 || eri[t] >= a.M) set_error(w.hdr, PGG_DEV_INDEX_RANGE, t);
  else verify_one(a, eri, w, t);
}

}  // namespace

hipError_t launch_prep_fused(const Plan& p, const int64_t* eri, const int64_t* gl,
                             const WsView& w, hipStream_t s) {
  // one wave for small problems: its scan barriers cost next to nothing
  const unsigned threads = (p.M <= 4096 && p.G <= 4096) ? 64u : unsigned(kPrepThreads);
  hipLaunchKernelGGL(prep_fused_kernel, dim3(1), dim3(threads), 0, s, prep_args(p), eri, gl, w);
  return hipGetLastError();
}

hipError_t launch_prep_groups(const Plan& p, const int64_t* gl, const WsView& w, hipStream_t s) {
  // Few rows: no more threads than groups keep busy, as every step of the scan is
  // a barrier of all of them.  Whole calls of the gradient in us at 1024 rows, D
  // and F 16, with 64, 256 and 1024 threads: 257 groups 10.8, 9.9, 11.1; 512 13.0,
  // 10.6, 11.5; 1024 18.9, 12.7, 12.8; 2048 30.3, 18.1, 16.4.  (At 64 groups 64
  // threads take 4 us and 1024 take 7.)
  const unsigned threads = p.M > 4096 || p.G > 1024 ? unsigned(kPrepThreads) : p.G > 64 ? 256u : 64u;
  hipLaunchKernelGGL(prep_groups_kernel, dim3(1), dim3(threads), 0, s, prep_args(p), gl, w);
  return hipGetLastError();
}

hipError_t launch_prep_tables(const Plan& p, const int64_t* eri, const int64_t* gl, const WsView& w,
                              hipStream_t s) {
  const unsigned blocks = 1 + static_cast<unsigned>((p.M + kPrepThreads - 1) / kPrepThreads);
  hipLaunchKernelGGL(prep_tables_kernel, dim3(blocks), dim3(kPrepThreads), 0, s, prep_args(p), eri, gl, w);
  return hipGetLastError();
}

hipError_t launch_prep_check(const Plan& p, const int64_t* eri, const WsView& w, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>((p.M + 255) / 256);
  hipLaunchKernelGGL(prep_check_kernel, dim3(blocks), dim3(256), 0, s, prep_args(p), eri, w);
  return hipGetLastError();
}

hipError_t launch_prep_index(const Plan& p, const int64_t* eri, const WsView& w, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>((p.M + 255) / 256);
  hipLaunchKernelGGL(prep_index_kernel, dim3(blocks), dim3(256), 0, s, prep_args(p), eri, w);
  return hipGetLastError();
}

hipError_t launch_prep_verify(const Plan& p, const int64_t* eri, const WsView& w, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>((p.M + 255) / 256);
  hipLaunchKernelGGL(prep_verify_kernel, dim3(blocks), dim3(256), 0, s, prep_args(p), eri, w);
  return hipGetLastError();
}

}  // namespace pgg
