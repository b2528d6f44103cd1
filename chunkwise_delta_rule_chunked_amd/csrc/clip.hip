// Global norm of a set of gradients and their clipping by it (include/delta_block.h).
//
// The tensors of a launch come by value in its arguments.  Each is cut into pieces of CLIP_PIECE
// elements; workgroup j sums the squares of pieces j, j + parts, ... in float64 and stores one
// partial sum, so the result does not depend on the order in which workgroups run.
#include <hip/hip_runtime.h>

#include "block_kernels.h"
#include "common.h"

namespace delta {
namespace {

constexpr int T = 256;

__device__ inline double block_sum(double x, double* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, WAVE);
  __syncthreads();
  if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = x;
  __syncthreads();
  double s = 0.;
  for (int i = 0; i < T / WAVE; ++i) s += lds[i];
  return s;
}

// The tensor that holds piece j: the last one whose first piece is at or before it.
__device__ inline int tensor_of(const ClipTable& t, int piece) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= piece) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ inline bool is_bf16(const ClipTable& t, int i) { return t.bf16[i / 32] >> (i % 32) & 1; }

__device__ inline float load(const void* p, long i, bool b) {
  return b ? to_float(static_cast<const bf16*>(p)[i]) : static_cast<const float*>(p)[i];
}

__global__ __launch_bounds__(T) void grad_sums_kernel(ClipTable t, double* sums, int parts) {
  __shared__ double lds[T / WAVE];
  double s = 0.;
  for (int piece = blockIdx.x; piece < t.first[t.count]; piece += parts) {
    const int i = tensor_of(t, piece);
    const long lo = (piece - t.first[i]) * CLIP_PIECE, hi = min(lo + CLIP_PIECE, (long)t.n[i]);
    const bool b = is_bf16(t, i);
    for (long k = lo + threadIdx.x; k < hi; k += T) {
      const double v = load(t.g[i], k, b);
      s += v * v;
    }
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

__global__ __launch_bounds__(T) void grad_finish_kernel(const double* sums, int parts, float* norm) {
  __shared__ double lds[T / WAVE];
  double s = 0.;
  for (int i = threadIdx.x; i < parts; i += T) s += sums[i];
  s = block_sum(s, lds);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

__global__ __launch_bounds__(T) void grad_scale_kernel(ClipTable t, const float* norm, float max_norm, float eps) {
  const float d = *norm + eps, r = max_norm / d;
  const float c = r >= 1.f || d == 0.f ? 1.f : r;  // NaN stays NaN
  const int piece = blockIdx.x, i = tensor_of(t, piece);
  const long lo = (piece - t.first[i]) * CLIP_PIECE, hi = min(lo + CLIP_PIECE, (long)t.n[i]);
  const bool b = is_bf16(t, i);
  if (c == 1.f && t.g[i] == t.out[i]) return;
  for (long k = lo + threadIdx.x; k < hi; k += T) {
    const float v = c * load(t.g[i], k, b);
    if (b) static_cast<bf16*>(t.out[i])[k] = to_elem<bf16>(v);
    else static_cast<float*>(t.out[i])[k] = v;
  }
}

}  // namespace

hipError_t launch_grad_sums(const ClipTable& t, double* sums, int parts, hipStream_t st) {
  hipLaunchKernelGGL(grad_sums_kernel, dim3(parts), dim3(T), 0, st, t, sums, parts);
  return hipGetLastError();
}
hipError_t launch_grad_finish(const double* sums, int parts, float* norm, hipStream_t st) {
  hipLaunchKernelGGL(grad_finish_kernel, dim3(1), dim3(T), 0, st, sums, parts, norm);
  return hipGetLastError();
}
hipError_t launch_grad_scale(const ClipTable& t, const float* norm, float max_norm, float eps, hipStream_t st) {
  if (t.first[t.count] == 0) return hipSuccess;
  hipLaunchKernelGGL(grad_scale_kernel, dim3(t.first[t.count]), dim3(T), 0, st, t, norm, max_norm, eps);
  return hipGetLastError();
}

}  // namespace delta
