// RMS norm of the residual stream with the residual's addition, its 8-bit form and its backward
// pass (include/delta_block.h).  One workgroup per row; sums in float32.
#include <hip/hip_runtime.h>

#include "block_kernels.h"
#include "common.h"

namespace delta {
namespace {

constexpr int T = 256;
constexpr float E4M3_MAX = 448.f;
constexpr float AMAX_MIN = 0x1p-100f;  // below it a group counts as zeros: 448 / max stays finite

__device__ inline float block_sum(float x, float* lds) {
  x = wave_sum(x);
  __syncthreads();
  if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = x;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < T / WAVE; ++i) s += lds[i];
  return s;
}

// max |v| as the bits of a non-negative float, whose order as integers puts infinity above every
// number and NaN above infinity
__device__ inline unsigned abs_bits(float v) { return __builtin_bit_cast(unsigned, v) & 0x7fffffffu; }
__device__ inline unsigned block_max(unsigned x, unsigned* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = max(x, (unsigned)__shfl_xor((int)x, o, WAVE));
  __syncthreads();
  if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = x;
  __syncthreads();
  unsigned s = 0;
  for (int i = 0; i < T / WAVE; ++i) s = max(s, lds[i]);
  return s;
}

__device__ inline uint8_t to_e4m3(float v) {
  return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xff);
}

template <typename E>
__global__ __launch_bounds__(T) void rmsnorm_kernel(RmsnormParams p) {
  __shared__ float lds[T / WAVE];
  __shared__ unsigned ldu[T / WAVE];
  const long row = blockIdx.x, base = row * p.width;
  const E* x = static_cast<const E*>(p.x) + base;
  const E* r = p.res ? static_cast<const E*>(p.res) + base : nullptr;
  E* sum = p.res ? static_cast<E*>(p.sum) + base : nullptr;
  float ss = 0.f;
  for (int i = threadIdx.x; i < p.width; i += T) {
    float s = to_float(x[i]);
    if (r) {
      const E e = to_elem<E>(s + to_float(r[i]));
      sum[i] = e;
      s = to_float(e);
    }
    ss += s * s;
  }
  const float rstd = 1.f / sqrtf(block_sum(ss, lds) / p.width + p.eps);
  const E* s = sum ? sum : x;  // what this thread itself wrote
  if (!p.y8) {
    E* y = static_cast<E*>(p.y) + base;
    for (int i = threadIdx.x; i < p.width; i += T) y[i] = to_elem<E>(to_float(s[i]) * rstd * p.weight[i]);
    return;
  }
  const int ng = (p.width + p.group - 1) / p.group;
  for (int n = 0; n < ng; ++n) {
    const int lo = n * p.group, hi = min(lo + p.group, p.width);
    unsigned m = 0;
    for (int i = threadIdx.x; i < p.width; i += T)
      if (i >= lo && i < hi) m = max(m, abs_bits(to_float(s[i]) * rstd * p.weight[i]));
    const float amax = __builtin_bit_cast(float, block_max(m, ldu));
    const bool zero = amax < AMAX_MIN;
    const float scale = zero ? 0.f : amax / E4M3_MAX, inv = zero ? 0.f : E4M3_MAX / amax;
    for (int i = threadIdx.x; i < p.width; i += T)
      if (i >= lo && i < hi) p.y8[base + i] = to_e4m3(to_float(s[i]) * rstd * p.weight[i] * inv);
    if (threadIdx.x == 0) p.scale[row * ng + n] = scale;
  }
}

// Workgroup j takes rows j, j + parts, ...; dweight's partial sums over its rows go to part[j].
template <typename E>
__global__ __launch_bounds__(T) void rmsnorm_bwd_kernel(RmsnormParams p, int parts) {
  __shared__ float lds[T / WAVE];
  if (p.dweight)
    for (int i = threadIdx.x; i < p.width; i += T) p.part[(long)blockIdx.x * p.width + i] = 0.f;
  for (long row = blockIdx.x; row < p.rows; row += parts) {
    const long base = row * p.width;
    const E* s = static_cast<const E*>(p.x) + base;
    const E* dy = static_cast<const E*>(p.dy) + base;
    const E* ds = p.dsum ? static_cast<const E*>(p.dsum) + base : nullptr;
    float ss = 0.f, dot = 0.f;
    for (int i = threadIdx.x; i < p.width; i += T) {
      const float v = to_float(s[i]);
      ss += v * v;
      dot += p.weight[i] * to_float(dy[i]) * v;
    }
    const float rstd = 1.f / sqrtf(block_sum(ss, lds) / p.width + p.eps);
    const float c = rstd * rstd * rstd * (block_sum(dot, lds) / p.width);
    for (int i = threadIdx.x; i < p.width; i += T) {
      const float v = to_float(s[i]), d = to_float(dy[i]);
      static_cast<E*>(p.dx)[base + i] = to_elem<E>((ds ? to_float(ds[i]) : 0.f) + rstd * (p.weight[i] * d) - v * c);
      if (p.dweight) p.part[(long)blockIdx.x * p.width + i] += d * v * rstd;
    }
  }
}

__global__ __launch_bounds__(T) void rmsnorm_dweight_kernel(const float* part, int parts, int width, float* dweight) {
  const int i = blockIdx.x * T + threadIdx.x;
  if (i >= width) return;
  float s = 0.f;
  for (int j = 0; j < parts; ++j) s += part[(long)j * width + i];
  dweight[i] = s;
}

}  // namespace

hipError_t launch_rmsnorm(const RmsnormParams& p, bool bf16_in, hipStream_t st) {
  const dim3 grid((unsigned)p.rows), block(T);
  if (bf16_in) hipLaunchKernelGGL((rmsnorm_kernel<bf16>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((rmsnorm_kernel<float>), grid, block, 0, st, p);
  return hipGetLastError();
}

int rmsnorm_bwd_parts(long rows, int) { return (int)(rows < 512 ? rows : 512); }

hipError_t launch_rmsnorm_bwd(const RmsnormParams& p, bool bf16_in, hipStream_t st) {
  const int parts = rmsnorm_bwd_parts(p.rows, p.width);
  if (parts > 0) {
    if (bf16_in) hipLaunchKernelGGL((rmsnorm_bwd_kernel<bf16>), dim3(parts), dim3(T), 0, st, p, parts);
    else hipLaunchKernelGGL((rmsnorm_bwd_kernel<float>), dim3(parts), dim3(T), 0, st, p, parts);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (!p.dweight) return hipSuccess;
  hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((p.width + T - 1) / T), dim3(T), 0, st, p.part, parts, p.width,
                     p.dweight);
  return hipGetLastError();
}

}  // namespace delta
