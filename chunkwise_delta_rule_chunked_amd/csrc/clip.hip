// Global norm of a set of gradients and their clipping by it (include/delta_block.h).
//
// The tensors of a launch come by value in its arguments, so nothing is copied to the device first.
// Each is cut into pieces of CLIP_PIECE elements; workgroup j sums the squares of pieces j, j + parts,
// ... in float64 and stores one partial sum, so the result does not depend on the order in which
// workgroups run.  Where one launch holds all tensors, every workgroup of the scaling then adds up the
// partial sums itself (in one fixed order, so all get the same norm), which saves a launch between the two.
//
// Bound by bytes: one read for the norm, one read and one write for the scaling.  Tensors start at any
// element: 16-byte accesses at element alignment, as gfx950 allows.  The sums load ordinarily, the scaling
// loads and stores non-temporally: what the sums leave in the 256 MB cache serves the scaling.  102M float32
// values (1.22 GB in all) take 197 us, 6.2 TB/s, the rate of a streaming copy; 206 with non-temporal loads
// in the sums, 209 with ordinary ones in the scaling, 202 scaling from the last piece to the first.
#include <hip/hip_runtime.h>

#include "block_kernels.h"
#include "common.h"

namespace delta {
namespace {

constexpr int T = 256;
constexpr int U = 4;  // vectors of a lane in flight

__device__ inline double block_sum(double x, double* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, WAVE);
  __syncthreads();
  if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = x;
  __syncthreads();
  double s = 0.;
#pragma unroll
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

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // at any element

template <typename E>
struct Vec {
  static constexpr int N = 16 / sizeof(E);
  __device__ static inline void unpack(u32x4 r, float* v) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if constexpr (sizeof(E) == 4) v[e] = __builtin_bit_cast(float, (uint32_t)r[e]);
      else v[e] = __builtin_bit_cast(float, e % 2 ? r[e / 2] & 0xffff0000u : r[e / 2] << 16);
    }
  }
  __device__ static inline u32x4 pack(const float* v) {
    E x[N];
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = to_elem<E>(v[e]);
    u32x4 r;
    __builtin_memcpy(&r, x, 16);
    return r;
  }
};

template <typename E>
__device__ inline double piece_sum(const E* g, long n) {
  constexpr int N = Vec<E>::N;
  double s[4] = {};
  long k = (long)threadIdx.x * N;
  for (; k + (U - 1) * T * N + N <= n; k += (long)U * T * N) {
    u32x4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = *reinterpret_cast<const u32x4_any*>(g + k + u * T * N);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[N];
      Vec<E>::unpack(r[u], v);
#pragma unroll
      for (int e = 0; e < N; ++e) s[e % 4] = __builtin_fma((double)v[e], (double)v[e], s[e % 4]);
    }
  }
  for (; k < n; k += T * N)
    for (int e = 0; e < N && k + e < n; ++e) {
      const double v = to_float(g[k + e]);
      s[0] += v * v;
    }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__global__ __launch_bounds__(T) void grad_sums_kernel(ClipTable t, double* sums, int parts) {
  __shared__ double lds[T / WAVE];
  double s = 0.;
  for (int piece = blockIdx.x; piece < t.first[t.count]; piece += parts) {
    const int i = tensor_of(t, piece);
    const long lo = (piece - t.first[i]) * CLIP_PIECE, n = min(CLIP_PIECE, (long)t.n[i] - lo);
    s += is_bf16(t, i) ? piece_sum(static_cast<const bf16*>(t.g[i]) + lo, n)
                       : piece_sum(static_cast<const float*>(t.g[i]) + lo, n);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

__device__ inline float norm_of(const double* sums, int parts, double* lds) {
  double s = 0.;
  for (int i = threadIdx.x; i < parts; i += T) s += sums[i];
  return (float)sqrt(block_sum(s, lds));
}

__global__ __launch_bounds__(T) void grad_finish_kernel(const double* sums, int parts, float* norm) {
  __shared__ double lds[T / WAVE];
  const float n = norm_of(sums, parts, lds);
  if (threadIdx.x == 0) *norm = n;
}

template <typename E>
__device__ inline void piece_scale(const E* g, E* out, long n, float c) {
  constexpr int N = Vec<E>::N;
  long k = (long)threadIdx.x * N;
  for (; k + (U - 1) * T * N + N <= n; k += (long)U * T * N) {
    u32x4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(g + k + u * T * N));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[N];
      Vec<E>::unpack(r[u], v);
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] *= c;
      __builtin_nontemporal_store(Vec<E>::pack(v), reinterpret_cast<u32x4_any*>(out + k + u * T * N));
    }
  }
  for (; k < n; k += T * N)
    for (int e = 0; e < N && k + e < n; ++e) out[k + e] = to_elem<E>(c * to_float(g[k + e]));
}

__global__ __launch_bounds__(T) void grad_scale_kernel(ClipTable t, const double* sums, int parts, float max_norm,
                                                      float eps, float* norm) {
  __shared__ double lds[T / WAVE];
  const float total = parts < 0 ? *norm : norm_of(sums, parts, lds);
  if (parts >= 0 && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  const float d = total + eps, r = max_norm / d;
  const float c = r >= 1.f || d == 0.f ? 1.f : r;  // NaN stays NaN
  const int piece = blockIdx.x;
  if (piece >= t.first[t.count]) return;  // no elements at all: the norm is all there is to write
  const int i = tensor_of(t, piece);
  const long lo = (piece - t.first[i]) * CLIP_PIECE, n = min(CLIP_PIECE, (long)t.n[i] - lo);
  if (c == 1.f && t.g[i] == t.out[i]) return;
  if (is_bf16(t, i)) piece_scale(static_cast<const bf16*>(t.g[i]) + lo, static_cast<bf16*>(t.out[i]) + lo, n, c);
  else piece_scale(static_cast<const float*>(t.g[i]) + lo, static_cast<float*>(t.out[i]) + lo, n, c);
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
hipError_t launch_grad_scale(const ClipTable& t, const double* sums, int parts, float max_norm, float eps, float* norm,
                             hipStream_t st) {
  const int wgs = t.first[t.count];
  hipLaunchKernelGGL(grad_scale_kernel, dim3(wgs > 0 ? wgs : 1), dim3(T), 0, st, t, sums, parts, max_norm, eps, norm);
  return hipGetLastError();
}

}  // namespace delta
