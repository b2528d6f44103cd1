// Gated linear recurrence: per channel h_t = a_t h_{t-1} + w_t x_t with a = exp(g), its gradients
// and its one-token step (include/delta_block.h).
//
// A hard reset (g = -inf, a = 0) drops the previous state by selection rather than by
// multiplication, so that nothing of it, NaN and infinities included, is seen after it; the same
// holds for the gradient that flows back.  State, gates and sums are float32.
//
// One thread per channel walks the sequence.
#include <hip/hip_runtime.h>

#include "block_kernels.h"
#include "common.h"

namespace delta {
namespace {

enum { NONE = 0, COMPLEMENT = 1, NORM = 2 };

// 1 - exp(z) for z <= 0 to a few units in the last place: the difference cancels near 0, where the
// series -z (1 + z/2 (1 + z/3 (...))) is used (|z| < 0.35: the first dropped term is below
// 0.35^8 / 9! = 6e-10 of the result).
__device__ inline float one_minus_exp(float z) {
  const float series =
      -z * (1.f + z * (1.f / 2) * (1.f + z * (1.f / 3) * (1.f + z * (1.f / 4) * (1.f + z * (1.f / 5) *
      (1.f + z * (1.f / 6) * (1.f + z * (1.f / 7) * (1.f + z * (1.f / 8))))))));
  return fabsf(z) < 0.35f ? series : 1.f - gate_exp(z);
}

template <int GATE>
__device__ inline float weight(float g) {
  if constexpr (GATE == NONE) return 1.f;
  if constexpr (GATE == COMPLEMENT) return one_minus_exp(g);
  return __builtin_amdgcn_sqrtf(fmaxf(one_minus_exp(2.f * g), 0.f));
}

// dw/dg
template <int GATE>
__device__ inline float slope(float a, float w) {
  if constexpr (GATE == NONE) return 0.f;
  if constexpr (GATE == COMPLEMENT) return -a;
  return w > 0.f ? -a * a * __builtin_amdgcn_rcpf(w) : 0.f;
}

__device__ inline float step(float a, float h, float u) { return a == 0.f ? u : a * h + u; }

template <typename E, int GATE>
__global__ __launch_bounds__(64) void glr_fwd_kernel(GlrParams p) {
  const int nb = (p.D + 63) / 64;
  const int b = blockIdx.x / nb, c = (blockIdx.x % nb) * 64 + threadIdx.x;
  if (c >= p.D) return;
  const long base = (long)b * p.L * p.D + c;
  const long sc = (long)b * p.D + c;
  const int nc = (p.L + GLR_CHUNK - 1) / GLR_CHUNK;
  float h = p.h0 ? p.h0[sc] : 0.f;
  for (int t = 0; t < p.L; ++t) {
    if (p.states && t % GLR_CHUNK == 0) p.states[((long)b * nc + t / GLR_CHUNK) * p.D + c] = h;
    const long i = base + (long)t * p.D;
    const float g = p.g[i];
    h = step(gate_exp(g), h, weight<GATE>(g) * to_float(static_cast<const E*>(p.x)[i]));
    static_cast<E*>(p.O)[i] = to_elem<E>(h);
  }
  if (p.h_final) p.h_final[sc] = h;
}

template <typename E, int GATE>
__global__ __launch_bounds__(64) void glr_bwd_kernel(GlrParams p) {
  const int nb = (p.D + 63) / 64;
  const int b = blockIdx.x / nb, c = (blockIdx.x % nb) * 64 + threadIdx.x;
  if (c >= p.D) return;
  const long base = (long)b * p.L * p.D + c;
  const long sc = (long)b * p.D + c;
  const int nc = (p.L + GLR_CHUNK - 1) / GLR_CHUNK;
  float flow = p.dh_final ? p.dh_final[sc] : 0.f;
  for (int n = nc - 1; n >= 0; --n) {
    // dh_t / dg_t of the chunk's tokens, from its start state; then the chunk in reverse
    float q[GLR_CHUNK];
    float h = p.states[((long)b * nc + n) * p.D + c];
#pragma unroll
    for (int j = 0; j < GLR_CHUNK; ++j) {
      const int t = n * GLR_CHUNK + j;
      q[j] = 0.f;
      if (t < p.L) {
        const long i = base + (long)t * p.D;
        const float g = p.g[i], a = gate_exp(g), w = weight<GATE>(g), x = to_float(static_cast<const E*>(p.x)[i]);
        q[j] = a == 0.f ? 0.f : a * h + slope<GATE>(a, w) * x;
        h = step(a, h, w * x);
      }
    }
#pragma unroll
    for (int j = GLR_CHUNK - 1; j >= 0; --j) {
      const int t = n * GLR_CHUNK + j;
      if (t < p.L) {
        const long i = base + (long)t * p.D;
        const float g = p.g[i], a = gate_exp(g), lam = to_float(static_cast<const E*>(p.dO)[i]) + flow;
        p.dx[i] = weight<GATE>(g) * lam;
        p.dg[i] = a == 0.f ? 0.f : lam * q[j];
        flow = a == 0.f ? 0.f : a * lam;
      }
    }
  }
  if (p.dh0) p.dh0[sc] = flow;
}

template <typename E, int GATE>
__global__ __launch_bounds__(256) void glr_decode_kernel(GlrParams p) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long)p.B * p.D) return;
  const float g = p.g[i];
  const float h = step(gate_exp(g), p.h_final[i], weight<GATE>(g) * to_float(static_cast<const E*>(p.x)[i]));
  p.h_final[i] = h;
  static_cast<E*>(p.O)[i] = to_elem<E>(h);
}

enum Which { FWD, BWD, DECODE };

template <typename E, int GATE>
hipError_t launch_one(const GlrParams& p, Which which, hipStream_t st) {
  const dim3 grid((unsigned)((p.D + 63) / 64) * p.B);
  if (which == FWD) hipLaunchKernelGGL((glr_fwd_kernel<E, GATE>), grid, dim3(64), 0, st, p);
  if (which == BWD) hipLaunchKernelGGL((glr_bwd_kernel<E, GATE>), grid, dim3(64), 0, st, p);
  if (which == DECODE) {
    const long n = (long)p.B * p.D;
    hipLaunchKernelGGL((glr_decode_kernel<E, GATE>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, p);
  }
  return hipGetLastError();
}

template <typename E>
hipError_t launch_gate(const GlrParams& p, Which which, hipStream_t st) {
  switch (p.gate) {
    case NONE: return launch_one<E, NONE>(p, which, st);
    case COMPLEMENT: return launch_one<E, COMPLEMENT>(p, which, st);
    case NORM: return launch_one<E, NORM>(p, which, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch(const GlrParams& p, bool bf16_in, Which which, hipStream_t st) {
  return bf16_in ? launch_gate<bf16>(p, which, st) : launch_gate<float>(p, which, st);
}

}  // namespace

hipError_t launch_glr_fwd(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, FWD, st); }
hipError_t launch_glr_bwd(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, BWD, st); }
hipError_t launch_glr_decode(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, DECODE, st); }

}  // namespace delta
