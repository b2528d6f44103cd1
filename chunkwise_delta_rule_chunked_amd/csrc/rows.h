// Rows of channels in vectors of eight, at any element: the accesses and reductions that the norms of the
// residual stream share.
#pragma once
#include "common.h"

namespace delta {
namespace rows {

constexpr int V = 8;  // channels of a vector

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // at any element
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef float floatx4_any __attribute__((ext_vector_type(4), aligned(4)));

typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

// The first n < 8 elements at p in pieces of 4, 2 and 1: accesses that do not wait for each other, as a
// row's last vector holds up its whole wavefront.  Elements of 2 bytes, the rest 0:
__device__ inline u32x4 load_part(const bf16* p, int n) {
  u32x2 four = {};
  uint32_t two = 0, one = 0;
  if (n & 4) four = *reinterpret_cast<const u32x2_any*>(p);
  if (n & 2) two = *reinterpret_cast<const u32_any*>(p + (n & 4));
  if (n & 1) one = *reinterpret_cast<const u16_any*>(p + (n & 6));
  const uint32_t lo = n & 2 ? two : one, hi = n & 2 ? one : 0;
  return u32x4{n & 4 ? four[0] : lo, n & 4 ? four[1] : hi, n & 4 ? lo : 0, n & 4 ? hi : 0};
}
__device__ inline void store_part(bf16* p, int n, u32x4 v) {
  if (n & 4) *reinterpret_cast<u32x2_any*>(p) = u32x2{v[0], v[1]};
  const uint32_t lo = n & 4 ? v[2] : v[0], hi = n & 4 ? v[3] : v[1];
  if (n & 2) *reinterpret_cast<u32_any*>(p + (n & 4)) = lo;
  if (n & 1) *reinterpret_cast<u16_any*>(p + (n & 6)) = (uint16_t)(n & 2 ? hi : lo);
}
// of 4 bytes
struct Eight {
  floatx4 lo, hi;
};
__device__ inline Eight load_part(const float* p, int n) {
  floatx4 four = {};
  u32x2 two = {};
  float one = 0.f;
  if (n & 4) four = *reinterpret_cast<const floatx4_any*>(p);
  if (n & 2) two = *reinterpret_cast<const u32x2_any*>(p + (n & 4));
  if (n & 1) one = p[n & 6];
  const float r0 = n & 2 ? __builtin_bit_cast(float, (uint32_t)two[0]) : one;
  const float r1 = __builtin_bit_cast(float, (uint32_t)two[1]), r2 = n & 2 ? one : 0.f;
  Eight v;
  v.lo = floatx4{n & 4 ? four[0] : r0, n & 4 ? four[1] : r1, n & 4 ? four[2] : r2, n & 4 ? four[3] : 0.f};
  v.hi = floatx4{n & 4 ? r0 : 0.f, n & 4 ? r1 : 0.f, n & 4 ? r2 : 0.f, 0.f};
  return v;
}
__device__ inline void store_part(float* p, int n, Eight v) {
  if (n & 4) *reinterpret_cast<floatx4_any*>(p) = v.lo;
  const floatx4 r = n & 4 ? v.hi : v.lo;
  if (n & 2)
    *reinterpret_cast<u32x2_any*>(p + (n & 4)) = u32x2{__builtin_bit_cast(uint32_t, (float)r[0]), __builtin_bit_cast(uint32_t, (float)r[1])};
  if (n & 1) p[n & 6] = n & 2 ? r[2] : r[0];
}
// of 1 byte
__device__ inline void store_part(uint8_t* p, int n, uint32_t lo, uint32_t hi) {
  if (n & 4) *reinterpret_cast<u32_any*>(p) = lo;
  const uint32_t rest = n & 4 ? hi : lo;
  if (n & 2) *reinterpret_cast<u16_any*>(p + (n & 4)) = (uint16_t)rest;
  if (n & 1) p[n & 6] = (uint8_t)(n & 2 ? rest >> 16 : rest);
}

// n of 8 channels (the rest 0; none for n <= 0); n < 8 only in a row's last vector
template <bool NT>
__device__ inline void load8(const bf16* p, int n, float* v) {
  u32x4 r = {};
  if (n >= V) {
    const auto* q = reinterpret_cast<const u32x4_any*>(p);
    r = NT ? __builtin_nontemporal_load(q) : *q;
  } else if (n > 0) {
    r = load_part(p, n);
  }
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = __builtin_bit_cast(float, e % 2 ? r[e / 2] & 0xffff0000u : r[e / 2] << 16);
}
template <bool NT>
__device__ inline void load8(const float* p, int n, float* v) {
  Eight r = {};
  if (n >= V) {
    const auto* q = reinterpret_cast<const floatx4_any*>(p);
    r.lo = NT ? __builtin_nontemporal_load(q) : *q;
    q = reinterpret_cast<const floatx4_any*>(p + 4);
    r.hi = NT ? __builtin_nontemporal_load(q) : *q;
  } else if (n > 0) {
    r = load_part(p, n);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = r.lo[e], v[4 + e] = r.hi[e];
}
__device__ inline void store8(bf16* p, int n, const float* v) {
  bf16 r[V];
#pragma unroll
  for (int e = 0; e < V; ++e) r[e] = to_elem<bf16>(v[e]);
  u32x4 q;
  __builtin_memcpy(&q, r, 16);
  if (n >= V) *reinterpret_cast<u32x4_any*>(p) = q;
  else if (n > 0) store_part(p, n, q);
}
__device__ inline void store8(float* p, int n, const float* v) {
  const Eight r{floatx4{v[0], v[1], v[2], v[3]}, floatx4{v[4], v[5], v[6], v[7]}};
  if (n >= V) {
    *reinterpret_cast<floatx4_any*>(p) = r.lo;
    *reinterpret_cast<floatx4_any*>(p + 4) = r.hi;
  } else if (n > 0) {
    store_part(p, n, r);
  }
}
// eight channels at a byte of a range, outside of which nothing is stored
__device__ inline void buffer_store8(__amdgpu_buffer_rsrc_t b, int off, const float* v, bf16) {
  bf16 r[V];
#pragma unroll
  for (int e = 0; e < V; ++e) r[e] = to_elem<bf16>(v[e]);
  floatx4 q;
  __builtin_memcpy(&q, r, 16);
  buffer_store16(b, off, q);
}
__device__ inline void buffer_store8(__amdgpu_buffer_rsrc_t b, int off, const float* v, float) {
  buffer_store16(b, off, floatx4{v[0], v[1], v[2], v[3]});
  buffer_store16(b, off + 16, floatx4{v[4], v[5], v[6], v[7]});
}
__device__ inline void store8_e4m3(uint8_t* p, int n, const float* v) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  if (n >= V) {
    *reinterpret_cast<u32x2_any*>(p) = u32x2{(uint32_t)lo, (uint32_t)hi};
  } else if (n > 0) {
    store_part(p, n, (uint32_t)lo, (uint32_t)hi);
  }
}

// Reductions over the LANES lanes of a row (a power of two; past a wavefront, over the workgroup,
// through `lds`, one slot per wavefront).  Every lane gets the same value.
template <int LANES>
__device__ inline float row_sum(float x, float* lds) {
#pragma unroll
  for (int o = (LANES < WAVE ? LANES : WAVE) / 2; o > 0; o >>= 1) x += __shfl_xor(x, o, WAVE);
  if constexpr (LANES > WAVE) {
    __syncthreads();
    if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < LANES / WAVE; ++i) x += lds[i];
  }
  return x;
}
// Two sums at once; `slot`: which row of the workgroup's (all slots of a workgroup take every step
// together).
template <int LANES, int W>
__device__ inline void row_sums(float& x, float& y, int slot, float (*lds)[W]) {
#pragma unroll
  for (int o = (LANES < WAVE ? LANES : WAVE) / 2; o > 0; o >>= 1) {
    x += __shfl_xor(x, o, WAVE);
    y += __shfl_xor(y, o, WAVE);
  }
  if constexpr (LANES > WAVE) {
    __syncthreads();
    if (threadIdx.x % WAVE == 0) lds[0][threadIdx.x / WAVE] = x, lds[1][threadIdx.x / WAVE] = y;
    __syncthreads();
    x = y = 0.f;
#pragma unroll
    for (int i = 0; i < LANES / WAVE; ++i) {
      x += lds[0][slot * (LANES / WAVE) + i];
      y += lds[1][slot * (LANES / WAVE) + i];
    }
  }
}

// Eight channels as they are in memory: half a float's registers each for bf16.  What is used twice is
// unpacked twice (`again` keeps the compiler from holding the floats between).
template <typename E>
struct Raw8;
template <>
struct Raw8<bf16> {
  u32x4 r;
  __device__ inline void load(__amdgpu_buffer_rsrc_t b, int off) { r = buffer_load16(b, off); }
  __device__ inline void load(const bf16* p, int n) {
    r = u32x4{};
    if (n >= V) {
      r = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
    } else if (n > 0) {
      r = load_part(p, n);
    }
  }
  __device__ inline float operator[](int e) const {
    return __builtin_bit_cast(float, e % 2 ? r[e / 2] & 0xffff0000u : r[e / 2] << 16);
  }
  __device__ inline void again() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t x = r[i];
      asm volatile("" : "+v"(x));
      r[i] = x;
    }
  }
};
template <>
struct Raw8<float> {
  float v[V];
  __device__ inline void load(__amdgpu_buffer_rsrc_t b, int off) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const floatx4 q = __builtin_bit_cast(floatx4, buffer_load16(b, off + 16 * h));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * h + e] = q[e];
    }
  }
  __device__ inline void load(const float* p, int n) { load8<true>(p, n, v); }
  __device__ inline float operator[](int e) const { return v[e]; }
  __device__ inline void again() {}
};

constexpr int threads(int lanes) { return lanes > WAVE ? lanes : 256; }

}  // namespace rows
}  // namespace delta
