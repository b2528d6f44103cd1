// RMS norm of the residual stream with the residual's addition, its 8-bit form and its backward
// pass (include/delta_block.h).  Sums in float32.
//
// Bound by bytes: each input is read once and each output written once, a row staying in registers
// between its sum and its use.  LANES lanes hold a row, J vectors of 8 channels each (lane l the
// vectors l, l + LANES, ...): one vector where that is possible, up to a workgroup of 512 lanes for 4096
// channels (`split` has what else was measured).  Workgroups walk over rows, keeping the weight (and,
// backward, their part of its gradient) in registers.  Rows that are not a multiple of 8 channels start
// at any element: the same wide accesses at element alignment, which gfx950 allows, with the row's last
// vector in three pieces.  Rows past 32768 channels (backward 16384) take a kernel that reads them twice.
//
// Measured, time on the card, bf16: 16384 rows of 2048, forward 44.5 us (6.0 TB/s), with y in 8 bits 43.5, backward
// 50 to 57 us by where its tensors lie in memory (5.3 to 4.7 TB/s; 5 us for adding up dweight's parts); 65536 x 512
// forward 44.4 us (6.0 TB/s); 32768 x 1003 forward 52 us (5.0 TB/s: accesses that cross their natural alignment),
// x 1008 47 us; 8192 x 1024 backward 20.5 us (3.3 TB/s); 64 x 2048 in 8 bits 3.4 us, the latency of two rounds to
// memory and a launch.  float32, 8192 x 2048: forward 51 us (5.2 TB/s), backward 55.7 us (4.8).  Non-temporal stores
// made no difference to 3% worse.
#include <hip/hip_runtime.h>

#include "block_kernels.h"
#include "common.h"

namespace delta {
namespace {

constexpr int V = 8;  // channels of a vector
constexpr float E4M3_MAX = 448.f;
constexpr float AMAX_MIN = 0x1p-100f;  // below it a group counts as zeros: 448 / max|z w| stays finite

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

// |v| as the bits of a non-negative float, whose order as integers puts infinity above every number
// and NaN above infinity
__device__ inline unsigned abs_bits(float v) { return __builtin_bit_cast(unsigned, v) & 0x7fffffffu; }

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
template <int LANES>
__device__ inline unsigned row_max(unsigned x, unsigned* lds) {
#pragma unroll
  for (int o = (LANES < WAVE ? LANES : WAVE) / 2; o > 0; o >>= 1) x = max(x, (unsigned)__shfl_xor((int)x, o, WAVE));
  if constexpr (LANES > WAVE) {
    __syncthreads();
    if (threadIdx.x % WAVE == 0) lds[threadIdx.x / WAVE] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int i = 0; i < LANES / WAVE; ++i) x = max(x, lds[i]);
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

// The two parts of a row's rstd in the 8-bit form: a power of two `up`, with which s becomes z of order 1
// (exactly), and the rest m in [1, 2).  The products z w are within a factor of 2 of y, so they leave float32's
// range only where y does, which s w would not.  An rstd that is 0, infinite or NaN is all in m.
struct Rstd {
  float up, m;
  __device__ inline explicit Rstd(float rstd) {
    const unsigned b = __builtin_bit_cast(unsigned, rstd), e = b & 0x7f800000u;
    const bool plain = e != 0 && e != 0x7f800000u;
    up = plain ? __builtin_bit_cast(float, e) : 1.f;
    m = plain ? __builtin_bit_cast(float, (b & 0x007fffffu) | 0x3f800000u) : rstd;
  }
};

// How a group's z w, the largest of which is `most` in magnitude, become 8 bits.  m cancels from
// y / scale = 448 z w / max|z w|.
struct Quant {
  float scale, f;  // the value is (z w) f
  __device__ inline Quant(float most, float m) {
    const float amax = most * m;
    const bool zero = amax < AMAX_MIN;
    scale = zero ? 0.f : amax / E4M3_MAX;
    f = zero ? 0.f : E4M3_MAX / most;
  }
};

constexpr int threads(int lanes) { return lanes > WAVE ? lanes : 256; }

// QUANT: 0 y, 1 y8 with a scale per row, 2 y8 with a scale per 128 channels (16 lanes).
template <typename E, int LANES, int J, int QUANT>
__global__ __launch_bounds__(threads(LANES)) void rmsnorm_kernel(RmsnormParams p) {
  constexpr int T = threads(LANES), RPW = T / LANES;
  static_assert(LANES <= WAVE || RPW == 1, "row_sum over wavefronts takes all of the workgroup's");
  __shared__ float lds[T / WAVE];
  __shared__ unsigned ldu[T / WAVE];
  const int lane = threadIdx.x % LANES;
  float w[J][V];
#pragma unroll
  for (int j = 0; j < J; ++j) load8<false>(p.weight + (lane + j * LANES) * V, p.width - (lane + j * LANES) * V, w[j]);
  // every lane of a workgroup takes the same number of steps (barriers inside)
  for (long row0 = (long)blockIdx.x * RPW; row0 < p.rows; row0 += (long)gridDim.x * RPW) {
    const long row = row0 + threadIdx.x / LANES;
    const bool ok = row < p.rows;
    const long base = row * p.width;
    float s[J][V], ss = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = (lane + j * LANES) * V, n = ok ? p.width - i : 0;
      load8<true>(static_cast<const E*>(p.x) + base + i, n, s[j]);
      if (p.res) {
        float r[V];
        load8<true>(static_cast<const E*>(p.res) + base + i, n, r);
#pragma unroll
        for (int e = 0; e < V; ++e) s[j][e] = to_float(to_elem<E>(s[j][e] + r[e]));
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = (lane + j * LANES) * V, n = ok ? p.width - i : 0;
      if (p.res) store8(static_cast<E*>(p.sum) + base + i, n, s[j]);
#pragma unroll
      for (int e = 0; e < V; ++e) ss += s[j][e] * s[j][e];
    }
    const float rstd = 1.f / sqrtf(row_sum<LANES>(ss, lds) / p.width + p.eps);
    const Rstd r(rstd);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) s[j][e] = s[j][e] * (QUANT ? r.up : rstd) * w[j][e];
    if constexpr (QUANT == 0) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int i = (lane + j * LANES) * V;
        store8(static_cast<E*>(p.y) + base + i, ok ? p.width - i : 0, s[j]);
      }
    } else {
      unsigned m[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int n = p.width - (lane + j * LANES) * V;  // what is past the row counts for nothing
        m[j] = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) m[j] = max(m[j], e < n ? abs_bits(s[j][e]) : 0u);
      }
      if constexpr (QUANT == 1) {
#pragma unroll
        for (int j = 1; j < J; ++j) m[0] = max(m[0], m[j]);
        m[0] = row_max<LANES>(m[0], ldu);
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int o = (LANES < 16 ? LANES : 16) / 2; o > 0; o >>= 1) m[j] = max(m[j], (unsigned)__shfl_xor((int)m[j], o, WAVE));
      }
      const int groups = (p.width + p.group - 1) / p.group;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int i = (lane + j * LANES) * V, n = ok ? p.width - i : 0;
        const Quant q(__builtin_bit_cast(float, m[QUANT == 1 ? 0 : j]), r.m);
#pragma unroll
        for (int e = 0; e < V; ++e) s[j][e] *= q.f;
        store8_e4m3(p.y8 + base + i, n, s[j]);
        if (n > 0 && i % p.group == 0) p.scale[row * groups + i / p.group] = q.scale;
      }
    }
  }
}

// Rows of any width, read again for each use.
template <typename E, int QUANT>
__global__ __launch_bounds__(1024) void rmsnorm_wide_kernel(RmsnormParams p) {
  constexpr int T = 1024;
  __shared__ float lds[T / WAVE];
  __shared__ unsigned ldu[T / WAVE];
  const long row = blockIdx.x, base = row * p.width;
  const E* x = static_cast<const E*>(p.x) + base;
  E* sum = static_cast<E*>(p.sum) + base;
  float ss = 0.f;
  for (int i = threadIdx.x * V; i < p.width; i += T * V) {
    float s[V];
    load8<false>(x + i, p.width - i, s);
    if (p.res) {
      float r[V];
      load8<false>(static_cast<const E*>(p.res) + base + i, p.width - i, r);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = to_float(to_elem<E>(s[e] + r[e]));
      store8(sum + i, p.width - i, s);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) ss += s[e] * s[e];
  }
  const float rstd = 1.f / sqrtf(row_sum<T>(ss, lds) / p.width + p.eps);
  const Rstd r(rstd);
  const E* s0 = p.res ? sum : x;  // what this thread itself wrote
  auto normed = [&](int i, float* y) {
    float w[V];
    load8<false>(s0 + i, p.width - i, y);
    load8<false>(p.weight + i, p.width - i, w);
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = y[e] * (QUANT ? r.up : rstd) * w[e];
  };
  const int groups = (p.width + p.group - 1) / p.group;
  unsigned all = 0;
  if constexpr (QUANT == 1) {
    for (int i = threadIdx.x * V; i < p.width; i += T * V) {
      float y[V];
      normed(i, y);
#pragma unroll
      for (int e = 0; e < V; ++e) all = max(all, i + e < p.width ? abs_bits(y[e]) : 0u);
    }
    all = row_max<T>(all, ldu);
  }
  // whole groups of 16 lanes take a step together
  for (int i = threadIdx.x * V; i - threadIdx.x % 16 * V < p.width; i += T * V) {
    const int n = p.width - i;
    float y[V] = {};
    if (n > 0) normed(i, y);
    if constexpr (QUANT == 0) {
      if (n > 0) store8(static_cast<E*>(p.y) + base + i, n, y);
    } else {
      unsigned m = all;
      if constexpr (QUANT == 2) {
#pragma unroll
        for (int e = 0; e < V; ++e) m = max(m, e < n ? abs_bits(y[e]) : 0u);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, (unsigned)__shfl_xor((int)m, o, WAVE));
      }
      const Quant q(__builtin_bit_cast(float, m), r.m);
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] *= q.f;
      if (n > 0) {
        store8_e4m3(p.y8 + base + i, n, y);
        if (i % p.group == 0) p.scale[row * groups + i / p.group] = q.scale;
      }
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
  __device__ inline void load(const float* p, int n) { load8<true>(p, n, v); }
  __device__ inline float operator[](int e) const { return v[e]; }
  __device__ inline void again() {}
};

constexpr int bwd_threads(int lanes) { return lanes > 512 ? lanes : 512; }

// Workgroup k takes rows k RPW .., then gridDim.x * RPW further on, and stores its part of dweight in
// part[k].  Every part is the sum over a fixed set of rows in a fixed order.
// With z = s rstd, dx = dsum + rstd (w dy - z mean(w dy z)), dweight = sum dy z: z is of order 1 whatever the
// row's size, where rstd^3 leaves float32's range from rms 1e13 on (and below 1e-13 with eps = 0).
template <typename E, int LANES, int J>
__global__ __launch_bounds__(bwd_threads(LANES), 4) void rmsnorm_bwd_kernel(RmsnormParams p) {
  constexpr int T = bwd_threads(LANES), RPW = T / LANES, COLS = LANES * J * V;
  __shared__ float lds[2][T / WAVE];
  const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
  float w[J][V], acc[J][V];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    load8<false>(p.weight + (lane + j * LANES) * V, p.width - (lane + j * LANES) * V, w[j]);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[j][e] = 0.f;
  }
  for (long row0 = (long)blockIdx.x * RPW; row0 < p.rows; row0 += (long)gridDim.x * RPW) {
    const long row = row0 + slot;
    const bool ok = row < p.rows;
    const long base = row * p.width;
    Raw8<E> s[J], d[J], o[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = (lane + j * LANES) * V, n = ok ? p.width - i : 0;
      s[j].load(static_cast<const E*>(p.x) + base + i, n);
      d[j].load(static_cast<const E*>(p.dy) + base + i, n);
    }
    if (p.dsum) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int i = (lane + j * LANES) * V;
        o[j].load(static_cast<const E*>(p.dsum) + base + i, ok ? p.width - i : 0);
      }
    }
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        ss += s[j][e] * s[j][e];
        dot += w[j][e] * d[j][e] * s[j][e];
      }
      s[j].again(), d[j].again();
      __builtin_amdgcn_sched_barrier(0);
    }
    row_sums<LANES>(ss, dot, slot, lds);
    const float rstd = 1.f / sqrtf(ss / p.width + p.eps);
    const float c = rstd * (dot / p.width);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = (lane + j * LANES) * V, n = ok ? p.width - i : 0;
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float z = s[j][e] * rstd;
        v[e] = (p.dsum ? o[j][e] : 0.f) + rstd * (w[j][e] * d[j][e] - z * c);
        if (ok) acc[j][e] += d[j][e] * z;  // a missing row's rstd is infinite for eps = 0
      }
      store8(static_cast<E*>(p.dx) + base + i, n, v);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (!p.dweight) return;
  float* part = p.part + (long)blockIdx.x * p.width;
  if constexpr (RPW == 1) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = (lane + j * LANES) * V;
      store8(part + i, p.width - i, acc[j]);
    }
  } else {
    // the RPW row slots add up in turn
    __shared__ float sums[COLS];
    for (int k = 0; k < RPW; ++k) {
      __syncthreads();
      if (slot == k) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            float* q = sums + (lane + j * LANES) * V + e;
            *q = k ? *q + acc[j][e] : acc[j][e];
          }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.width; i += T) part[i] = sums[i];
  }
}

template <typename E>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_wide_kernel(RmsnormParams p) {
  constexpr int T = 1024;
  __shared__ float lds[T / WAVE];
  float* part = p.part + (long)blockIdx.x * p.width;
  bool first = true;
  for (long row = blockIdx.x; row < p.rows; row += gridDim.x, first = false) {
    const long base = row * p.width;
    float ss = 0.f, dot = 0.f;
    for (int i = threadIdx.x * V; i < p.width; i += T * V) {
      float s[V], d[V], w[V];
      load8<false>(static_cast<const E*>(p.x) + base + i, p.width - i, s);
      load8<false>(static_cast<const E*>(p.dy) + base + i, p.width - i, d);
      load8<false>(p.weight + i, p.width - i, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        ss += s[e] * s[e];
        dot += w[e] * d[e] * s[e];
      }
    }
    const float rstd = 1.f / sqrtf(row_sum<T>(ss, lds) / p.width + p.eps);
    const float c = rstd * (row_sum<T>(dot, lds) / p.width);
    for (int i = threadIdx.x * V; i < p.width; i += T * V) {
      float s[V], d[V], w[V], o[V] = {}, a[V] = {};
      load8<false>(static_cast<const E*>(p.x) + base + i, p.width - i, s);
      load8<false>(static_cast<const E*>(p.dy) + base + i, p.width - i, d);
      load8<false>(p.weight + i, p.width - i, w);
      if (p.dsum) load8<false>(static_cast<const E*>(p.dsum) + base + i, p.width - i, o);
      if (!first && p.dweight) load8<false>(part + i, p.width - i, a);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float z = s[e] * rstd;
        o[e] = o[e] + rstd * (w[e] * d[e] - z * c);
        a[e] += d[e] * z;
      }
      store8(static_cast<E*>(p.dx) + base + i, p.width - i, o);
      if (p.dweight) store8(part + i, p.width - i, a);
    }
  }
}

// dweight = the sum of the parts: 16 columns and 64 lanes over the parts per workgroup.
constexpr int DW_THREADS = 1024;
__global__ __launch_bounds__(DW_THREADS) void rmsnorm_dweight_kernel(const float* part, int parts, int width, float* dweight) {
  __shared__ float sums[DW_THREADS / WAVE][17];
  const int col = threadIdx.x % 16, i = blockIdx.x * 16 + col;
  float s = 0.f;
  if (i < width)
#pragma unroll 8
    for (int k = threadIdx.x / 16; k < parts; k += DW_THREADS / 16) s += part[(long)k * width + i];
  s += __shfl_xor(s, 16, WAVE);
  s += __shfl_xor(s, 32, WAVE);
  if (threadIdx.x % WAVE < 16) sums[threadIdx.x / WAVE][col] = s;
  __syncthreads();
  if (threadIdx.x < 16 && i < width) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < DW_THREADS / WAVE; ++k) s += sums[k][col];
    dweight[i] = s;
  }
}

// Lanes and vectors per lane of a row (0: the kernels for any width), and the workgroups that walk over
// the rows where those are many: as many as the card holds, 2048 lanes on each of 256 compute units.  One
// vector per lane leaves the registers for all of them, which is worth as much as rows that need no barrier, and
// more for few rows; measured side by side, bf16, us, to y / to y8 per row: 16384 x 2048, 256 lanes 45.3 / 46.0, 64
// lanes of 4 vectors 49.2 / 46.5 (64 rows: 2.9 / 3.7, 4.4 / 5.3); 32768 x 1003, 128 lanes 54.5 / 52.0, 64 of 2
// 53.7 / 51.1, half the workgroups 68 / 71, twice 60 / 59; 8192 x 4096, 512 lanes 45.1 / 46.1, 256 of 2 46.8 / 46.8;
// 4096 x 8192, 512 of 2 46.5 / 45.1, 1024 lanes 44.8 / 60.5, 256 of 4 49.6 / 55.6, half the workgroups 51.3 / 49.2.
struct Split {
  int lanes, j, most;
};
Split split(int width) {
  if (width <= 64) return {8, 1, 2048};
  if (width <= 128) return {16, 1, 2048};
  if (width <= 256) return {32, 1, 2048};
  if (width <= 512) return {64, 1, 2048};
  if (width <= 1024) return {128, 1, 4096};
  if (width <= 2048) return {256, 1, 2048};
  if (width <= 4096) return {512, 1, 1024};
  if (width <= 8192) return {512, 2, 2048};
  if (width <= 16384) return {1024, 2, 512};
  if (width <= 32768) return {1024, 4, 512};
  return {0, 0, 0};
}
// Backward, with its sums for dweight in registers and a part of it per workgroup to add up, 16 wavefronts
// on a compute unit.  With dsum and dweight, us, side by side: 16384 x 2048, 256 lanes 56.9, 128 of 2 vectors 57.3
// (64 rows: 5.7 and 7.0); 8192 x 4096, 512 lanes 56.9, 256 of 2 60.9; but 32768 x 1003, 128 lanes 74.4, 64 of 2,
// which need no barrier, 66.3.
Split split_bwd(int width) {
  if (width <= 64) return {8, 1, 512};
  if (width <= 128) return {16, 1, 512};
  if (width <= 256) return {32, 1, 512};
  if (width <= 512) return {64, 1, 512};
  if (width <= 1024) return {64, 2, 512};
  if (width <= 2048) return {256, 1, 512};
  if (width <= 4096) return {512, 1, 512};
  if (width <= 8192) return {512, 2, 512};
  if (width <= 16384) return {1024, 2, 256};
  return {0, 0, 256};
}

// Workgroups: one step over the rows where that is no more than `most`, else `most` that walk.
long workgroups(long rows, Split s, int threads) {
  const long per = s.lanes == 0 ? 1 : threads / s.lanes;
  const long n = (rows + per - 1) / per;
  return n < s.most ? n : s.most;
}

template <typename E, int QUANT>
hipError_t launch_rows(const RmsnormParams& p, hipStream_t st) {
  const Split s = split(p.width);
  if (s.lanes == 0) {
    hipLaunchKernelGGL((rmsnorm_wide_kernel<E, QUANT>), dim3((unsigned)p.rows), dim3(1024), 0, st, p);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)workgroups(p.rows, s, threads(s.lanes)));
  switch (s.lanes * 16 + s.j) {
#define DELTA_ROWS_CASE(L, J)                                                                               \
  case L * 16 + J:                                                                                          \
    hipLaunchKernelGGL((rmsnorm_kernel<E, L, J, QUANT>), grid, dim3(threads(L)), 0, st, p);                 \
    break;
#define DELTA_ROWS_CASES(M) M(8, 1) M(16, 1) M(32, 1) M(64, 1) M(256, 1) M(512, 1) M(512, 2) M(1024, 2)
    DELTA_ROWS_CASES(DELTA_ROWS_CASE)
    DELTA_ROWS_CASE(128, 1) DELTA_ROWS_CASE(1024, 4)
#undef DELTA_ROWS_CASE
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <typename E>
hipError_t launch_rows_bwd(const RmsnormParams& p, hipStream_t st) {
  const Split s = split_bwd(p.width);
  const dim3 grid((unsigned)rmsnorm_bwd_parts(p.rows, p.width));
  switch (s.lanes * 16 + s.j) {
#define DELTA_ROWS_CASE(L, J)                                                                        \
  case L * 16 + J:                                                                                   \
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<E, L, J>), grid, dim3(bwd_threads(L)), 0, st, p);             \
    break;
    DELTA_ROWS_CASES(DELTA_ROWS_CASE)
    DELTA_ROWS_CASE(64, 2)
#undef DELTA_ROWS_CASE
#undef DELTA_ROWS_CASES
    case 0: hipLaunchKernelGGL((rmsnorm_bwd_wide_kernel<E>), grid, dim3(1024), 0, st, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <typename E>
hipError_t launch_quant(const RmsnormParams& p, hipStream_t st) {
  if (!p.y8) return launch_rows<E, 0>(p, st);
  return p.group == 128 ? launch_rows<E, 2>(p, st) : launch_rows<E, 1>(p, st);
}

}  // namespace

hipError_t launch_rmsnorm(const RmsnormParams& p, bool bf16_in, hipStream_t st) {
  return bf16_in ? launch_quant<bf16>(p, st) : launch_quant<float>(p, st);
}

// As many as the card holds: 2 workgroups of 512 threads on each of 256 compute units, or 1 of 1024.  Side by
// side, us, 16384 x 2048: 256 threads 56.5, 512 56.9, 1024 64.4, twice the workgroups 59; 32768 x 1003: 102, 66.3
// and 71.9.
int rmsnorm_bwd_parts(long rows, int width) {
  const Split s = split_bwd(width);
  return (int)workgroups(rows, s, bwd_threads(s.lanes));
}

hipError_t launch_rmsnorm_bwd(const RmsnormParams& p, bool bf16_in, hipStream_t st) {
  const int parts = rmsnorm_bwd_parts(p.rows, p.width);
  if (parts > 0)
    if (const hipError_t e = bf16_in ? launch_rows_bwd<bf16>(p, st) : launch_rows_bwd<float>(p, st)) return e;
  if (!p.dweight) return hipSuccess;
  hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((p.width + 15) / 16), dim3(DW_THREADS), 0, st, p.part, parts, p.width,
                     p.dweight);
  return hipGetLastError();
}

}  // namespace delta
