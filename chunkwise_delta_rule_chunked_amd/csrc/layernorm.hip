// Layer norm of the residual stream with the dropout of its branch and the residual's addition, its backward
// pass, and dropout alone (include/delta_layernorm.h).  Sums in float32.
//
// Bound by bytes, as the RMS norm next to it, whose accesses and split of a row over lanes it shares: a row
// stays in registers between its statistics and its use, and the mask of the dropout is formed again
// wherever it is needed and never stored.  Measured at 16384 x 2048 bf16 with p = 0.1: forward 46 us (5.8 TB/s; a copy
// 5.92), backward 75 (4.9 TB/s in its main launch of 69, whose vector instructions fill 62 % of the SIMDs' cycles; 62 us
// without a mask), dropout and residual 35 (5.7 TB/s).
#include <hip/hip_runtime.h>

#include "common.h"
#include "layernorm.h"
#include "rows.h"

namespace delta {
namespace {

using namespace rows;

// Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw: Parallel Random Numbers: As Easy as 1, 2, 3, SC 2011):
// 128 bits from a counter of 128 and a key of 64.  One counter serves eight channels of a row, 16 bits each: with 32
// bits the products of the rounds, not memory, would bound the kernels.
struct Bits {
  uint32_t w[4];
  __device__ inline bool keep(int e, uint32_t drop) const { return (w[e / 2] >> (16 * (e % 2)) & 0xffffu) >= drop; }
};
__device__ inline Bits random_bits(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b, c3 = (uint32_t)a;
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
  return Bits{{c0, c1, c2, c3}};
}

// v, a row's vector number `vec`, with its dropped channels 0 and the others scaled.
struct Dropper {
  uint32_t drop;
  float scale;
  uint64_t seed, offset, per_row;
  __device__ inline Dropper(const DropRule& r, int width)
      : drop(r.drop), scale(r.scale), seed(r.seed), offset(r.offset + (r.step ? *r.step : 0)), per_row((width + V - 1) / V) {}
  // the kept channels of a vector, a bit each, and what becomes of one
  __device__ inline unsigned mask(long row, int vec) const {
    const Bits b = random_bits(row * per_row + vec, offset, seed);
    unsigned m = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) m |= b.keep(e, drop) ? 1u << e : 0u;
    return m;
  }
  __device__ inline float apply(unsigned mask, int e, float v) const { return mask >> e & 1 ? v * scale : 0.f; }
  __device__ inline void operator()(long row, int vec, float* v) const {
    const Bits b = random_bits(row * per_row + vec, offset, seed);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = b.keep(e, drop) ? v[e] * scale : 0.f;
  }
};

// N sums over the LANES lanes of a row; `slot`: which row of the workgroup's.  All slots of a workgroup take every
// step together; `lds` has a place per sum and wavefront and is another one for each of a row's steps, so that one
// barrier does: a place is written again behind the barrier of the step that came after its reads.  The barriers wait
// for LDS alone, not for the loads and stores of rows.
template <int LANES, int N, int W>
__device__ inline void row_totals(float (&x)[N], int slot, float (*lds)[W]) {
#pragma unroll
  for (int o = (LANES < WAVE ? LANES : WAVE) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += __shfl_xor(x[i], o, WAVE);
  if constexpr (LANES > WAVE) {
    if (threadIdx.x % WAVE == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) lds[i][threadIdx.x / WAVE] = x[i];
    barrier_lds();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = 0.f;
#pragma unroll
      for (int k = 0; k < LANES / WAVE; ++k) x[i] += lds[i][slot * (LANES / WAVE) + k];
    }
  }
}

// A row's mean and 1 / sqrt(variance + eps) from a first mean and the sums of the deviations from it and of
// their squares: what rounding left of the first mean comes out again, so a row far from 0 loses nothing.
struct Stats {
  float shift, rstd;  // mean = first mean + shift
  __device__ inline Stats(float sum, float squares, float width, float eps) {
    shift = sum / width;
    rstd = 1.f / sqrtf(fmaxf(squares / width - shift * shift, 0.f) + eps);
    if (squares != squares) rstd = squares;  // fmaxf drops a NaN
  }
};

template <typename E, int LANES, int J, bool DROP>
__global__ __launch_bounds__(threads(LANES)) void layernorm_kernel(LayernormParams p) {
  constexpr int T = threads(LANES), RPW = T / LANES;
  constexpr bool KEEP = J == 1;  // weight and bias stay in registers
  __shared__ float lds[3][T / WAVE];
  const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
  const Dropper dropper(p.rule, p.width);
  float w[KEEP ? J : 1][V], b[KEEP ? J : 1][V] = {};
  if constexpr (KEEP) {
    load8<false>(p.weight + lane * V, p.width - lane * V, w[0]);
    if (p.bias) load8<false>(p.bias + lane * V, p.width - lane * V, b[0]);
  }
  // every lane of a workgroup takes the same number of steps (barriers inside)
  for (long row0 = (long)blockIdx.x * RPW; row0 < p.rows; row0 += (long)gridDim.x * RPW) {
    const long row = row0 + slot, base = row * p.width;
    const bool ok = row < p.rows;
    float s[J][V], total[1] = {0.f};
    Raw8<E> x[J], r[J];
    unsigned keep[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = (lane + j * LANES) * V, n = ok ? p.width - i : 0;
      x[j].load(static_cast<const E*>(p.x) + base + i, n);
      r[j].load(static_cast<const E*>(p.res) + base + i, p.res ? n : 0);
    }
    if constexpr (DROP) {
#pragma unroll
      for (int j = 0; j < J; ++j) keep[j] = dropper.mask(row, lane + j * LANES);  // while the loads are under way
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[j][e] = x[j][e];
        if constexpr (DROP) s[j][e] = dropper.apply(keep[j], e, s[j][e]);
        if (p.sum) s[j][e] = to_float(to_elem<E>(s[j][e] + r[j][e]));
      }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = (lane + j * LANES) * V, n = ok ? p.width - i : 0;
      if (p.sum) store8(static_cast<E*>(p.sum) + base + i, n, s[j]);
#pragma unroll
      for (int e = 0; e < V; ++e) total[0] += s[j][e];  // 0 past the row
    }
    row_totals<LANES>(total, slot, lds);
    const float mean = total[0] / p.width;
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int n = p.width - (lane + j * LANES) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[j][e] = e < n ? s[j][e] - mean : 0.f;
        sums[0] += s[j][e];
        sums[1] += s[j][e] * s[j][e];
      }
    }
    row_totals<LANES>(sums, slot, lds + 1);
    const Stats t(sums[0], sums[1], p.width, p.eps);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = (lane + j * LANES) * V;
      if constexpr (!KEEP) {
        load8<false>(p.weight + i, p.width - i, w[0]);
        if (p.bias) load8<false>(p.bias + i, p.width - i, b[0]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) s[j][e] = (s[j][e] - t.shift) * t.rstd * w[0][e] + b[0][e];
      store8(static_cast<E*>(p.y) + base + i, ok ? p.width - i : 0, s[j]);
    }
  }
}

// Rows of any width, read again for each use.
template <typename E, bool DROP>
__global__ __launch_bounds__(1024) void layernorm_wide_kernel(LayernormParams p) {
  constexpr int T = 1024;
  __shared__ float lds[3][T / WAVE];
  const Dropper dropper(p.rule, p.width);
  for (long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const long base = row * p.width;
    float total[1] = {0.f};
    for (int i = threadIdx.x * V; i < p.width; i += T * V) {
      float s[V], r[V] = {};
      load8<false>(static_cast<const E*>(p.x) + base + i, p.width - i, s);
      if (p.res) load8<false>(static_cast<const E*>(p.res) + base + i, p.width - i, r);
      if constexpr (DROP) dropper(row, i / V, s);
      if (p.sum) {
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] = to_float(to_elem<E>(s[e] + r[e]));
        store8(static_cast<E*>(p.sum) + base + i, p.width - i, s);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) total[0] += i + e < p.width ? s[e] : 0.f;
    }
    row_totals<T>(total, 0, lds);
    const float mean = total[0] / p.width;
    const E* s0 = static_cast<const E*>(p.sum ? p.sum : p.x) + base;  // what this thread itself wrote
    float sums[2] = {0.f, 0.f};
    for (int i = threadIdx.x * V; i < p.width; i += T * V) {
      float s[V];
      load8<false>(s0 + i, p.width - i, s);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = i + e < p.width ? s[e] - mean : 0.f;
        sums[0] += d;
        sums[1] += d * d;
      }
    }
    row_totals<T>(sums, 0, lds + 1);
    const Stats t(sums[0], sums[1], p.width, p.eps);
    for (int i = threadIdx.x * V; i < p.width; i += T * V) {
      float s[V], w[V], b[V] = {};
      load8<false>(s0 + i, p.width - i, s);
      load8<false>(p.weight + i, p.width - i, w);
      if (p.bias) load8<false>(p.bias + i, p.width - i, b);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = (s[e] - mean - t.shift) * t.rstd * w[e] + b[e];
      store8(static_cast<E*>(p.y) + base + i, p.width - i, s);
    }
  }
}

constexpr int bwd_threads(int lanes) { return lanes > 512 ? lanes : 512; }

// Workgroup k takes rows k RPW .., then gridDim.x * RPW further on, and stores its parts of dweight and dbias
// in part[k] and part[gridDim.x + k].  Every part is the sum over a fixed set of rows in a fixed order.
// WHOLE (rows of whole vectors, 16-byte aligned): the next step's rows are loaded ahead.
// With z = (s - mean) rstd: ds = dsum + rstd (w dy - mean(w dy) - z mean(w dy z)), dweight = sum dy z,
// dbias = sum dy.
template <typename E, int LANES, int J, bool DROP, bool WHOLE>
__global__ __launch_bounds__(bwd_threads(LANES), 4) void layernorm_bwd_kernel(LayernormParams p) {
  constexpr int T = bwd_threads(LANES), RPW = T / LANES, COLS = LANES * J * V;
  constexpr bool KEEP = J == 1;
  __shared__ float lds[5][T / WAVE];
  const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
  const Dropper dropper(p.rule, p.width);
  float w[KEEP ? J : 1][V], accw[J][V] = {}, accb[J][V] = {};
  if constexpr (KEEP) load8<false>(p.weight + lane * V, p.width - lane * V, w[0]);
  struct Row {
    Raw8<E> s[J], d[J], o[J];
  };
  // WHOLE: the rows of a step as one range of bytes; what is past it reads 0 and is not stored.  Without branches
  // around them the loads of the next step's rows are under way while this one's sums meet and are waited for by count
  // (16384 x 2048 bf16 69 to 62 us, 8192 x 2048 float32 63 to 53).
  const int off = lane * V < p.width ? (slot * p.width + lane * V) * (int)sizeof(E) : 1 << 30;
  auto window = [&](const void* q, long row0) {
    const long left = p.rows - row0, n = q ? (left < RPW ? (left > 0 ? left : 0) : RPW) : 0;
    return buffer_rsrc(static_cast<E*>(const_cast<void*>(q)) + row0 * p.width, (int)(n * p.width) * (int)sizeof(E));
  };
  auto fetch = [&](Row& r, long row0) {
    if constexpr (WHOLE) {
      r.s[0].load(window(p.x, row0), off);
      r.d[0].load(window(p.dy, row0), off);
      r.o[0].load(window(p.dsum, row0), off);
    } else {
      const long row = row0 + slot, base = row * p.width;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int i = (lane + j * LANES) * V, n = row < p.rows ? p.width - i : 0;
        r.s[j].load(static_cast<const E*>(p.x) + base + i, n);
        r.d[j].load(static_cast<const E*>(p.dy) + base + i, n);
        r.o[j].load(static_cast<const E*>(p.dsum) + base + i, p.dsum ? n : 0);
      }
    }
  };
  const long stride = (long)gridDim.x * RPW;
  Row now, next;
  if constexpr (WHOLE) fetch(next, (long)blockIdx.x * RPW);
  for (long row0 = (long)blockIdx.x * RPW; row0 < p.rows; row0 += stride) {
    const long row = row0 + slot, base = row * p.width;
    const bool ok = row < p.rows;
    if constexpr (WHOLE) {
      now = next;
      fetch(next, row0 + stride);
      __builtin_amdgcn_sched_barrier(0);
    } else {
      fetch(now, row0);
    }
    Raw8<E>(&s)[J] = now.s, (&d)[J] = now.d, (&o)[J] = now.o;
    auto store = [&](void* q, int i, const float* v) {
      if constexpr (WHOLE) buffer_store8(window(q, row0), off, v, E{});
      else store8(static_cast<E*>(q) + base + i, ok ? p.width - i : 0, v);
    };
    unsigned keep[J];
    if constexpr (DROP) {
#pragma unroll
      for (int j = 0; j < J; ++j) keep[j] = dropper.mask(row, lane + j * LANES);  // while the loads are under way
      __builtin_amdgcn_sched_barrier(0);
    }
    float first[2] = {0.f, 0.f};  // of s and of w dy
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if constexpr (!KEEP) load8<false>(p.weight + (lane + j * LANES) * V, p.width - (lane + j * LANES) * V, w[0]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        first[0] += s[j][e];
        first[1] += w[0][e] * d[j][e];
      }
      if constexpr (J > 1) s[j].again(), d[j].again();
    }
    row_totals<LANES>(first, slot, lds);
    const float mean = first[0] / p.width;
    float sums[3] = {0.f, 0.f, 0.f};  // of the deviations, their squares, and their products with w dy
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int n = p.width - (lane + j * LANES) * V;
      if constexpr (!KEEP) load8<false>(p.weight + (lane + j * LANES) * V, n, w[0]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float c = e < n ? s[j][e] - mean : 0.f;
        sums[0] += c;
        sums[1] += c * c;
        sums[2] += w[0][e] * d[j][e] * c;
      }
      if constexpr (J > 1) s[j].again(), d[j].again();
    }
    row_totals<LANES>(sums, slot, lds + 2);
    const Stats t(sums[0], sums[1], p.width, p.eps);
    const float c1 = first[1] / p.width, c2 = t.rstd * ((sums[2] - t.shift * first[1]) / p.width);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = (lane + j * LANES) * V;
      if constexpr (!KEEP) load8<false>(p.weight + i, p.width - i, w[0]);
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float z = (s[j][e] - mean - t.shift) * t.rstd;
        v[e] = o[j][e] + t.rstd * (w[0][e] * d[j][e] - c1 - z * c2);
        if (ok) {  // a missing row's rstd is infinite for eps = 0
          accw[j][e] += d[j][e] * z;
          accb[j][e] += d[j][e];
        }
      }
      store(p.dres, i, v);
      if constexpr (DROP) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = dropper.apply(keep[j], e, v[e]);
        store(p.dx, i, v);
      }
    }
  }
  // the RPW row slots add up in turn
  __shared__ float both[RPW == 1 ? 1 : COLS];
  auto give = [&](const float (&acc)[J][V], float* part) {
    if constexpr (RPW == 1) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int i = (lane + j * LANES) * V;
        store8(part + i, p.width - i, acc[j]);
      }
    } else {
      for (int k = 0; k < RPW; ++k) {
        __syncthreads();
        if (slot == k) {
#pragma unroll
          for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              float* q = both + (lane + j * LANES) * V + e;
              *q = k ? *q + acc[j][e] : acc[j][e];
            }
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < p.width; i += T) part[i] = both[i];
    }
  };
  if (p.dweight) give(accw, p.part + (long)blockIdx.x * p.width);
  if (p.dbias) give(accb, p.part + ((long)gridDim.x + blockIdx.x) * p.width);
}

template <typename E, bool DROP>
__global__ __launch_bounds__(1024) void layernorm_bwd_wide_kernel(LayernormParams p) {
  constexpr int T = 1024;
  __shared__ float lds[5][T / WAVE];
  const Dropper dropper(p.rule, p.width);
  float *partw = p.part + (long)blockIdx.x * p.width, *partb = p.part + ((long)gridDim.x + blockIdx.x) * p.width;
  bool begin = true;
  for (long row = blockIdx.x; row < p.rows; row += gridDim.x, begin = false) {
    const long base = row * p.width;
    const E *x = static_cast<const E*>(p.x) + base, *dy = static_cast<const E*>(p.dy) + base;
    float first[2] = {0.f, 0.f}, sums[3] = {0.f, 0.f, 0.f};
    for (int i = threadIdx.x * V; i < p.width; i += T * V) {
      float s[V], d[V], w[V];
      load8<false>(x + i, p.width - i, s);
      load8<false>(dy + i, p.width - i, d);
      load8<false>(p.weight + i, p.width - i, w);
#pragma unroll
      for (int e = 0; e < V; ++e) first[0] += s[e], first[1] += w[e] * d[e];
    }
    row_totals<T>(first, 0, lds);
    const float mean = first[0] / p.width;
    for (int i = threadIdx.x * V; i < p.width; i += T * V) {
      float s[V], d[V], w[V];
      load8<false>(x + i, p.width - i, s);
      load8<false>(dy + i, p.width - i, d);
      load8<false>(p.weight + i, p.width - i, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float c = i + e < p.width ? s[e] - mean : 0.f;
        sums[0] += c;
        sums[1] += c * c;
        sums[2] += w[e] * d[e] * c;
      }
    }
    row_totals<T>(sums, 0, lds + 2);
    const Stats t(sums[0], sums[1], p.width, p.eps);
    const float c1 = first[1] / p.width, c2 = t.rstd * ((sums[2] - t.shift * first[1]) / p.width);
    for (int i = threadIdx.x * V; i < p.width; i += T * V) {
      const int n = p.width - i;
      float s[V], d[V], w[V], o[V] = {}, aw[V] = {}, ab[V] = {};
      load8<false>(x + i, n, s);
      load8<false>(dy + i, n, d);
      load8<false>(p.weight + i, n, w);
      if (p.dsum) load8<false>(static_cast<const E*>(p.dsum) + base + i, n, o);
      if (!begin && p.dweight) load8<false>(partw + i, n, aw);
      if (!begin && p.dbias) load8<false>(partb + i, n, ab);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float z = (s[e] - mean - t.shift) * t.rstd;
        o[e] += t.rstd * (w[e] * d[e] - c1 - z * c2);
        aw[e] += d[e] * z;
        ab[e] += d[e];
      }
      store8(static_cast<E*>(p.dres) + base + i, n, o);
      if constexpr (DROP) {
        dropper(row, i / V, o);
        store8(static_cast<E*>(p.dx) + base + i, n, o);
      }
      if (p.dweight) store8(partw + i, n, aw);
      if (p.dbias) store8(partb + i, n, ab);
    }
  }
}

// dweight and dbias: the sums of their parts, 16 columns and 64 lanes over the parts per workgroup.
constexpr int DW_THREADS = 1024;
__global__ __launch_bounds__(DW_THREADS) void layernorm_dweight_kernel(const float* part, int parts, int width, float* dweight,
                                                                       float* dbias) {
  __shared__ float sums[DW_THREADS / WAVE][17];
  const int col = threadIdx.x % 16, i = blockIdx.x * 16 + col;
  float* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  part += (long)blockIdx.y * parts * width;
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
    out[i] = s;
  }
}

// Dropout alone: AHEAD vectors a lane.  RAGGED: rows that are no whole number of vectors.
constexpr int DROP_TH = 256, AHEAD = 4;
template <typename E, bool RAGGED>
__global__ __launch_bounds__(DROP_TH) void dropout_kernel(DropoutParams p) {
  const Dropper dropper(p.rule, p.width);
  const long per_row = (p.width + V - 1) / V, all = p.rows * per_row;
  const long at = (long)blockIdx.x * (DROP_TH * AHEAD) + threadIdx.x;
  float x[AHEAD][V], r[AHEAD][V] = {};
  long row[AHEAD];
  int vec[AHEAD], n[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const long v = at + k * DROP_TH;
    // without a ragged end the tensor is one long row to everything but the random bits, which count in vectors
    row[k] = RAGGED ? (all >> 32 ? v / per_row : (long)((uint32_t)v / (uint32_t)per_row)) : 0;
    vec[k] = RAGGED ? (int)(v - row[k] * per_row) : 0;
    n[k] = v >= all ? 0 : RAGGED ? min(p.width - vec[k] * V, V) : V;
    const long i = RAGGED ? row[k] * p.width + (long)vec[k] * V : v * V;
    load8<true>(static_cast<const E*>(p.x) + i, n[k], x[k]);
    if (p.res) load8<true>(static_cast<const E*>(p.res) + i, n[k], r[k]);
  }
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const long v = at + k * DROP_TH;
    if (p.rule.drop) {
      const Bits b = random_bits(v, dropper.offset, dropper.seed);
#pragma unroll
      for (int e = 0; e < V; ++e) x[k][e] = b.keep(e, dropper.drop) ? x[k][e] * dropper.scale : 0.f;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) x[k][e] += r[k][e];
    const long i = RAGGED ? row[k] * p.width + (long)vec[k] * V : v * V;
    store8(static_cast<E*>(p.y) + i, n[k], x[k]);
  }
}

// Lanes and vectors per lane of a row (0: the kernels for any width), and the workgroups that walk over the rows
// where those are many: enough that they do not all read, then all compute, then all write.  Forward with the mask,
// at 2048 / 6144 of them: 16384 x 2048 bf16 55.0 / 46.4 us, 32768 x 1003 69.5 / 59.3 us; without it 48.4 / 46.5 and
// 54.1 / 56.6.  Rows of 4096, at 1024 / 1536: 55.4 / 47.1 us.  Of two vectors a lane more do not help (52.0 / 54.4).
struct RowSplit {
  int lanes, j, most;
};
RowSplit split(int width) {
  if (width <= 64) return {8, 1, 6144};
  if (width <= 128) return {16, 1, 6144};
  if (width <= 256) return {32, 1, 6144};
  if (width <= 512) return {64, 1, 6144};
  if (width <= 1024) return {128, 1, 12288};
  if (width <= 2048) return {256, 1, 6144};
  if (width <= 4096) return {512, 1, 1536};
  if (width <= 8192) return {512, 2, 1024};
  if (width <= 16384) return {1024, 2, 512};
  return {0, 0, 4096};
}
// The backward pass keeps its parts of dweight and dbias for a workgroup's whole walk, so it has as many as the card
// runs at once (16384 x 2048 bf16: 512 62 us, 384 71, 768 68).  One vector a lane as far as a workgroup reaches: two
// leave no registers for the next row (4096 x 8192 bf16 in 1024 lanes 71 us, in 512 88; 3711 x 1003 float32 in 128
// lanes 24 us, in 64 33).
RowSplit split_bwd(int width) {
  if (width <= 64) return {8, 1, 512};
  if (width <= 128) return {16, 1, 512};
  if (width <= 256) return {32, 1, 512};
  if (width <= 512) return {64, 1, 512};
  if (width <= 1024) return {128, 1, 512};
  if (width <= 2048) return {256, 1, 512};
  if (width <= 4096) return {512, 1, 512};
  if (width <= 8192) return {1024, 1, 256};
  if (width <= 16384) return {1024, 2, 256};
  return {0, 0, 256};
}

// Workgroups: one step over the rows where that is no more than `most`, else `most` that walk.
long workgroups(long rows, RowSplit s, int threads) {
  const long per = s.lanes == 0 ? 1 : threads / s.lanes;
  const long n = (rows + per - 1) / per;
  return n < s.most ? n : s.most;
}

template <typename E, bool DROP>
hipError_t launch_rows(const LayernormParams& p, hipStream_t st) {
  const RowSplit s = split(p.width);
  if (s.lanes == 0) {
    hipLaunchKernelGGL((layernorm_wide_kernel<E, DROP>), dim3((unsigned)(p.rows < s.most ? p.rows : s.most)), dim3(1024), 0, st, p);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)workgroups(p.rows, s, threads(s.lanes)));
  switch (s.lanes * 16 + s.j) {
#define DELTA_ROWS_CASE(L, J)                                                                       \
  case L * 16 + J:                                                                                  \
    hipLaunchKernelGGL((layernorm_kernel<E, L, J, DROP>), grid, dim3(threads(L)), 0, st, p);        \
    break;
#define DELTA_ROWS_ONES(M) M(8, 1) M(16, 1) M(32, 1) M(64, 1) M(128, 1) M(256, 1) M(512, 1)
    DELTA_ROWS_ONES(DELTA_ROWS_CASE)
    DELTA_ROWS_CASE(512, 2)
    DELTA_ROWS_CASE(1024, 2)
#undef DELTA_ROWS_CASE
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <typename E, bool DROP>
hipError_t launch_rows_bwd(const LayernormParams& p, hipStream_t st) {
  const RowSplit s = split_bwd(p.width);
  const dim3 grid((unsigned)layernorm_bwd_parts(p.rows, p.width));
  const uintptr_t at = (uintptr_t)p.x | (uintptr_t)p.dy | (uintptr_t)p.dsum | (uintptr_t)p.dres | (uintptr_t)p.dx;
  // within a wavefront there is no barrier to wait at, and the next row's registers cost more than they give
  // (65536 x 512 bf16: 51 us as it is, 55 with them)
  const bool whole = p.width % V == 0 && at % 16 == 0 && s.lanes > WAVE && s.j == 1;
  switch ((s.lanes * 16 + s.j) * 2 + whole) {
#define DELTA_ROWS_CASE(L, J, W)                                                                          \
  case (L * 16 + J) * 2 + W:                                                                              \
    hipLaunchKernelGGL((layernorm_bwd_kernel<E, L, J, DROP, W>), grid, dim3(bwd_threads(L)), 0, st, p);   \
    break;
#define DELTA_ROWS_ONE(L, J) DELTA_ROWS_CASE(L, J, false)
    DELTA_ROWS_ONES(DELTA_ROWS_ONE)
    DELTA_ROWS_CASE(128, 1, true)
    DELTA_ROWS_CASE(256, 1, true)
    DELTA_ROWS_CASE(512, 1, true)
    DELTA_ROWS_CASE(1024, 1, true)
    DELTA_ROWS_CASE(1024, 1, false)
    DELTA_ROWS_CASE(1024, 2, false)
#undef DELTA_ROWS_ONE
#undef DELTA_ROWS_CASE
#undef DELTA_ROWS_ONES
    case 0: hipLaunchKernelGGL((layernorm_bwd_wide_kernel<E, DROP>), grid, dim3(1024), 0, st, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <typename E>
hipError_t dropout(const DropoutParams& p, hipStream_t st) {
  const long per_row = (p.width + V - 1) / V, all = p.rows * per_row;
  const dim3 grid((unsigned)((all + DROP_TH * AHEAD - 1) / (DROP_TH * AHEAD)));
  if (p.width % V) hipLaunchKernelGGL((dropout_kernel<E, true>), grid, dim3(DROP_TH), 0, st, p);
  else hipLaunchKernelGGL((dropout_kernel<E, false>), grid, dim3(DROP_TH), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layernorm(const LayernormParams& p, bool bf16_in, hipStream_t st) {
  if (p.rule.drop) return bf16_in ? launch_rows<bf16, true>(p, st) : launch_rows<float, true>(p, st);
  return bf16_in ? launch_rows<bf16, false>(p, st) : launch_rows<float, false>(p, st);
}

int layernorm_bwd_parts(long rows, int width) {
  const RowSplit s = split_bwd(width);
  return (int)workgroups(rows, s, bwd_threads(s.lanes));
}

hipError_t launch_layernorm_bwd(const LayernormParams& p, bool bf16_in, hipStream_t st) {
  const int parts = layernorm_bwd_parts(p.rows, p.width);
  if (parts > 0) {
    const hipError_t e = p.rule.drop ? (bf16_in ? launch_rows_bwd<bf16, true>(p, st) : launch_rows_bwd<float, true>(p, st))
                                     : (bf16_in ? launch_rows_bwd<bf16, false>(p, st) : launch_rows_bwd<float, false>(p, st));
    if (e != hipSuccess) return e;
  }
  if (!p.dweight && !p.dbias) return hipSuccess;
  hipLaunchKernelGGL(layernorm_dweight_kernel, dim3((p.width + 15) / 16, 2), dim3(DW_THREADS), 0, st, p.part, parts, p.width,
                     p.dweight, p.dbias);
  return hipGetLastError();
}

hipError_t launch_dropout(const DropoutParams& p, bool bf16_in, hipStream_t st) {
  return bf16_in ? dropout<bf16>(p, st) : dropout<float>(p, st);
}

}  // namespace delta
