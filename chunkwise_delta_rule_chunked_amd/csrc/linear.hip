// Linear attention with a decay for each head: the launches around the chain kernel (linear_chain.h), and
// the step for one token.
#include <hip/hip_runtime.h>
#include <math.h>

#include "common.h"
#include "linear.h"

namespace delta {
namespace {

__device__ inline double wave_total(double x) {
#pragma unroll
  for (int o = WAVE / 2; o > 0; o >>= 1) x += __shfl_xor(x, o, WAVE);
  return x;
}

// s e^d for a segment's sum of log gates.  With gates above 1 e^d may be no float32 number although s e^d is (s is small, or
// 0): then in three steps, each between s and the result.  Past e^240 every s is 0, infinite or 0 again.
__device__ inline floatx4 decayed(floatx4 s, double d) {
  if (!(fabs(d) > 80.0) || d == -INFINITY) return s * expf((float)d);
  const float third = expf((float)(fmin(fmax(d, -240.0), 240.0) / 3));
  return s * third * third * third;
}

// One chain's states of one place, four elements a lane, from segment to segment: a segment's result becomes its start,
// start_{p+1} = e^decay_p start_p + result_p.  BOUNDS: and the parts of the inner products with the other chain's starts
// (segment p of the reverse chain starts behind segment P - 1 - p of the other).
struct Walk {
  const floatx4* start;
  floatx4 *segs, *end;
  const double* decay;
};
template <bool BOUNDS>
__device__ inline void walk(const Walk& w, int P, long quads, long bh, long q, const floatx4* other, const floatx4* other0,
                            double* bounds) {
  auto dot = [](const floatx4& a, const floatx4& b) {
    double x = 0.0;
#pragma unroll
    for (int k = 0; k < 4; ++k) x += (double)a[k] * b[k];
    return x;
  };
  auto bound = [&](int place, double x) {
    x = wave_total(x);
    if (threadIdx.x % WAVE == 0) bounds[((bh * P + place) * quads + q) / WAVE] = x;
  };
  floatx4 s = w.start ? w.start[bh * quads + q] : floatx4{};
  floatx4* at = w.segs + bh * P * quads + q;
  const floatx4* ot = other + bh * P * quads + q;
  const int n = w.end ? P : P - 1;  // without an end the last segment has no result
  constexpr int AHEAD = 8;          // results loaded at a time
  for (int p0 = 0; p0 < n; p0 += AHEAD) {
    floatx4 r[AHEAD], o[BOUNDS ? AHEAD : 1];
    double x[AHEAD] = {};
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (p0 + k < n) {
        r[k] = at[(p0 + k) * quads];
        if constexpr (BOUNDS)
          if (p0 + k > 0) o[k] = ot[(P - p0 - k) * quads];
      }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (p0 + k < n) {
        at[(p0 + k) * quads] = s;
        if constexpr (BOUNDS)
          if (p0 + k > 0) x[k] = dot(s, o[k]);
        s = decayed(s, w.decay[bh * P + p0 + k]) + r[k];
      }
    if constexpr (BOUNDS) {
#pragma unroll
      for (int o2 = WAVE / 2; o2 > 0; o2 >>= 1)
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) x[k] += __shfl_xor(x[k], o2, WAVE);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (p0 + k > 0 && p0 + k < n && threadIdx.x % WAVE == 0) bounds[((bh * P + P - p0 - k) * quads + q) / WAVE] = x[k];
    }
  }
  if (w.end) {
    w.end[bh * quads + q] = s;
    if constexpr (BOUNDS) bound(0, other0 ? dot(s, other0[bh * quads + q]) : 0.0);
  } else if (P > 0) {
    at[(P - 1) * quads] = s;
    if constexpr (BOUNDS) {
      bound(1, dot(s, ot[quads]));
      bound(0, 0.0);
    }
  }
}

template <bool FORWARD, bool REVERSE, bool BOUNDS>
__global__ __launch_bounds__(256) void combine_kernel(int P, long quads, long all, Walk forward, Walk reverse, double* bounds) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x, bh = i / quads, q = i % quads;
  if (i >= all) return;  // whole wavefronts: a state is a multiple of 256 elements
  if constexpr (FORWARD) walk<false>(forward, P, quads, bh, q, nullptr, nullptr, nullptr);
  // the forward chain's starts are this lane's own
  if constexpr (REVERSE) walk<BOUNDS>(reverse, P, quads, bh, q, forward.segs, forward.start, bounds);
}

// d log g of the tokens of one segment.  With b the inner product of the state before a chunk and its
// gradient, and X = e^gc_C <G, S> what the chunk's two ends share,
//     b = X + sum e,   b' = X + sum f,   d log g_t = X + sum_{r < t} f_r + sum_{r >= t} e_r
// (e with the pairs' row and column sums, which cancel over a chunk).  b is formed from the states at the
// segment's start and carried on from chunk to chunk; a chunk that lets nothing through has X = 0.
constexpr int GATE_TH = 1024, GATE_WAVES = GATE_TH / WAVE, GATE_CHUNKS = 64;
__global__ __launch_bounds__(GATE_TH) void gates_kernel(LinGates p) {
  __shared__ double sums[GATE_WAVES], se[GATE_CHUNKS], sf[GATE_CHUNKS];
  __shared__ bool shut[GATE_CHUNKS];
  const int tid = threadIdx.x, lane = tid % WAVE, wave = tid / WAVE;
  const int seg = blockIdx.x % p.P;
  const long bh = blockIdx.x / p.P;
  const int h = (int)(bh % p.H);
  const long b = bh / p.H;
  double before = 0.0, all = 0.0;
  if (p.P > 1) {
    const int parts = lin_parts(p.dk, p.dv);
    for (int k = lane; k < parts; k += WAVE) before += p.bounds[(bh * p.P + seg) * parts + k];
    before = wave_total(before);
  } else if (p.S0) {
    const int size = p.dk * p.dv;
    for (int i = 4 * tid; i < size; i += 4 * GATE_TH) {
      const floatx4 s = *reinterpret_cast<const floatx4*>(p.S0 + bh * size + i), d = *reinterpret_cast<const floatx4*>(p.dS0 + bh * size + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) before += (double)s[k] * d[k];
    }
    before = wave_total(before);
    if (lane == 0) sums[wave] = before;
    __syncthreads();
    before = 0.0;
    for (int k = 0; k < GATE_WAVES; ++k) before += sums[k];
    __syncthreads();
  }
  const int first = seg * p.NS, count = min(p.NS, p.NT - first);
  auto token = [&](int n) { return n * p.C + lane; };
  auto gate = [&](int n) {
    if (lane >= p.C || token(n) >= p.L) return 0.f;
    return p.gate == LIN_GATE_TOKEN ? p.g[(b * p.L + token(n)) * p.H + h] : p.g[h];
  };
  for (int c0 = 0; c0 < count; c0 += GATE_CHUNKS) {
    const int nc = min(GATE_CHUNKS, count - c0);
    for (int c = wave; c < nc; c += GATE_WAVES) {
      const int n = first + c0 + c;
      const size_t i = (bh * p.NT + n) * p.C + lane;
      const float gl = gate(n);
      const double e = wave_total(lane < p.C ? p.e[i] : 0.0), f = wave_total(lane < p.C ? p.f[i] : 0.0);
      const double a = wave_total(lin_log_gate(gl));
      if (lane == 0) se[c] = e, sf[c] = f, shut[c] = expf((float)a) == 0.f;
    }
    __syncthreads();
    if (tid == 0)
      for (int c = 0; c < nc; ++c) {
        const double X = shut[c] ? 0.0 : before - se[c];
        before = X + sf[c];
        se[c] = X;
      }
    __syncthreads();
    for (int c = wave; c < nc; c += GATE_WAVES) {
      const int n = first + c0 + c;
      const size_t i = (bh * p.NT + n) * p.C + lane;
      const double e = lane < p.C ? p.e[i] : 0.0, f = lane < p.C ? p.f[i] : 0.0;
      // Sums from this token on and up to it, as far as the next reset: beyond one there is nothing to add but what
      // rounding leaves of sums that cancel.
      const bool reset = lin_log_gate(gate(n)) == LIN_RESET;
      const unsigned long long resets = __ballot(reset);
      double up = e, down = f;
#pragma unroll
      for (int o = 1; o < WAVE; o <<= 1) {
        const double u = __shfl_down(up, o, WAVE), d = __shfl_up(down, o, WAVE);
        const unsigned long long span = (1ull << o) - 1;  // o tokens
        if (lane + o < WAVE && !(resets >> (lane + 1) & span)) up += u;
        if (lane >= o && !(resets >> (lane - o + 1) & span)) down += d;
      }
      double past = __shfl_up(down, 1, WAVE);
      if (lane == 0) past = 0.0;
      const double dg = reset ? 0.0 : se[c] + up + past;  // nothing flows past a reset
      if (lane < p.C && token(n) < p.L) {
        if (p.gate == LIN_GATE_TOKEN) p.dg[(b * p.L + token(n)) * p.H + h] = (float)dg;
        else all += dg;
      }
    }
    __syncthreads();
  }
  if (p.gate == LIN_GATE_HEAD) {
    all = wave_total(all);
    __syncthreads();
    if (lane == 0) sums[wave] = all;
    __syncthreads();
    if (tid == 0) {
      double s = 0.0;
      for (int k = 0; k < GATE_WAVES; ++k) s += sums[k];
      p.part[bh * p.P + seg] = s;
    }
  }
}

// A fixed gate's gradient: the parts of all sequences and segments, one wavefront a head.
__global__ __launch_bounds__(WAVE) void gate_heads_kernel(int B, int H, int P, const double* part, float* dg) {
  const int h = blockIdx.x;
  double s = 0.0;
  for (long i = threadIdx.x; i < (long)B * P; i += WAVE) s += part[(i / P * H + h) * P + i % P];
  s = wave_total(s);
  if (threadIdx.x == 0) dg[h] = (float)s;
}

// The gradient of rows that `share` consecutive heads read: their float32 parts added up in order, rounded once.
template <typename E>
__global__ __launch_bounds__(256) void share_kernel(const float* dq_part, const float* dk_part, E* dq, E* dk, long quads, int share,
                                                    int width) {
  for (long t = (long)blockIdx.x * 256 + threadIdx.x; t < 2 * quads; t += (long)gridDim.x * 256) {
    const bool second = t >= quads;
    const long i = (second ? t - quads : t) * 4, row = i / width;
    const float* from = (second ? dk_part : dq_part) + row * share * width + i % width;
    floatx4 s = *reinterpret_cast<const floatx4*>(from);
    for (int k = 1; k < share; ++k) s += *reinterpret_cast<const floatx4*>(from + (long)k * width);
    store4<E>((second ? dk : dq) + i, s[0], s[1], s[2], s[3]);
  }
}

// One token: S <- a S + k v^T, o = scale S^T q.  Bound by the state, read and written once.  A workgroup has `pack`
// units, a unit being one head's state or a slab of its columns; of a unit, a thread has one of `quads` groups of four
// columns and U consecutive rows, in 16-byte accesses with non-temporal hints.  The sums over the rows of S^T q meet in
// LDS.  Measured at 64 x 16 states of 128 x 128 (a captured graph): 23.5 us, 5.8 TB/s; with 4 rows a thread 25.6, with 16
// 25.2, with 512 threads 24.8, with a loop over the rows of a state 28.6.  Accesses run along a state's rows, in one step:
// slabs of 16 columns where a width is no multiple of 32 took 72 us for 33M elements of 64 x 80 states, 47 like this.
// Small states share a workgroup: 33M elements of 16 x 16 states 49 us, one to a workgroup 64.
constexpr int DECODE_TH = 256, DECODE_WGS = 1024;
template <typename E, int DK, int U>
__global__ __launch_bounds__(DECODE_TH) void decode_kernel(LinDecode p, int quads, int slabs, int pack) {
  constexpr int GROUPS = DK / U;
  __shared__ floatx4 red[DECODE_TH];
  const int per = quads * GROUPS, tid = threadIdx.x, in = tid % per, r0 = in / quads * U;
  const long unit = (long)blockIdx.x * pack + tid / per, bh = unit / slabs;
  const int quad = (int)(unit % slabs) * quads + in % quads;
  const bool on = tid < per * pack && bh < (long)p.B * p.H && quad < p.DV / 4;
  typedef E E4 __attribute__((ext_vector_type(4)));
  floatx4 o = {};
  if (on) {
    const int h = (int)(bh % p.H);
    const long bk = bh / p.H * p.Hk + h / (p.H / p.Hk);
    float* Sg = p.S + (bh * DK + r0) * p.DV + quad * 4;
    floatx4 s[U];
#pragma unroll
    for (int i = 0; i < U; ++i) s[i] = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(Sg + (long)i * p.DV));
    const E *q = static_cast<const E*>(p.q) + bk * DK + r0, *k = static_cast<const E*>(p.k) + bk * DK + r0;
    const E4 v4 = *reinterpret_cast<const E4*>(static_cast<const E*>(p.v) + bh * p.DV + quad * 4);
    const float a = p.gate == LIN_GATE_NONE ? 1.f : expf(p.g[p.gate == LIN_GATE_TOKEN ? bh : h]);
#pragma unroll
    for (int i = 0; i < U; i += 4) {
      const E4 q4 = *reinterpret_cast<const E4*>(q + i), k4 = *reinterpret_cast<const E4*>(k + i);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i + j][e] = a * s[i + j][e] + to_float((E)k4[j]) * to_float((E)v4[e]);
          o[e] += to_float((E)q4[j]) * s[i + j][e];
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) __builtin_nontemporal_store(s[i], reinterpret_cast<floatx4*>(Sg + (long)i * p.DV));
  }
  red[tid] = o;
  barrier_lds();
  if (on && r0 == 0) {
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) o += red[tid + k * quads];
    store4<E>(static_cast<E*>(p.O) + bh * p.DV + quad * 4, p.scale * o[0], p.scale * o[1], p.scale * o[2], p.scale * o[3]);
  }
}

template <typename E, int DK, int U>
hipError_t decode(const LinDecode& p, hipStream_t st) {
  constexpr int GROUPS = DK / U, MOST = DECODE_TH / GROUPS / 4;  // tiles of 16 columns that a workgroup's threads reach
  const long heads = (long)p.B * p.H;
  const int tiles = p.DV / 16;
  long s = (DECODE_WGS + heads - 1) / heads;  // slabs: enough for the card, of two tiles at least
  if (s > (tiles + 1) / 2) s = (tiles + 1) / 2;
  if (s < (tiles + MOST - 1) / MOST) s = (tiles + MOST - 1) / MOST;
  const int per = (int)((tiles + s - 1) / s), slabs = (tiles + per - 1) / per, threads = 4 * per * GROUPS;
  const long units = heads * slabs, many = units / DECODE_WGS;
  const int fit = DECODE_TH / threads, pack = many < 1 ? 1 : many < fit ? (int)many : fit;
  const dim3 grid((unsigned)((units + pack - 1) / pack)), block((threads * pack + WAVE - 1) / WAVE * WAVE);
  hipLaunchKernelGGL((decode_kernel<E, DK, U>), grid, block, 0, st, p, 4 * per, slabs, pack);
  return hipGetLastError();
}

template <typename E>
hipError_t decode_by_dk(const LinDecode& p, hipStream_t st) {
  switch (p.DK) {
    case 16: return decode<E, 16, 4>(p, st);
    case 32: return decode<E, 32, 4>(p, st);
    case 64: return decode<E, 64, 8>(p, st);
    case 128: return decode<E, 128, 8>(p, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// Segments of a sequence, of NS chunks each.  A segment's chunks follow one another, so a call takes some time for each
// chunk of a segment; and it moves four states (backward: twelve, three chains being side by side) for each segment of
// each sequence and head.  The sum of the two is least where NS goes with the square root of (heads x chunks); the
// factors are measured.  Then the launch should fill the card: forward 512 workgroups, backward 256 of each chain, no
// more (a second round) and not much less.  Measured, us, 128 x 128 states, here and (segments: us) otherwise:
//   backward bf16  2 x 16 heads of 8K tokens in 8 segments 367 (6: 405, 9: 412, 10: 384, 16: 383); 4 x 16 of 2K in 4 193 (3:
//     214, 5: 220); 2 of 30000 in 79 164 (59: 161, 118: 196); 4 of 2K in 16 61 (8: 72, 32: 68)
//     (a number a little over a whole round of the three, 512, is worse than that round: 2 x 16 of 4K in 5 200, in 6 214)
//   backward float32  16 heads of 16K in 16 1067 (18: 1336, 23: 1279); 2 of 30000 in 79 355, in 86 418
//   forward bf16  4 x 16 of 2K in 8 77 (6: 85, 11: 104); 2 x 16 of 8K in 16 123 (8: 155); 64K of 16 heads in 32 417 (64: 528)
//   forward float32, whose workgroups are alone on a compute unit with such states and which therefore takes no number
//     between one and one and a half times 256: 2 of 30000 in 128 144 (188: 178); 2 x 16 of 8K, 64 x 64, in 16 136 (8: 182)
// Two segments (backward: three) are hardly ever worth the summaries' reads and launch: 8 x 16 of 2K backward 321 in one,
// 372 in two; 8 x 8 of 777 111 in one, 116 in three; 12 x 16 of 1K forward 69 in one, 76 in two.
void lin_split(int B, int L, int H, int dv, bool bf16, bool backward, int& NT, int& P, int& NS) {
  const int C = lin_chunk(bf16);
  NT = (L + C - 1) / C;
  P = NT > 0, NS = NT;
  const long units = (long)B * H * (backward ? 1 : (dv + LIN_SLAB - 1) / LIN_SLAB);
  if (NT == 0 || units == 0) return;
  const long card = backward ? 256 : 512, most = card / units;
  const double ns = sqrt((double)units * NT / (backward ? 24 : 64));
  const int n = ns < 1.5 ? 1 : (int)(ns + 0.5);
  long p = (NT + n - 1L) / n;
  // a round of workgroups and few more
  const long round = backward ? 512 / 3 : 256, few = backward ? 208 : 384;
  if ((backward ? dv <= 128 : !bf16) && units * p > round && units * p <= few) p = round / units;
  else if (4 * p >= 3 * most + backward) p = most;
  if (p > NT) p = NT;
  if (p < (backward ? 4 : 3)) return;
  NS = (int)((NT + p - 1) / p);  // as even as that many segments can be
  P = (NT + NS - 1) / NS;
}

hipError_t launch_lin_combine(const LinChain* forward, const LinChain* reverse, double* bounds, hipStream_t st) {
  const LinChain& c = forward ? *forward : *reverse;
  const long quads = (long)c.y.width * c.z.width / 4, all = quads * c.B * c.H;
  const dim3 grid((unsigned)((all + 255) / 256));
  auto of = [](const LinChain* c) {
    Walk w = {};
    if (c) {
      w.start = reinterpret_cast<const floatx4*>(c->start), w.segs = reinterpret_cast<floatx4*>(c->segs);
      w.end = reinterpret_cast<floatx4*>(c->end), w.decay = c->decay;
    }
    return w;
  };
  const Walk f = of(forward), r = of(reverse);
  if (!reverse) hipLaunchKernelGGL((combine_kernel<true, false, false>), grid, dim3(256), 0, st, c.P, quads, all, f, r, bounds);
  else if (!forward) hipLaunchKernelGGL((combine_kernel<false, true, false>), grid, dim3(256), 0, st, c.P, quads, all, f, r, bounds);
  else if (!bounds) hipLaunchKernelGGL((combine_kernel<true, true, false>), grid, dim3(256), 0, st, c.P, quads, all, f, r, bounds);
  else hipLaunchKernelGGL((combine_kernel<true, true, true>), grid, dim3(256), 0, st, c.P, quads, all, f, r, bounds);
  return hipGetLastError();
}

hipError_t launch_lin_gates(const LinGates& p, hipStream_t st) {
  const long n = (long)p.B * p.H * p.P;
  if (n > 0) {
    hipLaunchKernelGGL(gates_kernel, dim3((unsigned)n), dim3(GATE_TH), 0, st, p);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (p.gate == LIN_GATE_HEAD) hipLaunchKernelGGL(gate_heads_kernel, dim3(p.H), dim3(WAVE), 0, st, p.B, p.H, p.P, p.part, p.dg);
  return hipGetLastError();
}

hipError_t launch_lin_share(const float* dq_part, const float* dk_part, void* dq, void* dk, long rows, int heads, int share, int width,
                            bool bf16_out, hipStream_t st) {
  const long quads = rows * heads * width / 4;
  const long all = (2 * quads + 255) / 256, most = 1 << 16;  // more walk: a launch has fewer than 2^32 threads
  const dim3 grid((unsigned)(all < most ? all : most));
  if (bf16_out)
    hipLaunchKernelGGL((share_kernel<bf16>), grid, dim3(256), 0, st, dq_part, dk_part, static_cast<bf16*>(dq), static_cast<bf16*>(dk),
                       quads, share, width);
  else
    hipLaunchKernelGGL((share_kernel<float>), grid, dim3(256), 0, st, dq_part, dk_part, static_cast<float*>(dq), static_cast<float*>(dk),
                       quads, share, width);
  return hipGetLastError();
}

hipError_t launch_lin_decode(const LinDecode& p, bool bf16_in, hipStream_t st) {
  return bf16_in ? decode_by_dk<bf16>(p, st) : decode_by_dk<float>(p, st);
}

}  // namespace delta
