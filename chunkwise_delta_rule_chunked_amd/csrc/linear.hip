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

// e^d for a segment's sum d of log gates, as a factor to multiply by once or three times.  With gates above 1 e^d may be no
// float32 number although s e^d is (s is small, or 0): then in three steps, each between s and the result.  Past e^240
// every s is 0, infinite or 0 again.
struct Decay {
  float factor;
  bool thrice;
  __device__ inline Decay() {}
  __device__ inline Decay(double d) : thrice(fabs(d) > 80.0 && d != -INFINITY) {
    factor = expf((float)(thrice ? fmin(fmax(d, -240.0), 240.0) / 3 : d));
  }
  __device__ inline floatx4 operator()(floatx4 s) const {
    s *= factor;
    if (thrice) s = s * factor * factor;
    return s;
  }
};

// One chain's states of one place, four elements a lane, from segment to segment: a segment's result becomes its start,
// start_{p+1} = e^decay_p start_p + result_p.
struct Walk {
  const floatx4* start;
  floatx4 *segs, *end;
  const double* decay;
};
__device__ inline void walk(const Walk& w, int P, long quads, long bh, long q) {
  floatx4 s = w.start ? w.start[bh * quads + q] : floatx4{};
  floatx4* at = w.segs + bh * P * quads + q;
  const int n = w.end ? P : P - 1;  // without an end the last segment has no result
  constexpr int AHEAD = 8;          // results loaded at a time
  for (int p0 = 0; p0 < n; p0 += AHEAD) {
    floatx4 r[AHEAD];
    Decay decay[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (p0 + k < n) r[k] = at[(p0 + k) * quads], decay[k] = Decay(w.decay[bh * P + p0 + k]);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (p0 + k < n) {
        at[(p0 + k) * quads] = s;
        s = decay[k](s) + r[k];
      }
  }
  if (w.end) w.end[bh * quads + q] = s;
  else if (P > 0) at[(P - 1) * quads] = s;
}

template <bool FORWARD, bool REVERSE>
__global__ __launch_bounds__(256) void combine_kernel(int P, long quads, long all, Walk forward, Walk reverse) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x, bh = i / quads, q = i % quads;
  if (i >= all) return;
  if constexpr (FORWARD) walk(forward, P, quads, bh, q);
  if constexpr (REVERSE) walk(reverse, P, quads, bh, q);
}

// d log g_t = a_t <G_t, S_{t-1}>: every pair of a write before t and a read from t on.  For the tokens of a chunk these
// are
//     X + sum_{r >= t} e_r + sum_{r < t} f_r + pair_t
// with X = e^gc_C <G, S> what passes the chunk whole, e_r what the state at its start gives to token r's output (reads
// in it of writes before it), f_r the same in the other order, and pair_t the pairs in it around t.  All are formed from
// states with their decays, and sums run over terms that all cross t: a token's error goes by what crosses that token.
// (X carried from chunk to chunk by e and f, which differ by it, keeps the errors of far larger tokens that the state has
// long forgotten.)  A wavefront has a chunk.
constexpr int GATE_TH = 256, GATE_WAVES = GATE_TH / WAVE;
__global__ __launch_bounds__(GATE_TH) void gates_kernel(LinGates p, int groups) {
  __shared__ double sums[GATE_WAVES];
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  const long bh = blockIdx.x / groups;
  const int h = (int)(bh % p.H);
  const long b = bh / p.H;
  const int first = blockIdx.x % groups * LIN_GATE_CHUNKS, last = min(first + LIN_GATE_CHUNKS, p.NT);
  double all = 0.0;
  for (int n = first + wave; n < last; n += GATE_WAVES) {
    const size_t i = (bh * p.NT + n) * p.C + lane;
    const long token = (long)n * p.C + lane;
    const bool in = lane < p.C, on = in && token < p.L;
    double up = in ? p.e[i] : 0.0, down = in ? p.f[i] : 0.0, dg = in ? p.pair[i] : 0.0;
    const float gate = !on ? 0.f : p.gate == LIN_GATE_TOKEN ? p.g[(b * p.L + token) * p.H + h] : p.g[h];
    dg += p.edge[bh * p.NT + n];
#pragma unroll
    for (int o = 1; o < WAVE; o <<= 1) {
      const double u = __shfl_down(up, o, WAVE), d = __shfl_up(down, o, WAVE);
      if (lane + o < WAVE) up += u;
      if (lane >= o) down += d;
    }
    const double past = __shfl_up(down, 1, WAVE);
    dg += up;
    if (lane > 0) dg += past;
    if (lin_log_gate(gate) == LIN_RESET) dg = 0.0;  // nothing flows past a reset
    if (on) {
      if (p.gate == LIN_GATE_TOKEN) p.dg[(b * p.L + token) * p.H + h] = (float)dg;
      else all += dg;
    }
  }
  if (p.gate == LIN_GATE_HEAD) {
    all = wave_total(all);
    if (lane == 0) sums[wave] = all;
    __syncthreads();
    if (threadIdx.x == 0) {
      double s = 0.0;
      for (int k = 0; k < GATE_WAVES; ++k) s += sums[k];
      p.part[blockIdx.x] = s;
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
// more (a second round) and not much less.  Measured, us, 128 x 128 states, here and (segments: us) otherwise; backward
// with the gates' gradients:
//   backward bf16  2 x 16 heads of 8K tokens in 8 segments 461 (6: 500, 9: 516, 10: 491, 16: 489); 4 x 16 of 2K in 4 253 (3:
//     263, 5: 292); 2 of 30000 in 79 184 (59: 178, 118: 215); 4 of 2K in 16 69 (8: 82, 32: 82)
//   backward float32  16 heads of 16K in 16 1194 (18: 1480, 23: 1348); 2 of 30000 in 85 401, in 86 436
//   forward bf16  4 x 16 of 2K in 8 82 (6: 91, 11: 109); 2 x 16 of 8K in 16 128 (8: 161); 64K of 16 heads in 32 424 (64: 534)
// A number of backward workgroups a little over a third of 512, which is one round of the three chains on the card, is
// lowered to it: 16 heads of 4608 tokens would take 11 segments, 178 us (without gates' gradients 122), and take 10, 173
// (102).  Only for the chains that run side by side.  Float32 forward, whose workgroups are alone on a compute unit with
// such states, likewise takes no number between one and one and a half times 256: 2 of 30000 in 128 151 (188: 190); 2 x 16
// of 8K, 64 x 64, in 16 145 (8: 182).
// Two segments (backward: three) are hardly ever worth the summaries' reads and launch: 8 x 16 of 2K backward 365 in one,
// 465 in two; 8 x 8 of 777 134 in one, 142 in three; 12 x 16 of 1K forward 102 in one, 118 in two.
void lin_split(int B, int L, int H, int dv, bool bf16, bool backward, int& NT, int& P, int& NS, int& most_segments) {
  const int C = lin_chunk(bf16);
  NT = (L + C - 1) / C;
  P = most_segments = NT > 0, NS = NT;
  const long units = (long)B * H * (backward ? 1 : (dv + LIN_SLAB - 1) / LIN_SLAB);
  if (NT == 0 || units == 0) return;
  const long card = backward ? 256 : 512, most = card / units;  // no rule below takes more segments than `most`
  const double ns = sqrt((double)units * NT / (backward ? 24 : 64));
  const int n = ns < 1.5 ? 1 : (int)(ns + 0.5);
  long p = (NT + n - 1L) / n;
  const long round = backward ? 512 / 3 : 256, few = backward ? 208 : 384;
  if ((backward ? dv <= 128 : !bf16) && units * p > round && units * p <= few) p = round / units;
  else if (backward ? 4 * p > 3 * most : 4 * p >= 3 * most) p = most;
  if (p > NT) p = NT;
  const long least = backward ? 4 : 3, up_to = most < NT ? most : NT;
  if (up_to >= least) most_segments = (int)up_to;
  if (p < least) return;
  NS = (int)((NT + p - 1) / p);  // as even as that many segments can be
  P = (NT + NS - 1) / NS;
}

hipError_t launch_lin_combine(const LinChain* forward, const LinChain* reverse, hipStream_t st) {
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
  if (!reverse) hipLaunchKernelGGL((combine_kernel<true, false>), grid, dim3(256), 0, st, c.P, quads, all, f, r);
  else if (!forward) hipLaunchKernelGGL((combine_kernel<false, true>), grid, dim3(256), 0, st, c.P, quads, all, f, r);
  else hipLaunchKernelGGL((combine_kernel<true, true>), grid, dim3(256), 0, st, c.P, quads, all, f, r);
  return hipGetLastError();
}

hipError_t launch_lin_gates(const LinGates& p, hipStream_t st) {
  const int groups = (p.NT + LIN_GATE_CHUNKS - 1) / LIN_GATE_CHUNKS;
  const long n = (long)p.B * p.H * groups;
  if (n > 0) {
    hipLaunchKernelGGL(gates_kernel, dim3((unsigned)n), dim3(GATE_TH), 0, st, p, groups);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (p.gate == LIN_GATE_HEAD) hipLaunchKernelGGL(gate_heads_kernel, dim3(p.H), dim3(WAVE), 0, st, p.B, p.H, groups, p.part, p.dg);
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
