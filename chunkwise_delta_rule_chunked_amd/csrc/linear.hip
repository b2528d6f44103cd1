// Linear attention with a decay for each head: the launches around the chain kernel (linear_chain.h), and
// the step for one token.
#include <hip/hip_runtime.h>

#include "common.h"
#include "linear.h"

namespace delta {
namespace lin {
hipError_t chain_bf16(const LinChain& c, bool reverse, int form, hipStream_t st);
hipError_t chain_f32(const LinChain& c, bool reverse, int form, hipStream_t st);
hipError_t summary_bf16(const LinChain& c, bool reverse, hipStream_t st);
hipError_t summary_f32(const LinChain& c, bool reverse, hipStream_t st);
}  // namespace lin

namespace {

// Each segment's result becomes its start: start_{p+1} = e^decay_p start_p + result_p, four elements a lane.
__global__ __launch_bounds__(256) void combine_kernel(int P, long quads, long all, const floatx4* start, floatx4* segs,
                                                      const double* decay, floatx4* end) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x, bh = i / quads, q = i % quads;
  if (i >= all) return;
  floatx4 s = start ? start[bh * quads + q] : floatx4{};
  floatx4* at = segs + bh * P * quads + q;
  const int n = end ? P : P - 1;  // without an end the last segment has no result
  constexpr int AHEAD = 8;        // results loaded at a time
  for (int p0 = 0; p0 < n; p0 += AHEAD) {
    floatx4 r[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (p0 + k < n) r[k] = at[(p0 + k) * quads];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (p0 + k < n) {
        at[(p0 + k) * quads] = s;
        s = s * expf((float)decay[bh * P + p0 + k]) + r[k];
      }
  }
  if (end) end[bh * quads + q] = s;
  else if (P > 0) at[(P - 1) * quads] = s;
}

__device__ inline double wave_total(double x) {
#pragma unroll
  for (int o = WAVE / 2; o > 0; o >>= 1) x += __shfl_xor(x, o, WAVE);
  return x;
}

// d log g of the tokens of one segment.  With b the inner product of the state before a chunk and its
// gradient, and X = e^gc_C <G, S> what the chunk's two ends share,
//     b = X + sum e,   b' = X + sum f,   d log g_t = X + sum_{r < t} f_r + sum_{r >= t} e_r
// (e with the pairs' row and column sums, which cancel over a chunk).  b is formed from the states at the
// segment's start and carried on from chunk to chunk; a chunk that lets nothing through has X = 0.
constexpr int GATE_TH = 256, GATE_WAVES = GATE_TH / WAVE, GATE_CHUNKS = 64;
__global__ __launch_bounds__(GATE_TH) void gates_kernel(LinGates p) {
  __shared__ double sums[GATE_WAVES], se[GATE_CHUNKS], sf[GATE_CHUNKS];
  __shared__ bool shut[GATE_CHUNKS];
  const int tid = threadIdx.x, lane = tid % WAVE, wave = tid / WAVE;
  const int seg = blockIdx.x % p.P;
  const long bh = blockIdx.x / p.P;
  const int h = (int)(bh % p.H);
  const long b = bh / p.H;
  const float *S = nullptr, *G = nullptr;
  if (seg > 0) {
    S = p.segs + (bh * p.P + seg) * p.state;
    G = p.gsegs + (bh * p.P + p.P - seg) * p.state;  // behind segment seg - 1, the reverse chain's P - seg
  } else if (p.S0) {
    S = p.S0 + bh * p.state;
    G = p.dS0 + bh * p.state;
  }
  double x = 0.0;
  if (S)
    for (size_t i = 4 * tid; i < p.state; i += 4 * GATE_TH) {
      const floatx4 s = *reinterpret_cast<const floatx4*>(S + i), d = *reinterpret_cast<const floatx4*>(G + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) x += (double)s[k] * d[k];
    }
  x = wave_total(x);
  if (lane == 0) sums[wave] = x;
  __syncthreads();
  double before = 0.0, all = 0.0;
  for (int k = 0; k < GATE_WAVES; ++k) before += sums[k];
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
      const double a = wave_total((double)(gl < LOG_GATE_FLOOR ? LOG_GATE_FLOOR : gl));
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
      const bool reset = expf(gate(n)) == 0.f;
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
__global__ __launch_bounds__(256) void share_kernel(const float* part, E* out, long quads, int share, int width) {
  const long q = (long)blockIdx.x * 256 + threadIdx.x;
  if (q >= quads) return;
  const long i = q * 4, row = i / width;
  const float* from = part + row * share * width + i % width;
  floatx4 s = *reinterpret_cast<const floatx4*>(from);
  for (int k = 1; k < share; ++k) s += *reinterpret_cast<const floatx4*>(from + (long)k * width);
  store4<E>(out + i, s[0], s[1], s[2], s[3]);
}

// One token: S <- a S + k v^T, o = scale S^T q.  Bound by the state, read and written once: a workgroup has
// SW columns of one head's state, a thread 4 rows x 4 columns in 16-byte accesses with non-temporal hints,
// and the sums over the rows of S^T q meet in LDS.
template <typename E, int DK, int SW>
__global__ __launch_bounds__(DK * SW / 16) void decode_kernel(LinDecode p) {
  constexpr int CQ = SW / 4, TH = DK / 4 * CQ, NW = (TH + WAVE - 1) / WAVE;
  __shared__ floatx4 red[NW][CQ];
  const int tid = threadIdx.x, cq = tid % CQ, r0 = tid / CQ * 4;
  const int slabs = p.DV / SW, slab = blockIdx.x % slabs;
  const long bh = blockIdx.x / slabs;
  const int h = (int)(bh % p.H);
  const long bk = bh / p.H * p.Hk + h / (p.H / p.Hk);
  float* Sg = p.S + bh * DK * p.DV + slab * SW + cq * 4;
  floatx4 s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(Sg + (long)(r0 + i) * p.DV));
  const E *q = static_cast<const E*>(p.q) + bk * DK + r0, *k = static_cast<const E*>(p.k) + bk * DK + r0;
  const E* v = static_cast<const E*>(p.v) + bh * p.DV + slab * SW + cq * 4;
  typedef E E4 __attribute__((ext_vector_type(4)));
  const E4 q4 = *reinterpret_cast<const E4*>(q), k4 = *reinterpret_cast<const E4*>(k), v4 = *reinterpret_cast<const E4*>(v);
  const float a = p.gate == LIN_GATE_NONE ? 1.f : expf(p.g[p.gate == LIN_GATE_TOKEN ? bh : h]);
  floatx4 o = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      s[i][c] = a * s[i][c] + to_float((E)k4[i]) * to_float((E)v4[c]);
      o[c] += to_float((E)q4[i]) * s[i][c];
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) __builtin_nontemporal_store(s[i], reinterpret_cast<floatx4*>(Sg + (long)(r0 + i) * p.DV));
#pragma unroll
  for (int off = CQ; off < (TH < WAVE ? TH : WAVE); off <<= 1)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] += __shfl_xor(o[c], off, WAVE);
  if constexpr (NW > 1) {
    if (tid % WAVE < CQ) red[tid / WAVE][tid % WAVE] = o;
    barrier_lds();
    if (tid < CQ) {
      o = red[0][tid];
#pragma unroll
      for (int w = 1; w < NW; ++w) o += red[w][tid];
    }
  }
  if (tid < CQ) store4<E>(static_cast<E*>(p.O) + bh * p.DV + slab * SW + cq * 4, p.scale * o[0], p.scale * o[1], p.scale * o[2], p.scale * o[3]);
}

template <typename E, int DK>
hipError_t decode_by_slab(const LinDecode& p, hipStream_t st) {
  const unsigned heads = (unsigned)(p.B * p.H);
  if (p.DV % 32 == 0) hipLaunchKernelGGL((decode_kernel<E, DK, 32>), dim3(heads * (p.DV / 32)), dim3(DK * 2), 0, st, p);
  else hipLaunchKernelGGL((decode_kernel<E, DK, 16>), dim3(heads * (p.DV / 16)), dim3(DK), 0, st, p);
  return hipGetLastError();
}

template <typename E>
hipError_t decode_by_dk(const LinDecode& p, hipStream_t st) {
  switch (p.DK) {
    case 16: return decode_by_slab<E, 16>(p, st);
    case 32: return decode_by_slab<E, 32>(p, st);
    case 64: return decode_by_slab<E, 64>(p, st);
    case 128: return decode_by_slab<E, 128>(p, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// Segments of a sequence: about two workgroups of a chain for each of 256 compute units, none split where the
// sequences and heads alone fill the card.
void lin_split(int B, int L, int H, int dv, bool bf16, int& NT, int& P, int& NS) {
  const int C = lin_chunk(bf16);
  NT = (L + C - 1) / C;
  const long units = (long)B * H * ((dv + LIN_SLAB - 1) / LIN_SLAB);
  if (NT == 0 || units == 0 || units >= 256) {
    P = NT > 0, NS = NT;
    return;
  }
  const long want = (512 + units - 1) / units;
  NS = (int)((NT + want - 1) / want);
  P = (NT + NS - 1) / NS;
}

hipError_t launch_lin_chain(const LinChain& c, bool bf16, bool reverse, int form, hipStream_t st) {
  return bf16 ? lin::chain_bf16(c, reverse, form, st) : lin::chain_f32(c, reverse, form, st);
}

hipError_t launch_lin_summary(const LinChain& c, bool bf16, bool reverse, hipStream_t st) {
  if (c.run > 0) {
    const hipError_t e = bf16 ? lin::summary_bf16(c, reverse, st) : lin::summary_f32(c, reverse, st);
    if (e != hipSuccess) return e;
  }
  const long quads = (long)c.y.width * c.z.width / 4, all = quads * c.B * c.H;
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((all + 255) / 256)), dim3(256), 0, st, c.P, quads, all,
                     reinterpret_cast<const floatx4*>(c.start), reinterpret_cast<floatx4*>(c.segs), c.decay,
                     reinterpret_cast<floatx4*>(c.end));
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

hipError_t launch_lin_share(const float* part, void* out, long rows, int heads, int share, int width, bool bf16_out,
                            hipStream_t st) {
  const long quads = rows * heads * width / 4;
  const dim3 grid((unsigned)((quads + 255) / 256));
  if (bf16_out) hipLaunchKernelGGL((share_kernel<bf16>), grid, dim3(256), 0, st, part, static_cast<bf16*>(out), quads, share, width);
  else hipLaunchKernelGGL((share_kernel<float>), grid, dim3(256), 0, st, part, static_cast<float*>(out), quads, share, width);
  return hipGetLastError();
}

hipError_t launch_lin_decode(const LinDecode& p, bool bf16_in, hipStream_t st) {
  return bf16_in ? decode_by_dk<bf16>(p, st) : decode_by_dk<float>(p, st);
}

}  // namespace delta
