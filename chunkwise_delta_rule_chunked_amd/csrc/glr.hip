// Gated linear recurrence: per channel h_t = a_t h_{t-1} + w_t x_t with a = exp(g), its gradients
// and its one-token step (include/delta_block.h).
//
// A hard reset (g = -inf, a = 0) drops the previous state by selection rather than by
// multiplication, so that nothing of it, NaN and infinities included, is seen after it; the same
// holds for the gradient that flows back.  State, gates and sums are float32.
//
// Nothing but bytes bounds these kernels (an exp and about 20 other instructions per element), so
// the sequence kernels read each input once and write each output once, in one pass.  A workgroup
// takes a tile of TT tokens x 64 channels: 16 groups of 16 lanes, a group TPL consecutive tokens, a
// lane 4 channels.  The tile's gates and inputs stay in registers while its place in the sequence is
// found:
//   1. each lane reduces its tokens to the affine map of the state (A, H): h -> A h + H;
//   2. one wavefront, a lane per channel, folds the 16 groups' maps into the tile's, publishes it,
//      waits for a predecessor's state (below) and publishes the state behind the tile;
//   3. each group runs its tokens again from its start state, writing outputs.
// Tiles of one channel block and sequence form a chain.  A tile's predecessors publish their map as
// soon as they have read their tokens and the state behind them as soon as they know it; a tile
// starts from the nearest state it finds among its WINDOW predecessors and folds in the maps between.
// The fold is the same left fold whichever state it starts from, so the result does not depend on
// timing.  A published word carries its own readiness: the workspace starts as all ones, a NaN that
// no published value has, so no fence orders data and flag.  Tiles are handed out in chain order by a
// counter: whoever a tile waits for has started before it and waits for nobody behind it, so every
// wait ends (and is bounded besides: past POLLS polls, as can only happen if two calls share a
// workspace, the tile goes on with NaN).
//
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

// The gate's factor, with the sign bit (which exp never sets) marking a hard reset.  Products carry
// the mark along, so that a reset is told from a product that underflows.
__device__ inline unsigned bits(float x) { return __builtin_bit_cast(unsigned, x); }
__device__ inline float from_bits(unsigned x) { return __builtin_bit_cast(float, x); }
__device__ inline bool reset(float a) { return (int)bits(a) < 0; }
__device__ inline float gate_factor(float g) { return g == -__builtin_inff() ? -0.f : gate_exp(g); }
__device__ inline float times(float a, float b) {
  return from_bits((bits(a * b) & 0x7fffffffu) | ((bits(a) | bits(b)) & 0x80000000u));
}
__device__ inline float step(float a, float h, float u) { return reset(a) ? u : a * h + u; }

// Four consecutive channels.
__device__ inline void load4(const float* p, float* v) {
  const floatx4 r = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(p));
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = r[e];
}
__device__ inline void load4(const bf16* p, float* v) {
  const bf16x4 r = __builtin_bit_cast(bf16x4, __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p)));
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = to_float(r[e]);
}

constexpr int WG = 256, LPR = 16, NG = WG / LPR, CC = 4 * LPR;  // lanes per row, groups, channels of a tile
constexpr int TPL_FWD = 16, TPL_BWD = 8;                        // tokens per lane
constexpr int WINDOW = 8, POLLS = 1 << 22;
static_assert(NG * TPL_FWD % GLR_CHUNK == 0 && NG * TPL_BWD % GLR_CHUNK == 0, "a tile starts at a kept state");
static_assert(GLR_CHUNK % TPL_FWD == 0 && GLR_CHUNK % TPL_BWD == 0, "kept states fall between groups");

// What the tiles of one call publish: per tile and channel its map and the state behind it; then
// the counter that hands out tiles.
struct Chain {
  uint64_t* map;   // [B, tiles, D]: A in the low half, H in the high one
  uint32_t* state; // [B, tiles, D]
  uint32_t* next;
  int tiles;       // per sequence
};

__device__ inline unsigned plain_nan(float x) { return x != x ? (bits(x) & 0x80000000u) | 0x7fc00000u : bits(x); }
template <typename T>
__device__ inline void publish(T* p, T v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <typename T>
__device__ inline T look(const T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// The state this tile starts from, for the channel of this lane (of a whole wavefront; `live`: the
// channel exists), publishing the tile's map and the state behind it.  at: the tile's word.
__device__ inline float chain_state(const Chain& c, long at, long stride, int tile, bool live, float A, float H,
                                    float init) {
  if (c.tiles == 1) return init;
  float h = init;
  if (tile > 0) {
    if (live) publish(c.map + at, (uint64_t)plain_nan(H) << 32 | plain_nan(A));
    int found = -1;
    uint64_t m[WINDOW];
    uint32_t s[WINDOW];
    for (int poll = 0; poll < POLLS; ++poll) {
#pragma unroll
      for (int k = 0; k < WINDOW; ++k) {
        m[k] = 0, s[k] = 0;
        if (live && k < tile) {
          s[k] = look(c.state + at - (k + 1) * stride);
          m[k] = look(c.map + at - (k + 1) * stride);
        }
      }
      bool open = true;  // every map nearer than this one is there
#pragma unroll
      for (int k = 0; k < WINDOW; ++k) {
        if (open && k < tile && found < 0 && __all(s[k] != ~0u)) found = k;
        open = open && k < tile && __all(m[k] != ~0ull);
      }
      if (found >= 0) break;
      __builtin_amdgcn_s_sleep(1);
    }
    h = __builtin_nanf("");
#pragma unroll
    for (int k = WINDOW - 1; k >= 0; --k) {
      if (k == found) h = from_bits(s[k]);
      else if (k < found) h = step(from_bits((unsigned)m[k]), h, from_bits((unsigned)(m[k] >> 32)));
    }
  }
  if (live && tile + 1 < c.tiles) publish(c.state + at, plain_nan(step(A, h, H)));
  return h;
}

// This workgroup's tile of the whole call: tiles in chain order, channel blocks fastest.
__device__ inline unsigned take_tile(const Chain& c) {
  if (c.tiles == 1) return blockIdx.x;
  __shared__ unsigned mine;
  if (threadIdx.x == 0) mine = __hip_atomic_fetch_add(c.next, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
  __syncthreads();
  return mine;
}

__global__ __launch_bounds__(256) void glr_clear_kernel(u32x4* p, long n) {
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) p[i] = u32x4{~0u, ~0u, ~0u, ~0u};
}

template <typename E, int GATE>
__global__ __launch_bounds__(WG) void glr_fwd_kernel(GlrParams p, Chain chain) {
  constexpr int TPL = TPL_FWD, TT = NG * TPL;
  __shared__ float sA[NG][CC], sH[NG][CC];  // the groups' maps; then sH the groups' start states
  const unsigned job = take_tile(chain), nblk = (p.D + CC - 1) / CC, chains = nblk * p.B;
  const int tile = job / chains, b = job % chains / nblk, c0 = (int)(job % chains % nblk) * CC;
  const int tid = threadIdx.x, grp = tid / LPR, c = c0 + tid % LPR * 4;
  const int t0 = tile * TT + grp * TPL;
  const bool here = c < p.D;
  const long base = ((long)b * p.L + t0) * p.D + c;
  float a[TPL][4], u[TPL][4], A[4], H[4];
#pragma unroll
  for (int j = 0; j < TPL; ++j) {
    // tokens past the end are the identity: g = 0 (a = 1), x = 0
#pragma unroll
    for (int e = 0; e < 4; ++e) a[j][e] = u[j][e] = 0.f;
    if (here && t0 + j < p.L) {
      load4(p.g + base + (long)j * p.D, a[j]);
      load4(static_cast<const E*>(p.x) + base + (long)j * p.D, u[j]);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) A[e] = 1.f, H[e] = 0.f;
#pragma unroll
  for (int j = 0; j < TPL; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[j][e] *= weight<GATE>(a[j][e]);
      a[j][e] = gate_factor(a[j][e]);
      A[e] = times(A[e], a[j][e]);
      H[e] = step(a[j][e], H[e], u[j][e]);
    }
  const int col = tid % LPR * 4;
  *reinterpret_cast<floatx4*>(&sA[grp][col]) = floatx4{A[0], A[1], A[2], A[3]};
  *reinterpret_cast<floatx4*>(&sH[grp][col]) = floatx4{H[0], H[1], H[2], H[3]};
  __syncthreads();
  if (tid < CC) {
    const int ch = c0 + tid;
    const bool live = ch < p.D;
    float TA = 1.f, TH = 0.f;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      TH = step(sA[k][tid], TH, sH[k][tid]);
      TA = times(TA, sA[k][tid]);
    }
    float h = chain_state(chain, ((long)b * chain.tiles + tile) * p.D + ch, p.D, tile, live, TA, TH,
                          live && p.h0 ? p.h0[(long)b * p.D + ch] : 0.f);
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      const float next = step(sA[k][tid], h, sH[k][tid]);
      sH[k][tid] = h;
      h = next;
    }
    if (live && p.h_final && tile == chain.tiles - 1) p.h_final[(long)b * p.D + ch] = h;
  }
  __syncthreads();
  if (!here) return;
  floatx4 h = *reinterpret_cast<const floatx4*>(&sH[grp][col]);
  if (p.states && t0 % GLR_CHUNK == 0 && t0 < p.L) {
    const int nc = (p.L + GLR_CHUNK - 1) / GLR_CHUNK;
    *reinterpret_cast<floatx4*>(p.states + ((long)b * nc + t0 / GLR_CHUNK) * p.D + c) = h;
  }
#pragma unroll
  for (int j = 0; j < TPL; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = step(a[j][e], h[e], u[j][e]);
    if (t0 + j < p.L) store4<E>(static_cast<E*>(p.O) + base + (long)j * p.D, h[0], h[1], h[2], h[3]);
  }
}

// The same from the other end.  With flow_t = a_t lambda_t, the gradient that reaches the state
// before token t, flow_t = a_t (dO_t + flow_{t+1}): an affine recurrence over the same gates, tiles
// handed out from the last to the first.  A group's start state comes from the kept state of its
// 64 tokens and the maps of the groups between.
template <typename E, int GATE>
__global__ __launch_bounds__(WG) void glr_bwd_kernel(GlrParams p, Chain chain) {
  constexpr int TPL = TPL_BWD, TT = NG * TPL, GPC = GLR_CHUNK / TPL;  // groups per kept state
  __shared__ float sA[NG][CC], sH[NG][CC], sF[NG][CC];
  const unsigned job = take_tile(chain), nblk = (p.D + CC - 1) / CC, chains = nblk * p.B;
  const int order = job / chains, b = job % chains / nblk, c0 = (int)(job % chains % nblk) * CC;
  const int tid = threadIdx.x, grp = tid / LPR, c = c0 + tid % LPR * 4;
  const int tile0 = (chain.tiles - 1 - order) * TT, t0 = tile0 + grp * TPL;
  const bool here = c < p.D;
  const long base = ((long)b * p.L + t0) * p.D + c;
  float a[TPL][4], w[TPL][4], x[TPL][4], d[TPL][4], A[4], H[4], F[4];
#pragma unroll
  for (int j = 0; j < TPL; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) a[j][e] = x[j][e] = d[j][e] = 0.f;
    if (here && t0 + j < p.L) {
      load4(p.g + base + (long)j * p.D, a[j]);
      load4(static_cast<const E*>(p.x) + base + (long)j * p.D, x[j]);
      load4(static_cast<const E*>(p.dO) + base + (long)j * p.D, d[j]);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) A[e] = 1.f, H[e] = F[e] = 0.f;
#pragma unroll
  for (int j = 0; j < TPL; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[j][e] = weight<GATE>(a[j][e]);
      a[j][e] = gate_factor(a[j][e]);
      A[e] = times(A[e], a[j][e]);
      H[e] = step(a[j][e], H[e], w[j][e] * x[j][e]);
    }
#pragma unroll
  for (int j = TPL - 1; j >= 0; --j)
#pragma unroll
    for (int e = 0; e < 4; ++e) F[e] = step(a[j][e], d[j][e] + F[e], 0.f);
  const int col = tid % LPR * 4;
  *reinterpret_cast<floatx4*>(&sA[grp][col]) = floatx4{A[0], A[1], A[2], A[3]};
  *reinterpret_cast<floatx4*>(&sH[grp][col]) = floatx4{H[0], H[1], H[2], H[3]};
  *reinterpret_cast<floatx4*>(&sF[grp][col]) = floatx4{F[0], F[1], F[2], F[3]};
  __syncthreads();
  if (tid < CC) {
    const int ch = c0 + tid, nc = (p.L + GLR_CHUNK - 1) / GLR_CHUNK;
    const bool live = ch < p.D;
    float start[NG / GPC];
#pragma unroll
    for (int n = 0; n < NG / GPC; ++n) {
      const int chunk = tile0 / GLR_CHUNK + n;
      start[n] = live && chunk < nc ? p.states[((long)b * nc + chunk) * p.D + ch] : 0.f;
    }
    float TA = 1.f, TF = 0.f;
#pragma unroll
    for (int k = NG - 1; k >= 0; --k) {
      TF = step(sA[k][tid], TF, sF[k][tid]);
      TA = times(TA, sA[k][tid]);
    }
    float flow = chain_state(chain, ((long)b * chain.tiles + order) * p.D + ch, p.D, order, live, TA, TF,
                             live && p.dh_final ? p.dh_final[(long)b * p.D + ch] : 0.f);
#pragma unroll
    for (int k = NG - 1; k >= 0; --k) {
      const float next = step(sA[k][tid], flow, sF[k][tid]);
      sF[k][tid] = flow;
      flow = next;
    }
    if (live && p.dh0 && order == chain.tiles - 1) p.dh0[(long)b * p.D + ch] = flow;
#pragma unroll
    for (int n = 0; n < NG / GPC; ++n) {
      float h = start[n];
#pragma unroll
      for (int k = n * GPC; k < (n + 1) * GPC; ++k) {
        const float next = step(sA[k][tid], h, sH[k][tid]);
        sH[k][tid] = h;
        h = next;
      }
    }
  }
  __syncthreads();
  if (!here) return;
  floatx4 h = *reinterpret_cast<const floatx4*>(&sH[grp][col]), flow = *reinterpret_cast<const floatx4*>(&sF[grp][col]);
#pragma unroll
  for (int j = 0; j < TPL; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // x becomes dh_t / dg_t
      const float q = reset(a[j][e]) ? 0.f : a[j][e] * h[e] + slope<GATE>(a[j][e], w[j][e]) * x[j][e];
      h[e] = step(a[j][e], h[e], w[j][e] * x[j][e]);
      x[j][e] = q;
    }
#pragma unroll
  for (int j = TPL - 1; j >= 0; --j) {
    if (t0 + j < p.L) {
      floatx4 dx, dg;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lam = d[j][e] + flow[e];
        dx[e] = w[j][e] * lam;
        dg[e] = reset(a[j][e]) ? 0.f : lam * x[j][e];
        flow[e] = step(a[j][e], lam, 0.f);
      }
      *reinterpret_cast<floatx4*>(p.dx + base + (long)j * p.D) = dx;
      *reinterpret_cast<floatx4*>(p.dg + base + (long)j * p.D) = dg;
    }
  }
}

template <typename E, int GATE>
__global__ __launch_bounds__(256) void glr_decode_kernel(GlrParams p) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long)p.B * p.D) return;
  const float g = p.g[i];
  const float h = step(gate_factor(g), p.h_final[i], weight<GATE>(g) * to_float(static_cast<const E*>(p.x)[i]));
  p.h_final[i] = h;
  static_cast<E*>(p.O)[i] = to_elem<E>(h);
}

enum Which { FWD, BWD, DECODE };

int tile_tokens(Which which) { return NG * (which == FWD ? TPL_FWD : TPL_BWD); }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <typename E, int GATE>
hipError_t launch_one(const GlrParams& p, Which which, hipStream_t st) {
  if (which == DECODE) {
    const long n = (long)p.B * p.D;
    hipLaunchKernelGGL((glr_decode_kernel<E, GATE>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, p);
    return hipGetLastError();
  }
  const int TT = tile_tokens(which);
  Chain c{nullptr, nullptr, nullptr, p.L > TT ? (p.L + TT - 1) / TT : 1};
  if (c.tiles > 1) {
    const size_t n = (size_t)p.B * c.tiles * p.D, total = up256(n * 8) + up256(n * 4) + 256;
    char* ws = static_cast<char*>(p.ws);
    c.map = reinterpret_cast<uint64_t*>(ws);
    c.state = reinterpret_cast<uint32_t*>(ws + up256(n * 8));
    c.next = reinterpret_cast<uint32_t*>(ws + total - 256);
    const long v = (long)(total / 16);
    const long wgs = (v + 255) / 256;
    hipLaunchKernelGGL(glr_clear_kernel, dim3((unsigned)(wgs < 2048 ? wgs : 2048)), dim3(256), 0, st,
                       reinterpret_cast<u32x4*>(ws), v);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  const dim3 grid((unsigned)((p.D + CC - 1) / CC) * p.B * c.tiles);
  if (which == FWD) hipLaunchKernelGGL((glr_fwd_kernel<E, GATE>), grid, dim3(WG), 0, st, p, c);
  else hipLaunchKernelGGL((glr_bwd_kernel<E, GATE>), grid, dim3(WG), 0, st, p, c);
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

size_t glr_workspace(int B, int L, int D, bool backward) {
  const int TT = tile_tokens(backward ? BWD : FWD);
  if (L <= TT) return 0;
  const size_t n = (size_t)B * ((L + TT - 1) / TT) * D;
  return n ? up256(n * 8) + up256(n * 4) + 256 : 0;
}
bool glr_grid_fits(int B, int L, int D) {
  return (double)((D + CC - 1) / CC) * B * ((L + (double)NG * TPL_BWD - 1) / (NG * TPL_BWD)) < 0x1p31;
}

hipError_t launch_glr_fwd(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, FWD, st); }
hipError_t launch_glr_bwd(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, BWD, st); }
hipError_t launch_glr_decode(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, DECODE, st); }

}  // namespace delta
