// Gated linear recurrence: per channel h_t = a_t h_{t-1} + w_t x_t with a = exp(g), its gradients
// and its one-token step (include/delta_block.h).
//
// A hard reset (a = 0) drops the previous state by selection rather than by
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
// starts from the nearest state it finds among its 64 predecessors and folds in the maps between.
// The fold is the same left fold whichever state it starts from, so the result does not depend on
// timing.  Waiting reads one flag per predecessor (a lane each, a cache line in all).  A flag is only a
// hint: a published word carries its own readiness, since the workspace starts as all ones, a NaN that
// no published value has, so no fence orders data and flag.  A counter per chain hands out its tiles in
// order: whoever a tile waits for has started before it and waits for nobody behind it, so every
// wait ends (and is bounded besides: past POLLS polls, as can only happen if two calls share a
// workspace, the tile goes on with NaN).
//
#include <hip/hip_runtime.h>

#include "block_kernels.h"
#include "common.h"

namespace delta {
namespace {

enum { NONE = 0, COMPLEMENT = 1, NORM = 2 };

__device__ inline unsigned bits(float x) { return __builtin_bit_cast(unsigned, x); }
__device__ inline float from_bits(unsigned x) { return __builtin_bit_cast(float, x); }

// a = exp(g).  a = 0 (g = -inf, or an exp that underflows) is the hard reset.  Where a product of gates
// could underflow too, the sign bit, which no exp has (a NaN loses it here), marks a reset: products
// carry the mark along.
__device__ inline float factor(float g) { return fabsf(gate_exp(g)); }
__device__ inline float mark(float a) { return a == 0.f ? -0.f : a; }
__device__ inline bool reset(float a) { return (int)bits(a) < 0; }
__device__ inline float times(float a, float b) {
  return from_bits((bits(a * b) & 0x7fffffffu) | ((bits(a) | bits(b)) & 0x80000000u));
}
__device__ inline float step(float a, float h, float u) { return reset(a) ? u : a * h + u; }

// The same for the tokens a lane holds.  RESETS: whether a reset is among the wavefront's; without one
// (nearly always) the marks cost nothing.
template <bool RESETS>
struct Gates {
  __device__ static inline float marked(float a) { return RESETS ? mark(a) : a; }
  __device__ static inline float product(float a, float b) { return RESETS ? times(a, b) : a * b; }
  __device__ static inline float next(float a, float h, float u) { return RESETS ? step(a, h, u) : a * h + u; }
  // what multiplies into a gradient: nothing at a reset, whatever v is
  __device__ static inline float pass(float a, float v) { return RESETS && reset(a) ? 0.f : v; }
};

// w(g), from a = exp(g).  1 - exp(z) cancels near z = 0, where its series to z^7 takes over (|z| < 0.35:
// the first dropped term is below 0.35^7 / 8! = 2e-8 of the result); beyond, 1 - a or 1 - a^2 is good to
// a dozen units of 2^-24.  For the square root z = 2 g.
template <int GATE>
__device__ inline float weight(float g, float a) {
  if constexpr (GATE == NONE) return 1.f;
  constexpr float K = GATE == NORM ? 2.f : 1.f;
  float s = -K * K * K * K * K * K * K / 5040;
  s = s * g - K * K * K * K * K * K / 720;
  s = s * g - K * K * K * K * K / 120;
  s = s * g - K * K * K * K / 24;
  s = s * g - K * K * K / 6;
  s = s * g - K * K / 2;
  s = s * g - K;
  s *= g;
  const float direct = GATE == NORM ? 1.f - a * a : 1.f - a;
  const float v = fabsf(g) < 0.35f / K ? s : direct;
  return GATE == NORM ? __builtin_amdgcn_sqrtf(fmaxf(v, 0.f)) : v;
}

// dw/dg
template <int GATE>
__device__ inline float slope(float a, float w) {
  if constexpr (GATE == NONE) return 0.f;
  if constexpr (GATE == COMPLEMENT) return -a;
  return w > 0.f ? -a * a * __builtin_amdgcn_rcpf(w) : 0.f;
}

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

#ifndef GLR_WG
#define GLR_WG 256
#endif
#ifndef GLR_LPR
#define GLR_LPR 16
#endif
constexpr int WG = GLR_WG, LPR = GLR_LPR, NG = WG / LPR, CC = 4 * LPR;  // lanes per row, groups, channels of a tile
#ifndef GLR_TF
#define GLR_TF 16
#endif
#ifndef GLR_OF
#define GLR_OF 2
#endif
#ifndef GLR_OB
#define GLR_OB 2
#endif
#ifndef GLR_TB
#define GLR_TB 8
#endif
constexpr int TPL_FWD = GLR_TF, TPL_BWD = GLR_TB;                        // tokens per lane
constexpr int BATCH = 8, POLLS = 1 << 20;
static_assert(NG * TPL_FWD % GLR_CHUNK == 0 && NG * TPL_BWD % GLR_CHUNK == 0, "a tile starts at a kept state");
static_assert(GLR_CHUNK % TPL_FWD == 0 && GLR_CHUNK % TPL_BWD == 0, "kept states fall between groups");

// What the tiles of one call publish: per tile and channel its map and the state behind it; per chain a
// row of words, its counter and how far each tile is.
struct Chain {
  uint64_t* map;    // [B, tiles, D]: A in the low half, H in the high one
  uint32_t* state;  // [B, tiles, D]
  uint32_t* flag;   // [B * blocks, row]: the counter, then a word per tile
  int tiles;        // per sequence
  int row;
};
enum : uint32_t { HAS_MAP = 1, HAS_STATE = 2 };

__device__ inline unsigned plain_nan(float x) { return x != x ? (bits(x) & 0x80000000u) | 0x7fc00000u : bits(x); }
template <typename T>
__device__ inline void publish(T* p, T v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <typename T>
__device__ inline T look(const T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// The state this tile starts from, for the channel of this lane (of a whole wavefront; `live`: the
// channel exists), publishing the tile's map and the state behind it.  at: the tile's word; flag: the
// tile's flag.
__device__ inline float chain_state(const Chain& c, long at, long stride, uint32_t* flag, int tile, bool live, float A,
                                    float H, float init) {
  if (c.tiles == 1) return init;
  const int lane = threadIdx.x % WAVE;
  float h = init;
  if (tile > 0) {
    if (live) publish(c.map + at, (uint64_t)plain_nan(H) << 32 | plain_nan(A));
    if (lane == 0) publish(flag, (uint32_t)HAS_MAP);
    int polls = 0, found = -1;
    for (; polls < POLLS; ++polls) {
      const uint32_t f = lane < tile ? look(flag - 1 - lane) : 0;
      const uint64_t states = __ballot(f == HAS_STATE), maps = __ballot(f == HAS_STATE || f == HAS_MAP);
      if (states) {
        const int k = __builtin_ctzll(states);
        if ((~maps & ((1ull << k) - 1)) == 0) {
          found = k;
          break;
        }
      }
      __builtin_amdgcn_s_sleep(1);
    }
    // the state and the maps behind it, the farthest first, BATCH at a time
    for (int k0 = found - 1; found >= 0; k0 -= BATCH) {
      uint64_t m[BATCH];
      uint32_t first = 0;
      for (; polls < POLLS; ++polls) {
        if (live && k0 == found - 1) first = look(c.state + at - (found + 1) * stride);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) m[i] = live && i <= k0 ? look(c.map + at - (k0 - i + 1) * stride) : 0;
        bool there = first != ~0u;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) there = there && m[i] != ~0ull;
        if (__all(there)) break;
      }
      if (k0 == found - 1) h = from_bits(first);
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (i <= k0) h = step(from_bits((unsigned)m[i]), h, from_bits((unsigned)(m[i] >> 32)));
      if (k0 < BATCH) break;
    }
    if (polls >= POLLS) h = __builtin_nanf("");
  }
  if (tile + 1 < c.tiles) {
    if (live) publish(c.state + at, plain_nan(step(A, h, H)));
    if (lane == 0) publish(flag, (uint32_t)HAS_STATE);
  }
  return h;
}

__global__ __launch_bounds__(256) void glr_clear_kernel(u32x4* p, long n) {
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) p[i] = u32x4{~0u, ~0u, ~0u, ~0u};
}

// Where a lane's tokens are: `tile` (uniform) points at the tile's first token and channel of a
// [B, L, D] tensor, the lane's token j at element off + j D from there.  With the token's part in the
// uniform pointer the address costs a lane nothing.  Offsets stay within 32 bits: TT * D < 2^28.
struct Where {
  unsigned off;   // of the lane's first token (of an existing channel)
  int first;      // that token's place in the tile
  int left;       // tokens of the sequence from the tile's first one on; all of the tile's or fewer
  bool inside;    // all (uniform)
  int stride;     // D
};
template <typename E>
__device__ inline E* at_byte(E* p, unsigned off) {
  return reinterpret_cast<E*>(reinterpret_cast<uintptr_t>(p) + off);
}
// A lane's TPL tokens; past the end 0, the identity (g = 0, x = 0).
template <int TPL, typename E>
__device__ inline void load_tokens(const E* tile, const Where& w, float (*v)[4]) {
  if (w.inside) {
#pragma unroll
    for (int j = 0; j < TPL; ++j) load4(at_byte(tile + (long)j * w.stride, w.off * (unsigned)sizeof(E)), v[j]);
  } else if (w.left <= 0) {  // L = 0: there is no token to read
#pragma unroll
    for (int j = 0; j < TPL; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = 0.f;
  } else {
    const unsigned lane = w.off - (unsigned)w.first * w.stride;
#pragma unroll
    for (int j = 0; j < TPL; ++j) {
      const int t = w.first + j;
      load4(at_byte(tile, (lane + (unsigned)(t < w.left ? t : w.left - 1) * w.stride) * (unsigned)sizeof(E)), v[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = t < w.left ? v[j][e] : 0.f;
    }
  }
}

// Which tile a workgroup takes: the chain by its number, so that workgroups started one after another
// read along the rows, shifted by one from row to row, so that an XCD (every eighth workgroup) is not
// always at the same channels; in the chain the next one.
struct Tile {
  int b, order, c0;  // sequence, place in its chain, first channel
  uint32_t* flag;    // the tile's
  bool none;         // no such tile: a counter that another call moved
  __device__ inline Tile(const GlrParams& p, const Chain& c) {
    const unsigned nblk = (p.D + CC - 1) / CC, chains = nblk * p.B;
    const unsigned round = blockIdx.x / chains, chain = (blockIdx.x + round) % chains;
    order = 0;
    uint32_t* row = c.flag + (long)chain * c.row;
    if (c.tiles > 1) {
      __shared__ unsigned next;
      if (threadIdx.x == 0) next = __hip_atomic_fetch_add(row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
      __syncthreads();
      order = __builtin_amdgcn_readfirstlane(next);
    }
    flag = row + 1 + order;
    none = order < 0 || order >= c.tiles;
    b = chain / nblk;
    c0 = (int)(chain % nblk) * CC;
  }
};

// a <- the gates' factors; whether one of the wavefront's is 0
template <int TPL, int GATE>
__device__ inline bool factors(float (*a)[4], float (*w)[4]) {
  float m = 1.f;
#pragma unroll
  for (int j = 0; j < TPL; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float g = a[j][e];
      a[j][e] = factor(g);
      m = fminf(m, a[j][e]);
      w[j][e] = weight<GATE>(g, a[j][e]);
    }
  return __any(m == 0.f);
}

// The group's map.
template <int TPL, bool RESETS>
__device__ inline void fwd_map(float (*a)[4], const float (*u)[4], float* A, float* H) {
  typedef Gates<RESETS> G;
#pragma unroll
  for (int e = 0; e < 4; ++e) A[e] = 1.f, H[e] = 0.f;
#pragma unroll
  for (int j = 0; j < TPL; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[j][e] = G::marked(a[j][e]);
      A[e] = G::product(A[e], a[j][e]);
      H[e] = G::next(a[j][e], H[e], u[j][e]);
    }
}

template <int TPL, bool RESETS, typename E>
__device__ inline void fwd_out(const float (*a)[4], const float (*u)[4], floatx4 h, E* out, const Where& w, int left) {
#pragma unroll
  for (int j = 0; j < TPL; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = Gates<RESETS>::next(a[j][e], h[e], u[j][e]);
    if (j < left)
      store4<E>(at_byte(out + (long)j * w.stride, w.off * (unsigned)sizeof(E)), h[0], h[1], h[2], h[3]);
  }
}

template <typename E, int GATE>
__global__ __launch_bounds__(WG, GLR_OF) void glr_fwd_kernel(GlrParams p, Chain chain) {
  constexpr int TPL = TPL_FWD, TT = NG * TPL;
  __shared__ float sA[NG][CC], sH[NG][CC];  // the groups' maps; then sH the groups' start states
  const Tile tile(p, chain);
  if (tile.none) return;
  const int tid = threadIdx.x, grp = tid / LPR, col = tid % LPR * 4;
  const int tile0 = tile.order * TT;
  const bool here = tile.c0 + col < p.D;
  const Where w{(unsigned)(grp * TPL * p.D + (here ? col : 0)), grp * TPL, p.L - tile0, tile0 + TT <= p.L, p.D};
  const long base = ((long)tile.b * p.L + tile0) * p.D + tile.c0;
  float a[TPL][4], u[TPL][4], A[4], H[4];
  load_tokens<TPL>(p.g + base, w, a);
  load_tokens<TPL>(static_cast<const E*>(p.x) + base, w, u);
  bool resets;
  {
    float wt[TPL][4];
    resets = factors<TPL, GATE>(a, wt);
#pragma unroll
    for (int j = 0; j < TPL; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) u[j][e] *= wt[j][e];
  }
  if (resets) fwd_map<TPL, true>(a, u, A, H);
  else fwd_map<TPL, false>(a, u, A, H);
  *reinterpret_cast<floatx4*>(&sA[grp][col]) = floatx4{A[0], A[1], A[2], A[3]};
  *reinterpret_cast<floatx4*>(&sH[grp][col]) = floatx4{H[0], H[1], H[2], H[3]};
  __syncthreads();
  if (tid < CC) {
    const int ch = tile.c0 + tid;
    const bool live = ch < p.D;
    float TA = 1.f, TH = 0.f;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      TH = step(sA[k][tid], TH, sH[k][tid]);
      TA = times(TA, sA[k][tid]);
    }
    float h = chain_state(chain, ((long)tile.b * chain.tiles + tile.order) * p.D + ch, p.D,
                          tile.flag, tile.order, live, TA, TH,
                          live && p.h0 ? p.h0[(long)tile.b * p.D + ch] : 0.f);
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      const float next = step(sA[k][tid], h, sH[k][tid]);
      sH[k][tid] = h;
      h = next;
    }
    if (live && p.h_final && tile.order == chain.tiles - 1) p.h_final[(long)tile.b * p.D + ch] = h;
  }
  __syncthreads();
  const int mine = w.left - w.first;  // tokens of this lane and behind
  if (!here || mine <= 0) return;
  const floatx4 h = *reinterpret_cast<const floatx4*>(&sH[grp][col]);
  if (p.states && w.first % GLR_CHUNK == 0) {
    const int nc = (p.L + GLR_CHUNK - 1) / GLR_CHUNK;
    float* to = p.states + ((long)tile.b * nc + (tile0 + w.first) / GLR_CHUNK) * p.D + tile.c0 + col;
    *reinterpret_cast<floatx4*>(to) = h;
  }
  E* out = static_cast<E*>(p.O) + base;
  const int stores = w.inside ? TPL : mine;
  if (resets) fwd_out<TPL, true>(a, u, h, out, w, stores);
  else fwd_out<TPL, false>(a, u, h, out, w, stores);
}

// The same from the other end.  With flow_t = a_t lambda_t, the gradient that reaches the state
// before token t, flow_t = a_t (dO_t + flow_{t+1}): an affine recurrence over the same gates, tiles
// handed out from the last to the first.  A group's start state comes from the kept state of its
// 64 tokens and the maps of the groups between.
template <int TPL, bool RESETS>
__device__ inline void bwd_map(float (*a)[4], const float (*w)[4], const float (*x)[4], const float (*d)[4], float* A,
                               float* H, float* F) {
  typedef Gates<RESETS> G;
#pragma unroll
  for (int e = 0; e < 4; ++e) A[e] = 1.f, H[e] = F[e] = 0.f;
#pragma unroll
  for (int j = 0; j < TPL; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[j][e] = G::marked(a[j][e]);
      A[e] = G::product(A[e], a[j][e]);
      H[e] = G::next(a[j][e], H[e], w[j][e] * x[j][e]);
    }
#pragma unroll
  for (int j = TPL - 1; j >= 0; --j)
#pragma unroll
    for (int e = 0; e < 4; ++e) F[e] = G::pass(a[j][e], a[j][e] * (d[j][e] + F[e]));
}

template <int TPL, int GATE, bool RESETS>
__device__ inline void bwd_out(const float (*a)[4], const float (*w)[4], float (*x)[4], const float (*d)[4], floatx4 h,
                               floatx4 flow, float* dx, float* dg, const Where& at, int left) {
  typedef Gates<RESETS> G;
#pragma unroll
  for (int j = 0; j < TPL; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // x becomes dh_t / dg_t
      const float u = w[j][e] * x[j][e], ah = a[j][e] * h[e];
      x[j][e] = G::pass(a[j][e], ah + slope<GATE>(a[j][e], w[j][e]) * x[j][e]);
      h[e] = G::pass(a[j][e], ah) + u;
    }
#pragma unroll
  for (int j = TPL - 1; j >= 0; --j) {
    floatx4 px, pg;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lam = d[j][e] + flow[e];
      px[e] = w[j][e] * lam;
      pg[e] = G::pass(a[j][e], lam * x[j][e]);
      flow[e] = G::pass(a[j][e], a[j][e] * lam);
    }
    if (j < left) {
      *reinterpret_cast<floatx4*>(at_byte(dx + (long)j * at.stride, at.off * 4u)) = px;
      *reinterpret_cast<floatx4*>(at_byte(dg + (long)j * at.stride, at.off * 4u)) = pg;
    }
  }
}

template <typename E, int GATE>
__global__ __launch_bounds__(WG, GLR_OB) void glr_bwd_kernel(GlrParams p, Chain chain) {
  constexpr int TPL = TPL_BWD, TT = NG * TPL, GPC = GLR_CHUNK / TPL;  // groups per kept state
  __shared__ float sA[NG][CC], sH[NG][CC], sF[NG][CC];
  const Tile tile(p, chain);
  if (tile.none) return;
  const int tid = threadIdx.x, grp = tid / LPR, col = tid % LPR * 4;
  const int tile0 = (chain.tiles - 1 - tile.order) * TT;
  const bool here = tile.c0 + col < p.D;
  const Where at{(unsigned)(grp * TPL * p.D + (here ? col : 0)), grp * TPL, p.L - tile0, tile0 + TT <= p.L, p.D};
  const long base = ((long)tile.b * p.L + tile0) * p.D + tile.c0;
  float a[TPL][4], w[TPL][4], x[TPL][4], d[TPL][4], A[4], H[4], F[4];
  load_tokens<TPL>(p.g + base, at, a);
  load_tokens<TPL>(static_cast<const E*>(p.x) + base, at, x);
  load_tokens<TPL>(static_cast<const E*>(p.dO) + base, at, d);
  const bool resets = factors<TPL, GATE>(a, w);
  if (resets) bwd_map<TPL, true>(a, w, x, d, A, H, F);
  else bwd_map<TPL, false>(a, w, x, d, A, H, F);
  *reinterpret_cast<floatx4*>(&sA[grp][col]) = floatx4{A[0], A[1], A[2], A[3]};
  *reinterpret_cast<floatx4*>(&sH[grp][col]) = floatx4{H[0], H[1], H[2], H[3]};
  *reinterpret_cast<floatx4*>(&sF[grp][col]) = floatx4{F[0], F[1], F[2], F[3]};
  __syncthreads();
  if (tid < CC) {
    const int ch = tile.c0 + tid, nc = (p.L + GLR_CHUNK - 1) / GLR_CHUNK;
    const bool live = ch < p.D;
    float start[NG / GPC];
#pragma unroll
    for (int n = 0; n < NG / GPC; ++n) {
      const int chunk = tile0 / GLR_CHUNK + n;
      start[n] = live && chunk < nc ? p.states[((long)tile.b * nc + chunk) * p.D + ch] : 0.f;
    }
    float TA = 1.f, TF = 0.f;
#pragma unroll
    for (int k = NG - 1; k >= 0; --k) {
      TF = step(sA[k][tid], TF, sF[k][tid]);
      TA = times(TA, sA[k][tid]);
    }
    float flow = chain_state(chain, ((long)tile.b * chain.tiles + tile.order) * p.D + ch, p.D,
                             tile.flag, tile.order, live, TA, TF,
                             live && p.dh_final ? p.dh_final[(long)tile.b * p.D + ch] : 0.f);
#pragma unroll
    for (int k = NG - 1; k >= 0; --k) {
      const float next = step(sA[k][tid], flow, sF[k][tid]);
      sF[k][tid] = flow;
      flow = next;
    }
    if (live && p.dh0 && tile.order == chain.tiles - 1) p.dh0[(long)tile.b * p.D + ch] = flow;
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
  const int mine = at.left - at.first;
  if (!here || mine <= 0) return;
  const floatx4 h = *reinterpret_cast<const floatx4*>(&sH[grp][col]), flow = *reinterpret_cast<const floatx4*>(&sF[grp][col]);
  const int stores = at.inside ? TPL : mine;
  if (resets) bwd_out<TPL, GATE, true>(a, w, x, d, h, flow, p.dx + base, p.dg + base, at, stores);
  else bwd_out<TPL, GATE, false>(a, w, x, d, h, flow, p.dx + base, p.dg + base, at, stores);
}

template <typename E, int GATE>
__global__ __launch_bounds__(256) void glr_decode_kernel(GlrParams p) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long)p.B * p.D) return;
  const float g = p.g[i], a = mark(factor(g));
  const float h = step(a, p.h_final[i], weight<GATE>(g, a) * to_float(static_cast<const E*>(p.x)[i]));
  p.h_final[i] = h;
  static_cast<E*>(p.O)[i] = to_elem<E>(h);
}

enum Which { FWD, BWD, DECODE };

int tile_tokens(Which which) { return NG * (which == FWD ? TPL_FWD : TPL_BWD); }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

int flag_row(int tiles) { return (tiles + 1 + 31) / 32 * 32; }  // whole 128-byte lines

// Byte offsets of the chain's arrays in the workspace.
struct Layout {
  size_t state, flag, total;
};
Layout layout(int B, int tiles, int D) {
  const size_t n = (size_t)B * tiles * D, blocks = (D + CC - 1) / CC;
  Layout l;
  l.state = up256(n * 8);
  l.flag = l.state + up256(n * 4);
  l.total = l.flag + up256((size_t)B * blocks * flag_row(tiles) * 4);
  return l;
}

template <typename E, int GATE>
hipError_t launch_one(const GlrParams& p, Which which, hipStream_t st) {
  if (which == DECODE) {
    const long n = (long)p.B * p.D;
    hipLaunchKernelGGL((glr_decode_kernel<E, GATE>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, p);
    return hipGetLastError();
  }
  const int TT = tile_tokens(which);
  Chain c{nullptr, nullptr, nullptr, p.L > TT ? (p.L + TT - 1) / TT : 1, 0};
  if (c.tiles > 1) {
    const Layout l = layout(p.B, c.tiles, p.D);
    char* ws = static_cast<char*>(p.ws);
    c.map = reinterpret_cast<uint64_t*>(ws);
    c.state = reinterpret_cast<uint32_t*>(ws + l.state);
    c.flag = reinterpret_cast<uint32_t*>(ws + l.flag);
    c.row = flag_row(c.tiles);
    const long v = (long)(l.total / 16), wgs = (v + 255) / 256;
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
  return L > TT && B > 0 && D > 0 ? layout(B, (L + TT - 1) / TT, D).total : 0;
}
bool glr_grid_fits(int B, int L, int D) {
  return (double)((D + CC - 1) / CC) * B * ((L + (double)NG * TPL_BWD - 1) / (NG * TPL_BWD)) < 0x1p31;
}

hipError_t launch_glr_fwd(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, FWD, st); }
hipError_t launch_glr_bwd(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, BWD, st); }
hipError_t launch_glr_decode(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, DECODE, st); }

}  // namespace delta
