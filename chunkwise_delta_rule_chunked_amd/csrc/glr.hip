// Gated linear recurrence: per channel h_t = a_t h_{t-1} + w_t x_t with a = exp(g), its gradients
// and its one-token step (include/delta_block.h).
//
// A hard reset (a = 0) drops the previous state by selection rather than by multiplication, so that
// nothing of it, NaN and infinities included, is seen after it; the same holds for the gradient that flows
// back.  State, gates and sums are float32.
//
// Bytes bound these kernels (an exp and 20 to 30 other instructions per element take half as long at full
// issue), so the sequence kernels read each input once and write each output once, in one pass.  A workgroup
// takes a tile of 128 (backward 64) tokens x 64 channels: 16 groups of 16 lanes, a group 8 (4) consecutive
// tokens, a lane 4 channels.  The tile's gates and inputs stay in registers while its place in the sequence is
// found:
//   1. each lane reduces its tokens to the affine map of the state (A, H): h -> A h + H;
//   2. one wavefront, a lane per channel, folds the 16 groups' maps into the tile's, publishes it,
//      waits for a predecessor's state (below) and publishes the state behind the tile;
//   3. each group runs its tokens again from its start state, writing outputs.
// Tiles of one channel block and sequence form a chain (a scan with decoupled look-back).  A tile's
// predecessors publish their map as soon as they have read their tokens and the state behind them as soon as
// they know it; a tile starts from the nearest state it finds among its 64 predecessors and folds in the maps
// between.
// The fold is the same left fold whichever state it starts from, so the result does not depend on
// timing.  Waiting reads one flag per predecessor (a lane each, a cache line in all).  A flag is only a
// hint: a published word carries its own readiness, since the workspace starts as all ones, a NaN that
// no published value has, so no fence orders data and flag.  A counter per chain hands out its tiles in
// order: whoever a tile waits for has started before it and waits for nobody behind it, so every
// wait ends (and is bounded besides: past POLLS polls, as can only happen if two calls share a
// workspace, the tile goes on with NaN).
//
// Measured, 2048 channels, time on the card, bf16: 512 sequences of 128 tokens (no chain) 182 us, 5.9 TB/s; one of
// 64K tokens 205 us, 5.2 TB/s: clearing the workspace (6 us) and waiting along the chain cost the rest; backward
// 256 x 64 tokens (no chain) 96 us, 5.7 TB/s, 2 x 8K tokens 114 us, 4.7 TB/s.  float32, 2 x 8K: forward 82 us,
// 4.9 TB/s, backward 130 us, 5.2 TB/s.  HBM traffic is what the formulas need plus 7% (forward) and 6%.
// Tried and slower: workgroups that stay and load their next tile while they wait (its map is published a
// tile too late: 288 us); one counter for all chains (6 us more at the start of every call); a workgroup per
// narrow channel block that walks the whole sequence (its scans across lanes: 23 us for 4 x 2K x 1024
// channels, and 4096 tokens 345 us for 16 sequences, against 20 and 218).
//
#include <hip/hip_runtime.h>

#include "block_kernels.h"
#include "common.h"

namespace delta {
namespace {

enum { NONE = 0, COMPLEMENT = 1, NORM = 2 };

__device__ inline unsigned bits(float x) { return __builtin_bit_cast(unsigned, x); }
__device__ inline float from_bits(unsigned x) { return __builtin_bit_cast(float, x); }

// a = exp(g), as 2 to a rounded product: good to (2 + 2|g|) half steps of float32; subnormal results are 0.
// a = 0 (g = -inf, or an exp that underflows) is the hard reset.  Where a product of gates
// could underflow too, the sign bit, which no exp has (a NaN loses it here), marks a reset: products
// carry the mark along.
__device__ inline float factor(float g) { return fabsf(gate_exp(g)); }
__device__ inline float mark(float a) { return a == 0.f ? -0.f : a; }
__device__ inline bool reset(float a) { return (int)bits(a) < 0; }
__device__ inline float times(float a, float b) {
  return from_bits((bits(a * b) & 0x7fffffffu) | ((bits(a) | bits(b)) & 0x80000000u));
}
__device__ inline float step(float a, float h, float u) { return reset(a) ? u : __builtin_fmaf(a, h, u); }

// Gates above 1.  With factors up to GROWS the products of a tile's 128 stay below 2^75.  With larger ones a
// product can leave float32's range where no state does (a small or zero state, or decay behind it).  A map's
// factor of 2^127 or more is then held as minus its value times 2^-192; 2^319 stands for all above, where any state
// but 0 overflows.  Products are formed in 64 bits.  Ordinary factors give the same bits either way, so it does not
// matter to which of a chain's folds such a factor came too.  What this costs calls without such gates: 0.2 us of
// 10.7 on 3 x 1237 x 240, nothing that shows on 64K tokens.
constexpr float GROWS = 1.5f;
__device__ inline double whole(float a) { return a < 0.f ? -0x1p192 * a : a; }
__device__ inline float factor_of(double d) {
  if (d >= 0x1p127) return -(float)(d < 0x1p319 ? d * 0x1p-192 : 0x1p127);
  return d != d ? __builtin_nanf("") : (float)d;
}
template <bool GROWN>
struct Maps {
  __device__ static inline float product(float a, float b) {
    if constexpr (!GROWN) return times(a, b);
    return (a == 0.f && reset(a)) || (b == 0.f && reset(b)) ? -0.f : factor_of(whole(a) * whole(b));
  }
  __device__ static inline float next(float a, float h, float u) {
    if constexpr (!GROWN) return step(a, h, u);
    return a < 0.f ? (float)__builtin_fma(whole(a), (double)h, (double)u) : step(a, h, u);
  }
};

// The same for the tokens a lane holds.  RESETS: whether a reset, or a factor above GROWS, is among the
// wavefront's; without one (nearly always) the marks cost nothing.  Both round alike (the multiply-adds are
// written out), so a channel's bits do not depend on its neighbours.
template <bool RESETS>
struct Gates {
  __device__ static inline float marked(float a) { return RESETS ? mark(a) : a; }
  __device__ static inline float next(float a, float h, float u) { return RESETS ? step(a, h, u) : __builtin_fmaf(a, h, u); }
  // the product of a channel's factors; in 64 bits if one of them (whatever other channels have) is above GROWS
  struct Product {
    float v = 1.f;
    double v64 = 1.;
    bool forgets = false, grows = false;
    __device__ inline void by(float a) {
      v *= a;
      if constexpr (RESETS) {
        forgets = forgets || reset(a);
        grows = grows || a > GROWS;
        v64 *= a;
        if (v64 > 0x1p400) v64 = 0x1p400;
      }
    }
    __device__ inline float get() const { return forgets ? -0.f : grows ? factor_of(v64) : v; }
  };
  // what multiplies into a gradient: nothing at a reset, whatever v is
  __device__ static inline float pass(float a, float v) { return RESETS && reset(a) ? 0.f : v; }
};

// w(g), from a = exp(g).  1 - a and 1 - a^2 cancel near g = 0, where a series takes over.  For 1 - a it is
// that of 1 - exp(g) to g^7 (|g| < 0.35: the first dropped term is below 0.35^7 / 8! = 2e-8 of the result);
// for 1 - a^2 = -2 a sinh(g) that of sinh, two terms shorter (|g| < 0.25: 0.25^6 / 7! = 5e-8).  Beyond,
// the difference is good to a dozen units of 2^-24.  Root and reciprocal (in dw/dg) are the hardware's, good to a
// unit in the last place.
template <int GATE>
__device__ inline float weight(float g, float a) {
  if constexpr (GATE == NONE) {
    return 1.f;
  } else if constexpr (GATE == COMPLEMENT) {
    float s = -1.f / 5040;
    s = s * g - 1.f / 720;
    s = s * g - 1.f / 120;
    s = s * g - 1.f / 24;
    s = s * g - 1.f / 6;
    s = s * g - 1.f / 2;
    s = s * g - 1.f;
    return fabsf(g) < 0.35f ? s * g : 1.f - a;
  } else {
    const float t = g * g, s = (t * (t * (-2.f / 120) - 2.f / 6) - 2.f) * (g * a);
    const float v = fabsf(g) < 0.25f ? s : 1.f - a * a;
    return __builtin_amdgcn_sqrtf(__builtin_elementwise_maximum(v, 0.f));  // a NaN gate's is NaN, as fmaxf's is not
  }
}

// dw/dg
template <int GATE>
__device__ inline float slope(float a, float w) {
  if constexpr (GATE == NONE) return 0.f;
  if constexpr (GATE == COMPLEMENT) return -a;
  return w == 0.f ? 0.f : -a * a * __builtin_amdgcn_rcpf(w);
}

// Four consecutive channels as they are in memory.
template <typename E>
struct Raw;
template <>
struct Raw<float> {
  typedef floatx4 type;
};
template <>
struct Raw<bf16> {
  typedef u32x2 type;
};
template <typename E>
using raw4 = typename Raw<E>::type;
__device__ inline void unpack4(floatx4 r, float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = r[e];
}
__device__ inline void unpack4(u32x2 r, float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = from_bits(e % 2 ? r[e / 2] & 0xffff0000u : r[e / 2] << 16);
}

constexpr int WG = 256, LPR = 16, NG = WG / LPR, CC = 4 * LPR;  // lanes per row, groups, channels of a tile
// Tokens of a lane.  Fewer leave registers for more wavefronts, more make fewer and shorter chains.
// Measured on one 64K x 2048 sequence (forward) and 2 x 8K x 2048 (backward), us: forward 4: 263, 8: 206,
// 16: 228; backward 4: 113.5, 8: 119.  Forward with clearing, 4 x 2K x 1024: 27.4, 20.1 and 21.7; 32 x 512 x 2048:
// 63.6, 55.8 and 60.5; 3 x 1237 x 240 in float32: 11.4, 10.7 and 12.4.  A sequence of up to 64 tokens is one tile of
// TPL_SHORT tokens a lane with none left over (256 x 64 x 2048: 47.5 us, 64 with 8).
constexpr int TPL_FWD = 8, TPL_BWD = 4, TPL_SHORT = 4;
constexpr int BATCH = 8, POLLS = 1 << 20;
static_assert(NG * TPL_FWD % GLR_CHUNK == 0 && NG * TPL_BWD % GLR_CHUNK == 0, "a tile starts at a kept state");
static_assert(GLR_CHUNK % TPL_FWD == 0 && GLR_CHUNK % TPL_BWD == 0, "kept states fall between groups");

// What the tiles of one call publish: a word per tile and channel, first its map, then the state behind
// it, as the map that forgets what was before (a reset): a reader that expects the one and finds the other
// folds it in all the same.  Per chain a row of words: its counter and how far each tile is.
struct Chain {
  uint64_t* map;   // [B, tiles, D]: A in the low half, H in the high one
  uint32_t* flag;  // [B * blocks, row]: the counter, then a word per tile
  int tiles;       // per sequence
  int row;
};
enum : uint32_t { HAS_MAP = 1, HAS_STATE = 2, HAS_GROWN_MAP = 3 };  // grown: with factors that Maps<true> takes

__device__ inline unsigned plain_nan(float x) { return x != x ? (bits(x) & 0x80000000u) | 0x7fc00000u : bits(x); }
template <typename T>
__device__ inline void publish(T* p, T v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <typename T>
__device__ inline T look(const T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

__device__ inline uint64_t map_word(float A, float H) { return (uint64_t)plain_nan(H) << 32 | plain_nan(A); }

template <bool GROWN>
__device__ inline float fold_words(const uint64_t* m, int last, float h) {
#pragma unroll
  for (int i = 0; i < BATCH; ++i)
    if (i <= last) h = Maps<GROWN>::next(from_bits((unsigned)m[i]), h, from_bits((unsigned)(m[i] >> 32)));
  return h;
}

// The state this tile starts from, for the channel of this lane (of a whole wavefront; `live`: the
// channel exists), publishing the tile's map and the state behind it.  grown: a factor of the tile is above
// GROWS.  at: the tile's word; flag: the tile's flag.  init: the first tile's start state, which no other tile may
// read: where h_final is h0, the chain's last tile writes over it.
__device__ inline float chain_state(const Chain& c, long at, long stride, uint32_t* flag, int tile, bool live, bool grown,
                                    float A, float H, float init) {
  if (c.tiles == 1) return init;
  const int lane = threadIdx.x % WAVE;
  float h = init;
  if (tile > 0) {
    if (live) publish(c.map + at, map_word(A, H));
    if (lane == 0) publish(flag, (uint32_t)(grown ? HAS_GROWN_MAP : HAS_MAP));
    int polls = 0, found = -1;  // the nearest predecessor (0: the one before) with a state, and maps behind it
    bool any_grown = false;     // among those maps
    for (; polls < POLLS; ++polls) {
      const uint32_t f = lane < tile ? look(flag - 1 - lane) : 0;
      const uint64_t states = __ballot(f == HAS_STATE), words = __ballot(f - 1u < 3u);
      if (states) {
        const int k = __builtin_ctzll(states);
        if ((~words & ((1ull << k) - 1)) == 0) {
          any_grown = __ballot(f == HAS_GROWN_MAP) & ((1ull << k) - 1);
          found = k;
          break;
        }
      }
      __builtin_amdgcn_s_sleep(1);
    }
    // from the farthest on, BATCH at a time
    for (int k0 = found; k0 >= 0; k0 -= BATCH) {
      uint64_t m[BATCH];
      for (; polls < POLLS; ++polls) {
        bool there = true;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) m[i] = live && i <= k0 ? look(c.map + at - (k0 - i + 1) * stride) : 0;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) there = there && m[i] != ~0ull;
        // the flag may be seen before the state: what the fold starts from has to forget what was before
        if (k0 == found) there = there && (!live || (unsigned)m[0] == 0x80000000u);
        if (__all(there)) break;
      }
      if (__builtin_expect(any_grown, 0)) h = fold_words<true>(m, k0, h);
      else h = fold_words<false>(m, k0, h);
    }
    if (polls >= POLLS) h = __builtin_nanf("");
  }
  if (tile + 1 < c.tiles) {
    if (live) publish(c.map + at, map_word(-0.f, __builtin_expect(grown, 0) ? Maps<true>::next(A, h, H) : step(A, h, H)));
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
// A lane's TPL tokens; past the end 0, the identity (g = 0, x = 0).  (A tile has one token at least.)
template <int TPL, typename E>
__device__ inline void load_tokens(const E* tile, const Where& w, raw4<E>* v) {
  if (w.inside) {
#pragma unroll
    for (int j = 0; j < TPL; ++j)
      v[j] = __builtin_nontemporal_load(
          reinterpret_cast<const raw4<E>*>(at_byte(tile + (long)j * w.stride, w.off * (unsigned)sizeof(E))));
  } else {
    const unsigned lane = w.off - (unsigned)w.first * w.stride;
#pragma unroll
    for (int j = 0; j < TPL; ++j) {
      const int t = w.first + j < w.left ? w.first + j : w.left - 1;
      v[j] = *reinterpret_cast<const raw4<E>*>(at_byte(tile, (lane + (unsigned)t * w.stride) * (unsigned)sizeof(E)));
      if (w.first + j >= w.left) v[j] = raw4<E>{};
    }
  }
}
// What follows unpacks a token again rather than holding its floats (twice the registers) until then.
__device__ inline void again(u32x2& r) { asm volatile("" : "+v"(r)); }
__device__ inline void again(floatx4&) {}
// Ends a stretch of a few tokens: left to itself the compiler works on all of them at once, in more
// registers than there are.
__device__ inline void stretch(int j, int tokens) {
  if (j % tokens == tokens - 1) __builtin_amdgcn_sched_barrier(0);
}

// Workgroup k takes a tile of the chain that its number names; in its chain it takes the next one.  One
// sequence after the other (rows of many sequences at once would often be the same power of two apart and
// meet in the same memory channels), along the rows of each, shifted by one block from row to row, so that
// an XCD (every eighth workgroup) is not always at the same channels.
struct Jobs {
  unsigned nblk, per;  // channel blocks; tiles of a sequence
  __device__ inline Jobs(const GlrParams& p, const Chain& c) : nblk((p.D + CC - 1) / CC), per(nblk * c.tiles) {}
  __device__ inline unsigned chain(unsigned job) const {
    const unsigned in = job % per;
    return job / per * nblk + (in + in / nblk) % nblk;
  }
};
// The next tile of a chain, for one lane.
__device__ inline int take_tile(const Chain& c, unsigned chain) {
  if (c.tiles == 1) return 0;
  return (int)(__hip_atomic_fetch_add(c.flag + (long)chain * c.row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u);
}

// One tile as a lane sees it.
template <int TPL>
struct Tile {
  int b, order, c0, tile0;  // sequence, place in its chain, first channel and token
  unsigned chain;
  bool none;                // no such tile: the counter was moved by another call
  Where w;
  long base;                // of the tile's first token and channel
  __device__ inline void set(const GlrParams& p, const Chain& c, const Jobs& jobs, unsigned job, int taken, bool backward) {
    constexpr int TT = NG * TPL;
    chain = jobs.chain(job);
    order = taken;
    none = order < 0 || order >= c.tiles;
    if (none) order = 0;
    b = chain / jobs.nblk;
    c0 = (int)(chain % jobs.nblk) * CC;
    tile0 = (backward ? c.tiles - 1 - order : order) * TT;
    const int grp = threadIdx.x / LPR, col = threadIdx.x % LPR * 4;
    w = Where{(unsigned)(grp * TPL * p.D + (c0 + col < p.D ? col : 0)), grp * TPL, p.L - tile0, tile0 + TT <= p.L, p.D};
    base = ((long)b * p.L + tile0) * p.D + c0;
  }
};

// a <- the gates' factors, w <- their weights (FOLD: times the inputs); whether one of the wavefront's
// factors is a reset or above GROWS, and the lane's largest.  PIN: the weights are made here and now; left to itself the compiler
// holds what their roots are made from for many tokens (172 registers for 115).
struct Seen {
  bool special;
  float most;
};
template <int TPL, int GATE, bool FOLD, bool PIN = false, typename R>
__device__ inline Seen weigh(const floatx4* rg, const R* rx, float (*a)[4], float (*w)[4]) {
  float least = 1.f, most = 1.f;
#pragma unroll
  for (int j = 0; j < TPL; ++j) {
    float g[4], x[4];
    unpack4(rg[j], g);
    if (FOLD) unpack4(rx[j], x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[j][e] = factor(g[e]);
      least = fminf(least, a[j][e]);
      most = fmaxf(most, a[j][e]);
      w[j][e] = weight<GATE>(g[e], a[j][e]);
      if (FOLD) w[j][e] *= x[e];
      if (PIN) asm volatile("" : "+v"(w[j][e]));
    }
    stretch(j, 2);
  }
  return {(bool)__any(least == 0.f || most > GROWS), most};
}

// The groups' maps of a channel, from the first to the last (BACK: from the last to the first): the tile's, and the
// state each group starts from in the place of its H; what is behind the last comes back.
template <bool GROWN, bool BACK>
__device__ inline void fold_groups(const float (*sA)[CC], const float (*sH)[CC], int ch, float& A, float& H) {
  constexpr int UNROLL = GROWN ? 1 : NG;
  A = 1.f, H = 0.f;
#pragma unroll UNROLL
  for (int i = 0; i < NG; ++i) {
    const int k = BACK ? NG - 1 - i : i;
    H = Maps<GROWN>::next(sA[k][ch], H, sH[k][ch]);
    A = Maps<GROWN>::product(A, sA[k][ch]);
    stretch(i, 4);
  }
  if constexpr (!GROWN) A = reset(A) ? -0.f : A;
}
template <bool GROWN, bool BACK, int GROUPS>
__device__ inline float start_groups(const float (*sA)[CC], float (*sH)[CC], int ch, int first, float h) {
  constexpr int UNROLL = GROWN ? 1 : GROUPS;
#pragma unroll UNROLL
  for (int i = 0; i < GROUPS; ++i) {
    const int k = BACK ? first + GROUPS - 1 - i : first + i;
    const float behind = Maps<GROWN>::next(sA[k][ch], h, sH[k][ch]);
    sH[k][ch] = h;
    h = behind;
    stretch(i, 4);
  }
  return h;
}

// The group's map.
template <int TPL, bool RESETS>
__device__ inline void fwd_map(float (*a)[4], const float (*u)[4], float* A, float* H) {
  typedef Gates<RESETS> G;
  typename G::Product P[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) H[e] = 0.f;
#pragma unroll
  for (int j = 0; j < TPL; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[j][e] = G::marked(a[j][e]);
      P[e].by(a[j][e]);
      H[e] = G::next(a[j][e], H[e], u[j][e]);
    }
#pragma unroll
  for (int e = 0; e < 4; ++e) A[e] = P[e].get();
}

// Outputs are stored non-temporally (as the inputs are loaded), so that what streams through does not push
// out the chain's words: 4 x 2K x 1024 forward 20.1 us against 21.6 with ordinary stores, 512 x 32 x 2048 backward
// 116 against 126, one 64K sequence the same.  The other way round are 512 x 128 x 2048 forward, 184 against 179,
// and backward 2 x 8K, 113.5 against 110.
template <typename E>
__device__ inline void store_out(E* p, floatx4 h) {
  E v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = to_elem<E>(h[e]);
  raw4<E> r;
  __builtin_memcpy(&r, v, sizeof(r));
  __builtin_nontemporal_store(r, reinterpret_cast<raw4<E>*>(p));
}
__device__ inline void store_grad(float* p, floatx4 v) { __builtin_nontemporal_store(v, reinterpret_cast<floatx4*>(p)); }

template <int TPL, bool RESETS, typename E>
__device__ inline void fwd_out(const float (*a)[4], const float (*u)[4], floatx4 h, E* out, const Where& w, int left) {
#pragma unroll
  for (int j = 0; j < TPL; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = Gates<RESETS>::next(a[j][e], h[e], u[j][e]);
    if (j < left)
      store_out<E>(at_byte(out + (long)j * w.stride, w.off * (unsigned)sizeof(E)), h);
  }
}

template <typename E, int GATE, int TPL>
__global__ __launch_bounds__(WG) void glr_fwd_kernel(GlrParams p, Chain chain) {
  __shared__ float sA[NG][CC], sH[NG][CC];  // the groups' maps; then sH the groups' start states
  __shared__ int taken, grows;
  const Jobs jobs(p, chain);
  const int tid = threadIdx.x, grp = tid / LPR, col = tid % LPR * 4;
  if (tid == 0) taken = take_tile(chain, jobs.chain(blockIdx.x)), grows = 0;
  barrier_lds();
  Tile<TPL> tile;
  tile.set(p, chain, jobs, blockIdx.x, __builtin_amdgcn_readfirstlane(taken), false);
  if (tile.none) return;
  float a[TPL][4], u[TPL][4], A[4], H[4];
  Seen seen;
  {
    floatx4 rg[TPL];
    raw4<E> rx[TPL];
    load_tokens<TPL>(p.g + tile.base, tile.w, rg);
    load_tokens<TPL>(static_cast<const E*>(p.x) + tile.base, tile.w, rx);
    seen = weigh<TPL, GATE, true, GATE == NORM>(rg, rx, a, u);
  }
  if (seen.special) {
    if (seen.most > GROWS) grows = 1;
    fwd_map<TPL, true>(a, u, A, H);
  } else {
    fwd_map<TPL, false>(a, u, A, H);
  }
  *reinterpret_cast<floatx4*>(&sA[grp][col]) = floatx4{A[0], A[1], A[2], A[3]};
  *reinterpret_cast<floatx4*>(&sH[grp][col]) = floatx4{H[0], H[1], H[2], H[3]};
  barrier_lds();
  if (tid < CC) {
    const int ch = tile.c0 + tid;
    const bool live = ch < p.D;
    const bool grown = __builtin_amdgcn_readfirstlane(grows);
    float TA, TH;
    fold_groups<false, false>(sA, sH, tid, TA, TH);
    if (__builtin_expect(grown, 0)) fold_groups<true, false>(sA, sH, tid, TA, TH);
    float h = chain_state(chain, ((long)tile.b * chain.tiles + tile.order) * p.D + ch, p.D,
                          chain.flag + (long)tile.chain * chain.row + 1 + tile.order, tile.order, live, grown, TA, TH,
                          live && p.h0 && tile.order == 0 ? p.h0[(long)tile.b * p.D + ch] : 0.f);
    if (__builtin_expect(grown, 0)) h = start_groups<true, false, NG>(sA, sH, tid, 0, h);
    else h = start_groups<false, false, NG>(sA, sH, tid, 0, h);
    if (live && p.h_final && tile.order == chain.tiles - 1) p.h_final[(long)tile.b * p.D + ch] = h;
  }
  barrier_lds();
  const int have = tile.w.left - tile.w.first;  // tokens of this lane and behind
  if (tile.c0 + col >= p.D || have <= 0) return;
  const floatx4 h = *reinterpret_cast<const floatx4*>(&sH[grp][col]);
  if (p.states && tile.w.first % GLR_CHUNK == 0) {
    const int nc = (p.L + GLR_CHUNK - 1) / GLR_CHUNK;
    float* to = p.states + ((long)tile.b * nc + (tile.tile0 + tile.w.first) / GLR_CHUNK) * p.D + tile.c0 + col;
    *reinterpret_cast<floatx4*>(to) = h;
  }
  E* out = static_cast<E*>(p.O) + tile.base;
  const int stores = tile.w.inside ? TPL : have;
  if (seen.special) fwd_out<TPL, true>(a, u, h, out, tile.w, stores);
  else fwd_out<TPL, false>(a, u, h, out, tile.w, stores);
}

// The same from the other end.  With flow_t = a_t lambda_t, the gradient that reaches the state
// before token t, flow_t = a_t (dO_t + flow_{t+1}): an affine recurrence over the same gates, tiles
// handed out from the last to the first.  A group's start state comes from the kept state of its
// 64 tokens and the maps of the groups between.
template <int TPL, bool RESETS, typename R>
__device__ inline void bwd_map(float (*a)[4], const float (*w)[4], const R* rx, const R* rd, float* A, float* H,
                               float* F) {
  typedef Gates<RESETS> G;
  typename G::Product P[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) H[e] = 0.f;
#pragma unroll
  for (int j = 0; j < TPL; ++j) {
    float x[4];
    unpack4(rx[j], x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[j][e] = G::marked(a[j][e]);
      P[e].by(a[j][e]);
      H[e] = G::next(a[j][e], H[e], w[j][e] * x[e]);
    }
    stretch(j, 4);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) A[e] = P[e].get();
#pragma unroll
  for (int j = TPL - 1; j >= 0; --j) {
    float d[4];
    unpack4(rd[j], d);
#pragma unroll
    for (int e = 0; e < 4; ++e) F[e] = j == TPL - 1 ? d[e] : G::next(a[j + 1][e], F[e], d[e]);  // lambda
    stretch(j, 4);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) F[e] = G::pass(a[0][e], a[0][e] * F[e]);
}

template <int TPL, int GATE, bool RESETS, typename R>
__device__ inline void bwd_out(const float (*a)[4], const float (*w)[4], const R* rx, const R* rd, const Where& at,
                               floatx4 h, floatx4 flow, float* dx, float* dg, int left) {
  typedef Gates<RESETS> G;
  float q[TPL][4], lam[4];  // dh_t / dg_t; the gradient of h_t
#pragma unroll
  for (int j = 0; j < TPL; ++j) {
    float x[4];
    unpack4(rx[j], x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[j][e] = G::pass(a[j][e], __builtin_fmaf(slope<GATE>(a[j][e], w[j][e]), x[e], a[j][e] * h[e]));
      h[e] = G::next(a[j][e], h[e], w[j][e] * x[e]);
    }
    stretch(j, 2);
  }
#pragma unroll
  for (int j = TPL - 1; j >= 0; --j) {
    float d[4];
    unpack4(rd[j], d);
    floatx4 px, pg;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lam[e] = j == TPL - 1 ? d[e] + flow[e] : G::next(a[j + 1][e], lam[e], d[e]);
      px[e] = w[j][e] * lam[e];
      pg[e] = G::pass(a[j][e], lam[e] * q[j][e]);
    }
    if (j < left) {
      store_grad(at_byte(dx + (long)j * at.stride, at.off * 4u), px);
      store_grad(at_byte(dg + (long)j * at.stride, at.off * 4u), pg);
    }
    stretch(j, 2);
  }
}

template <typename E, int GATE>
__global__ __launch_bounds__(WG) void glr_bwd_kernel(GlrParams p, Chain chain) {
  constexpr int TPL = TPL_BWD, GPC = GLR_CHUNK / TPL;  // groups per kept state
  __shared__ float sA[NG][CC], sH[NG][CC], sF[NG][CC];
  __shared__ int taken, grows;
  const Jobs jobs(p, chain);
  const int tid = threadIdx.x, grp = tid / LPR, col = tid % LPR * 4;
  if (tid == 0) taken = take_tile(chain, jobs.chain(blockIdx.x)), grows = 0;
  barrier_lds();
  Tile<TPL> tile;
  tile.set(p, chain, jobs, blockIdx.x, __builtin_amdgcn_readfirstlane(taken), true);
  if (tile.none) return;
  floatx4 rg[TPL];
  raw4<E> rx[TPL], rd[TPL];
  load_tokens<TPL>(p.g + tile.base, tile.w, rg);
  load_tokens<TPL>(static_cast<const E*>(p.x) + tile.base, tile.w, rx);
  load_tokens<TPL>(static_cast<const E*>(p.dO) + tile.base, tile.w, rd);
  float a[TPL][4], w[TPL][4], A[4], H[4], F[4];
  const Seen seen = weigh<TPL, GATE, false>(rg, rx, a, w);
  if (seen.special) {
    if (seen.most > GROWS) grows = 1;
    bwd_map<TPL, true>(a, w, rx, rd, A, H, F);
  } else {
    bwd_map<TPL, false>(a, w, rx, rd, A, H, F);
  }
  *reinterpret_cast<floatx4*>(&sA[grp][col]) = floatx4{A[0], A[1], A[2], A[3]};
  *reinterpret_cast<floatx4*>(&sH[grp][col]) = floatx4{H[0], H[1], H[2], H[3]};
  *reinterpret_cast<floatx4*>(&sF[grp][col]) = floatx4{F[0], F[1], F[2], F[3]};
  barrier_lds();
  if (tid < CC) {
    const int ch = tile.c0 + tid, nc = (p.L + GLR_CHUNK - 1) / GLR_CHUNK;
    const bool live = ch < p.D;
    float start[NG / GPC];
#pragma unroll
    for (int n = 0; n < NG / GPC; ++n) {
      const int chunk = tile.tile0 / GLR_CHUNK + n;
      start[n] = live && chunk < nc ? p.states[((long)tile.b * nc + chunk) * p.D + ch] : 0.f;
    }
    const bool grown = __builtin_amdgcn_readfirstlane(grows);
    float TA, TF;
    fold_groups<false, true>(sA, sF, tid, TA, TF);
    if (__builtin_expect(grown, 0)) fold_groups<true, true>(sA, sF, tid, TA, TF);
    float flow = chain_state(chain, ((long)tile.b * chain.tiles + tile.order) * p.D + ch, p.D,
                             chain.flag + (long)tile.chain * chain.row + 1 + tile.order, tile.order, live, grown, TA, TF,
                             live && p.dh_final && tile.order == 0 ? p.dh_final[(long)tile.b * p.D + ch] : 0.f);
    if (__builtin_expect(grown, 0)) flow = start_groups<true, true, NG>(sA, sF, tid, 0, flow);
    else flow = start_groups<false, true, NG>(sA, sF, tid, 0, flow);
    if (live && p.dh0 && tile.order == chain.tiles - 1) p.dh0[(long)tile.b * p.D + ch] = flow;
#pragma unroll
    for (int n = 0; n < NG / GPC; ++n) {
      if (__builtin_expect(grown, 0)) start_groups<true, false, GPC>(sA, sH, tid, n * GPC, start[n]);
      else start_groups<false, false, GPC>(sA, sH, tid, n * GPC, start[n]);
    }
  }
  barrier_lds();
  const int have = tile.w.left - tile.w.first;
  if (tile.c0 + col >= p.D || have <= 0) return;
  const floatx4 h = *reinterpret_cast<const floatx4*>(&sH[grp][col]), flow = *reinterpret_cast<const floatx4*>(&sF[grp][col]);
  const int stores = tile.w.inside ? TPL : have;
#pragma unroll
  for (int j = 0; j < TPL; ++j) again(rx[j]), again(rd[j]);
  float* dx = p.dx + tile.base;
  float* dg = p.dg + tile.base;
  if (seen.special) bwd_out<TPL, GATE, true>(a, w, rx, rd, tile.w, h, flow, dx, dg, stores);
  else bwd_out<TPL, GATE, false>(a, w, rx, rd, tile.w, h, flow, dx, dg, stores);
}

// Sequences of up to SHORT tokens: a lane runs its 4 channels from the first token to the last, STEP at a
// time, where a tile would leave most of its groups without tokens.  Nothing is shared between lanes.
// Measured at 2048 channels, bf16: 512 sequences of 32 tokens here 53.5 us (backward 116), of 33 tokens in tiles
// 77 us (132) and here 57 (125); but 256 of 64 tokens 49 us in tiles (95) and 56 here (124), 4 of 64 tokens 4.9 us
// (6.3) and 21.6 (41).
constexpr int SHORT = 32, STEP = 8;

// Sequence, first channel and the lane's place in every [B, L, D] tensor; false past the last lane.
struct Lane {
  long first;  // element of token 0
  long state;  // element of a [B, D] tensor
  __device__ inline bool set(const GlrParams& p) {
    const long i = (long)blockIdx.x * 256 + threadIdx.x, per = p.D / 4;
    const long b = i / per;
    state = i * 4;
    first = b * p.L * p.D + i % per * 4;
    return b < p.B;
  }
  __device__ inline Where where(const GlrParams& p, int t0) const { return Where{0, 0, p.L - t0, t0 + STEP <= p.L, p.D}; }
};

template <int TPL, typename E>
__device__ inline void load_lane(const E* at, const Where& w, raw4<E>* v) {
#pragma unroll
  for (int j = 0; j < TPL; ++j) {
    v[j] = *reinterpret_cast<const raw4<E>*>(at + (long)(j < w.left ? j : w.left - 1) * w.stride);
    if (j >= w.left) v[j] = raw4<E>{};
  }
}

template <typename E, int GATE>
__global__ __launch_bounds__(256) void glr_fwd_short_kernel(GlrParams p) {
  Lane lane;
  if (!lane.set(p)) return;
  floatx4 h = {};
  if (p.h0) h = *reinterpret_cast<const floatx4*>(p.h0 + lane.state);
  if (p.states && p.L > 0) *reinterpret_cast<floatx4*>(p.states + lane.state) = h;
  for (int t0 = 0; t0 < p.L; t0 += STEP) {
    const Where w = lane.where(p, t0);
    const long at = lane.first + (long)t0 * p.D;
    floatx4 rg[STEP];
    raw4<E> rx[STEP];
    float a[STEP][4], u[STEP][4];
    load_lane<STEP>(p.g + at, w, rg);
    load_lane<STEP>(static_cast<const E*>(p.x) + at, w, rx);
    weigh<STEP, GATE, true>(rg, rx, a, u);
#pragma unroll
    for (int j = 0; j < STEP; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = step(mark(a[j][e]), h[e], u[j][e]);
      if (j < w.left) store4<E>(static_cast<E*>(p.O) + at + (long)j * p.D, h[0], h[1], h[2], h[3]);
    }
  }
  if (p.h_final) *reinterpret_cast<floatx4*>(p.h_final + lane.state) = h;
}

template <typename E, int GATE>
__global__ __launch_bounds__(256) void glr_bwd_short_kernel(GlrParams p) {
  Lane lane;
  if (!lane.set(p)) return;
  floatx4 flow = {};
  if (p.dh_final) flow = *reinterpret_cast<const floatx4*>(p.dh_final + lane.state);
  // the states before every STEP tokens, then the steps from the last to the first (their tokens are in
  // the caches by then)
  floatx4 start[SHORT / STEP];
  if (p.L > 0) start[0] = *reinterpret_cast<const floatx4*>(p.states + lane.state);
#pragma unroll
  for (int n = 1; n < SHORT / STEP; ++n) {
    start[n] = start[n - 1];
    if (n * STEP < p.L) {
      const Where w = lane.where(p, (n - 1) * STEP);
      const long at = lane.first + (long)(n - 1) * STEP * p.D;
      floatx4 rg[STEP];
      raw4<E> rx[STEP];
      float a[STEP][4], u[STEP][4];
      load_lane<STEP>(p.g + at, w, rg);
      load_lane<STEP>(static_cast<const E*>(p.x) + at, w, rx);
      weigh<STEP, GATE, true>(rg, rx, a, u);
#pragma unroll
      for (int j = 0; j < STEP; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) start[n][e] = step(mark(a[j][e]), start[n][e], u[j][e]);
    }
  }
#pragma unroll
  for (int n = SHORT / STEP - 1; n >= 0; --n) {
    if (n * STEP >= p.L) continue;
    const Where w = lane.where(p, n * STEP);
    const long at = lane.first + (long)n * STEP * p.D;
    floatx4 rg[STEP];
    raw4<E> rx[STEP], rd[STEP];
    float a[STEP][4], wt[STEP][4];
    load_lane<STEP>(p.g + at, w, rg);
    load_lane<STEP>(static_cast<const E*>(p.x) + at, w, rx);
    load_lane<STEP>(static_cast<const E*>(p.dO) + at, w, rd);
    weigh<STEP, GATE, false>(rg, rx, a, wt);
#pragma unroll
    for (int j = 0; j < STEP; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) a[j][e] = mark(a[j][e]);
    bwd_out<STEP, GATE, true>(a, wt, rx, rd, w, start[n], flow, p.dx + at, p.dg + at, w.inside ? STEP : w.left);
#pragma unroll
    for (int j = STEP - 1; j >= 0; --j) {
      float d[4];
      unpack4(rd[j], d);
#pragma unroll
      for (int e = 0; e < 4; ++e) flow[e] = Gates<true>::pass(a[j][e], a[j][e] * (d[e] + flow[e]));
    }
  }
  if (p.dh0) *reinterpret_cast<floatx4*>(p.dh0 + lane.state) = flow;
}

// One token, 4 channels of one sequence a lane: a launch's latency (2.3 us for 64 x 2048 channels).
template <typename E, int GATE>
__global__ __launch_bounds__(256) void glr_decode_kernel(GlrParams p) {
  const long i = ((long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= (long)p.B * p.D) return;
  float g[4], x[4];
  unpack4(*reinterpret_cast<const floatx4*>(p.g + i), g);
  unpack4(*reinterpret_cast<const raw4<E>*>(static_cast<const E*>(p.x) + i), x);
  floatx4 h = *reinterpret_cast<const floatx4*>(p.h_final + i);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a = mark(factor(g[e]));
    h[e] = step(a, h[e], weight<GATE>(g[e], a) * x[e]);
  }
  *reinterpret_cast<floatx4*>(p.h_final + i) = h;
  store4<E>(static_cast<E*>(p.O) + i, h[0], h[1], h[2], h[3]);
}

enum Which { FWD, BWD, DECODE };

int tile_tokens(Which which) { return NG * (which == FWD ? TPL_FWD : TPL_BWD); }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

int flag_row(int tiles) { return (tiles + 1 + 31) / 32 * 32; }  // whole 128-byte lines

// Byte offsets of the chain's arrays in the workspace.
struct Layout {
  size_t flag, total;
};
Layout layout(int B, int tiles, int D) {
  const size_t n = (size_t)B * tiles * D, blocks = (D + CC - 1) / CC;
  Layout l;
  l.flag = up256(n * 8);
  l.total = l.flag + up256((size_t)B * blocks * flag_row(tiles) * 4);
  return l;
}

template <typename E, int GATE>
hipError_t launch_one(const GlrParams& p, Which which, hipStream_t st) {
  if (which == DECODE) {
    const long n = (long)p.B * p.D / 4;
    hipLaunchKernelGGL((glr_decode_kernel<E, GATE>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, p);
    return hipGetLastError();
  }
  if (p.L <= SHORT) {
    const dim3 grid((unsigned)(((long)p.B * p.D / 4 + 255) / 256));
    if (which == FWD) hipLaunchKernelGGL((glr_fwd_short_kernel<E, GATE>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((glr_bwd_short_kernel<E, GATE>), grid, dim3(256), 0, st, p);
    return hipGetLastError();
  }
  const int TT = tile_tokens(which);
  Chain c{nullptr, nullptr, p.L > TT ? (p.L + TT - 1) / TT : 1, 0};
  if (c.tiles > 1) {
    const Layout l = layout(p.B, c.tiles, p.D);
    char* ws = static_cast<char*>(p.ws);
    c.map = reinterpret_cast<uint64_t*>(ws);
    c.flag = reinterpret_cast<uint32_t*>(ws + l.flag);
    c.row = flag_row(c.tiles);
    const long v = (long)(l.total / 16), wgs = (v + 255) / 256;
    hipLaunchKernelGGL(glr_clear_kernel, dim3((unsigned)(wgs < 2048 ? wgs : 2048)), dim3(256), 0, st,
                       reinterpret_cast<u32x4*>(ws), v);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  const unsigned jobs = (unsigned)((p.D + CC - 1) / CC) * p.B * c.tiles;
  const dim3 grid(jobs);
  if (which == FWD && p.L <= NG * TPL_SHORT) hipLaunchKernelGGL((glr_fwd_kernel<E, GATE, TPL_SHORT>), grid, dim3(WG), 0, st, p, c);
  else if (which == FWD) hipLaunchKernelGGL((glr_fwd_kernel<E, GATE, TPL_FWD>), grid, dim3(WG), 0, st, p, c);
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
bool glr_grid_fits(int B, int L, int D) {  // a launch holds fewer than 2^32 lanes
  return L <= 1 << 30 && (double)((D + CC - 1) / CC) * B * ((L + (double)NG * TPL_BWD - 1) / (NG * TPL_BWD)) < 0x1p24;
}

hipError_t launch_glr_fwd(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, FWD, st); }
hipError_t launch_glr_bwd(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, BWD, st); }
hipError_t launch_glr_decode(const GlrParams& p, bool bf16_in, hipStream_t st) { return launch(p, bf16_in, DECODE, st); }

}  // namespace delta
