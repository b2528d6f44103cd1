// Linear attention with a decay for each head, over a sequence in chunks: the chain kernel that the
// forward pass and each gradient are an instance of.
//
// With S_t = a_t S_{t-1} + k_t v_t^T and o_t = scale S_t^T q_t, cut into chunks of C tokens and gc_i the sum
// of the log gates from the chunk's start to token i:
//
//     o_i = scale (e^gc_i S^T q_i + sum_{j <= i} e^(gc_i - gc_j) (q_i . k_j) v_j)
//     S  <- e^gc_C S + sum_j e^(gc_C - gc_j) k_j v_j^T
//
// dq is the same map of (dO, v, k) with the state transposed, and dv and dk are its mirror image in time of
// (k, q, dO) and (v, dO, q): one kernel, out = chain(x, y, z), with roles for its operands, REV for the
// mirrored order, and forms that also leave what the gates' gradients need while its operands are at hand.
// Every exponent goes from a later token back to an earlier one, so decays are at most 1 for log gates up to 0; for
// gates above 1 the products within a chunk have to be float32 numbers.  The sums of log gates are held in 64
// bits, because their differences are what is used.  What spans a hard reset is an exact 0 (lin_log_gate).
//
// A workgroup has a segment of the sequence for one head and some columns of the state: each wavefront has
// CT tiles of 16 columns and all rows, in MFMA accumulators for the whole segment.  The two row tiles 2u,
// 2u + 1 interleave their rows so that the accumulators of a pair, converted, are the operand of a 32-deep
// product, in the order in which a 16-byte piece of an x row lies in LDS.  out is formed transposed, and a
// wavefront's tiles interleave their columns, so a lane ends with 4 CT consecutive columns of a token.
//
// Measured, 16 heads of 128 x 128 states in bf16.  Forward over 64K tokens: summaries 152 us (3.8 TB/s, matrix unit 28 %,
// vector instructions 47 %), chain 256 us (4.5 TB/s, 21 %, 40 %); the rest to the rate of a copy is the states' loads and
// the tail.  The three chains of a backward pass over 2 x 8K with the gates' gradients: 221 and 135 us in two
// launches (4.3 and 4.5 TB/s, matrix unit 16 and 18 %, vector instructions 30 and 33 %), of which the states that meet are
// a third of the bytes.  The state's registers allow two wavefronts a SIMD, and nothing is saturated: what is left is
// waiting between a chunk's two barriers.
// Four wavefronts of two column tiles against eight of one: chain 246 and 269 us.  Tiles of the next chunk go through
// registers; straight to a second LDS stage the summaries gain 3 us and the other forms have no LDS for it.
#pragma once
#include "common.h"
#include "linear.h"

namespace delta {
namespace lin {

template <typename E>
struct Frag;  // 8 elements along a product's depth, lane group g the indices 8 g .. 8 g + 7 of 32
template <>
struct Frag<bf16> {
  bf16x8 v;
};
template <>
struct Frag<float> {
  float v[8];
};

__device__ inline floatx4 mma(const Frag<bf16>& a, const Frag<bf16>& b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ inline floatx4 mma(const Frag<float>& a, const Frag<float>& b, floatx4 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

// Tile of rows of W elements, 16-byte chunks permuted within a row by its key.
template <typename E, int W>
struct Rows {
  static constexpr int MASK = PackedLayout<E, W>::MASK, VEC = 16 / (int)sizeof(E);
  static __device__ inline int at(int r, int e) {
    const unsigned u = e;
    return r * W + (int)(((u / VEC) ^ (unsigned)swz_key(r, MASK)) * VEC + u % VEC);
  }
  // elements e .. e + 7 of row r (e a multiple of 8)
  static __device__ inline Frag<E> row(const E* t, int r, int e) {
    Frag<E> f;
    if constexpr (sizeof(E) == 2) {
      f.v = *reinterpret_cast<const bf16x8*>(t + at(r, e));
    } else {
      const floatx4 a = *reinterpret_cast<const floatx4*>(t + at(r, e)), b = *reinterpret_cast<const floatx4*>(t + at(r, e + 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) f.v[i] = a[i], f.v[4 + i] = b[i];
    }
    return f;
  }
  // column col(lane % 16) of rows r0 + 8 (lane / 16) .. + 7, where col(i) = c0 + 16 (i / 4) / 4 step + i % 4
  // with `step` columns from one group of four to the next (4: sixteen consecutive ones)
  static __device__ inline Frag<E> col(const E* t, int r0, int c0, int step, int lane) {
    const int g = lane >> 4, i = lane & 15;
    Frag<E> f;
    if constexpr (sizeof(E) == 2) {
      const int r = r0 + 8 * g + (i >> 2), e = c0 + step * (i & 3);
      f.v = __builtin_shufflevector(read_tr4(t + at(r, e)), read_tr4(t + at(r + 4, e)), 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
#pragma unroll
      for (int n = 0; n < 8; ++n) f.v[n] = t[at(r0 + 8 * g + n, c0 + step * (i >> 2) + (i & 3))];
    }
    return f;
  }
};

// Eight float32 values as operands whose sum they are: bf16 takes three terms of eight bits of the mantissa each, cut
// off one after another, which is exact; one term is rounded to nearest.  (Two would be good to 2^-16.)
template <typename E, int TERMS>
struct Split;
template <int TERMS>
struct Split<bf16, TERMS> {
  Frag<bf16> t[TERMS];
  __device__ inline void set(const float* x) {
    if constexpr (TERMS == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[0].v[i] = (bf16)x[i];
    } else {
      u32x4 w[TERMS];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a = __builtin_bit_cast(uint32_t, x[2 * i]), b = __builtin_bit_cast(uint32_t, x[2 * i + 1]);
#pragma unroll
        for (int k = 0; k < TERMS; ++k) {
          w[k][i] = __builtin_amdgcn_perm(b, a, 0x07060302);  // the upper halves
          if (k + 1 < TERMS) a = rest(a), b = rest(b);
        }
      }
#pragma unroll
      for (int k = 0; k < TERMS; ++k) t[k].v = __builtin_bit_cast(bf16x8, w[k]);
    }
  }
  static __device__ inline uint32_t rest(uint32_t x) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, x) - __builtin_bit_cast(float, x & 0xffff0000u));
  }
};
template <int TERMS>
struct Split<float, TERMS> {
  Frag<float> t[1];
  __device__ inline void set(const float* x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[0].v[i] = x[i];
  }
};
template <typename E>
constexpr int terms(int n) {
  return sizeof(E) == 2 ? n : 1;
}

// The sum of the four lanes l % 16, + 16, + 32, + 48, in each of them: a product with ones, which costs no LDS access.
__device__ inline float sum_groups(float x) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(1.f, x, floatx4{}, 0, 0, 0)[0];
}
// The sum of the lanes l % 16, l % 16 + 16, ... below l's own group of 16.
__device__ inline float sum_groups_below(float x, int lane) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32((lane >> 4) < ((lane & 15) >> 2) ? 1.f : 0.f, x, floatx4{}, 0, 0, 0)[0];
}
// The sum over a group of 16 lanes, in each of them.
template <int CTRL>
__device__ inline float from_dpp(float x) {  // 0 from outside the group
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ inline float add_dpp(float x) {
  return x + from_dpp<CTRL>(x);
}
__device__ inline float sum_row(float x) {
  x = add_dpp<0xb1>(x);    // lanes 1, 0, 3, 2 of each four
  x = add_dpp<0x4e>(x);    // 2, 3, 0, 1
  x = add_dpp<0x141>(x);   // mirrored in each eight
  return add_dpp<0x140>(x);  // and in all sixteen
}
// Sums within a group of 16 lanes: from each lane on (itself too), and of the lanes below it.
__device__ inline float sum_from(float x) {
  x = add_dpp<0x101>(x);
  x = add_dpp<0x102>(x);
  x = add_dpp<0x104>(x);
  return add_dpp<0x108>(x);
}
__device__ inline float sum_below(float x) {
  x = from_dpp<0x111>(x);
  x = add_dpp<0x111>(x);
  x = add_dpp<0x112>(x);
  x = add_dpp<0x114>(x);
  return add_dpp<0x118>(x);
}

template <int N>
struct Int {
  static constexpr int value = N;
};

// What a chain forms beside out.  SUMS: per token the sum over columns of w_i times the state's share of out_i.
// PAIRS: also, for pairs j < i of a chunk, M_ij = e^(gc_i - gc_j) (x_i . y_j)(w_i . z_j), and per token t the sum of M over
// j < t <= i.  And these two, which walk in opposite orders over states in the same registers, form the inner product of S
// and G at every chunk: the one that comes to it first leaves its state as the registers hold it, the other multiplies.
// STATE: the state behind the last token.  A state that is an output, or that the gates' gradients are formed from,
// takes in float32 weights whole (three bf16 terms).  One that only out reads takes in two, good to 2^-16, and is rounded to
// bf16 as the operand of out's product, as A is for the chunk's own share: out carries one operand's rounding and its own,
// 2.4e-3 in the 2-norm where its own is 1.7e-3.  (One term into the state makes it 2.7e-3 where decays are slow, and takes 417
// us for 424 of the 64K forward, 295 for 307 of 2 x 16 heads of 8K backward without gates.  Two terms as the operand too: 440
// and 326, for 2.25e-3; the rest is A, for a second term of which the chains with gates have no LDS at two workgroups to a
// compute unit.)
constexpr int PLAIN = LIN_PLAIN, PAIRS = LIN_PAIRS, SUMS = LIN_SUMS, STATE = LIN_STATE;
constexpr bool for_gates(int form) { return form == PAIRS || form == SUMS; }

template <typename E, int KW, int NW, int CT, bool REV, int FORM, bool SUM>
struct Config {
  static constexpr int C = lin_chunk(sizeof(E) == 2), NB = C / 16, VW = 16 * NW * CT, TH = NW * WAVE;
  static constexpr int NT = KW / 16, NU = KW / 32;
  static constexpr int VEC = 16 / (int)sizeof(E);
  static constexpr int PX = C * KW / VEC, PZ = C * VW / VEC;            // 16-byte pieces of a tile
  static constexpr int NX = (PX + TH - 1) / TH, NZ = (PZ + TH - 1) / TH;  // of a thread
  // LDS, in bytes
  static constexpr int X = 0, Y = X + (SUM ? 0 : C * KW * (int)sizeof(E)), Z = Y + C * KW * (int)sizeof(E),
                       W = Z + C * VW * (int)sizeof(E), A = W + (for_gates(FORM) ? C * VW * (int)sizeof(E) : 0),
                       TAB = A + (SUM ? 0 : C * C * (int)sizeof(E));
  // A chunk's gate tables: sums of log gates (64 bits); x's and y's factors; decays of a token since the block of 16 it
  // is in, and from it to each later block; the chunk's
  static constexpr int BACK = 16 * (NB * (NB - 1) / 2), TABLE = 4 * (5 * C + BACK) + 16;
  static constexpr int PART = TAB + 2 * TABLE, PARTS = FORM == PAIRS ? NW + 2 * NB : FORM == SUMS ? NW : 0;
  static constexpr int EDGE = PART + PARTS * C * 4, LDS = EDGE + (for_gates(FORM) ? 4 * NW : 0);
};

// PARTED: a launch may have a part of the walk (p.part).
template <typename E, int KW, int NW, int CT, bool REV, int FORM, bool SUM, bool PARTED>
__device__ __forceinline__ void walk(const LinChain& p, unsigned block) {
  typedef Config<E, KW, NW, CT, REV, FORM, SUM> K;
  constexpr int C = K::C, NB = K::NB, VW = K::VW, NT = K::NT, NU = K::NU, VEC = K::VEC, TH = K::TH;
  constexpr bool GATES = for_gates(FORM);
  constexpr int INT = terms<E>(GATES ? 3 : 1), UPD = terms<E>(SUM || FORM != PLAIN ? 3 : 2);
  typedef Rows<E, KW> RX;
  typedef Rows<E, VW> RZ;
  typedef Rows<E, C> RA;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  E* const xt = reinterpret_cast<E*>(smem + K::X);
  E* const yt = reinterpret_cast<E*>(smem + K::Y);
  E* const zt = reinterpret_cast<E*>(smem + K::Z);
  E* const wt = reinterpret_cast<E*>(smem + K::W);
  E* const at = reinterpret_cast<E*>(smem + K::A);
  float* const part = reinterpret_cast<float*>(smem + K::PART);
  float* const dots = reinterpret_cast<float*>(smem + K::EDGE);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = p.z.width / 16, slabs = (tiles + NW * CT - 1) / (NW * CT), per = (tiles + slabs - 1) / slabs;
  const int slab = block % slabs, seg = block / slabs % p.run;
  const long bh = block / slabs / p.run;
  const int h = (int)(bh % p.H);
  const long b = bh / p.H;
  const int c0 = 16 * per * slab, cols = min(16 * per, p.z.width - c0);  // columns of this workgroup
  const int w0 = 16 * CT * wave;  // this wavefront's columns w0 ..: its tile c holds w0 + 4 CT (i / 4) + 4 c + i % 4, i < 16
  const bool live = w0 < cols;
  // the segments are the same ones in either order
  const int first = (REV ? p.P - 1 - seg : seg) * p.NS, count = min(p.NS, p.NT - first);
  auto chunk_at = [&](int i) { return REV ? first + count - 1 - i : first + i; };
  // the chunks of this launch; either order's first half is the other's second
  const int half = PARTED ? p.part : 0;
  const int cut = half == 0 ? count : REV ? count / 2 : (count + 1) / 2;
  const int first_step = half == 2 ? cut : 0, stop = half == 1 ? cut : count;
  if (first_step == stop) return;

  // ---- tiles: registers for the next chunk's pieces
  struct Source {
    const E* base;
    int stride;  // bytes between tokens
    int left;    // bytes of a row to read
  };
  auto source = [&](const LinRole& r, int col, int width) {
    const int head = h / (p.H / r.heads);
    return Source{static_cast<const E*>(r.p) + (b * p.L * r.heads + head) * r.width + col, r.heads * r.width * (int)sizeof(E),
                  width * (int)sizeof(E)};
  };
  // Offsets are formed again for every chunk, from a thread index that the optimiser cannot see through: kept, they
  // spill, and each load then waits for its offset behind the loads before it.
  auto hidden = [](int x) {
    asm volatile("" : "+v"(x));
    return x;
  };
  auto load = [&](auto& regs, const Source& s, int n, auto cpr) {
    constexpr int CPR = decltype(cpr)::value, N = sizeof(regs) / 16;
    static_assert(TH % CPR == 0 && N * TH == C * CPR, "whole rounds of whole rows");
    const int rows = min(C, p.L - n * C);
    const __amdgpu_buffer_rsrc_t r = buffer_rsrc(
        const_cast<char*>(reinterpret_cast<const char*>(s.base) + (long)n * C * s.stride), rows * s.stride);
    const int q = hidden(tid), c = q % CPR * 16;
    // rows past the sequence and columns past the width read 0 (no range reaches 2^30)
    const int from = q / CPR * s.stride + (c < s.left ? c : 1 << 30);
#pragma unroll
    for (int k = 0; k < N; ++k) regs[k] = buffer_load16(r, from + k * (TH / CPR) * s.stride);
  };
  auto put = [&](const auto& regs, E* tile, auto cpr) {
    constexpr int CPR = decltype(cpr)::value, MASK = pow2_part(CPR) - 1, N = sizeof(regs) / 16;
    const int q = hidden(tid);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int row = q / CPR + k * (TH / CPR), c = q % CPR;
      *reinterpret_cast<u32x4*>(tile + row * CPR * VEC + (c ^ swz_key(row, MASK)) * VEC) = regs[k];
    }
  };
  typedef Int<KW / VEC> CX;  // 16-byte pieces of a row
  typedef Int<VW / VEC> CZ;
  const Source sx = source(p.x, 0, p.x.width), sy = source(p.y, 0, p.y.width), sz = source(p.z, c0, cols),
               sw = source(GATES ? p.w : p.z, c0, cols);
  u32x4 rx[SUM ? 1 : K::NX], ry[K::NX], rz[K::NZ], rw[GATES ? K::NZ : 1];
  const bool keeper = wave == NW - 1;  // forms the gate tables
  auto gate_of = [&](int i) {
    const int tok = chunk_at(i) * C + lane;
    if (p.gate == LIN_GATE_NONE || lane >= C || tok >= p.L) return 0.f;
    return p.gate == LIN_GATE_TOKEN ? p.g[(b * p.L + tok) * p.H + h] : p.g[h];
  };
  float gate = 0.f;  // of this lane's token of the chunk after the one in the registers (keeper)
  auto load_all = [&](int i) {
    const int n = chunk_at(i);
    if (keeper && i + 1 < stop) gate = gate_of(i + 1);
    if constexpr (!SUM) load(rx, sx, n, CX{});
    load(ry, sy, n, CX{});
    load(rz, sz, n, CZ{});
    if constexpr (GATES) load(rw, sw, n, CZ{});
  };
  auto put_all = [&]() {
    if constexpr (!SUM) put(rx, xt, CX{});
    put(ry, yt, CX{});
    put(rz, zt, CZ{});
    if constexpr (GATES) put(rw, wt, CZ{});
    asm volatile("" : "+v"(gate));  // waited for here, not behind the next chunk's loads
  };

  // ---- a chunk's gate tables, by one wavefront (gc as a power of two)
  struct Table {
    double* gc;
    float *fx, *fy, *in, *back, *whole;
  };
  auto table = [&](int i) {
    char* t = smem + K::TAB + (i & 1) * K::TABLE;
    float* f = reinterpret_cast<float*>(t + 8 * C);
    return Table{reinterpret_cast<double*>(t), f, f + C, f + 2 * C, f + 3 * C, f + 3 * C + K::BACK};
  };
  auto back_of = [](int hi) { return 8 * hi * (hi - 1); };  // where the decays to block hi begin
  double sum = 0.0;  // log gates of the chunks so far, -inf with a reset among them (keeper)
  auto tables = [&](int i, float gl) {
    const int ln = GATES ? hidden(lane) : lane;
    double a = lin_log_gate(gl);
#pragma unroll
    for (int o = 1; o < C; o <<= 1) {
      const double up = __shfl_up(a, o, WAVE);
      if (ln >= o) a += up;
    }
    const double last = __shfl(a, C - 1, WAVE);
    sum += last < LIN_RESET / 2 ? -INFINITY : last;
    const Table t = table(i);
    const float begin = expf((float)a), end = expf((float)(last - a));
    const double ref = __shfl(a, max(16 * (ln >> 4) - 1, 0), WAVE);
    if (ln < C) {
      t.gc[ln] = a * 1.4426950408889634074;
      t.fx[ln] = (REV ? end : begin) * p.outer;
      t.fy[ln] = (REV ? begin : end) * p.write;
      t.in[ln] = expf((float)(ln < 16 ? a : a - ref));
    }
#pragma unroll
    for (int hi = 1; hi < NB; ++hi) {
      const float to = expf((float)(__shfl(a, 16 * hi - 1, WAVE) - a));
      if (ln < 16 * hi) t.back[back_of(hi) + ln] = to;
    }
    if (ln == 0) *t.whole = expf((float)last);
  };

  // ---- the state: rows srow(t, 4 g + j) of column m of this wavefront's tiles
  auto srow = [](int t, int r) { return 32 * (t >> 1) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3); };
  const int width = p.y.width;
  const int size = width * p.z.width;
  floatx4 S[CT][NT];
  // A lane's four rows of a tile lie next to each other in a flipped state, and are z.width apart in another one.
  auto each = [&](auto four, auto one) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int row = srow(t, 4 * (lane >> 4)), own = w0 + 4 * CT * ((lane & 15) >> 2) + 4 * c + (lane & 3);
        const bool in = own < cols && row < width;
        if (p.flip) {
          four(c, t, in ? ((c0 + own) * width + row) * 4 : 1 << 30);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) one(c, t, j, in ? ((row + j) * p.z.width + c0 + own) * 4 : 1 << 30);
        }
      }
  };
  // A state as the registers hold it: 16 x 16 tiles of a lane's four elements each.
  const int slot = (tiles + 1) / 2 * 2 * NT * (4 * WAVE);
  auto raw = [&](float* base, long i, int ln) { return reinterpret_cast<floatx4*>(base + i * slot) + wave * (CT * NT * WAVE) + ln; };
  const float first_gate = keeper ? gate_of(first_step) : 0.f;
  load_all(first_step);  // under way while the state is loaded
  const float* from = SUM ? nullptr : p.P > 1 ? p.segs + (bh * p.P + seg) * size : p.start ? p.start + bh * size : nullptr;
  const __amdgpu_buffer_rsrc_t start = buffer_rsrc(const_cast<float*>(from), from ? size * 4 : 0);  // else all 0
  if constexpr (SUM) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int t = 0; t < NT; ++t) S[c][t] = floatx4{};
  } else if (first_step > 0) {
    if (live) {
      const floatx4* q = raw(p.wait, bh * p.P + seg, lane);
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int t = 0; t < NT; ++t) S[c][t] = q[(c * NT + t) * WAVE];
    }
  } else {
    each([&](int c, int t, int i) { S[c][t] = __builtin_bit_cast(floatx4, buffer_load16(start, i)); },
         [&](int c, int t, int j, int i) { S[c][t][j] = buffer_load4(start, i); });
  }

  // what is never written again: blocks of A past the diagonal, slots of wavefronts without columns
  if constexpr (!SUM)
    for (int i = tid; i < C * C; i += TH) at[i] = (E)0.f;
  for (int i = tid; i < K::PARTS * C + (GATES ? NW : 0); i += TH) part[i] = 0.f;

  if (keeper) tables(first_step, first_gate);
  put_all();
  float next = gate;  // gates of the chunk whose tables come next
  if (first_step + 1 < stop) load_all(first_step + 1);
  barrier_lds();

  for (int i = first_step; i < stop; ++i) {
    const int n = chunk_at(i);
    const Table tab = table(i);
    // LDS addresses are formed again in every chunk, from a lane that the optimiser cannot see through: hoisted
    // out of the loop they take a hundred registers
    const int ln = hidden(lane);
    const int g4 = ln >> 4, m = ln & 15;
    if (keeper && i + 1 < stop) tables(i + 1, next);

    // S before the chunk, or G behind it, left for the other order's walk or met by it; a chunk that lets nothing through
    // needs neither
    [[maybe_unused]] const bool meets = GATES && (FORM == PAIRS ? half == 2 : half != 1);
    if constexpr (GATES) {
      const bool open = __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, *tab.whole)) != 0;
      if (live && open) {
        floatx4* q = raw(p.states, bh * p.NT + n, ln);
        if (meets) {
          // two groups on their way (when measured, 16 heads of 2 x 8K tokens 452 us; all 64 registers of them spill, 472; half
          // of them a phase ahead spill too, 554)
          constexpr int GROUP = CT * NT < 4 ? CT * NT : 4, AHEAD = 2, GROUPS = CT * NT / GROUP;
          floatx4 other[AHEAD][GROUP], dot = {};
          auto fetch = [&](int k) {
#pragma unroll
            for (int e = 0; e < GROUP; ++e) other[k % AHEAD][e] = __builtin_nontemporal_load(q + (k * GROUP + e) * WAVE);
          };
#pragma unroll
          for (int k = 0; k < AHEAD && k < GROUPS; ++k) fetch(k);
#pragma unroll
          for (int k = 0; k < GROUPS; ++k) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < GROUP; ++e) dot += S[(k * GROUP + e) / NT][(k * GROUP + e) % NT] * other[k % AHEAD][e];
            if (k + AHEAD < GROUPS) fetch(k + AHEAD);
          }
          __builtin_amdgcn_sched_barrier(0);
          const float all = sum_groups(sum_row((dot[0] + dot[1]) + (dot[2] + dot[3])));
          if (ln == 0) dots[wave] = all;
        } else {
#pragma unroll
          for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int t = 0; t < NT; ++t) __builtin_nontemporal_store(S[c][t], q + (c * NT + t) * WAVE);
        }
      }
    }

    // A = inner Gamma (x y^T), block by block: rows j of the product are y's tokens, so a lane has four
    // consecutive j of one token i
    if constexpr (!SUM) {
#pragma unroll
      for (int k = 0; k < (NB * (NB + 1) / 2 + NW - 1) / NW; ++k) {
        const int q = wave + k * NW;
        if (q < NB * (NB + 1) / 2) {
          const int hi = q < 1 ? 0 : q < 3 ? 1 : q < 6 ? 2 : 3, lo = q - hi * (hi + 1) / 2;
          const int ib = REV ? lo : hi, jb = REV ? hi : lo;
          floatx4 d = {}, d2 = {};
#pragma unroll
          for (int u = 0; u < NU; ++u)
            d = mma(RX::row(yt + 16 * jb * KW, m, 32 * u + 8 * g4), RX::row(xt + 16 * ib * KW, m, 32 * u + 8 * g4), d);
          if constexpr (FORM == PAIRS) {
#pragma unroll
            for (int u = 0; u < (VW + 31) / 32; ++u)
              if (32 * u < cols)
                d2 = mma(RZ::row(zt + 16 * jb * VW, m, 32 * u + 8 * g4), RZ::row(wt + 16 * ib * VW, m, 32 * u + 8 * g4), d2);
          }
          const int ti = 16 * ib + m, tj = 16 * jb + 4 * g4;
          float v[4];
          if (hi == lo) {
            const double gi = tab.gc[ti];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const double e = REV ? tab.gc[tj + r] - gi : gi - tab.gc[tj + r];
              const bool on = REV ? tj + r >= ti : tj + r <= ti;
              const float factor = p.inner * __builtin_amdgcn_exp2f(on ? (float)e : -INFINITY);
              v[r] = on ? d[r] * factor : 0.f;
              if constexpr (FORM == PAIRS) d2[r] = tj + r < ti ? v[r] * d2[r] : 0.f;
            }
          } else {  // through the end of the block before hi: two decays
            const float* back = tab.back + back_of(hi);
            const float fi = p.inner * (REV ? back[ti] : tab.in[ti]);
            const floatx4 fj = *reinterpret_cast<const floatx4*>((REV ? tab.in : back) + tj);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              v[r] = d[r] * (fi * fj[r]);
              if constexpr (FORM == PAIRS) d2[r] *= v[r];
            }
          }
          store4<E>(at + RA::at(ti, tj), v[0], v[1], v[2], v[3]);
          // Pairs around a token t: of another block's two halves their row sums from t on, or column sums before t; of
          // its own block the sum over j < t in each row, then over the rows from t on.
          if constexpr (FORM == PAIRS) {
            const float four = (d2[0] + d2[1]) + (d2[2] + d2[3]);
            if (hi == lo) {
              float before = sum_groups_below(four, ln);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float own = d2[r];
                d2[r] = ti >= tj + r ? before : 0.f;
                before += own;
              }
            } else {
              const float row = sum_groups(four);
              if (g4 == 0) part[(NW + jb) * C + ti] = row;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) d2[r] = sum_row(d2[r]);
            if (m == 0) *reinterpret_cast<floatx4*>(part + (NW + NB + ib) * C + tj) = d2;
          }
        }
      }
    }

    [[maybe_unused]] floatx4 out[CT][NB];
    Frag<E> zf[CT][C / 32];
    if (live) {
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int s = 0; s < C / 32; ++s) zf[c][s] = RZ::col(zt, 32 * s, w0 + 4 * c, 4 * CT, ln);

      // the state's share of out
      if constexpr (!SUM) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int ib = 0; ib < NB; ++ib) out[c][ib] = floatx4{};
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          Split<E, INT> sf[CT];
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            float s8[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) s8[j] = S[c][2 * u][j], s8[4 + j] = S[c][2 * u + 1][j];
            sf[c].set(s8);
          }
#pragma unroll
          for (int ib = 0; ib < NB; ++ib) {
            const Frag<E> xf = RX::row(xt + 16 * ib * KW, m, 32 * u + 8 * g4);
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
              for (int k = INT - 1; k >= 0; --k) out[c][ib] = mma(sf[c].t[k], xf, out[c][ib]);
          }
        }
#pragma unroll
        for (int ib = 0; ib < NB; ++ib) {
          const float fx = tab.fx[16 * ib + m];
#pragma unroll
          for (int c = 0; c < CT; ++c) out[c][ib] *= fx;
          if constexpr (GATES) {
            float e = 0.f;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              const E* wr = wt + RZ::at(16 * ib + m, w0 + 4 * CT * g4 + 4 * c);
#pragma unroll
              for (int r = 0; r < 4; ++r) e += out[c][ib][r] * to_float(wr[r]);
            }
            e = sum_groups(e);
            if (g4 == 0) part[wave * C + 16 * ib + m] = e;
          }
        }
      }

      // the state behind the chunk
      const float whole = *tab.whole;
      const int lu = hidden(lane);
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int t = 0; t < NT; ++t) S[c][t] *= whole;
#pragma unroll
      for (int s = 0; s < C / 32; ++s) {
        Split<E, UPD> zw[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          float z8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) z8[k] = to_float((E)zf[c][s].v[k]) * tab.fy[32 * s + 8 * g4 + k];
          zw[c].set(z8);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const Frag<E> yf = RX::col(yt + 32 * s * KW, 0, 32 * (t >> 1) + 4 * (t & 1), 8, lu);
#pragma unroll
          for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int k = UPD - 1; k >= 0; --k) S[c][t] = mma(yf, zw[c].t[k], S[c][t]);
        }
      }
    }
    barrier_lds();  // A is whole; the tiles have been read

    if (i + 1 < stop) {
      put_all();
      next = gate;
      if (i + 2 < stop) load_all(i + 2);
    }
    if constexpr (!SUM) {
      if (live) {
        // the chunk's own share
#pragma unroll
        for (int s = 0; s < C / 32; ++s)
#pragma unroll
          for (int ib = 0; ib < NB; ++ib)
            if (REV ? 2 * s + 1 >= ib : 2 * s <= ib) {
              const Frag<E> af = RA::row(at + 16 * ib * C, m, 32 * s + 8 * g4);
#pragma unroll
              for (int c = 0; c < CT; ++c) out[c][ib] = mma(zf[c][s], af, out[c][ib]);
            }
        const int rows = min(C, p.L - n * C), stride = p.H * p.z.width;
        const long head = (b * p.L + (long)n * C) * p.H + h;
        const int size_of = sizeof(E) == 2 && !p.out_f32 ? 2 : 4;
        const __amdgpu_buffer_rsrc_t r = buffer_rsrc(static_cast<char*>(p.out) + head * p.z.width * size_of, rows * stride * size_of);
        const int own = w0 + 4 * CT * g4, to = own < cols ? m * stride + c0 + own : 1 << 28;  // past every range
#pragma unroll
        for (int ib = 0; ib < NB; ++ib) {
          const int at = (to + 16 * ib * stride) * size_of;
          if (size_of == 4) {
#pragma unroll
            for (int c = 0; c < CT; ++c) buffer_store16(r, at + 16 * c, out[c][ib]);
          } else if constexpr (CT == 2) {
            bf16x8 v;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = (bf16)out[0][ib][k], v[4 + k] = (bf16)out[1][ib][k];
            buffer_store16(r, at, __builtin_bit_cast(floatx4, v));
          } else {
            const floatx4 o = out[0][ib];
            buffer_store8(r, at, bf16x4{(bf16)o[0], (bf16)o[1], (bf16)o[2], (bf16)o[3]});
          }
        }
      }
      if constexpr (GATES) {
        const int tok = hidden(lane);
        if (wave == 0 && tok < C) {
          float e = 0.f;
#pragma unroll
          for (int k = 0; k < NW; ++k) e += part[k * C + tok];
          p.tok[(bh * p.NT + n) * C + tok] = e;
          if constexpr (FORM == PAIRS) {
            const int own = tok >> 4;
            float row = 0.f, col = 0.f, around = part[(NW + NB + own) * C + tok];
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              row += part[(NW + k) * C + tok];  // none from blocks behind
              const float down = part[(NW + NB + k) * C + tok];
              col += k > own ? down : 0.f;
              if (NB == 4 && k >= 2) {  // blocks 0 and 2, 0 and 3, 1 and 3 lie on either side of others
                const int whole = __builtin_bit_cast(int, sum_row(down));
                const float from0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(whole, 0));
                const float from1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(whole, 16));
                around += own == 1 ? from0 : own == 2 && k == 3 ? from0 + from1 : 0.f;
              }
            }
            p.pair[(bh * p.NT + n) * C + tok] = around + sum_from(row) + sum_below(col);
          }
        }
        if (meets && tid == 0) {
          float dot = 0.f;
#pragma unroll
          for (int k = 0; k < NW; ++k) dot += dots[k];
          const float whole = *tab.whole;
          p.edge[bh * p.NT + n] = whole == 0.f ? 0.f : whole * dot;
        }
      }
    }
    barrier_lds();
  }

  float* to = SUM ? p.segs + (bh * p.P + seg) * size : FORM == STATE ? p.end + bh * size : nullptr;
  if (half == 1) {
    if (live) {
      floatx4* q = raw(p.wait, bh * p.P + seg, lane);
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int t = 0; t < NT; ++t) q[(c * NT + t) * WAVE] = S[c][t];
    }
  } else if (to) {
    const __amdgpu_buffer_rsrc_t end = buffer_rsrc(to, size * 4);
    each([&](int c, int t, int i) { buffer_store16(end, i, S[c][t]); },
         [&](int c, int t, int j, int i) { buffer_store4(end, i, S[c][t][j]); });
  }
  if (SUM && keeper && slab == 0 && lane == 0) p.decay[bh * p.P + seg] = sum;
}

// Wavefronts on a SIMD that the registers are shared out for: bf16 chains of up to 128 rows and 128 columns fit twice on
// a compute unit.
template <typename E, int KW, int NW, int CT>
constexpr int waves() {
  return NW * CT == 8 && KW <= 128 && sizeof(E) == 2 ? 2 : 1;
}

template <typename E, int KW, int NW, int CT, bool REV, int FORM>
__global__ __launch_bounds__(NW * WAVE, (waves<E, KW, NW, CT>())) void chain_kernel(LinChain p) {
  walk<E, KW, NW, CT, REV, FORM, false, false>(p, blockIdx.x);
}

// The summaries of one chain, or of a chain and one in the other order behind it.
template <typename E, int KW, int CT>
__global__ __launch_bounds__(4 * WAVE, (waves<E, KW, 4, CT>())) void summary_kernel(LinChain forward, LinChain reverse, unsigned split) {
  if (blockIdx.x < split) walk<E, KW, 4, CT, false, PLAIN, true, false>(forward, blockIdx.x);
  else walk<E, KW, 4, CT, true, PLAIN, true, false>(reverse, blockIdx.x - split);
}

// The three chains of a backward pass side by side: workgroups bound by products run next to ones bound by memory, and
// there is one tail.  dv's come first, which may walk twice as far (linear_abi.cpp).  KQ, KV: the rows for q's and k's width,
// and for v's; LAST: dv's form, which may leave its state.
template <typename E, int KQ, int KV, bool GATES, int LAST>
__global__ __launch_bounds__(4 * WAVE, sizeof(E) == 2 ? 2 : 1) void backward_kernel(LinChain dq, LinChain dv, LinChain dk, unsigned first,
                                                                               unsigned second) {
  constexpr int CQ = KQ == 128 ? 2 : 1, CV = KV == 128 ? 2 : 1;
  if (blockIdx.x < first) walk<E, KQ, 4, CV, true, LAST, false, GATES>(dv, blockIdx.x);
  else if (blockIdx.x < second) walk<E, KV, 4, CQ, false, GATES ? PAIRS : PLAIN, false, GATES>(dq, blockIdx.x - first);
  else walk<E, KV, 4, CQ, true, GATES ? SUMS : PLAIN, false, GATES>(dk, blockIdx.x - second);
}

constexpr int max_of(int a, int b) { return a > b ? a : b; }

// Workgroups of a chain with 16 NW CT columns each.
inline unsigned blocks(const LinChain& c, int tiles_each) {
  const int tiles = c.z.width / 16;
  return (unsigned)((long)c.B * c.H * c.run * ((tiles + tiles_each - 1) / tiles_each));
}

template <typename E, int KW, int NW, int CT, bool REV, int FORM>
hipError_t run(const LinChain& c, hipStream_t st) {
  typedef Config<E, KW, NW, CT, REV, FORM, false> K;
  static_assert(K::LDS <= 160 * 1024, "a workgroup's LDS");
  hipLaunchKernelGGL((chain_kernel<E, KW, NW, CT, REV, FORM>), dim3(blocks(c, NW * CT)), dim3(K::TH), K::LDS, st, c);
  return hipGetLastError();
}

// Workgroups of 64 or 128 columns, four wavefronts with one tile or two each; states of 256 rows (the backward pass of
// values of more than 128 channels) leave the registers of a wavefront room for one tile.
template <typename E, int KW, bool REV, int FORM>
hipError_t by_columns(const LinChain& c, hipStream_t st) {
  // a reverse chain alone is one of more columns than the three together take
  if constexpr (!REV)
    if (c.z.width <= 64) return run<E, KW, 4, 1, REV, FORM>(c, st);
  return run<E, KW, 4, 2, REV, FORM>(c, st);
}

template <typename E, bool REV, int FORM>
hipError_t by_width(const LinChain& c, hipStream_t st) {
  const int w = c.y.width;
  if (w <= 32) return by_columns<E, 32, REV, FORM>(c, st);
  return w <= 64 ? by_columns<E, 64, REV, FORM>(c, st) : by_columns<E, 128, REV, FORM>(c, st);
}

template <typename E>
hipError_t chain(const LinChain& c, bool reverse, int form, hipStream_t st) {
  if (c.y.width > 128) {
    switch (form) {
      case PLAIN: return reverse ? run<E, 256, 8, 1, true, PLAIN>(c, st) : run<E, 256, 8, 1, false, PLAIN>(c, st);
      case PAIRS: return run<E, 256, 8, 1, false, PAIRS>(c, st);
      case SUMS: return run<E, 256, 8, 1, true, SUMS>(c, st);
      default: return hipErrorInvalidValue;
    }
  }
  switch (form) {
    case PLAIN: return reverse ? by_width<E, true, PLAIN>(c, st) : by_width<E, false, PLAIN>(c, st);
    case STATE: return reverse ? by_width<E, true, STATE>(c, st) : by_width<E, false, STATE>(c, st);
    default: return hipErrorInvalidValue;
  }
}

template <typename E, int KW, int CT>
hipError_t run_summary(const LinChain& forward, const LinChain* reverse, hipStream_t st) {
  const unsigned split = blocks(forward, 4 * CT), all = split + (reverse ? blocks(*reverse, 4 * CT) : 0);
  if (all == 0) return hipSuccess;
  hipLaunchKernelGGL((summary_kernel<E, KW, CT>), dim3(all), dim3(4 * WAVE), (Config<E, KW, 4, CT, false, PLAIN, true>::LDS), st,
                     forward, reverse ? *reverse : forward, split);
  return hipGetLastError();
}
template <typename E>
hipError_t summary(const LinChain& forward, const LinChain* reverse, hipStream_t st) {
  const int w = forward.y.width;
  const bool wide = forward.z.width > 64;
  if (w <= 32) return wide ? run_summary<E, 32, 2>(forward, reverse, st) : run_summary<E, 32, 1>(forward, reverse, st);
  if (w <= 64) return wide ? run_summary<E, 64, 2>(forward, reverse, st) : run_summary<E, 64, 1>(forward, reverse, st);
  return wide ? run_summary<E, 128, 2>(forward, reverse, st) : run_summary<E, 128, 1>(forward, reverse, st);
}

template <typename E, int KQ, int KV, bool GATES, int LAST>
hipError_t run_backward(const LinChain& dq, const LinChain& dv, const LinChain& dk, hipStream_t st) {
  constexpr int CQ = KQ == 128 ? 2 : 1, CV = KV == 128 ? 2 : 1;
  constexpr int LDS = max_of(Config<E, KV, 4, CQ, false, GATES ? PAIRS : PLAIN, false>::LDS, Config<E, KQ, 4, CV, true, LAST, false>::LDS);
  const unsigned first = blocks(dv, 4 * CV), second = first + blocks(dq, 4 * CQ);
  hipLaunchKernelGGL((backward_kernel<E, KQ, KV, GATES, LAST>), dim3(second + blocks(dk, 4 * CQ)), dim3(4 * WAVE), LDS, st, dq, dv,
                     dk, first, second);
  return hipGetLastError();
}
template <typename E, bool GATES, int LAST, int KQ>
hipError_t backward_by_values(const LinChain& dq, const LinChain& dv, const LinChain& dk, hipStream_t st) {
  if (dv.z.width <= 32) return run_backward<E, KQ, 32, GATES, LAST>(dq, dv, dk, st);
  return dv.z.width <= 64 ? run_backward<E, KQ, 64, GATES, LAST>(dq, dv, dk, st) : run_backward<E, KQ, 128, GATES, LAST>(dq, dv, dk, st);
}
template <typename E, bool GATES, int LAST>
hipError_t backward(const LinChain& dq, const LinChain& dv, const LinChain& dk, hipStream_t st) {
  if (dq.z.width <= 32) return backward_by_values<E, GATES, LAST, 32>(dq, dv, dk, st);
  return dq.z.width <= 64 ? backward_by_values<E, GATES, LAST, 64>(dq, dv, dk, st) : backward_by_values<E, GATES, LAST, 128>(dq, dv, dk, st);
}
template <typename E, bool GATES>
hipError_t backward(const LinChain& dq, const LinChain& dv, const LinChain& dk, bool state, hipStream_t st) {
  return state ? backward<E, GATES, STATE>(dq, dv, dk, st) : backward<E, GATES, PLAIN>(dq, dv, dk, st);
}

}  // namespace lin
}  // namespace delta
