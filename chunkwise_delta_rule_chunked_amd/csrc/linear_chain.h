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
// mirrored order, and a hook that forms what the gates' gradients need while its operands are at hand.
// Every exponent goes from a later token back to an earlier one, so decays never overflow; the sums of log
// gates are held in 64 bits, because their differences are what is used (behind a hard reset of -150 a
// float32 sum has lost 1e-5).
//
// A workgroup has a segment of the sequence for one head and up to 128 columns of the state: 8 wavefronts,
// each with 16 columns and all rows, in MFMA accumulators for the whole segment.  The two row tiles 2u,
// 2u + 1 interleave their rows so that the accumulators of a pair, converted, are the operand of a 32-deep
// product, in the order in which a 16-byte piece of an x row lies in LDS.  out is formed transposed, so a
// lane ends with four consecutive columns of a token.
#pragma once
#include "common.h"
#include "linear.h"

namespace delta {
namespace lin {

constexpr int NW = 8, TH = NW * WAVE;

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

// Eight float32 values as `terms` operands whose sum they are to within 2^-9 of the last one's step: bf16
// products of the terms carry float32 values to 2^-17 (two terms) or 2^-26 (three).
template <typename E, int TERMS>
struct Split;
template <int TERMS>
struct Split<bf16, TERMS> {
  Frag<bf16> t[TERMS];
  __device__ inline explicit Split(const float* x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float r = x[i];
#pragma unroll
      for (int k = 0; k < TERMS; ++k) {
        t[k].v[i] = (bf16)r;
        if (k + 1 < TERMS) r -= (float)t[k].v[i];
      }
    }
  }
};
template <int TERMS>
struct Split<float, TERMS> {
  Frag<float> t[1];
  __device__ inline explicit Split(const float* x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[0].v[i] = x[i];
  }
};
template <typename E>
constexpr int terms(int n) {
  return sizeof(E) == 2 ? n : 1;
}

template <int N>
struct Int {
  static constexpr int value = N;
};

// Hooks: 1, with the sum over columns of w_i times the state's share of out_i (e) and, for pairs j < i,
// M_ij = e^(gc_i - gc_j) (x_i . y_j)(w_i . z_j): e + M's row sums - its column sums per token.  2: e alone.
template <typename E, int KW, bool REV, int HOOK, bool SUM>
struct Config {
  static constexpr int C = lin_chunk(sizeof(E) == 2), NB = C / 16, VW = LIN_SLAB;
  static constexpr int NT = KW / 16, NU = KW / 32;
  static constexpr int VEC = 16 / (int)sizeof(E);
  static constexpr int PX = C * KW / VEC, PZ = C * VW / VEC;            // 16-byte pieces of a tile
  static constexpr int NX = (PX + TH - 1) / TH, NZ = (PZ + TH - 1) / TH;  // of a thread
  // LDS, in bytes
  static constexpr int X = 0, Y = X + (SUM ? 0 : C * KW * (int)sizeof(E)), Z = Y + C * KW * (int)sizeof(E),
                       W = Z + C * VW * (int)sizeof(E), A = W + (HOOK ? C * VW * (int)sizeof(E) : 0),
                       TAB = A + (SUM ? 0 : C * C * (int)sizeof(E));
  static constexpr int TABLE = 4 * C * 4 + 16;  // sums of log gates (64 bits), x's and y's factors, the chunk's
  static constexpr int PART = TAB + 2 * TABLE, PARTS = HOOK == 1 ? NW + 2 * NB : HOOK == 2 ? NW : 0;
  static constexpr int LDS = PART + PARTS * C * 4;
};

template <typename E, int KW, bool REV, int HOOK, bool SUM>
__global__ __launch_bounds__(TH) void chain_kernel(LinChain p) {
  typedef Config<E, KW, REV, HOOK, SUM> K;
  constexpr int C = K::C, NB = K::NB, VW = K::VW, NT = K::NT, NU = K::NU, VEC = K::VEC;
  constexpr int INT = terms<E>(HOOK ? 3 : 1);
  // A state that is an output, or that the gates' gradients are formed from, takes float32 weights in whole (three
  // terms); one that only out reads, whose products round it to bf16, one term.
  const bool whole_terms = SUM || HOOK || (p.P == 1 && p.end);
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

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g4 = lane >> 4, m = lane & 15;
  const int tiles = p.z.width / 16, slabs = (tiles + NW - 1) / NW, per = (tiles + slabs - 1) / slabs;
  const int slab = blockIdx.x % slabs, seg = blockIdx.x / slabs % p.run;
  const long bh = blockIdx.x / slabs / p.run;
  const int h = (int)(bh % p.H);
  const long b = bh / p.H;
  const int c0 = 16 * per * slab, cols = min(16 * per, p.z.width - c0);  // columns of this workgroup
  const bool live = 16 * wave < cols;
  // the segments are the same ones in either order
  const int first = (REV ? p.P - 1 - seg : seg) * p.NS, count = min(p.NS, p.NT - first);
  auto chunk_at = [&](int i) { return REV ? first + count - 1 - i : first + i; };

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
  auto load = [&](auto& regs, const Source& s, int n, auto cpr, int pieces) {
    constexpr int CPR = decltype(cpr)::value;
    const int rows = min(C, p.L - n * C);
    const __amdgpu_buffer_rsrc_t r = buffer_rsrc(
        const_cast<char*>(reinterpret_cast<const char*>(s.base) + (long)n * C * s.stride), rows * s.stride);
#pragma unroll
    for (int k = 0; k < (int)(sizeof(regs) / 16); ++k) {
      const int q = tid + k * TH, row = q / CPR, c = q % CPR * 16;
      // rows past the sequence and columns past the width read 0
      regs[k] = buffer_load16(r, q < pieces && c < s.left ? row * s.stride + c : 0x7fffffff);
    }
  };
  auto put = [&](const auto& regs, E* tile, auto cpr, int pieces) {
    constexpr int CPR = decltype(cpr)::value, MASK = pow2_part(CPR) - 1;
#pragma unroll
    for (int k = 0; k < (int)(sizeof(regs) / 16); ++k) {
      const int q = tid + k * TH, row = q / CPR, c = q % CPR;
      if (q < pieces) *reinterpret_cast<u32x4*>(tile + row * CPR * VEC + (c ^ swz_key(row, MASK)) * VEC) = regs[k];
    }
  };
  typedef Int<KW / VEC> CX;  // 16-byte pieces of a row
  typedef Int<VW / VEC> CZ;
  const Source sx = source(p.x, 0, p.x.width), sy = source(p.y, 0, p.y.width), sz = source(p.z, c0, cols),
               sw = source(HOOK ? p.w : p.z, c0, cols);
  u32x4 rx[SUM ? 1 : K::NX], ry[K::NX], rz[K::NZ], rw[HOOK ? K::NZ : 1];
  auto load_all = [&](int i) {
    const int n = chunk_at(i);
    if constexpr (!SUM) load(rx, sx, n, CX{}, K::PX);
    load(ry, sy, n, CX{}, K::PX);
    load(rz, sz, n, CZ{}, K::PZ);
    if constexpr (HOOK != 0) load(rw, sw, n, CZ{}, K::PZ);
  };
  auto put_all = [&]() {
    if constexpr (!SUM) put(rx, xt, CX{}, K::PX);
    put(ry, yt, CX{}, K::PX);
    put(rz, zt, CZ{}, K::PZ);
    if constexpr (HOOK != 0) put(rw, wt, CZ{}, K::PZ);
  };

  // ---- a chunk's gate tables, by one wavefront: gc log2 e, x's factors, y's factors, the chunk's
  struct Table {
    const double* gc;
    const float *fx, *fy, *whole;
  };
  auto table = [&](int i) {
    char* t = smem + K::TAB + (i & 1) * K::TABLE;
    return Table{reinterpret_cast<double*>(t), reinterpret_cast<float*>(t + 8 * C), reinterpret_cast<float*>(t + 12 * C),
                 reinterpret_cast<float*>(t + 16 * C)};
  };
  const bool keeper = wave == NW - 1;
  double sum = 0.0;  // log gates of the chunks so far (keeper)
  auto gate_of = [&](int i) {  // this lane's token's
    const int tok = chunk_at(i) * C + lane;
    if (p.gate == LIN_GATE_NONE || lane >= C || tok >= p.L) return 0.f;
    return p.gate == LIN_GATE_TOKEN ? p.g[(b * p.L + tok) * p.H + h] : p.g[h];
  };
  auto tables = [&](int i, float gl) {
    double a = (double)(gl < LOG_GATE_FLOOR ? LOG_GATE_FLOOR : gl);
#pragma unroll
    for (int o = 1; o < C; o <<= 1) {
      const double up = __shfl_up(a, o, WAVE);
      if (lane >= o) a += up;
    }
    const double last = __shfl(a, C - 1, WAVE);
    sum += last;
    const Table t = table(i);
    const float begin = expf((float)a), end = expf((float)(last - a));
    if (lane < C) {
      const_cast<double*>(t.gc)[lane] = a * 1.4426950408889634074;
      const_cast<float*>(t.fx)[lane] = (REV ? end : begin) * p.outer;
      const_cast<float*>(t.fy)[lane] = (REV ? begin : end) * p.write;
    }
    if (lane == 0) *const_cast<float*>(t.whole) = expf((float)last);
  };

  // ---- the state: rows srow(t, 4 g + j) of column m of this wavefront's 16
  auto srow = [](int t, int r) { return 32 * (t >> 1) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3); };
  const int width = p.y.width, col = c0 + 16 * wave + m;
  const long size = (long)width * p.z.width;
  auto element = [&](int row) { return p.flip ? (long)col * width + row : (long)row * p.z.width + col; };
  floatx4 S[NT];
  const float* from = SUM ? nullptr : p.P > 1 ? p.segs + (bh * p.P + seg) * size : p.start ? p.start + bh * size : nullptr;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = srow(t, 4 * g4 + j);
      S[t][j] = from && live && row < width ? from[element(row)] : 0.f;
    }

  // what is never written again: blocks of A past the diagonal, hooks' slots of wavefronts without columns
  if constexpr (!SUM)
    for (int i = tid; i < C * C; i += TH) at[i] = (E)0.f;
  for (int i = tid; i < K::PARTS * C; i += TH) part[i] = 0.f;

  float gnext = 0.f;
  if (keeper) {
    tables(0, gate_of(0));
    if (count > 1) gnext = gate_of(1);
  }
  load_all(0);
  put_all();
  if (count > 1) load_all(1);
  barrier_lds();

  for (int i = 0; i < count; ++i) {
    const int n = chunk_at(i);
    const Table tab = table(i);
    if (keeper && i + 1 < count) {
      tables(i + 1, gnext);
      if (i + 2 < count) gnext = gate_of(i + 2);
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
            d = mma(RX::row(yt, 16 * jb + m, 32 * u + 8 * g4), RX::row(xt, 16 * ib + m, 32 * u + 8 * g4), d);
          if constexpr (HOOK == 1) {
#pragma unroll
            for (int u = 0; u < VW / 32; ++u)
              if (32 * u < cols) d2 = mma(RZ::row(zt, 16 * jb + m, 32 * u + 8 * g4), RZ::row(wt, 16 * ib + m, 32 * u + 8 * g4), d2);
          }
          const int ti = 16 * ib + m, tj = 16 * jb + 4 * g4;
          const double gi = tab.gc[ti];
          float v[4], row = 0.f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const double e = REV ? tab.gc[tj + r] - gi : gi - tab.gc[tj + r];
            const bool on = REV ? tj + r >= ti : tj + r <= ti;
            v[r] = on ? d[r] * p.inner * __builtin_amdgcn_exp2f((float)e) : 0.f;
            if constexpr (HOOK == 1) {
              d2[r] = tj + r == ti ? 0.f : v[r] * d2[r];
              row += d2[r];
            }
          }
          store4<E>(at + RA::at(ti, tj), v[0], v[1], v[2], v[3]);
          if constexpr (HOOK == 1) {
            row += __shfl_xor(row, 16, WAVE);
            row += __shfl_xor(row, 32, WAVE);
            if (g4 == 0) part[(NW + jb) * C + ti] = row;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
              for (int o = 1; o < 16; o <<= 1) d2[r] += __shfl_xor(d2[r], o, WAVE);
              if (m == 0) part[(NW + NB + ib) * C + tj + r] = d2[r];
            }
          }
        }
      }
    }

    Frag<E> zf[C / 32];
#pragma unroll
    for (int s = 0; s < C / 32; ++s) zf[s] = RZ::col(zt, 32 * s, 16 * wave, 4, lane);

    // the state's share of out
    [[maybe_unused]] floatx4 out[NB];
    if constexpr (!SUM) {
#pragma unroll
      for (int ib = 0; ib < NB; ++ib) out[ib] = floatx4{};
      if (live) {
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          float s8[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) s8[j] = S[2 * u][j], s8[4 + j] = S[2 * u + 1][j];
          const Split<E, INT> sf(s8);
#pragma unroll
          for (int ib = 0; ib < NB; ++ib) {
            const Frag<E> xf = RX::row(xt, 16 * ib + m, 32 * u + 8 * g4);
#pragma unroll
            for (int k = INT - 1; k >= 0; --k) out[ib] = mma(sf.t[k], xf, out[ib]);
          }
        }
#pragma unroll
        for (int ib = 0; ib < NB; ++ib) {
          out[ib] *= tab.fx[16 * ib + m];
          if constexpr (HOOK != 0) {
            const E* wr = wt + RZ::at(16 * ib + m, 16 * wave + 4 * g4);
            float e = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) e += out[ib][r] * to_float(wr[r]);
            e += __shfl_xor(e, 16, WAVE);
            e += __shfl_xor(e, 32, WAVE);
            if (g4 == 0) part[wave * C + 16 * ib + m] = e;
          }
        }
      }
    }

    // the state behind the chunk
    const float whole = *tab.whole;
#pragma unroll
    for (int t = 0; t < NT; ++t) S[t] *= whole;
    auto update = [&](auto n) {
      constexpr int UPD = terms<E>(decltype(n)::value);
#pragma unroll
      for (int s = 0; s < C / 32; ++s) {
        float z8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) z8[k] = to_float((E)zf[s].v[k]) * tab.fy[32 * s + 8 * g4 + k];
        const Split<E, UPD> zw(z8);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const Frag<E> yf = RX::col(yt, 32 * s, 32 * (t >> 1) + 4 * (t & 1), 8, lane);
#pragma unroll
          for (int k = UPD - 1; k >= 0; --k) S[t] = mma(yf, zw.t[k], S[t]);
        }
      }
    };
    if (whole_terms) update(Int<3>{});
    else update(Int<1>{});
    barrier_lds();  // A is whole; the tiles have been read

    if (i + 1 < count) {
      put_all();
      if (i + 2 < count) load_all(i + 2);
    }
    if constexpr (!SUM) {
      if (live) {
        // the chunk's own share
#pragma unroll
        for (int s = 0; s < C / 32; ++s)
#pragma unroll
          for (int ib = 0; ib < NB; ++ib)
            if (REV ? 2 * s + 1 >= ib : 2 * s <= ib) out[ib] = mma(zf[s], RA::row(at, 16 * ib + m, 32 * s + 8 * g4), out[ib]);
        const int rows = min(C, p.L - n * C);
        const long head = (b * p.L + (long)n * C) * p.H + h;
        const int stride = p.H * p.z.width;
        if (sizeof(E) == 2 && !p.out_f32) {
          const __amdgpu_buffer_rsrc_t r = buffer_rsrc(static_cast<bf16*>(p.out) + head * p.z.width, rows * stride * 2);
#pragma unroll
          for (int ib = 0; ib < NB; ++ib)
            buffer_store8(r, ((16 * ib + m) * stride + c0 + 16 * wave + 4 * g4) * 2,
                          bf16x4{(bf16)out[ib][0], (bf16)out[ib][1], (bf16)out[ib][2], (bf16)out[ib][3]});
        } else {
          const __amdgpu_buffer_rsrc_t r = buffer_rsrc(static_cast<float*>(p.out) + head * p.z.width, rows * stride * 4);
#pragma unroll
          for (int ib = 0; ib < NB; ++ib) buffer_store16(r, ((16 * ib + m) * stride + c0 + 16 * wave + 4 * g4) * 4, out[ib]);
        }
      }
      if constexpr (HOOK != 0) {
        if (wave == 0 && lane < C) {
          float e = 0.f;
#pragma unroll
          for (int k = 0; k < NW; ++k) e += part[k * C + lane];
          if constexpr (HOOK == 1) {
            float row = 0.f, down = 0.f;
#pragma unroll
            for (int k = 0; k < NB; ++k) row += part[(NW + k) * C + lane], down += part[(NW + NB + k) * C + lane];
            e += row - down;
          }
          p.tok[(bh * p.NT + n) * C + lane] = e;
        }
      }
    }
    barrier_lds();
  }

  float* to = SUM ? p.segs + (bh * p.P + seg) * size : p.P == 1 && p.end ? p.end + bh * size : nullptr;
  if (to && live)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = srow(t, 4 * g4 + j);
        if (row < width) to[element(row)] = S[t][j];
      }
  if (SUM && keeper && slab == 0 && lane == 0) p.decay[bh * p.P + seg] = sum;
}

template <typename E, int KW, bool REV, int HOOK, bool SUM>
hipError_t run(const LinChain& c, hipStream_t st) {
  typedef Config<E, KW, REV, HOOK, SUM> K;
  static_assert(K::LDS <= 160 * 1024, "a workgroup's LDS");
  const int tiles = c.z.width / 16, slabs = (tiles + NW - 1) / NW;
  hipLaunchKernelGGL((chain_kernel<E, KW, REV, HOOK, SUM>), dim3((unsigned)((long)c.B * c.H * c.run * slabs)), dim3(TH), K::LDS,
                     st, c);
  return hipGetLastError();
}

template <typename E, bool REV, int HOOK, bool SUM>
hipError_t by_width(const LinChain& c, hipStream_t st) {
  const int w = c.y.width;
  if (w <= 32) return run<E, 32, REV, HOOK, SUM>(c, st);
  if (w <= 64) return run<E, 64, REV, HOOK, SUM>(c, st);
  if (w <= 128) return run<E, 128, REV, HOOK, SUM>(c, st);
  if constexpr (!SUM) return run<E, 256, REV, HOOK, SUM>(c, st);
  return hipErrorInvalidValue;
}

template <typename E>
hipError_t chain(const LinChain& c, bool reverse, int hook, hipStream_t st) {
  if (reverse) return hook ? by_width<E, true, 2, false>(c, st) : by_width<E, true, 0, false>(c, st);
  return hook ? by_width<E, false, 1, false>(c, st) : by_width<E, false, 0, false>(c, st);
}
template <typename E>
hipError_t summary(const LinChain& c, bool reverse, hipStream_t st) {
  return reverse ? by_width<E, true, 0, true>(c, st) : by_width<E, false, 0, true>(c, st);
}

hipError_t chain_bf16(const LinChain& c, bool reverse, int hook, hipStream_t st);
hipError_t chain_f32(const LinChain& c, bool reverse, int hook, hipStream_t st);
hipError_t summary_bf16(const LinChain& c, bool reverse, hipStream_t st);
hipError_t summary_f32(const LinChain& c, bool reverse, hipStream_t st);

}  // namespace lin
}  // namespace delta
