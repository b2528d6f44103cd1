// Launch interface between the linear attention entry points (linear_abi.cpp) and their kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace delta {

enum { LIN_GATE_NONE = 0, LIN_GATE_TOKEN = 1, LIN_GATE_HEAD = 2 };

constexpr int LIN_SLAB = 128;  // columns of a workgroup's state at most

// What a chain forms beside its outputs (linear_chain.h)
enum { LIN_PLAIN = 0, LIN_PAIRS = 1, LIN_SUMS = 2, LIN_STATE = 3 };

// Tokens of a chunk: float32 tiles are twice as large, and their products run at a sixteenth of the rate.
constexpr int lin_chunk(bool bf16) { return bf16 ? 64 : 32; }

// Rows that a chain's registers hold for a state of `rows`, and the bytes of such a state as they hold it (linear_chain.h):
// 16 x 16 tiles, an even number of them across.
constexpr int lin_rows(int rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256; }
constexpr size_t lin_state_bytes(int rows, int cols) { return (size_t)((cols / 16 + 1) / 2 * 2) * (lin_rows(rows) / 16) * 1024; }

// Chunks of a workgroup of the gates' gradients.
constexpr int LIN_GATE_CHUNKS = 16;

// A log gate as a term of a chunk's sums.  One whose exp is 0 in float32 (below ln 2^-150) is a hard reset, and so far
// from the others that no chunk of 64 gates whose products are float32 numbers makes up for it: the exp of a sum with
// a reset in it is 0.  Differences of such sums are still good to 2^-29.
constexpr double LIN_RESET = -131072.0;
__device__ inline double lin_log_gate(float g) { return g < -103.972076f ? LIN_RESET : (double)g; }

// One operand of a chain: [B, L, heads, width], head h of the chain reading head h / (H / heads).
struct LinRole {
  const void* p;
  int heads, width;
};

// One chain over chunks (linear.hip has the formulas).  The state's rows are x's and y's width, its
// columns z's; it is stored [rows][cols], or [cols][rows] where `flip`.
struct LinChain {
  int B, L, H, NT, P, NS;  // chunks in all, segments, chunks of a segment
  int run;                 // segments of this launch: P, or fewer for a summary whose end nobody asks for
  LinRole x, y, z, w;      // w: PAIRS and SUMS only
  const float* g;          // [B, L, H], [H] or nullptr
  int gate;
  float outer, inner, write;  // scales of the state's share of out, of the chunk's share, of what the state takes in
  const float* start;      // [B, H] states before the first segment in the chain's order, or nullptr
  float* segs;             // P > 1: [B, H, P] states, the summary's results and then each segment's start
  double* decay;           // P > 1: [B, H, P] sums of log gates
  float* end;              // [B, H] states behind the last segment: form STATE, or the summary's (or nullptr)
  bool flip;
  void* out;               // [B, L, H, z.width] in the inputs' type, or float32
  bool out_f32;
  float* tok;              // PAIRS, SUMS: [B, H, NT chunks] a value per token
  float* pair;             // PAIRS: the same of the pairs within its chunk
  int part;                // of a backward pass: 0 the whole walk, 1 the first half of its chunks, 2 the rest
  float* wait;             // part 1, 2: [B, H, P] states between the two, as the registers hold them
  float *states, *edge;    // PAIRS, SUMS: [B, H, NT] states left by the one for the other; e^gc_C <S, G> of the chunk
};

// Gradients of the log gates from what the two backward chains left.
struct LinGates {
  int B, L, H, C, NT;
  const float *e, *f, *pair;  // [B, H, NT * C]
  const float* edge;          // [B, H, NT]
  const float* g;
  int gate;
  float* dg;                  // [B, L, H], or [H] through `part`
  double* part;               // gate HEAD: [B, H, workgroups of a head]
};

struct LinDecode {
  int B, H, Hk, DK, DV, gate;
  float scale;
  const void *q, *k, *v;
  const float* g;
  float* S;
  void* O;
};

// Chunks, segments, chunks of a segment; and the most segments of any sequence of up to this length.
void lin_split(int B, int L, int H, int dv, bool bf16, bool backward, int& NT, int& P, int& NS, int& most_segments);
// bf16 inputs in one file, float32 in another
hipError_t lin_chain_bf16(const LinChain& c, bool reverse, int form, hipStream_t st);
hipError_t lin_chain_f32(const LinChain& c, bool reverse, int form, hipStream_t st);
hipError_t lin_summary_bf16(const LinChain& forward, const LinChain* reverse, hipStream_t st);
hipError_t lin_summary_f32(const LinChain& forward, const LinChain* reverse, hipStream_t st);
hipError_t lin_backward_bf16(const LinChain& dq, const LinChain& dv, const LinChain& dk, bool gates, bool state, hipStream_t st);
hipError_t lin_backward_f32(const LinChain& dq, const LinChain& dv, const LinChain& dk, bool gates, bool state, hipStream_t st);

inline hipError_t launch_lin_chain(const LinChain& c, bool bf16, bool reverse, int form, hipStream_t st) {
  return bf16 ? lin_chain_bf16(c, reverse, form, st) : lin_chain_f32(c, reverse, form, st);
}
// Each segment's state from zero, of `forward` and (unless nullptr) `reverse` in one launch; either may have run = 0.
inline hipError_t launch_lin_summary(const LinChain& forward, const LinChain* reverse, bool bf16, hipStream_t st) {
  return bf16 ? lin_summary_bf16(forward, reverse, st) : lin_summary_f32(forward, reverse, st);
}
// The three chains of a backward pass side by side in one launch, forms PAIRS, PLAIN and SUMS, or all PLAIN without `gates`;
// dv's STATE with `state`.  Only for values of up to 128 channels.  A chain with run = 0 is left out.
inline hipError_t launch_lin_backward(const LinChain& dq, const LinChain& dv, const LinChain& dk, bool gates, bool state, bool bf16,
                                      hipStream_t st) {
  return bf16 ? lin_backward_bf16(dq, dv, dk, gates, state, st) : lin_backward_f32(dq, dv, dk, gates, state, st);
}
// The segments' results become their starts, of both chains (either nullptr).
hipError_t launch_lin_combine(const LinChain* forward, const LinChain* reverse, hipStream_t st);
hipError_t launch_lin_gates(const LinGates& p, hipStream_t st);
// The parts of dq and of dk, each [rows, heads, share, width], added up over `share`.
hipError_t launch_lin_share(const float* dq_part, const float* dk_part, void* dq, void* dk, long rows, int heads, int share, int width,
                            bool bf16, hipStream_t st);
hipError_t launch_lin_decode(const LinDecode& p, bool bf16, hipStream_t st);

}  // namespace delta
