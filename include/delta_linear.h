/*
 * delta_linear.h -- C ABI of linear attention with a decay for each head: the mixer that the delta
 * rule of delta.h becomes without its erase term.
 *
 *     S_t = a_t S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t,   a_t = exp(g_t)
 *
 * Conventions, return codes, delta_shape and the environment switches are those of delta.h: device
 * pointers owned by the caller, contiguous row-major tensors, work enqueued on `stream`, argument
 * errors detected before anything is enqueued, no device memory allocated, no state kept between
 * calls.  Every call can be captured into a graph.  A workspace belongs to one call at a time: calls
 * (or replays of captured calls) that may overlap need a workspace each.  The same arguments give the
 * same bits, whatever the device's load or the call's timing.
 *
 * Shapes: s->n_h must be 1, s->chunk is ignored, dk in {16, 32, 64, 128}, dv a multiple of 16 up to
 * 256, H * max(dk, dv) <= 2^20, B * H <= 2^20, B * H * dk * dv <= 2^33, L <= 2^30.  `qk_heads` heads of q
 * and k, which divides H: value head h reads query and key head h / (H / qk_heads).
 *
 * Gates: log decays in float32, one of DELTA_LIN_GATE_*.  g <= 0 is expected; a positive value is
 * computed as given, as long as the products of the gates within a chunk of 64 tokens (up to the next
 * reset) and the states themselves stay in float32's range.  g = -inf, or any g whose exp is 0 in float32
 * (below -103.972), is the hard reset: the state before it is multiplied by an exact 0, whatever gates follow.  Non-finite q, k or v propagate as in delta_fwd: such a value in one
 * chunk reaches that chunk's outputs and every later state and output of its sequence and head, and
 * nothing before the chunk nor any other sequence or head that does not read it.
 */
#ifndef DELTA_LINEAR_H
#define DELTA_LINEAR_H

#include "delta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What g_log holds. */
enum {
  DELTA_LIN_GATE_NONE = 0,  /* g_log is NULL: a = 1 */
  DELTA_LIN_GATE_TOKEN = 1, /* [B, L, H]: a gate for each token and head */
  DELTA_LIN_GATE_HEAD = 2   /* [H]: a fixed decay for each head */
};

/*
 * Forward pass over a sequence.
 *   q, k    [B, L, qk_heads, dk] dtype;  v [B, L, H, dv] dtype
 *   S0      [B, H, dk, dv] float32   initial state, or NULL for zeros
 *   O       [B, L, H, dv] dtype      written
 *   S_final [B, H, dk, dv] float32   written, or NULL; may equal S0 exactly (in place)
 *   workspace   at least delta_fwd_lin_workspace_bytes bytes, 16-byte aligned; contents on entry are
 *               ignored; may be NULL when that size is 0.  The size never falls with L: a workspace for the
 *               longest sequence serves shorter ones of the same B, heads, widths and type
 * States are float32, as if from float32 products, in either type; O is rounded once, from products
 * of operands in the inputs' type summed in float32 (for bf16 the state and the pairs' weights are
 * rounded to bf16 as operands).  No other overlap of outputs with inputs or with each other; 16-byte aligned
 * pointers (g_log: 4).  L = 0 writes S_final = S0 (or zeros).
 */
int delta_fwd_lin_workspace_bytes(const delta_shape* s, int32_t qk_heads, size_t* bytes);
int delta_fwd_lin(const delta_shape* s, int32_t qk_heads, int32_t gate, const void* q, const void* k, const void* v,
                  const float* g_log, const float* S0, void* O, float* S_final, void* workspace, size_t workspace_bytes,
                  void* stream);

/*
 * Backward pass of delta_fwd_lin for the same arguments: the gradients of <O, dO> + <S_final, dS_final>.
 * The forward pass's states are formed again.  With G_t the gradient of S_t,
 *
 *     G_t = scale q_t dO_t^T + a_{t+1} G_{t+1},   dq_t = scale S_t dO_t,   dk_t = G_t v_t,
 *     dv_t = G_t^T k_t,   dg_t = a_t <G_t, S_{t-1}>,   dS0 = a_1 G_1
 *
 * Precision as the forward pass's.  For bf16 with dg_log, dq and dk take the state's operands as three bf16 terms
 * (as good as float32), without it as one: dq's and dk's last bits depend on whether dg_log is asked for.
 *   dO       [B, L, H, dv] dtype
 *   dS_final [B, H, dk, dv] float32   or NULL for zero
 *   dq, dk   [B, L, qk_heads, dk] dtype   written: the sums over the heads that share them, rounded once
 *   dv       [B, L, H, dv] dtype          written
 *   dg_log   as g_log, float32            written, or NULL; must be NULL for DELTA_LIN_GATE_NONE
 *   dS0      [B, H, dk, dv] float32       written, or NULL
 *   workspace   as above, delta_bwd_lin_workspace_bytes.  With gates it holds a state for each chunk (64 tokens,
 *               float32 32); a call without dg_log takes the size for DELTA_LIN_GATE_NONE
 * At a hard reset dg = 0 and nothing flows back.  dg_t is formed from the states before and the gradients
 * behind its chunk and the pairs of tokens around t, so its error goes by the magnitudes that cross
 * t, whatever the sequence holds elsewhere.  A fixed decay's gradient is the sum of such terms over all
 * tokens and sequences, added up in 64 bits.  Outputs may not overlap the inputs, each other or the workspace.
 */
int delta_bwd_lin_workspace_bytes(const delta_shape* s, int32_t qk_heads, int32_t gate, size_t* bytes);
int delta_bwd_lin(const delta_shape* s, int32_t qk_heads, int32_t gate, const void* q, const void* k, const void* v,
                  const float* g_log, const float* S0, const void* dO, const float* dS_final, void* dq, void* dk, void* dv,
                  float* dg_log, float* dS0, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token (s->L must be 1), the state updated in place: S [B, H, dk, dv] float32, read and written;
 * O [B, 1, H, dv] dtype, written.  No overlap of S or O with an input or each other.
 */
int delta_decode_lin(const delta_shape* s, int32_t qk_heads, int32_t gate, const void* q, const void* k, const void* v,
                     const float* g_log, float* S, void* O, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DELTA_LINEAR_H */
