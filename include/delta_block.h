/*
 * delta_block.h -- C ABI of the operators a residual block needs around the delta-rule mixers of
 * delta.h: a gated linear recurrence (a second, diagonal mixer), the RMS norm of the residual
 * stream, and the clipping of the gradients a training step leaves behind.
 *
 * Conventions, return codes, delta_shape and the environment switches are those of delta.h:
 * device pointers owned by the caller, contiguous row-major tensors, work enqueued on `stream`,
 * argument errors detected before anything is enqueued, no device memory allocated, no state
 * kept between calls.  Every call's work is complete when the stream reaches its end, and all of
 * it can be captured into a graph.  A workspace belongs to one call at a time: calls (or replays
 * of captured calls) that may overlap need a workspace each, or their results are undefined
 * (they still end).  Results do not depend on the device, the stream or the timing of the call:
 * the same arguments give the same bits.
 */
#ifndef DELTA_BLOCK_H
#define DELTA_BLOCK_H

#include "delta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How the gate weighs the input of the gated linear recurrence (a = exp(g_log)). */
enum {
  DELTA_GLR_NONE = 0,       /* w = 1 */
  DELTA_GLR_COMPLEMENT = 1, /* w = 1 - a */
  DELTA_GLR_NORM = 2        /* w = sqrt(1 - a^2) (0 where a > 1) */
};

/* Tokens between the states delta_fwd_glr keeps for delta_bwd_glr. */
#define DELTA_GLR_CHUNK 64

/*
 * Gated linear recurrence over a sequence, per channel (H * dv independent channels):
 *
 *     a_t = exp(g_t),   h_t = a_t h_{t-1} + w_t x_t,   o_t = h_t
 *
 * the diagonal counterpart of the delta rule's matrix state, with the same layout, log gates and
 * float32 state.  g_t <= 0 is expected; a positive value is computed as given, also where a product
 * of several a_t, which no state takes part in, would leave float32's range.  What such a product of up
 * to 128 factors takes below 2^-126 of its value counts as 0.  g_t = -inf, or any
 * g_t whose exp is 0 in float32 (below about -87), is the hard reset: h_t = w_t x_t exactly, whatever
 * h_{t-1} holds (also infinities and NaN), so packed sequences do not see each other.  Other NaN and
 * infinite inputs propagate.
 *   s->n_h must be 1; s->dk, s->chunk and s->scale are ignored; input_gate is DELTA_GLR_*; at most
 *   2^20 channels and 2^30 tokens.  A channel's results do not depend on the batch it is in or on other
 *   channels.
 *   x       [B, L, H, dv]       dtype
 *   g_log   [B, L, H, dv]       float32
 *   h0      [B, H, dv]          float32   initial state, or NULL for zeros
 *   O       [B, L, H, dv]       dtype     written
 *   h_final [B, H, dv]          float32   written, or NULL; may equal h0 exactly (in place)
 *   states  [B, ceil(L / DELTA_GLR_CHUNK), H, dv] float32   written, or NULL: the state before
 *                                         tokens 0, 64, 128, ... (what delta_bwd_glr reads)
 *   workspace                   at least delta_fwd_glr_workspace_bytes bytes, 16-byte aligned;
 *                               contents on entry are ignored; may be NULL when that size is 0
 * State and gates are float32; each output is rounded once.  No other overlap of outputs with
 * inputs or with each other.  16-byte aligned pointers.  L = 0 writes h_final = h0 (or zeros).
 */
int delta_fwd_glr_workspace_bytes(const delta_shape* s, size_t* bytes);
int delta_fwd_glr(const delta_shape* s, int32_t input_gate, const void* x, const float* g_log, const float* h0,
                  void* O, float* h_final, float* states, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward pass of delta_fwd_glr: the gradients of <O, dO> + <h_final, dh_final>.  With
 * lambda_t = dO_t + a_{t+1} lambda_{t+1} (the last token's also gets dh_final),
 *
 *     dx_t = w_t lambda_t,  dg_t = lambda_t (a_t h_{t-1} + w'_t x_t),  dh0 = a_1 lambda_1,
 *
 * w' = dw/dg = 0, -a or -a^2 / w (taken as 0 where w = 0).  h is recomputed from `states` and equals
 * the forward pass's to within float32 rounding.  At a hard reset dg = 0 and nothing flows back.
 *   x, g_log, states             as passed to and written by delta_fwd_glr
 *   dO       [B, L, H, dv]       dtype
 *   dh_final [B, H, dv]          float32   or NULL for zero
 *   dx, dg_log [B, L, H, dv]     float32   written
 *   dh0      [B, H, dv]          float32   written, or NULL
 *   workspace                    as above, delta_bwd_glr_workspace_bytes
 * Outputs may not overlap the inputs, each other or the workspace.
 */
int delta_bwd_glr_workspace_bytes(const delta_shape* s, size_t* bytes);
int delta_bwd_glr(const delta_shape* s, int32_t input_gate, const void* x, const float* g_log, const float* states,
                  const void* dO, const float* dh_final, float* dx, float* dg_log, float* dh0, void* workspace,
                  size_t workspace_bytes, void* stream);

/*
 * One token of the recurrence, the state updated in place (s->L must be 1).
 *   x [B, 1, H, dv] dtype; g_log [B, 1, H, dv] float32; h [B, H, dv] float32, read and written;
 *   O [B, 1, H, dv] dtype, written.  No overlap of h or O with an input or each other.
 */
int delta_decode_glr(const delta_shape* s, int32_t input_gate, const void* x, const float* g_log, float* h, void* O,
                     void* stream);

/*
 * RMS norm of the residual stream, the step before a layer's projections.  Per row of `width`
 * channels (1 <= width <= 2^20; rows >= 0; dtype DELTA_F32 or DELTA_BF16):
 *
 *     s = x + residual  (rounded to dtype),   y = s / sqrt(mean(s^2) + eps) * weight
 *
 *   x        [rows, width] dtype
 *   residual [rows, width] dtype, or NULL: then s is x itself and `sum` is not written
 *   weight   [width] float32
 *   sum      [rows, width] dtype, written with s; may equal x or residual exactly
 *   y        [rows, width] dtype, written
 * The norm is that of the rounded s, the value the next layer adds to and the backward pass
 * reads.  Sums in float32, so a row's sum of squares has to be one: of rows longer than 1.8e19 (the
 * 2-norm) it is infinite and y is 0, and with eps = 0 rows shorter than 1e-19 count as zeros.  16-byte
 * aligned pointers; no other overlap.  eps >= 0.
 */
int delta_layer_rmsnorm(int64_t rows, int32_t width, int32_t dtype, float eps, const void* x, const void* residual,
                        const float* weight, void* sum, void* y, void* stream);

/*
 * The same norm with its output in 8 bits (OCP e4m3, largest value 448), for projections that
 * take 8-bit operands: per group of `group` consecutive channels of a row (the last group may be
 * shorter), from the unrounded y,
 *
 *     scale = max|y| / 448,   y8 = e4m3(y / scale)  (to nearest, ties to even)
 *
 * A group whose largest |y| is below 2^-100 gets scale 0 and zeros.  A NaN or infinity makes its
 * group's scale NaN or infinite, and so every product of that scale with y8 NaN or infinite.
 *   group  0 (one scale per row) or 128
 *   y8     [rows, width] one byte each, written
 *   scale  [rows, ceil(width / group)] float32 ([rows] for group 0), written; 4-byte aligned
 * Otherwise as delta_layer_rmsnorm.
 */
int delta_layer_rmsnorm_quant(int64_t rows, int32_t width, int32_t dtype, float eps, int32_t group, const void* x,
                              const void* residual, const float* weight, void* sum, void* y8, float* scale,
                              void* stream);

/*
 * Backward pass of delta_layer_rmsnorm.  With r = 1 / sqrt(mean(s^2) + eps), per row
 *
 *     dx = dsum + r weight dy - s r^3 mean(weight dy s),    dweight = sum over rows of dy s r
 *
 * dx is the gradient of x and of residual alike.
 *   dy, s   [rows, width] dtype      gradient of y; the s of the forward pass
 *   weight  [width] float32
 *   dsum    [rows, width] dtype      gradient reaching s from the residual path, or NULL for zero
 *   dx      [rows, width] dtype      written
 *   dweight [width] float32          written, or NULL
 *   workspace   at least delta_layer_rmsnorm_bwd_workspace_bytes bytes, 16-byte aligned; not used where
 *               dweight is NULL
 * Outputs may not overlap the inputs, each other or the workspace.
 */
int delta_layer_rmsnorm_bwd_workspace_bytes(int64_t rows, int32_t width, int32_t dtype, size_t* bytes);
int delta_layer_rmsnorm_bwd(int64_t rows, int32_t width, int32_t dtype, float eps, const void* dy, const void* s,
                            const float* weight, const void* dsum, void* dx, float* dweight, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * The global norm of a set of gradients, and their clipping by it:
 *
 *     norm = sqrt(sum over all elements of g^2),   c = min(1, max_norm / (norm + eps)),   out = c g
 *
 * n tensors, described by host arrays read during the call: grads[i] a device pointer (aligned to
 * its element only), sizes[i] >= 0 its elements, dtypes[i] DELTA_F32 or DELTA_BF16.  The sum is
 * held in 64 bits.  A NaN or infinity in any gradient reaches norm (and, as c, every output).
 *   norm   one float32, device, written
 *   out    host array of n device pointers, or NULL to clip in place; out[i] may equal grads[i].
 *          No other overlap between outputs, or between an output and a gradient (a tensor may
 *          not be listed twice).
 *   max_norm >= 0, eps >= 0
 *   workspace   at least delta_grad_norm_workspace_bytes bytes, 16-byte aligned.  The size depends on
 *               how many tensors there are and on each one's size, not on their total alone; it never
 *               falls when a tensor is added or one grows
 */
int delta_grad_norm_workspace_bytes(int32_t n, const int64_t* sizes, size_t* bytes);
int delta_grad_norm(int32_t n, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, float* norm,
                    void* workspace, size_t workspace_bytes, void* stream);
int delta_clip_grads(int32_t n, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, float max_norm,
                     float eps, void* const* out, float* norm, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DELTA_BLOCK_H */
