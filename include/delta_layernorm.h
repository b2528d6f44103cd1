/*
 * delta_layernorm.h -- C ABI of the layer norm of the residual stream and of dropout: what a residual
 * block that normalises with a mean, or trains with dropout on its branches, needs around the mixers
 * of delta.h and delta_linear.h (the RMS norm is in delta_block.h).
 *
 * Conventions, return codes and the environment switches are those of delta.h: device pointers owned
 * by the caller, contiguous row-major tensors, work enqueued on `stream`, argument errors detected
 * before anything is enqueued, no device memory allocated, no state kept between calls.  Every call
 * can be captured into a graph.  A workspace belongs to one call at a time.  The same arguments give
 * the same bits.  Rows: 0 <= rows < 2^31, 1 <= width <= 2^20; dtype DELTA_F32 or DELTA_BF16.  Tensors of
 * rows may start at any element; the others, and workspaces, at 16 bytes.
 */
#ifndef DELTA_LAYERNORM_H
#define DELTA_LAYERNORM_H

#include "delta.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Dropout of one call.  p in [0, 1] is taken to the nearest 65536th (ties to even), d = p * 65536:
 * channel c of row r is kept if its 16 random bits are at least d, and then multiplied by
 * 65536 / (65536 - d), so that the expectation is exact; a dropped channel counts as 0 whatever it
 * holds.  The bits are those of Philox4x32-10 with the key `seed` and the counter
 * (r * ceil(width / 8) + c / 8, offset + *step), each low word first: word (c % 8) / 2, its low half
 * for even c.  They depend on nothing else, so the backward pass forms the same mask from the same
 * seed and offset; calls that are to differ take another seed or offset.
 */
typedef struct {
  double p;
  uint64_t seed, offset;
  const uint64_t* step; /* device, 8-byte aligned, read when the work runs (so that replays of a captured
                           call can draw anew); NULL counts as 0 */
} delta_dropout;

/*
 * y = dropout(x) + residual, rounded once.
 *   x, residual [rows, width] dtype; residual may be NULL for none
 *   y           [rows, width] dtype, written; may equal x or residual exactly
 * The gradient of x is the same call on the gradient of y, without a residual.  No other
 * overlap.  rows * ceil(width / 8) <= 2^34 - 2^10 (a launch's threads).
 */
int delta_layer_dropout(int64_t rows, int32_t width, int32_t dtype, const delta_dropout* drop, const void* x,
                        const void* residual, void* y, void* stream);

/*
 * Layer norm of the residual stream.  Per row
 *
 *     s = dropout(x) + residual  (rounded to dtype),   y = (s - mean(s)) / sqrt(var(s) + eps) * weight + bias
 *
 *   x, residual  [rows, width] dtype; residual may be NULL for none
 *   weight, bias [width] float32; bias may be NULL for none
 *   drop         NULL: nothing is dropped
 *   sum          [rows, width] dtype, written with s; may equal x or residual exactly.  Without a
 *                residual and with nothing dropped (drop NULL or p = 0) s is x and sum is not written
 *   y            [rows, width] dtype, written
 * The norm is that of the rounded s; var is the mean of the squared deviations.  Sums in float32 about
 * the row's mean: a row's size against its spread costs nothing beyond the rounding of s itself, but
 * sums of s, and of squared deviations, have to be float32 numbers.  eps >= 0 (with eps = 0 a constant
 * row is 0 / 0).  No other overlap.
 */
int delta_layer_layernorm(int64_t rows, int32_t width, int32_t dtype, float eps, const delta_dropout* drop, const void* x,
                          const void* residual, const float* weight, const float* bias, void* sum, void* y, void* stream);

/*
 * Backward pass of delta_layer_layernorm.  With z = (s - mean) / sqrt(var + eps), per row
 *
 *     ds = dsum + (weight dy - mean(weight dy) - z mean(weight dy z)) / sqrt(var + eps),
 *     dx = dropout(ds),   dweight = sum over rows of dy z,   dbias = sum over rows of dy
 *
 *   dy, s     [rows, width] dtype      gradient of y; the s of the forward pass
 *   weight    [width] float32
 *   drop      as in the forward pass
 *   dsum      [rows, width] dtype      gradient reaching s from the residual path, or NULL for zero
 *   dresidual [rows, width] dtype      written with ds
 *   dx        [rows, width] dtype      written, from the unrounded ds; with nothing dropped it is dresidual
 *                                      and dx is not written
 *   dweight, dbias [width] float32     written, or NULL
 *   workspace   at least delta_layer_layernorm_bwd_workspace_bytes bytes; not used
 *               where dweight and dbias are NULL
 * Outputs may not overlap the inputs, each other or the workspace.
 */
int delta_layer_layernorm_bwd_workspace_bytes(int64_t rows, int32_t width, int32_t dtype, size_t* bytes);
int delta_layer_layernorm_bwd(int64_t rows, int32_t width, int32_t dtype, float eps, const delta_dropout* drop, const void* dy,
                              const void* s, const float* weight, const void* dsum, void* dresidual, void* dx, float* dweight,
                              float* dbias, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DELTA_LAYERNORM_H */
