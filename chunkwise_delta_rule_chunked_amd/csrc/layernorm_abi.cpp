// C ABI of the layer norm and of dropout (include/delta_layernorm.h): argument validation and dispatch, in the
// manner of block_abi.cpp.  Nothing here throws or allocates.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/delta_layernorm.h"
#include "abi_common.h"
#include "layernorm.h"

using delta::DropoutParams;
using delta::DropRule;
using delta::LayernormParams;
using namespace delta::abi;

namespace {

int rows_shape(int64_t rows, int32_t width, int32_t dtype, float eps) {
  if (rows < 0 || rows > 0x7fffffff || width < 1 || width > (1 << 20) || !(eps >= 0.f)) return DELTA_ERR_BAD_SHAPE;
  if (dtype != DELTA_F32 && dtype != DELTA_BF16) return DELTA_ERR_UNSUPPORTED_DIM;
  return DELTA_OK;
}

int drop_rule(const delta_dropout* d, DropRule& r) {
  memset(&r, 0, sizeof(r));
  if (!d) return DELTA_OK;
  if (!(d->p >= 0.0 && d->p <= 1.0)) return DELTA_ERR_BAD_SHAPE;
  if (!aligned(d->step, 8)) return DELTA_ERR_MISALIGNED;
  r.drop = (uint32_t)nearbyint(d->p * 65536.0);
  r.scale = r.drop == 65536 ? 0.f : (float)(65536.0 / (65536 - (int)r.drop));
  r.seed = d->seed, r.offset = d->offset, r.step = d->step;
  return DELTA_OK;
}

// Rows may start at any element, the other tensors at 16 bytes.
template <int NR, int NT>
int check_aligned(int32_t dtype, const void* const (&rows)[NR], const void* const (&tensors)[NT]) {
  for (const void* p : rows)
    if (!aligned(p, (unsigned)esize(dtype))) return DELTA_ERR_MISALIGNED;
  for (const void* p : tensors)
    if (!aligned16(p)) return DELTA_ERR_MISALIGNED;
  return DELTA_OK;
}

Range span(const void* p, size_t bytes) { return range(p, p ? bytes : 0); }

}  // namespace

extern "C" {

int delta_layer_dropout(int64_t rows, int32_t width, int32_t dtype, const delta_dropout* drop, const void* x,
                        const void* residual, void* y, void* stream) {
  int rc = rows_shape(rows, width, dtype, 0.f);
  if (rc) return rc;
  if (!drop) return DELTA_ERR_NULL_ARG;
  // one launch has fewer than 2^32 threads, four vectors of eight channels each
  if (rows * ((width + 7LL) / 8) > (1LL << 34) - 1024) return DELTA_ERR_BAD_SHAPE;
  DropoutParams p;
  if ((rc = drop_rule(drop, p.rule))) return rc;
  if (rows == 0) return DELTA_OK;
  if (!x || !y) return DELTA_ERR_NULL_ARG;
  if ((rc = check_aligned(dtype, {x, residual, y}, {nullptr}))) return rc;
  const size_t n = (size_t)rows * width * esize(dtype);
  const Range in[] = {span(y == x ? nullptr : x, n), span(y == residual ? nullptr : residual, n), span(p.rule.step, 8)};
  const Range out[] = {span(y, n)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  if ((rc = launch_guard())) return rc;
  p.rows = rows, p.width = width, p.x = x, p.res = residual, p.y = y;
  return hip_status(delta::launch_dropout(p, dtype == DELTA_BF16, static_cast<hipStream_t>(stream)));
}

int delta_layer_layernorm(int64_t rows, int32_t width, int32_t dtype, float eps, const delta_dropout* drop, const void* x,
                          const void* residual, const float* weight, const float* bias, void* sum, void* y, void* stream) {
  int rc = rows_shape(rows, width, dtype, eps);
  if (rc) return rc;
  LayernormParams p;
  memset(&p, 0, sizeof(p));
  if ((rc = drop_rule(drop, p.rule))) return rc;
  if (rows == 0) return DELTA_OK;
  if (!residual && !p.rule.drop) sum = nullptr;
  if (!x || !weight || !y || ((residual || p.rule.drop) && !sum)) return DELTA_ERR_NULL_ARG;
  if ((rc = check_aligned(dtype, {x, residual, sum, y}, {weight, bias}))) return rc;
  const size_t n = (size_t)rows * width * esize(dtype), nw = (size_t)width * 4;
  // sum may be x or residual itself (each vector is read by the lane that writes it, before)
  const Range in[] = {span(sum && sum == x ? nullptr : x, n), span(sum && sum == residual ? nullptr : residual, n),
                      span(weight, nw), span(bias, nw), span(p.rule.step, 8)};
  const Range out[] = {span(sum, n), span(y, n)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  if ((rc = launch_guard())) return rc;
  p.rows = rows, p.width = width, p.eps = eps, p.x = x, p.res = residual, p.weight = weight, p.bias = bias, p.sum = sum, p.y = y;
  return hip_status(delta::launch_layernorm(p, dtype == DELTA_BF16, static_cast<hipStream_t>(stream)));
}

int delta_layer_layernorm_bwd_workspace_bytes(int64_t rows, int32_t width, int32_t dtype, size_t* bytes) {
  const int rc = rows_shape(rows, width, dtype, 0.f);
  if (rc) return rc;
  if (!bytes) return DELTA_ERR_NULL_ARG;
  *bytes = align_up((size_t)delta::layernorm_bwd_parts(rows, width) * width * 8);
  return DELTA_OK;
}

int delta_layer_layernorm_bwd(int64_t rows, int32_t width, int32_t dtype, float eps, const delta_dropout* drop, const void* dy,
                              const void* s, const float* weight, const void* dsum, void* dresidual, void* dx, float* dweight,
                              float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = rows_shape(rows, width, dtype, eps);
  if (rc) return rc;
  LayernormParams p;
  memset(&p, 0, sizeof(p));
  if ((rc = drop_rule(drop, p.rule))) return rc;
  if (!p.rule.drop) dx = nullptr;
  if (rows > 0 && (!dy || !s || !weight || !dresidual || (p.rule.drop && !dx))) return DELTA_ERR_NULL_ARG;
  size_t need = 0;  // the workspace holds the parts of dweight and dbias
  if (dweight || dbias) delta_layer_layernorm_bwd_workspace_bytes(rows, width, dtype, &need);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DELTA_ERR_WORKSPACE;
  if ((rc = check_aligned(dtype, {dy, s, dsum, dresidual, dx}, {weight, dweight, dbias, workspace}))) return rc;
  const size_t n = (size_t)rows * width * esize(dtype), nw = (size_t)width * 4;
  const Range in[] = {span(dy, n), span(s, n), span(weight, nw), span(dsum, n), span(p.rule.step, 8)};
  const Range out[] = {span(dresidual, n), span(dx, n), span(dweight, nw), span(dbias, nw), span(workspace, need)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  if (rows == 0 && !dweight && !dbias) return DELTA_OK;
  if ((rc = launch_guard())) return rc;
  p.rows = rows, p.width = width, p.eps = eps, p.x = s, p.weight = weight, p.dy = dy, p.dsum = dsum;
  p.dres = dresidual, p.dx = dx, p.dweight = dweight, p.dbias = dbias, p.part = static_cast<float*>(workspace);
  return hip_status(delta::launch_layernorm_bwd(p, dtype == DELTA_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
