// C ABI of the residual-block operators (include/delta_block.h): argument validation, workspace
// layout and kernel dispatch, in the manner of delta_abi.cpp.  Nothing here throws or allocates
// device memory.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <memory>
#include <new>

#include "../../include/delta_block.h"
#include "abi_common.h"
#include "block_kernels.h"

using delta::ClipTable;
using delta::GlrParams;
using delta::RmsnormParams;
using namespace delta::abi;

static_assert(DELTA_GLR_CHUNK == delta::GLR_CHUNK, "the kept states' spacing is part of the interface");

namespace {

// ---- gated linear recurrence ----

struct GlrSizes {
  size_t x, g, state, states;  // bytes of x/O/dO, of g/dx/dg, of one state, of the kept states
};

int glr_shape(const delta_shape* s, int32_t gate, GlrParams& p, GlrSizes& z) {
  if (!s) return DELTA_ERR_NULL_ARG;
  delta_shape t = *s;
  t.dk = 16;  // not used by this recurrence
  const int rc = check_shape(&t);
  if (rc) return rc;
  if (s->n_h != 1) return DELTA_ERR_BAD_SHAPE;
  if (gate != DELTA_GLR_NONE && gate != DELTA_GLR_COMPLEMENT && gate != DELTA_GLR_NORM) return DELTA_ERR_UNSUPPORTED_DIM;
  const long long D = (long long)s->H * s->dv;
  if (D > (1LL << 20) || !delta::glr_grid_fits(s->B, s->L, (int)D)) return DELTA_ERR_BAD_SHAPE;
  memset(&p, 0, sizeof(p));
  p.B = s->B, p.L = s->L, p.D = (int)D, p.gate = gate;
  const size_t n = (size_t)s->B * s->L * D;
  z.x = n * esize(s->dtype), z.g = n * 4, z.state = (size_t)s->B * D * 4;
  z.states = z.state * (((size_t)s->L + delta::GLR_CHUNK - 1) / delta::GLR_CHUNK);
  return DELTA_OK;
}

// ---- gradients ----

struct Clip {
  int64_t pieces;
  int64_t parts;  // at most: every launch but the last takes CLIP_TENSORS tensors
};

int clip_sizes(int32_t n, const int64_t* sizes, Clip& c) {
  if (n < 0) return DELTA_ERR_BAD_SHAPE;
  if (n > 0 && !sizes) return DELTA_ERR_NULL_ARG;
  c.pieces = 0;
  for (int i = 0; i < n; ++i) {
    if (sizes[i] < 0 || sizes[i] > (1LL << 40)) return DELTA_ERR_BAD_SHAPE;
    c.pieces += (sizes[i] + delta::CLIP_PIECE - 1) / delta::CLIP_PIECE;
    if (c.pieces > 0x7fffffff) return DELTA_ERR_BAD_SHAPE;
  }
  int64_t m = 0;
  for (int i = 0; i < n; ++i) m += sizes[i] > 0;
  c.parts = std::min<int64_t>(c.pieces, (m + delta::CLIP_TENSORS - 1) / delta::CLIP_TENSORS * delta::CLIP_PARTS);
  return DELTA_OK;
}

// Fills `t` from tensor `i` on; returns the next tensor to take (n when all are in).
int fill_table(ClipTable& t, int i, int n, const void* const* grads, void* const* out, const int64_t* sizes,
               const int32_t* dtypes) {
  memset(t.bf16, 0, sizeof(t.bf16));
  int m = 0;
  int32_t pieces = 0;
  for (; i < n && m < delta::CLIP_TENSORS; ++i) {
    if (sizes[i] == 0) continue;
    t.g[m] = grads[i];
    t.out[m] = out ? out[i] : const_cast<void*>(grads[i]);
    t.n[m] = sizes[i];
    t.first[m] = pieces;
    if (dtypes[i] == DELTA_BF16) t.bf16[m / 32] |= 1u << (m % 32);
    pieces += (int32_t)((sizes[i] + delta::CLIP_PIECE - 1) / delta::CLIP_PIECE);
    ++m;
  }
  t.first[m] = pieces;
  t.count = m;
  return i;
}

int run_clip(int32_t n, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, bool scale,
             float max_norm, float eps, void* const* out, float* norm, void* workspace, size_t workspace_bytes,
             void* stream) {
  Clip c;
  int rc = clip_sizes(n, sizes, c);
  if (rc) return rc;
  if ((n > 0 && (!grads || !dtypes)) || !norm) return DELTA_ERR_NULL_ARG;
  if (scale && (!(max_norm >= 0.f) || !(eps >= 0.f))) return DELTA_ERR_BAD_SHAPE;
  for (int i = 0; i < n; ++i) {
    if (dtypes[i] != DELTA_F32 && dtypes[i] != DELTA_BF16) return DELTA_ERR_UNSUPPORTED_DIM;
    if (sizes[i] > 0 && (!grads[i] || (out && !out[i]))) return DELTA_ERR_NULL_ARG;
    const unsigned es = (unsigned)esize(dtypes[i]);
    if (!aligned(grads[i], es) || (out && !aligned(out[i], es))) return DELTA_ERR_MISALIGNED;
  }
  if (!aligned(norm, 4) || !aligned16(workspace)) return DELTA_ERR_MISALIGNED;
  size_t need = 0;
  delta_grad_norm_workspace_bytes(n, sizes, &need);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DELTA_ERR_WORKSPACE;
  // what is written may overlap nothing else: neighbours in address order are enough to look at,
  // an output that is its own gradient standing for both
  struct Region {
    Range r;
    bool written;
  };
  const size_t count = 2 * (size_t)n + 2;
  std::unique_ptr<Region[]> all(new (std::nothrow) Region[count]);
  if (!all) return DELTA_ERR_HIP;
  size_t m = 0;
  all[m++] = {range(norm, 4), true};
  if (need) all[m++] = {range(workspace, need), true};
  for (int i = 0; i < n; ++i) {
    const size_t b = (size_t)sizes[i] * esize(dtypes[i]);
    if (b == 0) continue;
    const void* o = scale ? (out ? out[i] : grads[i]) : nullptr;
    if (o) all[m++] = {range(o, b), true};
    if (o != grads[i]) all[m++] = {range(grads[i], b), false};
  }
  std::sort(all.get(), all.get() + m, [](const Region& a, const Region& b) { return a.r.lo < b.r.lo; });
  uintptr_t hi = 0, hi_written = 0;  // ends of everything, and of what is written, so far
  for (size_t i = 0; i < m; ++i) {
    if (all[i].r.lo < (all[i].written ? hi : hi_written)) return DELTA_ERR_ALIAS;
    hi = std::max(hi, all[i].r.hi);
    if (all[i].written) hi_written = std::max(hi_written, all[i].r.hi);
  }
  if ((rc = launch_guard())) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  double* sums = static_cast<double*>(workspace);
  ClipTable t;
  int parts = 0, tables = 0;
  for (int i = 0; i < n; ++tables) {
    i = fill_table(t, i, n, grads, out, sizes, dtypes);
    if (t.count == 0) break;
    const int np = delta::clip_parts(t.first[t.count]);
    if ((rc = hip_status(delta::launch_grad_sums(t, sums + parts, np, st)))) return rc;
    parts += np;
  }
  // all tensors in one table: the scaling adds the sums up itself
  if (scale && tables <= 1) {
    fill_table(t, 0, n, grads, out, sizes, dtypes);
    return hip_status(delta::launch_grad_scale(t, sums, parts, max_norm, eps, norm, st));
  }
  if ((rc = hip_status(delta::launch_grad_finish(sums, parts, norm, st)))) return rc;
  for (int i = 0; scale && i < n;) {
    i = fill_table(t, i, n, grads, out, sizes, dtypes);
    if (t.count && (rc = hip_status(delta::launch_grad_scale(t, sums, -1, max_norm, eps, norm, st)))) return rc;
  }
  return DELTA_OK;
}

}  // namespace

extern "C" {

int delta_fwd_glr_workspace_bytes(const delta_shape* s, size_t* bytes) {
  GlrParams p;
  GlrSizes z;
  const int rc = glr_shape(s, DELTA_GLR_NONE, p, z);
  if (rc) return rc;
  if (!bytes) return DELTA_ERR_NULL_ARG;
  *bytes = delta::glr_workspace(p.B, p.L, p.D, false);
  return DELTA_OK;
}

int delta_fwd_glr(const delta_shape* s, int32_t input_gate, const void* x, const float* g_log, const float* h0,
                  void* O, float* h_final, float* states, void* workspace, size_t workspace_bytes, void* stream) {
  GlrParams p;
  GlrSizes z;
  int rc = glr_shape(s, input_gate, p, z);
  if (rc) return rc;
  if (z.x > 0 && (!x || !g_log || !O)) return DELTA_ERR_NULL_ARG;
  size_t need = 0;
  delta_fwd_glr_workspace_bytes(s, &need);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DELTA_ERR_WORKSPACE;
  const void* ptrs[] = {x, g_log, h0, O, h_final, states, workspace};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return DELTA_ERR_MISALIGNED;
  const bool in_place = h0 && h0 == h_final;
  const Range in[] = {range(x, x ? z.x : 0), range(g_log, g_log ? z.g : 0), range(h0, h0 && !in_place ? z.state : 0)};
  const Range out[] = {range(O, O ? z.x : 0), range(h_final, h_final ? z.state : 0), range(states, states ? z.states : 0),
                       range(workspace, need)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  if (z.state == 0 || (s->L == 0 && !h_final)) return DELTA_OK;
  if ((rc = launch_guard())) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (validate_on() && (rc = validate_gates(g_log, z.g / 4, st))) return rc;
  p.x = x, p.g = g_log, p.h0 = h0, p.O = O, p.h_final = h_final, p.states = states;
  p.ws = workspace;
  return hip_status(delta::launch_glr_fwd(p, s->dtype == DELTA_BF16, st));
}

int delta_bwd_glr_workspace_bytes(const delta_shape* s, size_t* bytes) {
  GlrParams p;
  GlrSizes z;
  const int rc = glr_shape(s, DELTA_GLR_NONE, p, z);
  if (rc) return rc;
  if (!bytes) return DELTA_ERR_NULL_ARG;
  *bytes = delta::glr_workspace(p.B, p.L, p.D, true);
  return DELTA_OK;
}

int delta_bwd_glr(const delta_shape* s, int32_t input_gate, const void* x, const float* g_log, const float* states,
                  const void* dO, const float* dh_final, float* dx, float* dg_log, float* dh0, void* workspace,
                  size_t workspace_bytes, void* stream) {
  GlrParams p;
  GlrSizes z;
  int rc = glr_shape(s, input_gate, p, z);
  if (rc) return rc;
  if (z.x > 0 && (!x || !g_log || !states || !dO || !dx || !dg_log)) return DELTA_ERR_NULL_ARG;
  size_t need = 0;
  delta_bwd_glr_workspace_bytes(s, &need);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DELTA_ERR_WORKSPACE;
  const void* ptrs[] = {x, g_log, states, dO, dh_final, dx, dg_log, dh0, workspace};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return DELTA_ERR_MISALIGNED;
  const Range in[] = {range(x, x ? z.x : 0), range(g_log, g_log ? z.g : 0), range(states, states ? z.states : 0),
                      range(dO, dO ? z.x : 0), range(dh_final, dh_final ? z.state : 0)};
  const Range out[] = {range(dx, dx ? z.g : 0), range(dg_log, dg_log ? z.g : 0), range(dh0, dh0 ? z.state : 0),
                       range(workspace, need)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  if (z.state == 0 || (s->L == 0 && !dh0)) return DELTA_OK;
  if ((rc = launch_guard())) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (validate_on() && (rc = validate_gates(g_log, z.g / 4, st))) return rc;
  p.x = x, p.g = g_log, p.states = const_cast<float*>(states), p.dO = dO, p.dh_final = dh_final;
  p.dx = dx, p.dg = dg_log, p.dh0 = dh0, p.ws = workspace;
  return hip_status(delta::launch_glr_bwd(p, s->dtype == DELTA_BF16, st));
}

int delta_decode_glr(const delta_shape* s, int32_t input_gate, const void* x, const float* g_log, float* h, void* O,
                     void* stream) {
  GlrParams p;
  GlrSizes z;
  int rc = glr_shape(s, input_gate, p, z);
  if (rc) return rc;
  if (s->L != 1) return DELTA_ERR_BAD_SHAPE;
  if (z.x > 0 && (!x || !g_log || !h || !O)) return DELTA_ERR_NULL_ARG;
  const void* ptrs[] = {x, g_log, h, O};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return DELTA_ERR_MISALIGNED;
  const Range in[] = {range(x, z.x), range(g_log, z.g)};
  const Range out[] = {range(h, z.state), range(O, z.x)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  if (z.x == 0) return DELTA_OK;
  if ((rc = launch_guard())) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (validate_on() && (rc = validate_gates(g_log, z.g / 4, st))) return rc;
  p.x = x, p.g = g_log, p.h_final = h, p.O = O;
  return hip_status(delta::launch_glr_decode(p, s->dtype == DELTA_BF16, st));
}

}  // extern "C"

namespace {

int rows_shape(int64_t rows, int32_t width, int32_t dtype, float eps) {
  if (rows < 0 || rows > 0x7fffffff || width < 1 || width > (1 << 20) || !(eps >= 0.f)) return DELTA_ERR_BAD_SHAPE;
  if (dtype != DELTA_F32 && dtype != DELTA_BF16) return DELTA_ERR_UNSUPPORTED_DIM;
  return DELTA_OK;
}

// The two forward forms: y in dtype, or y8 with its scales.
int run_rmsnorm(int64_t rows, int32_t width, int32_t dtype, float eps, int group, const void* x, const void* residual,
                const float* weight, void* sum, void* y, void* y8, float* scale, void* stream) {
  int rc = rows_shape(rows, width, dtype, eps);
  if (rc) return rc;
  if (rows == 0) return DELTA_OK;
  if (!x || !weight || (residual && !sum) || !(y || (y8 && scale))) return DELTA_ERR_NULL_ARG;
  if (!residual) sum = nullptr;
  const void* ptrs[] = {x, residual, weight, sum, y, y8};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return DELTA_ERR_MISALIGNED;
  if (!aligned(scale, 4)) return DELTA_ERR_MISALIGNED;
  const size_t n = (size_t)rows * width, es = esize(dtype);
  const size_t groups = group ? ((size_t)width + group - 1) / group : 1;
  // sum may be x or residual itself (each row is read whole before it is written)
  const bool over_x = sum == x, over_r = sum && sum == residual;
  const Range in[] = {range(x, over_x ? 0 : n * es), range(residual, residual && !over_r ? n * es : 0),
                      range(weight, (size_t)width * 4)};
  const Range out[] = {range(sum, sum ? n * es : 0), range(y, y ? n * es : 0), range(y8, y8 ? n : 0),
                       range(scale, scale ? (size_t)rows * groups * 4 : 0)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  if ((rc = launch_guard())) return rc;
  RmsnormParams p;
  memset(&p, 0, sizeof(p));
  p.rows = rows, p.width = width, p.group = group ? group : width, p.eps = eps;
  p.x = x, p.res = residual, p.weight = weight, p.sum = sum, p.y = y, p.y8 = static_cast<uint8_t*>(y8), p.scale = scale;
  return hip_status(delta::launch_rmsnorm(p, dtype == DELTA_BF16, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int delta_layer_rmsnorm(int64_t rows, int32_t width, int32_t dtype, float eps, const void* x, const void* residual,
                        const float* weight, void* sum, void* y, void* stream) {
  return run_rmsnorm(rows, width, dtype, eps, 0, x, residual, weight, sum, y, nullptr, nullptr, stream);
}

int delta_layer_rmsnorm_quant(int64_t rows, int32_t width, int32_t dtype, float eps, int32_t group, const void* x,
                              const void* residual, const float* weight, void* sum, void* y8, float* scale,
                              void* stream) {
  if (group != 0 && group != 128) return DELTA_ERR_UNSUPPORTED_DIM;
  return run_rmsnorm(rows, width, dtype, eps, group, x, residual, weight, sum, nullptr, y8, scale, stream);
}

int delta_layer_rmsnorm_bwd_workspace_bytes(int64_t rows, int32_t width, int32_t dtype, size_t* bytes) {
  const int rc = rows_shape(rows, width, dtype, 0.f);
  if (rc) return rc;
  if (!bytes) return DELTA_ERR_NULL_ARG;
  *bytes = align_up((size_t)delta::rmsnorm_bwd_parts(rows, width) * width * 4);
  return DELTA_OK;
}

int delta_layer_rmsnorm_bwd(int64_t rows, int32_t width, int32_t dtype, float eps, const void* dy, const void* s,
                            const float* weight, const void* dsum, void* dx, float* dweight, void* workspace,
                            size_t workspace_bytes, void* stream) {
  int rc = rows_shape(rows, width, dtype, eps);
  if (rc) return rc;
  if (rows > 0 && (!dy || !s || !weight || !dx)) return DELTA_ERR_NULL_ARG;
  size_t need = 0;  // the workspace holds the parts of dweight
  if (dweight) delta_layer_rmsnorm_bwd_workspace_bytes(rows, width, dtype, &need);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DELTA_ERR_WORKSPACE;
  const void* ptrs[] = {dy, s, weight, dsum, dx, dweight, workspace};
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return DELTA_ERR_MISALIGNED;
  const size_t n = (size_t)rows * width * esize(dtype), nw = (size_t)width * 4;
  const Range in[] = {range(dy, dy ? n : 0), range(s, s ? n : 0), range(weight, weight ? nw : 0), range(dsum, dsum ? n : 0)};
  const Range out[] = {range(dx, dx ? n : 0), range(dweight, dweight ? nw : 0), range(workspace, need)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  if (rows == 0 && !dweight) return DELTA_OK;
  if ((rc = launch_guard())) return rc;
  RmsnormParams p;
  memset(&p, 0, sizeof(p));
  p.rows = rows, p.width = width, p.eps = eps;
  p.dy = dy, p.x = s, p.weight = weight, p.dsum = dsum, p.dx = dx, p.dweight = dweight;
  p.part = static_cast<float*>(workspace);
  return hip_status(delta::launch_rmsnorm_bwd(p, dtype == DELTA_BF16, static_cast<hipStream_t>(stream)));
}

int delta_grad_norm_workspace_bytes(int32_t n, const int64_t* sizes, size_t* bytes) {
  Clip c;
  const int rc = clip_sizes(n, sizes, c);
  if (rc) return rc;
  if (!bytes) return DELTA_ERR_NULL_ARG;
  // one float64 per workgroup of every launch over the tensors
  *bytes = align_up((size_t)c.parts * 8);
  return DELTA_OK;
}

int delta_grad_norm(int32_t n, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, float* norm,
                    void* workspace, size_t workspace_bytes, void* stream) {
  return run_clip(n, grads, sizes, dtypes, false, 0.f, 0.f, nullptr, norm, workspace, workspace_bytes, stream);
}

int delta_clip_grads(int32_t n, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, float max_norm,
                     float eps, void* const* out, float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  return run_clip(n, grads, sizes, dtypes, true, max_norm, eps, out, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
