// Launch interface between the residual-block entry points (block_abi.cpp) and their kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace delta {

// One gated linear recurrence after validation: D = H * dv channels.
constexpr int GLR_CHUNK = 64;  // tokens between kept states
struct GlrParams {
  int B, L, D, gate;
  const void* x;          // [B, L, D]
  const float* g;         // [B, L, D] log gates
  const float* h0;        // [B, D] or nullptr (decode: unused)
  void* O;                // [B, L, D]
  float* h_final;         // [B, D] or nullptr (decode: the state, in place)
  float* states;          // [B, ceil(L / GLR_CHUNK), D]: written forward (or nullptr), read backward
  const void* dO;         // [B, L, D]
  const float* dh_final;  // [B, D] or nullptr
  float *dx, *dg;         // [B, L, D]
  float* dh0;             // [B, D] or nullptr
  void* ws;               // glr_workspace bytes
};
size_t glr_workspace(int B, int L, int D, bool backward);
bool glr_grid_fits(int B, int L, int D);  // whether the number of tiles is one a launch takes
hipError_t launch_glr_fwd(const GlrParams& p, bool bf16, hipStream_t st);
hipError_t launch_glr_bwd(const GlrParams& p, bool bf16, hipStream_t st);
hipError_t launch_glr_decode(const GlrParams& p, bool bf16, hipStream_t st);

struct RmsnormParams {
  long rows;
  int width, group;     // group: channels per scale of y8
  float eps;
  const void *x, *res;  // [rows, width]; res may be nullptr
  const float* weight;  // [width]
  void *sum, *y;        // [rows, width]; y nullptr where y8 is wanted
  uint8_t* y8;
  float* scale;
  const void *dy, *dsum;  // backward; dsum may be nullptr, x is s
  void* dx;
  float* dweight;         // [width] or nullptr
  float* part;            // backward: rmsnorm_bwd_parts(rows, width) partial rows of dweight
};
hipError_t launch_rmsnorm(const RmsnormParams& p, bool bf16, hipStream_t st);
int rmsnorm_bwd_parts(long rows, int width);
hipError_t launch_rmsnorm_bwd(const RmsnormParams& p, bool bf16, hipStream_t st);

// Tensors of one launch of the gradient kernels, passed by value (no table in device memory).
constexpr int CLIP_TENSORS = 96;
struct ClipTable {
  const void* g[CLIP_TENSORS];
  void* out[CLIP_TENSORS];
  int64_t n[CLIP_TENSORS];
  int32_t first[CLIP_TENSORS + 1];  // first piece of each tensor; first[count]: pieces in all
  uint32_t bf16[CLIP_TENSORS / 32];
  int32_t count;
};
constexpr long CLIP_PIECE = 16384;  // elements of one piece
constexpr int CLIP_PARTS = 2048;    // workgroups of the sums at most
// Workgroups for so many pieces: the fewest that take no more rounds over them than CLIP_PARTS would.
inline int clip_parts(int64_t pieces) {
  const int64_t rounds = (pieces + CLIP_PARTS - 1) / CLIP_PARTS;
  return pieces ? (int)((pieces + rounds - 1) / rounds) : 0;
}
// The sums of one table's squares, sums[0 .. parts); then the norm of `parts` sums in all, alone or with
// the scaling of one table (there parts = -1: *norm is there already)
hipError_t launch_grad_sums(const ClipTable& t, double* sums, int parts, hipStream_t st);
hipError_t launch_grad_finish(const double* sums, int parts, float* norm, hipStream_t st);
hipError_t launch_grad_scale(const ClipTable& t, const double* sums, int parts, float max_norm, float eps, float* norm,
                             hipStream_t st);

}  // namespace delta
