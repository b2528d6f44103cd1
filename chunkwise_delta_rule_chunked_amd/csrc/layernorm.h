// Launch interface between the layer norm and dropout entry points (layernorm_abi.cpp) and their kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace delta {

// Dropout of one call: an element is kept where its 16 bits reach `drop`, and then multiplied by `scale`.
struct DropRule {
  uint32_t drop;  // 0: nothing dropped, 65536: everything
  float scale;
  uint64_t seed, offset;
  const uint64_t* step;  // added to offset when the kernel runs, or nullptr
};

struct LayernormParams {
  long rows;
  int width;
  float eps;
  DropRule rule;
  const void *x, *res;  // [rows, width]; res may be nullptr
  const float *weight, *bias;  // [width]; bias may be nullptr
  void *sum, *y;               // sum: nullptr where it would be x
  // backward: x is the sum
  const void *dy, *dsum;       // dsum may be nullptr
  void *dres, *dx;             // dx: nullptr where it would be dres
  float *dweight, *dbias;      // [width] or nullptr
  float* part;                 // layernorm_bwd_parts partial rows of dweight, and as many of dbias
};
hipError_t launch_layernorm(const LayernormParams& p, bool bf16, hipStream_t st);
int layernorm_bwd_parts(long rows, int width);
hipError_t launch_layernorm_bwd(const LayernormParams& p, bool bf16, hipStream_t st);

struct DropoutParams {
  long rows;
  int width;
  DropRule rule;
  const void *x, *res;  // res may be nullptr
  void* y;
};
hipError_t launch_dropout(const DropoutParams& p, bool bf16, hipStream_t st);

}  // namespace delta
