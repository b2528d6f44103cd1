// The chain kernels of linear attention for float32 inputs.
#include "linear_chain.h"

namespace delta {

hipError_t lin_chain_f32(const LinChain& c, bool reverse, int form, hipStream_t st) { return lin::chain<float>(c, reverse, form, st); }

hipError_t lin_summary_f32(const LinChain& forward, const LinChain* reverse, hipStream_t st) {
  return lin::summary<float>(forward, reverse, st);
}

hipError_t lin_backward_f32(const LinChain& dq, const LinChain& dv, const LinChain& dk, bool gates, bool state, hipStream_t st) {
  return gates ? lin::backward<float, true>(dq, dv, dk, state, st) : lin::backward<float, false>(dq, dv, dk, state, st);
}

}  // namespace delta
