// The chain kernels of linear attention for bf16 inputs.
#include "linear_chain.h"

namespace delta {

hipError_t lin_chain_bf16(const LinChain& c, bool reverse, int form, hipStream_t st) { return lin::chain<bf16>(c, reverse, form, st); }

hipError_t lin_summary_bf16(const LinChain& forward, const LinChain* reverse, hipStream_t st) {
  return lin::summary<bf16>(forward, reverse, st);
}

hipError_t lin_backward_bf16(const LinChain& dq, const LinChain& dv, const LinChain& dk, bool gates, bool state, hipStream_t st) {
  return gates ? lin::backward<bf16, true>(dq, dv, dk, state, st) : lin::backward<bf16, false>(dq, dv, dk, state, st);
}

}  // namespace delta
