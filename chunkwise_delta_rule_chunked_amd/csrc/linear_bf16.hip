// The chain kernel of linear attention for bf16 inputs.
#include "linear_chain.h"

namespace delta {
namespace lin {

hipError_t chain_bf16(const LinChain& c, bool reverse, int form, hipStream_t st) { return chain<bf16>(c, reverse, form, st); }
hipError_t summary_bf16(const LinChain& c, bool reverse, hipStream_t st) { return summary<bf16>(c, reverse, st); }

}  // namespace lin
}  // namespace delta
