// The chain kernel of linear attention for float32 inputs.
#include "linear_chain.h"

namespace delta {
namespace lin {

hipError_t chain_f32(const LinChain& c, bool reverse, int form, hipStream_t st) { return chain<float>(c, reverse, form, st); }
hipError_t summary_f32(const LinChain& c, bool reverse, hipStream_t st) { return summary<float>(c, reverse, st); }

}  // namespace lin
}  // namespace delta
