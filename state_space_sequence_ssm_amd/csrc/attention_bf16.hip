// The walk of linear attention on bf16 inputs.
#include "attention_impl.hpp"

namespace m3 {
hipError_t launch_walk_bf16(const WalkPlan& p, int kb, int nct, bool states_only, hipStream_t s) {
  return walk::dispatch<bf16_t>(p, kb, nct, states_only, s);
}
}  // namespace m3
