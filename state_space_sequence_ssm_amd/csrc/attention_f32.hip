// The walk of linear attention on fp32 inputs.
#include "attention_impl.hpp"

namespace m3 {
hipError_t launch_walk_f32(const WalkPlan& p, int kb, int nct, bool states_only, hipStream_t s) {
  return walk::dispatch<float>(p, kb, nct, states_only, s);
}
}  // namespace m3
