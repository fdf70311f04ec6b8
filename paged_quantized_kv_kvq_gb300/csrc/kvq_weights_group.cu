// kvq_weights_group.cu -- the attention-weights kernel for pools with per-group
// scales.
#include "kvq_weights_impl.cuh"

namespace kvq {

cudaError_t launch_weights_int8(const WeightsLaunch& l) { return run_weights_group<FMT_INT8_GROUP>(l); }
cudaError_t launch_weights_int4(const WeightsLaunch& l) { return run_weights_group<FMT_INT4_GROUP>(l); }

}  // namespace kvq
