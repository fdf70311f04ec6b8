// kvq_decode_fp4.cu -- paged decode over pools of 4-bit floats.
#include "kvq_decode_impl.cuh"
#include "kvq_internal.h"

namespace kvq {

cudaError_t launch_decode_fp4(const DecodeLaunch& l) { return run_decode_d<FMT_FP4>(l); }

}  // namespace kvq
