// kvq_decode_fp4.cu -- paged decode over pools of 4-bit floats (kvq_decode4_impl.cuh).
#include "kvq_decode4_impl.cuh"

namespace kvq {

cudaError_t launch_decode_fp4(const DecodeLaunch& l) { return run_decode4_any<false>(l); }
cudaError_t launch_diff_fp4(const DecodeLaunch& l) { return run_decode4_any<true>(l); }

}  // namespace kvq
