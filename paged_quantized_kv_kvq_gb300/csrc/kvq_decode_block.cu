// kvq_decode_block.cu -- paged decode over pools with one K and one V scale per
// (block, kv head): INT8 and FP8 e4m3 codes, every block size.
#include "kvq_decode_impl.cuh"
#include "kvq_internal.h"

namespace kvq {

cudaError_t launch_decode_block(const DecodeLaunch& l) {
  const bool fp8 = l.p.pool.fmt == FMT_FP8_BLOCK;
  if (l.p.pool.bs == 8)
    return fp8 ? run_decode_d<FMT_FP8_BLOCK, true>(l) : run_decode_d<FMT_INT8_BLOCK, true>(l);
  return fp8 ? run_decode_d<FMT_FP8_BLOCK>(l) : run_decode_d<FMT_INT8_BLOCK>(l);
}

}  // namespace kvq
