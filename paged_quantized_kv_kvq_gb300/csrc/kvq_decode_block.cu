// kvq_decode_block.cu -- paged decode over pools with one K and one V scale per
// (block, kv head): INT8 and FP8 e4m3 codes, every block size.
#include "kvq_decode_impl.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

template <int FMT>
cudaError_t run_block(const DecodeLaunch& l) {
  if (l.p.pool.bs == 8) return run_decode_d<FMT, true>(l);
  if (!l.two_ctas) return run_decode_d<FMT>(l);
  return l.p.pool.D == 64 ? run_decode<FMT, 64, 1, false, 2>(l) : run_decode<FMT, 128, 1, false, 2>(l);
}

}  // namespace

cudaError_t launch_decode_block(const DecodeLaunch& l) {
  return l.p.pool.fmt == FMT_FP8_BLOCK ? run_block<FMT_FP8_BLOCK>(l) : run_block<FMT_INT8_BLOCK>(l);
}

}  // namespace kvq
