// kvq_diff_decode.cu -- differential decode kernels (kvq_decode_impl.cuh) but for
// the per-group formats.  The two maps of a head are two rows of a head tile, the channels of
// the other map zero in each: an mma has idle columns for them, and the pages are what
// bounds it.  Their lane has both in hand at the end, for the difference and the norm.
// Measured, replayed: 64 x 2048, 16 heads over 8 kv heads, INT8 blocks: 57.2 us (269 MB,
// 0.69 of the copy rate).
#include "kvq_decode_impl.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

template <int FMT>
cudaError_t run_block(const DecodeLaunch& l) {
  if (l.p.pool.bs == 8) return run_decode_d<FMT, true, true>(l);
  if (!l.two_ctas) return run_decode_d<FMT, false, true>(l);
  return l.p.pool.D == 64 ? run_decode<FMT, 64, 1, false, 2, true>(l)
                          : run_decode<FMT, 128, 1, false, 2, true>(l);
}

template <int FMT>
cudaError_t run_any(const DecodeLaunch& l) {
  return l.p.pool.bs == 8 ? run_decode_d<FMT, true, true>(l) : run_decode_d<FMT, false, true>(l);
}

}  // namespace

cudaError_t launch_diff_block(const DecodeLaunch& l) {
  return l.p.pool.fmt == FMT_FP8_BLOCK ? run_block<FMT_FP8_BLOCK>(l) : run_block<FMT_INT8_BLOCK>(l);
}

cudaError_t launch_diff_misc(const DecodeLaunch& l) {
  switch (l.p.pool.fmt) {
    case FMT_FP16: return run_any<FMT_FP16>(l);
    case FMT_INT8_TOKEN: return run_any<FMT_INT8_TOKEN>(l);
    case FMT_FP8_TOKEN: return run_any<FMT_FP8_TOKEN>(l);
    case FMT_INT8_CHANNEL: return run_any<FMT_INT8_CHANNEL>(l);
    case FMT_FP8_E5M2: return run_any<FMT_FP8_E5M2>(l);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
