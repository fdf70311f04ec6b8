// kvq_diff_decode_group.cu -- differential decode kernels (kvq_decode_impl.cuh) of the
// per-group formats.
#include "kvq_decode_impl.cuh"
#include "kvq_internal.h"

namespace kvq {

cudaError_t launch_diff_group(const DecodeLaunch& l) {
  if (l.p.pool.fmt == FMT_INT4_GROUP) return run_decode_group<FMT_INT4_GROUP, false, true>(l);
  return l.p.pool.bs == 8 ? run_decode_group<FMT_INT8_GROUP, true, true>(l)
                          : run_decode_group<FMT_INT8_GROUP, false, true>(l);
}

}  // namespace kvq
