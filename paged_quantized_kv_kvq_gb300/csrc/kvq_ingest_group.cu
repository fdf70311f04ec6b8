// kvq_ingest_group.cu -- the ingest kernel for pools with per-group scales.
#include "kvq_ingest_impl.cuh"

namespace kvq {

cudaError_t launch_ingest_group(const IngestLaunch& l) {
  return l.p.pool.fmt == FMT_INT4_GROUP ? run_ingest<FMT_INT4_GROUP>(l)
                                        : run_ingest<FMT_INT8_GROUP>(l);
}

}  // namespace kvq
