// kvq_ingest_group.cu -- the ingest kernel for pools with per-group scales and of 4-bit floats.
#include "kvq_ingest_impl.cuh"

namespace kvq {

cudaError_t launch_ingest_group(const IngestLaunch& l) {
  switch (l.p.pool.fmt) {
    case FMT_INT4_GROUP: return run_ingest<FMT_INT4_GROUP>(l);
    case FMT_FP4: return run_ingest<FMT_FP4>(l);
    default: return run_ingest<FMT_INT8_GROUP>(l);
  }
}

}  // namespace kvq
