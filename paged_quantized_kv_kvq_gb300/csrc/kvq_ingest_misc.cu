// kvq_ingest_misc.cu -- the ingest kernel for FP16, per-channel, unscaled and
// per-token pools.
#include "kvq_ingest_impl.cuh"

namespace kvq {

cudaError_t launch_ingest_misc(const IngestLaunch& l) {
  switch (l.p.pool.fmt) {
    case FMT_FP16: return run_ingest<FMT_FP16>(l);
    case FMT_INT8_CHANNEL: return run_ingest<FMT_INT8_CHANNEL>(l);
    case FMT_FP8_E5M2: return run_ingest<FMT_FP8_E5M2>(l);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_ingest_token(const IngestLaunch& l) {
  return l.p.pool.fmt == FMT_FP8_TOKEN ? run_ingest<FMT_FP8_TOKEN>(l)
                                       : run_ingest<FMT_INT8_TOKEN>(l);
}

}  // namespace kvq
