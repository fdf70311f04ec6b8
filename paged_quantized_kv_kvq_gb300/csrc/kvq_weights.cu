// kvq_weights.cu -- launch and format dispatch of the attention-weights kernel
// (kvq_weights_impl.cuh).
#include "kvq_weights_impl.cuh"

namespace kvq {

cudaError_t launch_weights(const WeightsArgs& a, cudaStream_t st) {
  WeightsLaunch l;
  l.st = st;
  l.sms = a.sms;
  WeightsParams& p = l.p;
  p = WeightsParams{};
  p.d.pool = a.pool;
  p.d.q = a.q;
  p.d.table = a.table;
  p.d.lens = a.lens;
  p.d.q_stride = (int64_t)a.Hq * a.pool.D;
  p.d.S = a.S;
  p.d.Hq = a.Hq;
  p.d.G = a.Hq / a.pool.Hkv;
  p.d.n_ht = (p.d.G + 7) / 8;
  p.d.max_blocks = a.max_blocks;
  p.d.max_ctx = a.max_ctx;
  p.d.sm_scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.d.wait_tries = kWaitTries;
  p.lse = a.lse;
  p.prev = a.prev;
  p.scores = a.scores;
  p.stride = a.stride;
  p.decay = a.decay;
  switch (a.pool.fmt) {
    case FMT_FP16: return run_weights_d<FMT_FP16>(l);
    case FMT_INT8_TOKEN: return run_weights_d<FMT_INT8_TOKEN>(l);
    case FMT_INT8_CHANNEL: return run_weights_d<FMT_INT8_CHANNEL>(l);
    case FMT_INT8_GROUP: return launch_weights_int8(l);
    case FMT_FP8_TOKEN: return run_weights_d<FMT_FP8_TOKEN>(l);
    case FMT_INT4_GROUP: return launch_weights_int4(l);
    case FMT_FP8_E5M2: return run_weights_d<FMT_FP8_E5M2>(l);
    case FMT_INT8_BLOCK: return run_weights_d<FMT_INT8_BLOCK>(l);
    case FMT_FP8_BLOCK: return run_weights_d<FMT_FP8_BLOCK>(l);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
