// kvq_ingest.cu -- launch planning of the ingest kernel (kvq_ingest_impl.cuh),
// its formats with one scale per block, and the read-back of slots as values.
#include <algorithm>

#include "kvq_ingest_impl.cuh"

namespace kvq {

namespace {

// K and V of 16 slots of one kv head per CTA, as fp16: code times scale in
// fp32, rounded once.  The 16 slots of a sub-tile share its bytes, so its
// sectors come from L2 once; the bound is the write of the values.
constexpr int kValueSlots = 16;

__global__ void __launch_bounds__(256) kvq_read_values_kernel(PoolView pool, const int64_t* slots,
                                                              int64_t n, __half* k, __half* v) {
  const int D = pool.D, lph = D / 8;
  const int kv = threadIdx.x / (kValueSlots * 8) ;  // 128 threads each for K and V
  const int h = blockIdx.y;
  for (int u = threadIdx.x % (kValueSlots * 8); u < kValueSlots * lph; u += kValueSlots * 8) {
    const int64_t i = (int64_t)blockIdx.x * kValueSlots + u / lph;
    if (i >= n) return;
    const int d0 = u % lph * 8;
    const int64_t slot = slots[i];
    if (slot < 0) continue;
    if (slot >= pool.num_blocks * pool.bs) {
      set_error(pool.err, ERR_RANGE);
      continue;
    }
    const int64_t blk = slot / pool.bs;
    const int off = static_cast<int>(slot % pool.bs), tt = off & 15;
    const char* page = pool.pages + (blk * pool.Hkv + h) * pool.page_bytes;
    const char* tile = page + (kv == 0 ? 0 : pool.code_bytes) + (off >> 4) * pool.sub_bytes;
    const float* sc = reinterpret_cast<const float*>(page + 2 * pool.code_bytes);
    float s = 1.f;
    if (pool.fmt == FMT_INT8_GROUP || pool.fmt == FMT_INT4_GROUP)
      s = sc[(kv * pool.bs + off) * pool.ng + d0 / pool.group];
    else if (fmt_block(pool.fmt))
      s = sc[kv];
    else if (pool.fmt == FMT_INT8_TOKEN || pool.fmt == FMT_FP8_TOKEN)
      s = pool.tok_scales[(blk * 2 + kv) * pool.bs + off];
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = d0 + e;
      if (pool.fmt == FMT_INT4_GROUP) {
        int sh;
        const int o = kv == 0 ? k_nibble(tt, d, sh) : v_nibble(tt, d, sh);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + o);
        x[e] = static_cast<float>(static_cast<int>(w >> sh & 0xFu) - static_cast<int>(kInt4Bias)) * s;
        continue;
      }
      const char* at = tile + (kv == 0 ? k_tile_offset(tt, d, D, pool.esize)
                                       : v_code_offset(tt, d, D, pool.esize, pool.bs));
      if (pool.fmt == FMT_FP16) {
        x[e] = __half2float(*reinterpret_cast<const __half*>(at));
        continue;
      }
      const uint8_t c = *reinterpret_cast<const uint8_t*>(at);
      if (pool.fmt == FMT_FP8_E5M2)
        x[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E5M2)));
      else if (fmt_e4m3(pool.fmt))
        x[e] = code_value<FMT_FP8_BLOCK>(c) * s;
      else
        x[e] = code_value<FMT_INT8_BLOCK>(c) *
               (pool.fmt == FMT_INT8_CHANNEL ? pool.chan_scales[((int64_t)kv * pool.Hkv + h) * D + d] : s);
    }
    *reinterpret_cast<uint4*>((kv == 0 ? k : v) + (i * pool.Hkv + h) * D + d0) = narrow8(x);
  }
}

}  // namespace

cudaError_t launch_read_values(const PoolView& pool, const int64_t* slots, int64_t n, __half* k,
                               __half* v, cudaStream_t st) {
  const int64_t gx = (n + kValueSlots - 1) / kValueSlots;
  if (gx > 0x7fffffffLL || pool.Hkv > 65535) return cudaErrorInvalidValue;
  kvq_read_values_kernel<<<dim3(static_cast<unsigned>(gx), pool.Hkv), 256, 0, st>>>(pool, slots, n, k, v);
  return phase_mark(st, cudaGetLastError());
}

cudaError_t launch_ingest_block(const IngestLaunch& l) {
  return l.p.pool.fmt == FMT_FP8_BLOCK ? run_ingest<FMT_FP8_BLOCK>(l) : run_ingest<FMT_INT8_BLOCK>(l);
}

cudaError_t launch_ingest(const IngestArgs& a, cudaStream_t st, bool dependent) {
  IngestLaunch l;
  IngestParams& p = l.p;
  p = IngestParams{};
  p.pool = a.pool;
  p.q = RopeRows{a.q, a.q_stride, a.q_out, a.q_out_stride, a.q_weight};
  p.Hq = a.Hq;
  p.x[0] = a.k;
  p.x[1] = a.v;
  p.stride[0] = a.k_stride;
  p.stride[1] = a.v_stride;
  p.k_weight = a.k_weight;
  p.positions = a.positions;
  p.slots = a.slots;
  p.table = a.table;
  p.lens = a.lens;
  p.max_blocks = a.max_blocks;
  p.max_ctx = a.max_ctx;
  p.T = a.T;
  p.eps = a.eps;
  p.bf16 = a.bf16;
  if (a.plan != nullptr) p.plan = *a.plan;
  while ((1 << p.bs_log2) < a.pool.bs) ++p.bs_log2;
  // Few tokens (a decode step): one per CTA and one head per CTA, for the
  // latency of a run.  Many: a block's worth of tokens per CTA, its angles
  // shared by the heads.  Formats with one scale per token need every head of
  // a token in one CTA.
  const bool many = a.T >= 1024;
  const bool tok = a.pool.fmt == FMT_INT8_TOKEN || a.pool.fmt == FMT_FP8_TOKEN;
  p.tpc = many && a.slots != nullptr ? a.pool.bs : 1;
  p.hpc = many || tok ? a.pool.Hkv : 1;
  p.hsplit = (a.pool.Hkv + p.hpc - 1) / p.hpc;
  p.kv_ctas = (a.T + p.tpc - 1) / p.tpc * p.hsplit * 2;
  int64_t q_ctas = 0;
  if (a.Hq > 0) {
    const int rpp = kIngestThreads / (a.pool.D / 8);
    p.q_parts = a.T >= 512 ? 1 : (a.Hq + rpp - 1) / rpp;
    p.q_inv = rope_inverse(a.Hq);
    p.q_tpc = a.T >= 4096 ? kRopeTokens : 1;
    q_ctas = (a.T + p.q_tpc - 1) / p.q_tpc * p.q_parts;
  }
  if (p.kv_ctas + q_ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  l.grid = static_cast<unsigned>(p.kv_ctas + q_ctas);
  l.smem = ingest_smem(a.pool, p.plan.rotary_dim);
  l.st = st;
  l.dependent = dependent;
  switch (a.pool.fmt) {
    case FMT_INT8_BLOCK:
    case FMT_FP8_BLOCK: return launch_ingest_block(l);
    case FMT_INT8_GROUP:
    case FMT_INT4_GROUP: return launch_ingest_group(l);
    case FMT_INT8_TOKEN:
    case FMT_FP8_TOKEN: return launch_ingest_token(l);
    default: return launch_ingest_misc(l);
  }
}

}  // namespace kvq
