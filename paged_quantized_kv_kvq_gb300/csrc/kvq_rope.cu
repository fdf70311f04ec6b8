// kvq_rope.cu -- per-head norms and rotary positions of query and key rows, and
// the host side of a rotation plan.
#include <algorithm>
#include <cmath>

#include "kvq_context.h"
#include "kvq_internal.h"
#include "kvq_rope_math.cuh"

namespace kvq {

namespace {

constexpr int kRopeThreads = 320;  // at most; 48 registers let four such CTAs share an SM

struct RopeParams {
  RopeRows rows[2];
  int heads[2];
  const int64_t* positions;
  int64_t T;
  int tpc;    // tokens per CTA
  int parts;  // CTAs a token's rows are spread over
  float eps;
  bool beside;  // launched while the kernel before it runs
  kvq_rope_plan plan;
};

template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 4) kvq_rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) float smem[rope_smem(D) / 4];
  const int64_t t0 = (blockIdx.x / p.parts) * (int64_t)p.tpc;
  const int part = blockIdx.x % p.parts, rpc = blockDim.x / (D / 8);  // rows of the CTA
  rope_tokens<D, BF16, INTER>(p.rows[0], p.heads[0], p.rows[1], p.heads[1], p.positions, t0,
                              static_cast<int>(min((int64_t)p.tpc, p.T - t0)),
                              part * rpc + threadIdx.x / (D / 8), p.eps, p.plan, smem);
  // A kernel after this one may itself be a programmatic dependent and wait for
  // this grid alone: so this grid ends no earlier than the one it runs beside.  One
  // CTA waits for that; all of the other grid's are resident by now.
  if (p.beside && blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D>
cudaError_t run_rope(const cudaLaunchConfig_t& cfg, const RopeParams& p, bool bf16) {
  if (p.plan.layout == KVQ_ROPE_INTERLEAVED)
    return bf16 ? cudaLaunchKernelEx(&cfg, kvq_rope_kernel<D, true, true>, p)
                : cudaLaunchKernelEx(&cfg, kvq_rope_kernel<D, false, true>, p);
  return bf16 ? cudaLaunchKernelEx(&cfg, kvq_rope_kernel<D, true, false>, p)
              : cudaLaunchKernelEx(&cfg, kvq_rope_kernel<D, false, false>, p);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st, bool beside) {
  RopeParams p{};
  for (int i = 0; i < 2; ++i) {
    p.rows[i] = RopeRows{a.x[i], a.x_stride[i], a.out[i], a.out_stride[i], a.weight[i]};
    p.heads[i] = a.heads[i];
  }
  p.positions = a.positions;
  p.T = a.T;
  p.eps = a.eps;
  p.beside = beside;
  if (a.plan != nullptr) p.plan = *a.plan;
  // A thread takes one head row of up to kRopeTokens tokens; a token's rows are
  // spread evenly over CTAs of at most 10 warps.  A warp holds 2 rows of 128
  // channels or 4 of 64.  One token per CTA while that fills the SMs: 8192 tokens x
  // 40 heads of 128 take 53.9 us with one and 29.9 with four, 2048 (the first that takes
  // four) 15.4 and 10.5, 1024 9.1 and 6.7, 256 3.2 either way; 10 heads of 64: 4096 tokens 5.5 and 4.5,
  // 2048 3.7 and 3.6, 256 2.4 and 3.2.
  const int H = a.heads[0] + a.heads[1], rpw = 256 / a.D;
  const int warps = (H + rpw - 1) / rpw;
  p.parts = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  // (at least a thread per pair of channels, for the angles)
  const int threads = std::max(KVQ_ROPE_MAX_PAIRS, 32 * ((warps + p.parts - 1) / p.parts));
  p.tpc = a.T * p.parts >= 4096 ? kRopeTokens : 1;
  const int64_t grid = (a.T + p.tpc - 1) / p.tpc * p.parts;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 1 : 0;
  return phase_mark(st, a.D == 64 ? run_rope<64>(cfg, p, a.bf16) : run_rope<128>(cfg, p, a.bf16));
}

}  // namespace kvq

extern "C" kvq_status kvq_rope_init(const kvq_rope_config* c, kvq_rope_plan* out) {
  if (c == nullptr || out == nullptr) return KVQ_ERR_INVALID_ARG;
  const int r = c->rotary_dim;
  if (r < 2 || r > 2 * KVQ_ROPE_MAX_PAIRS || r % 2 != 0) return KVQ_ERR_INVALID_ARG;
  if (r % 16 != 0) return KVQ_ERR_UNSUPPORTED;
  if (c->layout != KVQ_ROPE_HALF && c->layout != KVQ_ROPE_INTERLEAVED) return KVQ_ERR_INVALID_ARG;
  const double s = c->factor, n = c->orig_len, pi = 3.14159265358979323846;
  if (!(c->base > 1.0) || !std::isfinite(c->base) || !(c->magnitude >= 0.0) ||
      !(c->magnitude <= 3e38))  // (kept as fp32)
    return KVQ_ERR_INVALID_ARG;
  if (c->scaling < KVQ_ROPE_NONE || c->scaling > KVQ_ROPE_BANDS) return KVQ_ERR_INVALID_ARG;
  if (c->scaling != KVQ_ROPE_NONE && (!(s >= 1.0) || !std::isfinite(s))) return KVQ_ERR_INVALID_ARG;
  const bool by_turns = c->scaling == KVQ_ROPE_PARTS || c->scaling == KVQ_ROPE_BANDS;
  if (by_turns && (!(n >= 1.0) || !std::isfinite(n) || !(c->low > 0.0) || !(c->high > c->low) ||
                   !std::isfinite(c->high)))
    return KVQ_ERR_INVALID_ARG;
  double base = c->base, lo = 0.0, hi = 0.0;
  bool all = false, none = false;  // KVQ_ROPE_PARTS: every pair is divided, or no pair
  if (c->scaling == KVQ_ROPE_BASE) {
    base *= std::pow(s, r / (r - 2.0));
    if (!std::isfinite(base)) return KVQ_ERR_INVALID_ARG;
  }
  if (c->scaling == KVQ_ROPE_PARTS) {
    // the (fractional) pair that turns `high` / `low` times over orig_len
    const double ln = 2.0 * std::log(base);
    lo = std::floor(r * std::log(n / (2.0 * pi * c->high)) / ln);
    hi = std::ceil(r * std::log(n / (2.0 * pi * c->low)) / ln);
    // even pair 0 turns no more than `low` times, or every pair more than `high`:
    // the ends, each kept within 0 .. r-1, would meet or cross there
    all = hi <= 0.0;
    none = lo >= r - 1.0;
    lo = std::max(lo, 0.0);
    hi = std::min(hi, r - 1.0);
  }
  kvq_rope_plan p{};
  p.rotary_dim = r;
  p.layout = c->layout;
  p.magnitude = static_cast<float>(c->magnitude > 0.0 ? c->magnitude
                                   : c->scaling == KVQ_ROPE_PARTS ? 0.1 * std::log(s) + 1.0 : 1.0);
  for (int i = 0; i < r / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (c->scaling == KVQ_ROPE_LINEAR) {
      f /= s;
    } else if (c->scaling == KVQ_ROPE_PARTS) {
      const double width = hi != lo ? hi - lo : 0.001;
      const double ramp = all ? 1.0 : none ? 0.0 : std::min(std::max((i - lo) / width, 0.0), 1.0);
      f = f / s * ramp + f * (1.0 - ramp);
    } else if (c->scaling == KVQ_ROPE_BANDS) {
      const double turns = n * f / (2.0 * pi);
      const double mix = std::min(std::max((turns - c->low) / (c->high - c->low), 0.0), 1.0);
      f = (1.0 - mix) * f / s + mix * f;
    }
    // f <= 1 radian, so f / 2pi < 0.16: its 64-bit fraction
    p.turns[i] = static_cast<uint64_t>(std::ldexp(f / (2.0 * pi), 64));
  }
  *out = p;
  return KVQ_OK;
}
