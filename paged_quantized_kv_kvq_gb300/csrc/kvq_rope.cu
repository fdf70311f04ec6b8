// kvq_rope.cu -- per-head norms and rotary positions of query and key rows, and
// the host side of a rotation plan.
#include <algorithm>
#include <cmath>

#include "kvq_context.h"
#include "kvq_internal.h"
#include "kvq_rope_math.cuh"

namespace kvq {

namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  RopeRows rows[2];
  int heads[2];
  bool bf16;
  const int64_t* positions;
  int64_t T;
  int tpc;    // tokens per CTA
  int parts;  // CTAs a token's rows are spread over
  uint32_t inv;
  float eps;
  kvq_rope_plan plan;
};

template <int D>
__global__ void __launch_bounds__(kRopeThreads) kvq_rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) char smem[rope_smem(D, D)];
  const int64_t t0 = (blockIdx.x / p.parts) * (int64_t)p.tpc;
  rope_tokens<D, kRopeThreads>(p.rows[0], p.heads[0], p.rows[1], p.heads[1], p.inv, p.bf16,
                               p.positions, t0, static_cast<int>(min((int64_t)p.tpc, p.T - t0)),
                               blockIdx.x % p.parts, p.parts, p.eps, p.plan, smem);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
  RopeParams p{};
  for (int i = 0; i < 2; ++i) {
    p.rows[i] = RopeRows{a.x[i], a.x_stride[i], a.out[i], a.out_stride[i], a.weight[i]};
    p.heads[i] = a.heads[i];
  }
  p.bf16 = a.bf16;
  p.positions = a.positions;
  p.T = a.T;
  p.eps = a.eps;
  if (a.plan != nullptr) p.plan = *a.plan;
  // Few tokens: spread a token's rows over CTAs so that every thread has one
  // chunk; many: several tokens per CTA share its set-up.
  const int H = a.heads[0] + a.heads[1];
  p.inv = rope_inverse(H);
  const int rpp = kRopeThreads / (a.D / 8);
  const int passes = (H + rpp - 1) / rpp;
  p.parts = a.T >= 512 ? 1 : passes;
  p.tpc = a.T >= 4096 ? kRopeTokens : 1;
  const int64_t grid = (a.T + p.tpc - 1) / p.tpc * p.parts;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.D == 64)
    kvq_rope_kernel<64><<<static_cast<unsigned>(grid), kRopeThreads, 0, st>>>(p);
  else
    kvq_rope_kernel<128><<<static_cast<unsigned>(grid), kRopeThreads, 0, st>>>(p);
  return phase_mark(st, cudaGetLastError());
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
      !std::isfinite(c->magnitude))
    return KVQ_ERR_INVALID_ARG;
  if (c->scaling < KVQ_ROPE_NONE || c->scaling > KVQ_ROPE_BANDS) return KVQ_ERR_INVALID_ARG;
  if (c->scaling != KVQ_ROPE_NONE && (!(s >= 1.0) || !std::isfinite(s))) return KVQ_ERR_INVALID_ARG;
  const bool by_turns = c->scaling == KVQ_ROPE_PARTS || c->scaling == KVQ_ROPE_BANDS;
  if (by_turns && (!(n >= 1.0) || !std::isfinite(n) || !(c->low > 0.0) || !(c->high > c->low) ||
                   !std::isfinite(c->high)))
    return KVQ_ERR_INVALID_ARG;
  double base = c->base, lo = 0.0, hi = 0.0;
  if (c->scaling == KVQ_ROPE_BASE) {
    base *= std::pow(s, r / (r - 2.0));
    if (!std::isfinite(base)) return KVQ_ERR_INVALID_ARG;
  }
  if (c->scaling == KVQ_ROPE_PARTS) {
    // the (fractional) pair that turns `high` / `low` times over orig_len
    const double ln = 2.0 * std::log(base);
    lo = std::max(std::floor(r * std::log(n / (2.0 * pi * c->high)) / ln), 0.0);
    hi = std::min(std::ceil(r * std::log(n / (2.0 * pi * c->low)) / ln), r - 1.0);
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
      const double ramp = std::min(std::max((i - lo) / width, 0.0), 1.0);
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
