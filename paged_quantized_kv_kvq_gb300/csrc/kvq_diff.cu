// kvq_diff.cu -- differential attention over a paged pool: format dispatch of the decode
// (kvq_decode_impl.cuh's DIFF kernels), and prompts.
//
// Prompts go through the two-pass prefill, whose attention kernel has a form for two maps
// (kvq_prefill_ws_impl.cuh).  Formats that it does not take (per-channel scales, several scale
// groups per head): every head becomes two Q rows, one per map with the other map's
// channels zero, the prefill kernels attend them, and a last kernel takes the
// difference of the two results of a head, norms it and rounds it.  The form for two maps
// does half the score products and needs no expanded queries and no fp32 results.  Calls of 8 x
// 2048, 16 heads over 4 kv heads of 128: two maps 359 us over 4-bit floats, 369 over FP16, 399 over INT8
// blocks and INT8 groups of 128; expanded 1299 per channel (two fp16 parts of q, one tile a CTA), 2930 over INT8
// groups of 32 and 2550 over INT4 groups of 32 (whose prompts have no tcgen05 kernel).
#include <algorithm>

#include "kvq_decode_impl.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kDiffThreads = 256;

// q [T][H][D] -> [T][2H][D]: rows 2h and 2h + 1 of a token are the maps of head h.  Tokens of
// the sequences alone: others are not read.
__global__ void __launch_bounds__(kDiffThreads) kvq_diff_expand_kernel(const __half* q, __half* out, const int* q_start,
                                                                       int S, int64_t chunks, int H, int cpr_log2) {
  // a thread: 8 channels of one map's half row, and zeros in the other map's row
  const int64_t i = (int64_t)blockIdx.x * kDiffThreads + threadIdx.x;
  if (i >= chunks || i < (int64_t)q_start[0] * H << cpr_log2 || i >= (int64_t)q_start[S] * H << cpr_log2) return;
  const uint4 v = reinterpret_cast<const uint4*>(q)[i];
  const int64_t row = i >> cpr_log2;
  const int c = static_cast<int>(i & ((1 << cpr_log2) - 1)), map = c >> (cpr_log2 - 1);
  uint4* dst = reinterpret_cast<uint4*>(out) + (row << (cpr_log2 + 1)) + c;
  dst[map << cpr_log2] = v;
  dst[(map ^ 1) << cpr_log2] = make_uint4(0, 0, 0, 0);
}

// o [T][2H][D] -> the normed differences [T][H][D], a warp for each.  Rows that the prefill
// did not write are left as they were: before the first sequence, behind the last, and past
// max_q_len in one.
template <int D>
__global__ void __launch_bounds__(kDiffThreads) kvq_diff_combine_kernel(const float* o, const int* q_start, int S,
                                                                        int max_q_len, int64_t heads, int H, DiffOut p) {
  constexpr int NE = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (kDiffThreads / 32) + (threadIdx.x >> 5);
  if (i >= heads) return;
  const float* a = o + i * 2 * D + lane * NE;
  float y0[NE], y1[NE];  // (on their way while the row's sequence is looked up)
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    y0[e] = a[e];
    y1[e] = a[D + e];
  }
  const int row = static_cast<int>(i / H);
  if (row < q_start[0] || row >= q_start[S]) return;
  int lo = 0;  // q_start[lo] <= row: of 32 at a time
  for (int n = S; n > 1;) {
    const int step = (n + 31) / 32, at = lane * step;
    const int last = __popc(__ballot_sync(0xffffffffu, at < n && q_start[lo + min(at, n - 1)] <= row)) - 1;
    lo += last * step;
    n = min(step, n - last * step);
  }
  if (row - q_start[lo] >= max_q_len) return;
  const float lam = p.lambda[i - (int64_t)row * H];
  float y[NE], ss = 0.f;
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    y[e] = y0[e] - lam * y1[e];
    ss = fmaf(y[e], y[e], ss);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
  const float f = diff_factor<D>(p, ss);
  __half* dst = p.out + i * D + lane * NE;
#pragma unroll
  for (int e = 0; e < NE; ++e)
    dst[e] = __float2half_rn(y[e] * (p.weight != nullptr ? f * p.weight[lane * NE + e] : f));
}

bool two_maps(const PoolView& pool) {
  return prefill_tc_supported(pool) && pool.fmt != FMT_INT8_CHANNEL;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_diff_block(const DecodeLaunch& l);  // kvq_diff_decode.cu
cudaError_t launch_diff_misc(const DecodeLaunch& l);
cudaError_t launch_diff_group(const DecodeLaunch& l);  // kvq_diff_decode_group.cu
cudaError_t launch_diff_fp4(const DecodeLaunch& l);    // kvq_decode_fp4.cu

cudaError_t launch_decode_diff(const DecodeLaunch& l) {
  const int f = l.p.pool.fmt;
  if (fmt_block(f)) return launch_diff_block(l);
  if (f == FMT_FP4) return launch_diff_fp4(l);
  return f == FMT_INT8_GROUP || f == FMT_INT4_GROUP ? launch_diff_group(l) : launch_diff_misc(l);
}

size_t diff_prefill_ws_bytes(const PoolView& pool, int64_t T, int S, int H, int max_ctx) {
  if (two_maps(pool)) return prefill_ws_bytes(pool, S, max_ctx);
  const size_t rows = (size_t)T * 2 * H * pool.D;
  return up256(rows * sizeof(__half)) + up256(rows * sizeof(float)) + prefill_ws_bytes(pool, S, max_ctx);
}

cudaError_t launch_diff_prefill(const PoolView& pool, const __half* q, int64_t T, int S, int H,
                                const int* q_start, int max_q_len, const int* table, int max_blocks,
                                const int* lens, int max_ctx, float sm_scale, const DiffOut& diff,
                                void* ws, cudaStream_t st) {
  if (two_maps(pool))
    return launch_prefill_ws(pool, q, S, H, q_start, max_q_len, table, max_blocks, lens, max_ctx, sm_scale,
                             nullptr, ws, st, &diff);
  const int D = pool.D;
  const size_t rows = (size_t)T * 2 * H * D;
  __half* qx = static_cast<__half*>(ws);
  float* o = reinterpret_cast<float*>(static_cast<char*>(ws) + up256(rows * sizeof(__half)));
  void* rec = reinterpret_cast<char*>(o) + up256(rows * sizeof(float));
  const int64_t chunks = T * H * (D / 8), heads = T * H;
  const int64_t eg = (chunks + kDiffThreads - 1) / kDiffThreads, cg = (heads + 7) / 8;
  if (eg > 0x7fffffffLL || cg > 0x7fffffffLL) return cudaErrorInvalidValue;
  kvq_diff_expand_kernel<<<static_cast<unsigned>(eg), kDiffThreads, 0, st>>>(q, qx, q_start, S, chunks, H, D == 64 ? 3 : 4);
  cudaError_t e = phase_mark(st, cudaGetLastError());
  if (e != cudaSuccess) return e;
  e = prefill_ws_bytes(pool, S, max_ctx) > 0
          ? launch_prefill_ws(pool, qx, S, 2 * H, q_start, max_q_len, table, max_blocks, lens, max_ctx,
                              sm_scale, o, rec, st)
          : launch_prefill(pool, qx, S, 2 * H, q_start, max_q_len, table, max_blocks, lens, max_ctx,
                           sm_scale, o, st);
  if (e != cudaSuccess) return e;
  if (D == 64)
    kvq_diff_combine_kernel<64><<<static_cast<unsigned>(cg), kDiffThreads, 0, st>>>(o, q_start, S, max_q_len, heads, H, diff);
  else
    kvq_diff_combine_kernel<128><<<static_cast<unsigned>(cg), kDiffThreads, 0, st>>>(o, q_start, S, max_q_len, heads, H, diff);
  return phase_mark(st, cudaGetLastError());
}

}  // namespace kvq
