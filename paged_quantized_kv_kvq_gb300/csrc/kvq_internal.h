// kvq_internal.h -- host-side declarations shared by the C ABI and the kernel
// translation units.  Not part of the public interface.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime_api.h>

#include "kvq.h"
#include "kvq_common.cuh"

namespace kvq {

// Differential attention: the two halves of a head's channels are two maps over one V,
//   y = softmax(s q1.k1) V - lambda softmax(s q2.k2) V,
//   out = out_scale * y / sqrt(mean(y^2) + eps) * weight  (no norm without a weight).
// To the kernels a head is two Q rows, 2i and 2i + 1 of its group, each q with the other
// half zero: what the heads of a group share -- the page, its conversion, the products'
// n dimension -- the maps share too.
struct DiffOut {
  const float* lambda = nullptr;  // [heads]
  const float* weight = nullptr;  // [D] or null
  __half* out = nullptr;          // [rows][heads][D]
  float eps = 0.f, out_scale = 1.f;
};

cudaError_t launch_append(const PoolView& pool, const __half* k, const __half* v,
                          const int64_t* slots, int64_t T, cudaStream_t st);
// Append with slots from `slots`, or -- when slots is null -- the decode-step
// form: token t is sequence t's new token, stored at position lens[t]-1.
// `dependent`: launch as a programmatic dependent of the previous kernel (the
// kernel waits for its completion before reading anything).  `x_stride`:
// elements between consecutive tokens of k and v (0 = kv_heads * head_dim).
cudaError_t launch_step_append(const PoolView& pool, const __half* k, const __half* v,
                               const int64_t* slots, int64_t T, const int* table, const int* lens,
                               int max_blocks, int max_ctx, cudaStream_t st, bool dependent,
                               int64_t x_stride = 0);
cudaError_t launch_copy_blocks(const PoolView& pool, const int* src, const int* dst, int n,
                               cudaStream_t st);
cudaError_t launch_calibrate(const PoolView& pool, const __half* k, const __half* v, int64_t T,
                             cudaStream_t st);
cudaError_t launch_read_slots(const PoolView& pool, const int64_t* slots, int64_t n,
                              void* codes_out, float* scales_out, cudaStream_t st);

// Norm, rotation, quantization and scatter of new tokens in one kernel
// (kvq_ingest_impl.cuh).  Q rows (when there are any) are normed, rotated and
// written as fp16; K rows are normed, rotated, quantized from fp32 and stored
// with V in the pool.  With `slots` null the slots come from table / lens as in
// launch_step_append.
struct IngestArgs {
  PoolView pool;
  const void* q = nullptr;
  const void* k = nullptr;
  const void* v = nullptr;
  int64_t q_stride = 0, k_stride = 0, v_stride = 0;  // elements between tokens
  bool bf16 = false;                                 // q, k, v are bfloat16 (else fp16)
  const int64_t* positions = nullptr;
  const int64_t* slots = nullptr;
  const int* table = nullptr;
  const int* lens = nullptr;
  int max_blocks = 0, max_ctx = 0;
  int64_t T = 0;
  int Hq = 0;
  const float* q_weight = nullptr;  // null: no norm
  const float* k_weight = nullptr;
  float eps = 0.f;
  __half* q_out = nullptr;
  int64_t q_out_stride = 0;
  const kvq_rope_plan* plan = nullptr;  // null: no rotation
};
cudaError_t launch_ingest(const IngestArgs& a, cudaStream_t st, bool dependent);

// Norm and rotation of Q and K rows to fp16 (kvq_rope.cu).
struct RopeArgs {
  const void* x[2] = {};  // q, k
  int64_t x_stride[2] = {};
  __half* out[2] = {};
  int64_t out_stride[2] = {};
  int heads[2] = {};
  const float* weight[2] = {};
  bool bf16 = false;
  const int64_t* positions = nullptr;
  int64_t T = 0;
  int D = 0;
  float eps = 0.f;
  const kvq_rope_plan* plan = nullptr;
};
// `beside`: launch while the kernel before it on the stream still runs (which
// must let its dependents launch and touch nothing that this call touches); the
// call's kernel ends after that one.
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st, bool beside = false);

// Dequantized fp16 K and V of n slots, [n][Hkv][D] each.
cudaError_t launch_read_values(const PoolView& pool, const int64_t* slots, int64_t n, __half* k,
                               __half* v, cudaStream_t st);

// Long appends to pools of 4-bit floats, and their read-back (kvq_fp4_rows.cu).
cudaError_t launch_append4(const PoolView& pool, const __half* k, const __half* v, int64_t stride,
                           const int64_t* slots, int64_t T, cudaStream_t st);
cudaError_t launch_read_values4(const PoolView& pool, const int64_t* slots, int64_t n, __half* k,
                                __half* v, cudaStream_t st);

// Attention weights of the cached tokens (kvq_weights_impl.cuh), from the
// log-sum-exps of a decode of the same rows.
struct WeightsArgs {
  PoolView pool;
  const __half* q;
  const int* table;
  const int* lens;
  const float* lse;   // [S][Hq]
  const float* prev;  // [S][Hkv][stride] or null
  float* scores;      // [S][Hkv][stride]
  int64_t stride;
  float decay;
  int S, Hq, max_blocks, max_ctx;
  float sm_scale;
  int sms;  // SMs of the device
};
cudaError_t launch_weights(const WeightsArgs& a, cudaStream_t st);

// Blocks with the least accumulated weight leave their sequences (kvq_evict.cu).
constexpr int kEvictMaxBlocks = 28672;  // of one sequence: two words each in shared memory
struct EvictArgs {
  const float* scores;  // [S][Hkv][stride]
  int64_t stride;
  const int* lens;
  const int* table;
  int* table_out;
  int* lens_out;
  int* kept;          // [S][budget] or null
  float* scores_out;  // [S][Hkv][out_stride] or null
  int64_t out_stride;
  int* err;
  int S, Hkv, bs, max_blocks, max_ctx, budget, sink, recent;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st);

// Launch geometry of one decode call.
struct DecodePlan {
  int grid = 0;         // persistent CTAs
  int ppw_fixed = 0;    // pages per warp when forced; 0 = balanced
  int n_ht = 0;         // head tiles of 8 Q heads per kv head
  int nstage = 0;  // pipeline stages per warp
  int part_rows = 0;    // rows of a split partial
  int stage_bytes = 0;  // bytes of one stage
  int smem_bytes = 0;   // dynamic shared memory per CTA
  int merge_grid = 0;   // CTAs of the merge kernel
  int merge_chunk = 8;  // pieces the merge loads per round trip
  bool two_ctas = false;  // two resident CTAs per SM instead of three
  size_t ps_bytes = 0;  // page prefix at the start of the workspace
  size_t ws_bytes = 0;  // page prefix + split partials
};

// Plan a decode call; `sms` is the device's SM count.  Returns false for an
// unsupported geometry.
bool plan_decode(const PoolView& pool, int S, int Hq, int max_ctx, int split_blocks, int sms,
                 DecodePlan* plan);

struct DecodeArgs {
  PoolView pool;
  const __half* q;
  const int* table;
  const int* lens;
  float* out;
  void* workspace;
  int S, Hq, max_blocks, max_ctx;
  float sm_scale;
  // shared-prefix cascade: skip the first `skip` blocks of every sequence and
  // fold in the prefix partials `pre` ([S][Hq][D+2]); 0 / null otherwise
  int skip = 0;
  const float* pre = nullptr;
  int64_t q_stride = 0, out_stride = 0;  // elements between sequences' rows; 0 = Hq * D
  float* lse = nullptr;  // [S][Hq] log of the softmax denominators; null = not wanted
  DiffOut diff;          // differential attention (Hq counts both maps) if diff.lambda is set
  int wait_tries = kWaitTries;  // bound of each pipeline wait, in ~1 ms tries
  int fault_issue = -1;   // self-test only: withhold warp 0's copy of this index
};

// `dependent`: launch the decode as a programmatic dependent of the kernel
// just before it on the stream (the decode-step append).
cudaError_t launch_decode(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t st,
                          bool dependent = false);

// Shared-prefix attention (kvq_rows_impl.cuh): the first P blocks of every
// sequence (those of table row 0) attended once per kv head for all
// sequences' Q rows, writing the partial rows out[S][Hq][D+2] (m, l, O) that
// a decode with skip = P folds in.
struct RowsPlan {
  int grid = 0, ntiles = 0, nstage = 0, stage_bytes = 0, bar_off = 0, smem_bytes = 0;
};
bool plan_rows(const PoolView& pool, int S, int Hq, RowsPlan* plan);
struct RowsArgs {
  PoolView pool;
  const __half* q;
  const int* table;
  const int* lens;
  float* out;
  int S, Hq, max_blocks, max_ctx;
  int P = 0;
  float sm_scale;
};
cudaError_t launch_rows(const RowsArgs& a, const RowsPlan& plan, cudaStream_t st, bool dependent);

// Prefill / chunked prefill (kvq_prefill_impl.cuh): the query tokens
// q_start[s]..q_start[s+1]-1 of each sequence attend causally to its cache.
cudaError_t launch_prefill(const PoolView& pool, const __half* q, int S, int Hq, const int* q_start,
                           int max_q_len, const int* table, int max_blocks, const int* lens,
                           int max_ctx, float sm_scale, float* out, cudaStream_t st);

// The same on the 5th-generation tensor cores (kvq_prefill_tc_impl.cuh): for
// formats with at most one scale per token and K|V (per-group only when the
// group is the whole head), head_dim 64 or 128, blocks of 16 tokens or more.
bool prefill_tc_supported(const PoolView& pool);
cudaError_t launch_prefill_tc(const PoolView& pool, const __half* q, int S, int Hq,
                              const int* q_start, int max_q_len, const int* table, int max_blocks,
                              const int* lens, int max_ctx, float sm_scale, float* out,
                              cudaStream_t st);

// Prefill in two passes through a workspace (kvq_prefill_ws_impl.cuh): the
// codes of every 64-token key step staged once as fp16 tiles, then the
// attention pass.  Same formats as launch_prefill_tc; 0 bytes otherwise.
size_t prefill_ws_bytes(const PoolView& pool, int S, int max_ctx);
cudaError_t launch_prefill_ws(const PoolView& pool, const __half* q, int S, int Hq,
                              const int* q_start, int max_q_len, const int* table, int max_blocks,
                              const int* lens, int max_ctx, float sm_scale, float* out, void* ws,
                              cudaStream_t st, const DiffOut* diff = nullptr);
// (diff: differential attention, Hq heads, rows to diff->out; not for per-channel pools.)

// Differential attention of prompts (kvq_diff.cu); T rows of q and out, H heads.
size_t diff_prefill_ws_bytes(const PoolView& pool, int64_t T, int S, int H, int max_ctx);
cudaError_t launch_diff_prefill(const PoolView& pool, const __half* q, int64_t T, int S, int H,
                                const int* q_start, int max_q_len, const int* table, int max_blocks,
                                const int* lens, int max_ctx, float sm_scale, const DiffOut& diff,
                                void* ws, cudaStream_t st);

// Block tables, slot map and positions of a step (kvq_blocks.cu).
struct ExtendArgs {
  const int* n;     // [S] new tokens
  const int* lens;  // [S]
  int* table;       // [S][max_blocks]
  const int* free_list;
  const int* count;
  int* lens_out;
  int* count_out;
  int* q_start;        // [S + 1]
  int64_t* slots;      // [max_tokens]
  int64_t* positions;  // [max_tokens]
  int* err;
  int64_t num_blocks;
  int S, max_blocks, capacity, max_tokens, bs;
  bool wide;  // slots and positions lie at 16-byte boundaries (set by the launcher)
};
cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t st);
struct ReleaseArgs {
  const int* table;
  const int* old_lens;
  const int* new_lens;
  int* free_list;
  const int* count;
  int* count_out;
  int* err;
  int64_t num_blocks;
  int S, max_blocks, capacity, shared, bs;
};
cudaError_t launch_release(const ReleaseArgs& a, cudaStream_t st);

// Per-format kernel launchers (one translation unit each, compiled in parallel).
struct DecodeLaunch;
cudaError_t launch_decode_int8_group(const DecodeLaunch& l);
cudaError_t launch_decode_int4_group(const DecodeLaunch& l);
cudaError_t launch_decode_fp16(const DecodeLaunch& l);
cudaError_t launch_decode_token(const DecodeLaunch& l);
cudaError_t launch_decode_channel(const DecodeLaunch& l);
cudaError_t launch_decode_e5m2(const DecodeLaunch& l);
cudaError_t launch_decode_bs8_group(const DecodeLaunch& l);  // block size 8, INT8 per-group
cudaError_t launch_decode_bs8_misc(const DecodeLaunch& l);   // block size 8, the other formats
cudaError_t launch_decode_fp4(const DecodeLaunch& l);
cudaError_t launch_decode_diff(const DecodeLaunch& l);  // differential, every format
cudaError_t launch_decode_block(const DecodeLaunch& l);      // one scale per block, every block size

}  // namespace kvq
