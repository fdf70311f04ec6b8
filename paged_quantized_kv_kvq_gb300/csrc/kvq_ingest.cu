// kvq_ingest.cu -- launch planning of the ingest kernel (kvq_ingest_impl.cuh),
// its formats with one scale per block, and the read-back of slots as values.
#include <algorithm>

#include "kvq_ingest_impl.cuh"

namespace kvq {

namespace {

// K and V of 16 slots (long calls: 32 or 64) of one kv head per CTA, as fp16: code
// times scale in fp32, rounded once.  A thread takes 8 channels of one slot: its K
// codes are two neighbouring words of the page, its V codes lie in eight words 64 bytes
// apart, each shared with three other tokens, so a sub-tile's sectors come from
// L2 once and from L1 for its other slots.  The bound for few slots is one chain
// of loads.  Where the 16 slots are a sub-tile in its order (long calls), a thread
// takes 8 channels of the four tokens that share V words instead and every word
// is read once; the bound then is HBM and the instructions that widen and round
// (16384 slots x 8 heads of INT8: 18 us, of which HBM would take 15; 25 with 128
// threads to a sub-tile, half of them idle).
constexpr int kValueSlots = 16;

// Channels 8ci .. 8ci+7 of tokens 2j, 2j+1, 2j+8, 2j+9 of the sub-tile at offset
// `off` of block blk (one-byte codes); token t's values go to out + t rows.
template <int FMT>
__device__ __forceinline__ void read_tile(const PoolView& pool, int64_t blk, int off, int kv, int h,
                                          int ci, int j, __half* out) {
  const int D = pool.D, d0 = 8 * ci;
  const int64_t row = (int64_t)pool.Hkv * D;
  const char* page = pool.pages + (blk * pool.Hkv + h) * pool.page_bytes;
  const char* tile = page + (kv == 0 ? 0 : pool.v_off) + (off >> 4) * pool.sub_bytes;
  const float* sc = reinterpret_cast<const float*>(page + 2 * pool.code_bytes);
  uint32_t w[8];  // K: token c's two words; V: a word per channel, a byte per token
  if (kv == 0) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const char* at = tile + k_tile_offset(2 * j + (c & 1) + 8 * (c >> 1), d0, D, 1);
      w[2 * c] = *reinterpret_cast<const uint32_t*>(at);
      w[2 * c + 1] = *reinterpret_cast<const uint32_t*>(at + 16);
    }
  } else {
    const char* at = tile + v_tile_offset(2 * j, d0, D, 1);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = *reinterpret_cast<const uint32_t*>(at + 64 * e);
  }
  float s[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int t = off + 2 * j + (c & 1) + 8 * (c >> 1);
    if constexpr (FMT == FMT_INT8_GROUP)
      s[c] = sc[(kv * pool.bs + t) * pool.ng + d0 / pool.group];
    else if constexpr (fmt_block(FMT))
      s[c] = sc[kv];
    else if constexpr (FMT == FMT_INT8_TOKEN || FMT == FMT_FP8_TOKEN)
      s[c] = pool.tok_scales[(blk * 2 + kv) * pool.bs + t];
  }
  __half2 q[8][2];  // the words' codes, exact in fp16
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t lo, hi;
    if constexpr (fmt_e4m3(FMT))
      e4m3x4_to_h2x2(w[i], lo, hi);
    else if constexpr (FMT == FMT_FP8_E5M2)
      e5m2x4_to_h2x2(w[i], lo, hi);
    else
      i8x4_to_h2x2(w[i], lo, hi);
    q[i][0] = *reinterpret_cast<__half2*>(&lo);
    q[i][1] = *reinterpret_cast<__half2*>(&hi);
  }
  float chs[8];
  if constexpr (FMT == FMT_INT8_CHANNEL)
#pragma unroll
    for (int e = 0; e < 8; ++e) chs[e] = pool.chan_scales[((int64_t)kv * pool.Hkv + h) * D + d0 + e];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __half2 pr = kv == 0 ? q[2 * c + (e >> 2)][(e >> 1) & 1] : q[e][c >> 1];
      const bool odd = kv == 0 ? e & 1 : c & 1;
      x[e] = (odd ? __high2float(pr) : __low2float(pr)) * (FMT == FMT_INT8_CHANNEL ? chs[e] : s[c]);
    }
    const int t = 2 * j + (c & 1) + 8 * (c >> 1);
    *reinterpret_cast<uint4*>(out + t * row) = narrow8(x);
  }
}

template <int FMT>
__global__ void __launch_bounds__(256) kvq_read_values_kernel(PoolView pool, int bs_log2, int tpt_log2,
                                                              const int64_t* slots, int64_t n,
                                                              __half* k, __half* v) {
  // (powers of two throughout: a division costs as much as the rest of a row)
  const int D = pool.D, lph_log2 = D == 64 ? 3 : 4, lph = 1 << lph_log2, tpt = 1 << tpt_log2;
  const int kv = threadIdx.x >> 7;  // 128 threads each for K and V
  const int h = blockIdx.y;
  const int unit = threadIdx.x & 127 & (tpt - 1);  // of the tpt threads (whole warps) of its 16 slots
  const int64_t i0 = (((int64_t)blockIdx.x << (7 - tpt_log2)) + ((threadIdx.x & 127) >> tpt_log2)) * kValueSlots;
  if (FMT != FMT_FP16 && !fmt_4bit(FMT) && pool.bs >= 16 && i0 + kValueSlots <= n) {
    const int64_t first = slots[i0];
    const int lane = threadIdx.x & 15;
    if (__all_sync(0xffffffffu, slots[i0 + lane] == first + lane) && first >= 0 && (first & 15) == 0 &&
        first < pool.num_blocks * pool.bs) {
      const int ci = unit & (lph - 1), j = unit >> lph_log2;
      if (j < 4)
        read_tile<FMT>(pool, first >> bs_log2, static_cast<int>(first & (pool.bs - 1)), kv, h, ci, j,
                       (kv == 0 ? k : v) + (i0 * pool.Hkv + h) * D + 8 * ci);
      return;
    }
  }
  for (int u = unit; u < kValueSlots * lph; u += tpt) {
    const int64_t i = i0 + (u >> lph_log2);
    if (i >= n) return;
    const int ci = u & (lph - 1), d0 = 8 * ci;
    const int64_t slot = slots[i];
    if (slot < 0) continue;
    if (slot >= pool.num_blocks * pool.bs) {
      set_error(pool.err, ERR_RANGE);
      continue;
    }
    const int64_t blk = slot >> bs_log2;
    const int off = static_cast<int>(slot & (pool.bs - 1)), t = off & 15;
    const char* page = pool.pages + (blk * pool.Hkv + h) * pool.page_bytes;
    const char* tile = page + (kv == 0 ? 0 : pool.v_off) + (off >> 4) * pool.sub_bytes;
    const float* sc = reinterpret_cast<const float*>(page + 2 * pool.code_bytes);
    // the first of the thread's words: lane and word of (t, d0) in the sub-tile
    int lane, word;
    if (kv == 0) {
      lane = (t & 7) * 4 + 2 * (ci & 1);
      word = (fmt_4bit(FMT) ? 0 : (t >> 3) * (D >> 4)) + (ci >> 1);
    } else {
      lane = (t & 7) >> 1;
      word = fmt_4bit(FMT) || pool.bs == 8 ? ci >> 1 : ci;
    }
    constexpr int WB = FMT == FMT_FP16 ? 8 : 4;  // bytes of a word of four elements (4-bit codes: eight)
    const char* at = tile + (word / (16 / WB)) * 512 + lane * 16 + word % (16 / WB) * WB;
    uint2 w[8];  // V: one word per channel; K: one per four channels
    if (kv == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[e] = FMT == FMT_FP16 ? *reinterpret_cast<const uint2*>(at + 16 * e)
                               : make_uint2(*reinterpret_cast<const uint32_t*>(at + 16 * e), 0);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = FMT == FMT_FP16 ? *reinterpret_cast<const uint2*>(at + 64 * e)
                               : make_uint2(*reinterpret_cast<const uint32_t*>(at + 64 * e), 0);
    }
    float s = 1.f;
    if constexpr (FMT == FMT_INT8_GROUP || FMT == FMT_INT4_GROUP)
      s = sc[(kv * pool.bs + off) * pool.ng + d0 / pool.group];
    else if constexpr (FMT == FMT_FP4)
      s = fp4_scale_value(static_cast<uint8_t>(
          page[(kv == 0 ? 0 : pool.v_off) + pool.code_bytes + (off >> 4) * D +
               (kv == 0 ? fp4_k_scale(t, ci >> 1, pool.ng) : fp4_v_scale(t, ci >> 1, pool.ng))]));
    else if constexpr (fmt_block(FMT))
      s = sc[kv];
    else if constexpr (FMT == FMT_INT8_TOKEN || FMT == FMT_FP8_TOKEN)
      s = pool.tok_scales[(blk * 2 + kv) * pool.bs + off];
    const float* chs = pool.chan_scales + ((int64_t)kv * pool.Hkv + h) * D + d0;
    // element of this token in a V word
    const int ev = pool.bs == 8 ? (t & 1) + 2 * (ci & 1) : (t & 1) + 2 * (t >> 3);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint2 q = kv == 0 ? w[e >> 2] : w[e];
      const int el = kv == 0 ? e & 3 : ev;
      if constexpr (FMT == FMT_FP4) {
        const int sh = kv == 0 ? fp4_k_shift(t, el) : fp4_v_shift(t, d0);
        x[e] = fp4_code_value(q.x >> sh & 0xFu) * s;
      } else if constexpr (FMT == FMT_INT4_GROUP) {
        const int sh = kv == 0 ? nib_shift((t >> 3) * 4 + el) : nib_shift(el + 4 * (ci & 1));
        x[e] = static_cast<float>(static_cast<int>(q.x >> sh & 0xFu) - static_cast<int>(kInt4Bias)) * s;
      } else if constexpr (FMT == FMT_FP16) {
        const uint32_t hw = el & 2 ? q.y : q.x;
        x[e] = __half2float(__ushort_as_half(static_cast<unsigned short>(hw >> (16 * (el & 1)))));
      } else {
        const uint8_t c = static_cast<uint8_t>(q.x >> (8 * el));
        if constexpr (FMT == FMT_FP8_E5M2)
          x[e] = __half2float(__ushort_as_half(static_cast<unsigned short>(c << 8)));
        else
          x[e] = code_value<FMT>(c) * (FMT == FMT_INT8_CHANNEL ? chs[e] : s);
      }
    }
    *reinterpret_cast<uint4*>((kv == 0 ? k : v) + (i * pool.Hkv + h) * D + d0) = narrow8(x);
  }
}

}  // namespace

cudaError_t launch_read_values(const PoolView& pool, const int64_t* slots, int64_t n, __half* k,
                               __half* v, cudaStream_t st) {
  // Threads of 16 slots: all 128 for a short call's latency, the 4 per 8 channels that
  // a sub-tile takes for a long one.  (8 heads of 128, slots in order: 1024 slots 2.7 and
  // 2.8 us, 2048 4.0 and 3.7, 16384 22.2 and 19.4; scattered: 256 2.9 and 3.7, 2048 5.9
  // and 6.1, 16384 36.1 and 32.4.)
  const int tpt_log2 = n < 2048 ? 7 : pool.D == 64 ? 5 : 6;
  const int64_t spc = kValueSlots << (7 - tpt_log2), gx = (n + spc - 1) / spc;
  if (gx > 0x7fffffffLL || pool.Hkv > 65535) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(gx), pool.Hkv);
  int log2 = 0;
  while ((1 << log2) < pool.bs) ++log2;
  auto run = [&](auto kernel) { kernel<<<grid, 256, 0, st>>>(pool, log2, tpt_log2, slots, n, k, v); };
  switch (pool.fmt) {
    case FMT_FP16: run(kvq_read_values_kernel<FMT_FP16>); break;
    case FMT_INT8_TOKEN: run(kvq_read_values_kernel<FMT_INT8_TOKEN>); break;
    case FMT_INT8_CHANNEL: run(kvq_read_values_kernel<FMT_INT8_CHANNEL>); break;
    case FMT_INT8_GROUP: run(kvq_read_values_kernel<FMT_INT8_GROUP>); break;
    case FMT_FP8_TOKEN: run(kvq_read_values_kernel<FMT_FP8_TOKEN>); break;
    case FMT_INT4_GROUP: run(kvq_read_values_kernel<FMT_INT4_GROUP>); break;
    case FMT_FP8_E5M2: run(kvq_read_values_kernel<FMT_FP8_E5M2>); break;
    case FMT_INT8_BLOCK: run(kvq_read_values_kernel<FMT_INT8_BLOCK>); break;
    case FMT_FP8_BLOCK: run(kvq_read_values_kernel<FMT_FP8_BLOCK>); break;
    case FMT_FP4:  // (n = 1024, this kernel and that one: slots in order 3.9 and 3.3 us,
                   // scattered 4.3 and 5.3; 2048: 6.6 and 4.6, 7.3 and 6.9; 16384: 34 and 18, 49 and 48)
      if (n >= 2048) return launch_read_values4(pool, slots, n, k, v, st);
      run(kvq_read_values_kernel<FMT_FP4>);
      break;
    default: return cudaErrorInvalidValue;
  }
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
  // Few tokens (a decode step, a short prompt): one per CTA, and one head per CTA
  // (four above 128 tokens) for the latency of a run.  Many: several tokens per
  // CTA, and heads for kIngestRounds rounds of its warps, which share its angles.
  // (Prompts with 32 query heads: 1000 tokens 19.7 us as few, 23.5 as many, 2048
  // tokens 34.5 and 17.7; single tokens 24.4 and 26.0, 47.0 and 30.4.  One head per CTA
  // against four: 128 tokens 7.5 and 8.0 us, 256 tokens 10.5 and 8.8, single tokens
  // 7.6 and 5.2, 11.7 and 6.5.)  Formats with one scale per token need every head of a
  // token in one CTA.
  // A long call's query rows go to a kernel of their own, launched beside this
  // one: this one's 128 registers leave an SM 16 warps, too few loads in flight
  // for the rows that are most of the bytes (16384 tokens, 32 Q and 8 kv heads:
  // 154 us in one kernel).
  const bool many = a.T >= 1024;
  const bool tok = a.pool.fmt == FMT_INT8_TOKEN || a.pool.fmt == FMT_FP8_TOKEN;
  // A long call's CTA takes 8 tokens whatever the call's length: its runs may be whole
  // blocks, chunks that begin inside one, or single tokens, and the last two it takes one
  // after the other.  8 kv heads, blocks of 16, 16384 tokens with 4, 8 and 16 a CTA:
  // prompts of whole blocks 54.5, 47.5 and 44.3 us (the CTAs that own no run cost that
  // much), chunks from inside a block 89.1, 80.5 and 85.3, single tokens 154.7, 159.3
  // and 163.8, a prompt with 64 single tokens 54.7, 56.3 and 71.5; 2048 tokens: 17.1,
  // 15.5 and 13.4; 40.9, 38.9 and 48.6; 29.8, 27.7 and 44.5; 17.4, 23.8 and 40.0.
  p.tpc = !many || a.slots == nullptr ? 1 : std::min(a.pool.bs, 8);
  const int round_heads = std::max(1, kIngestWarps * 1024 / (std::max(a.pool.bs, 16) * a.pool.D));
  p.hpc = tok ? a.pool.Hkv : many ? kIngestRounds * round_heads : a.T > 128 ? 4 : 1;
  p.hsplit = (a.pool.Hkv + p.hpc - 1) / p.hpc;
  p.kv_ctas = (a.T + p.tpc - 1) / p.tpc * p.hsplit * 2;
  int64_t q_ctas = 0;
  if (a.Hq > 0 && !many) {
    const int rpp = kIngestThreads / (a.pool.D / 8);
    p.q_parts = (a.Hq + rpp - 1) / rpp;
    q_ctas = a.T * p.q_parts;
  }
  if (p.kv_ctas + q_ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  l.grid = static_cast<unsigned>(p.kv_ctas + q_ctas);
  l.smem = ingest_smem(a.pool, p.plan.rotary_dim);
  l.st = st;
  l.dependent = dependent;
  cudaError_t e;
  switch (a.pool.fmt) {
    case FMT_INT8_BLOCK:
    case FMT_FP8_BLOCK: e = launch_ingest_block(l); break;
    case FMT_INT8_GROUP:
    case FMT_INT4_GROUP:
    case FMT_FP4: e = launch_ingest_group(l); break;
    case FMT_INT8_TOKEN:
    case FMT_FP8_TOKEN: e = launch_ingest_token(l); break;
    default: e = launch_ingest_misc(l);
  }
  if (e != cudaSuccess || a.Hq == 0 || !many) return e;
  RopeArgs q;
  q.x[0] = a.q;
  q.x_stride[0] = a.q_stride;
  q.out[0] = a.q_out;
  q.out_stride[0] = a.q_out_stride;
  q.heads[0] = a.Hq;
  q.weight[0] = a.q_weight;
  q.bf16 = a.bf16;
  q.positions = a.positions;
  q.T = a.T;
  q.D = a.pool.D;
  q.eps = a.eps;
  q.plan = a.plan;
  return launch_rope(q, st, /*beside=*/true);
}

}  // namespace kvq
