// kvq_ingest_impl.cuh -- new tokens into the cache in one kernel: query rows
// normed and rotated to fp16; key rows normed, rotated and quantized straight
// from fp32; value rows quantized; keys and values stored in their slots.
//
// A CTA either turns query rows (kvq_rope_math.cuh) or takes runs of tokens: a
// run is a maximal stretch of the call's tokens whose slots lie in one block,
// and the CTA that owns its first token quantizes and stores the whole run,
// K or V, for `hpc` kv heads.  So
//  * the one scale of a (block, head) is an absmax inside one CTA, with no
//    atomics and no second kernel, whatever number of tokens the call brings;
//  * a 16-token sub-tile that the run covers is assembled in shared memory and
//    leaves as 16-byte stores, although its bytes interleave tokens.
// Bounds: the instructions that norm, rotate and quantize for prompts (16384
// tokens x 8 heads into INT8 blocks: 47 us, 27 million warp instructions, where HBM
// would take 15), latency for a decode step (one token per run: slot -> rows ->
// absmax -> codes; 5.9 us for 64 tokens with their 32 query heads into INT8 groups;
// into INT8 blocks 61 tokens take 4.4 us where no scale grows and 11 where nearly
// every one does, whose older codes are read, rounded again and written).
//
// One scale per (block, head): s = max(s_old, absmax / top) in fp32, where top
// is 127 or 448 and s_old the block's scale, unless the run writes offset 0,
// which starts the block anew.  Where s grew, the codes the block keeps are
// rounded again: code' = rne(code * s_old / s).
#pragma once
#include <cstdint>
#include <type_traits>

#include "kvq_context.h"
#include "kvq_fp4.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"
#include "kvq_rope_math.cuh"

namespace kvq {

constexpr int kIngestThreads = 128;
constexpr int kIngestWarps = kIngestThreads / 32;
constexpr int kMaxBlock = 64;  // largest block size
constexpr int kIngestRounds = 4;  // of ingest_whole per CTA

struct IngestParams {
  PoolView pool;
  RopeRows q;
  int Hq;
  const void* x[2];     // k, v
  int64_t stride[2];
  const float* k_weight;
  const int64_t* positions;
  const int64_t* slots;  // null: the decode-step form, from table and lens
  const int* table;
  const int* lens;
  int max_blocks, max_ctx;
  int64_t T;
  float eps;
  bool bf16;
  int bs_log2;
  int tpc, hpc, hsplit;  // tokens and heads per K/V CTA, CTAs over the heads
  int64_t kv_ctas;       // CTAs 0 .. kv_ctas-1 take K/V, the rest query rows
  int q_parts;           // CTAs a token's query rows are spread over
  kvq_rope_plan plan;
};

// Shared memory of a K/V CTA; `tile` and `cs` follow it.
struct IngestShared {
  int blk[2 * kMaxBlock + 1];  // block of window token i - 1 (-1: none)
  uint8_t off[2 * kMaxBlock];  // its offset in the block
  uint32_t cut[4];             // bit i: token i begins a new block
  uint32_t has[2];             // offsets the run writes
  float red[2 * kIngestWarps];
  uint32_t tok[kMaxBlock];     // per-token absmax, as bits
  int grown;                   // heads of a pass whose block scale grew
  int grown_head[16];
  float grown_from[16], grown_to[16];
};

// Slot of token t, or -1 (nothing to store).
__device__ __forceinline__ int64_t ingest_slot(const IngestParams& p, int64_t t) {
  if (p.slots != nullptr) return p.slots[t];
  const int L = p.lens[t];  // the decode flags a length beyond max_ctx; nothing is stored
  if (L <= 0 || L > p.max_ctx) return -1;
  const int b = p.table[t * p.max_blocks + ((L - 1) >> p.bs_log2)];
  return b < 0 ? p.pool.num_blocks * p.pool.bs
               : ((int64_t)b << p.bs_log2) + ((L - 1) & (p.pool.bs - 1));
}

// Store 8 codes of channels d0 .. d0+7 of token offset `off` into K (or V)
// codes at `base` (a page's, or its image in shared memory).
__device__ __forceinline__ void store_codes8(char* base, int kv, int off, int d0, int D, int bs,
                                             int sub_bytes, const uint8_t (&c)[8]) {
  char* tile = base + (off >> 4) * sub_bytes;
  const int tt = off & 15;
  if (kv == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint32_t*>(tile + k_tile_offset(tt, d0 + 4 * h, D, 1)) =
          c[4 * h] | (c[4 * h + 1] << 8) | (c[4 * h + 2] << 16) | ((uint32_t)c[4 * h + 3] << 24);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      tile[v_code_offset(tt, d0 + i, D, 1, bs)] = static_cast<char>(c[i]);
  }
}

// The scale byte of channels 16gi .. +15 of token offset `off` (4-bit floats).
template <int D>
__device__ __forceinline__ void store_fp4_scale(char* page, int kv, int off, int gi, const PoolView& pool,
                                                uint32_t code) {
  constexpr int NG = D / 16;
  page[(kv == 0 ? 0 : pool.v_off) + pool.code_bytes + (off >> 4) * D +
       (kv == 0 ? fp4_k_scale(off & 15, gi, NG) : fp4_v_scale(off & 15, gi, NG))] = static_cast<char>(code);
}

template <int FMT>
__device__ __forceinline__ uint8_t quant_byte(float x, float s) {
  if constexpr (fmt_e4m3(FMT))
    return quant_e4m3(x, s);
  else if constexpr (FMT == FMT_FP8_E5M2)
    return static_cast<uint8_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E5M2));
  else
    return quant_i8(x, s);
}

template <int FMT>
__device__ __forceinline__ float code_value(uint8_t c) {
  if constexpr (fmt_e4m3(FMT))
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
  else
    return static_cast<float>(static_cast<int>(c) - 128);
}

// Four codes (channel or token neighbours) of one scale, as a 32-bit word.
// (Not inlined: it would be there some thirty times, and is reached for one word
// in thousands where quant4_i8 serves.)
template <int FMT>
__device__ __noinline__ uint32_t quant_word(float x0, float x1, float x2, float x3, float s) {
  return quant_byte<FMT>(x0, s) | (uint32_t)quant_byte<FMT>(x1, s) << 8 |
         (uint32_t)quant_byte<FMT>(x2, s) << 16 | (uint32_t)quant_byte<FMT>(x3, s) << 24;
}

// The same with the scale's reciprocal where the format is INT8 (see quant4_i8).
template <int FMT>
__device__ __forceinline__ uint32_t quant_word_fast(const float (&x)[4], float s, float inv) {
  if constexpr (FMT == FMT_INT8_BLOCK || FMT == FMT_INT8_GROUP) {
    bool ok = inv > 0.f;
    const uint32_t w = quant4_i8(x, inv, ok);
    if (ok) return w;
  }
  return quant_word<FMT>(x[0], x[1], x[2], x[3], s);
}

// Four codes at scale s_old, rounded again at s (whose quant_inverse is inv).
template <int FMT>
__device__ __forceinline__ uint32_t rescale_word(uint32_t v, float s_old, float s, float inv) {
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = code_value<FMT>(v >> (8 * e) & 0xFF) * s_old;
  return quant_word_fast<FMT>(x, s, inv);
}

// A run of one token, K or V of every head: a row of lanes per head, a decode
// step's form.  Nothing is staged; with one scale per block the codes that the
// block keeps are touched only where its scale grows.
template <int FMT, int D>
__device__ __forceinline__ void ingest_token(const IngestParams& p, IngestShared& sh, float2* cs,
                                             int64_t t, int off, int64_t blk, int kv, uint4 first) {
  constexpr int LPH = D / 8, RPP = kIngestThreads / LPH;
  constexpr bool kBlock = fmt_block(FMT);
  constexpr bool kToken = FMT == FMT_INT8_TOKEN || FMT == FMT_FP8_TOKEN;
  constexpr float kTop = fmt_e4m3(FMT) ? 448.f : FMT == FMT_INT4_GROUP ? 7.f : 127.f;
  const PoolView& pool = p.pool;
  const int tid = threadIdx.x, ci = tid % LPH, r0 = tid / LPH, d0 = 8 * ci;
  const int bs = pool.bs, tt = off & 15, r = p.plan.rotary_dim;
  const bool turn = kv == 0 && r > 0, norm = kv == 0 && p.k_weight != nullptr;
  if (turn) rope_table<kIngestThreads>(p.plan, p.positions + t, 1, cs);
  if (tid == 0) {
    sh.tok[0] = 0;
    sh.grown = 0;
  }
  float w[8];
  if (norm)
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = p.k_weight[d0 + i];
  __syncthreads();
  float x[8];
  auto load = [&](int hb) {
    const int h = hb + r0;
    uint4 raw = first;
    if (hb > 0)
      raw = h < pool.Hkv ? *reinterpret_cast<const uint4*>(static_cast<const __half*>(p.x[kv]) +
                                                           t * p.stride[kv] + h * D + d0)
                         : make_uint4(0, 0, 0, 0);
    widen8(raw, p.bf16, x);
    if (norm) norm8<D>(x, w, p.eps);
    if (turn) rotate8<D>(x, ci, r, p.plan.layout == KVQ_ROPE_INTERLEAVED, cs);
  };
  auto absmax = [&](int lanes) {  // over the chunk and its neighbours
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
    for (int o = lanes >> 1; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
  };
  float s_tok = 0.f;
  if constexpr (kToken) {  // the scale of a token spans every head
    for (int hb = 0; hb < pool.Hkv; hb += RPP) {
      load(hb);
      const float a = absmax(32);
      if ((tid & 31) == 0) atomicMax(&sh.tok[0], __float_as_uint(a));
    }
    __syncthreads();
    s_tok = __fdiv_rn(__uint_as_float(sh.tok[0]), kTop);
    if (tid == 0) pool.tok_scales[(blk * 2 + kv) * bs + off] = s_tok;
  }
  for (int hb = 0; hb < pool.Hkv; hb += RPP) {
    if (!kToken || pool.Hkv > RPP) load(hb);
    const int h = hb + r0;
    const bool act = h < pool.Hkv;
    char* page = pool.pages + (blk * pool.Hkv + (act ? h : 0)) * pool.page_bytes;
    char* codes = page + (kv == 0 ? 0 : pool.v_off);
    float* scales = reinterpret_cast<float*>(page + 2 * pool.code_bytes);
    float s = s_tok;
    if constexpr (kBlock) {
      const float a = absmax(LPH);
      const float s_old = off == 0 || !act ? 0.f : scales[kv];
      s = fmaxf(s_old, __fdiv_rn(a, kTop));
      if (act && ci == 0 && off != 0 && s > s_old) {
        const int i = atomicAdd(&sh.grown, 1);
        sh.grown_head[i] = h;
        sh.grown_from[i] = s_old;
        sh.grown_to[i] = s;
      }
      __syncthreads();  // (every lane has read the old scales)
      const int grown = sh.grown;
      for (int i = 0; i < grown; ++i) {
        uint4* tile = reinterpret_cast<uint4*>(pool.pages + (blk * pool.Hkv + sh.grown_head[i]) * pool.page_bytes +
                                               (kv == 0 ? 0 : pool.v_off));
        const float from = sh.grown_from[i], to = sh.grown_to[i], inv = quant_inverse(to);
        for (int u = tid; u < pool.code_bytes / 16; u += kIngestThreads) {
          uint4 v = tile[u];
          v.x = rescale_word<FMT>(v.x, from, to, inv);
          v.y = rescale_word<FMT>(v.y, from, to, inv);
          v.z = rescale_word<FMT>(v.z, from, to, inv);
          v.w = rescale_word<FMT>(v.w, from, to, inv);
          tile[u] = v;
        }
      }
      __syncthreads();  // the rescaled codes are there, and the list has been read
      if (tid == 0) sh.grown = 0;
      if (act && ci == 0) scales[kv] = s;
      if (hb + RPP < pool.Hkv) __syncthreads();
    }
    char* tile = codes + (off >> 4) * pool.sub_bytes;
    if constexpr (FMT == FMT_INT8_GROUP || FMT == FMT_INT4_GROUP) {
      s = __fdiv_rn(absmax(pool.group >> 3), kTop);
      if (act && d0 % pool.group == 0) scales[(kv * bs + off) * pool.ng + d0 / pool.group] = s;
    }
    uint32_t sc4 = 0;
    if constexpr (FMT == FMT_FP4) {
      sc4 = fp4_scale_code(absmax(2));
      if (act && (d0 & 15) == 0) store_fp4_scale<D>(page, kv, off, d0 >> 4, pool, sc4);
    }
    if (!act) continue;
    if constexpr (FMT == FMT_FP16) {
      const uint4 o = narrow8(x);
      if (kv == 0) {
        *reinterpret_cast<uint2*>(tile + k_tile_offset(tt, d0, D, 2)) = make_uint2(o.x, o.y);
        *reinterpret_cast<uint2*>(tile + k_tile_offset(tt, d0 + 4, D, 2)) = make_uint2(o.z, o.w);
      } else {
        const uint16_t* half = reinterpret_cast<const uint16_t*>(&o);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint16_t*>(tile + v_code_offset(tt, d0 + i, D, 2, bs)) = half[i];
      }
    } else if constexpr (FMT == FMT_FP4) {
      store_fp4x8<false>(tile, kv, tt, d0, quant8_fp4(x, fp4_scale_value(sc4)));
    } else if constexpr (FMT == FMT_INT4_GROUP) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int sh4;
        const int o = kv == 0 ? k_nibble(tt, d0 + i, sh4) : v_nibble(tt, d0 + i, sh4);
        store_nibbles(tile + o, 0xFu << sh4, quant_i4(x[i], s) << sh4);
      }
    } else {
      uint8_t q[8];
      if constexpr (FMT == FMT_INT8_CHANNEL) {
        const float* chs = pool.chan_scales + ((int64_t)kv * pool.Hkv + h) * D + d0;
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = quant_byte<FMT>(x[i], chs[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = quant_byte<FMT>(x[i], s);
      }
      store_codes8(codes, kv, off, d0, D, bs, pool.sub_bytes, q);
    }
  }
  __syncthreads();
}

// One run: tokens t0 .. t0+n-1 of the call (window indices w0 ..), block blk.
template <int FMT, int D, int CPT>
__device__ __forceinline__ void ingest_run(const IngestParams& p, IngestShared& sh, char* tile,
                                           float2* cs, int64_t t0, int n, int w0, int64_t blk,
                                           int h0, int h1, int kv) {
  constexpr int LPH = D / 8, RPP = kIngestThreads / LPH;
  constexpr bool kBlock = fmt_block(FMT);
  constexpr bool kToken = FMT == FMT_INT8_TOKEN || FMT == FMT_FP8_TOKEN;
  constexpr float kTop = fmt_e4m3(FMT) ? 448.f : FMT == FMT_INT4_GROUP ? 7.f : 127.f;
  const PoolView& pool = p.pool;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ci = tid % LPH, r0 = tid / LPH, d0 = 8 * ci;
  const int bs = pool.bs;
  const int r = p.plan.rotary_dim, rp = r >> 1;
  const bool turn = kv == 0 && r > 0, norm = kv == 0 && p.k_weight != nullptr;

  if (tid < 2) sh.has[tid] = 0;
  if (kToken && tid < kMaxBlock) sh.tok[tid] = 0;
  __syncthreads();
  if (tid < n) {
    const int off = sh.off[w0 + tid];
    atomicOr(&sh.has[off >> 5], 1u << (off & 31));
  }
  if (turn) rope_table<kIngestThreads>(p.plan, p.positions + t0, n, cs);
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = norm ? p.k_weight[d0 + i] : 1.f;
  __syncthreads();
  const uint64_t has = (uint64_t)sh.has[1] << 32 | sh.has[0];
  const bool fresh = has & 1;
  // sub-tiles (8-token pages: the page) whose every token the run writes
  auto covered = [&](int off) {
    const uint64_t m = bs == 8 ? 0xFFull : 0xFFFFull;
    return (~has >> (off & ~15) & m) == 0;
  };

  float x[CPT][8];
  int off[CPT];
  auto load_head = [&](int h) {  // rows of head h, normed and rotated
    uint4 raw[CPT];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int row = c * RPP + r0;
      off[c] = row < n ? sh.off[w0 + row] : -1;
      raw[c] = row < n ? *reinterpret_cast<const uint4*>(static_cast<const __half*>(p.x[kv]) +
                                                         (t0 + row) * p.stride[kv] + h * D + d0)
                       : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      widen8(raw[c], p.bf16, x[c]);
      if (norm) norm8<D>(x[c], w, p.eps);
      if (turn)
        rotate8<D>(x[c], ci, r, p.plan.layout == KVQ_ROPE_INTERLEAVED,
                   cs + min(c * RPP + r0, n - 1) * rp);
    }
  };
  auto absmax = [&](const float (&v)[8]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
    return a;
  };

  if constexpr (kToken) {  // the scale of a token spans every head: a first pass over them
    for (int h = 0; h < pool.Hkv; ++h) {
      load_head(h);
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        float a = absmax(x[c]);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        if (ci == 0 && off[c] >= 0) atomicMax(&sh.tok[c * RPP + r0], __float_as_uint(a));
      }
    }
    __syncthreads();
    if (tid < n)
      pool.tok_scales[(blk * 2 + kv) * bs + sh.off[w0 + tid]] =
          __fdiv_rn(__uint_as_float(sh.tok[tid]), kTop);
  }

  for (int h = h0; h < h1; ++h) {
    char* page = pool.pages + (blk * pool.Hkv + h) * pool.page_bytes;
    char* codes = page + (kv == 0 ? 0 : pool.v_off);
    float* scales = reinterpret_cast<float*>(page + 2 * pool.code_bytes);
    load_head(h);
    float s_block = 0.f;
    if constexpr (kBlock) {
      float a = 0.f;
#pragma unroll
      for (int c = 0; c < CPT; ++c) a = fmaxf(a, absmax(x[c]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      const float s_old = fresh ? 0.f : scales[kv];
      if (lane == 0) sh.red[warp] = a;
      __syncthreads();  // (also: the previous head's tile has left)
      a = sh.red[0];
#pragma unroll
      for (int i = 1; i < kIngestWarps; ++i) a = fmaxf(a, sh.red[i]);
      s_block = fmaxf(s_old, __fdiv_rn(a, kTop));
      const float inv_block = quant_inverse(s_block);
      // the codes the block keeps
      const uint32_t zero = fmt_e4m3(FMT) ? 0u : 0x80808080u;
      for (int i = tid; i < pool.code_bytes / 4; i += kIngestThreads) {
        uint32_t v = fresh ? zero : reinterpret_cast<const uint32_t*>(codes)[i];
        if (!fresh && s_block > s_old) v = rescale_word<FMT>(v, s_old, s_block, inv_block);
        reinterpret_cast<uint32_t*>(tile)[i] = v;
      }
      if (tid == 0) scales[kv] = s_block;
    } else if constexpr (fmt_4bit(FMT)) {
      __syncthreads();
      for (int i = tid; i < pool.code_bytes / 4; i += kIngestThreads)
        reinterpret_cast<uint32_t*>(tile)[i] = 0;
    }
    __syncthreads();

#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const bool act = off[c] >= 0;
      const bool staged = kBlock || (act && covered(off[c]));
      char* dst = staged ? tile : codes;
      if constexpr (FMT == FMT_FP16) {
        if (!act) continue;
        const uint4 o = narrow8(x[c]);
        char* t = dst + (off[c] >> 4) * pool.sub_bytes;
        const int tt = off[c] & 15;
        if (kv == 0) {
          *reinterpret_cast<uint2*>(t + k_tile_offset(tt, d0, D, 2)) = make_uint2(o.x, o.y);
          *reinterpret_cast<uint2*>(t + k_tile_offset(tt, d0 + 4, D, 2)) = make_uint2(o.z, o.w);
        } else {
          const uint16_t* hb = reinterpret_cast<const uint16_t*>(&o);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint16_t*>(t + v_code_offset(tt, d0 + i, D, 2, bs)) = hb[i];
        }
        continue;
      }
      float s = 0.f;
      if constexpr (FMT == FMT_FP4) {
        float a = absmax(x[c]);
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
        const uint32_t sc4 = fp4_scale_code(a);
        s = fp4_scale_value(sc4);
        if (act && (d0 & 15) == 0) store_fp4_scale<D>(page, kv, off[c], d0 >> 4, pool, sc4);
      } else if constexpr (FMT == FMT_INT8_GROUP || FMT == FMT_INT4_GROUP) {
        // a group is group/8 consecutive lanes
        float a = absmax(x[c]);
        for (int o = pool.group >> 4; o > 0; o >>= 1)
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        s = __fdiv_rn(a, kTop);
        if (act && d0 % pool.group == 0)
          scales[(kv * bs + off[c]) * pool.ng + d0 / pool.group] = s;
      } else if constexpr (kToken) {
        s = act ? __fdiv_rn(__uint_as_float(sh.tok[c * RPP + r0]), kTop) : 0.f;
      } else if constexpr (kBlock) {
        s = s_block;
      }
      if (!act) continue;
      if constexpr (FMT == FMT_FP4) {
        char* t = dst + (off[c] >> 4) * pool.sub_bytes;
        const uint32_t q = quant8_fp4(x[c], s);
        if (staged)
          store_fp4x8<true>(t, kv, off[c] & 15, d0, q);
        else
          store_fp4x8<false>(t, kv, off[c] & 15, d0, q);
      } else if constexpr (FMT == FMT_INT4_GROUP) {
        char* t = dst + (off[c] >> 4) * pool.sub_bytes;
        const int tt = off[c] & 15;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          int sh4;
          const int o = kv == 0 ? k_nibble(tt, d0 + i, sh4) : v_nibble(tt, d0 + i, sh4);
          const uint32_t val = quant_i4(x[c][i], s) << sh4;
          if (staged)
            atomicOr(reinterpret_cast<uint32_t*>(t + o), val);
          else
            store_nibbles(t + o, 0xFu << sh4, val);
        }
      } else {
        uint8_t q[8];
        if constexpr (FMT == FMT_INT8_CHANNEL) {
          const float* chs = pool.chan_scales + ((int64_t)kv * pool.Hkv + h) * D + d0;
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = quant_byte<FMT>(x[c][i], chs[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = quant_byte<FMT>(x[c][i], s);
        }
        store_codes8(dst, kv, off[c], d0, D, bs, pool.sub_bytes, q);
      }
    }
    __syncthreads();
    for (int i = tid; i < pool.code_bytes / 16; i += kIngestThreads) {
      const int sub = i * 16 / pool.sub_bytes;
      if (kBlock || covered(16 * sub))
        reinterpret_cast<uint4*>(codes)[i] = reinterpret_cast<const uint4*>(tile)[i];
    }
    if constexpr (!kBlock) __syncthreads();
  }
  if constexpr (kBlock) __syncthreads();
}

// A whole block of tokens (t0 .. t0+bs-1 in the order of their slots).  A lane
// holds 8 channels of the four tokens that share V words (2j, 2j+1, 2j+8, 2j+9 of
// a sub-tile), so that both K words (4 channels of a token) and V words (those 4
// tokens of a channel) are complete in one lane and go straight to the page, a
// sector per 8 of them; only the one scale of a block passes through shared
// memory.  A warp's unit is 8 such tokens of one head of 128 channels (16 of one of
// 64): 32 values a lane.  (Whole sub-tiles, 64 values, left an SM 16 warps and the
// kernel waiting for its loads: 75 us for 16384 tokens x 8 heads.)
// 4-bit codes, whose words pack tokens t and t + 8, and the formats whose scale spans a
// token's heads are not built this way; they take every run through shared memory, the
// latter loading and rotating each row twice: 16384 tokens x 8 heads of 128 in 133 us
// and 112 to 120, where FP16 takes 36, e5m2 39, INT8 blocks 47, INT8 groups and e4m3
// blocks 60, per-channel 72.
template <int FMT>
constexpr bool whole_blocks() {
  return !fmt_4bit(FMT) && FMT != FMT_INT8_TOKEN && FMT != FMT_FP8_TOKEN;
}

template <int FMT, int D>
__device__ __forceinline__ void ingest_whole(const IngestParams& p, IngestShared& sh, float2* cs,
                                             int64_t t0, int64_t blk, int h0, int h1, int kv) {
  constexpr int LPH = D / 8, RG = 32 / LPH;
  constexpr int UPT = 4 / RG;  // units per sub-tile
  constexpr bool kBlock = fmt_block(FMT);
  constexpr float kTop = fmt_e4m3(FMT) ? 448.f : 127.f;
  const PoolView& pool = p.pool;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ci = lane % LPH, rg = lane / LPH;
  const int bs = pool.bs;
  // (powers of two: units of a head, warps per head, units per warp -- 1, or 2 for 64
  // tokens x 128 -- and heads at a time)
  const int units = (bs >> 4) * UPT;
  const int wl = units >= 4 ? 2 : units - 1, wph = 1 << wl;
  const int ul = units >> (wl + 1), upw = 1 << ul;
  const int hpi = kIngestWarps >> wl;
  const int r = p.plan.rotary_dim, rp = r >> 1;
  const bool turn = kv == 0 && r > 0, norm = kv == 0 && p.k_weight != nullptr;
  const bool inter = p.plan.layout == KVQ_ROPE_INTERLEAVED;
  // Half layout: a lane takes both channels of its pairs (as in rope_tokens),
  // unless scale groups are narrower than the head, whose lanes must adjoin.
  const bool split = turn && !inter && (FMT != FMT_INT8_GROUP || pool.ng == 1) && 8 * ci < r;
  const int da = split ? 4 * ci : 8 * ci, db = split ? 4 * ci + rp : 8 * ci + 4;
  // Rounds: a head's (or several heads') units, one per warp.  With several units per
  // warp the first rounds of a head only find the block's absmax.
  const int rl = kBlock && ul > 0 ? ul + 1 : ul, rounds = 1 << rl;
  const int total = ((h1 - h0 + hpi - 1) >> (2 - wl)) << rl;
  const int wu = (warp & (wph - 1)) << ul, wh = h0 + (warp >> wl);
  uint32_t next[4][4];  // rows of the round to come
  auto load = [&](int it) {
    const int u = wu + (it & (upw - 1)), h = wh + ((it >> rl) << (2 - wl));
    const int tok = 16 * (u / UPT) + 2 * (rg + RG * (u % UPT));  // chunk c: token tok + (c & 1) + 8 (c >> 1)
    const __half* src = static_cast<const __half*>(p.x[kv]) + (t0 + tok) * p.stride[kv] + h * D;
    const bool act = h < h1;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const __half* at = src + ((c & 1) + 8 * (c >> 1)) * p.stride[kv];
      if (!turn) {  // (channels da .. db+3 adjoin)
        const uint4 a = act ? *reinterpret_cast<const uint4*>(at + da) : make_uint4(0, 0, 0, 0);
        next[c][0] = a.x;
        next[c][1] = a.y;
        next[c][2] = a.z;
        next[c][3] = a.w;
      } else {
        const uint2 a = act ? *reinterpret_cast<const uint2*>(at + da) : make_uint2(0, 0);
        const uint2 b = act ? *reinterpret_cast<const uint2*>(at + db) : make_uint2(0, 0);
        next[c][0] = a.x;
        next[c][1] = a.y;
        next[c][2] = b.x;
        next[c][3] = b.y;
      }
    }
  };
  load(0);
  if (turn) rope_table<kIngestThreads>(p.plan, p.positions + t0, bs, cs);
  float w[8];
  if (norm)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = p.k_weight[da + i];
      w[4 + i] = p.k_weight[db + i];
    }
  // K words of token 2j + (c & 1) + 8 (c >> 1): 64 bytes further for c & 1, half a
  // sub-tile for c >> 1
  constexpr int ES = FMT == FMT_FP16 ? 2 : 1;
  const int ka = k_tile_offset(0, da, D, ES), kb = k_tile_offset(0, db, D, ES);
  __syncthreads();
  int it = 0;
  for (int hb = h0; hb < h1; hb += hpi) {
    const int h = hb + (warp >> wl);
    const bool act = h < h1;
    char* page = pool.pages + (blk * pool.Hkv + (act ? h : 0)) * pool.page_bytes;
    float* scales = reinterpret_cast<float*>(page + 2 * pool.code_bytes);
    float amax = 0.f, s = 0.f, inv = 0.f;
    for (int k = 0; k < rounds; ++k, ++it) {
      const bool last = k >= rounds - upw;
      const int u = wu + (k & (upw - 1));
      const int sub = u / UPT, j = rg + RG * (u % UPT);
      const int tok = 16 * sub + 2 * j;
      float x[4][8];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        widen8(make_uint4(next[c][0], next[c][1], next[c][2], next[c][3]), p.bf16, x[c]);
      if (it + 1 < total) load(it + 1);
      if (norm)
#pragma unroll
        for (int c = 0; c < 4; ++c) norm8<D>(x[c], w, p.eps);
      if (turn) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2* t = cs + (tok + (c & 1) + 8 * (c >> 1)) * rp;
          if (split) {
            const float4 c0 = *reinterpret_cast<const float4*>(t + 4 * ci);
            const float4 c1 = *reinterpret_cast<const float4*>(t + 4 * ci + 2);
            const float cv[4] = {c0.x, c0.z, c1.x, c1.z}, sv[4] = {c0.y, c0.w, c1.y, c1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[c][i], d = x[c][4 + i];
              x[c][i] = fmaf(a, cv[i], -d * sv[i]);
              x[c][4 + i] = fmaf(a, sv[i], d * cv[i]);
            }
          } else if (inter || (FMT == FMT_INT8_GROUP && pool.ng > 1)) {
            rotate8<D>(x[c], ci, r, inter, t);
          }
        }
      }
      if constexpr (kBlock) {
        if (k < upw) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[c][i]));
        }
        if (k == upw - 1) {  // every unit of the block seen: its warps agree on the scale
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          if (wph > 1) {  // (the two halves in turn: one barrier)
            float* red = sh.red + (hb - h0 & hpi) * (kIngestWarps / hpi);
            if (lane == 0) red[warp] = amax;
            __syncthreads();
            for (int i = 0; i < wph; ++i) amax = fmaxf(amax, red[(warp & ~(wph - 1)) + i]);
          }
          s = __fdiv_rn(amax, kTop);
          inv = quant_inverse(s);
          if (act && warp % wph == 0 && lane == 0) scales[kv] = s;
        }
      }
      if (!last || !act) continue;
      char* tile = page + (kv == 0 ? 0 : pool.v_off) + sub * pool.sub_bytes;
      if constexpr (FMT == FMT_FP16) {
        uint32_t o[4][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 v = narrow8(x[c]);
          o[c][0] = v.x;
          o[c][1] = v.y;
          o[c][2] = v.z;
          o[c][3] = v.w;
        }
        if (kv == 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            char* at = tile + (2 * j + (c & 1)) * 64 + (c >> 1) * (16 * D);
            *reinterpret_cast<uint2*>(at + ka) = make_uint2(o[c][0], o[c][1]);
            *reinterpret_cast<uint2*>(at + kb) = make_uint2(o[c][2], o[c][3]);
          }
        } else {
          char* at = tile + v_tile_offset(2 * j, da, D, 2);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t sel = i & 1 ? 0x7632u : 0x5410u;
            *reinterpret_cast<uint2*>(at + 64 * i) =
                make_uint2(prmt(o[0][i >> 1], o[1][i >> 1], sel), prmt(o[2][i >> 1], o[3][i >> 1], sel));
          }
        }
      } else {
        uint32_t k4[4][2];  // per token: channels da .. da+3 and db .. db+3
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if constexpr (FMT == FMT_INT8_GROUP) {
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[c][i]));
            for (int o = pool.group >> 4; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            s = __fdiv_rn(a, kTop);
            inv = quant_inverse(s);
            if (8 * ci % pool.group == 0)
              scales[(kv * bs + tok + (c & 1) + 8 * (c >> 1)) * pool.ng + 8 * ci / pool.group] = s;
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float y[4] = {x[c][4 * q], x[c][4 * q + 1], x[c][4 * q + 2], x[c][4 * q + 3]};
            if constexpr (FMT == FMT_INT8_CHANNEL) {
              const float* chs = pool.chan_scales + ((int64_t)kv * pool.Hkv + h) * D + (q ? db : da);
              uint32_t v = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) v |= (uint32_t)quant_i8(y[i], chs[i]) << (8 * i);
              k4[c][q] = v;
            } else {
              k4[c][q] = quant_word_fast<FMT>(y, s, inv);
            }
          }
        }
        if (kv == 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            char* at = tile + (2 * j + (c & 1)) * 64 + (c >> 1) * (8 * D);
            *reinterpret_cast<uint32_t*>(at + ka) = k4[c][0];
            *reinterpret_cast<uint32_t*>(at + kb) = k4[c][1];
          }
        } else {  // transpose 4 tokens x 4 channels, twice
          char* at = tile + v_tile_offset(2 * j, da, D, 1);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t a = prmt(k4[0][q], k4[1][q], 0x5140u), b = prmt(k4[2][q], k4[3][q], 0x5140u);
            const uint32_t c = prmt(k4[0][q], k4[1][q], 0x7362u), d = prmt(k4[2][q], k4[3][q], 0x7362u);
            *reinterpret_cast<uint32_t*>(at + 64 * (4 * q)) = prmt(a, b, 0x5410u);
            *reinterpret_cast<uint32_t*>(at + 64 * (4 * q + 1)) = prmt(a, b, 0x7632u);
            *reinterpret_cast<uint32_t*>(at + 64 * (4 * q + 2)) = prmt(c, d, 0x5410u);
            *reinterpret_cast<uint32_t*>(at + 64 * (4 * q + 3)) = prmt(c, d, 0x7632u);
          }
        }
      }
    }
  }
  __syncthreads();
}

// Resident CTAs to compile for: whole blocks need some 96 registers with the rows of
// the next round on their way, a run held in registers 8 more per chunk.  (16384
// tokens with their queries and the read-back, 16 tokens a CTA: 96.1 us; with four
// CTAs 96.6, with six 98.0, with six and no rows ahead 96.9.)
constexpr int ingest_ctas(int cpt) { return cpt <= 4 ? 5 : 3; }

template <int FMT, int D, int CPT>
__global__ void __launch_bounds__(kIngestThreads, ingest_ctas(CPT)) kvq_ingest_kernel(const __grid_constant__ IngestParams p) {
  extern __shared__ __align__(16) char smem[];
  // The decode-step form launches as a programmatic dependent: wait for what
  // ran before, then let the decode launch (see kvq_append_kernel).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x >= p.kv_ctas) {
    const int64_t b = blockIdx.x - p.kv_ctas;
    constexpr int rows = kIngestThreads / (D / 8);
    const int h = static_cast<int>(b % p.q_parts) * rows + threadIdx.x / (D / 8);
    auto turn = [&](auto bf, auto in) {
      rope_tokens<D, decltype(bf)::value, decltype(in)::value>(
          p.q, p.Hq, RopeRows{}, 0, p.positions, b / p.q_parts, 1, h, p.eps, p.plan,
          reinterpret_cast<float*>(smem));
    };
    using Y = std::true_type;
    using N = std::false_type;
    if (p.plan.layout == KVQ_ROPE_INTERLEAVED)
      p.bf16 ? turn(Y{}, Y{}) : turn(N{}, Y{});
    else
      p.bf16 ? turn(Y{}, N{}) : turn(N{}, N{});
    return;
  }
  __shared__ IngestShared sh;
  const PoolView& pool = p.pool;
  const int kv = static_cast<int>(blockIdx.x & 1);
  const int64_t b = blockIdx.x >> 1;
  const int h0 = static_cast<int>(b % p.hsplit) * p.hpc;
  const int64_t c0 = b / p.hsplit * p.tpc;
  // Window of tokens c0 .. c0+tpc+bs-1: the runs that begin among the first tpc
  // and, for the last of them, as far as a run can go.
  const int tid = threadIdx.x, lane = tid & 31;
  // one token per CTA: its row's first chunks come while its slot is looked up
  auto first_rows = [&](int64_t t) {
    return tid / (D / 8) < pool.Hkv ? *reinterpret_cast<const uint4*>(static_cast<const __half*>(p.x[kv]) +
                                                                      t * p.stride[kv] + tid * 8)
                                    : make_uint4(0, 0, 0, 0);
  };
  const uint4 row0 = p.tpc == 1 && h0 == 0 ? first_rows(c0) : make_uint4(0, 0, 0, 0);
  const int win = static_cast<int>(min((int64_t)p.tpc + pool.bs, p.T - c0));
  for (int i = tid; i <= win; i += kIngestThreads) {
    const int64_t t = c0 + i - 1;
    int blk = -1;
    if (t >= 0) {
      const int64_t slot = ingest_slot(p, t);
      if (slot >= pool.num_blocks * pool.bs) {
        if (i > 0 && i <= p.tpc && h0 == 0) set_error(pool.err, ERR_RANGE);
      } else if (slot >= 0) {
        blk = static_cast<int>(slot >> p.bs_log2);
        if (i > 0) sh.off[i - 1] = static_cast<uint8_t>(slot & (pool.bs - 1));
      }
    }
    sh.blk[i] = blk;
  }
  __syncthreads();
  {
    // the step form's tokens are of different sequences: each is a run
    const bool cut = tid >= win || sh.blk[tid] != sh.blk[tid + 1] || p.slots == nullptr;
    const uint32_t m = __ballot_sync(0xffffffffu, cut);
    if (lane == 0) sh.cut[tid >> 5] = m;
  }
  __syncthreads();
  char* tile = smem;
  float2* cs = reinterpret_cast<float2*>(smem + pool.code_bytes);
  const int h1 = min(h0 + p.hpc, pool.Hkv);
  const int nown = min(p.tpc, win);
  const uint64_t cuts[2] = {(uint64_t)sh.cut[1] << 32 | sh.cut[0], (uint64_t)sh.cut[3] << 32 | sh.cut[2]};
  auto next_cut = [&](int i) {  // the first cut at or behind token i of the window
    const uint64_t a = i < 64 ? cuts[0] >> i : 0, b = i < 64 ? cuts[1] : i < 128 ? cuts[1] >> (i - 64) : 0;
    return a != 0 ? i + __ffsll(a) - 1 : b != 0 ? max(i, 64) + __ffsll(b) - 1 : 128;
  };
  // (what lies before the first cut belongs to a run of an earlier CTA; what a run
  // has beyond a block's tokens, slots given twice, is dropped)
  for (int i = next_cut(0); i < nown; i = next_cut(i)) {
    const int e = min(next_cut(i + 1), i + pool.bs);  // (every place behind the window is a cut)
    const int blk = sh.blk[i + 1];
    if (e - i == 1) {  // one token: the CTA of the first heads takes all of them
      if (blk >= 0 && h0 == 0)
        ingest_token<FMT, D>(p, sh, cs, c0 + i, sh.off[i], blk, kv, p.tpc == 1 ? row0 : first_rows(c0 + i));
      i = e;
      continue;
    }
    if constexpr (whole_blocks<FMT>()) {
      if (blk >= 0 && e - i == pool.bs && pool.bs >= 16 &&
          __syncthreads_and(tid >= pool.bs || sh.off[i + min(tid, pool.bs - 1)] == tid)) {
        ingest_whole<FMT, D>(p, sh, cs, c0 + i, blk, h0, h1, kv);
        i = e;
        continue;
      }
    }
    if (blk >= 0)
      ingest_run<FMT, D, CPT>(p, sh, tile, cs, c0 + i, e - i, i, blk, h0, h1, kv);
    i = e;
  }
}

// Shared memory of a launch: the tile image and the run's cosines and sines (the
// query CTAs' own, if that is more).
inline int ingest_smem(const PoolView& pool, int rotary_dim) {
  const int kv = pool.code_bytes + pool.bs * rotary_dim / 2 * 8;
  const int q = rope_smem(rotary_dim);
  return kv > q ? kv : q;
}

struct IngestLaunch {
  IngestParams p;
  unsigned grid;
  int smem;
  cudaStream_t st;
  bool dependent;
};

template <int FMT, int D, int CPT>
cudaError_t run_ingest_c(const IngestLaunch& l) {
  constexpr int own = sizeof(IngestShared);  // (FP16 blocks of 64 x 128, wholly rotated: 48 KB beside it)
  if (l.smem + own > 48 * 1024) {
    const cudaError_t e = allow_big_smem<kvq_ingest_kernel<FMT, D, CPT>, own>();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(l.grid);
  cfg.blockDim = dim3(kIngestThreads);
  cfg.dynamicSmemBytes = l.smem;
  cfg.stream = l.st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = l.dependent ? 1 : 0;
  return phase_mark(l.st, cudaLaunchKernelEx(&cfg, kvq_ingest_kernel<FMT, D, CPT>, l.p));
}

// CPT: 16-byte chunks of a whole block's rows of one head per thread.
template <int FMT>
cudaError_t run_ingest(const IngestLaunch& l) {
  const int chunks = l.p.pool.bs * l.p.pool.D / 8;
  if (l.p.pool.D == 64) {
    if (chunks <= kIngestThreads) return run_ingest_c<FMT, 64, 1>(l);
    if (chunks <= 2 * kIngestThreads) return run_ingest_c<FMT, 64, 2>(l);
    return run_ingest_c<FMT, 64, 4>(l);
  }
  if (chunks <= 2 * kIngestThreads) return run_ingest_c<FMT, 128, 2>(l);
  if (chunks <= 4 * kIngestThreads) return run_ingest_c<FMT, 128, 4>(l);
  return run_ingest_c<FMT, 128, 8>(l);
}

cudaError_t launch_ingest_block(const IngestLaunch& l);
cudaError_t launch_ingest_group(const IngestLaunch& l);
cudaError_t launch_ingest_token(const IngestLaunch& l);
cudaError_t launch_ingest_misc(const IngestLaunch& l);

}  // namespace kvq
