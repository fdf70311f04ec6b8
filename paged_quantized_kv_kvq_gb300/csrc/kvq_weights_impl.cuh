// kvq_weights_impl.cuh -- attention weights of every cached token, summed over
// the Q heads of its kv head and accumulated over steps:
//
//   scores[s][h][t] = decay * prev[s][h][t] + sum_{q in group h} exp(z_q,t - lse_q)
//
// with z_q,t = q . k^_t * sm_scale over the quantized cache and lse_q the
// log-sum-exp that the decode of the same rows handed out.  With the
// denominators known no token depends on another, so one pass over K does it:
// no running maximum, no split to join, no workspace.
//
// Bound: HBM -- the K half of the pages once (half of a decode's bytes) and
// 8 bytes of scores per (token, kv head).  A warp walks a stretch of tokens of one
// (sequence, kv head), 4 KB of K words a step, straight into the registers that
// are its tensor-core fragments (pages are stored in that order); nothing passes
// through shared memory.  The next step's words are loaded before this step's
// products, so that 16 warps keep 64 KB an SM in flight throughout; one step per
// warp, without that overlap, left the loads of 10 warps waiting behind three
// round trips (lengths, table, pages): 110 us for 8 x 32768 tokens of INT8 blocks.
// The Q heads sit on the n dimension of mma.m16n8k16 as in the decode; groups of
// more than 8 heads take their products 8 at a time.
#pragma once
#include "kvq_decode_impl.cuh"
#include "kvq_internal.h"

namespace kvq {

constexpr int kWeightsWarps = 4;

// 16-token sub-tiles per step: 4 KB of codes (INT4: 2 KB).
template <int FMT, int D>
constexpr int weights_tiles() {
  return 256 / D / (FMT == FMT_FP16 ? 2 : 1);
}
// Resident CTAs to compile for: two steps' words and a head tile's fragments fit
// 128 registers; per-channel scales keep a second set of fragments, INT4 twice the
// sub-tiles' sums, narrow groups a scale each per token.
template <int FMT, int NG>
constexpr int weights_ctas() {
  return NG > 2 ? 2 : FMT == FMT_INT8_CHANNEL || FMT == FMT_INT4_GROUP || NG > 1 ? 3 : 4;
}

struct WeightsParams {
  DecodeParams d;  // q, table, lens and sizes as the decode has them
  const float* lse;
  const float* prev;
  float* scores;
  int64_t stride;
  float decay;
  int per;     // tokens per warp (a multiple of a step's)
  int nchunk;  // CTAs per (sequence, kv head)
};

template <int FMT, int D, int NG>
__global__ void __launch_bounds__(kWeightsWarps * 32, weights_ctas<FMT, NG>())
    kvq_weights_kernel(const __grid_constant__ WeightsParams p) {
  using T = FmtTraits<FMT>;
  constexpr int KS = D / 16, KPG = KS / NG, SUB = KPG >= 2 ? 2 : 1;
  constexpr int NU32 = lane_words<FMT, D>(), NC = NU32 / 4;  // 32-bit words, 16-byte chunks per lane
  constexpr int TL = weights_tiles<FMT, D>();
  constexpr int NS = T::group_scales ? NG : 1;
  const float kInf = __int_as_float(0x7f800000u);
  const PoolView& pool = p.d.pool;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, j = lane & 3;
  const int sh = blockIdx.x / p.nchunk, s = sh / pool.Hkv, h = sh - s * pool.Hkv;
  const int t0 = ((blockIdx.x - sh * p.nchunk) * kWeightsWarps + warp) * p.per;
  int L = p.d.lens[s];
  if (L > p.d.max_ctx) {
    if (t0 == 0 && h == 0 && lane == 0) set_error(pool.err, ERR_RANGE);
    L = p.d.max_ctx;
  }
  if (t0 >= L) return;
  const int bs = pool.bs, bl = 31 - __clz(bs), end = min(L, t0 + p.per);
  const int64_t row = ((int64_t)s * pool.Hkv + h) * p.stride;

  // Block-table entries of the stretch, one per lane, 32 at a time; an entry
  // outside the pool is flagged once and skipped.
  const int* trow = p.d.table + (int64_t)s * p.d.max_blocks;
  const int n0 = t0 >> bl, n1 = (end - 1) >> bl;
  int held = n0, entry = 0;
  auto hold = [&](int n) {  // entries n .. n+31
    held = n;
    entry = n + lane <= n1 ? trow[n + lane] : 0;
    if (entry < 0 || (int64_t)entry >= pool.num_blocks) {
      entry = -1;
      if (h == 0) set_error(pool.err, ERR_RANGE);
    }
  };
  hold(n0);

  // One step's loads.  ok: bit 2x + b, half b (tokens 8b .. 8b+7) of sub-tile x is there.
  struct Step {
    uint32_t kw[TL][NU32];
    float ks[TL][2][NS];
    float before[TL];
    uint32_t ok;
  };
  auto fetch = [&](int t, Step& S) {
    if (((t + 16 * TL - 1) >> bl) - held >= 32) hold(t >> bl);
    S.ok = 0;
#pragma unroll
    for (int x = 0; x < TL; ++x) {
      const char* page[2];
      int off[2], phys[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int tt = t + 16 * x + 8 * b;
        phys[b] = __shfl_sync(0xffffffffu, entry, (tt >> bl) - held);
        off[b] = tt & (bs - 1);
        page[b] = nullptr;
        if (tt < end && phys[b] >= 0) {
          page[b] = pool.pages + ((int64_t)phys[b] * pool.Hkv + h) * pool.page_bytes;
          S.ok |= 1u << (2 * x + b);
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        // chunks of the first half hold tokens 0..7, of the second 8..15
        // (INT4 words hold both; 8-token pages hold a half each)
        constexpr bool kBoth = FMT == FMT_INT4_GROUP;
        const int b = !kBoth && c >= NC / 2 ? 1 : 0;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (page[b] != nullptr) {
          const int chunk = bs == 8 && b ? c - NC / 2 : c;
          v = __ldg(reinterpret_cast<const uint4*>(page[b] + (off[b] >> 4) * pool.sub_bytes +
                                                   chunk * 512 + lane * 16));
        }
        S.kw[x][4 * c] = v.x;
        S.kw[x][4 * c + 1] = v.y;
        S.kw[x][4 * c + 2] = v.z;
        S.kw[x][4 * c + 3] = v.w;
      }
      if constexpr (T::row_scales) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int gi = 0; gi < NS; ++gi) {
            float v = 0.f;
            if (page[b] != nullptr) {
              const float* sc = reinterpret_cast<const float*>(page[b] + 2 * pool.code_bytes);
              if constexpr (T::block_scales) {
                v = sc[0];
              } else if constexpr (T::group_scales) {
                v = sc[(off[b] + g) * NS + gi];
              } else {
                v = pool.tok_scales[(int64_t)phys[b] * 2 * bs + off[b] + g];
              }
            }
            S.ks[x][b][gi] = v;
          }
      }
      // the accumulated weight so far of the token this lane writes
      const int tw = t + 16 * x + 8 * (j & 1) + g;
      S.before[x] = p.prev != nullptr && j < 2 && tw < end ? p.prev[row + tw] : 0.f;
    }
  };

  uint32_t qb[KS][2];
  uint32_t ql[T::channel ? KS : 1][2];
  float csc, lse2[2];
  auto load_heads = [&](int ht) {
    load_q<FMT, D>(p.d, s, h, ht, lane, qb, ql, csc);
    // heads 2j, 2j+1 of the tile; one that is not there, or attends nothing, weighs 0
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int hq = 8 * ht + 2 * j + c;
      const float v = hq < p.d.G ? p.lse[(int64_t)s * p.d.Hq + h * p.d.G + hq] : -kInf;
      lse2[c] = v == -kInf ? kInf : v * 1.4426950408889634f;
    }
  };

  Step cur, nxt;
  fetch(t0, cur);
  if (p.d.n_ht == 1) load_heads(0);
  for (int t = t0; t < end; t += 16 * TL) {
    if (t + 16 * TL < end) fetch(t + 16 * TL, nxt);
    float w[TL][2];
#pragma unroll
    for (int x = 0; x < TL; ++x) w[x][0] = w[x][1] = 0.f;
    for (int ht = 0; ht < p.d.n_ht; ++ht) {
      if (p.d.n_ht > 1) load_heads(ht);
#pragma unroll
      for (int x = 0; x < TL; ++x) {
        float acc[NG * SUB][4];
#pragma unroll
        for (int a = 0; a < NG * SUB; ++a) acc[a][0] = acc[a][1] = acc[a][2] = acc[a][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          const int ai = (kk / KPG) * SUB + (SUB == 2 ? (kk & 1) : 0);
          uint32_t a0, a1, a2, a3;
          k_frag<FMT, D>(cur.kw[x], kk, a0, a1, a2, a3);
          mma_16816(acc[ai], a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
          if constexpr (T::channel) mma_16816(acc[ai], a0, a1, a2, a3, ql[kk][0], ql[kk][1]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {  // tokens g and g + 8
          float z0 = -lse2[0], z1 = -lse2[1];
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) {
            const float a = SUB == 2 ? acc[gi * SUB][2 * r] + acc[gi * SUB + 1][2 * r] : acc[gi][2 * r];
            const float b = SUB == 2 ? acc[gi * SUB][2 * r + 1] + acc[gi * SUB + 1][2 * r + 1] : acc[gi][2 * r + 1];
            const float sc = T::row_scales ? csc * cur.ks[x][r][T::group_scales ? gi : 0] : csc;
            z0 = fmaf(a, sc, z0);
            z1 = fmaf(b, sc, z1);
          }
          w[x][r] += (lse2[0] == kInf ? 0.f : fast_exp2(z0)) + (lse2[1] == kInf ? 0.f : fast_exp2(z1));
        }
      }
    }
#pragma unroll
    for (int x = 0; x < TL; ++x) {
      // the sum over the lanes' heads; lane j = 0 takes token g, j = 1 token g + 8
      const float give = j & 1 ? w[x][0] : w[x][1];
      float mine = (j & 1 ? w[x][1] : w[x][0]) + __shfl_xor_sync(0xffffffffu, give, 1);
      mine += __shfl_xor_sync(0xffffffffu, mine, 2);
      const int tw = t + 16 * x + 8 * (j & 1) + g;
      if (j < 2 && tw < end && (cur.ok >> (2 * x + j) & 1))
        p.scores[row + tw] = fmaf(p.decay, cur.before[x], mine);
    }
    cur = nxt;
  }
}

struct WeightsLaunch {
  WeightsParams p;
  cudaStream_t st;
};

template <int FMT, int D, int NG>
cudaError_t run_weights(const WeightsLaunch& l) {
  WeightsParams p = l.p;
  // Tokens per warp: whole steps, as many as leave every SM four times the warps
  // it holds (a warp's first loads wait; the ragged ends of sequences idle), 512
  // at most.
  constexpr int step = 16 * weights_tiles<FMT, D>();
  const int64_t tokens = (int64_t)p.d.max_ctx * p.d.S * p.d.pool.Hkv;
  const int64_t want = tokens / (152 * 16 * 4) / step * step;
  p.per = static_cast<int>(want < step ? step : want > 512 ? 512 : want);
  p.nchunk = static_cast<int>((p.d.max_ctx + (int64_t)kWeightsWarps * p.per - 1) / (kWeightsWarps * p.per));
  const int64_t grid = (int64_t)p.nchunk * p.d.S * p.d.pool.Hkv;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  kvq_weights_kernel<FMT, D, NG><<<static_cast<unsigned>(grid), kWeightsWarps * 32, 0, l.st>>>(p);
  return phase_mark(l.st, cudaGetLastError());
}

template <int FMT>
cudaError_t run_weights_d(const WeightsLaunch& l) {
  return l.p.d.pool.D == 64 ? run_weights<FMT, 64, 1>(l) : run_weights<FMT, 128, 1>(l);
}

template <int FMT>
cudaError_t run_weights_group(const WeightsLaunch& l) {
  const int D = l.p.d.pool.D, ng = l.p.d.pool.ng;
  switch (D * 16 + ng) {
    case 64 * 16 + 1: return run_weights<FMT, 64, 1>(l);
    case 64 * 16 + 2: return run_weights<FMT, 64, 2>(l);
    case 64 * 16 + 4: return run_weights<FMT, 64, 4>(l);
    case 128 * 16 + 1: return run_weights<FMT, 128, 1>(l);
    case 128 * 16 + 2: return run_weights<FMT, 128, 2>(l);
    case 128 * 16 + 4: return run_weights<FMT, 128, 4>(l);
    case 128 * 16 + 8: return run_weights<FMT, 128, 8>(l);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_weights_int8(const WeightsLaunch& l);
cudaError_t launch_weights_int4(const WeightsLaunch& l);

}  // namespace kvq
