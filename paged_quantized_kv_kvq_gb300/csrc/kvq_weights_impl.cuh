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
// 8 bytes of scores per (token, kv head).  A warp takes one stretch of tokens
// of one (sequence, kv head) and loads all of its K words before the first
// product, straight into the registers that are its tensor-core fragments
// (pages are stored in that order); nothing passes through shared memory.  The
// Q heads sit on the n dimension of mma.m16n8k16 as in the decode; groups of
// more than 8 heads read the stretch again per 8, from L1.
#pragma once
#include "kvq_decode_impl.cuh"
#include "kvq_internal.h"

namespace kvq {

constexpr int kWeightsWarps = 4;

// 16-token sub-tiles per warp: 64 tokens, 32 for fp16 codes (their words would
// take 128 registers).
template <int FMT>
constexpr int weights_tiles() {
  return FMT == FMT_FP16 ? 2 : 4;
}

struct WeightsParams {
  DecodeParams d;  // q, table, lens and sizes as the decode has them
  const float* lse;
  const float* prev;
  float* scores;
  int64_t stride;
  float decay;
  int nchunk;  // CTAs per (sequence, kv head)
};

template <int FMT, int D, int NG>
__global__ void __launch_bounds__(kWeightsWarps * 32) kvq_weights_kernel(const __grid_constant__ WeightsParams p) {
  using T = FmtTraits<FMT>;
  constexpr int KS = D / 16, KPG = KS / NG, SUB = KPG >= 2 ? 2 : 1;
  constexpr int NU32 = lane_words<FMT, D>(), NC = NU32 / 4;  // 32-bit words, 16-byte chunks per lane
  constexpr int TL = weights_tiles<FMT>();
  constexpr int NS = T::group_scales ? NG : 1;
  const PoolView& pool = p.d.pool;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, j = lane & 3;
  const int sh = blockIdx.x / p.nchunk, s = sh / pool.Hkv, h = sh - s * pool.Hkv;
  const int t0 = ((blockIdx.x - sh * p.nchunk) * kWeightsWarps + warp) * 16 * TL;
  int L = p.d.lens[s];
  if (L > p.d.max_ctx) {
    if (t0 == 0 && h == 0 && lane == 0) set_error(pool.err, ERR_RANGE);
    L = p.d.max_ctx;
  }
  if (t0 >= L) return;
  const int bs = pool.bs;
  const int* trow = p.d.table + (int64_t)s * p.d.max_blocks;

  // page of the 8 tokens from t, and their offset in it; null when the block
  // lies outside the pool (its tokens are skipped) or t behind the sequence
  const char* page[2 * TL];
  int off[2 * TL];
#pragma unroll
  for (int i = 0; i < 2 * TL; ++i) {
    const int t = t0 + 8 * i;
    page[i] = nullptr;
    off[i] = t & (bs - 1);
    if (t < L) {
      const int phys = trow[t / bs];
      if (phys >= 0 && (int64_t)phys < pool.num_blocks)
        page[i] = pool.pages + ((int64_t)phys * pool.Hkv + h) * pool.page_bytes;
      else if (lane == 0)
        set_error(pool.err, ERR_RANGE);
    }
  }
  uint32_t kw[TL][NU32];
  auto load_k = [&]() {
#pragma unroll
    for (int x = 0; x < TL; ++x)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        // chunks of the first half hold tokens 0..7, of the second 8..15
        // (INT4 words hold both; 8-token pages hold a half each)
        const bool b = FMT != FMT_INT4_GROUP && c >= NC / 2;
        const char* pg = page[2 * x + b];
        uint4 v = make_uint4(0, 0, 0, 0);
        if (pg != nullptr) {
          const int chunk = bs == 8 && b ? c - NC / 2 : c;
          v = __ldg(reinterpret_cast<const uint4*>(pg + (off[2 * x + b] >> 4) * pool.sub_bytes +
                                                   chunk * 512 + lane * 16));
        }
        kw[x][4 * c] = v.x;
        kw[x][4 * c + 1] = v.y;
        kw[x][4 * c + 2] = v.z;
        kw[x][4 * c + 3] = v.w;
      }
  };
  load_k();
  float ks[TL][2][NS];
  if constexpr (T::row_scales) {
#pragma unroll
    for (int i = 0; i < 2 * TL; ++i)
#pragma unroll
      for (int gi = 0; gi < NS; ++gi) {
        float v = 0.f;
        if (page[i] != nullptr) {
          const float* sc = reinterpret_cast<const float*>(page[i] + 2 * pool.code_bytes);
          if constexpr (T::block_scales) {
            v = sc[0];
          } else if constexpr (T::group_scales) {
            v = sc[(off[i] + g) * NS + gi];
          } else {
            const int64_t blk = (page[i] - pool.pages) / ((int64_t)pool.Hkv * pool.page_bytes);
            v = pool.tok_scales[blk * 2 * bs + off[i] + g];
          }
        }
        ks[i >> 1][i & 1][gi] = v;
      }
  }
  // the accumulated weights so far, of the token this lane writes
  const int64_t row = ((int64_t)s * pool.Hkv + h) * p.stride;
  float before[TL];
#pragma unroll
  for (int x = 0; x < TL; ++x) {
    const int t = t0 + 16 * x + 8 * (j & 1) + g;
    before[x] = p.prev != nullptr && j < 2 && t < L ? p.prev[row + t] : 0.f;
  }

  float w[TL][2];
#pragma unroll
  for (int x = 0; x < TL; ++x) w[x][0] = w[x][1] = 0.f;
  for (int ht = 0; ht < p.d.n_ht; ++ht) {
    if (ht > 0) load_k();
    uint32_t qb[KS][2];
    uint32_t ql[T::channel ? KS : 1][2];
    float csc;
    load_q<FMT, D>(p.d, s, h, ht, lane, qb, ql, csc);
    // heads 2j, 2j+1 of the tile; one that is not there, or attends nothing, weighs 0
    float lse2[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int hq = 8 * ht + 2 * j + c;
      const float v = hq < p.d.G ? p.lse[(int64_t)s * p.d.Hq + h * p.d.G + hq] : __int_as_float(0xff800000u);
      lse2[c] = v == __int_as_float(0xff800000u) ? __int_as_float(0x7f800000u) : v * 1.4426950408889634f;
    }
#pragma unroll
    for (int x = 0; x < TL; ++x) {
      float acc[NG * SUB][4];
#pragma unroll
      for (int a = 0; a < NG * SUB; ++a) acc[a][0] = acc[a][1] = acc[a][2] = acc[a][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        const int ai = (kk / KPG) * SUB + (SUB == 2 ? (kk & 1) : 0);
        uint32_t a0, a1, a2, a3;
        k_frag<FMT, D>(kw[x], kk, a0, a1, a2, a3);
        mma_16816(acc[ai], a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
        if constexpr (T::channel) mma_16816(acc[ai], a0, a1, a2, a3, ql[kk][0], ql[kk][1]);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {  // tokens g and g + 8
        float z0 = 0.f, z1 = 0.f;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          const float a = SUB == 2 ? acc[gi * SUB][2 * r] + acc[gi * SUB + 1][2 * r] : acc[gi][2 * r];
          const float b = SUB == 2 ? acc[gi * SUB][2 * r + 1] + acc[gi * SUB + 1][2 * r + 1] : acc[gi][2 * r + 1];
          const float sc = T::row_scales ? csc * ks[x][r][T::group_scales ? gi : 0] : csc;
          z0 = fmaf(a, sc, z0);
          z1 = fmaf(b, sc, z1);
        }
        w[x][r] += fast_exp2(z0 - lse2[0]) + fast_exp2(z1 - lse2[1]);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < TL; ++x) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      w[x][r] += __shfl_xor_sync(0xffffffffu, w[x][r], 1);
      w[x][r] += __shfl_xor_sync(0xffffffffu, w[x][r], 2);
    }
    // lanes j = 0 write token g, lanes j = 1 token g + 8
    const int t = t0 + 16 * x + 8 * (j & 1) + g;
    if (j < 2 && t < L && page[2 * x + 1] != nullptr && j == 1)
      p.scores[row + t] = fmaf(p.decay, before[x], w[x][1]);
    else if (j == 0 && t < L && page[2 * x] != nullptr)
      p.scores[row + t] = fmaf(p.decay, before[x], w[x][0]);
  }
}

struct WeightsLaunch {
  WeightsParams p;
  cudaStream_t st;
};

template <int FMT, int D, int NG>
cudaError_t run_weights(const WeightsLaunch& l) {
  WeightsParams p = l.p;
  constexpr int per = kWeightsWarps * 16 * weights_tiles<FMT>();
  p.nchunk = (p.d.max_ctx + per - 1) / per;
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
