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
// 8 bytes of scores per (token, kv head) -- and close behind it the conversion of
// the codes: a 16-token sub-tile of 128 channels is 2 KB and some 240 warp
// instructions (counted over 8 x 32768 tokens x 8 heads), 64 of them to make fp16
// fragments and 8 products; the rest looks after pages, stages and partial sums.
// The grid is persistent and balanced like the decode's: the stages (32 tokens or
// a page) of all (sequence, kv head) rows form one index space that the warps cut
// into equal contiguous ranges, so no warp idles behind a short sequence and the
// start of a stream (lengths, table, first pages: three round trips) is paid once
// a warp, not once a stretch.  Pages come by bulk copies into stages of the warp's
// own, some 200 KB in flight an SM, and are read back as the tensor-core fragments
// they are stored as, two sub-tiles side by side.
// Measured: 8 x 32768 tokens of INT8 blocks in 65 us (285 MB, 0.66 of the copy
// rate; its page stream without the arithmetic takes 62), 64 x ~1050 tokens of INT8
// groups in 22 us.  Stretches of 256 tokens per warp took 67 and 24 us with the
// next 4 KB held in registers, 67 and 27 with stages; pages aligned to 64 or 128
// bytes, waits that suspend, or the heads of a block side by side changed nothing
// or lost; a fourth CTA per SM spills, and two wait for their arithmetic.
// The Q heads sit on the n dimension of mma.m16n8k16 as in the decode; groups of
// more than 8 heads take their products 8 at a time.
#pragma once
#include "kvq_decode_impl.cuh"
#include "kvq_internal.h"

namespace kvq {

constexpr int kWeightsWarps = 4;
constexpr int kWeightsCtas = 3;    // resident per SM
constexpr int kWeightsStages = 8;  // per warp at most
constexpr int kWeightsStagePages = 4;  // of 8 tokens; fewer of larger ones

struct WeightsParams {
  DecodeParams d;  // q, table, lens and sizes as the decode has them
  const float* lse;
  const float* prev;
  float* scores;
  int64_t stride;
  float decay;
  int scale_bytes;  // K scales of a page copied behind its codes (per token, per group)
  int slot_bytes;   // room of a page in a stage
  int nstage;
};

// What the consumer of a stage has to know of its pages.
struct StageInfo {
  float scale[kWeightsStagePages];  // K scale (one scale per block)
  int there;                        // bit k: page k is in the pool
  int pad[3];
};

template <int FMT, int D, int NG>
__global__ void __launch_bounds__(kWeightsWarps * 32, kWeightsCtas)
    kvq_weights_kernel(const __grid_constant__ WeightsParams p) {
  using T = FmtTraits<FMT>;
  constexpr int KS = D / 16, KPG = KS / NG;
  constexpr int NU32 = lane_words<FMT, D>(), NC = NU32 / 4;  // 32-bit words, 16-byte chunks per lane
  constexpr int NS = T::group_scales ? NG : 1;
  constexpr bool kCopied = T::group_scales || T::token_scales;  // scales come with the codes
  const float kInf = __int_as_float(0x7f800000u);
  extern __shared__ __align__(128) char smem[];
  const PoolView& pool = p.d.pool;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, j = lane & 3;
  const int bs = pool.bs, bl = 31 - __clz(bs), nstage = p.nstage;
  const int sps = bs < 32 ? 32 / bs : 1;  // pages per stage
  const int span = bs * sps;              // tokens per stage
  const int stage_bytes = sps * p.slot_bytes;

  char* at = smem;
  char* stages = at + warp * nstage * stage_bytes;
  at += kWeightsWarps * nstage * stage_bytes;
  float* part = reinterpret_cast<float*>(at) + warp * 128;  // partial sums of 32 tokens x 4 lanes j
  at += kWeightsWarps * 512;
  StageInfo* info = reinterpret_cast<StageInfo*>(at) + warp * nstage;
  at += kWeightsWarps * nstage * sizeof(StageInfo);
  uint64_t* bars = reinterpret_cast<uint64_t*>(at) + warp * nstage;
  at += kWeightsWarps * nstage * 8;
  int* wtot = reinterpret_cast<int*>(at);
  int* PS = wtot + kWeightsWarps;  // [S + 1] stages before each sequence

  // ---- stages per sequence and their prefix (every CTA computes the same)
  {
    int carry = 0;
    for (int base = 0; base < p.d.S; base += kWeightsWarps * 32) {
      const int s = base + threadIdx.x;
      int v = 0;
      if (s < p.d.S) {
        int L = p.d.lens[s];
        if (L > p.d.max_ctx) {
          if (blockIdx.x == 0) set_error(pool.err, ERR_RANGE);
          L = p.d.max_ctx;
        }
        v = L > 0 ? (L + span - 1) / span * pool.Hkv : 0;
      }
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) wtot[warp] = x;
      __syncthreads();
      int before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kWeightsWarps; ++w) {
        before += w < warp ? wtot[w] : 0;
        all += wtot[w];
      }
      if (s < p.d.S) PS[s + 1] = carry + before + x;
      carry += all;
      __syncthreads();
    }
    if (threadIdx.x == 0) PS[0] = 0;
    __syncthreads();
  }
  const int Ttot = PS[p.d.S], nwarps = gridDim.x * kWeightsWarps;
  const int spw = (Ttot + nwarps - 1) / nwarps;  // stages per warp
  const int a0 = static_cast<int>(min((int64_t)(blockIdx.x * kWeightsWarps + warp) * spw, (int64_t)Ttot));
  const int n_w = min(spw, Ttot - a0);
  if (n_w <= 0) return;

  struct Cursor {
    int s, h, i, Ps;  // sequence, kv head, stage of the row, stages of the row
  };
  auto locate = [&](int x) {
    int lo = 0, hi = p.d.S;  // PS[lo] <= x < PS[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (PS[mid] <= x) lo = mid; else hi = mid;
    }
    Cursor c;
    c.s = lo;
    c.Ps = (PS[lo + 1] - PS[lo]) / pool.Hkv;
    const int r = x - PS[lo];
    c.h = r / c.Ps;
    c.i = r - c.h * c.Ps;
    return c;
  };
  auto advance = [&](Cursor& c) {  // true: another row
    if (++c.i < c.Ps) return false;
    c.i = 0;
    if (++c.h < pool.Hkv) return true;
    c.h = 0;
    do { ++c.s; } while (c.s < p.d.S && PS[c.s + 1] == PS[c.s]);
    c.Ps = c.s < p.d.S ? (PS[c.s + 1] - PS[c.s]) / pool.Hkv : 1;
    return true;
  };

  // ---- pages on their way.  A lane looks after one page of each batch of 32: its
  // table entry (negative: outside the pool, or behind the sequence), looked up a
  // batch ahead, and its scale, which needs the entry, half a batch ahead.
  struct Page {
    int entry, h;
    float scale;
  };
  const int batch = 32 / sps;  // stages of a batch
  auto look_up = [&](int n0) {  // the batch of stages n0 .. n0+batch-1 of this warp's range
    Page q{-1, 0, 0.f};
    const int n = n0 + lane / sps;
    if (n < n_w) {
      const Cursor c = locate(a0 + n);
      const int pg = c.i * sps + lane % sps;
      q.h = c.h;
      if (pg << bl < min(p.d.lens[c.s], p.d.max_ctx)) {
        q.entry = p.d.table[(int64_t)c.s * p.d.max_blocks + pg];
        if (q.entry < 0 || (int64_t)q.entry >= pool.num_blocks) {
          q.entry = -1;
          set_error(pool.err, ERR_RANGE);
        }
      }
    }
    return q;
  };
  auto page_at = [&](const Page& q) {
    return pool.pages + ((int64_t)q.entry * pool.Hkv + q.h) * pool.page_bytes;
  };
  auto look_scale = [&](Page& q) {
    if constexpr (T::block_scales)
      if (q.entry >= 0) q.scale = *reinterpret_cast<const float*>(page_at(q) + 2 * pool.code_bytes);
  };
  if (lane < nstage) mbar_init(&bars[lane], 1);
  fence_barrier_init();
  __syncwarp();
  Page now = look_up(0), next = look_up(batch);
  look_scale(now);
  look_scale(next);
  int base = 0;  // first stage of `now`'s batch
  const uint32_t page_tx = pool.code_bytes + p.scale_bytes;
  auto issue = [&](int n, int st) {  // all lanes call: stage n of the range into st
    if (n - base == batch) {
      now = next;
      base = n;
      next = look_up(n + batch);
    } else if (n - base == batch / 2) {
      look_scale(next);
    }
    const int first = (n - base) * sps, k = lane - first;
    const uint32_t there = __ballot_sync(0xffffffffu, now.entry >= 0) >> first & ((1u << sps) - 1);
    if (lane == 0) {
      info[st].there = there;
      if (there == 0) mbar_arrive(&bars[st]);
      else mbar_arrive_expect_tx(&bars[st], __popc(there) * page_tx);
    }
    __syncwarp();
    if (k >= 0 && k < sps) {  // the lanes that look after its pages
      if constexpr (T::block_scales) info[st].scale[k] = now.scale;
      if (now.entry >= 0) {
        char* dst = stages + st * stage_bytes + k * p.slot_bytes;
        const char* page = page_at(now);
        bulk_g2s(dst, page, pool.code_bytes, &bars[st]);
        if constexpr (T::token_scales)
          bulk_g2s(dst + pool.code_bytes, pool.tok_scales + (int64_t)now.entry * 2 * bs, p.scale_bytes, &bars[st]);
        else if constexpr (T::group_scales)
          bulk_g2s(dst + pool.code_bytes, page + 2 * pool.code_bytes, p.scale_bytes, &bars[st]);
      }
    }
  };
  for (int n = 0; n < min(n_w, nstage); ++n) issue(n, n);
  __syncwarp();  // (what issue wrote about its pages; later ones pass the loop's barriers)

  // ---- the row being weighed
  Cursor c = locate(a0);
  uint32_t qb[KS][2];
  uint32_t ql[T::channel ? KS : 1][2];
  float csc, lse2[2];
  int L = 0;
  int64_t row = 0;
  auto load_heads = [&](int ht) {
    load_q<FMT, D>(p.d, c.s, c.h, ht, lane, qb, ql, csc);
    // heads 2j, 2j+1 of the tile; one that is not there, or attends nothing, weighs 0
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int hq = 8 * ht + 2 * j + e;
      const float v = hq < p.d.G ? p.lse[(int64_t)c.s * p.d.Hq + c.h * p.d.G + hq] : -kInf;
      lse2[e] = v == -kInf ? kInf : v * 1.4426950408889634f;
    }
  };
  auto start_row = [&]() {
    L = min(p.d.lens[c.s], p.d.max_ctx);
    row = ((int64_t)c.s * pool.Hkv + c.h) * p.stride;
    if (p.d.n_ht == 1) load_heads(0);
  };
  start_row();

  // A stage's two sub-tiles: where this lane's words of tokens 0..7 and 8..15 lie in
  // it, and the scales of tokens g and g + 8
  int lo_at[2], hi_at[2], lo_sc[2], hi_sc[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int k = 16 * x >> bl, sub = (16 * x & (bs - 1)) >> 4;
    lo_at[x] = k * p.slot_bytes + sub * pool.sub_bytes + lane * 16;
    hi_at[x] = bs == 8 ? lo_at[x] + p.slot_bytes - NC / 2 * 512 : lo_at[x];
    lo_sc[x] = k * p.slot_bytes + pool.code_bytes + (16 * sub + g) * NS * 4;
    hi_sc[x] = lo_sc[x] + (bs == 8 ? p.slot_bytes : 8 * NS * 4);
  }
  int st = 0;
  uint32_t phase = 0;
  bool failed = false;
  int n = 0;
  for (; n < n_w; ++n) {
    // the weights so far, on their way while the stage is waited for
    float before[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int tw = c.i * span + 32 * e + lane;
      before[e] = p.prev != nullptr && tw < L && 32 * e < span ? p.prev[row + tw] : 0.f;
    }
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[st], phase, p.d.wait_tries))) {
      failed = true;
      break;
    }
    const char* stage = stages + st * stage_bytes;
    const int there = info[st].there;
    // two sub-tiles (32 tokens) at a time; what lies behind the sequence computes on
    // whatever the stage holds and is not stored
#pragma unroll 1
    for (int o = 0; o < span; o += 32) {
      const int t = c.i * span + o;
      if (t >= L) break;
      uint32_t kw[2][NU32];
      float ks[2][2][NS];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int more = (o >> 4) * pool.sub_bytes;  // (blocks of 64 tokens: the second pair)
#pragma unroll
        for (int q = 0; q < NC; ++q) {
          // chunks of the first half hold tokens 0..7, of the second 8..15 (INT4
          // words hold both; 8-token pages a half each)
          const bool second = FMT != FMT_INT4_GROUP && q >= NC / 2;
          const uint4 v = *reinterpret_cast<const uint4*>(stage + (second ? hi_at[x] : lo_at[x]) + more + q * 512);
          kw[x][4 * q] = v.x;
          kw[x][4 * q + 1] = v.y;
          kw[x][4 * q + 2] = v.z;
          kw[x][4 * q + 3] = v.w;
        }
        if constexpr (T::block_scales) {
          ks[x][0][0] = info[st].scale[16 * x >> bl];
          ks[x][1][0] = info[st].scale[(16 * x + 8) >> bl];
        } else if constexpr (kCopied) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float* sc = reinterpret_cast<const float*>(stage + (r ? hi_sc[x] : lo_sc[x])) + o * NS;
#pragma unroll
            for (int gi = 0; gi < NS; ++gi) ks[x][r][gi] = sc[gi];
          }
        }
      }
      float w[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
      for (int ht = 0; ht < p.d.n_ht; ++ht) {
        if (p.d.n_ht > 1) load_heads(ht);
        float acc[2][NG][4];
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t f0, f1, f2, f3;
            k_frag<FMT, D>(kw[x], kk, f0, f1, f2, f3);
            if (kk % KPG == 0)
              mma_16816_from0(acc[x][kk / KPG], f0, f1, f2, f3, qb[kk][0], qb[kk][1]);
            else
              mma_16816(acc[x][kk / KPG], f0, f1, f2, f3, qb[kk][0], qb[kk][1]);
            if constexpr (T::channel)
              mma_16816(acc[x][kk / KPG], f0, f1, f2, f3, ql[kk][0], ql[kk][1]);
          }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int r = 0; r < 2; ++r) {  // tokens g and g + 8
            float z0 = -lse2[0], z1 = -lse2[1];
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
              const float sc = T::row_scales ? csc * ks[x][r][T::group_scales ? gi : 0] : csc;
              z0 = fmaf(acc[x][gi][2 * r], sc, z0);
              z1 = fmaf(acc[x][gi][2 * r + 1], sc, z1);
            }
            float e0 = fast_exp2(z0), e1 = fast_exp2(z1);
            if constexpr (T::maybe_nan) {  // (an infinite k makes 0 * k of an absent head NaN)
              e0 = lse2[0] == kInf ? 0.f : e0;
              e1 = lse2[1] == kInf ? 0.f : e1;
            }
            w[x][r] += e0 + e1;
          }
      }
      __syncwarp();  // the sums before these have been read
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 2; ++r) part[(16 * x + 8 * r + g) * 4 + j] = w[x][r];
      __syncwarp();
      const float4 v = *reinterpret_cast<const float4*>(part + lane * 4);
      if (t + lane < L && (there >> ((o + lane) >> bl) & 1))
        p.scores[row + t + lane] = fmaf(p.decay, o == 0 ? before[0] : before[1],
                                        (v.x + v.y) + (v.z + v.w));
    }
    __syncwarp();  // every lane has read the stage
    if (n + nstage < n_w) issue(n + nstage, st);
    if (++st == nstage) {
      st = 0;
      phase ^= 1u;
    }
    if (advance(c) && n + 1 < n_w) start_row();
  }
  if (failed) {
    // A wait ran out: flag it, then wait (bounded again) for this warp's copies
    // still in flight so that none lands after the CTA has exited.
    if (lane == 0) set_error(pool.err, ERR_TIMEOUT);
    for (int k = n; k < min(n_w, n + nstage); ++k) {
      mbar_wait_bounded(&bars[st], phase, p.d.wait_tries);
      if (++st == nstage) {
        st = 0;
        phase ^= 1u;
      }
    }
    __syncwarp();
  }
}

struct WeightsLaunch {
  WeightsParams p;
  int sms;
  cudaStream_t st;
};

template <int FMT, int D, int NG>
cudaError_t run_weights(const WeightsLaunch& l) {
  WeightsParams p = l.p;
  const PoolView& pool = p.d.pool;
  using T = FmtTraits<FMT>;
  p.scale_bytes = T::group_scales ? pool.bs * NG * 4 : T::token_scales ? pool.bs * 4 : 0;
  p.slot_bytes = (pool.code_bytes + p.scale_bytes + 127) / 128 * 128;
  // stages: what kWeightsCtas CTAs leave each of their warps of an SM's 228 KB
  const int span = pool.bs < 32 ? 32 : pool.bs;
  const int stage = p.slot_bytes * span / pool.bs + static_cast<int>(sizeof(StageInfo)) + 8;
  if (p.d.S > 227 * 1024 / 4) return cudaErrorInvalidValue;  // (its prefix alone: the sums below stay in 32 bits)
  const int fixed = kWeightsWarps * (512 + 4) + (p.d.S + 1) * 4;
  auto stages_of = [&](int ctas) { return (228 * 1024 / ctas - 1024 - fixed) / kWeightsWarps / stage; };
  int room = stages_of(kWeightsCtas);
  if (room < 3) room = stages_of(2);  // (large pages: fewer warps with deeper streams)
  p.nstage = room < 2 ? 2 : room < kWeightsStages ? room : kWeightsStages;
  const int smem = kWeightsWarps * p.nstage * stage + fixed;
  if (smem > 227 * 1024) return cudaErrorInvalidValue;
  // one warp per stage at most
  const int64_t stages = (int64_t)((p.d.max_ctx + span - 1) / span) * p.d.S * pool.Hkv;
  if (stages > 0x7fffffffLL - (1 << 17)) return cudaErrorInvalidValue;  // (the kernel rounds them up to its warps)
  const int fit = 228 * 1024 / (smem + 1024);
  const int64_t full = (int64_t)l.sms * (fit < kWeightsCtas ? fit : kWeightsCtas), need = (stages + kWeightsWarps - 1) / kWeightsWarps;
  const int64_t grid = need < full ? need : full;
  const cudaError_t e = allow_big_smem<kvq_weights_kernel<FMT, D, NG>>();
  if (e != cudaSuccess) return e;
  kvq_weights_kernel<FMT, D, NG><<<static_cast<unsigned>(grid), kWeightsWarps * 32, smem, l.st>>>(p);
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
