// kvq_decode4_impl.cuh -- paged decode attention over a pool of 4-bit floats.
//
// The mathematics is that of kvq_decode_impl.cuh: softmax(q . k^T) v per row, k and v
// dequantized on the way, one pass with a running maximum and sum, long sequences cut
// over warps and joined by the merge kernel.  What differs is what bounds it.  At 4.5
// bits a value a page is a quarter of an FP16 one while its tokens want the same products and
// weights, so the work per token decides, not the bytes (64 x 2048 tokens, 8 kv
// heads of 128: 22 us of HBM time; the general kernel took 53):
//  * A step is 64 tokens whatever the block size: one barrier, one softmax update, one look
//    at the bookkeeping for four sub-tiles instead of two or one.
//  * The lanes that look after a step's pages issue their copies side by side, from table
//    entries they hold 32 pages ahead; no lane walks a cursor.
//  * Dequantized values are exact fp16 fragments (kvq_fp4.cuh): no scale is left for the
//    scores, the weights or the sums.
//  * P.V of a step is summed from zero and added to O in fp32 together with O's rescaling, one
//    multiply-add an output; the sums of long ranges never pass through the tensor core's
//    truncating accumulator.
//  * DUP: groups of up to 4 rows leave half of the 8 columns of an mma idle.  Columns 4..7
//    take the same heads once more: their lanes carry the low parts of the weights
//    (p - fp16(p)) where the others carry the high parts, so that one product does what
//    two did.
// The range of a warp and the partials are as in the general kernel with
// steps in the place of pages; kvq_merge_kernel joins them.
// Measured, calls replayed back to back: 64 x 2048 37.7 us (151 MB, 4.0 TB/s, 0.59 of the copy
// rate), 64 x 512 16.4, 64 x 8192 116.9: some 26 us for 2048 more tokens (0.84 of the copy
// rate) and 11 us of start, merge and uneven ends; 8 x 16384..32768 in blocks of 32: 47.0.
// Neither HBM (52%) nor the issue slots (48%) are full: with 2.8 warps a scheduler one is ready in 56% of
// the cycles, so a step's waits -- conversion, softmax and P.V follow each other in a warp -- bound it.
// (One stage of 16 warps a CTA instead of two stages for each of 4: more instructions,
// slower at every length.)
#pragma once
#include "kvq_decode_impl.cuh"

namespace kvq {

constexpr int kDecode4Span = 64;   // tokens of a step
constexpr int kDecode4Ctas = 3;    // resident per SM
// Rows of a head tile that fit 4 columns take the DUP kernel.
constexpr bool decode4_dup(int G) { return G <= 4; }
constexpr float kDecode4Exp = 14;  // weights are 2^14 p, so that their low parts stay normal fp16

template <int D, bool DUP, bool DIFF>
__global__ void __launch_bounds__(kDecodeThreads, kDecode4Ctas)
    kvq_decode4_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int KS = D / 16, NG = D / 16, NC = NG / 4;  // 16-channel steps; 16-byte chunks per lane
  constexpr int NL = DUP ? 1 : 2;                       // weight fragments of a sub-tile: hi, lo
  const float kNegInf = __int_as_float(0xff800000u);

  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, j = lane & 3;
  const PoolView& pool = p.pool;
  const int bl = 31 - __clz(pool.bs), nstage = p.nstage;
  const int sps = kDecode4Span >> bl;  // pages per step
  const int U = pool.Hkv * p.n_ht;     // units per sequence

  char* stages = smem + warp * nstage * p.stage_bytes;
  uint64_t* bars_base = reinterpret_cast<uint64_t*>(smem + kDecodeWarps * nstage * p.stage_bytes);
  uint64_t* bars = bars_base + warp * nstage;
  if (lane < nstage) mbar_init(&bars[lane], 1);
  fence_barrier_init();
  // Launched while the kernel before it ends; only the decode step's append vouches for
  // the lengths and the table.
  if (!p.inputs_early) asm volatile("griddepcontrol.wait;" ::: "memory");
  // The join may launch now: it waits for this grid, but reads the lengths before that.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int* there_base = reinterpret_cast<int*>(bars_base + kDecodeWarps * nstage);
  int* there_at = there_base + warp * nstage;  // pages of each stage that are in the pool, a bit each
  int* wtot = there_base + kDecodeWarps * nstage;  // [kDecodeWarps]
  int* PS = wtot + kDecodeWarps;                   // [S + 1] steps before each sequence

  // tokens of sequence s to attend here (the cascade has seen its first `skip` blocks)
  auto tokens_of = [&](int s) { return tokens_behind(p.lens[s], p.max_ctx, p.skip, pool.bs); };

  // ---- steps per sequence and their prefix (every CTA computes the same)
  {
    int carry = 0;
    for (int base = 0; base < p.S; base += kDecodeThreads) {
      const int s = base + threadIdx.x;
      int v = 0;
      if (s < p.S) {
        if (p.lens[s] > p.max_ctx && blockIdx.x == 0) set_error(pool.err, ERR_RANGE);
        v = (tokens_of(s) + kDecode4Span - 1) / kDecode4Span * U;
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
      for (int w = 0; w < kDecodeWarps; ++w) {
        before += w < warp ? wtot[w] : 0;
        all += wtot[w];
      }
      if (s < p.S) PS[s + 1] = carry + before + x;
      carry += all;
      __syncthreads();
    }
    if (threadIdx.x == 0) PS[0] = 0;
    __syncthreads();
  }
  const int Ttot = PS[p.S];
  const int nwarps = gridDim.x * kDecodeWarps;
  const int gw = blockIdx.x * kDecodeWarps + warp;
  const int ppw = p.ppw_fixed > 0 ? p.ppw_fixed : (Ttot + nwarps - 1) / nwarps;
  const int a0 = static_cast<int>(min((int64_t)gw * ppw, (int64_t)Ttot));
  const int n_w = static_cast<int>(min((int64_t)a0 + ppw, (int64_t)Ttot)) - a0;

  // Writes come only after griddepcontrol.wait: the merge before may still be reading.
  auto after_wait = [&]() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (gw == 0)  // the prefix, for the merge kernel
      for (int s = lane; s <= p.S; s += 32) p.ps[s] = PS[s];
    // sequences with nothing (left) to attend: zeros, or the cascade's normalised prefix
    for (int s = gw; s < p.S; s += nwarps) {
      if (PS[s + 1] != PS[s]) continue;
      if constexpr (DIFF) {
        __half* o = p.diff.out + (int64_t)s * (p.Hq / 2) * D;
        for (int i = lane; i < p.Hq / 2 * D; i += 32) o[i] = __ushort_as_half(0);
        continue;
      }
      float* o = p.out + (int64_t)s * p.out_stride;
      if (p.lse != nullptr)
        for (int i = lane; i < p.Hq; i += 32) p.lse[(int64_t)s * p.Hq + i] = kNegInf;
      for (int hq = 0; hq < p.Hq; ++hq) {
        const float* pr = p.pre + ((int64_t)s * p.Hq + hq) * (D + 2);
        const float f = p.pre != nullptr && pr[1] > 0.f ? 1.f / pr[1] : 0.f;
        for (int d = lane; d < D; d += 32) o[(int64_t)hq * D + d] = f != 0.f ? pr[2 + d] * f : 0.f;
      }
    }
  };
  if (n_w <= 0) {
    after_wait();
    return;
  }

  struct Cursor4 {
    int s, lu, i, Ps;  // sequence, unit within it, step within the unit, steps per unit
  };
  auto locate = [&](int x) {
    int lo = 0, hi = p.S;  // PS[lo] <= x < PS[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (PS[mid] <= x) lo = mid; else hi = mid;
    }
    Cursor4 c;
    c.s = lo;
    c.Ps = (PS[lo + 1] - PS[lo]) / U;
    const int r = x - PS[lo];
    c.lu = r / c.Ps;
    c.i = r - c.lu * c.Ps;
    return c;
  };
  auto advance = [&](Cursor4& c) {
    if (++c.i < c.Ps) return;
    c.i = 0;
    if (++c.lu < U) return;
    c.lu = 0;
    do { ++c.s; } while (c.s < p.S && PS[c.s + 1] == PS[c.s]);
    c.Ps = c.s < p.S ? (PS[c.s + 1] - PS[c.s]) / U : 1;
  };

  // ---- pages on their way: a lane looks after one page of each batch of 32.  Its table
  // entry is asked for a batch ahead and looked at when the batch begins, so that no
  // copy waits for it.
  struct Entry {
    int block, h;  // kv head; -1: behind the sequence
    bool last;     // of the sequence's last step
  };
  struct Page {
    const char* at;  // null: nothing to copy
    bool last;
  };
  const int batch = 32 / sps;  // steps of a batch
  auto look_up = [&](int n0) {
    Entry q{0, -1, false};
    const int n = n0 + lane / sps;
    if (n < n_w) {
      const Cursor4 c = locate(a0 + n);
      const int pg = c.i * sps + lane % sps;
      q.last = c.i + 1 == c.Ps;
      if (pg << bl < tokens_of(c.s)) {
        q.block = p.table[(int64_t)c.s * p.max_blocks + p.skip + pg];
        q.h = c.lu / p.n_ht;
      }
    }
    return q;
  };
  auto page_of = [&](const Entry& q) {
    const bool in = q.block >= 0 && (int64_t)q.block < pool.num_blocks;
    if (q.h >= 0 && !in) set_error(pool.err, ERR_RANGE);
    return Page{q.h >= 0 && in ? pool.pages + ((int64_t)q.block * pool.Hkv + q.h) * pool.page_bytes : nullptr,
                q.last};
  };
  Page now = page_of(look_up(0));
  Entry next = look_up(batch);
  int base = 0;  // first step of `now`'s batch
  auto issue = [&](int n, int st) {  // all lanes: step n of the range into stage st
    if (n - base == batch) {
      now = page_of(next);
      base = n;
      next = look_up(n + batch);
    }
    const int first = (n - base) * sps, k = lane - first;
    const uint32_t there = __ballot_sync(0xffffffffu, now.at != nullptr) >> first & ((1u << sps) - 1);
    if (lane == 0) {
      there_at[st] = there;
      if (there == 0) mbar_arrive(&bars[st]);
      else mbar_arrive_expect_tx(&bars[st], __popc(there) * pool.page_bytes);
    }
    __syncwarp();
    const bool held = p.fault_issue >= 0 && gw == 0 && n == p.fault_issue;  // (bytes that never come)
    if (k >= 0 && k < sps && now.at != nullptr && !held)
      bulk_g2s(stages + st * p.stage_bytes + k * pool.page_bytes, now.at, pool.page_bytes, &bars[st]);
  };
  // Everything above reads only inputs.  As a dependent of the decode step's append, which
  // writes each sequence's last page, the steps up to the first one that holds such a page
  // are fetched before griddepcontrol.wait (see kvq_decode_impl.cuh).
  {
    const int npre = min(n_w, nstage);
    int n = 0;
    for (; n < npre; ++n) {
      if (__shfl_sync(0xffffffffu, now.last, (n - base) * sps & 31)) break;
      issue(n, n);
    }
    after_wait();
    for (; n < npre; ++n) issue(n, n);
    __syncwarp();
  }

  // ---- a sub-tile's codes and scales in a stage (the same for the whole warp)
  int tile_at[4], scale_at[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int k = 16 * t >> bl, sub = (16 * t & (pool.bs - 1)) >> 4;
    tile_at[t] = k * pool.page_bytes + sub * pool.sub_bytes;
    scale_at[t] = k * pool.page_bytes + pool.code_bytes + sub * D;
  }
  const int v_off = pool.v_off;

  // ---- the unit being attended: columns 2j, 2j+1 are this lane's.  The scale is kept
  // positive (its sign goes to q; zero is a zero q), so that it leaves the order of scores.
  const float csc0 = p.sm_scale_log2, csc = csc0 == 0.f ? 1.f : fabsf(csc0);
  uint32_t qb[KS][2];
  float m[2], l[2], o[KS][4];
  Cursor4 cc = locate(a0);
  const Cursor4 first = cc;
  int seg0 = cc.i, L = 0;
  auto start_unit = [&]() {
    L = tokens_of(cc.s);
    const int h = cc.lu / p.n_ht, ht = cc.lu % p.n_ht;
    const int Gt = min(8, p.G - 8 * ht), row = DUP ? g & 3 : g;
    const int hq = h * p.G + 8 * ht + (row < Gt ? row : 0);
    const __half* qp = p.q + (int64_t)cc.s * p.q_stride + (int64_t)(DIFF ? hq >> 1 : hq) * D + 4 * j;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      // a map has its half of the channels
      const bool has = row < Gt && csc0 != 0.f && (!DIFF || (kk >= KS / 2) == ((hq & 1) != 0));
      const uint2 v = has ? *reinterpret_cast<const uint2*>(qp + 16 * kk) : make_uint2(0, 0);
      qb[kk][0] = csc0 < 0.f ? v.x ^ 0x80008000u : v.x;
      qb[kk][1] = csc0 < 0.f ? v.y ^ 0x80008000u : v.y;
    }
    m[0] = m[1] = kNegInf;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    seg0 = cc.i;
  };

  // Result of a unit that lies within this range, or its partial (m, l, O in true units).
  auto finish_unit = [&](const Cursor4& u, int seg_end) {
    const int h = u.lu / p.n_ht, ht = u.lu % p.n_ht;
    const int Gt = min(8, p.G - 8 * ht);
    if constexpr (DUP) {  // high and low parts
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][e] += __shfl_xor_sync(0xffffffffu, o[mt][e], 2);
    }
    const float lt[2] = {warp_sum_over_rows(l[0]), warp_sum_over_rows(l[1])};
    // (with DUP the lanes j >= 2 hold the heads of j - 2 once more)
    const bool v0 = 2 * j < Gt && (!DUP || j < 2), v1 = 2 * j + 1 < Gt && (!DUP || j < 2);
    const bool whole = seg0 == 0 && seg_end == u.Ps;
    if (DIFF && whole) {  // both maps of a head are this lane's
      const float f0 = lt[0] > 0.f ? 1.f / lt[0] : 0.f, f1 = lt[1] > 0.f ? 1.f / lt[1] : 0.f;
      const int head = h * (p.G / 2) + 4 * ht + j;
      const float f1l = v0 ? f1 * p.diff.lambda[head] : 0.f;
      float ss = 0.f;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        o[mt][0] = diff_of(o[mt][0], f0, o[mt][1], f1l);
        o[mt][2] = diff_of(o[mt][2], f0, o[mt][3], f1l);
        ss = fmaf(o[mt][0], o[mt][0], fmaf(o[mt][2], o[mt][2], ss));
      }
      const float f = diff_factor<D>(p.diff, warp_sum_over_rows(ss));
      if (!v0) return;
      __half* dst = p.diff.out + ((int64_t)u.s * (p.Hq / 2) + head) * D;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        const int d0 = 16 * mt + g;
        const float w0 = p.diff.weight != nullptr ? f * p.diff.weight[d0] : f;
        const float w8 = p.diff.weight != nullptr ? f * p.diff.weight[d0 + 8] : f;
        dst[d0] = __float2half_rn(o[mt][0] * w0);
        dst[d0 + 8] = __float2half_rn(o[mt][2] * w8);
      }
      return;
    }
    const float down = pow2f(-static_cast<int>(kDecode4Exp));
    const int64_t row0 = (int64_t)u.s * p.Hq + h * p.G + 8 * ht;
    if (whole) {
      float* obase = p.out + (int64_t)u.s * p.out_stride + (int64_t)(h * p.G + 8 * ht) * D;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!(c ? v1 : v0)) continue;
        if (p.lse != nullptr && g == 0) p.lse[row0 + 2 * j + c] = row_lse(m[c], lt[c] * down);
        float* dst = obase + (2 * j + c) * D;
        if (p.pre == nullptr) {
          const float f = lt[c] > 0.f ? 1.f / lt[c] : 0.f;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            dst[16 * mt + g] = o[mt][c] * f;
            dst[16 * mt + g + 8] = o[mt][2 + c] * f;
          }
        } else {  // cascade: log-sum-exp with the row's prefix partial
          const float* pr = p.pre + (row0 + 2 * j + c) * (D + 2);
          const float mp = pr[0], lp = pr[1], lu = lt[c] * down;
          const float M = fmaxf(m[c], mp);
          const float wu = m[c] == kNegInf ? 0.f : fast_exp2(m[c] - M);
          const float wp = mp == kNegInf ? 0.f : fast_exp2(mp - M);
          const float den = fmaf(lu, wu, lp * wp);
          const float inv = den > 0.f ? 1.f / den : 0.f;
          const float fu = wu * down * inv, fp = wp * inv;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            const int d0 = 16 * mt + g;
            dst[d0] = fmaf(o[mt][c], fu, pr[2 + d0] * fp);
            dst[d0 + 8] = fmaf(o[mt][2 + c], fu, pr[2 + d0 + 8] * fp);
          }
        }
      }
      return;
    }
    const int slot = (u.s == first.s && u.lu == first.lu) ? 0 : 1;
    float* pbase = p.part + ((int64_t)gw * 2 + slot) * p.part_rows * (D + 2);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (!(c ? v1 : v0)) continue;
      float* r = pbase + (2 * j + c) * (D + 2);
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        r[2 + 16 * mt + g] = o[mt][c] * down;
        r[2 + 16 * mt + g + 8] = o[mt][2 + c] * down;
      }
      if (g == 0) {
        r[0] = m[c];
        r[1] = lt[c] * down;
      }
    }
  };

  start_unit();
  int st = 0;
  uint32_t phase = 0;
  bool failed = false;
  int n = 0;
  for (; n < n_w; ++n) {
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[st], phase, p.wait_tries))) {
      failed = true;
      break;
    }
    const char* stage = stages + st * p.stage_bytes;
    const int there = there_at[st];
    const int left = L - cc.i * kDecode4Span;  // tokens from this step on
    const bool full = left >= kDecode4Span && there == (1 << sps) - 1;
    auto rows_of = [&](int t) {
      return there >> (16 * t >> bl) & 1 ? min(max(left - 16 * t, 0), 16) : 0;
    };

    // ---- scores of 4 x 16 tokens (g and g + 8 of each) for this lane's two columns
    float z[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float acc[2][4];
      const char* tile = stage + tile_at[t] + lane * 16;
      const char* sc = stage + scale_at[t] + g * 2 * NG;
      uint32_t sw[2][NC];  // scales of tokens g, g + 8
      if constexpr (NC == 2) {
        const uint4 v = *reinterpret_cast<const uint4*>(sc);
        sw[0][0] = v.x;
        sw[0][1] = v.y;
        sw[1][0] = v.z;
        sw[1][1] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(sc);
        sw[0][0] = v.x;
        sw[1][0] = v.y;
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(tile + c * 512);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        __half2 s0[2], s8[2];
        fp4_scales(sw[0][c], s0[0], s0[1]);
        fp4_scales(sw[1][c], s8[0], s8[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = 4 * c + i;
          uint32_t a[4];
          fp4_k_frag(w[i], i & 2 ? __high2half2(s0[i & 1]) : __low2half2(s0[i & 1]),
                     i & 2 ? __high2half2(s8[i & 1]) : __low2half2(s8[i & 1]), a);
          if (kk < 2) mma_16816_from0(acc[kk & 1], a[0], a[1], a[2], a[3], qb[kk][0], qb[kk][1]);
          else mma_16816(acc[kk & 1], a[0], a[1], a[2], a[3], qb[kk][0], qb[kk][1]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) z[t][e] = acc[0][e] + acc[1][e];
    }
    uint32_t keep[4][2];  // bits of the V scales that count: tokens 2j, 2j+1 | 2j+8, 2j+9
#pragma unroll
    for (int t = 0; t < 4; ++t) keep[t][0] = keep[t][1] = 0x7F807F80u;
    if (!full) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int rows = rows_of(t);
        if (g >= rows) z[t][0] = z[t][1] = kNegInf;
        if (g + 8 >= rows) z[t][2] = z[t][3] = kNegInf;
        const uint32_t mk = fp4_v_mask(j, rows);
        keep[t][0] &= mk << 7;
        keep[t][1] &= mk >> 1;
      }
    }

    // ---- softmax update (base 2); weights p 2^14 as B fragments
    float al[2];
    uint32_t pb[4][NL][2];
    {
      float mb[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float t = fmaxf(fmaxf(fmaxf(z[0][c], z[0][2 + c]), fmaxf(z[1][c], z[1][2 + c])),
                        fmaxf(fmaxf(z[2][c], z[2][2 + c]), fmaxf(z[3][c], z[3][2 + c])));
        const float mn = fmaxf(m[c], warp_max_over_rows(t) * csc);
        const float ms = mn == kNegInf ? 0.f : mn;
        al[c] = fast_exp2(m[c] - ms);
        m[c] = mn;
        mb[c] = ms - kDecode4Exp;
      }
      float add[2] = {0.f, 0.f};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) z[t][e] = fast_exp2(fmaf(z[t][e], csc, -mb[e & 1]));
        add[0] += z[t][0] + z[t][2];
        add[1] += z[t][1] + z[t][3];
        if constexpr (DUP) {
          uint32_t hA, lA, hB, lB;
          split_h2(z[t][0], z[t][1], hA, lA);
          split_h2(z[t][2], z[t][3], hB, lB);
          pb[t][0][0] = movmatrix_t(j < 2 ? hA : lA);
          pb[t][0][1] = movmatrix_t(j < 2 ? hB : lB);
        } else {
          uint32_t hA, lA, hB, lB;
          split_h2(z[t][0], z[t][1], hA, lA);
          split_h2(z[t][2], z[t][3], hB, lB);
          pb[t][0][0] = movmatrix_t(hA);
          pb[t][0][1] = movmatrix_t(hB);
          pb[t][NL - 1][0] = movmatrix_t(lA);
          pb[t][NL - 1][1] = movmatrix_t(lB);
        }
      }
      l[0] = fmaf(l[0], al[0], add[0]);
      l[1] = fmaf(l[1], al[1], add[1]);
    }

    // ---- O = al O + V^T P, 64 channels at a time
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float acc[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint4 v = *reinterpret_cast<const uint4*>(stage + tile_at[t] + v_off + lane * 16 + c * 512);
        const uint4 q = *reinterpret_cast<const uint4*>(stage + scale_at[t] + v_off + j * 4 * NG + 16 * c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w}, sw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo = sw[i] << 7 & keep[t][0], hi = sw[i] >> 1 & keep[t][1];
          uint32_t a[4];
          fp4_v_frag(w[i], *reinterpret_cast<const __half2*>(&lo), *reinterpret_cast<const __half2*>(&hi), a);
          if (t == 0) mma_16816_from0(acc[i], a[0], a[1], a[2], a[3], pb[t][0][0], pb[t][0][1]);
          else mma_16816(acc[i], a[0], a[1], a[2], a[3], pb[t][0][0], pb[t][0][1]);
          if constexpr (!DUP) mma_16816(acc[i], a[0], a[1], a[2], a[3], pb[t][NL - 1][0], pb[t][NL - 1][1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[4 * c + i][e] = fmaf(o[4 * c + i][e], al[e & 1], acc[i][e]);
    }
    __syncwarp();  // every lane has read the stage
    if (n + nstage < n_w) issue(n + nstage, st);
    if (++st == nstage) {
      st = 0;
      phase ^= 1u;
    }
    const Cursor4 done = cc;
    advance(cc);
    if (done.i + 1 == done.Ps || n + 1 == n_w) {
      finish_unit(done, done.i + 1);
      if (n + 1 < n_w) start_unit();
    }
  }
  if (failed) {
    // flag it, leave empty partials for the merge, wait (bounded again) for the copies
    // still in flight so that none lands after the CTA has exited
    if (lane == 0) set_error(pool.err, ERR_TIMEOUT);
    if (lane < 2 * p.part_rows) {
      float* r = p.part + ((int64_t)gw * 2 * p.part_rows + lane) * (D + 2);
      r[0] = kNegInf;
      r[1] = 0.f;
    }
    for (int k = n; k < min(n_w, n + nstage); ++k) {
      mbar_wait_bounded(&bars[st], phase, p.wait_tries);
      if (++st == nstage) {
        st = 0;
        phase ^= 1u;
      }
    }
    __syncwarp();
  }
}

template <int D, bool DUP, bool DIFF>
cudaError_t run_decode4(const DecodeLaunch& l) {
  const cudaError_t e = allow_big_smem<kvq_decode4_kernel<D, DUP, DIFF>>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t dc = {};
  dc.gridDim = l.grid;
  dc.blockDim = dim3(kDecodeThreads);
  dc.dynamicSmemBytes = l.smem;
  dc.stream = l.st;
  cudaLaunchAttribute da[1];
  da[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  da[0].val.programmaticStreamSerializationAllowed = 1;
  dc.attrs = da;
  dc.numAttrs = 1;
  const cudaError_t f = phase_mark(l.st, cudaLaunchKernelEx(&dc, kvq_decode4_kernel<D, DUP, DIFF>, l.p));
  return f != cudaSuccess ? f : run_merge<D, DIFF>(l);
}

template <bool DIFF>
cudaError_t run_decode4_any(const DecodeLaunch& l) {
  const bool dup = decode4_dup(l.p.G);
  if (l.p.pool.D == 64) return dup ? run_decode4<64, true, DIFF>(l) : run_decode4<64, false, DIFF>(l);
  return dup ? run_decode4<128, true, DIFF>(l) : run_decode4<128, false, DIFF>(l);
}

}  // namespace kvq
