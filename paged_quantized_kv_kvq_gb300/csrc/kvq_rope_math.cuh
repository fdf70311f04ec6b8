// kvq_rope_math.cuh -- per-head RMS norm and rotary positions of 8-channel
// chunks held in registers (sm_103a).
//
// A head of D channels lies over D/8 consecutive lanes, 8 channels each.  The
// norm is y = x / sqrt(mean(x^2) + eps) * w with the mean over the head in
// fp32.  Pair i of the first r channels turns by the angle pos * f_i:
//   (u, v) -> m (u cos - v sin, u sin + v cos),
// the pair being channels (i, i + r/2) or (2i, 2i+1).
//
// The angle.  A plan holds f_i / 2pi -- turns per position -- as a 64-bit
// fraction; pos times it, modulo 2^64, is the position's fraction of a turn
// without a rounding, where an fp32 angle at position 10^5 would be off by 2^-8.
// What is off is the fraction itself: it comes from fp64 and is good to 2^-52 of a
// turn (2^-55 measured), so 2^-23.3 radians at position 2^26, in proportion beyond.
// The top 32 bits, less the nearest quarter turn, give an angle in [-pi/4, pi/4] within
// 2^-23.6 (the conversion 2^-25.3, the factor 2^-25.4, the product 2^-25), and the
// Taylor series of sine and cosine there, to x^9 and x^10 (the next terms are below
// 2^-29), round by 2^-24: 2^-23 in all, 2^-22 with the fraction up to position 2^26.
// That is at the level of the norm's and the rotation's own roundings, so that a key
// falls on the other side of a code's border no more often for it.  (The hardware's
// sine and cosine, 2^-21, did so three times as often: 12 codes of 64 x 8 x 128 x 60
// against 4 of fp64 angles.)  No table of positions is read, so there is no longest
// position and no cache traffic.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq.h"
#include "kvq_f32x2.cuh"

namespace kvq {

// cos and sin (times the plan's magnitude) of `pos` at `turn` turns per position.
__device__ __forceinline__ float2 rope_cs(uint64_t turn, int64_t pos, float magnitude) {
  const uint32_t frac = static_cast<uint32_t>(turn * static_cast<uint64_t>(pos) >> 32);
  const uint32_t quarter = (frac + 0x20000000u) >> 30;  // the nearest, modulo four
  const float a = static_cast<float>(static_cast<int32_t>(frac - (quarter << 30))) * 1.4629180792671596e-9f;
  const float x = a * a;  // (a: 2 pi / 2^32 times what is left)
  const float s = fmaf(a * x, fmaf(fmaf(fmaf(1.f / 362880, x, -1.f / 5040), x, 1.f / 120), x, -1.f / 6), a);
  const float c = fmaf(fmaf(fmaf(fmaf(fmaf(-1.f / 3628800, x, 1.f / 40320), x, -1.f / 720), x, 1.f / 24), x, -0.5f), x, 1.f);
  // a quarter turn takes (cos, sin) to (-sin, cos)
  const uint32_t u = __float_as_uint(quarter & 1 ? s : c) ^ ((quarter + 1) & 2) << 30;
  const uint32_t v = __float_as_uint(quarter & 1 ? c : s) ^ (quarter & 2) << 30;
  return make_float2(__uint_as_float(u) * magnitude, __uint_as_float(v) * magnitude);
}

// Cosines and sines of tokens 0 .. n-1 (their positions at `pos`): cs[t][pair].
// A thread keeps its pair.
template <int THREADS>
__device__ __forceinline__ void rope_table(const kvq_rope_plan& plan, const int64_t* pos, int n,
                                           float2* cs) {
  static_assert(THREADS % KVQ_ROPE_MAX_PAIRS == 0, "a thread per pair");
  const int rp = plan.rotary_dim >> 1, q = threadIdx.x % KVQ_ROPE_MAX_PAIRS;
  if (q >= rp) return;
  const uint64_t turn = plan.turns[q];
  for (int t = threadIdx.x / KVQ_ROPE_MAX_PAIRS; t < n; t += THREADS / KVQ_ROPE_MAX_PAIRS)
    cs[t * rp + q] = rope_cs(turn, pos[t], plan.magnitude);
}

// 8 values of a 16-byte chunk, widened exactly.
__device__ __forceinline__ void widen8(uint4 raw, bool bf16, float (&x)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// RMS norm of the head this thread's chunk belongs to; every lane of the warp
// calls it (lanes without a row carry zeros).
template <int D>
__device__ __forceinline__ void norm8(float (&x)[8], const float (&w)[8], float eps) {
  uint64_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2_pack(x[2 * i], x[2 * i + 1]);
  uint64_t q = f2_mul(v[0], v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) q = f2_madd(v[i], v[i], q);
  float s, s1;
  f2_unpack(q, s, s1);
  s += s1;
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float r = rsqrtf(fmaf(s, 1.f / D, eps));
  const uint64_t rr = f2_pack(r, r);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f2_unpack(f2_mul(v[i], f2_mul(f2_pack(w[2 * i], w[2 * i + 1]), rr)), x[2 * i], x[2 * i + 1]);
}

// Rotation of chunk `ci` (channels 8ci .. 8ci+7) of a head whose token's cos
// and sin are cs[0 .. r/2); every lane of the warp calls it.
template <int D>
__device__ __forceinline__ void rotate8(float (&x)[8], int ci, int r, bool interleaved,
                                        const float2* cs) {
  if (interleaved) {
    if (8 * ci < r) {
      const float4* t = reinterpret_cast<const float4*>(cs + 4 * ci);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 c = t[i];
        const float u0 = x[4 * i], v0 = x[4 * i + 1], u1 = x[4 * i + 2], v1 = x[4 * i + 3];
        x[4 * i] = fmaf(u0, c.x, -v0 * c.y);
        x[4 * i + 1] = fmaf(u0, c.y, v0 * c.x);
        x[4 * i + 2] = fmaf(u1, c.z, -v1 * c.w);
        x[4 * i + 3] = fmaf(u1, c.w, v1 * c.z);
      }
    }
    return;
  }
  // the partner channel of pair i sits r/2 channels, i.e. half = r/16 lanes, away
  const int half = r >> 4;
  const bool lo = ci < half, in = ci < 2 * half;
  const int lane = threadIdx.x & 31;
  const int partner = in ? (lane & ~(D / 8 - 1)) | (lo ? ci + half : ci - half) : lane;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner);
  if (in) {
    const float4* t = reinterpret_cast<const float4*>(cs + 8 * (lo ? ci : ci - half));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 c = t[i];
      const float s0 = lo ? -c.y : c.y, s1 = lo ? -c.w : c.w;
      x[2 * i] = fmaf(x[2 * i], c.x, y[2 * i] * s0);
      x[2 * i + 1] = fmaf(x[2 * i + 1], c.z, y[2 * i + 1] * s1);
    }
  }
}

// Rows (token, head) of one set of heads, normed and rotated to fp16.
struct RopeRows {
  const void* x;
  int64_t x_stride;
  __half* out;
  int64_t out_stride;
  const float* weight;  // null: no norm
};

constexpr int kRopeTokens = 4;  // tokens per CTA at most

// Shared memory of rope_tokens: cosines, sines and negated sines of its tokens.
__host__ __device__ constexpr int rope_smem(int rotary_dim) {
  return kRopeTokens * 3 * (rotary_dim / 2) * 4;
}

// Head row `h` of tokens t0 .. t0+nt-1 (nt <= kRopeTokens): set A's hA heads
// followed by set B's hB.  Every thread of the CTA calls it; LPH = D/8
// consecutive threads share a row (h >= hA + hB: none); at least 64 threads.
//
// In the half layout a lane holds channels 4c .. 4c+3 and, where they are
// rotated, their partners r/2 further on, so that a rotation stays within a lane
// (two 8-byte accesses, each still whole sectors over the row); otherwise
// channels 8c .. 8c+7 (one 16-byte access).  Either way its pairs are
// 4c .. 4c+3.  The row's pointers and weights are set up once for all nt tokens,
// whose loads are issued together, and the arithmetic is packed two by two:
// after HBM it is the instructions that bound this (16384 tokens x 40 heads with
// norms, interleaved: 52.0 us, 0.95 of the copy rate, at 117 instructions per 16 bytes of input;
// half layout 56.0 with the whole head turned, 54.0 interleaved; with
// checks of rows and tokens 142 and 55.5 us, one row at a time 161 and 65 us).
template <int D, bool BF16, bool INTER, bool full>
__device__ __forceinline__ void rope_tokens_of(const RopeRows& A, int hA, const RopeRows& B, int hB,
                                               const int64_t* positions, int64_t t0, int nt, int h,
                                               float eps, const kvq_rope_plan& plan, float* smem) {
  constexpr int LPH = D / 8;
  const int r = plan.rotary_dim, rp = r >> 1;
  const int ci = threadIdx.x % LPH;
  const bool rot = 8 * ci < r;
  const int da = !INTER && rot ? 4 * ci : 8 * ci, db = !INTER && rot ? 4 * ci + rp : 8 * ci + 4;
  const bool act = full || h < hA + hB, b = act && h >= hA;
  const RopeRows& R = b ? B : A;
  const int64_t at = act ? (b ? h - hA : h) * D : 0;
  const __half* x = static_cast<const __half*>(R.x) + t0 * R.x_stride + at;
  const int64_t xs = R.x_stride, os = R.out_stride;
  uint32_t raw[kRopeTokens][4];
#pragma unroll
  for (int t = 0; t < kRopeTokens; ++t) {
    if (!full) raw[t][0] = raw[t][1] = raw[t][2] = raw[t][3] = 0;
    if (full || (act && t < nt)) {
      if constexpr (INTER) {
        const uint4 v = *reinterpret_cast<const uint4*>(x + t * xs + da);
        raw[t][0] = v.x;
        raw[t][1] = v.y;
        raw[t][2] = v.z;
        raw[t][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(x + t * xs + da);
        const uint2 u = *reinterpret_cast<const uint2*>(x + t * xs + db);
        raw[t][0] = v.x;
        raw[t][1] = v.y;
        raw[t][2] = u.x;
        raw[t][3] = u.y;
      }
    }
  }
  const bool norm = R.weight != nullptr;
  const bool warp_norm = __any_sync(0xffffffffu, norm);
  uint64_t w[4];
  if (warp_norm) {
    const float4 a = norm ? *reinterpret_cast<const float4*>(R.weight + da) : make_float4(1, 1, 1, 1);
    const float4 c = norm ? *reinterpret_cast<const float4*>(R.weight + db) : make_float4(1, 1, 1, 1);
    w[0] = f2_pack(a.x, a.y);
    w[1] = f2_pack(a.z, a.w);
    w[2] = f2_pack(c.x, c.y);
    w[3] = f2_pack(c.z, c.w);
  }
  float* cs = smem;  // [nt][3][rp]: cos, sin, -sin
  const int q = threadIdx.x % KVQ_ROPE_MAX_PAIRS;  // (a division by rp would cost more)
  if (q < rp)
    for (int t = threadIdx.x / KVQ_ROPE_MAX_PAIRS; t < (full ? kRopeTokens : nt);
         t += blockDim.x / KVQ_ROPE_MAX_PAIRS) {
      const float2 v = rope_cs(plan.turns[q], positions[t0 + t], plan.magnitude);
      cs[3 * t * rp + q] = v.x;
      cs[(3 * t + 1) * rp + q] = v.y;
      cs[(3 * t + 2) * rp + q] = -v.y;
    }
  __syncthreads();
  const float* my = cs + 4 * ci;
  __half* out = R.out + t0 * os + at;
#pragma unroll
  for (int t = 0; t < kRopeTokens; ++t) {
    if (!full && t >= nt) break;
    uint64_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16) {
        v[i] = f2_pack(__uint_as_float(raw[t][i] << 16), __uint_as_float(raw[t][i] & 0xFFFF0000u));
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&raw[t][i]));
        v[i] = f2_pack(f.x, f.y);
      }
    }
    if (warp_norm) {
      uint64_t q = f2_mul(v[0], v[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) q = f2_madd(v[i], v[i], q);
      float s, s1;
      f2_unpack(q, s, s1);
      s += s1;
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float f = norm ? rsqrtf(fmaf(s, 1.f / D, eps)) : 1.f;
      const uint64_t ff = f2_pack(f, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2_mul(v[i], f2_mul(w[i], ff));
    }
    if (rot) {
      const float* c = my + 3 * t * rp;
      const float4 cc = *reinterpret_cast<const float4*>(c);
      const float4 ss = *reinterpret_cast<const float4*>(c + rp);
      if constexpr (INTER) {
        const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a, d;
          f2_unpack(v[i], a, d);
          v[i] = f2_pack(fmaf(a, cv[i], -d * sv[i]), fmaf(a, sv[i], d * cv[i]));
        }
      } else {
        const float4 nn = *reinterpret_cast<const float4*>(c + 2 * rp);
        const uint64_t c2[2] = {f2_pack(cc.x, cc.y), f2_pack(cc.z, cc.w)};
        const uint64_t s2[2] = {f2_pack(ss.x, ss.y), f2_pack(ss.z, ss.w)};
        const uint64_t n2[2] = {f2_pack(nn.x, nn.y), f2_pack(nn.z, nn.w)};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t a = v[i], d = v[2 + i];
          v[i] = f2_madd(d, n2[i], f2_mul(a, c2[i]));
          v[2 + i] = f2_madd(a, s2[i], f2_mul(d, c2[i]));
        }
      }
    }
    if (act) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, d;
        f2_unpack(v[i], a, d);
        const __half2 hh = __floats2half2_rn(a, d);
        o[i] = *reinterpret_cast<const uint32_t*>(&hh);
      }
      if constexpr (INTER) {
        *reinterpret_cast<uint4*>(out + t * os + da) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        *reinterpret_cast<uint2*>(out + t * os + da) = make_uint2(o[0], o[1]);
        *reinterpret_cast<uint2*>(out + t * os + db) = make_uint2(o[2], o[3]);
      }
    }
  }
}

template <int D, bool BF16, bool INTER>
__device__ __forceinline__ void rope_tokens(const RopeRows& A, int hA, const RopeRows& B, int hB,
                                            const int64_t* positions, int64_t t0, int nt, int h,
                                            float eps, const kvq_rope_plan& plan, float* smem) {
  // a CTA whose tokens and rows are all there goes without the checks
  const int h_end = h - static_cast<int>(threadIdx.x) / (D / 8) + static_cast<int>(blockDim.x) / (D / 8);
  if (nt == kRopeTokens && h_end <= hA + hB)
    rope_tokens_of<D, BF16, INTER, true>(A, hA, B, hB, positions, t0, nt, h, eps, plan, smem);
  else
    rope_tokens_of<D, BF16, INTER, false>(A, hA, B, hB, positions, t0, nt, h, eps, plan, smem);
}

}  // namespace kvq
