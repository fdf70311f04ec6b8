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
// fraction; pos times it, modulo 2^64, is the position's fraction of a turn,
// exact but for the 2^-65 of f_i itself (2^-34 of a turn at position 2^31),
// where an fp32 angle at position 10^5 would be off by 2^-8.  Its top 32 bits,
// taken as signed, give an angle in [-pi, pi) within 2^-23, and there the
// hardware's sine and cosine are good to 2^-21: both sit far below the
// rounding of what is stored (fp16, 2^-11, or 8-bit codes).  No table of
// positions is read, so there is no longest position and no cache traffic.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq.h"

namespace kvq {

// cos and sin (times the plan's magnitude) of `pos` at `turn` turns per position.
__device__ __forceinline__ float2 rope_cs(uint64_t turn, int64_t pos, float magnitude) {
  const uint64_t frac = turn * static_cast<uint64_t>(pos);
  const float a = static_cast<float>(static_cast<int32_t>(frac >> 32)) * 1.4629180792671596e-9f;
  float s, c;
  __sincosf(a, &s, &c);  // a = 2 pi * fraction of a turn
  return make_float2(c * magnitude, s * magnitude);
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
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float r = rsqrtf(fmaf(s, 1.f / D, eps));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
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

// Tokens t0 .. t0+nt-1 (nt <= kRopeTokens) of sets A (hA heads) and B (hB
// heads), head rows `part`, part + parts, ... of each; `cs` is shared memory for
// nt * r/2 pairs.
constexpr int kRopeTokens = 4;

template <int D, int THREADS>
__device__ __forceinline__ void rope_tokens(const RopeRows& A, int hA, const RopeRows& B, int hB,
                                            bool bf16, const int64_t* positions, int64_t t0, int nt,
                                            int part, int parts, float eps,
                                            const kvq_rope_plan& plan, float2* cs) {
  constexpr int LPH = D / 8, RPP = THREADS / LPH;  // lanes per head, rows per pass
  const int r = plan.rotary_dim, rp = r >> 1;
  for (int i = threadIdx.x; i < nt * rp; i += THREADS)
    cs[i] = rope_cs(plan.turns[i % rp], positions[t0 + i / rp], plan.magnitude);
  const int ci = threadIdx.x % LPH, row0 = threadIdx.x / LPH;
  float wA[8], wB[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wA[i] = A.weight != nullptr ? A.weight[8 * ci + i] : 1.f;
    wB[i] = B.weight != nullptr ? B.weight[8 * ci + i] : 1.f;
  }
  __syncthreads();
  const int H = hA + hB, rows = nt * H;
  constexpr int U = 2;  // rows in flight per thread
  for (int base = part * RPP; base < rows; base += parts * RPP * U) {
    uint4 raw[U];
    int tok[U], head[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = base + u * parts * RPP + row0;
      tok[u] = row < rows ? row / H : -1;
      head[u] = row - (row / H) * H;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (tok[u] >= 0) {
        const bool b = head[u] >= hA;
        const RopeRows& R = b ? B : A;
        raw[u] = *reinterpret_cast<const uint4*>(
            static_cast<const __half*>(R.x) + (t0 + tok[u]) * R.x_stride +
            (b ? head[u] - hA : head[u]) * D + 8 * ci);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool b = head[u] >= hA;
      const RopeRows& R = b ? B : A;
      float x[8], w[8];
      widen8(raw[u], bf16, x);
      // a row's lanes agree on its set; a warp may hold rows of both, so all of
      // its lanes reduce and only those with a weight take the result
      if (A.weight != nullptr || B.weight != nullptr) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = x[i];
          w[i] = b ? wB[i] : wA[i];
        }
        norm8<D>(y, w, eps);
        if (R.weight != nullptr)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = y[i];
      }
      if (r > 0) rotate8<D>(x, ci, r, plan.layout == KVQ_ROPE_INTERLEAVED, cs + max(tok[u], 0) * rp);
      if (tok[u] >= 0)
        *reinterpret_cast<uint4*>(R.out + (t0 + tok[u]) * R.out_stride +
                                  (b ? head[u] - hA : head[u]) * D + 8 * ci) = narrow8(x);
    }
  }
}

}  // namespace kvq
