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

constexpr int kRopeTokens = 4;

// Shared memory of rope_tokens: cosines and sines of its tokens, both sets' weights.
__host__ __device__ constexpr int rope_smem(int rotary_dim, int D) {
  return kRopeTokens * rotary_dim / 2 * 8 + 2 * D * 4;
}

// ceil(2^32 / h), h > 1: the high word of row * that is row / h for row * h < 2^32
// (here row < kRopeTokens * h + 2 * 32 and h <= 2^14).
inline uint32_t rope_inverse(int h) {
  return h > 1 ? static_cast<uint32_t>((0x100000000ull + h - 1) / h) : 0;
}

// Tokens t0 .. t0+nt-1 (nt <= kRopeTokens) of sets A (hA heads) and B (hB
// heads), every parts-th stretch of their rows; `inv` = rope_inverse(hA + hB).
//
// A pass of the CTA takes one row per D/8 lanes.  In the half layout a lane
// holds channels 4c .. 4c+3 and, where they are rotated, their partners r/2
// further on, so that a rotation stays within a lane (two 8-byte accesses, each
// still whole sectors over the row); otherwise channels 8c .. 8c+7 (one 16-byte
// access).  Either way its pairs are 4c .. 4c+3.
// The kernel that uses this is bound by its instructions as much as by HBM: a
// row's lane costs about 90 of them for its 32 bytes, so the row index is split
// by a multiplication, and the weights come from shared memory.
template <int D, int THREADS>
__device__ __forceinline__ void rope_tokens(const RopeRows& A, int hA, const RopeRows& B, int hB,
                                            uint32_t inv, bool bf16, const int64_t* positions,
                                            int64_t t0, int nt, int part, int parts, float eps,
                                            const kvq_rope_plan& plan, char* smem) {
  constexpr int LPH = D / 8, RPP = THREADS / LPH;  // lanes per head, rows per pass
  const int r = plan.rotary_dim, rp = r >> 1;
  float2* cs = reinterpret_cast<float2*>(smem);
  float* wsm = reinterpret_cast<float*>(cs + kRopeTokens * rp);
  for (int i = threadIdx.x; i < nt * rp; i += THREADS)
    cs[i] = rope_cs(plan.turns[i % rp], positions[t0 + i / rp], plan.magnitude);
  for (int i = threadIdx.x; i < 2 * D; i += THREADS) {
    const float* w = i < D ? A.weight : B.weight;
    wsm[i] = w != nullptr ? w[i % D] : 1.f;
  }
  const int ci = threadIdx.x % LPH, row0 = threadIdx.x / LPH;
  const bool inter = plan.layout == KVQ_ROPE_INTERLEAVED, rot = 8 * ci < r;
  const bool norm = A.weight != nullptr || B.weight != nullptr;
  const int da = !inter && rot ? 4 * ci : 8 * ci, db = !inter && rot ? 4 * ci + rp : 8 * ci + 4;
  const __half* xA = static_cast<const __half*>(A.x) + t0 * A.x_stride;
  const __half* xB = static_cast<const __half*>(B.x) + t0 * B.x_stride - hA * D;
  __half* oA = A.out + t0 * A.out_stride;
  __half* oB = B.out + t0 * B.out_stride - hA * D;
  __syncthreads();
  const int H = hA + hB, rows = nt * H;
  constexpr int U = 2;  // rows in flight per thread
  for (int base = part * RPP; base < rows; base += parts * RPP * U) {
    uint2 raw[U][2];
    int tok[U], head[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = base + u * parts * RPP + row0;
      tok[u] = H > 1 ? static_cast<int>(__umulhi(row, inv)) : row;
      head[u] = row - tok[u] * H;
      raw[u][0] = raw[u][1] = make_uint2(0, 0);
      if (row < rows) {
        const bool b = head[u] >= hA;
        const __half* x = (b ? xB : xA) + tok[u] * (b ? B.x_stride : A.x_stride) + head[u] * D;
        if (inter) {
          const uint4 v = *reinterpret_cast<const uint4*>(x + da);
          raw[u][0] = make_uint2(v.x, v.y);
          raw[u][1] = make_uint2(v.z, v.w);
        } else {
          raw[u][0] = *reinterpret_cast<const uint2*>(x + da);
          raw[u][1] = *reinterpret_cast<const uint2*>(x + db);
        }
      } else {
        tok[u] = -1;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool b = head[u] >= hA;
      float x[8];
      widen8(make_uint4(raw[u][0].x, raw[u][0].y, raw[u][1].x, raw[u][1].y), bf16, x);
      if (norm) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float f = (b ? B.weight : A.weight) != nullptr ? rsqrtf(fmaf(s, 1.f / D, eps)) : 1.f;
        const float4 wa = *reinterpret_cast<const float4*>(wsm + (b ? D : 0) + da);
        const float4 wb = *reinterpret_cast<const float4*>(wsm + (b ? D : 0) + db);
        x[0] *= f * wa.x;
        x[1] *= f * wa.y;
        x[2] *= f * wa.z;
        x[3] *= f * wa.w;
        x[4] *= f * wb.x;
        x[5] *= f * wb.y;
        x[6] *= f * wb.z;
        x[7] *= f * wb.w;
      }
      if (rot) {
        const float4* t = reinterpret_cast<const float4*>(cs + max(tok[u], 0) * rp + 4 * ci);
        const float4 c0 = t[0], c1 = t[1];
        const float c[4] = {c0.x, c0.z, c1.x, c1.z}, s[4] = {c0.y, c0.w, c1.y, c1.w};
        if (inter) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], d = x[2 * i + 1];
            x[2 * i] = fmaf(a, c[i], -d * s[i]);
            x[2 * i + 1] = fmaf(a, s[i], d * c[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[i], d = x[4 + i];
            x[i] = fmaf(a, c[i], -d * s[i]);
            x[4 + i] = fmaf(a, s[i], d * c[i]);
          }
        }
      }
      if (tok[u] >= 0) {
        __half* out = (b ? oB : oA) + tok[u] * (b ? B.out_stride : A.out_stride) + head[u] * D;
        const uint4 o = narrow8(x);
        if (inter) {
          *reinterpret_cast<uint4*>(out + da) = o;
        } else {
          *reinterpret_cast<uint2*>(out + da) = make_uint2(o.x, o.y);
          *reinterpret_cast<uint2*>(out + db) = make_uint2(o.z, o.w);
        }
      }
    }
  }
}

}  // namespace kvq
