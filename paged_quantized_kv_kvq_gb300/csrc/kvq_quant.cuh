// kvq_quant.cuh -- the quantizers of the append kernels: absmax of a 16-byte
// chunk, the INT8 / INT4 / FP8 codes of a value at a scale (IEEE division,
// round-half-even, saturating; a zero scale gives the zero code), and the
// nibble stores of INT4 words.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kvq_common.cuh"
#include "kvq_f32x2.cuh"

namespace kvq {

__device__ __forceinline__ float absmax8(const __half2 (&x)[4]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a = fmaxf(a, fabsf(__low2float(x[i])));
    a = fmaxf(a, fabsf(__high2float(x[i])));
  }
  return a;
}

// INT8 code, returned biased (c + 128) as stored in the pool.
__device__ __forceinline__ uint8_t quant_i8(float x, float s) {
  if (s == 0.f) return static_cast<uint8_t>(kInt8Bias);
  float q = rintf(__fdiv_rn(x, s));
  q = fminf(fmaxf(q, -127.f), 127.f);
  return static_cast<uint8_t>(static_cast<int>(q) + 128);
}

// INT4 code, returned biased (c + 8) as stored in the pool.
__device__ __forceinline__ uint32_t quant_i4(float x, float s) {
  if (s == 0.f) return kInt4Bias;
  float q = rintf(__fdiv_rn(x, s));
  q = fminf(fmaxf(q, -7.f), 7.f);
  return static_cast<uint32_t>(static_cast<int>(q) + 8);
}

// Replace the nibbles under `mask` of a shared 32-bit word: other tokens own
// the word's other nibbles and may be written by other CTAs at the same time.
__device__ __forceinline__ void store_nibbles(char* word, uint32_t mask, uint32_t val) {
  uint32_t* w = reinterpret_cast<uint32_t*>(word);
  atomicAnd(w, ~mask);
  atomicOr(w, val);
}

__device__ __forceinline__ uint8_t quant_e4m3(float x, float s) {
  if (s == 0.f) return 0;
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(__fdiv_rn(x, s), __NV_SATFINITE, __NV_E4M3));
}


// A scale's reciprocal for quant4_i8, or 0 where that is not to be used (a zero
// scale, or one whose reciprocal leaves fp32's normal range).
__device__ __forceinline__ float quant_inverse(float s) {
  return s > 1e-30f && s < 1e30f ? __fdividef(1.f, s) : 0.f;
}

// Largest magnitude of four values; NaN if one is NaN.
__device__ __forceinline__ float absmax4_nan(float a, float b, float c, float d) {
  float m, r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(d)));
  return r;
}

// Codes of x[0..3] (biased, packed in a word, x[0] lowest) at a scale s whose
// quant_inverse is inv > 0: the bits of quant_i8, unless `ok` is cleared.
// x * inv and the rounded x / s are within 2^-21 of each other relative (2^-22 from
// the reciprocal, a rounding each), 6.1e-5 for |x / s| <= 127.5, so the two round to
// the same integer unless x * inv lies that close to a half, i.e. unless its
// distance from the integer exceeds 0.49993; then, and for NaN, ok is cleared and
// the caller takes quant_i8.  (Adding 1.5 * 2^23 rounds half to even
// and leaves the integer in the low bits.  Five instructions a value; an IEEE
// division alone is twice that.)
__device__ __forceinline__ uint32_t quant4_i8(const float (&x)[4], float inv, bool& ok) {
  const uint64_t vi = f2_pack(inv, inv), big = f2_pack(12582912.f, 12582912.f),
                 neg = f2_pack(-1.f, -1.f);
  float m[4], t[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t r = f2_mul(f2_pack(x[2 * i], x[2 * i + 1]), vi);
    const uint64_t b = f2_add(r, big);
    const uint64_t d = f2_add(r, f2_madd(b, neg, big));  // r minus its integer
    f2_unpack(b, m[2 * i], m[2 * i + 1]);
    f2_unpack(d, t[2 * i], t[2 * i + 1]);
  }
  ok = ok && absmax4_nan(t[0], t[1], t[2], t[3]) < 0.49993f;
  return prmt(prmt(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0040u),
              prmt(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0040u), 0x5410u) ^
         0x80808080u;
}

}  // namespace kvq
