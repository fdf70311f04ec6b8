// kvq_quant.cuh -- the quantizers of the append kernels: absmax of a 16-byte
// chunk, the INT8 / INT4 / FP8 codes of a value at a scale (IEEE division,
// round-half-even, saturating; a zero scale gives the zero code), and the
// nibble stores of INT4 words.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kvq_common.cuh"

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

}  // namespace kvq
