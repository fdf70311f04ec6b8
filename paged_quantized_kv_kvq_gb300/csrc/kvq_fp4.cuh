// kvq_fp4.cuh -- 4-bit floats with a scale for every 16 channels (KVQ_FP4_E2M1):
// the scale's 8 bits, the code's 4, where they lie in a page, and their values as
// tensor-core fragments.
//
// A value of a (token, head, K|V) vector is code * scale.  Codes are e2m1: a sign,
// two exponent bits, one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6.  A scale has no
// sign, 5 exponent bits and 3 of mantissa -- the upper bits of an fp16 without its
// sign (fp16 bits = byte << 7), subnormals among them -- and is the group's absmax / 6
// rounded to nearest (even), at most 10240 so that 6 of it is an fp16 value.  A scale of
// fp16's range needs no second one for the tensor; 3 mantissa bits put the absmax
// within 1/16 of the largest code.  The product has 6 significant bits and fp16's range,
// so dequantized values are exact fp16 operands: no scale is left for the scores, the
// weights or the sums.  4.5 bits a value.
//
// Sub-tiles of 16 tokens hold one 32-bit word per lane and 16-channel step, at the
// place that INT4's words have (int4_word_offset): K word kk of lane 4g + j has
// channels 16kk + 4j .. +3 of tokens g and g + 8, V word mt tokens 2j, 2j+1, 2j+8, 2j+9
// of channels 16mt + g and 16mt + g + 8.  Each byte is the pair of one fragment register.
// The 16 * D/16 scale bytes of a sub-tile lie as the lanes want them: K's for
// token row g, then g + 8, side by side; V's in words of the four tokens of a lane.  A
// page is its K codes and their scales, then the same of V, so that either half is one
// copy.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "kvq_common.cuh"

namespace kvq {

// Bit of element (t, d) in its K (V) word, t in [0, 16).
__host__ __device__ inline int fp4_k_shift(int t, int d) { return (t >> 3) * 16 + (d & 3) * 4; }
__host__ __device__ inline int fp4_v_shift(int t, int d) {
  return (t >> 3) * 16 + ((d >> 3) & 1) * 8 + (t & 1) * 4;
}
// Byte of the scale of token t, channels 16gi .. +15 in a sub-tile's K (V) scales.
__host__ __device__ inline int fp4_k_scale(int t, int gi, int ng) {
  return (t & 7) * 2 * ng + (t >> 3) * ng + gi;
}
__host__ __device__ inline int fp4_v_scale(int t, int gi, int ng) {
  return ((t & 7) >> 1) * 4 * ng + gi * 4 + (t & 1) * 2 + (t >> 3);
}

// The scale's byte for a group whose largest magnitude is amax (not NaN).
__device__ __forceinline__ uint32_t fp4_scale_code(float amax) {
  const float y = fminf(__fdiv_rn(amax, 6.f), 10240.f);
  if (y < 6.103515625e-5f) return static_cast<uint32_t>(rintf(y * 131072.f));  // steps of 2^-17
  const uint32_t u = __float_as_uint(y);
  return ((u + 0x7FFFFu + (u >> 20 & 1u)) >> 20) - (112u << 3);
}
__device__ __forceinline__ float fp4_scale_value(uint32_t code) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(code << 7)));
}

// Codes of a (lower nibble) and b, both already divided by their scale: to nearest,
// ties to the even code, saturating at 6; NaN gives 6.
__device__ __forceinline__ uint32_t e2m1x2(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tmov.b32 %0, {c, 0, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b));
  return r;
}
// Codes of 8 values at scale s, x[0] in the lowest nibble; zeros where s is 0.
__device__ __forceinline__ uint32_t quant8_fp4(const float (&x)[8], float s) {
  if (s == 0.f) return 0;
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= e2m1x2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s)) << (8 * i);
  return r;
}
__device__ __forceinline__ float fp4_code_value(uint32_t code) {
  const uint32_t m = code & 7u;  // 0 and 0.5 are the subnormals
  const float v = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  return code & 8u ? -v : v;
}

// Store the codes of channels d0 .. d0+7 (packed as quant8_fp4 gives them) of token tt of
// a sub-tile.  K: a token's four channels of a word are 16 bits of their own.  V: a
// byte holds two tokens' codes, which other threads may be writing; OR alone where
// the word's other nibbles are known to be clear.
template <bool Clear>
__device__ __forceinline__ void store_fp4x8(char* tile, int kv, int tt, int d0, uint32_t codes) {
  if (kv == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = d0 + 4 * h;
      char* w = tile + int4_word_offset((tt & 7) * 4 + ((d & 15) >> 2), d >> 4);
      *reinterpret_cast<uint16_t*>(w + (tt >> 3) * 2) = static_cast<uint16_t>(codes >> (16 * h));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = d0 + i, sh = fp4_v_shift(tt, d);
      uint32_t* w = reinterpret_cast<uint32_t*>(
          tile + int4_word_offset((d & 7) * 4 + ((tt & 7) >> 1), d >> 4));
      if constexpr (!Clear) atomicAnd(w, ~(0xFu << sh));
      atomicOr(w, (codes >> (4 * i) & 0xFu) << sh);
    }
  }
}

// Eight codes -> the fp16 pairs of the word's bytes (exact).
__device__ __forceinline__ void e2m1x8_to_h2x4(uint32_t w, uint32_t (&p)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
      : "r"(w));
}
// Four scale bytes -> fp16 pairs (bytes 0, 2) and (1, 3).
__device__ __forceinline__ void fp4_scales(uint32_t w, __half2& even, __half2& odd) {
  const uint32_t e = w << 7 & 0x7F807F80u, o = w >> 1 & 0x7F807F80u;
  even = *reinterpret_cast<const __half2*>(&e);
  odd = *reinterpret_cast<const __half2*>(&o);
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, __half2 s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), s);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A word's values as fragment registers: K with the scales of rows g and g + 8 (a0, a2
// of row g; a1, a3 of row g + 8), V with those of token pairs (2j, 2j+1) and
// (2j+8, 2j+9) (a0, a1; a2, a3).
__device__ __forceinline__ void fp4_k_frag(uint32_t w, __half2 sg, __half2 sg8, uint32_t (&a)[4]) {
  uint32_t p[4];
  e2m1x8_to_h2x4(w, p);
  a[0] = h2_mul(p[0], sg);
  a[2] = h2_mul(p[1], sg);
  a[1] = h2_mul(p[2], sg8);
  a[3] = h2_mul(p[3], sg8);
}
__device__ __forceinline__ void fp4_v_frag(uint32_t w, __half2 lo, __half2 hi, uint32_t (&a)[4]) {
  uint32_t p[4];
  e2m1x8_to_h2x4(w, p);
  a[0] = h2_mul(p[0], lo);
  a[1] = h2_mul(p[1], lo);
  a[2] = h2_mul(p[2], hi);
  a[3] = h2_mul(p[3], hi);
}

// Mask of a V scale word's bytes whose tokens 2j, 2j+1, 2j+8, 2j+9 are below `rows`: the
// scales of tokens that were never written may be infinities or NaN.
__device__ __forceinline__ uint32_t fp4_v_mask(int j, int rows) {
  return (2 * j < rows ? 0xFFu : 0u) | (2 * j + 8 < rows ? 0xFF00u : 0u) |
         (2 * j + 1 < rows ? 0xFF0000u : 0u) | (2 * j + 9 < rows ? 0xFF000000u : 0u);
}

// A lane's share of a K (V) sub-tile as fp16 words in the order that FP16 sub-tiles have
// them (D/4 words).  `sc`: the sub-tile's scales.  V tokens at or past `rows` are zeros.
template <int D>
__device__ __forceinline__ void fp4_load_k(const char* tile, const char* sc, int lane,
                                           uint32_t* words) {
  constexpr int NG = D / 16;
  const int g = lane >> 2;
#pragma unroll
  for (int c = 0; c < NG / 4; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(tile + c * 512 + lane * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    __half2 s[2][2];
    fp4_scales(*reinterpret_cast<const uint32_t*>(sc + g * 2 * NG + 4 * c), s[0][0], s[0][1]);
    fp4_scales(*reinterpret_cast<const uint32_t*>(sc + g * 2 * NG + NG + 4 * c), s[1][0], s[1][1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int kk = 4 * c + i;
      uint32_t a[4];
      const __half2 x = s[0][i & 1], y = s[1][i & 1];
      fp4_k_frag(w[i], i & 2 ? __high2half2(x) : __low2half2(x),
                 i & 2 ? __high2half2(y) : __low2half2(y), a);
      words[2 * kk] = a[0];
      words[2 * kk + 1] = a[2];
      words[2 * (NG + kk)] = a[1];
      words[2 * (NG + kk) + 1] = a[3];
    }
  }
}
template <int D>
__device__ __forceinline__ void fp4_load_v(const char* tile, const char* sc, int lane, int rows,
                                           uint32_t* words) {
  constexpr int NG = D / 16;
  const int j = lane & 3;
  const uint32_t mask = fp4_v_mask(j, rows);
#pragma unroll
  for (int c = 0; c < NG / 4; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(tile + c * 512 + lane * 16);
    const uint4 q = *reinterpret_cast<const uint4*>(sc + j * 4 * NG + 16 * c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w}, sw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int mt = 4 * c + i;
      __half2 lo, hi;
      fp4_scales(sw[i] & mask, lo, hi);
      uint32_t a[4];
      fp4_v_frag(w[i], lo, hi, a);
      words[4 * mt] = a[0];
      words[4 * mt + 1] = a[2];
      words[4 * mt + 2] = a[1];
      words[4 * mt + 3] = a[3];
    }
  }
}

}  // namespace kvq
