// kvq_fp4_rows.cu -- long appends to pools of 4-bit floats, and their read-back as fp16.
//
// A warp takes 16 consecutive tokens of the call and one head's K or V (two heads of 64
// channels).  Lane 4 gi + j has the 16 channels of scale group gi of the tokens 2j, 2j+1,
// 2j+8 and 2j+9 of a sub-tile: the ones that share its V words, and both tokens of two
// rows of its K words.  So a group's absmax, scale and 16 codes are one lane's, and every
// 32-bit word of the page is complete in one lane: no shuffle, no shared tile, two byte
// permutes a word.
//
// Tokens come in runs: neighbours of the call whose slots follow each other inside one
// sub-tile.  A run belongs to the warp in whose 16 tokens it begins, with all of its
// tokens, so that a prompt that starts inside a block still fills whole sub-tiles.  Runs of
// kRows4Run tokens or more are taken one after the other, the tokens of shorter ones (a
// decode step's) all at once, a lane then holding four tokens of any slots.  A word that
// a run does not fill is merged into the page (V nibbles by atomics: other warps may
// hold its other tokens).
// Bound: HBM (4 bytes a channel in, 1.125 out, for K and V together), the instructions (760 of
// a warp for its 16 tokens, counted) and the wait for the slots, then the rows: issue slots
// 46% busy from a cold cache, DRAM 40%.  Measured, 16384 tokens x 8 heads of 128: whole
// blocks 16.9 us replayed (86 MB, part of which the L2 keeps between replays; 21.9 from a
// cold cache, 0.58 of the copy rate), from inside a block 17.1, single tokens 76; read
// back 17.2, 18.2 and 47.  (Sub-tile by sub-tile of the 16 tokens instead of runs: 16.6 us
// for whole blocks, but 32 from inside a block and 235 for single tokens.)
#include "kvq_context.h"
#include "kvq_f32x2.cuh"
#include "kvq_fp4.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kRows4Threads = 128;
constexpr int kRows4Warps = kRows4Threads / 32;

// Codes of 16 fp16 values at the scale whose reciprocal is inv (0 for a zero scale): the
// bits of quant8_fp4.  A quotient x / s of an 11-bit x and a 4-bit s is either a border
// between codes (0.25, 0.75, .. 5) or at least 1/2047 of it away: with x = X 2^a, s = S 2^b,
// border T 2^c (T in 1, 3, 5, 7) the difference X 2^a - T S 2^(b+c) is 0 or a multiple of
// the smaller power.  That is 2^-13 or more, so rounding x * inv (within 2^-21 of itself)
// to a multiple of 2^-13 -- what adding and taking away 1536 does -- lands on the border
// or stays on its side of it.  The sign is x's, also of what rounds to zero.
__device__ __forceinline__ uint2 quant16_fp4(const uint4 (&raw)[2], float inv) {
  const uint64_t vi = f2_pack(inv, inv), up = f2_pack(1536.f, 1536.f), down = f2_pack(-1536.f, -1536.f);
  const uint32_t h[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    float q0, q1;
    f2_unpack(f2_add(f2_madd(f2_pack(x.x, x.y), vi, up), down), q0, q1);
    q0 = __uint_as_float((__float_as_uint(q0) & ~0x80000000u) | (__float_as_uint(x.x) & 0x80000000u));
    q1 = __uint_as_float((__float_as_uint(q1) & ~0x80000000u) | (__float_as_uint(x.y) & 0x80000000u));
    b[i] = e2m1x2(q0, q1);
  }
  if (inv == 0.f) return make_uint2(0, 0);
  return make_uint2(prmt(prmt(b[0], b[1], 0x0040u), prmt(b[2], b[3], 0x0040u), 0x5410u),
                    prmt(prmt(b[4], b[5], 0x0040u), prmt(b[6], b[7], 0x0040u), 0x5410u));
}

// fp4_scale_code of an fp16 value without the division: the same argument with 6 for s and
// the middle between two scales (5 bits) for the border holds amax / 6 off every middle
// that it is not by 1/2047 of itself, so amax * (1/6) rounded to 14 mantissa bits is on the
// same side of it or on it.  (Below 2^-14 middles are multiples of 2^-18, which that leaves
// exact, too.)
__device__ __forceinline__ uint32_t scale_code16(float amax) {
  const uint32_t y = __float_as_uint(fminf(amax * 0.16666667f, 10240.f)), u = (y + 0x100u) & ~0x1FFu;
  const uint32_t sub = __float2uint_rn(__uint_as_float(u) * 131072.f);  // steps of 2^-17
  return u < 0x38800000u ? sub : ((u + 0x7FFFFu + (u >> 20 & 1u)) >> 20) - (112u << 3);
}

__device__ __forceinline__ float absmax16(const uint4 (&raw)[2]) {
  const uint32_t h[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
  __half2 m = __half2half2(__ushort_as_half(0));
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&h[i])));
  return fmaxf(__low2float(m), __high2float(m));  // (NaN loses every comparison)
}

// Bytes i of four words as word i.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&o)[4]) {
  const uint32_t ab0 = prmt(a, b, 0x5140u), ab1 = prmt(a, b, 0x7362u);  // a0 b0 a1 b1 | a2 b2 a3 b3
  const uint32_t cd0 = prmt(c, d, 0x5140u), cd1 = prmt(c, d, 0x7362u);
  o[0] = prmt(ab0, cd0, 0x5410u);
  o[1] = prmt(ab0, cd0, 0x7632u);
  o[2] = prmt(ab1, cd1, 0x5410u);
  o[3] = prmt(ab1, cd1, 0x7632u);
}

// Nibble c of t0 and t1 side by side: bytes 0, 2, 4, 6 in `even`, 1, 3, 5, 7 in `odd`.
__device__ __forceinline__ void interleave(uint32_t t0, uint32_t t1, uint32_t& even, uint32_t& odd) {
  even = (t0 & 0x0F0F0F0Fu) | (t1 << 4 & 0xF0F0F0F0u);
  odd = (t0 >> 4 & 0x0F0F0F0Fu) | (t1 & 0xF0F0F0F0u);
}

// The runs that begin among a warp's 16 tokens: lane l has the call's token i0 + l.
struct Runs {
  int64_t slot;       // of the lane's token; negative: none
  uint32_t follows;   // tokens that continue the run of the one before
  uint32_t leaders;   // tokens (of the first 16) that begin a run

  __device__ __forceinline__ Runs(const int64_t* slots, int64_t i0, int64_t T, int64_t limit, int* err) {
    const int lane = threadIdx.x & 31;
    slot = i0 + lane < T ? slots[i0 + lane] : -1;
    const int64_t before = lane == 0 && i0 > 0 ? slots[i0 - 1] : -1;
    if (slot >= limit) {
      set_error(err, ERR_RANGE);
      slot = -1;
    }
    int64_t prev = __shfl_up_sync(0xffffffffu, slot, 1);
    if (lane == 0) prev = before < limit ? before : -1;
    const bool cont = slot >= 0 && slot == prev + 1 && (slot & 15) != 0;
    follows = __ballot_sync(0xffffffffu, cont);
    leaders = __ballot_sync(0xffffffffu, slot >= 0 && !cont) & 0xFFFFu;
  }
  __device__ __forceinline__ int length(int l) const {  // of the run that token l < 16 begins
    return __ffs(~(follows >> (l + 1)));
  }
};

constexpr int kRows4Run = 4;

// Calls take(first slot, idx) for the runs: lane quarter j's token idx[c] (of the call's from
// i0 on; -1: none) at place 2j + (c & 1) + 8 (c >> 1) of the sub-tile; and each(slot, idx)
// with four tokens of any slots.
template <class Take, class Each>
__device__ __forceinline__ void for_runs(const Runs& r, int j, Take&& take, Each&& each) {
  uint32_t shorts = 0;
  for (uint32_t todo = r.leaders; todo != 0; todo &= todo - 1) {
    const int l = __ffs(todo) - 1, n = r.length(l);
    if (n < kRows4Run) {
      shorts |= ((1u << n) - 1) << l;
      continue;
    }
    const int64_t first = __shfl_sync(0xffffffffu, r.slot, l);
    const int t0 = static_cast<int>(first & 15);
    int idx[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int k = 2 * j + (c & 1) + 8 * (c >> 1) - t0;
      idx[c] = k >= 0 && k < n ? l + k : -1;
    }
    take(first, idx);
  }
  for (int b = 0; b < 32; b += 16) {
    if ((shorts >> b & 0xFFFFu) == 0) continue;
    int idx[4];
    int64_t slot[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int l = b + 4 * c + j;
      slot[c] = __shfl_sync(0xffffffffu, r.slot, l);
      idx[c] = shorts >> l & 1 ? l : -1;
    }
    each(slot, idx);
  }
}

// Where a warp's lanes stand: scale group gi of head h, K or V, quarter j of the tokens.
template <int D>
struct Rows4Lane {
  static constexpr int NG = D / 16, HPW = 8 / NG;  // heads per warp
  int kv, h, gi, j;
  bool unit, act;

  __device__ __forceinline__ Rows4Lane(int Hkv) {
    const int lane = threadIdx.x & 31, hu = (Hkv + HPW - 1) / HPW;  // units of K (of V)
    const int u = blockIdx.y * kRows4Warps + (threadIdx.x >> 5);
    unit = u < 2 * hu;
    kv = u >= hu;
    h = (u - kv * hu) * HPW + (HPW == 2 ? lane >> 4 : 0);
    gi = (lane >> 2) & (NG - 1);
    j = lane & 3;
    act = unit && h < Hkv;
  }
};

// K (V) half of the page of a slot, from the first byte of its sub-tile's codes (16-byte
// chunk and word of the group) and of its scales.
template <int D>
__device__ __forceinline__ char* half_of(const PoolView& pool, int64_t slot, int bs_log2, int h, int kv) {
  return pool.pages + ((slot >> bs_log2) * pool.Hkv + h) * pool.page_bytes + (kv ? pool.v_off : 0);
}
template <int D>
__device__ __forceinline__ int codes_at(const PoolView& pool, int64_t slot, int gi) {
  return static_cast<int>(slot & (pool.bs - 1)) / 16 * pool.sub_bytes + (gi >> 2) * 512 + (gi & 3) * 4;
}
template <int D>
__device__ __forceinline__ int scales_at(const PoolView& pool, int64_t slot) {
  return pool.code_bytes + static_cast<int>(slot & (pool.bs - 1)) / 16 * D;
}

template <int D>
__global__ void __launch_bounds__(kRows4Threads) kvq_append4_kernel(PoolView pool, const __half* k, const __half* v,
                                                                    int64_t stride, const int64_t* slots, int64_t T,
                                                                    int bs_log2) {
  constexpr int NG = D / 16;
  const Rows4Lane<D> me(pool.Hkv);
  if (!me.unit) return;
  const int gi = me.gi, j = me.j, kv = me.kv, h = me.h;
  const int64_t i0 = (int64_t)blockIdx.x * 16;
  const Runs runs(slots, i0, T, pool.num_blocks << bs_log2, pool.err);
  const __half* x = (kv ? v : k) + i0 * stride + h * D + 16 * gi;
  uint32_t lo[4], hi[4], sc[4];  // codes of channels 0 .. 7, 8 .. 15 of the group, scales
  auto quantize = [&](const int (&idx)[4]) {
    uint4 raw[4][2];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4* at = reinterpret_cast<const uint4*>(x + idx[c] * stride);
      raw[c][0] = me.act && idx[c] >= 0 ? at[0] : make_uint4(0, 0, 0, 0);
      raw[c][1] = me.act && idx[c] >= 0 ? at[1] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      sc[c] = scale_code16(absmax16(raw[c]));
      const float s = fp4_scale_value(sc[c]);
      const uint2 q = quant16_fp4(raw[c], s != 0.f ? __fdividef(1.f, s) : 0.f);
      lo[c] = q.x;
      hi[c] = q.y;
    }
  };
  for_runs(
      runs, j,
      [&](int64_t first, const int (&idx)[4]) {
        quantize(idx);
        if (!me.act) return;
        const bool whole = idx[0] >= 0 && idx[1] >= 0 && idx[2] >= 0 && idx[3] >= 0;
        char* half = half_of<D>(pool, first, bs_log2, h, kv);
        char* codes = half + codes_at<D>(pool, first, gi);
        char* scales = half + scales_at<D>(pool, first);
        if (kv == 0) {
          // rows 2j + p (tokens c = p and p + 2), channels 4q .. 4q+3: a word each
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t word = prmt(q < 2 ? lo[p] : hi[p], q < 2 ? lo[p + 2] : hi[p + 2], q & 1 ? 0x7632u : 0x5410u);
              char* to = codes + j * 128 + (p * 4 + q) * 16;
              if (whole) {
                *reinterpret_cast<uint32_t*>(to) = word;
              } else {
                if (idx[p] >= 0) *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(word);
                if (idx[p + 2] >= 0) *reinterpret_cast<uint16_t*>(to + 2) = static_cast<uint16_t>(word >> 16);
              }
            }
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (idx[c] >= 0) scales[fp4_k_scale(2 * j + (c & 1) + 8 * (c >> 1), gi, NG)] = static_cast<char>(sc[c]);
        } else {
          // channel c of the group's lower (bytes 0, 2) and upper (1, 3) eight: a word each
          uint32_t e[4], o[4], word[2][4];
          interleave(lo[0], lo[1], e[0], o[0]);
          interleave(hi[0], hi[1], e[1], o[1]);
          interleave(lo[2], lo[3], e[2], o[2]);
          interleave(hi[2], hi[3], e[3], o[3]);
          transpose4(e[0], e[1], e[2], e[3], word[0]);
          transpose4(o[0], o[1], o[2], o[3], word[1]);
          const uint32_t mask = (idx[0] >= 0 ? 0x00000F0Fu : 0u) | (idx[1] >= 0 ? 0x0000F0F0u : 0u) |
                                (idx[2] >= 0 ? 0x0F0F0000u : 0u) | (idx[3] >= 0 ? 0xF0F00000u : 0u);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t* to = reinterpret_cast<uint32_t*>(codes + (c * 4 + j) * 16);
            const uint32_t wd = word[c & 1][c >> 1];
            if (whole) {
              *to = wd;
            } else if (mask != 0) {
              atomicAnd(to, ~mask);
              atomicOr(to, wd & mask);
            }
          }
          char* at = scales + fp4_v_scale(2 * j, gi, NG);
          if (whole) {
            *reinterpret_cast<uint32_t*>(at) = sc[0] | sc[2] << 8 | sc[1] << 16 | sc[3] << 24;
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (idx[c] >= 0) at[(c & 1) * 2 + (c >> 1)] = static_cast<char>(sc[c]);
          }
        }
      },
      [&](const int64_t (&slot)[4], const int (&idx)[4]) {
        quantize(idx);
        if (!me.act) return;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (idx[c] < 0) continue;
          const int tt = static_cast<int>(slot[c] & 15);
          char* half = half_of<D>(pool, slot[c], bs_log2, h, kv);
          char* codes = half + codes_at<D>(pool, slot[c], gi);
          char* scales = half + scales_at<D>(pool, slot[c]);
          if (kv == 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint16_t*>(codes + ((tt & 7) * 4 + q) * 16 + (tt >> 3) * 2) =
                  static_cast<uint16_t>((q < 2 ? lo[c] : hi[c]) >> 16 * (q & 1));
            scales[fp4_k_scale(tt, gi, NG)] = static_cast<char>(sc[c]);
          } else {
            const int sh = fp4_v_shift(tt, 0);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              uint32_t* to = reinterpret_cast<uint32_t*>(codes + (q * 4 + ((tt & 7) >> 1)) * 16);
              atomicAnd(to, ~(0x0F0Fu << sh));
              atomicOr(to, ((lo[c] >> 4 * q & 0xFu) | (hi[c] >> 4 * q & 0xFu) << 8) << sh);
            }
            scales[fp4_v_scale(tt, gi, NG)] = static_cast<char>(sc[c]);
          }
        }
      });
}

// Four tokens' 16 channels from the words of their sub-tiles, as fp16 rows.
__device__ __forceinline__ void put16(__half* out, const uint32_t (&y)[8], __half2 s) {
  uint4* to = reinterpret_cast<uint4*>(out);
  to[0] = make_uint4(h2_mul(y[0], s), h2_mul(y[1], s), h2_mul(y[2], s), h2_mul(y[3], s));
  to[1] = make_uint4(h2_mul(y[4], s), h2_mul(y[5], s), h2_mul(y[6], s), h2_mul(y[7], s));
}
__device__ __forceinline__ __half2 scale2(char byte) {
  return __half2half2(__ushort_as_half(static_cast<unsigned short>(static_cast<uint8_t>(byte) << 7)));
}

template <int D>
__global__ void __launch_bounds__(kRows4Threads) kvq_read_values4_kernel(PoolView pool, const int64_t* slots, int64_t T,
                                                                         __half* k, __half* v, int bs_log2) {
  constexpr int NG = D / 16;
  const Rows4Lane<D> me(pool.Hkv);
  if (!me.unit) return;
  const int gi = me.gi, j = me.j, kv = me.kv, h = me.h;
  const int64_t i0 = (int64_t)blockIdx.x * 16, row = (int64_t)pool.Hkv * D;
  const Runs runs(slots, i0, T, pool.num_blocks << bs_log2, pool.err);
  __half* out = (kv ? v : k) + i0 * row + h * D + 16 * gi;
  for_runs(
      runs, j,
      [&](int64_t first, const int (&idx)[4]) {
        if (!me.act) return;
        const char* half = half_of<D>(pool, first, bs_log2, h, kv);
        const char* codes = half + codes_at<D>(pool, first, gi);
        const char* scales = half + scales_at<D>(pool, first);
        uint32_t wd[8], y[4][8];  // channel pairs of the four tokens
        __half2 s[4];
        if (kv == 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) wd[i] = *reinterpret_cast<const uint32_t*>(codes + j * 128 + i * 16);
#pragma unroll
          for (int c = 0; c < 4; ++c) s[c] = scale2(scales[fp4_k_scale(2 * j + (c & 1) + 8 * (c >> 1), gi, NG)]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // row 2j + (i >> 2): tokens (i >> 2) and (i >> 2) + 2
            uint32_t p[4];
            e2m1x8_to_h2x4(wd[i], p);
            y[i >> 2][2 * (i & 3)] = p[0];
            y[i >> 2][2 * (i & 3) + 1] = p[1];
            y[(i >> 2) + 2][2 * (i & 3)] = p[2];
            y[(i >> 2) + 2][2 * (i & 3) + 1] = p[3];
          }
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) wd[c] = *reinterpret_cast<const uint32_t*>(codes + (c * 4 + j) * 16);
          __half2 a, b;  // tokens 2j, 2j+1 | 2j+8, 2j+9
          fp4_scales(*reinterpret_cast<const uint32_t*>(scales + fp4_v_scale(2 * j, gi, NG)), a, b);
          s[0] = __low2half2(a);
          s[1] = __high2half2(a);
          s[2] = __low2half2(b);
          s[3] = __high2half2(b);
          // channels 2q, 2q+1 of the lower and the upper eight
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t e[4], o[4];
            e2m1x8_to_h2x4(wd[2 * q], e);
            e2m1x8_to_h2x4(wd[2 * q + 1], o);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int u = 0; u < 2; ++u)
                y[c][q + 4 * u] = prmt(e[(c & 2) + u], o[(c & 2) + u], c & 1 ? 0x7632u : 0x5410u);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (idx[c] >= 0) put16(out + idx[c] * row, y[c], s[c]);
      },
      [&](const int64_t (&slot)[4], const int (&idx)[4]) {
        if (!me.act) return;
        uint32_t lo[4], hi[4];  // the codes of channels 0 .. 7, 8 .. 15
        __half2 s[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (idx[c] < 0) continue;
          const int tt = static_cast<int>(slot[c] & 15);
          const char* half = half_of<D>(pool, slot[c], bs_log2, h, kv);
          const char* codes = half + codes_at<D>(pool, slot[c], gi);
          const char* scales = half + scales_at<D>(pool, slot[c]);
          s[c] = scale2(scales[kv == 0 ? fp4_k_scale(tt, gi, NG) : fp4_v_scale(tt, gi, NG)]);
          if (kv == 0) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = *reinterpret_cast<const uint16_t*>(codes + ((tt & 7) * 4 + q) * 16 + (tt >> 3) * 2);
            lo[c] = w[0] | w[1] << 16;
            hi[c] = w[2] | w[3] << 16;
          } else {
            const int sh = fp4_v_shift(tt, 0);
            lo[c] = hi[c] = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + (q * 4 + ((tt & 7) >> 1)) * 16) >> sh;
              lo[c] |= (w & 0xFu) << 4 * q;
              hi[c] |= (w >> 8 & 0xFu) << 4 * q;
            }
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (idx[c] < 0) continue;
          uint32_t a[4], b[4];
          e2m1x8_to_h2x4(lo[c], a);
          e2m1x8_to_h2x4(hi[c], b);
          const uint32_t y[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
          put16(out + idx[c] * row, y, s[c]);
        }
      });
}

struct Rows4Grid {
  dim3 grid;
  int bs_log2 = 0;
  bool ok;
};

Rows4Grid rows4_grid(const PoolView& pool, int64_t n) {
  Rows4Grid g;
  const int hpw = pool.D == 64 ? 2 : 1;
  const int64_t gx = (n + 15) / 16, gy = (2 * ((pool.Hkv + hpw - 1) / hpw) + kRows4Warps - 1) / kRows4Warps;
  g.ok = gx <= 0x7fffffffLL && gy <= 65535;
  if (g.ok) g.grid = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  while ((1 << g.bs_log2) < pool.bs) ++g.bs_log2;
  return g;
}

}  // namespace

cudaError_t launch_append4(const PoolView& pool, const __half* k, const __half* v, int64_t stride,
                           const int64_t* slots, int64_t T, cudaStream_t st) {
  const Rows4Grid g = rows4_grid(pool, T);
  if (!g.ok) return cudaErrorInvalidValue;
  if (pool.D == 64)
    kvq_append4_kernel<64><<<g.grid, kRows4Threads, 0, st>>>(pool, k, v, stride, slots, T, g.bs_log2);
  else
    kvq_append4_kernel<128><<<g.grid, kRows4Threads, 0, st>>>(pool, k, v, stride, slots, T, g.bs_log2);
  return phase_mark(st, cudaGetLastError());
}

cudaError_t launch_read_values4(const PoolView& pool, const int64_t* slots, int64_t n, __half* k, __half* v,
                                cudaStream_t st) {
  const Rows4Grid g = rows4_grid(pool, n);
  if (!g.ok) return cudaErrorInvalidValue;
  if (pool.D == 64)
    kvq_read_values4_kernel<64><<<g.grid, kRows4Threads, 0, st>>>(pool, slots, n, k, v, g.bs_log2);
  else
    kvq_read_values4_kernel<128><<<g.grid, kRows4Threads, 0, st>>>(pool, slots, n, k, v, g.bs_log2);
  return phase_mark(st, cudaGetLastError());
}

}  // namespace kvq
