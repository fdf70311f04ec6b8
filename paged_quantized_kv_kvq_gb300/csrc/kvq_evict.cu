// kvq_evict.cu -- blocks with the least accumulated attention weight leave their
// sequences.
//
// A block's weight is the sum of its tokens' over the kv heads; the first `sink`
// and the last `recent` blocks stay, and of the others the heaviest, up to
// `budget` in all (ties: the lower index stays).  Nothing of the cache moves:
// the table row is permuted -- kept blocks in their order, then the evicted
// ones -- and the accumulators of the kept blocks are gathered behind it.
//
// One thread-block cluster per sequence.  Its CTAs share the reading (the one
// cost that grows with the context: 4 bytes per token and head, HBM or L2
// bound) and the gather; every CTA gets every block's key through distributed
// shared memory and makes the same selection, so that one cluster barrier
// orders everything.  The selection is a search for the budget-th largest key,
// one bit of the key per step.
//
// Sums.  Two blocks next to the border may differ in the last bits, and which
// of them stays must not depend on the order of a sum: each block's is carried
// as an fp32 pair (exact additions, good to 2^-44) and rounded to fp32 once, the
// same value that a sum in fp64 rounds to.  (fp64 itself runs at 1/64 of the
// fp32 rate here.)
#include <cooperative_groups.h>

#include <algorithm>

#include "kvq_context.h"
#include "kvq_internal.h"

namespace cg = cooperative_groups;

namespace kvq {

namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;

struct Pair {
  float hi, lo;
};

// a + b to twice fp32's precision (a, b normalised pairs); a sum that fp32 cannot
// hold stays what it is, an infinity or NaN.
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const float s = __fadd_rn(a.hi, b.hi);
  if (!isfinite(s)) return Pair{s, 0.f};
  const float t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
  const float l = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
  const float hi = __fadd_rn(s, l);
  return Pair{hi, __fsub_rn(l, __fsub_rn(hi, s))};
}

// Order of block weights as an unsigned key: larger weight, larger key; NaN
// counts as -inf, and -0 as 0.  The largest key is kept for blocks that stay.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) w = __int_as_float(0xff800000u);
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int block_sum(int v, int* red) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int i = 0; i < kEvictWarps; ++i) s += red[i];
  __syncthreads();
  return s;
}

// Sum of v over the threads before this one.
__device__ __forceinline__ int block_before(int v, int* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  int b = 0;
#pragma unroll
  for (int i = 0; i < kEvictWarps; ++i) b += i < warp ? red[i] : 0;
  __syncthreads();
  return b + x - v;
}

__global__ void __launch_bounds__(kEvictThreads) kvq_evict_kernel(const EvictArgs p, int cap) {
  extern __shared__ uint32_t smem[];
  int* red = reinterpret_cast<int*>(smem);               // [kEvictWarps]
  uint32_t* keys = smem + kEvictWarps;                   // [cap], later the table row
  int* perm = reinterpret_cast<int*>(keys + cap);        // [cap] kept blocks, then evicted ones
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
  const int s = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int L = p.lens[s];
  if (L > p.max_ctx) {
    if (rank == 0 && tid == 0) set_error(p.err, ERR_RANGE);
    L = p.max_ctx;
  }
  L = max(L, 0);
  const int bs = p.bs, n = (L + bs - 1) / bs;
  const int nkept = min(n, p.budget);
  const float* sc = p.scores + (int64_t)s * p.Hkv * p.stride;

  cluster.sync();  // every CTA's shared memory exists before anyone writes to it
  if (n > nkept) {
    // ---- weights of the blocks: lane = token (two tokens of a 64-token block)
    const int span = max(32, bs), width = min(bs, 32);
    for (int t0 = (rank * kEvictWarps + warp) * span; t0 < n * bs; t0 += ranks * kEvictWarps * span) {
      Pair a{0.f, 0.f};
      for (int t = t0 + lane; t < t0 + span; t += 32)
        if (t < L)
          for (int h = 0; h < p.Hkv; ++h) a = pair_add(a, Pair{sc[h * p.stride + t], 0.f});
      for (int o = width >> 1; o > 0; o >>= 1) {
        Pair b;
        b.hi = __shfl_xor_sync(0xffffffffu, a.hi, o);
        b.lo = __shfl_xor_sync(0xffffffffu, a.lo, o);
        // (the sum of a pair is the same from both sides)
        a = lane & o ? pair_add(b, a) : pair_add(a, b);
      }
      const int jb = (t0 + lane) / bs;
      if (lane % width == 0 && jb < n) {
        const uint32_t key = jb < p.sink || jb >= n - p.recent ? 0xffffffffu
                                                               : weight_key(__fadd_rn(a.hi, a.lo));
        for (int r = 0; r < ranks; ++r) cluster.map_shared_rank(keys, r)[jb] = key;
      }
    }
  }
  cluster.sync();

  // ---- the selection (every CTA the same): the largest T with at least
  // `budget` keys >= T; of the keys equal to T the first few stay
  if (n > nkept) {
    uint32_t T = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t c = T | 1u << bit;
      int v = 0;
      for (int j = tid; j < n; j += kEvictThreads) v += keys[j] >= c;
      if (block_sum(v, red) >= p.budget) T = c;
    }
    const int per = (n + kEvictThreads - 1) / kEvictThreads;
    const int j0 = min(tid * per, n), j1 = min(j0 + per, n);
    int above = 0, equal = 0;
    for (int j = j0; j < j1; ++j) {
      above += keys[j] > T;
      equal += keys[j] == T;
    }
    const int ties = p.budget - block_sum(above, red);  // of the keys equal to T
    int tie = block_before(equal, red);
    int pos = block_before(above + max(0, min(equal, ties - tie)), red);
    for (int j = j0; j < j1; ++j) {
      bool keep = keys[j] > T;
      if (keys[j] == T) keep = tie++ < ties;
      perm[keep ? pos : nkept + j - pos] = j;
      pos += keep;
    }
  } else {
    for (int j = tid; j < n; j += kEvictThreads) perm[j] = j;
  }
  __syncthreads();
  const int lens_new = L - (n - nkept) * bs;

  // ---- accumulators of the kept blocks, spread over the cluster
  if (p.scores_out != nullptr) {
    float* dst = p.scores_out + (int64_t)s * p.Hkv * p.out_stride;
    const int bl = 31 - __clz(bs);
    for (int h = warp + rank * kEvictWarps; h < p.Hkv * ((lens_new + 255) >> 8);
         h += ranks * kEvictWarps) {
      // a warp takes 256 tokens of one head
      const int hd = h % p.Hkv, base = h / p.Hkv << 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = base + 32 * i + lane;
        if (t < lens_new)
          dst[hd * p.out_stride + t] = sc[hd * p.stride + ((int64_t)perm[t >> bl] << bl) + (t & (bs - 1))];
      }
    }
  }
  // ---- the row, its length and the list (the row may be permuted in place)
  if (rank == 0) {
    const int* row = p.table + (int64_t)s * p.max_blocks;
    int* out = p.table_out + (int64_t)s * p.max_blocks;
    for (int j = tid; j < n; j += kEvictThreads) keys[j] = static_cast<uint32_t>(row[j]);
    __syncthreads();
    for (int j = tid; j < p.max_blocks; j += kEvictThreads)
      out[j] = j < n ? static_cast<int>(keys[perm[j]]) : row[j];
    if (p.kept != nullptr)
      for (int j = tid; j < p.budget; j += kEvictThreads)
        p.kept[(int64_t)s * p.budget + j] = j < nkept ? perm[j] : -1;
    if (tid == 0) p.lens_out[s] = lens_new;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  const int cap = (std::min(a.max_blocks, (a.max_ctx + a.bs - 1) / a.bs) + 3) / 4 * 4;
  const int smem = (kEvictWarps + std::max(cap, 4) * 2) * static_cast<int>(sizeof(uint32_t));
  // CTAs per sequence: as many as its longest possible row keeps busy
  const int64_t words = (int64_t)a.max_ctx * a.Hkv;
  const int ranks = words > 32768 ? 8 : words > 4096 ? 4 : 1;
  if ((int64_t)a.S * ranks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (smem > 40 * 1024) {
    const cudaError_t e = allow_big_smem<kvq_evict_kernel>();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.S * ranks));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return phase_mark(st, cudaLaunchKernelEx(&cfg, kvq_evict_kernel, a, std::max(cap, 4)));
}

}  // namespace kvq
