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
// orders everything.  The selection halves the interval of keys until exactly
// `budget` of them lie above (or ties are all that is left): some 15 counts for
// weights as attention gives them, 32 at most.  A short row costs one launch and
// a chain of such steps; the reading loads eight heads of two tokens at once, so
// that a long row is not a chain of round trips.  Measured: 16 rows of up to 1000
// tokens 7.1 us, 8 rows of 32768 tokens x 8 heads 14.2 us (12.8 with clusters of 16
// CTAs, which not every part of the chip can place; 256 threads 6.4 and 18.4, 1024
// threads 7.9 and 13.9).
//
// Sums.  Two blocks next to the border may differ in the last bits, and which
// of them stays must not depend on the order of a sum: each block's is carried
// as an fp32 sum with the sum of its rounding errors and rounded to fp32 once.  Over
// n additions in a chain (heads and log2 of the block size) the errors sum to at most
// n 2^-25 of the magnitudes and are themselves rounded n times: good to n^2 2^-49 (12
// for 8 heads, 2^-41), so the value is that of a sum in fp64 unless this one
// lies that close to the middle between two fp32 values.  (fp64 itself runs at 1/64 of
// the fp32 rate here.)
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

// a.hi + a.lo + x, the rounding error of the new hi added to lo.
__device__ __forceinline__ Pair pair_add(Pair a, float x) {
  const float s = __fadd_rn(a.hi, x);
  const float t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(x, t));
  return Pair{s, __fadd_rn(a.lo, e)};
}

__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const Pair c = pair_add(a, b.hi);
  return Pair{c.hi, __fadd_rn(c.lo, b.lo)};
}

// The sum, rounded once; an infinity or NaN (whose errors are NaN) as it is.
__device__ __forceinline__ float pair_value(Pair a) {
  return isfinite(a.hi) ? __fadd_rn(a.hi, a.lo) : a.hi;
}

// Order of block weights as an unsigned key: larger weight, larger key; NaN
// counts as -inf, and -0 as 0.  The largest key is kept for blocks that stay.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) w = __int_as_float(0xff800000u);
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sums over the CTA, one barrier each: consecutive calls use the two halves of
// `red` in turn.
struct BlockSum {
  int* red;  // [2][kEvictWarps]
  int turn = 0;

  __device__ __forceinline__ int* next() {
    turn ^= 1;
    return red + turn * kEvictWarps;
  }
  __device__ __forceinline__ int all(int v) {
    int* r = next();
    v = __reduce_add_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < kEvictWarps ? r[threadIdx.x & 31] : 0);
  }
  // Sum over the threads before this one, and over all.
  __device__ __forceinline__ uint32_t before(uint32_t v, uint32_t* total) {
    uint32_t* r = reinterpret_cast<uint32_t*>(next());
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) r[warp] = x;
    __syncthreads();
    const uint32_t w = lane < kEvictWarps ? r[lane] : 0;
    *total = __reduce_add_sync(0xffffffffu, w);
    return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + x - v;
  }
};

__global__ void __launch_bounds__(kEvictThreads) kvq_evict_kernel(const __grid_constant__ EvictArgs p, int cap) {
  extern __shared__ uint32_t smem[];
  BlockSum sum{reinterpret_cast<int*>(smem)};            // [2][kEvictWarps]
  uint32_t* range = smem + 2 * kEvictWarps;              // [2]: smallest and largest key
  uint32_t* keys = range + 2;                            // [cap], later the table row
  int* perm = reinterpret_cast<int*>(keys + cap);        // [cap] kept blocks, then evicted ones
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
  const int s = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int* row = p.table + (int64_t)s * p.max_blocks;
  if (tid == 0) {
    range[0] = 0xffffffffu;
    range[1] = 0;
  }
  cluster.barrier_arrive();  // (waited for before anything is written to another CTA)
  int L = p.lens[s];
  if (L > p.max_ctx) {
    if (rank == 0 && tid == 0) set_error(p.err, ERR_RANGE);
    L = p.max_ctx;
  }
  L = max(L, 0);
  const int bs = p.bs, bl = 31 - __clz(bs), n = (L + bs - 1) >> bl;
  const int nkept = min(n, p.budget);
  const float* sc = p.scores + (int64_t)s * p.Hkv * p.stride;
  // the row's first entries, on their way while the rest happens
  constexpr int kAhead = 4;
  int ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int j = tid + i * kEvictThreads;
    ahead[i] = rank == 0 && j < n ? row[j] : 0;
  }
  cluster.barrier_wait();

  if (n > nkept) {
    // ---- weights of the blocks.  A warp takes 64 tokens, a lane tokens l and
    // l + 32; blocks are bs consecutive lanes (of both tokens for bs = 64)
    const int width = min(bs, 32);
    for (int t0 = (rank * kEvictWarps + warp) * 64; t0 < n << bl; t0 += ranks * kEvictWarps * 64) {
      const int t = t0 + lane;
      Pair a[2] = {{0.f, 0.f}, {0.f, 0.f}};
      for (int h0 = 0; h0 < p.Hkv; h0 += 8) {
        float v[2][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float* at = sc + (int64_t)(h0 + i) * p.stride + t;
          v[0][i] = h0 + i < p.Hkv && t < L ? at[0] : 0.f;
          v[1][i] = h0 + i < p.Hkv && t + 32 < L ? at[32] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[0] = pair_add(a[0], v[0][i]);
          a[1] = pair_add(a[1], v[1][i]);
        }
      }
      if (bs == 64) {
        a[0] = pair_add(a[0], a[1]);
        a[1] = Pair{0.f, 0.f};
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        for (int o = width >> 1; o > 0; o >>= 1) {
          Pair b;
          b.hi = __shfl_xor_sync(0xffffffffu, a[c].hi, o);
          b.lo = __shfl_xor_sync(0xffffffffu, a[c].lo, o);
          a[c] = lane & o ? pair_add(b, a[c]) : pair_add(a[c], b);  // (the same on both sides)
        }
        const int jb = (t + 32 * c) >> bl;
        // lanes 0 .. ranks-1 of a block's hand its key to the CTAs
        for (int r = lane & (width - 1); r < ranks; r += width)
          if (jb < n && !(bs == 64 && c == 1)) {
            const uint32_t key =
                jb < p.sink || jb >= n - p.recent ? 0xffffffffu : weight_key(pair_value(a[c]));
            cluster.map_shared_rank(keys, r)[jb] = key;
          }
      }
    }
  }
  cluster.sync();

  // ---- the selection (every CTA the same): the largest T with at least
  // `budget` keys >= T; of the keys equal to T the first few stay
  if (n > nkept) {
    uint32_t lo = 0xffffffffu, hi = 0;
    for (int j = tid; j < n; j += kEvictThreads)
      if (keys[j] != 0xffffffffu) {
        lo = min(lo, keys[j]);
        hi = max(hi, keys[j]);
      }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      atomicMin(&range[0], lo);
      atomicMax(&range[1], hi);
    }
    __syncthreads();
    // at least `budget` keys are >= lo (all of them are); fewer are >= hi, unless
    // the blocks that stay anyway fill the budget
    lo = range[0];
    hi = range[1] + 1;
    if (p.sink + p.recent >= p.budget) lo = 0xffffffffu;
    while (lo != 0xffffffffu && hi - lo > 1) {
      const uint32_t mid = lo + (hi - lo) / 2;
      int v = 0;
      for (int j = tid; j < n; j += kEvictThreads) v += keys[j] >= mid;
      v = sum.all(v);
      if (v >= p.budget) lo = mid; else hi = mid;
      if (v == p.budget) break;
    }
    const uint32_t T = lo;
    const int per = (n + kEvictThreads - 1) / kEvictThreads;
    const int j0 = min(tid * per, n), j1 = min(j0 + per, n);
    uint32_t mine = 0;  // keys above T, and (high half) equal to it
    for (int j = j0; j < j1; ++j) mine += keys[j] > T ? 1u : keys[j] == T ? 0x10000u : 0u;
    uint32_t total;
    const uint32_t was = sum.before(mine, &total);
    const int ties = p.budget - static_cast<int>(total & 0xffffu);  // of the keys equal to T
    int tie = static_cast<int>(was >> 16);
    int pos = static_cast<int>(was & 0xffffu) + min(tie, ties);
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

  // ---- the row, its length and the list (the row may be permuted in place)
  if (rank == 0) {
    int* out = p.table_out + (int64_t)s * p.max_blocks;
    if (p.kept != nullptr)
      for (int j = tid; j < p.budget; j += kEvictThreads)
        p.kept[(int64_t)s * p.budget + j] = j < nkept ? perm[j] : -1;
    if (tid == 0) p.lens_out[s] = lens_new;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (tid + i * kEvictThreads < n) keys[tid + i * kEvictThreads] = static_cast<uint32_t>(ahead[i]);
    for (int j = tid + kAhead * kEvictThreads; j < n; j += kEvictThreads)
      keys[j] = static_cast<uint32_t>(row[j]);
    __syncthreads();
    for (int j = tid; j < n; j += kEvictThreads) out[j] = static_cast<int>(keys[perm[j]]);
    if (out != row)
      for (int j = n + tid; j < p.max_blocks; j += kEvictThreads) out[j] = row[j];
  }
  // ---- accumulators of the kept blocks, spread over the cluster: a warp takes
  // 256 tokens of one head
  if (p.scores_out != nullptr) {
    float* dst = p.scores_out + (int64_t)s * p.Hkv * p.out_stride;
    const int spans = (lens_new + 255) >> 8;
    for (int i = warp * ranks + rank; i < p.Hkv * spans; i += ranks * kEvictWarps) {
      const int h = i / spans, base = (i - h * spans) << 8;
      const float* from = sc + (int64_t)h * p.stride;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int t = base + 32 * k + lane;
        v[k] = t < lens_new ? from[((int64_t)perm[t >> bl] << bl) + (t & (bs - 1))] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int t = base + 32 * k + lane;
        if (t < lens_new) dst[(int64_t)h * p.out_stride + t] = v[k];
      }
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  const int cap = (std::min(a.max_blocks, (a.max_ctx + a.bs - 1) / a.bs) + 3) / 4 * 4;
  const int smem = (2 * kEvictWarps + 2 + std::max(cap, 4) * 2) * static_cast<int>(sizeof(uint32_t));
  // CTAs per sequence: as many as its longest possible row keeps busy.  8 rows, 1, 4
  // and 8 CTAs each: 1000 words 7.4, 7.5 and 7.4 us, 4096 11.5, 7.7 and 7.7, 32768
  // 15.5, 8.8 and 8.6, 262144 77.5, 25.1 and 16.5.  (Where the rows alone fill the
  // SMs fewer would do: 256 rows of 16384 words take 14.7, 25.2 and 42.2 us.)
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
