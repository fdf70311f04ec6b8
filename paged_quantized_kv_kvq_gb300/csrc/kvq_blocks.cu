// kvq_blocks.cu -- a step's block tables, slot map and positions from the requests'
// lengths, and the blocks of requests that shrank or ended back on the free list, so
// that a serving step (a captured one, too) needs no host to plan it.
//
//   need_s = ceil((L_s + n_s) / bs) - ceil(L_s / bs)     blocks sequence s takes
//   q_s    = n_0 + .. + n_{s-1}                          its first row
//   b_s    = need_0 + .. + need_{s-1}                    blocks taken before it
//   row q_s + i: position L_s + i, in block (L_s + i) / bs of its table row, which
//   is an older entry or free_list[count - 1 - (b_s + .. )]
//
// Two prefix sums over the sequences, then one independent lookup per row and per new
// table entry.  Bound: latency -- a launch, a chain of loads (lengths, then free-list
// entries) and the scan's barriers; the bytes are 16 a row.  One thread-block cluster
// does it all: every CTA makes the whole scan for itself (8 bytes a sequence, from L2)
// and keeps it in shared memory, the rows and entries are shared out among the CTAs, and
// one cluster barrier stands between the last read of the lengths and the count and the
// first write to them, so that both may be updated in place.  Measured, replayed: a decode
// step of 64 sequences 3.0 us for the tables and 3.2 for the blocks that come back; 32768
// rows of 512 sequences 6.0, 32768 freed blocks 7.8; the cases below the launch rules.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvq_context.h"
#include "kvq_internal.h"

namespace cg = cooperative_groups;

namespace kvq {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
// CTAs of a cluster (of 8 instead: 32768 rows of 512 sequences 8.1 us where 16 take 6.0, 16384
// freed entries 7.1 and 5.1; small calls alike).  A partition of a GPU whose processing
// clusters have fewer SMs cannot place 16: it gets the 8 that every one places.
constexpr int kPlanCluster = 16, kPlanClusterSmall = 8;
// Rows and table entries up to which one CTA does it alone, without the cluster's barriers.
// Rows, alone and as a cluster: 64 3.0 and 4.1 us, 512 3.2 and 3.7, 1024 4.4 and 4.4, 2048
// 5.6 and 4.4.  Entries (the host does not know how many go; a tenth): 2048 3.2 and 5.0,
// 8192 3.2 and 4.9, 16384 4.4 and 5.0, 32768 5.5 and 5.2; all of 16384: 20 and 5.2.
constexpr int kPlanAlone = 1024;
constexpr int64_t kPlanAloneEntries = 16384;
// Neighbouring entries a thread frees at a time (1, 2, 4: alone, 768 of 8192 4.1, 3.2 and 3.6
// us), and rows a thread of a cluster's (alone 1: 64 rows take 3.0, 3.6 and 4.4 us).  Both
// calls for 512 sequences, 64 ended and 64 begun with up to 1024 tokens, with 1, 2 and 4 of
// each: 17.2, 12.6 and 14.5 us (1 with 8 CTAs).
constexpr int kPlanEntries = 2, kPlanRows = 2;
constexpr uint32_t kPlanCap = 0x7fffffffu;  // prefix sums stop here

// a + b of two sums that are at most the cap, at most the cap (associative).
__device__ __forceinline__ uint32_t cap_add(uint32_t a, uint32_t b) { return min(a + b, kPlanCap); }

// Sums (capped) of two values over the threads before this one and over all of them.
struct PairScan {
  uint2* part;  // [kPlanWarps]

  __device__ __forceinline__ uint2 before(uint2 v, uint2* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint2 x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
      if (lane >= o) x = make_uint2(cap_add(x.x, a), cap_add(x.y, b));
    }
    uint2 e = make_uint2(__shfl_up_sync(0xffffffffu, x.x, 1), __shfl_up_sync(0xffffffffu, x.y, 1));
    if (lane == 0) e = make_uint2(0, 0);
    __syncthreads();  // (the sums of the call before have been read)
    if (lane == 31) part[warp] = x;
    __syncthreads();
    uint2 w = make_uint2(0, 0), all = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < kPlanWarps; ++i) {
      const uint2 p = part[i];
      if (i < warp) w = make_uint2(cap_add(w.x, p.x), cap_add(w.y, p.y));
      all = make_uint2(cap_add(all.x, p.x), cap_add(all.y, p.y));
    }
    *total = all;
    return make_uint2(cap_add(w.x, e.x), cap_add(w.y, e.y));
  }
};

// Last index s in [0, n) with first[s] <= x (first[0] = 0 <= x).
__device__ __forceinline__ int last_at_most(const uint32_t* first, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

template <int R>
__global__ void __launch_bounds__(kPlanThreads) kvq_extend_kernel(const __grid_constant__ ExtendArgs p,
                                                                 int bs_log2) {
  extern __shared__ uint32_t smem[];
  const int S = p.S, tid = threadIdx.x;
  PairScan scan{reinterpret_cast<uint2*>(smem)};  // [kPlanWarps]
  uint32_t* rows = smem + 2 * kPlanWarps;         // [S + 1] rows before each sequence
  uint32_t* taken = rows + S + 1;                 // [S + 1] blocks before it
  int* len = reinterpret_cast<int*>(taken + S + 1);  // [S] its length, or ~length where it is not served
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
  const int bs = 1 << bs_log2;

  const int given = *p.count, count = min(max(given, 0), p.capacity);
  // ---- prefix sums; who is served
  uint2 carry = make_uint2(0, 0);
  uint32_t served = 0;  // blocks that served sequences take
  int L_next = tid < S ? p.lens[tid] : 0, n_next = tid < S ? p.n[tid] : 0;
  for (int base = 0; base < S; base += kPlanThreads) {
    const int s = base + tid, L = L_next, n = n_next;
    const bool more = s + kPlanThreads < S;  // (loaded while this turn's sums are made)
    L_next = more ? p.lens[s + kPlanThreads] : 0;
    n_next = more ? p.n[s + kPlanThreads] : 0;
    const bool ok = n >= 0 && L >= 0 && (int64_t)L + n <= (int64_t)p.max_blocks << bs_log2;
    const uint32_t need = ok ? static_cast<uint32_t>((((int64_t)L + n + bs - 1) >> bs_log2) - (((int64_t)L + bs - 1) >> bs_log2)) : 0;
    uint2 all;
    const uint2 own = make_uint2(max(n, 0), need);
    uint2 at = scan.before(own, &all);
    at = make_uint2(cap_add(carry.x, at.x), cap_add(carry.y, at.y));
    const uint2 end = make_uint2(cap_add(at.x, own.x), cap_add(at.y, own.y));
    carry = make_uint2(cap_add(carry.x, all.x), cap_add(carry.y, all.y));
    // (a sum at the cap is more than any call has of either)
    const bool serve = ok && end.x <= static_cast<uint32_t>(p.max_tokens) &&
                       (need == 0 || end.y <= static_cast<uint32_t>(count));
    if (s < S) {
      rows[s] = min(at.x, static_cast<uint32_t>(p.max_tokens));
      taken[s] = at.y;
      len[s] = serve ? L : ~max(L, 0);
      if (serve && need > 0) served = end.y;  // (they take the first blocks: the last one's end is their sum)
      if (!serve && rank == 0) set_error(p.err, ERR_RANGE);
    }
  }
  if (tid == 0) {
    rows[S] = min(carry.x, static_cast<uint32_t>(p.max_tokens));
    taken[S] = carry.y;
  }
  served = __reduce_max_sync(0xffffffffu, served);
  __syncthreads();  // rows, taken, len; the scan's sums have been read
  if ((tid & 31) == 0) smem[tid >> 5] = served;
  __syncthreads();
  served = __reduce_max_sync(0xffffffffu, smem[tid & (kPlanWarps - 1)]);

  // every CTA has read the lengths and the count
  if (ranks > 1) cluster.sync();
  const int step = ranks * kPlanThreads, me = rank * kPlanThreads + tid;
  if (me == 0) {
    if (given != count) set_error(p.err, ERR_RANGE);
    *p.count_out = count - static_cast<int>(served);
  }
  for (int s = me; s <= S; s += step) {
    p.q_start[s] = static_cast<int>(rows[s]);
    if (s == S) break;
    const int L = len[s];
    if (L >= 0) p.lens_out[s] = L + static_cast<int>(rows[s + 1] - rows[s]);
    else if (p.lens_out != p.lens) p.lens_out[s] = p.lens[s];
  }
  auto pool_block = [&](int id) { return id >= 0 && (int64_t)id < p.num_blocks; };
  // ---- new table entries
  for (uint32_t k = me; k < served; k += step) {
    const int s = last_at_most(taken, S, k);
    const int64_t j = (((int64_t)len[s] + bs - 1) >> bs_log2) + (k - taken[s]);
    const int id = p.free_list[count - 1 - static_cast<int>(k)];
    if (!pool_block(id)) set_error(p.err, ERR_RANGE);
    p.table[(int64_t)s * p.max_blocks + j] = id;
  }
  // ---- rows, R neighbours at a time: one search, their lookups side by side
  const int64_t last = rows[S];
  for (int64_t r0 = (int64_t)me * R; r0 < p.max_tokens; r0 += (int64_t)step * R) {
    int64_t slot[R], pos[R];
    int id[R];
    int s = r0 < last ? last_at_most(rows, S, static_cast<uint32_t>(r0)) : 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = r0 + i;
      slot[i] = -1;
      pos[i] = 0;
      id[i] = 0;
      if (r >= last) continue;
      if (rows[s + 1] <= r) s = last_at_most(rows, S, static_cast<uint32_t>(r));
      const int L = len[s];
      pos[i] = (L >= 0 ? L : ~L) + (r - rows[s]);
      if (L < 0) continue;
      const int64_t held = ((int64_t)L + bs - 1) >> bs_log2, j = pos[i] >> bs_log2;
      id[i] = j < held ? p.table[(int64_t)s * p.max_blocks + j]
                       : p.free_list[count - 1 - static_cast<int>(taken[s] + (j - held))];
      slot[i] = pos[i] & (bs - 1);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (slot[i] < 0) continue;
      if (pool_block(id[i])) slot[i] += (int64_t)id[i] << bs_log2;
      else {
        slot[i] = -1;
        set_error(p.err, ERR_RANGE);
      }
    }
    if (R % 2 == 0 && p.wide && r0 + R <= p.max_tokens) {
#pragma unroll
      for (int i = 0; i + 1 < R; i += 2) {
        *reinterpret_cast<longlong2*>(p.slots + r0 + i) = make_longlong2(slot[i], slot[i + 1]);
        *reinterpret_cast<longlong2*>(p.positions + r0 + i) = make_longlong2(pos[i], pos[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (r0 + i >= p.max_tokens) break;
        p.slots[r0 + i] = slot[i];
        p.positions[r0 + i] = pos[i];
      }
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) kvq_release_kernel(const __grid_constant__ ReleaseArgs p,
                                                                  int bs_log2) {
  constexpr int R = kPlanEntries;
  extern __shared__ uint32_t smem[];
  const int S = p.S, tid = threadIdx.x;
  PairScan scan{reinterpret_cast<uint2*>(smem)};  // [kPlanWarps]
  uint32_t* here = smem + 2 * kPlanWarps;         // blocks of the pool among this CTA's entries
  uint32_t* gone = here + 1;                      // [S] entries before each sequence
  int* first = reinterpret_cast<int*>(gone + S);  // [S] its first entry that goes
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
  const int bs = 1 << bs_log2;

  const int given = *p.count, count = min(max(given, 0), p.capacity);
  uint2 carry = make_uint2(0, 0);
  int a_next = tid < S ? p.old_lens[tid] : 0, b_next = tid < S ? p.new_lens[tid] : 0;
  for (int base = 0; base < S; base += kPlanThreads) {
    const int s = base + tid, a = a_next, b = b_next;
    const bool more = s + kPlanThreads < S;  // (loaded while this turn's sums are made)
    a_next = more ? p.old_lens[s + kPlanThreads] : 0;
    b_next = more ? p.new_lens[s + kPlanThreads] : 0;
    int64_t from = 0, to = 0;
    if (s < S) {
      to = ((int64_t)max(a, 0) + bs - 1) >> bs_log2;
      from = max(((int64_t)max(b, 0) + bs - 1) >> bs_log2, (int64_t)p.shared);
      if (a < 0 || b < 0 || to > p.max_blocks) {
        if (rank == 0) set_error(p.err, ERR_RANGE);
        to = min(to, (int64_t)p.max_blocks);
      }
    }
    uint2 all;
    const uint2 at = scan.before(make_uint2(from < to ? static_cast<uint32_t>(to - from) : 0, 0), &all);
    if (s < S) {
      gone[s] = cap_add(carry.x, at.x);
      first[s] = static_cast<int>(min(from, (int64_t)p.max_blocks));
    }
    carry.x = cap_add(carry.x, all.x);
  }
  const uint32_t total = carry.x;
  if (tid == 0) *here = 0;
  __syncthreads();

  // ---- this CTA's entries: how many are blocks of the pool, then each to its place
  const uint32_t per = (total + ranks - 1) / ranks;
  const uint32_t e0 = static_cast<uint32_t>(min((uint64_t)rank * per, (uint64_t)total));
  const uint32_t e1 = static_cast<uint32_t>(min((uint64_t)e0 + per, (uint64_t)total));
  int ids[R];
  auto entries = [&](uint32_t e) {  // R neighbours: one search, their loads side by side
    int q = e < e1 ? last_at_most(gone, S, e) : 0;
#pragma unroll
    for (int i = 0; i < R; ++i, ++e) {
      ids[i] = -1;
      if (e >= e1) continue;
      if (q + 1 < S && gone[q + 1] <= e) q = last_at_most(gone, S, e);
      ids[i] = p.table[(int64_t)q * p.max_blocks + first[q] + (e - gone[q])];
    }
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (!(ids[i] >= 0 && (int64_t)ids[i] < p.num_blocks)) ids[i] = -1;
      n += ids[i] >= 0;
    }
    return n;
  };
  const uint32_t round = kPlanThreads * R;
  uint32_t mine = 0;
  if (ranks > 1) {
    for (uint32_t base = e0; base < e1; base += round) mine += entries(base + tid * R);
    const uint32_t sum = __reduce_add_sync(0xffffffffu, mine);
    if ((tid & 31) == 0 && sum > 0) atomicAdd(here, sum);
    cluster.sync();  // (and every CTA has read the count)
  }
  uint32_t at = 0;
  for (int q = 0; q < rank; ++q) at += *cluster.map_shared_rank(here, q);
  for (uint32_t base = e0; base < e1; base += round) {
    // (a single round's entries are the ones just counted)
    if (ranks == 1 || e1 - e0 > round) mine = entries(base + tid * R);
    uint32_t e = base + tid * R;
    uint2 all;
    uint32_t k = at + scan.before(make_uint2(mine, 0), &all).x;
#pragma unroll
    for (int i = 0; i < R; ++i, ++e) {
      if (ids[i] >= 0) {
        if ((int64_t)count + k < p.capacity) p.free_list[count + k] = ids[i];
        else set_error(p.err, ERR_RANGE);
        ++k;
      } else if (e < e1) {
        set_error(p.err, ERR_RANGE);
      }
    }
    at += all.x;
  }
  // the last CTA has counted them all
  if (rank == ranks - 1 && tid == 0) {
    if (given != count) set_error(p.err, ERR_RANGE);
    *p.count_out = static_cast<int>(min((int64_t)count + at, (int64_t)p.capacity));
  }
  if (ranks > 1) cluster.sync();  // no CTA leaves while its count may be read
}

template <auto Kernel, class Args>
cudaError_t launch_plan(const Args& a, bool alone, size_t smem, cudaStream_t st) {
  static PerContext<int> most;  // CTAs of a cluster that this context's device places
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kPlanThreads);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto ctas_of = [&](int n) { cfg.gridDim = dim3(attr[0].val.clusterDim.x = static_cast<unsigned>(n)); };
  int ctas = 0;
  const cudaError_t e = most.get(&ctas, [&](int* n) {
    const size_t big = cfg.dynamicSmemBytes = 227 * 1024;
    cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(big));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    int fit = 0;
    ctas_of(kPlanCluster);
    if (cudaOccupancyMaxActiveClusters(&fit, Kernel, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      fit = 0;
    }
    *n = fit > 0 ? kPlanCluster : kPlanClusterSmall;
    return cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  ctas_of(alone ? 1 : ctas);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  int log2 = 0;
  while ((1 << log2) < a.bs) ++log2;
  return phase_mark(st, cudaLaunchKernelEx(&cfg, Kernel, a, log2));
}

}  // namespace

cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t st) {
  const size_t smem = (2 * kPlanWarps + 3 * (size_t)a.S + 2) * 4;
  ExtendArgs b = a;
  b.wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0;
  if (a.max_tokens <= kPlanAlone) return launch_plan<kvq_extend_kernel<1>>(b, true, smem, st);
  return launch_plan<kvq_extend_kernel<kPlanRows>>(b, false, smem, st);
}

cudaError_t launch_release(const ReleaseArgs& a, cudaStream_t st) {
  const size_t smem = (2 * kPlanWarps + 1 + 2 * (size_t)a.S) * 4;
  return launch_plan<kvq_release_kernel>(a, (int64_t)a.S * a.max_blocks <= kPlanAloneEntries, smem, st);
}

}  // namespace kvq
