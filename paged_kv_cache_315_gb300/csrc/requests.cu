// requests.cu -- block tables, slot map and free list from request lengths (sm_103a).
//
// One call moves every request s from its cached length old_s to a target length new_s.
// With had_s = ceil(old_s / bs) and has_s = ceil(new_s / bs) blocks,
//     grow_s = max(0, new_s - old_s) tokens,   need_s = max(0, has_s - had_s) blocks taken,
//     give_s = max(0, had_s - has_s) blocks given back,
// and the exclusive prefix sums of the three over the requests place everything: request s
// takes free-ring entries head + excl(need)_s + j, its tokens own rows excl(grow)_s + i of
// the slot map, and its returned blocks go to ring entries head + count + excl(give)_s + j.
// Taken and returned entries are disjoint (the ring holds each block at most once), so
// every entry can be moved independently once the sums are known.
//
// The work is a few bytes per request and token, far below one launch's latency for any
// decode batch, so what counts is the number of launches and of dependent memory
// round trips.  One launch of a cluster of 8 CTAs does it all: every CTA computes the sums for
// itself in shared memory, moves its share of the entries, and when all CTAs have read the old
// lengths (the cluster's barrier) the first one writes the new ones and the pool's state.  Many
// requests or rows take two grids: one CTA for the sums, then as many as the entries want.
#include <algorithm>
#include <climits>

#include "device_common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCluster = 8;
constexpr int kMaxClusterSeqs = 8192;     // sums of 128 KB of shared memory
// Rows up to which one launch of 8 CTAs beats two grids.  Measured there and back (two calls):
// 128 requests with 128 rows 8.0 us in a cluster, 9.5 in two grids; 2000 requests with 32000 rows
// 20 against 17, with 128000 rows 36 against 17.
constexpr int kMaxClusterRows = 1 << 14;

struct Totals {
  int head, count, taken, given, tokens;
};

struct ResizeParams {
  int32_t* block_tables;
  int32_t* context_lens;
  const int32_t* target_lens;
  int32_t* ring;
  int32_t* pool;
  int64_t* slots;
  int32_t* query_start;
  int32_t* ws;  // two-grid form: Totals, then the sums
  int n, num_rows, ring_size, block_size, max_blocks_per_seq, num_blocks;
  unsigned* err;
};

constexpr int kWsWords = 8;

// The requests' old lengths (-1: refused) and exclusive sums, n + 1 entries each.
struct Sums {
  int32_t *old_len, *grow_off, *need_off, *give_off;
  __host__ __device__ Sums(int32_t* at, int n)
      : old_len(at), grow_off(at + n + 1), need_off(at + 2 * (n + 1)), give_off(at + 3 * (n + 1)) {}
};

struct Counts {
  long long grow;
  int need, give;
};

__device__ __forceinline__ Counts operator+(Counts a, Counts b) {
  return {a.grow + b.grow, a.need + b.need, a.give + b.give};
}

__device__ __forceinline__ Counts shfl_up(Counts c, int o) {
  return {__shfl_up_sync(0xffffffffu, c.grow, o), __shfl_up_sync(0xffffffffu, c.need, o),
          __shfl_up_sync(0xffffffffu, c.give, o)};
}

// Request s's counts; a length outside the table leaves the request as it is (and says so).
__device__ __forceinline__ Counts counts_of(const ResizeParams& P, int s, int& old_len,
                                            int& new_len, bool report) {
  const int bs = P.block_size;
  const int cap = P.max_blocks_per_seq * bs;
  old_len = P.context_lens[s];
  new_len = P.target_lens[s];
  if (old_len < 0 || old_len > cap || new_len < 0 || new_len > cap) {
    if (report) raise_error(P.err, PKV_DERR_CONTEXT);
    new_len = old_len;
    return {0, 0, 0};
  }
  const int had = (old_len + bs - 1) / bs, has = (new_len + bs - 1) / bs;
  return {max(0, new_len - old_len), max(0, has - had), max(0, had - has)};
}

// Largest s in [0, n) with off[s] <= i (off non-decreasing, off[0] = 0 <= i < off[n]).
__device__ __forceinline__ int owner(const int32_t* off, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Entries i, i + stride, ... of the slot map, the taken blocks and the returned blocks.
__device__ __forceinline__ void fill(const ResizeParams& P, const Sums& S, const Totals& tot,
                                     long long i, long long stride) {
  const int head = tot.head, count = tot.count;
  const int taken = tot.taken, given = tot.given, tokens = tot.tokens;
  const int bs = P.block_size;
  const long long end = static_cast<long long>(P.num_rows) + taken + given;
#pragma unroll 2
  for (; i < end; i += stride) {
    if (i < P.num_rows) {
      const int row = static_cast<int>(i);
      int64_t slot = -1;
      if (row < tokens) {
        const int s = owner(S.grow_off, P.n, row);
        const int old_len = S.old_len[s];
        if (old_len >= 0) {  // admitted
          const int pos = old_len + row - S.grow_off[s];
          const int j = pos / bs, had = (old_len + bs - 1) / bs;
          const int id =
              j < had ? P.block_tables[static_cast<size_t>(s) * P.max_blocks_per_seq + j]
                      : P.ring[(static_cast<long long>(head) + S.need_off[s] + j - had) %
                               P.ring_size];
          if (id >= 0 && id < P.num_blocks)
            slot = static_cast<int64_t>(id) * bs + pos % bs;
          else
            raise_error(P.err, PKV_DERR_BLOCK_ID);
        }
      }
      P.slots[row] = slot;
    } else if (i < static_cast<long long>(P.num_rows) + taken) {
      const int a = static_cast<int>(i - P.num_rows);
      const int s = owner(S.need_off, P.n, a);
      const int had = (S.old_len[s] + bs - 1) / bs;
      P.block_tables[static_cast<size_t>(s) * P.max_blocks_per_seq + had + a - S.need_off[s]] =
          P.ring[(static_cast<long long>(head) + a) % P.ring_size];
    } else {
      const int b = static_cast<int>(i - P.num_rows - taken);
      const int s = owner(S.give_off, P.n, b);
      // old_len's blocks end at had; the returned ones are the last give_s of them
      const int had = (S.old_len[s] + bs - 1) / bs;
      const int give = S.give_off[s + 1] - S.give_off[s];
      if (static_cast<long long>(count) + b < P.ring_size)
        P.ring[(static_cast<long long>(head) + count + b) % P.ring_size] =
            P.block_tables[static_cast<size_t>(s) * P.max_blocks_per_seq + had - give + b -
                           S.give_off[s]];
    }
  }
}

// One CTA's threads: the three prefix sums, which growths are admitted, and the totals.  `report`:
// say what is wrong with lengths, pool or growths.
__device__ Totals plan(const ResizeParams& P, const Sums& S, bool report) {
  __shared__ long long tot_grow[kPlanWarps];
  __shared__ int tot_need[kPlanWarps], tot_give[kPlanWarps], most_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int head = P.pool[0], count = P.pool[1];
  // each thread owns a run of `per` requests
  const int per = (P.n + kPlanThreads - 1) / kPlanThreads;
  const int s0 = min(P.n, tid * per), s1 = min(P.n, s0 + per);
  Counts own{0, 0, 0}, c{0, 0, 0};
  int old_len = 0, new_len = 0;
  for (int s = s0; s < s1; ++s) {
    c = counts_of(P, s, old_len, new_len, report);
    own = own + c;
  }
  if (head < 0 || head >= P.ring_size || count < 0 || count > P.ring_size) {
    if (report && tid == 0) raise_error(P.err, PKV_DERR_POOL);
    head = 0;
    count = 0;
  }
  if (tid == 0) most_taken = 0;
  Counts incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Counts y = shfl_up(incl, o);
    if (lane >= o) incl = incl + y;
  }
  if (lane == 31) {
    tot_grow[warp] = incl.grow;
    tot_need[warp] = incl.need;
    tot_give[warp] = incl.give;
  }
  __syncthreads();
  if (warp == 0) {
    Counts v{tot_grow[lane], tot_need[lane], tot_give[lane]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Counts y = shfl_up(v, o);
      if (lane >= o) v = v + y;
    }
    tot_grow[lane] = v.grow;
    tot_need[lane] = v.need;
    tot_give[lane] = v.give;
  }
  __syncthreads();
  Counts at{incl.grow - own.grow, incl.need - own.need, incl.give - own.give};
  if (warp > 0) at = at + Counts{tot_grow[warp - 1], tot_need[warp - 1], tot_give[warp - 1]};
  int taken = 0;
  for (int s = s0; s < s1; ++s) {
    if (per > 1) c = counts_of(P, s, old_len, new_len, false);
    const Counts next = at + c;
    // a growth is admitted while the rows and, if it takes blocks, the free blocks reach:
    // both sums are over every request before it, so no later growth overtakes a refused one
    const bool ok = c.grow == 0 ||
                    (next.grow <= P.num_rows && (c.need == 0 || next.need <= count));
    if (ok)
      taken = c.need > 0 ? next.need : taken;
    else if (report)
      raise_error(P.err, PKV_DERR_POOL);
    S.old_len[s] = ok ? old_len : -1;
    S.grow_off[s] = static_cast<int>(min(at.grow, static_cast<long long>(INT_MAX)));
    S.need_off[s] = at.need;
    S.give_off[s] = at.give;
    at = next;
  }
  if (taken > 0) atomicMax(&most_taken, taken);
  const int last = kPlanWarps - 1;
  const int rows = static_cast<int>(min(tot_grow[last], static_cast<long long>(INT_MAX)));
  if (tid == 0) {
    S.grow_off[P.n] = rows;
    S.need_off[P.n] = tot_need[last];
    S.give_off[P.n] = tot_give[last];
  }
  __syncthreads();
  return {head, count, most_taken, tot_give[last], min(rows, P.num_rows)};
}

// One CTA's threads: the new lengths, the rows' starts and the pool's state.
__device__ void commit(const ResizeParams& P, const Sums& S, const Totals& tot) {
  const int tid = threadIdx.x;
  for (int s = tid; s <= P.n; s += kPlanThreads) {
    if (P.query_start) P.query_start[s] = S.grow_off[s];
    if (s < P.n && S.old_len[s] >= 0) {
      int old_len, new_len;
      counts_of(P, s, old_len, new_len, false);
      P.context_lens[s] = new_len;
    }
  }
  if (tid == 0) {
    long long left = static_cast<long long>(tot.count) + tot.given;
    if (left > P.ring_size) {  // more blocks come back than the ring has places for
      raise_error(P.err, PKV_DERR_POOL);
      left = P.ring_size;
    }
    P.pool[0] = static_cast<int>((static_cast<long long>(tot.head) + tot.taken) % P.ring_size);
    P.pool[1] = static_cast<int>(left - tot.taken);
  }
}

__global__ void __launch_bounds__(kPlanThreads) resize_cluster_kernel(const ResizeParams P) {
  extern __shared__ int32_t sums[];
  const Sums S(sums, P.n);
  const bool first = blockIdx.x == 0;
  const Totals tot = plan(P, S, first);
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  fill(P, S, tot, blockIdx.x * kPlanThreads + threadIdx.x, gridDim.x * kPlanThreads);
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (first) commit(P, S, tot);
}

__global__ void __launch_bounds__(kPlanThreads) resize_plan_kernel(const ResizeParams P) {
  griddep_launch_dependents();
  const Sums S(P.ws + kWsWords, P.n);
  const Totals tot = plan(P, S, true);
  if (threadIdx.x == 0) *reinterpret_cast<Totals*>(P.ws) = tot;
  commit(P, S, tot);
}

__global__ void __launch_bounds__(kFillThreads) resize_fill_kernel(const ResizeParams P) {
  griddep_wait();
  fill(P, Sums(P.ws + kWsWords, P.n), *reinterpret_cast<const Totals*>(P.ws),
       static_cast<long long>(blockIdx.x) * kFillThreads + threadIdx.x,
       static_cast<long long>(gridDim.x) * kFillThreads);
}

}  // namespace

size_t resize_workspace_size(int num_seqs) {
  return (kWsWords + 4ull * (static_cast<size_t>(num_seqs) + 1)) * sizeof(int32_t);
}

int launch_resize_requests(const ResizeArgs& a, cudaStream_t stream) {
  ResizeParams P{};
  P.block_tables = a.block_tables;
  P.context_lens = a.context_lens;
  P.target_lens = a.target_lens;
  P.ring = a.free_ring;
  P.pool = a.pool_state;
  P.slots = a.slot_mapping;
  P.query_start = a.query_start;
  P.ws = static_cast<int32_t*>(a.workspace);
  P.n = a.num_seqs;
  P.num_rows = a.num_rows;
  P.ring_size = a.ring_size;
  P.block_size = a.block_size;
  P.max_blocks_per_seq = a.max_blocks_per_seq;
  P.num_blocks = a.num_blocks;
  P.err = a.err;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.num_seqs <= kMaxClusterSeqs && a.num_rows <= kMaxClusterRows) {
    const int smem = static_cast<int>(4 * sizeof(int32_t) * (a.num_seqs + 1));
    if (smem > 47 * 1024 &&
        cudaFuncSetAttribute(reinterpret_cast<const void*>(resize_cluster_kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return PKV_ECUDA;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {kCluster, 1, 1};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    return cudaLaunchKernelEx(&cfg, resize_cluster_kernel, P) == cudaSuccess ? PKV_OK : PKV_ECUDA;
  }
  resize_plan_kernel<<<1, kPlanThreads, 0, stream>>>(P);
  if (cudaGetLastError() != cudaSuccess) return PKV_ECUDA;
  // rows, and the blocks that they may take; blocks that come back share the threads
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const long long entries = static_cast<long long>(a.num_rows) + a.num_rows / a.block_size + 65536;
  cfg.gridDim = dim3(static_cast<unsigned>(
      std::min((entries + kFillThreads - 1) / kFillThreads, 8LL * 152)));
  cfg.blockDim = dim3(kFillThreads);
  return cudaLaunchKernelEx(&cfg, resize_fill_kernel, P) == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

}  // namespace pkv
