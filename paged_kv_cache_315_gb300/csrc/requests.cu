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
// round trips: one CTA computes the sums, and for small batches the same CTA then moves
// the entries; larger ones launch a grid for that.
#include <algorithm>
#include <climits>

#include "device_common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;

// Header of the workspace, in int32 words; then old[n], grow_off[n + 1], need_off[n + 1],
// give_off[n + 1].
enum { kWsHead = 0, kWsCount, kWsTaken, kWsGiven, kWsTokens, kWsWords = 8 };

struct ResizeParams {
  int32_t* block_tables;
  int32_t* context_lens;
  const int32_t* target_lens;
  int32_t* ring;
  int32_t* pool;
  int64_t* slots;
  int32_t* query_start;
  int32_t *ws, *old_len, *grow_off, *need_off, *give_off;
  int n, num_rows, ring_size, block_size, max_blocks_per_seq, num_blocks;
  unsigned* err;
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
__device__ __forceinline__ void fill(const ResizeParams& P, long long i, long long stride) {
  const int head = P.ws[kWsHead], count = P.ws[kWsCount];
  const int taken = P.ws[kWsTaken], given = P.ws[kWsGiven], tokens = P.ws[kWsTokens];
  const int bs = P.block_size;
  const long long end = static_cast<long long>(P.num_rows) + taken + given;
  for (; i < end; i += stride) {
    if (i < P.num_rows) {
      const int row = static_cast<int>(i);
      int64_t slot = -1;
      if (row < tokens) {
        const int s = owner(P.grow_off, P.n, row);
        const int old_len = P.old_len[s];
        if (old_len >= 0) {  // admitted
          const int pos = old_len + row - P.grow_off[s];
          const int j = pos / bs, had = (old_len + bs - 1) / bs;
          const int id =
              j < had ? P.block_tables[static_cast<size_t>(s) * P.max_blocks_per_seq + j]
                      : P.ring[(static_cast<long long>(head) + P.need_off[s] + j - had) %
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
      const int s = owner(P.need_off, P.n, a);
      const int had = (P.old_len[s] + bs - 1) / bs;
      P.block_tables[static_cast<size_t>(s) * P.max_blocks_per_seq + had + a - P.need_off[s]] =
          P.ring[(static_cast<long long>(head) + a) % P.ring_size];
    } else {
      const int b = static_cast<int>(i - P.num_rows - taken);
      const int s = owner(P.give_off, P.n, b);
      // old_len's blocks end at had; the returned ones are the last give_s of them
      const int had = (P.old_len[s] + bs - 1) / bs;
      const int give = P.give_off[s + 1] - P.give_off[s];
      if (static_cast<long long>(count) + b < P.ring_size)
        P.ring[(static_cast<long long>(head) + count + b) % P.ring_size] =
            P.block_tables[static_cast<size_t>(s) * P.max_blocks_per_seq + had - give + b -
                           P.give_off[s]];
    }
  }
}

// One CTA: the three prefix sums, which growths are admitted, the new lengths and the
// pool's state; with FILL the entries too.
template <bool FILL>
__global__ void __launch_bounds__(kPlanThreads) resize_plan_kernel(const ResizeParams P) {
  if (!FILL) griddep_launch_dependents();
  __shared__ long long tot_grow[kPlanWarps];
  __shared__ int tot_need[kPlanWarps], tot_give[kPlanWarps], most_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int head = P.pool[0], count = P.pool[1];
  if (head < 0 || head >= P.ring_size || count < 0 || count > P.ring_size) {
    if (tid == 0) raise_error(P.err, PKV_DERR_POOL);
    head = 0;
    count = 0;
  }
  if (tid == 0) most_taken = 0;
  // each thread owns a run of `per` requests
  const int per = (P.n + kPlanThreads - 1) / kPlanThreads;
  const int s0 = min(P.n, tid * per), s1 = min(P.n, s0 + per);
  Counts own{0, 0, 0};
  int old_len, new_len;
  for (int s = s0; s < s1; ++s) own = own + counts_of(P, s, old_len, new_len, true);
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
    const Counts c = counts_of(P, s, old_len, new_len, false);
    const Counts next = at + c;
    // a growth is admitted while the rows and, if it takes blocks, the free blocks reach:
    // both sums are over every request before it, so no later growth overtakes a refused one
    const bool ok = c.grow == 0 ||
                    (next.grow <= P.num_rows && (c.need == 0 || next.need <= count));
    if (ok)
      taken = c.need > 0 ? next.need : taken;
    else
      raise_error(P.err, PKV_DERR_POOL);
    P.old_len[s] = ok ? old_len : -1;
    const int row = static_cast<int>(min(at.grow, static_cast<long long>(INT_MAX)));
    P.grow_off[s] = row;
    P.need_off[s] = at.need;
    P.give_off[s] = at.give;
    if (P.query_start) P.query_start[s] = row;
    if (ok) P.context_lens[s] = new_len;
    at = next;
  }
  if (taken > 0) atomicMax(&most_taken, taken);
  if (tid == kPlanThreads - 1) {
    const int last = kPlanWarps - 1;
    const int rows = static_cast<int>(min(tot_grow[last], static_cast<long long>(INT_MAX)));
    P.grow_off[P.n] = rows;
    P.need_off[P.n] = tot_need[last];
    P.give_off[P.n] = tot_give[last];
    if (P.query_start) P.query_start[P.n] = rows;
    P.ws[kWsHead] = head;
    P.ws[kWsCount] = count;
    P.ws[kWsGiven] = tot_give[last];
    P.ws[kWsTokens] = min(rows, P.num_rows);
  }
  __syncthreads();
  if (tid == 0) {
    const int given = tot_give[kPlanWarps - 1];
    P.ws[kWsTaken] = most_taken;
    long long left = static_cast<long long>(count) + given;
    if (left > P.ring_size) {  // more blocks come back than the ring has places for
      raise_error(P.err, PKV_DERR_POOL);
      left = P.ring_size;
    }
    P.pool[0] = static_cast<int>((static_cast<long long>(head) + most_taken) % P.ring_size);
    P.pool[1] = static_cast<int>(left - most_taken);
  }
  if (FILL) {
    __syncthreads();
    fill(P, tid, kPlanThreads);
  }
}

__global__ void __launch_bounds__(kFillThreads) resize_fill_kernel(const ResizeParams P) {
  griddep_wait();
  fill(P, static_cast<long long>(blockIdx.x) * kFillThreads + threadIdx.x,
       static_cast<long long>(gridDim.x) * kFillThreads);
}

}  // namespace

size_t resize_workspace_size(int num_seqs) {
  return (kWsWords + 4ull * num_seqs + 3) * sizeof(int32_t);
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
  P.old_len = P.ws + kWsWords;
  P.grow_off = P.old_len + a.num_seqs;
  P.need_off = P.grow_off + a.num_seqs + 1;
  P.give_off = P.need_off + a.num_seqs + 1;
  P.n = a.num_seqs;
  P.num_rows = a.num_rows;
  P.ring_size = a.ring_size;
  P.block_size = a.block_size;
  P.max_blocks_per_seq = a.max_blocks_per_seq;
  P.num_blocks = a.num_blocks;
  P.err = a.err;
  resize_plan_kernel<true><<<1, kPlanThreads, 0, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

}  // namespace pkv
