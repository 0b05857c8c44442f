// decode_fp4.cu -- paged single-token decode attention over 4-bit caches (sm_103a).
//
// Per cached token and KV head the cache holds two rows (key, value) of head_dim E2M1 codes
// and one bf16 scale each: head_dim + 4 bytes.  Element d of a key is code_d * ks, so
//     score(p) = scale * <q, K_p> = (scale * ks_p) * <q, codes(K_p)>,
//     out      = sum_p softmax(score)_p * vs_p * codes(V_p),
// and both scales stay outside the products over the codes.
//
// Work split.  A sequence of L tokens has ceil(L / 128) tiles.  The tiles of all sequences,
// in order, are cut into R ranges of equal cost (to one tile), and one CTA runs one range
// for one (KV head, chunk of query heads) unit; the units of a range are neighbouring CTAs,
// so the heads of one token, which lie side by side in memory, are read together.  A range
// may begin inside one sequence and end inside another: a CTA leaves (m, l, o) partials for
// those two, writes the rows of every sequence that lies inside its range itself, and a
// second grid merges the partials by log-sum-exp.  Equal ranges keep every CTA busy to the
// end whatever the lengths are, and there are at most 2 partials per CTA.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <mutex>
#include <type_traits>

#include "device_common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "umma.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;       // tokens of a tile
constexpr int kHeads = 8;        // query heads of a unit, at most
constexpr int kRangeCtas = 456;  // CTAs the ranges aim for: three on each of 152 SMs,
constexpr int kMaxRanges = 912;  // or six of the CUDA-core kernel's
constexpr int kSimtWarps = 4;
constexpr int kSimtThreads = 32 * kSimtWarps;

struct Fp4Params {
  void* out;
  const void* q;
  const uint8_t *k_cache, *v_cache;
  const __nv_bfloat16 *k_scales, *v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* part_o;    // [ranges][2][num_q_heads][head_dim]
  float2* part_ml;  // [ranges][2][num_q_heads]: (m in log2 units, l)
  int2* info;       // [ranges]: the sequence that begins in the range and goes on past it
                    // (or -1), and the last range that holds tiles of it
  unsigned* err;
  int num_seqs, num_q_heads, num_kv_heads, group, chunk, num_chunks;
  int max_blocks_per_seq, num_blocks, block_size, ranges, seq_cost;
  float scale_log2;
};

// Where a range begins: `tiles` tiles from tile `tile` of sequence `s` on.  Ranges behind the
// batch's last tile have none.
struct Span {
  int s, tile, tiles;
};

__device__ __forceinline__ int live_len(const Fp4Params& P, int s) {
  const int L = P.context_lens[s], cap = P.max_blocks_per_seq * P.block_size;
  return L < 0 ? 0 : min(L, cap);
}

// Quotient of non-negative numbers, mostly small ones (a 64-bit division takes three times as
// long).
__device__ __forceinline__ long long divide(long long a, int b) {
  return (a >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b))
                        : a / b;
}

// The batch lies along a line on which a tile is kTileCost long and each sequence with a context
// starts with a stretch of P.seq_cost before its second tile, what its query and its rows cost.  The
// line is cut into equal ranges, and a tile belongs to the range in which it starts.  Cuts lie as far
// apart as two neighbouring starts at least, so no range is empty.
//
// What a sequence costs was measured with 2048 of them, of one tile each: a tile more with 5 to 8
// query heads in a unit, a sixth of one with fewer.  128 sequences of 128 to 8192 tokens in order of
// length, 64 query heads over 8 KV heads: 55.8 us (a cost of 0: 56.6, of 7: 56.1).
constexpr int kTileCost = 4;
constexpr int kSeqCostMany = 4;
constexpr int kSeqCostFew = 1;

// A line of length `total` in `ranges` pieces: the first `extra` of them are base + 1 long, the
// others base.
struct Cut {
  long long base;
  int extra;
  __device__ __forceinline__ Cut(long long total, int ranges) {
    base = ranges > 0 ? divide(total, ranges) : 0;
    extra = static_cast<int>(total - base * ranges);
  }
  __device__ __forceinline__ long long begin(int r) const { return base * r + min(r, extra); }
  // The range that holds point x.
  __device__ __forceinline__ int of(long long x) const {
    const long long big = (base + 1) * extra;
    return static_cast<int>(x < big ? x / (base + 1) : extra + (x - big) / base);
  }
};

// Finds range r; called by all THREADS threads of the CTA.  `notes` (one CTA of each range):
// say so where a context length is outside the block table, and leave P.info[r], which the
// merge grid reads: the sequence that begins in the range and goes on past it, if there is one.
// `lens` (shared memory, may be null) receives the context lengths of the range's first sequence
// and of the kLens - 1 behind it.
constexpr int kLens = 64;
template <int THREADS>
__device__ Span find_span(const Fp4Params& P, int r, bool notes, int* lens) {
  constexpr int W = THREADS / 32;
  __shared__ long long warp_tiles[W];
  __shared__ int warp_seqs[W];
  __shared__ int found_s, found_tile;
  __shared__ long long found[2];  // the batch's tiles before the range's begin and before its end
  __shared__ int2 past;           // the sequence that the range's end cuts (or -1), and its last range
  __shared__ long long past_first;  // and the batch's tiles before it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = P.max_blocks_per_seq * P.block_size;
  const int per = (P.num_seqs + THREADS - 1) / THREADS;
  const int s0 = min(P.num_seqs, tid * per), s1 = min(P.num_seqs, s0 + per);
  long long own = 0;
  int own_seqs = 0;
  for (int s = s0; s < s1; ++s) {
    const int L = P.context_lens[s];
    if (notes && r == 0 && (L < 0 || L > cap)) raise_error(P.err, PKV_DERR_CONTEXT);
    own += (min(max(L, 0), cap) + kTile - 1) / kTile;
    own_seqs += min(L, cap) > 0;
  }
  long long incl = own;
  int seqs = own_seqs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    const int z = __shfl_up_sync(0xffffffffu, seqs, o);
    if (lane >= o) {
      incl += y;
      seqs += z;
    }
  }
  if (lane == 31) {
    warp_tiles[warp] = incl;
    warp_seqs[warp] = seqs;
  }
  if (tid == 0) past = make_int2(-1, 0);
  __syncthreads();
  long long before = incl - own, total = 0;
  int before_seqs = seqs - own_seqs, total_seqs = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) {
      before += warp_tiles[w];
      before_seqs += warp_seqs[w];
    }
    total += warp_tiles[w];
    total_seqs += warp_seqs[w];
  }
  // (few tiles: as many ranges as can be, whatever they cost)
  const int cost = total >= 4LL * P.ranges ? P.seq_cost : 0;
  const long long line = total * kTileCost + static_cast<long long>(total_seqs) * cost;
  const int ranges = static_cast<int>(min(static_cast<long long>(P.ranges), total));
  const Cut cuts(line, ranges);
  const long long begin = r < ranges ? cuts.begin(r) : line;
  const long long end = r < ranges ? cuts.begin(r + 1) : line;
  const long long at = before * kTileCost + static_cast<long long>(before_seqs) * cost;
  const long long own_end = at + own * kTileCost + static_cast<long long>(own_seqs) * cost;
  // The first tile that starts at point x or behind it, x lying in sequence s of this thread, whose
  // `tiles` tiles begin with the batch's tile `first`: its number in the sequence, or `tiles` (then it
  // is the next sequence's first).  `last` is where the sequence's last tile starts.
  auto tile_at = [&](long long x, int& s, long long& first, int& tiles, long long& last) {
    long long start = at;
    first = before;
    for (s = s0;; ++s) {  // one of them holds it
      tiles = (live_len(P, s) + kTile - 1) / kTile;
      const long long length = tiles > 0 ? static_cast<long long>(tiles) * kTileCost + cost : 0;
      if (x < start + length) break;
      start += length;
      first += tiles;
    }
    last = tiles > 1 ? start + cost + static_cast<long long>(tiles - 1) * kTileCost : start;
    if (x == start) return 0;
    const long long in = x - start - cost;
    return in <= kTileCost ? 1 : static_cast<int>((in + kTileCost - 1) / kTileCost);
  };
  int s, tiles;
  long long first, last;
  if (at <= begin && begin < own_end) {
    int tile = tile_at(begin, s, first, tiles, last);
    found[0] = first + tile;
    if (tile >= tiles) {  // r < ranges: a tile starts in the range, so a sequence with tiles follows
      tile = 0;
      do ++s;
      while (live_len(P, s) == 0);
    }
    found_s = s;
    found_tile = tile;
  }
  if (at <= end && end < own_end) {
    const int tile = tile_at(end, s, first, tiles, last);
    found[1] = first + tile;
    if (notes && tile > 0 && tile < tiles) {
      past = make_int2(s, cuts.of(last));
      past_first = first;
    }
  } else if (tid == 0 && end >= line) {
    found[1] = total;
  }
  __syncthreads();
  Span sp;
  sp.tiles = r < ranges ? static_cast<int>(found[1] - found[0]) : 0;
  sp.s = sp.tiles > 0 ? found_s : 0;
  sp.tile = sp.tiles > 0 ? found_tile : 0;
  // (a sequence that begins before the range is noted by the range it begins in)
  if (notes && tid == 0 && P.ranges > 1)
    P.info[r] = sp.tiles > 0 && past.x >= 0 && past_first >= found[0] ? past : make_int2(-1, 0);
  if (lens != nullptr) {
    for (int i = max(s0, sp.s); i < min(s1, sp.s + kLens); ++i) lens[i - sp.s] = live_len(P, i);
    __syncthreads();
  }
  return sp;
}

// The part of one sequence that a range holds.
struct Segment {
  int s, L, t0, t1;  // tokens [t0, t1) of sequence s, whose context is L
  bool whole;        // all of the sequence: its rows are written, not left as partials
  int slot;          // partial slot: 0 = the sequence began before the range, 1 = it goes on
};

__device__ __forceinline__ Segment next_segment(const Fp4Params& P, int& s, int& tile,
                                                int& left) {
  Segment g;
  int L = live_len(P, s);
  while (L == 0) L = live_len(P, ++s);  // left > 0: a sequence with tiles follows
  const int tiles = (L + kTile - 1) / kTile;
  const int n = min(left, tiles - tile);
  g.s = s;
  g.L = L;
  g.t0 = tile * kTile;
  g.t1 = min(L, (tile + n) * kTile);
  g.whole = n == tiles;
  g.slot = tile > 0 ? 0 : 1;
  left -= n;
  tile = 0;
  ++s;
  return g;
}

template <typename T>
__device__ __forceinline__ void zero_empty_rows(const Fp4Params& P, int D, int r, int h0, int hc,
                                                int tid, int threads) {
  for (int s = r; s < P.num_seqs; s += P.ranges) {
    if (live_len(P, s) > 0) continue;
    T* out = static_cast<T*>(P.out) + (static_cast<size_t>(s) * P.num_q_heads + h0) * D;
    for (int i = tid; i < hc * D; i += threads) out[i] = from_f32<T>(0.f);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

#include "decode_fp4_umma.cuh"

// ------------------------------------------------------------------------------------------
// CUDA-core path: any type, head_dim 32, 64, 128 or 256, any block size
// ------------------------------------------------------------------------------------------
//
// A lane holds head_dim / 32 neighbouring elements of each row and of each query head.  A warp takes
// U tokens at a time, whose rows it loads together; their U HN dot products (at most 32) are summed
// over the lanes by one exchange that leaves each lane with the score of one (token, head), so the
// softmax of all of them takes one exponential per lane, and the weights go back by broadcasts.
// The loads in flight bound it (U rows of head_dim / 2 bytes per warp), and with several heads the
// exchanges.  64 contexts of 1024 to 2048 tokens, 32 query and KV heads: head_dim 64 214 us, with U 16
// 304 and with 8 404; head_dim 256 325, with U 32, for which registers lack, 432 and with 8 425.

constexpr int simt_tokens(int HN, int E) { return HN == 1 && E >= 4 ? 16 : 32 / HN; }

// A lane's E codes of a row, in the low bits.
template <int E>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* row, int lane) {
  if constexpr (E == 1)
    return __ldg(row + (lane >> 1)) >> (4 * (lane & 1));
  else if constexpr (E == 2)
    return __ldg(row + lane);
  else if constexpr (E == 4)
    return __ldg(reinterpret_cast<const uint16_t*>(row) + lane);
  else
    return __ldg(reinterpret_cast<const uint32_t*>(row) + lane);
}

template <typename T, int E, int HN>
__global__ void __launch_bounds__(kSimtThreads) decode_fp4_simt_kernel(const Fp4Params P) {
  constexpr int D = 32 * E;
  constexpr int U = simt_tokens(HN, E), N = U * HN;
  constexpr int G = 32 / N;  // lanes that hold the same (head, token)
  __shared__ float o_s[kSimtWarps][HN][D];
  __shared__ float2 ml_s[kSimtWarps][HN];
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int own_u = lane / G % U, own_h = lane / (G * U);
  const int units = P.num_kv_heads * P.num_chunks;
  const int r = blockIdx.x / units, u0 = blockIdx.x - r * units;
  const int g = u0 / P.num_chunks, c = u0 - g * P.num_chunks;
  const int h0 = g * P.group + c * P.chunk, hc = min(P.chunk, P.group - c * P.chunk);
  const int BS = P.block_size;
  griddep_wait();
  const Span sp = find_span<kSimtThreads>(P, r, u0 == 0, nullptr);
  zero_empty_rows<T>(P, D, r, h0, hc, tid, kSimtThreads);

  int s = sp.s, tile = sp.tile, left = sp.tiles;
  while (left > 0) {
    const Segment seg = next_segment(P, s, tile, left);
    float qr[HN][E], acc[HN][E];
    const T* qs = static_cast<const T*>(P.q) +
                  (static_cast<size_t>(seg.s) * P.num_q_heads + h0) * D + lane * E;
#pragma unroll
    for (int h = 0; h < HN; ++h) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        qr[h][e] = h < hc ? to_f32(qs[h * D + e]) : 0.f;
        acc[h][e] = 0.f;
      }
    }
    float m = -INFINITY, l = 0.f;  // of head own_h; l over this lane's tokens alone
    const int32_t* bt = P.block_tables + static_cast<size_t>(seg.s) * P.max_blocks_per_seq;
    for (int tb = seg.t0 + warp * U; tb < seg.t1; tb += kSimtWarps * U) {
      // each lane finds its own token's row and scales; the rows' places go round by shuffles
      const int t = tb + own_u;
      const bool live = t < seg.t1;
      int own_row = -1;  // within the cache (num_blocks * block_size < 2^31), -1: reads as zeros
      float ks = 0.f, vs = 0.f;
      if (live) {
        const int j = t / BS, off = t - j * BS;
        const int id = __ldg(&bt[j]);
        if (id >= 0 && id < P.num_blocks) {
          own_row = id * BS + off;
          const size_t at = (static_cast<size_t>(id) * P.num_kv_heads + g) * BS + off;
          ks = __bfloat162float(P.k_scales[at]);
          vs = __bfloat162float(P.v_scales[at]);
        } else {
          raise_error(P.err, PKV_DERR_BLOCK_ID);
        }
      }
      uint32_t kw[U], vw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = __shfl_sync(0xffffffffu, own_row, u * G);
        kw[u] = vw[u] = 0;
        if (row >= 0) {
          const size_t at = (static_cast<size_t>(row) * P.num_kv_heads + g) * (D / 2);
          kw[u] = load_codes<E>(P.k_cache + at, lane);
          vw[u] = load_codes<E>(P.v_cache + at, lane);
        }
      }
      float dot[N];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float kf[8];
        decode8(kw[u], 1.f, kf);
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          float d = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) d = fmaf(qr[h][e], kf[e], d);
          dot[h * U + u] = d;
        }
      }
      const float sum = reduce_heads(dot, [](float x, float y) { return x + y; });
      const float sl = live ? sum * (ks * P.scale_log2) : -INFINITY;
      float mn = sl;
#pragma unroll
      for (int o = G; o < G * U; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mn = fmaxf(m, mn);
      const float a = exp2f(m - mn), p = live ? exp2f(sl - mn) : 0.f;
      m = mn;
      l = fmaf(l, a, p);
      const float pv = p * vs;
#pragma unroll
      for (int h = 0; h < HN; ++h) {
        const float ah = __shfl_sync(0xffffffffu, a, h * U * G);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[h][e] *= ah;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float vf[8];
        decode8(vw[u], 1.f, vf);
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          const float w = __shfl_sync(0xffffffffu, pv, (h * U + u) * G);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[h][e] = fmaf(w, vf[e], acc[h][e]);
        }
      }
    }
#pragma unroll
    for (int o = G; o < G * U; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane % (G * U) == 0) ml_s[warp][own_h] = make_float2(m, l);
#pragma unroll
    for (int h = 0; h < HN; ++h)
#pragma unroll
      for (int e = 0; e < E; ++e) o_s[warp][h][lane * E + e] = acc[h][e];
    __syncthreads();
    for (int i = tid; i < hc * D; i += kSimtThreads) {
      const int h = i / D, d = i - h * D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kSimtWarps; ++w) M = fmaxf(M, ml_s[w][h].x);
      float num = 0.f, den = 0.f;
#pragma unroll
      for (int w = 0; w < kSimtWarps; ++w) {
        const float2 ml = ml_s[w][h];
        // a warp without a token of the segment has m = -inf, l = 0 and o = 0
        const float cw = ml.x == -INFINITY && ml.y == 0.f ? 0.f : exp2f(ml.x - M);
        num = fmaf(cw, o_s[w][h][d], num);
        den = fmaf(cw, ml.y, den);
      }
      const int head = h0 + h;
      if (seg.whole) {
        static_cast<T*>(P.out)[(static_cast<size_t>(seg.s) * P.num_q_heads + head) * D + d] =
            from_f32<T>(num / den);
      } else {
        const size_t idx = (static_cast<size_t>(r) * 2 + seg.slot) * P.num_q_heads + head;
        P.part_o[idx * D + d] = num;
        if (d == 0) P.part_ml[idx] = make_float2(M, den);
      }
    }
    __syncthreads();  // the merge buffers are read before the next segment writes them
  }
}

// ------------------------------------------------------------------------------------------
// Merge of the partials of sequences cut by a range's end
// ------------------------------------------------------------------------------------------

constexpr int kMergeWarps = 4;

// One CTA per (range, query head): if a sequence begins in the range and goes on past it,
// its partials are slot 1 of this range and slot 0 of every later range up to the last that
// holds tiles of it:
//   M = max m_p,  out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
// The threads first turn the (m, l) into weights; then warp w adds partials w, w + 4, ..., whose
// loads depend on nothing any more, eight at a time: a single sequence may have a partial in each
// range (131072 tokens, one KV head, 456 partials: 37 us a call with loads four at a time behind
// their weights, 31 like this).
template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_fp4_kernel(const Fp4Params P) {
  constexpr int V = D / 32;
  constexpr int kThreads = 32 * kMergeWarps;
  constexpr int kOwn = (kMaxRanges + kThreads - 1) / kThreads;
  using Vec = typename std::conditional<V == 1, float,
                                        typename std::conditional<V == 2, float2, float4>::type>::type;
  constexpr int kVecs = V * sizeof(float) / sizeof(Vec);
  __shared__ float red[2][kMergeWarps];
  __shared__ float weight[kMaxRanges];
  __shared__ float o_s[kMergeWarps][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.x, head = blockIdx.y;
  // No early launch of the grid behind this one: a decode CTA placed between merge CTAs leaves
  // their registers as gaps too small for a third decode CTA on the SM, and the CTAs left over run
  // after all others (32 contexts of 32k tokens: 277 us a call for 173).
  griddep_wait();
  const int2 info = __ldcg(&P.info[r]);
  if (info.x < 0) return;
  const int np = info.y - r + 1;
  auto index = [&](int p) {
    return (static_cast<size_t>(r + p) * 2 + (p == 0 ? 1 : 0)) * P.num_q_heads + head;
  };
  float2 ml[kOwn];
  float M = -INFINITY;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    const int p = tid + k * kThreads;
    ml[k] = p < np ? __ldcg(&P.part_ml[index(p)]) : make_float2(-INFINITY, 0.f);
  }
#pragma unroll
  for (int k = 0; k < kOwn; ++k) M = fmaxf(M, ml[k].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) M = fmaxf(M, red[0][w]);
  float den = 0.f;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    const int p = tid + k * kThreads;
    if (p < np) {
      const float w = exp2f(ml[k].x - M);
      weight[p] = w;
      den = fmaf(w, ml[k].y, den);
    }
  }
  den = warp_sum(den);
  if (lane == 0) red[1][warp] = den;
  __syncthreads();
  float acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll 8
  for (int p = warp; p < np; p += kMergeWarps) {
    const Vec* src = reinterpret_cast<const Vec*>(P.part_o + index(p) * D) + lane;
    const float w = weight[p];
    Vec x[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) x[k] = __ldcg(src + 32 * k);
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = fmaf(w, reinterpret_cast<const float*>(x)[k], acc[k]);
  }
  constexpr int kWide = V / kVecs;
#pragma unroll
  for (int k = 0; k < V; ++k) o_s[warp][(k / kWide * 32 + lane) * kWide + k % kWide] = acc[k];
  __syncthreads();
  den = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) den += red[1][w];
  T* out = static_cast<T*>(P.out) + (static_cast<size_t>(info.x) * P.num_q_heads + head) * D;
  for (int d = tid; d < D; d += kThreads) {
    float num = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) num += o_s[w][d];
    out[d] = from_f32<T>(num / den);
  }
}

// The same with a warp per (range, query head), for batches whose sequences have few partials: a
// quarter of the CTAs, all resident at once, and no exchange between warps.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_few_fp4_kernel(const Fp4Params P) {
  constexpr int V = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x, head = blockIdx.y * kMergeWarps + warp;
  griddep_wait();  // (no early launch of the grid behind this one, as above)
  const int2 info = __ldcg(&P.info[r]);
  if (info.x < 0 || head >= P.num_q_heads) return;
  const int np = info.y - r + 1;
  auto index = [&](int p) {
    return (static_cast<size_t>(r + p) * 2 + (p == 0 ? 1 : 0)) * P.num_q_heads + head;
  };
  float M = -INFINITY;
  for (int p = lane; p < np; p += 32) M = fmaxf(M, __ldcg(&P.part_ml[index(p)]).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[V], den = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
  for (int p0 = 0; p0 < np; p0 += 32) {
    const int p = p0 + lane, count = min(32, np - p0);
    float w = 0.f;
    if (p < np) {
      const float2 ml = __ldcg(&P.part_ml[index(p)]);
      w = exp2f(ml.x - M);
      den = fmaf(w, ml.y, den);
    }
#pragma unroll 4
    for (int j = 0; j < count; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const float* src = P.part_o + index(p0 + j) * D + lane;
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] = fmaf(wj, __ldcg(src + 32 * k), acc[k]);
    }
  }
  den = warp_sum(den);
  T* out = static_cast<T*>(P.out) + (static_cast<size_t>(info.x) * P.num_q_heads + head) * D + lane;
#pragma unroll
  for (int k = 0; k < V; ++k) out[32 * k] = from_f32<T>(acc[k] / den);
}

// ------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

struct Fp4Layout {
  int chunk, num_chunks, ranges;
  size_t o_offset, ml_offset, info_offset, total;
};

// Block sizes that the tensor-core kernel's copies serve: they divide a tile, and a block of one KV
// head is 8 rows of shared memory or more.
bool umma_shape(int head_dim, int block_size) {
  return head_dim == 128 && (block_size == 8 || block_size == 16 || block_size == 32 ||
                             block_size == 64 || block_size == 128);
}

Fp4Layout layout(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                 int max_blocks_per_seq) {
  Fp4Layout w{};
  const int group = num_q_heads / num_kv_heads;
  w.num_chunks = (group + kHeads - 1) / kHeads;
  w.chunk = (group + w.num_chunks - 1) / w.num_chunks;
  const long long units = static_cast<long long>(num_kv_heads) * w.num_chunks;
  const long long tiles =
      static_cast<long long>(num_seqs) *
      ((static_cast<long long>(max_blocks_per_seq) * block_size + kTile - 1) / kTile);
  const long long ctas = umma_shape(head_dim, block_size) ? kRangeCtas : kMaxRanges;
  w.ranges = static_cast<int>(std::max(1LL, std::min(ctas / units, tiles)));
  if (w.ranges <= 1) return w;
  const size_t rows = static_cast<size_t>(w.ranges) * 2 * num_q_heads;
  w.ml_offset = align_up(rows * head_dim * sizeof(float), 256);
  w.info_offset = w.ml_offset + align_up(rows * sizeof(float2), 256);
  w.total = w.info_offset + align_up(w.ranges * sizeof(int2), 256);
  return w;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// The codes of a cache as a 2-D tensor of 4-bit elements: x = num_kv_heads * 128, y = slots.
// A box is one block of one KV head: 128 elements (64 bytes, 128 in shared memory) a row.
bool make_codes_map(CUtensorMap* map, const void* base, int Hkv, long long slots, int block_size) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(Hkv) * 128, static_cast<cuuint64_t>(slots)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(Hkv) * 64};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(block_size)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<void*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using Fp4Fn = void (*)(const Fp4Params);
using UmmaFn = void (*)(CUtensorMap, CUtensorMap, Fp4Params);

// The tensor-core kernel of a unit of `chunk` query heads, and its shared memory.
template <typename T>
UmmaFn umma_for(int chunk, int& smem) {
  const int HN = chunk <= 1 ? 1 : chunk <= 2 ? 2 : chunk <= 4 ? 4 : 8;
  smem = u_smem(u_cols(u_terms<T>(), HN));
  switch (HN) {
    case 1: return decode_fp4_umma_kernel<T, 1>;
    case 2: return decode_fp4_umma_kernel<T, 2>;
    case 4: return decode_fp4_umma_kernel<T, 4>;
    default: return decode_fp4_umma_kernel<T, 8>;
  }
}

// Whether the tensor-core kernel serves a call.  Its products read 8-bit terms of 16-bit numbers,
// and its copies of scales 16 bytes.  It is the faster one of the two at every size measured: 11 us
// against 15 for one sequence of 100 tokens, 61 against 795 for 128 sequences of 128 to 8192 tokens
// with 8 query heads per KV head.
bool uses_umma(const DecodeFp4Args& a) {
  return a.dtype != PKV_F32 && umma_shape(a.head_dim, a.block_size) &&
         reinterpret_cast<uintptr_t>(a.k_scales) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(a.v_scales) % 16 == 0;
}

template <typename T, int E>
Fp4Fn simt_heads(int chunk) {
  return chunk <= 1   ? decode_fp4_simt_kernel<T, E, 1>
         : chunk <= 2 ? decode_fp4_simt_kernel<T, E, 2>
         : chunk <= 4 ? decode_fp4_simt_kernel<T, E, 4>
                      : decode_fp4_simt_kernel<T, E, 8>;
}

template <typename T>
Fp4Fn simt_for(int D, int chunk) {
  switch (D) {
    case 32: return simt_heads<T, 1>(chunk);
    case 64: return simt_heads<T, 2>(chunk);
    case 128: return simt_heads<T, 4>(chunk);
    case 256: return simt_heads<T, 8>(chunk);
    default: return nullptr;
  }
}

template <typename T>
Fp4Fn merge_for(int D, bool few) {
  switch (D) {
    case 32: return few ? merge_few_fp4_kernel<T, 32> : merge_fp4_kernel<T, 32>;
    case 64: return few ? merge_few_fp4_kernel<T, 64> : merge_fp4_kernel<T, 64>;
    case 128: return few ? merge_few_fp4_kernel<T, 128> : merge_fp4_kernel<T, 128>;
    case 256: return few ? merge_few_fp4_kernel<T, 256> : merge_fp4_kernel<T, 256>;
    default: return nullptr;
  }
}

}  // namespace

size_t decode_fp4_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                 int block_size, int max_blocks_per_seq) {
  return layout(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq)
      .total;
}

bool decode_fp4_supported(int head_dim, int block_size) {
  return (head_dim == 32 || head_dim == 64 || head_dim == 128 || head_dim == 256) &&
         block_size >= 1;
}

int launch_decode_fp4(const DecodeFp4Args& a, cudaStream_t stream) {
  const Fp4Layout w = layout(a.num_seqs, a.num_q_heads, a.num_kv_heads, a.head_dim, a.block_size,
                             a.max_blocks_per_seq);
  if (w.total > 0 && (a.workspace == nullptr || a.workspace_bytes < w.total)) return PKV_ENOMEM;
  Fp4Params P{};
  P.out = a.out;
  P.q = a.q;
  P.k_cache = static_cast<const uint8_t*>(a.k_cache);
  P.v_cache = static_cast<const uint8_t*>(a.v_cache);
  P.k_scales = static_cast<const __nv_bfloat16*>(a.k_scales);
  P.v_scales = static_cast<const __nv_bfloat16*>(a.v_scales);
  P.block_tables = a.block_tables;
  P.context_lens = a.context_lens;
  char* ws = static_cast<char*>(a.workspace);
  if (w.total > 0) {
    P.part_o = reinterpret_cast<float*>(ws + w.o_offset);
    P.part_ml = reinterpret_cast<float2*>(ws + w.ml_offset);
    P.info = reinterpret_cast<int2*>(ws + w.info_offset);
  }
  P.err = a.err;
  P.num_seqs = a.num_seqs;
  P.num_q_heads = a.num_q_heads;
  P.num_kv_heads = a.num_kv_heads;
  P.group = a.num_q_heads / a.num_kv_heads;
  P.chunk = w.chunk;
  P.num_chunks = w.num_chunks;
  P.max_blocks_per_seq = a.max_blocks_per_seq;
  P.num_blocks = a.num_blocks;
  P.block_size = a.block_size;
  const bool umma = uses_umma(a);
  // The variant that has two CTAs on an SM takes as many ranges as are resident at a time (128
  // sequences of 2048 tokens, fp16, 8 query heads per KV head: 72 us, with half as many again 94).
  P.ranges = umma && a.dtype == PKV_F16 && w.chunk > 4
                 ? std::max(1, std::min(w.ranges, kRangeCtas * 2 / 3 / (a.num_kv_heads * w.num_chunks)))
                 : w.ranges;
  P.seq_cost = umma && w.chunk > 4 ? kSeqCostMany : kSeqCostFew;
  P.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  const long long grid = static_cast<long long>(P.ranges) * a.num_kv_heads * w.num_chunks;
  if (grid > INT_MAX || (P.ranges > 1 && a.num_q_heads > 65535)) return PKV_EUNSUPPORTED;
  const Fp4Fn fn = a.dtype == PKV_F32    ? simt_for<float>(a.head_dim, w.chunk)
                   : a.dtype == PKV_BF16 ? simt_for<__nv_bfloat16>(a.head_dim, w.chunk)
                                         : simt_for<__half>(a.head_dim, w.chunk);
  // At most five partials a sequence on average, if all are as long: a warp each takes them.  Measured
  // against a CTA each: 57 ranges and 128 sequences of 128 to 8192 tokens, 64 query heads, 59 us for 62;
  // 16 of 32k tokens 99 for 101, with 8 heads 91.5 for 91.0; a single long sequence has 57 partials in
  // a row, and CTAs of four warps take them.
  const bool few = P.ranges <= 4 * a.num_seqs;
  const Fp4Fn merge = a.dtype == PKV_F32    ? merge_for<float>(a.head_dim, few)
                      : a.dtype == PKV_BF16 ? merge_for<__nv_bfloat16>(a.head_dim, few)
                                            : merge_for<__half>(a.head_dim, few);
  if (!fn || !merge) return PKV_EUNSUPPORTED;
  // Both grids may be launched while the grid ahead of them drains, and wait for its end on the
  // device before they touch memory: that hides the launches and the first grid's set-up.
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  if (umma) {
    CUtensorMap kmap, vmap;
    const long long slots = static_cast<long long>(a.num_blocks) * a.block_size;
    if (!make_codes_map(&kmap, a.k_cache, a.num_kv_heads, slots, a.block_size) ||
        !make_codes_map(&vmap, a.v_cache, a.num_kv_heads, slots, a.block_size))
      return PKV_ECUDA;
    int smem = 0;
    const UmmaFn ufn = a.dtype == PKV_BF16 ? umma_for<__nv_bfloat16>(w.chunk, smem)
                                           : umma_for<__half>(w.chunk, smem);
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(ufn),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return PKV_ECUDA;
    cfg.blockDim = dim3(kUThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    if (cudaLaunchKernelEx(&cfg, ufn, kmap, vmap, P) != cudaSuccess) return PKV_ECUDA;
  } else {
    cfg.blockDim = dim3(kSimtThreads);
    if (cudaLaunchKernelEx(&cfg, fn, P) != cudaSuccess) return PKV_ECUDA;
  }
  if (P.ranges > 1) {
    cfg.gridDim = dim3(static_cast<unsigned>(P.ranges - 1), static_cast<unsigned>(
                       few ? (a.num_q_heads + kMergeWarps - 1) / kMergeWarps : a.num_q_heads));
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, merge, P) != cudaSuccess) return PKV_ECUDA;
  }
  return PKV_OK;
}

}  // namespace pkv
