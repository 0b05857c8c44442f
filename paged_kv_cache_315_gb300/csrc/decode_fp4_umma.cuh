// decode_fp4_umma.cuh -- 4-bit decode on the 5th-generation tensor cores: head_dim 128, query
// and output in 16 bits, block sizes 8, 16, 32, 64 and 128.  Included by decode_fp4.cu.
//
// Why tensor cores: a token and KV head bring 132 bytes, so at the copy bandwidth of HBM an
// SM has about 6 clocks for each of them, some 24 warp instructions.  Turning its 256 codes
// into 16-bit operands of mma.sync alone takes more than half of that.  kind::f8f6f4 reads the
// codes as they are: TMA spreads a row's 64 bytes over 128 (4-bit elements lie 16 to a 16-byte
// chunk) and no thread touches a code.
//
// Both products have the tile's 128 tokens or the 128 dimensions as M, and the query heads as
// N, on the smallest N the instruction has:
//     S^T [128 tokens x heads] = K . Q^T       (A = K rows, K-major; B = Q, E4M3)
//     O^T [128 dims x heads]   = V^T . P^T     (A = V rows, MN-major; B = P, E4M3)
// so thread t of the four softmax warps owns token t of S^T and dimension t of O^T.
//
// The 8-bit operands B carry 16-bit precision as sums of E4M3 terms in columns of their own:
// x 2^e = x_0 + x_1 / 16 + x_2 / 256, where x_i is what the terms before it leave, times
// 16^i, rounded to E4M3's 4 significant bits.  Two terms hold a bf16 number exactly (8 bits:
// after 4 rounded bits the rest is a multiple of 2^-7 below 2^-4), three terms an fp16 number.
//   - Q: e per head, from its largest element, so that |q 2^e| < 256; below 2^-9 / 16 of that
//     range, 2^-22 of the largest element, bits are lost.
//   - P: the weights of one tile relative to that tile's own largest score, times the V scale
//     over the tile's largest V scale, times 256.  A weight is lost only below 2^-21 of the
//     tile's largest one, whatever the running maximum is: a token that takes nearly all of the
//     weight cannot push the many small ones of other tiles out of range.
// Since a tile has its own reference, O^T is not accumulated in tensor memory: each tile's
// product is added to fp32 registers, times 2^(m_tile - m) (2^e of the V scales), where the
// running reference m only moves when a tile exceeds it by 2^64.
//
// Codes have no NaN, so rows that no copy wrote (past the context, or of an earlier tile) only
// need a weight of zero.
//
// Roles: warps 0-3 softmax and output, warp 4 loads K tiles, warp 5 issues the products, warp 6
// loads V tiles, warp 7 scales, notes and each sequence's query; the last four walk the range's
// tiles each for itself.  K, V, S and O are double buffered, and the products run ahead: S(i + 1)
// is issued before O(i), so the tensor cores score a tile while the softmax warps work on the one
// before.  The small scales and notes have four slots.  Buffers are released like this:
//   - the K slot of tile i by S(i), the V slot and the P buffer by O(i);
//   - the S buffer by P(i), which follows its reading; S(i + 2) waits for it;
//   - the O buffer by P(i + 2): O(i) is read before P(i + 2) arrives;
//   - the scales and notes of tile i (four slots) by S(i + 2), which waits for P(i), which follows
//     their reading; a query buffer by the last S that reads it.
// The barrier of S(i) also counts the arrival of tile i's scales and notes: one wait for the
// softmax warps instead of two.
// A wait by parity must not be lapped: a warp may wait for a barrier's use by tile i only while
// the use by the next tile of that slot cannot complete without the warp itself (K(i + 2) and
// scales(i + 2) are what S(i + 2)'s barrier waits for, V(i + 2) what O(i + 2)'s does).
// HBM's copy bandwidth gives each of three CTAs on an SM 2150 clocks for a tile, and the warps'
// chains have to stay below that one by one.  With all loads in one warp that warp was the bound
// (16 TMA copies of a 16-token block each, at 45-60 clocks from an elected thread in straight-line
// code, 80 from eight lanes side by side).  The registers follow the roles: 80 a thread at launch,
// then 88 for softmax warps and 72 for the others.
//
// Measured on one GB300 (clocks per tile and SM at 1.92 GHz, 700 being the copy bandwidth): 16
// contexts of 32k tokens with 1, 2, 4 and 8 query heads for each of 8 KV heads take 806, 814, 826 and
// 886 with the start and the merge (91 to 99 us); 32 of them with 4 heads 169-173 us, 6.4-6.6 TB/s.
// Up to 4 heads HBM bounds the steady state.  With 8 the softmax warps' chain does: 2400 clocks a
// tile in each of the three CTAs, 1600 of them work, with 60% of the issue slots taken.  A call
// starts with 6 us to the first scores (launch, range, block ids, K), and a sequence of one tile
// costs a CTA twice what a tile inside a long one does, by its query and its rows.

constexpr int kUTileBytes = kTile * 128;  // a K or V tile in shared memory (64 of 128 bytes data)
constexpr int kUThreads = 256;
constexpr int kTries = 1 << 18;  // of a wait: a second, at the 4 us that hardware holds each
constexpr int kUScaleBytes = 4 * 2 * kTile * 2;  // [4 slots][K, V][128 tokens] bf16

// Terms of a 16-bit number, and the columns of S and O: term * HN + head, padded to an N that
// the instruction has for M = 128.
template <typename T>
constexpr int u_terms() { return std::is_same<T, __half>::value ? 3 : 2; }
__host__ __device__ constexpr int u_cols(int terms, int HN) { return terms * HN <= 16 ? 16 : 32; }
__host__ __device__ constexpr int u_smem(int NC) {
  return 1024 + 4 * kUTileBytes + 2 * NC * 128 + NC * kTile + kUScaleBytes + 1600;
}

// What the warps tell each other, behind the tiles.
struct alignas(16) USmem {
  int4 meta[4];          // per tile: flags, sequence, live tokens
  float f[4][2][kHeads]; // per sequence: score factor of each head, and its negative
  float top[2][4][kHeads];
  uint32_t vtop[2][4];
  float lsum[2][4][kHeads];  // per sequence: the warps' sums of weights
  uint64_t bars[15];
  int lens[kLens];       // of the range's first sequence and those behind it
  int4 rows[2][4];       // of K, of V: the cache row of each block of a tile
  uint32_t tmem;
};
static_assert(sizeof(USmem) <= 1600, "bookkeeping area");

enum { kFirst = 1, kLast = 2, kWhole = 4, kSlot1 = 8, kSeqShift = 4 };  // and sequence mod 4

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ uint32_t redux_max(uint32_t v) {
  return __reduce_max_sync(0xffffffffu, v);
}

// Barrier of the softmax warps; true if `ok` was true in all of them.  Every one of them
// comes to each of these barriers whatever its own waits gave, so that none is left behind.
__device__ __forceinline__ bool softmax_sync_and(bool ok) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(ok))
      : "memory");
  return r != 0;
}

// 16 bytes from global to shared memory, and an arrival on `bar` once this thread's copies
// before it are complete.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The `np` blocks of a tile, `step` bytes apart in shared memory, from the cache rows in `rows`;
// issued by one thread.
__device__ __forceinline__ void load_blocks(uint32_t dst, uint32_t step, const CUtensorMap* map,
                                            uint32_t bar, int x, const int4* rows, int np,
                                            uint32_t bytes) {
  mbar_arrive_expect_tx(bar, bytes);
#pragma unroll 2
  for (int p = 0; p < np; p += 4, dst += 4 * step) {
    const int4 y = rows[p >> 2];
    tma_load_2d(dst, map, bar, x, y.x);
    if (p + 1 < np) tma_load_2d(dst + step, map, bar, x, y.y);
    if (p + 2 < np) tma_load_2d(dst + 2 * step, map, bar, x, y.z);
    if (p + 3 < np) tma_load_2d(dst + 3 * step, map, bar, x, y.w);
  }
}

__device__ __forceinline__ float pow2_bits(int field) {
  return __uint_as_float(static_cast<uint32_t>(field) << 23);
}

// Combines the lanes' values of each head: every step halves the heads a lane still holds, so H
// heads take H + 4 - log2(H) exchanges instead of 5 H.  Returns head lane / (32 / H)'s result.
template <int H, typename Op>
__device__ __forceinline__ float reduce_heads(const float (&v)[H], Op op) {
  const int lane = threadIdx.x & 31;
  float x[H];
#pragma unroll
  for (int h = 0; h < H; ++h) x[h] = v[h];
  int o = 16;
#pragma unroll
  for (int c = H / 2; c > 0; c >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int h = 0; h < c; ++h) {
      const float give = up ? x[h] : x[h + c], keep = up ? x[h + c] : x[h];
      x[h] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
#pragma unroll
  for (; o > 0; o >>= 1) x[0] = op(x[0], __shfl_xor_sync(0xffffffffu, x[0], o));
  return x[0];
}

// Two heads' fp32 values in a register pair, for the instructions that work on both.  (One head
// alone has a pair's other half unused.)
using Pair = unsigned long long;

__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(Pair p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Columns that a row of S or O is read in.
template <int N>
__device__ __forceinline__ void read_columns(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 24) {
    uint32_t a[16], b[8];
    tmem_ld(taddr, a);
    tmem_ld(taddr + 16, b);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = a[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[16 + i] = b[i];
  } else if constexpr (N == 12) {
    uint32_t a[8], b[4];
    tmem_ld(taddr, a);
    tmem_ld(taddr + 8, b);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = a[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[8 + i] = b[i];
  } else if constexpr (N == 6 || N == 3) {
    uint32_t a[N == 6 ? 8 : 4];
    tmem_ld(taddr, a);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = a[i];
  } else {
    tmem_ld(taddr, r);
    tmem_ld_wait();
  }
}

// The sum of each head's terms.
template <int NT, int HN>
__device__ __forceinline__ void join_terms(const uint32_t (&r)[NT * HN], Pair (&v)[(HN + 1) / 2]) {
  auto term = [&](int q, int h) {
    return pair(__uint_as_float(r[q * HN + h]), h + 1 < HN ? __uint_as_float(r[q * HN + h + 1]) : 0.f);
  };
#pragma unroll
  for (int h = 0; h < HN; h += 2) {
    v[h / 2] = fma2(term(1, h), pair(0.0625f, 0.0625f), term(0, h));
    if constexpr (NT == 3) v[h / 2] = fma2(term(2, h), pair(0.00390625f, 0.00390625f), v[h / 2]);
  }
}

// Waits for the phase of `bar` with the given parity; false when that takes more than kTries tries.
// The plain try_wait is one instruction in which the hardware holds the thread for a while (given a
// time to hold it becomes a loop of its own, with sleeps and clock reads).  A limit on tries rather
// than on time keeps the loop small: five roles' code shares an SM's instruction caches, and with
// clock reads at every wait the kernel was 1-3% slower.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < kTries; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

// Registers of a thread from here on, for the four warps of a warpgroup.
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The context lengths that a range's walks meet, the first kLens of them in shared memory.
struct Lens {
  const int* near;
  int s0;
  __device__ __forceinline__ int of(const Fp4Params& P, int s) const {
    return s - s0 < kLens ? near[s - s0] : live_len(P, s);
  }
};

// The tiles of a range in order.
struct Walk {
  int s, L, tile;  // the tile's sequence, its context length, the tile within it
  bool first;      // the sequence's first tile in this range

  __device__ __forceinline__ void next_sequence(const Fp4Params& P, const Lens& lens) {
    do {
      L = lens.of(P, ++s);
    } while (L == 0);
    tile = 0;
  }
  // the sequence ends with this tile
  __device__ __forceinline__ bool ends() const { return (tile + 1) * kTile >= L; }
  // (not called behind the range's last tile: a sequence with tiles follows)
  __device__ __forceinline__ void advance(const Fp4Params& P, const Lens& lens) {
    first = ends();
    if (first)
      next_sequence(P, lens);
    else
      ++tile;
  }
};

// The block ids of a range's tiles.  They come 32 at a time, one per lane, and one window ahead:
// under load a row of the block table takes longer to arrive than a tile takes.
struct Ids {
  int s, j, id;         // the lane's id is that of logical block j + lane of sequence s
  int ns, nj, nid, nL;  // the window behind it, and its sequence's length

  __device__ __forceinline__ int load(const Fp4Params& P, int seq, int L, int j0) const {
    const int x = j0 + static_cast<int>(threadIdx.x & 31);
    return static_cast<long long>(x) * P.block_size < L
               ? __ldg(&P.block_tables[static_cast<size_t>(seq) * P.max_blocks_per_seq + x])
               : -1;
  }
  __device__ __forceinline__ void load_next(const Fp4Params& P, const Lens& lens) {
    nj = j + 32;
    if (static_cast<long long>(nj) * P.block_size >= nL) {
      nj = nL = 0;
      while (++ns < P.num_seqs && (nL = lens.of(P, ns)) == 0) {
      }
    }
    nid = load(P, ns, nL, nj);
  }
  __device__ __forceinline__ void begin(const Fp4Params& P, const Lens& lens, const Walk& w,
                                        int pages) {
    s = ns = w.s;
    nL = w.L;
    j = w.tile * pages / 32 * 32;
    id = load(P, s, w.L, j);
    load_next(P, lens);
  }
  // This lane's block of the walk's tile, `block` saying whether it has one: its id, or -1 (and
  // an error) where that is out of range.
  __device__ __forceinline__ int of(const Fp4Params& P, const Lens& lens, const Walk& w, int pages,
                                    bool block) {
    if (w.s != s || w.tile * pages >= j + 32) {
      s = ns;
      j = nj;
      id = nid;
      load_next(P, lens);
    }
    int x = __shfl_sync(0xffffffffu, id, (w.tile * pages - j + (threadIdx.x & 31)) & 31);
    if (block && static_cast<unsigned>(x) >= static_cast<unsigned>(P.num_blocks)) {
      raise_error(P.err, PKV_DERR_BLOCK_ID);
      x = -1;
    }
    return x;
  }
};

template <typename T, int HN>
__global__ void __launch_bounds__(kUThreads, u_cols(u_terms<T>(), HN) == 16 ? 3 : 2)
    decode_fp4_umma_kernel(const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, const Fp4Params P) {
  constexpr int D = 128;
  constexpr int NT = u_terms<T>();
  constexpr int COLS = NT * HN;
  constexpr int NC = u_cols(NT, HN);
  constexpr uint32_t kIdS = umma_idesc_e2m1_e4m3(kTile, NC, false, false);
  constexpr uint32_t kIdO = umma_idesc_e2m1_e4m3(D, 16, true, true);
  constexpr uint32_t kTmemCols = NC == 16 ? 64 : 128;
  // 4 (kManyRegs + kFewRegs) registers of 4 warps are what 8 warps have at launch: 80 or 128 each
  constexpr int kManyRegs = NC == 16 ? 88 : 168, kFewRegs = NC == 16 ? 72 : 88;
  extern __shared__ uint8_t smem_raw[];
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = P.num_kv_heads * P.num_chunks;
  const int r = blockIdx.x / units, u = blockIdx.x - r * units;
  const int g = u / P.num_chunks, c = u - g * P.num_chunks;
  const int h0 = g * P.group + c * P.chunk, hc = min(P.chunk, P.group - c * P.chunk);
  const int BS = P.block_size;
  uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* k_tiles = base;
  uint8_t* v_tiles = k_tiles + 2 * kUTileBytes;
  uint8_t* q_rows = v_tiles + 2 * kUTileBytes;        // [2][NC][128], 128-byte swizzle
  uint8_t* p_rows = q_rows + 2 * NC * 128;            // [NC / 16][128 tokens][16]
  __nv_bfloat16* scales = reinterpret_cast<__nv_bfloat16*>(p_rows + NC * kTile);
  USmem& sm = *reinterpret_cast<USmem*>(reinterpret_cast<uint8_t*>(scales) + kUScaleBytes);
  // barriers: K, V loaded, S, O complete, P written, Q written, Q read (two slots each), drain
  enum { kK = 0, kV, kS, kP, kO, kQ };
  auto bar = [&](int kind, int slot) { return smem_addr(&sm.bars[2 * kind + slot]); };
  auto query_free_bar = [&](int seg) { return smem_addr(&sm.bars[12 + (seg & 1)]); };
  const uint32_t drain_bar = smem_addr(&sm.bars[14]);

  if (tid == 0) {
    // P: four warps; S: the products, every lane's copies of scales, and the notes
    for (int k = 0; k < 15; ++k)
      mbar_init(smem_addr(&sm.bars[k]), k / 2 == kP ? 4 : k / 2 == kS ? 34 : 1);
    fence_mbar_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  // query rows of absent heads and terms stay zero
  for (int i = tid; i < 2 * NC * 128 / 16; i += kUThreads)
    reinterpret_cast<uint4*>(q_rows)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 5) {
    tmem_alloc(smem_addr(&sm.tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  griddep_wait();  // nothing above depends on what the grid ahead writes
  // (synchronises all threads; u == 0 also leaves the merge's notes)
  const Span sp = find_span<kUThreads>(P, r, u == 0, sm.lens);
  tc_fence_after_sync();
  const int n = sp.tiles;
  const uint32_t tm_s = sm.tmem, tm_o = tm_s + 2 * NC;

  // A whole warp's wait; false when it ran out (the call's output is void): the warp ends its role,
  // and the others' waits for it run out in turn.
  bool failed = false;
  auto warp_wait_bar = [&](uint32_t at, uint32_t parity) -> bool {
    failed = !__all_sync(0xffffffffu, wait_phase(at, parity));
    return !failed;
  };
  // The same for tile i's use of a two-slot barrier.
  auto warp_wait = [&](int kind, int i) {
    return warp_wait_bar(bar(kind, i & 1), (i >> 1) & 1);
  };

  if (warp >= 4) {
    fewer_registers<kFewRegs>();
    const int pages = kTile / BS;
    const Lens lens{sm.lens, sp.s};
    Walk w{sp.s, n > 0 ? sm.lens[0] : 0, sp.tile, true};
    if (warp == 4 || warp == 6) {
      // ---- K tiles (warp 4), V tiles (warp 6) ----------------------------------------------
      const bool is_k = warp == 4;
      const int kind = is_k ? kK : kV, freed = is_k ? kS : kO;
      const CUtensorMap* map = is_k ? &kmap : &vmap;
      const uint32_t tiles = smem_addr(is_k ? k_tiles : v_tiles);
      int4* rows = sm.rows[is_k ? 0 : 1];
      Ids ids;
      int i = 0;
      if (n > 0) ids.begin(P, lens, w, pages);
      for (; i < n; ++i) {
        const int b = i & 1;
        const int valid = min(kTile, w.L - w.tile * kTile);
        const bool block = lane * BS < valid;  // this lane has a block
        const int np = (valid + BS - 1) / BS;
        const int id = ids.of(P, lens, w, pages, block);
        // (an id out of range reads zeros, past the cache's end)
        if (block) reinterpret_cast<int*>(rows)[lane] = (id >= 0 ? id : P.num_blocks) * BS;
        __syncwarp();
        if (i >= 2 && !warp_wait(freed, i - 2)) break;
        if (elect_one())
          load_blocks(tiles + b * kUTileBytes, BS * 128, map, bar(kind, b), g * D, rows, np,
                      np * BS * 64);
        __syncwarp();
        if (i + 1 < n) w.advance(P, lens);
      }
      // after a wait that ran out, no copy may be in flight when the CTA ends
      if (i < n && lane == 0)
        for (int j = max(0, i - 2); j < i; ++j)
          mbar_wait_for(bar(kind, j & 1), (j >> 1) & 1, kWaitLimitNs / 8);
    } else if (warp == 5) {
      // ---- products -------------------------------------------------------------------------
      const uint64_t dk = smem_desc_sw128(smem_addr(k_tiles), 16, 1024);
      const uint64_t dv = smem_desc_sw128(smem_addr(v_tiles), 1024, 1024);
      const uint64_t dq = smem_desc_sw128(smem_addr(q_rows), 16, 1024);
      const uint64_t dp = smem_desc_plain(smem_addr(p_rows), 128, 128);
      constexpr uint64_t kSlot = kUTileBytes / 16;
      int seg = -1;
      for (int j = 0; n > 0 && j <= n; ++j) {
        const int b = j & 1;
        if (j < n) {
          // S(j) overwrites S(j - 2), which was read before P(j - 2) arrived; this warp waited
          // for that arrival when it issued O(j - 2)
          if (!warp_wait(kK, j)) break;
          if (w.first) {
            ++seg;
            if (!warp_wait(kQ, seg)) break;
          }
          if (elect_one()) {
            tc_fence_after_sync();
            const uint64_t a = dk + b * kSlot, q = dq + (seg & 1) * (NC * 8);
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              umma_f8_ss(tm_s + b * NC, a + kk * 2, q + kk * 2, kIdS, kk > 0 ? 1u : 0u);
            umma_commit(bar(kS, b));
            if (w.ends()) umma_commit(query_free_bar(seg));
          }
          __syncwarp();
          if (j + 1 < n) w.advance(P, lens);
        }
        if (j > 0) {
          // O(i) overwrites O(i - 2), which was read before P(i) arrived
          const int i = j - 1, bi = i & 1;
          if (!warp_wait(kV, i) || !warp_wait(kP, i)) break;
          if (elect_one()) {
            tc_fence_after_sync();
            const uint64_t a = dv + bi * kSlot;
#pragma unroll
            for (int half = 0; half < NC / 16; ++half) {
#pragma unroll
              for (int kk = 0; kk < kTile / 32; ++kk)
                umma_f8_ss(tm_o + bi * NC + half * 16, a + kk * 256, dp + half * kTile + kk * 32,
                           kIdO, kk > 0 ? 1u : 0u);
            }
            umma_commit(bar(kO, bi));
          }
          __syncwarp();
        }
      }
      // every product is complete before tensor memory is released
      if (elect_one()) {
        umma_commit(drain_bar);
        failed = !mbar_wait_bounded(drain_bar, 0) || failed;
      }
    } else {
      // ---- scales, notes, queries -----------------------------------------------------------
      // Queries are prepared one sequence ahead: `query` walks the sequences, whose first tile is
      // the range's tile `query_at`.
      Walk query = w;
      int query_at = 0, query_seg = 0;
      uint2 qraw[HN];
      auto load_query = [&]() {
        const T* q = static_cast<const T*>(P.q) +
                     (static_cast<size_t>(query.s) * P.num_q_heads + h0) * D + 4 * lane;
#pragma unroll
        for (int h = 0; h < HN; ++h)
          qraw[h] = h < hc ? __ldg(reinterpret_cast<const uint2*>(q + h * D)) : make_uint2(0, 0);
      };
      // The query rows as E4M3 terms; false when a wait ran out.
      auto put_query = [&]() -> bool {
        const int buf = query_seg & 1;
        if (query_seg >= 2 && !warp_wait_bar(query_free_bar(buf), ((query_seg - 2) >> 1) & 1))
          return false;
        uint8_t* rows = q_rows + buf * NC * 128;
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          float x[4];
          const float2 a = Mma<T>::unpack(qraw[h].x), bb = Mma<T>::unpack(qraw[h].y);
          x[0] = a.x, x[1] = a.y, x[2] = bb.x, x[3] = bb.y;
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
          top = redux_max(top);
          // |x| 2^(134 - E) < 256 for the exponent field E of the largest; a query that is not
          // finite becomes NaN, and a scale of zero leaves scores of zero
          const int E = max(8, static_cast<int>(top >> 23));
          float up = P.scale_log2 == 0.f ? 0.f : pow2_bits(261 - E);
          if (E == 255) up = __uint_as_float(0x7fffffffu);
          float factor = P.scale_log2 == 0.f ? 1.f : fabsf(P.scale_log2) * pow2_bits(E - 7);
          if (factor < FLT_MIN) factor = FLT_MIN;  // masked scores times it stay -inf
          // (S of the sequence two before is complete, so the softmax warps are done with the one
          // four before, whose place this is)
          if (lane == 0) {
            sm.f[query_seg & 3][0][h] = factor;
            sm.f[query_seg & 3][1][h] = -factor;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] *= up;
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            const uint32_t lo = f32x2_to_e4m3x2(x[0], x[1]), hi = f32x2_to_e4m3x2(x[2], x[3]);
            const int row = q * HN + h;
            *reinterpret_cast<uint32_t*>(rows + row * 128 + (((lane >> 2) ^ (row & 7)) << 4) +
                                         (lane & 3) * 4) = lo | (hi << 16);
            const uint32_t w0 = e4m3x2_to_f16x2(lo), w1 = e4m3x2_to_f16x2(hi);
            const float2 f0 = Mma<__half>::unpack(w0), f1 = Mma<__half>::unpack(w1);
            x[0] = (x[0] - f0.x) * 16.f;
            x[1] = (x[1] - f0.y) * 16.f;
            x[2] = (x[2] - f1.x) * 16.f;
            x[3] = (x[3] - f1.y) * 16.f;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kQ, buf));
        query_at += (query.L + kTile - 1) / kTile - query.tile;
        ++query_seg;
        if (query_at < n) {
          query.next_sequence(P, lens);
          load_query();
        }
        return true;
      };
      // the 16 lanes of K and of V take the scales of 8 tokens each
      const int chunk_page = 8 * (lane & 15) / BS, chunk_off = 8 * (lane & 15) - chunk_page * BS;
      const __nv_bfloat16* scale_src =
          (lane < 16 ? P.k_scales : P.v_scales) + static_cast<size_t>(g) * BS + chunk_off;
      const uint32_t scale_dst = smem_addr(scales + (lane >> 4) * kTile + 8 * (lane & 15));
      const size_t scale_block = static_cast<size_t>(P.num_kv_heads) * BS;
      Ids ids;
      int i = 0, seg = 0, first_tile = sp.tile;
      if (n > 0) {
        load_query();
        ids.begin(P, lens, w, pages);
        put_query();
      }
      for (; i < n; ++i) {
        const int valid = min(kTile, w.L - w.tile * kTile);
        const int id = ids.of(P, lens, w, pages, lane * BS < valid);
        const int cid = __shfl_sync(0xffffffffu, lane * BS < valid ? id : -1, chunk_page);
        const int flags = (w.first ? kFirst : 0) | (w.ends() || i + 1 == n ? kLast : 0) |
                          (first_tile == 0 && w.ends() ? kWhole : 0) |
                          (first_tile == 0 ? kSlot1 : 0) | (seg & 3) << kSeqShift;
        if (i >= 2 && !warp_wait(kS, i - 2)) break;
        // (a plain asynchronous copy: TMA takes about as long for 32 bytes as for a block of codes)
        const uint32_t dst = scale_dst + (i & 3) * (4 * kTile);
        if (cid >= 0)
          copy16_async(dst, scale_src + cid * scale_block);
        else
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
        __syncwarp();
        copy_async_arrive(bar(kS, i & 1));
        if (lane == 0) {
          sm.meta[i & 3] = make_int4(flags, w.s, valid, 0);
          mbar_arrive(bar(kS, i & 1));
        }
        __syncwarp();
        // the query of the next sequence, whose buffer frees with the first product of this one
        if (w.first && query_at < n && !put_query()) break;
        if (i + 1 < n) {
          w.advance(P, lens);
          if (w.first) {
            first_tile = 0;
            ++seg;
          }
        }
      }
      if (i < n && lane == 0)
        for (int j = max(0, i - 1); j <= i; ++j)
          mbar_wait_for(bar(kS, j & 1), (j >> 1) & 1, kWaitLimitNs / 8);
      __syncwarp();
      // rows of sequences without a context, dealt out over the ranges
      for (int s0 = r; s0 < P.num_seqs; s0 += 32 * P.ranges) {
        const long long s = s0 + static_cast<long long>(lane) * P.ranges;
        uint32_t empty = __ballot_sync(0xffffffffu, s < P.num_seqs && live_len(P, s) == 0);
        for (; empty != 0; empty &= empty - 1) {
          const size_t row = s0 + static_cast<size_t>(__ffs(empty) - 1) * P.ranges;
          T* out = static_cast<T*>(P.out) + (row * P.num_q_heads + h0) * D;
          for (int e = lane; e < hc * D; e += 32) out[e] = from_f32<T>(0.f);
        }
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: token tid of S^T, dimension tid of O^T -----------------------------------
    more_registers<kManyRegs>();
    const uint32_t lane_off = static_cast<uint32_t>(32 * warp) << 16;
    // Sums of weights l and outputs acc are relative to a running reference, held as its negative
    // nm.  A tile's product joins acc one iteration later, and a sequence's rows are written when P
    // of the next tile is on its way: nothing waits for a product just issued.
    constexpr int HP = (HN + 1) / 2;
    Pair acc[HP], l[HP], nm[HP], beta[HP];
    const float sign = P.scale_log2 < 0.f ? -1.f : 1.f;
    int before = 0, before_s = 0;  // flags and sequence of the tile before
    bool ok = true;
#pragma unroll
    for (int p = 0; p < HP; ++p) acc[p] = 0;
    // (whether all four warps go on after a wait is decided at the barriers below)
    // acc += O(i) beta.  The columns are read before P(i + 2) arrives, which lets another product
    // overwrite them.
    auto add_output = [&](int i) {
      uint32_t o[COLS];
      Pair v[HP];
      tc_fence_after_sync();
      read_columns<COLS>(tm_o + lane_off + (i & 1) * NC, o);
      tc_fence_before_sync();
      join_terms<NT, HN>(o, v);
#pragma unroll
      for (int p = 0; p < HP; ++p) acc[p] = fma2(v[p], beta[p], acc[p]);
    };
    // The rows of the sequence that ended with the tile before.
    auto write_rows = [&]() {
      const int seq = (before >> kSeqShift) & 1;
      Pair den[HP];  // > 0, or NaN
#pragma unroll
      for (int p = 0; p < HP; ++p) {
        auto part = [&](int w) { return *reinterpret_cast<const Pair*>(&sm.lsum[seq][w][2 * p]); };
        den[p] = add2(add2(part(0), part(1)), add2(part(2), part(3)));
      }
      if (before & kWhole) {
        T* out = static_cast<T*>(P.out) +
                 (static_cast<size_t>(before_s) * P.num_q_heads + h0) * D + tid;
#pragma unroll
        for (int p = 0; p < HP; ++p) {
          float a0, a1, d0, d1;
          split(acc[p], a0, a1);
          split(den[p], d0, d1);
          if (2 * p < hc) out[2 * p * D] = from_f32<T>(__fdividef(a0, d0));
          if (2 * p + 1 < hc) out[(2 * p + 1) * D] = from_f32<T>(__fdividef(a1, d1));
          acc[p] = 0;
        }
      } else {
        const size_t idx =
            (static_cast<size_t>(r) * 2 + ((before & kSlot1) ? 1 : 0)) * P.num_q_heads + h0;
        float* part = P.part_o + idx * D + tid;
#pragma unroll
        for (int p = 0; p < HP; ++p) {
          float a0, a1, d0, d1;
          split(acc[p], a0, a1);
          split(den[p], d0, d1);
          if (2 * p < hc) part[2 * p * D] = a0;
          if (2 * p + 1 < hc) part[(2 * p + 1) * D] = a1;
          if (tid == 0 && 2 * p < hc) P.part_ml[idx + 2 * p].y = d0;
          if (tid == 0 && 2 * p + 1 < hc) P.part_ml[idx + 2 * p + 1].y = d1;
          acc[p] = 0;
        }
      }
    };
    for (int i = 0; i < n; ++i) {
      const int b = i & 1;
      ok = ok && warp_wait(kS, i);
      const int4 meta = sm.meta[i & 3];
      const int flags = meta.x;
      const __nv_bfloat16* sc = scales + (i & 3) * 2 * kTile + tid;
      const float ks = __bfloat162float(sc[0]) * sign;
      float vs = __bfloat162float(sc[kTile]);
      // scores but for the head's factor f > 0, which the exponent below applies
      Pair x[HP];
      float xs[2 * HP];  // their halves
      if (ok) {
        uint32_t sr[COLS];
        tc_fence_after_sync();
        read_columns<COLS>(tm_s + lane_off + b * NC, sr);
        tc_fence_before_sync();
        join_terms<NT, HN>(sr, x);
#pragma unroll
        for (int p = 0; p < HP; ++p) x[p] = mul2(x[p], pair(ks, ks));
      } else {
#pragma unroll
        for (int p = 0; p < HP; ++p) x[p] = 0;
      }
      if (meta.z < kTile && tid >= meta.z) {  // past the context
        vs = 0.f;
#pragma unroll
        for (int p = 0; p < HP; ++p) x[p] = pair(-INFINITY, -INFINITY);
      }
#pragma unroll
      for (int p = 0; p < HP; ++p) split(x[p], xs[2 * p], xs[2 * p + 1]);
      // the tile's largest score of each head and largest |V scale|
      {
        float t[HN];
#pragma unroll
        for (int h = 0; h < HN; ++h) t[h] = redux_max(xs[h]);
        const uint32_t tv = redux_max(__float_as_uint(vs) & 0x7fffffffu);
        if (lane == 0) {
#pragma unroll
          for (int h = 0; h < HN; ++h) sm.top[b][warp][h] = t[h];
          sm.vtop[b][warp] = tv;
        }
      }
      // the product of the tile before (it has read the buffer of the weights); beta is that tile's
      if (i > 0 && (ok = ok && warp_wait(kO, i - 1))) add_output(i - 1);
      ok = softmax_sync_and(ok);
      if (!ok) break;
      // (the query's factors are in place: they were written before the first tile's notes)
      const int seq = flags >> kSeqShift;
      Pair nt[HP], d[HP];  // nt: the tile's reference in log2 units, negated
      float most = -INFINITY;
      const uint32_t tv = max(max(sm.vtop[b][0], sm.vtop[b][1]), max(sm.vtop[b][2], sm.vtop[b][3]));
#pragma unroll
      for (int p = 0; p < HP; ++p) {
        const int h = 2 * p;
        auto top = [&](int w) { return *reinterpret_cast<const float2*>(&sm.top[b][w][h]); };
        const float2 t0 = top(0), t1 = top(1), t2 = top(2), t3 = top(3);
        nt[p] = mul2(pair(fmaxf(max3(t0.x, t1.x, t2.x), t3.x), fmaxf(max3(t0.y, t1.y, t2.y), t3.y)),
                     *reinterpret_cast<const Pair*>(&sm.f[seq][1][h]));
      }
      // |vs| 2^(134 - E) < 256 for the exponent field E of the largest
      const int E = min(254, max(8, static_cast<int>(tv >> 23)));
      const float cv = tv >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : vs * pow2_bits(261 - E);
      const float back = pow2_bits(E - 7);
      if (flags & kFirst) {
#pragma unroll
        for (int p = 0; p < HP; ++p) {
          nm[p] = nt[p];
          l[p] = 0;
        }
      }
      // how far the tile's reference exceeds the running one
#pragma unroll
      for (int p = 0; p < HP; ++p) {
        d[p] = fma2(nt[p], pair(-1.f, -1.f), nm[p]);
        float lo, hi;
        split(d[p], lo, hi);
        most = HN == 1 ? lo : max3(most, lo, hi);
      }
      if (most > 64.f) {  // the running reference moves
#pragma unroll
        for (int p = 0; p < HP; ++p) {
          float n0, n1, t0, t1;
          split(nm[p], n0, n1);
          split(nt[p], t0, t1);
          const float m0 = fminf(n0, t0), m1 = fminf(n1, t1);
          const Pair a = pair(fast_exp2(m0 - n0), fast_exp2(m1 - n1));
          acc[p] = mul2(acc[p], a);
          l[p] = mul2(l[p], a);
          nm[p] = pair(m0, m1);
          d[p] = pair(m0 - t0, m1 - t1);
        }
      }
      uint32_t w[HP];  // the weights times the V scale, as fp16 pairs
#pragma unroll
      for (int p = 0; p < HP; ++p) {
        float lo, hi;
        split(d[p], lo, hi);
        d[p] = pair(fast_exp2(lo), HN == 1 ? 0.f : fast_exp2(hi));  // to the running reference
        split(fma2(x[p], *reinterpret_cast<const Pair*>(&sm.f[seq][0][2 * p]), nt[p]), lo, hi);
        const Pair e = pair(fast_exp2(lo), HN == 1 ? 0.f : fast_exp2(hi));
        l[p] = fma2(e, d[p], l[p]);
        split(mul2(e, pair(cv, cv)), lo, hi);
        w[p] = Mma<__half>::pack(lo, HN == 1 ? 0.f : hi);
      }
      // the weights' E4M3 terms: byte term * HN + head of the token's row
      {
        uint32_t code[NT][HP];
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int p = 0; p < HP; ++p) {
            code[q][p] = f16x2_to_e4m3x2(w[p]);
            if (q + 1 < NT) {
              const uint32_t got = e4m3x2_to_f16x2(code[q][p]);
              const __half2 rest = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&w[p]),
                                                   *reinterpret_cast<const __half2*>(&got)),
                                           __float2half2_rn(16.f));
              w[p] = *reinterpret_cast<const uint32_t*>(&rest);
            }
          }
        uint32_t row[NC / 4];
        if constexpr (HN >= 4) {
#pragma unroll
          for (int k = 0; k < NC / 4; ++k) {
            const int q = 4 * k / HN, p = (4 * k - q * HN) / 2;
            row[k] = q < NT ? __byte_perm(code[q < NT ? q : 0][p], code[q < NT ? q : 0][p + 1], 0x5410)
                            : 0u;
          }
        } else {
          uint32_t first = 0;  // all terms fit 8 bytes
          uint32_t second = 0;
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            const uint32_t bits = HN == 1 ? code[q][0] & 0xffu : code[q][0];
            const int at = q * HN;
            if (at < 4)
              first |= bits << (8 * at);
            else
              second |= bits << (8 * (at - 4));
          }
          row[0] = first;
          row[1] = second;
          row[2] = row[3] = 0u;
        }
#pragma unroll
        for (int half = 0; half < NC / 16; ++half)
          *reinterpret_cast<uint4*>(p_rows + half * 16 * kTile + tid * 16) =
              make_uint4(row[4 * half], row[4 * half + 1], row[4 * half + 2], row[4 * half + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kP, b));
      if (before & kLast) write_rows();  // while the tensor cores work on this tile
#pragma unroll
      for (int p = 0; p < HP; ++p) beta[p] = mul2(d[p], pair(back, back));
      if (flags & kLast) {
        float ls[2 * HP], some[HN];
#pragma unroll
        for (int p = 0; p < HP; ++p) split(l[p], ls[2 * p], ls[2 * p + 1]);
#pragma unroll
        for (int h = 0; h < HN; ++h) some[h] = ls[h];
        const float sum = reduce_heads(some, [](float p, float q) { return p + q; });
        if (lane % (32 / HN) == 0) sm.lsum[seq & 1][warp][lane / (32 / HN)] = sum;
        if (!(flags & kWhole) && tid == 0) {
          const size_t idx =
              (static_cast<size_t>(r) * 2 + ((flags & kSlot1) ? 1 : 0)) * P.num_q_heads + h0;
#pragma unroll
          for (int h = 0; h < HN; ++h) {
            float both[2];
            split(nm[h / 2], both[0], both[1]);
            if (h < hc) P.part_ml[idx + h].x = -both[h & 1];
          }
        }
      }
      before = flags;
      before_s = meta.y;
      // (a wait that ran out shows at the next barrier)
    }
    if (n > 0) {  // the last tile; every warp comes to this barrier
      if ((ok = ok && warp_wait(kO, n - 1))) add_output(n - 1);
      ok = softmax_sync_and(ok);
      if (ok) write_rows();  // (a range's last tile ends its sequence's part)
    }
    tc_fence_before_sync();
  }
  if (failed) raise_error(P.err, PKV_DERR_TIMEOUT);
  __syncthreads();
  if (warp == 5) {
    tc_fence_after_sync();
    tmem_dealloc(tm_s, kTmemCols);
  }
}
