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
// Roles: warps 0-3 softmax and output, warp 4 loads (K, V and scale tiles, and each sequence's
// query), warp 5 issues the products.  S, P and O are double buffered, and the products run
// ahead: S(i + 1) is issued before O(i), so the tensor cores score a tile while the softmax
// warps work on the one before.  Every buffer is released by a barrier that the releasing
// product or read implies:
//   - the K slot of tile i by S(i); the V slot, the P buffer, the scales and the notes by O(i),
//     which follows P(i), which follows their reading;
//   - the S buffer by P(i), the O buffer by P(i + 2): O(i) is read before P(i + 2) arrives.

constexpr int kUStages = 2;
constexpr int kUTileBytes = kTile * 128;  // a K or V tile in shared memory (64 of 128 bytes data)
constexpr int kUSoftmax = 128;
constexpr int kUThreads = 192;

// Terms of a 16-bit number, and the columns of S and O: term * HN + head, padded to an N that
// the instruction has for M = 128.
template <typename T>
constexpr int u_terms() { return std::is_same<T, __half>::value ? 3 : 2; }
__host__ __device__ constexpr int u_cols(int terms, int HN) { return terms * HN <= 16 ? 16 : 32; }
__host__ __device__ constexpr int u_smem(int NC) {
  return 1024 + 4 * kUTileBytes + 2 * NC * 128 + 2 * NC * kTile + 1024 + 704;
}

// What the warps tell each other, behind the tiles.
struct USmem {
  int4 meta[2];          // per tile slot: flags, sequence, live tokens
  float f[2][kHeads];    // per tile slot: score factor of each head, 2^-e scale log2(e)
  float top[2][4][kHeads];
  uint32_t vtop[2][4];
  float lsum[4][kHeads];
  uint64_t bars[16];
  uint32_t tmem;
  int qslot[2];          // per tile slot: query buffer | first tile of a sequence << 1
  volatile int abort;
};
static_assert(sizeof(USmem) <= 704, "bookkeeping area");

enum { kFirst = 1, kLast = 2, kWhole = 4, kSlot1 = 8 };

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

// Untiled bulk copy (16-byte aligned addresses and size) with completion on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float pow2_bits(int field) {
  return __uint_as_float(static_cast<uint32_t>(field) << 23);
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

// The sum of a head's terms.
template <int NT, int HN>
__device__ __forceinline__ float join_terms(const uint32_t (&r)[NT * HN], int h) {
  float v = fmaf(__uint_as_float(r[HN + h]), 0.0625f, __uint_as_float(r[h]));
  if constexpr (NT == 3) v = fmaf(__uint_as_float(r[2 * HN + h]), 0.00390625f, v);
  return v;
}

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
  extern __shared__ uint8_t smem_raw[];
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = P.num_kv_heads * P.num_chunks;
  const int r = blockIdx.x / units, u = blockIdx.x - r * units;
  const int g = u / P.num_chunks, c = u - g * P.num_chunks;
  const int h0 = g * P.group + c * P.chunk, hc = min(P.chunk, P.group - c * P.chunk);
  const int BS = P.block_size;
  const Span sp = find_span<kUThreads>(P, r, u == 0);  // u == 0 also leaves the merge's notes
  zero_empty_rows<T>(P, D, r, h0, hc, tid, kUThreads);
  if (sp.tiles == 0) return;
  const int n = sp.tiles;

  uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* k_tiles = base;
  uint8_t* v_tiles = k_tiles + 2 * kUTileBytes;
  uint8_t* q_rows = v_tiles + 2 * kUTileBytes;        // [2][NC][128], 128-byte swizzle
  uint8_t* p_rows = q_rows + 2 * NC * 128;            // [2][NC / 16][128 tokens][16]
  __nv_bfloat16* scales = reinterpret_cast<__nv_bfloat16*>(p_rows + 2 * NC * kTile);
  USmem& sm = *reinterpret_cast<USmem*>(reinterpret_cast<uint8_t*>(scales) + 1024);
  // bars: K full, V full, scales full, S full, P full, O full, Q full (two each), drain
  auto bar = [&](int kind, int slot) { return smem_addr(&sm.bars[2 * kind + slot]); };
  enum { kK = 0, kV, kSc, kS, kP, kO, kQ, kDrain };

  if (tid == 0) {
    for (int kind = kK; kind <= kDrain; ++kind)
      for (int b = 0; b < 2; ++b) mbar_init(bar(kind, b), kind == kP ? 4 : 1);
    sm.abort = 0;
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
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm_s = sm.tmem, tm_o = tm_s + 2 * NC;

  auto fail = [&]() {
    raise_error(P.err, PKV_DERR_TIMEOUT);
    sm.abort = 1;
  };
  // one lane's wait for tile i's use of a two-slot barrier, for the whole warp
  auto warp_wait = [&](int kind, int i) -> bool {
    int ok = 1;
    if (lane == 0) {
      ok = mbar_wait_bounded(bar(kind, i & 1), (i >> 1) & 1) ? 1 : 0;
      if (!ok) fail();
      if (sm.abort) ok = 0;
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();  // what lane 0 acquired holds for the whole warp
    return ok != 0;
  };

  if (warp == 4) {
    // ---- loads ----------------------------------------------------------------------------
    const int pages = kTile / BS;
    int lens_at = sp.s, lens = 0;  // context lengths of 32 sequences, one per lane
    auto load_lens = [&](int s) {
      lens_at = s;
      lens = s + lane < P.num_seqs ? live_len(P, s + lane) : 0;
    };
    auto len_of = [&](int s) {
      if (s >= lens_at + 32) load_lens(s);
      return __shfl_sync(0xffffffffu, lens, s - lens_at);
    };
    auto load_id = [&](int s, int tile, int L) {
      const int j = tile * pages + lane;
      return lane < pages && j * BS < L
                 ? __ldg(&P.block_tables[static_cast<size_t>(s) * P.max_blocks_per_seq + j])
                 : -1;
    };
    uint2 qraw[HN];
    auto load_query = [&](int s) {
      const T* q = static_cast<const T*>(P.q) +
                   (static_cast<size_t>(s) * P.num_q_heads + h0) * D + 4 * lane;
#pragma unroll
      for (int h = 0; h < HN; ++h)
        qraw[h] = h < hc ? __ldg(reinterpret_cast<const uint2*>(q + h * D)) : make_uint2(0, 0);
    };
    load_lens(sp.s);
    int s = sp.s, tile = sp.tile, L = len_of(s), first_tile = tile, seg = 0;
    bool first = true;
    int id = load_id(s, tile, L);
    load_query(s);
    int i = 0;
    for (; i < n; ++i) {
      const int b = i & 1;
      const int cs = s, cL = L, ct = tile, cid = id;
      const bool cfirst = first;
      const int tiles = (cL + kTile - 1) / kTile;
      const bool clast = ct + 1 == tiles || i + 1 == n;
      const int valid = min(kTile, cL - ct * kTile);
      const int np = (valid + BS - 1) / BS;
      const bool good = lane < np && cid >= 0 && cid < P.num_blocks;
      if (lane < np && !good) raise_error(P.err, PKV_DERR_BLOCK_ID);
      const int y = (good ? cid : P.num_blocks) * BS;  // past the cache: reads zeros
      // the K slot: S(i - 2) has read it
      if (i >= 2 && !warp_wait(kS, i - 2)) break;
      if (lane == 0) {
        sm.qslot[b] = (seg & 1) | (cfirst ? 2 : 0);
        mbar_arrive_expect_tx(bar(kK, b), np * BS * 64);
      }
      __syncwarp();
      if (lane < np)
        tma_load_2d(smem_addr(k_tiles + b * kUTileBytes) + lane * BS * 128, &kmap, bar(kK, b),
                    g * D, y);
      float factor[HN];
      if (cfirst) {
        // the query rows as E4M3 terms.  The buffer's last reader was a product of the
        // sequence before the last one, no later than S(i - 2).
        uint8_t* rows = q_rows + (seg & 1) * NC * 128;
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
          // finite becomes NaN
          const int E = max(8, static_cast<int>(top >> 23));
          const float up = E == 255 ? __uint_as_float(0x7fffffffu) : pow2_bits(261 - E);
          factor[h] = P.scale_log2 * pow2_bits(E - 7);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] *= up;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint32_t lo = f32x2_to_e4m3x2(x[0], x[1]), hi = f32x2_to_e4m3x2(x[2], x[3]);
            const int row = t * HN + h;
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
        if (lane == 0) mbar_arrive(bar(kQ, seg & 1));
      }
      // what the next tile needs from global memory, while this one waits for its V slot
      int flags = (cfirst ? kFirst : 0) | (clast ? kLast : 0) |
                  (first_tile == 0 && ct + 1 == tiles ? kWhole : 0) |
                  (first_tile == 0 ? kSlot1 : 0);
      if (i + 1 < n) {
        first = ct + 1 == tiles;
        if (first) {
          ++s;
          while ((L = len_of(s)) == 0) ++s;
          tile = first_tile = 0;
          ++seg;
          load_query(s);
        } else {
          tile = ct + 1;
        }
        id = load_id(s, tile, L);
      }
      // the V slot, the scales and the tile's notes: O(i - 2) is complete, and P(i - 2), which
      // it waited for, came after the softmax warps had read tile i - 2's scales and notes
      if (i >= 2 && !warp_wait(kO, i - 2)) break;
      if (lane == 0) mbar_arrive_expect_tx(bar(kV, b), np * BS * 64);
      __syncwarp();
      if (lane < np)
        tma_load_2d(smem_addr(v_tiles + b * kUTileBytes) + lane * BS * 128, &vmap, bar(kV, b),
                    g * D, y);
      __nv_bfloat16* sk = scales + b * 2 * kTile + lane * BS;
      if (lane < np && !good) {
        for (int e = 0; e < BS; ++e) sk[e] = sk[kTile + e] = __float2bfloat16_rn(0.f);
        fence_proxy_async_smem();
      }
      const uint32_t copies = __popc(__ballot_sync(0xffffffffu, good));
      if (lane == 0) {
        sm.meta[b] = make_int4(flags, cs, valid, 0);
        if (cfirst) {
#pragma unroll
          for (int h = 0; h < HN; ++h) sm.f[b][h] = factor[h];
        }
        mbar_arrive_expect_tx(bar(kSc, b), copies * BS * 4);
      }
      __syncwarp();
      if (good) {
        const size_t at = (static_cast<size_t>(cid) * P.num_kv_heads + g) * BS;
        bulk_load(smem_addr(sk), P.k_scales + at, BS * 2, bar(kSc, b));
        bulk_load(smem_addr(sk + kTile), P.v_scales + at, BS * 2, bar(kSc, b));
      }
    }
    // after a wait that ran out, no copy may be in flight when the CTA ends
    if (i < n) {
      if (lane == 0) {
        for (int j = max(0, i - 2); j <= i; ++j) {
          if (j < i || j >= 2) mbar_wait_for(bar(kK, j & 1), (j >> 1) & 1, kWaitLimitNs / 8);
          if (j < i) {
            mbar_wait_for(bar(kV, j & 1), (j >> 1) & 1, kWaitLimitNs / 8);
            mbar_wait_for(bar(kSc, j & 1), (j >> 1) & 1, kWaitLimitNs / 8);
          }
        }
      }
      __syncwarp();
    }
  } else if (warp == 5) {
    // ---- products ---------------------------------------------------------------------------
    bool ok = true;
    int issued = 0, seg = -1;
    for (int j = 0; ok && j <= n; ++j) {
      const int b = j & 1;
      if (j < n) {
        // S(j) overwrites S(j - 2), which was read before P(j - 2) arrived; this warp waited
        // for that arrival when it issued O(j - 2)
        ok = warp_wait(kK, j);
        if (!ok) break;
        const int note = sm.qslot[b];
        if (note & 2) {
          ++seg;
          ok = warp_wait(kQ, seg);
          if (!ok) break;
        }
        if (lane == 0) {
          tc_fence_after_sync();
          const uint64_t dk = smem_desc_sw128(smem_addr(k_tiles + b * kUTileBytes), 16, 1024);
          const uint64_t dq =
              smem_desc_sw128(smem_addr(q_rows + (note & 1) * NC * 128), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            umma_f8_ss(tm_s + b * NC, dk + kk * 2, dq + kk * 2, kIdS, kk > 0 ? 1u : 0u);
          umma_commit(bar(kS, b));
        }
        __syncwarp();
        issued = 1;
      }
      if (j > 0) {
        // O(i) overwrites O(i - 2), which was read before P(i) arrived
        const int i = j - 1, bi = i & 1;
        ok = warp_wait(kP, i) && warp_wait(kV, i);
        if (!ok) break;
        if (lane == 0) {
          tc_fence_after_sync();
          const uint64_t dv = smem_desc_sw128(smem_addr(v_tiles + bi * kUTileBytes), 1024, 1024);
#pragma unroll
          for (int half = 0; half < NC / 16; ++half) {
            const uint64_t dp = smem_desc_plain(
                smem_addr(p_rows + bi * NC * kTile + half * 16 * kTile), 128, 128);
#pragma unroll
            for (int kk = 0; kk < kTile / 32; ++kk)
              umma_f8_ss(tm_o + bi * NC + half * 16, dv + kk * 256, dp + kk * 32, kIdO,
                         kk > 0 ? 1u : 0u);
          }
          umma_commit(bar(kO, bi));
        }
        __syncwarp();
      }
    }
    // every product is complete before tensor memory is released
    if (issued && lane == 0) {
      umma_commit(bar(kDrain, 0));
      if (!mbar_wait_bounded(bar(kDrain, 0), 0)) fail();
    }
    __syncwarp();
  } else {
    // ---- softmax: token tid of S^T, dimension tid of O^T -----------------------------------
    const uint32_t lane_off = static_cast<uint32_t>(32 * warp) << 16;
    float f[HN], acc[HN], l[HN], m[HN], beta[HN];
    bool ok = true;
    // every lane waits; whether all four warps go on is decided at the barriers below
    auto wait = [&](int kind, int i) -> bool {
      const bool got = mbar_wait_bounded(bar(kind, i & 1), (i >> 1) & 1);
      const bool all = __all_sync(0xffffffffu, got);
      if (!all && lane == 0) fail();
      return all;
    };
    auto add_output = [&](int i) {  // acc += O(i) beta
      uint32_t o[COLS];
      tc_fence_after_sync();
      read_columns<COLS>(tm_o + lane_off + (i & 1) * NC, o);
      tc_fence_before_sync();
#pragma unroll
      for (int h = 0; h < HN; ++h) acc[h] = fmaf(join_terms<NT, HN>(o, h), beta[h], acc[h]);
    };
    for (int i = 0; i < n; ++i) {
      const int b = i & 1;
      ok = ok && wait(kSc, i);
      const int4 meta = sm.meta[b];
      const int flags = meta.x;
      const bool live = tid < meta.z;
      const float ks = __bfloat162float(scales[b * 2 * kTile + tid]);
      const float vs = live ? __bfloat162float(scales[b * 2 * kTile + kTile + tid]) : 0.f;
      if (flags & kFirst) {
#pragma unroll
        for (int h = 0; h < HN; ++h) f[h] = sm.f[b][h];
      }
      ok = ok && wait(kS, i);
      float x[HN];
      if (ok) {
        uint32_t sr[COLS];
        tc_fence_after_sync();
        read_columns<COLS>(tm_s + lane_off + b * NC, sr);
        tc_fence_before_sync();
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          const float v = join_terms<NT, HN>(sr, h) * (ks * f[h]);
          x[h] = live ? v : -INFINITY;
        }
      } else {
#pragma unroll
        for (int h = 0; h < HN; ++h) x[h] = 0.f;
      }
      // the tile's largest score of each head and largest |V scale|
      {
        float t[HN];
#pragma unroll
        for (int h = 0; h < HN; ++h) t[h] = redux_max(x[h]);
        const uint32_t tv = redux_max(__float_as_uint(vs) & 0x7fffffffu);
        if (lane == 0) {
#pragma unroll
          for (int h = 0; h < HN; ++h) sm.top[b][warp][h] = t[h];
          sm.vtop[b][warp] = tv;
        }
      }
      ok = softmax_sync_and(ok);
      if (!ok) break;
      float t[HN];
#pragma unroll
      for (int h = 0; h < HN; ++h)
        t[h] = fmaxf(fmaxf(sm.top[b][0][h], sm.top[b][1][h]),
                     fmaxf(sm.top[b][2][h], sm.top[b][3][h]));
      const uint32_t tv = max(max(sm.vtop[b][0], sm.vtop[b][1]), max(sm.vtop[b][2], sm.vtop[b][3]));
      // |vs| 2^(134 - E) < 256 for the exponent field E of the largest
      const int E = min(254, max(8, static_cast<int>(tv >> 23)));
      const float cv = tv >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : vs * pow2_bits(261 - E);
      const float back = pow2_bits(E - 7);
      if (flags & kFirst) {
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          m[h] = t[h];
          acc[h] = 0.f;
          l[h] = 0.f;
        }
      } else {
        bool up = false;
#pragma unroll
        for (int h = 0; h < HN; ++h) up = up || t[h] > m[h] + 64.f;
        if (up) {
#pragma unroll
          for (int h = 0; h < HN; ++h) {
            const float mn = fmaxf(m[h], t[h]);
            const float a = fast_exp2(m[h] - mn);
            acc[h] *= a;
            l[h] *= a;
            beta[h] *= a;
            m[h] = mn;
          }
        }
      }
      float w[HN], bh[HN];
#pragma unroll
      for (int h = 0; h < HN; ++h) {
        bh[h] = fast_exp2(t[h] - m[h]);
        const float p = fast_exp2(x[h] - t[h]);
        l[h] = fmaf(p, bh[h], l[h]);
        w[h] = p * cv;
      }
      // the weights' E4M3 terms: byte term * HN + head of the token's row
      {
        uint32_t row[NC / 4];
#pragma unroll
        for (int k = 0; k < NC / 4; ++k) row[k] = 0u;
#pragma unroll
        for (int h = 0; h < HN; h += 2) {
          uint32_t a = Mma<__half>::pack(w[h], h + 1 < HN ? w[h + 1] : 0.f);
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            const uint32_t code = f16x2_to_e4m3x2(a);
            const int at = q * HN + h;
            if constexpr (HN == 1)
              row[at >> 2] |= (code & 0xffu) << (8 * (at & 3));
            else
              row[at >> 2] |= code << (8 * (at & 3));
            if (q + 1 < NT) {
              const uint32_t back2 = e4m3x2_to_f16x2(code);
              const __half2 rest = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&a),
                                                   *reinterpret_cast<const __half2*>(&back2)),
                                           __float2half2_rn(16.f));
              a = *reinterpret_cast<const uint32_t*>(&rest);
            }
          }
        }
#pragma unroll
        for (int half = 0; half < NC / 16; ++half)
          *reinterpret_cast<uint4*>(p_rows + b * NC * kTile + half * 16 * kTile + tid * 16) =
              make_uint4(row[4 * half], row[4 * half + 1], row[4 * half + 2], row[4 * half + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kP, b));
      // the output of the tile before, of the same sequence, while the tensor cores work on
      // this one's; it is read before P(i + 1) arrives, which lets O(i + 1) overwrite it
      if (!(flags & kFirst)) {
        ok = wait(kO, i - 1);
        if (ok) add_output(i - 1);
      }
#pragma unroll
      for (int h = 0; h < HN; ++h) beta[h] = bh[h] * back;
      if (flags & kLast) {
        ok = ok && wait(kO, i);
        if (ok) add_output(i);
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          const float sum = warp_sum(l[h]);
          if (lane == 0) sm.lsum[warp][h] = sum;
        }
        ok = softmax_sync_and(ok);
        if (!ok) break;
        const bool whole = flags & kWhole;
        const size_t idx = (static_cast<size_t>(r) * 2 + ((flags & kSlot1) ? 1 : 0)) *
                               P.num_q_heads + h0;
#pragma unroll
        for (int h = 0; h < HN; ++h) {
          if (h < hc) {
            const float den = (sm.lsum[0][h] + sm.lsum[1][h]) + (sm.lsum[2][h] + sm.lsum[3][h]);
            if (whole) {
              static_cast<T*>(P.out)[(static_cast<size_t>(meta.y) * P.num_q_heads + h0 + h) * D +
                                     tid] = from_f32<T>(acc[h] / den);
            } else {
              P.part_o[(idx + h) * D + tid] = acc[h];
              if (tid == 0) P.part_ml[idx + h] = make_float2(m[h], den);
            }
          }
        }
      }
      // (a wait that ran out shows at the next of the barriers)
    }
    tc_fence_before_sync();
  }
  __syncthreads();
  if (warp == 5) {
    tc_fence_after_sync();
    tmem_dealloc(tm_s, kTmemCols);
  }
}
