// cache_fp4.cu -- quantising writes into and reads out of the 4-bit cache (sm_103a).
//
// A row is the head_dim elements of one token and one KV head.  Its scale is the bf16
// nearest to amax / 6 (6 is the largest E2M1 magnitude) and each element's code the E2M1
// value nearest to x / scale, ties to the even code.  Both kernels are byte movement with a
// little arithmetic: per element the write reads 2 bytes (16-bit types) and stores half a
// byte, and at the copy bandwidth of HBM an SM has 14 clocks for 128 of them, that is 14
// instructions for each element of a lane.
#include <algorithm>
#include <type_traits>

#include "device_common.cuh"
#include "fp4.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWriteCtas = 4, kReadCtas = 5;  // on an SM; the grids hold no more than are resident
constexpr int kElems = 8;        // elements of a run: 16 bytes of a 16-bit type
constexpr int kLaneElems = 16;   // elements a lane holds of a row, in runs D / 2 (or D / 4) apart

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[kElems]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Mma<T>::unpack(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// 16 bytes of values: 8 of a 16-bit type, or the first 4.
template <typename T>
__device__ __forceinline__ void store_run(T* p, const float (&x)[kElems]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    uint4 a;
    a.x = Mma<T>::pack(x[0], x[1]);
    a.y = Mma<T>::pack(x[2], x[3]);
    a.z = Mma<T>::pack(x[4], x[5]);
    a.w = Mma<T>::pack(x[6], x[7]);
    *reinterpret_cast<uint4*>(p) = a;
  }
}

// The IEEE quotient x / d, given r, the correctly rounded reciprocal of d: with y = x r and
// e = y d - x (exact in one FMA), y - e r is the correctly rounded quotient (Markstein, 1990), three
// operations where the division takes some ten.  With e taken this way round a zero keeps its sign:
// x = -0 gives y = -0, e = +0 and -0 r + y = -0.  Divisors near the ends of fp32's range, where e or
// r could leave it, take the division.
__device__ __forceinline__ float quotient(float x, float d, float r) {
  const float y = x * r, e = fmaf(y, d, -x);
  return fmaf(-e, r, y);
}

// The 8 codes (element 0 in the lowest four bits) of x / scale.
__device__ __forceinline__ uint32_t encode8(const float (&x)[kElems], float scale) {
  uint32_t word = 0;
  if (scale > 0x1p-100f && scale < 0x1p100f) {
    const float r = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      word |= f32x2_to_e2m1x2(quotient(x[2 * i], scale, r), quotient(x[2 * i + 1], scale, r))
              << (8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      word |= f32x2_to_e2m1x2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale))
              << (8 * i);
  }
  return word;
}

// The largest of three magnitudes, NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

// A row of D elements is held by D / 16 lanes of a warp, two runs of 8 in each.  Returns its codes
// and, in `scale`, its scale (the same in each of those lanes).
template <int D>
__device__ __forceinline__ uint2 quantise(const float (&x)[2][kElems], __nv_bfloat16& scale) {
  // magnitudes' bits order like the magnitudes, and a NaN above infinity above every number
  float most[2];
#pragma unroll
  for (int c = 0; c < 2; ++c)
    most[c] = max_abs(max_abs(x[c][0], x[c][1], x[c][2]), max_abs(x[c][3], x[c][4], x[c][5]),
                      max_abs(x[c][6], x[c][7], 0.f));
  uint32_t top = __float_as_uint(max_abs(most[0], most[1], 0.f));
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (top >= 0x7f800000u) {  // a NaN or an infinity in the row: every element reads as NaN
    scale = __ushort_as_bfloat16(0x7fff);
    return make_uint2(0, 0);
  }
  const float amax = __uint_as_float(top);
  scale = __float2bfloat16_rn(amax > 0x1p-100f ? quotient(amax, 6.f, 1.f / 6.f)
                                               : __fdiv_rn(amax, 6.f));
  const float s = __bfloat162float(scale);
  return s > 0.f ? make_uint2(encode8(x[0], s), encode8(x[1], s)) : make_uint2(0, 0);
}

// The (token, head) rows a group of lanes takes, `stride` rows apart, without a division in the
// loop.
struct RowWalk {
  long long row;
  int token, head, heads, step_tokens, step_heads;
  __device__ __forceinline__ RowWalk(long long first, long long stride, int num_heads)
      : row(first), heads(num_heads) {
    token = static_cast<int>(first / heads);
    head = static_cast<int>(first - static_cast<long long>(token) * heads);
    step_tokens = static_cast<int>(stride / heads);
    step_heads = static_cast<int>(stride - static_cast<long long>(step_tokens) * heads);
  }
  __device__ __forceinline__ void next(long long stride) {
    row += stride;
    token += step_tokens;
    head += step_heads;
    if (head >= heads) {
      head -= heads;
      ++token;
    }
  }
};

// Place of a row's scale.
__device__ __forceinline__ size_t scale_at(uint32_t slot, int head, int num_heads, int block_size) {
  const uint32_t block = slot / static_cast<uint32_t>(block_size);
  return (static_cast<size_t>(block) * num_heads + head) * block_size +
         (slot - block * static_cast<uint32_t>(block_size));
}

// One group of D / 16 lanes per (token, head) row, its key and its value row together.  131072 x 8
// bf16 rows take 135 us, 5.0 TB/s, with 67% of the issue slots taken and the loads' latency hidden by
// other CTAs alone.  With 8 elements a lane instead of 16 the exchanges, the scale and the addresses
// weigh twice as much: 174 us.  Four CTAs of one row a lane beat fewer of two rows (2 CTAs: 166 us, 3:
// 163) and more, which lack registers (5: 141, 6: 157).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kWriteCtas)
    write_fp4_kernel(const T* __restrict__ k, const T* __restrict__ v, uint8_t* __restrict__ kc,
                     uint8_t* __restrict__ vc, __nv_bfloat16* __restrict__ ks,
                     __nv_bfloat16* __restrict__ vs, const int64_t* __restrict__ slots,
                     long long num_rows, int num_heads, int block_size, long long num_slots,
                     unsigned* err) {
  constexpr int LPR = D / kLaneElems;
  const int sub = threadIdx.x % LPR;
  const long long stride = static_cast<long long>(gridDim.x) * (kThreads / LPR);
  RowWalk w(static_cast<long long>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR, stride,
            num_heads);
  // every lane of a warp runs the same number of iterations: the shuffles are warp-wide
  for (long long base = static_cast<long long>(blockIdx.x) * (kThreads / LPR); base < num_rows;
       base += stride) {
    const bool in = w.row < num_rows;
    const long long r = in ? w.row : num_rows - 1;
    const long long slot = in ? __ldg(&slots[w.token]) : -1;
    const int head = w.head;
    w.next(stride);
    float xk[2][kElems], xv[2][kElems];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      load8(k + r * D + (c * LPR + sub) * kElems, xk[c]);
      load8(v + r * D + (c * LPR + sub) * kElems, xv[c]);
    }
    __nv_bfloat16 sk, sv;
    const uint2 ck = quantise<D>(xk, sk), cv = quantise<D>(xv, sv);
    if (slot < 0) continue;  // padding, or past the last row
    if (slot >= num_slots) {
      if (head == 0 && sub == 0) raise_error(err, PKV_DERR_SLOT);
      continue;
    }
    const long long at = slot * num_heads + head;
    uint32_t* krow = reinterpret_cast<uint32_t*>(kc + at * (D / 2));
    uint32_t* vrow = reinterpret_cast<uint32_t*>(vc + at * (D / 2));
    krow[sub] = ck.x;
    krow[LPR + sub] = ck.y;
    vrow[sub] = cv.x;
    vrow[LPR + sub] = cv.y;
    if (sub == 0) {
      const size_t place = scale_at(static_cast<uint32_t>(slot), head, num_heads, block_size);
      ks[place] = sk;
      vs[place] = sv;
    }
  }
}

// A lane takes 16 elements of a row in runs whose values are 16 bytes, so that neighbouring lanes'
// stores lie side by side (fp32 rows with a lane's 32 bytes in a row: 274 us for 212).  HBM bounds
// it: 131072 x 8 bf16 rows in 112 us, 6.0 TB/s.  Four CTAs that keep two rows of a lane in flight
// take 116.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kReadCtas)
    read_fp4_kernel(T* __restrict__ k, T* __restrict__ v, const uint8_t* __restrict__ kc,
                    const uint8_t* __restrict__ vc, const __nv_bfloat16* __restrict__ ks,
                    const __nv_bfloat16* __restrict__ vs, const int64_t* __restrict__ slots,
                    long long num_rows, int num_heads, int block_size, long long num_slots,
                    unsigned* err) {
  constexpr int LPR = D / kLaneElems;
  constexpr int kRun = 16 / sizeof(T), kRuns = kLaneElems / kRun;
  using Codes = typename std::conditional<kRun == 8, uint32_t, uint16_t>::type;
  const int sub = threadIdx.x % LPR;
  const long long stride = static_cast<long long>(gridDim.x) * (kThreads / LPR);
  for (RowWalk w(static_cast<long long>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR, stride,
                 num_heads);
       w.row < num_rows; w.next(stride)) {
    const long long slot = __ldg(&slots[w.token]);
    if (slot < 0) continue;  // padding
    if (slot >= num_slots) {
      if (w.head == 0 && sub == 0) raise_error(err, PKV_DERR_SLOT);
      continue;
    }
    const long long at = slot * num_heads + w.head;
    const size_t place = scale_at(static_cast<uint32_t>(slot), w.head, num_heads, block_size);
    Codes ck[kRuns], cv[kRuns];
#pragma unroll
    for (int c = 0; c < kRuns; ++c) {
      ck[c] = __ldg(reinterpret_cast<const Codes*>(kc + at * (D / 2)) + c * LPR + sub);
      cv[c] = __ldg(reinterpret_cast<const Codes*>(vc + at * (D / 2)) + c * LPR + sub);
    }
    const float sk = __bfloat162float(ks[place]), sv = __bfloat162float(vs[place]);
#pragma unroll
    for (int c = 0; c < kRuns; ++c) {
      float x[kElems];
      decode8(ck[c], sk, x);
      store_run(k + w.row * D + (c * LPR + sub) * kRun, x);
      decode8(cv[c], sv, x);
      store_run(v + w.row * D + (c * LPR + sub) * kRun, x);
    }
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 152;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 152;
  return n;
}

template <typename T, int D>
int run(const CacheFp4Args& a, bool write, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.num_tokens) * a.num_kv_heads;
  const long long slots = static_cast<long long>(a.num_blocks) * a.block_size;
  const long long per_cta = kThreads / (D / kLaneElems);
  const long long resident = static_cast<long long>(write ? kWriteCtas : kReadCtas) * sm_count();
  const int grid =
      static_cast<int>(std::max(1LL, std::min((rows + per_cta - 1) / per_cta, resident)));
  uint8_t *kc = static_cast<uint8_t*>(a.k_cache), *vc = static_cast<uint8_t*>(a.v_cache);
  __nv_bfloat16 *ks = static_cast<__nv_bfloat16*>(a.k_scales),
                *vs = static_cast<__nv_bfloat16*>(a.v_scales);
  T *k = static_cast<T*>(a.k), *v = static_cast<T*>(a.v);
  if (write)
    write_fp4_kernel<T, D><<<grid, kThreads, 0, stream>>>(k, v, kc, vc, ks, vs, a.slot_mapping,
                                                          rows, a.num_kv_heads, a.block_size,
                                                          slots, a.err);
  else
    read_fp4_kernel<T, D><<<grid, kThreads, 0, stream>>>(k, v, kc, vc, ks, vs, a.slot_mapping,
                                                         rows, a.num_kv_heads, a.block_size, slots,
                                                         a.err);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

template <typename T>
int run_dim(const CacheFp4Args& a, bool write, cudaStream_t stream) {
  switch (a.head_dim) {
    case 32: return run<T, 32>(a, write, stream);
    case 64: return run<T, 64>(a, write, stream);
    case 128: return run<T, 128>(a, write, stream);
    case 256: return run<T, 256>(a, write, stream);
    default: return PKV_EUNSUPPORTED;
  }
}

}  // namespace

int launch_cache_fp4(const CacheFp4Args& a, bool write, cudaStream_t stream) {
  if (a.num_tokens == 0) return PKV_OK;
  switch (a.dtype) {
    case PKV_F32: return run_dim<float>(a, write, stream);
    case PKV_BF16: return run_dim<__nv_bfloat16>(a, write, stream);
    default: return run_dim<__half>(a, write, stream);
  }
}

}  // namespace pkv
