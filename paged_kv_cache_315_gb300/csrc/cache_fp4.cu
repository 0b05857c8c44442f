// cache_fp4.cu -- quantising writes into and reads out of the 4-bit cache (sm_103a).
//
// A row is the head_dim elements of one token and one KV head.  Its scale is the bf16
// nearest to amax / 6 (6 is the largest E2M1 magnitude) and each element's code the E2M1
// value nearest to x / scale, ties to the even code.  Both kernels are byte movement with a
// little arithmetic: per element the write reads 2 bytes (16-bit types) and stores half a
// byte, so the arithmetic per element has to stay within a few instructions for HBM to
// remain the bound.
#include <algorithm>

#include "device_common.cuh"
#include "fp4.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kElems = 8;  // elements a lane holds of a row: 16 bytes of a 16-bit type

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

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[kElems]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint4 a;
    a.x = Mma<T>::pack(x[0], x[1]);
    a.y = Mma<T>::pack(x[2], x[3]);
    a.z = Mma<T>::pack(x[4], x[5]);
    a.w = Mma<T>::pack(x[6], x[7]);
    *reinterpret_cast<uint4*>(p) = a;
  }
}

// The 8 codes (element 0 in the lowest four bits) of x / scale, the IEEE quotient.
__device__ __forceinline__ uint32_t encode8(const float (&x)[kElems], float scale) {
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    word |= f32x2_to_e2m1x2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale)) << (8 * i);
  return word;
}

// A row of D elements is held by D / 8 lanes of a warp.  Returns its codes and, in `scale`,
// its scale (the same in each of those lanes).
template <int D>
__device__ __forceinline__ uint32_t quantise(const float (&x)[kElems], __nv_bfloat16& scale) {
  // |x| as bits orders like |x|, and a NaN above infinity above every number
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kElems; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (top >= 0x7f800000u) {  // a NaN or an infinity in the row: every element reads as NaN
    scale = __ushort_as_bfloat16(0x7fff);
    return 0;
  }
  scale = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(top), 6.f));
  const float s = __bfloat162float(scale);
  return s > 0.f ? encode8(x, s) : 0u;
}

// One group of D / 8 lanes per (token, head) row, its key and its value row together.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    write_fp4_kernel(const T* __restrict__ k, const T* __restrict__ v, uint8_t* __restrict__ kc,
                     uint8_t* __restrict__ vc, __nv_bfloat16* __restrict__ ks,
                     __nv_bfloat16* __restrict__ vs, const int64_t* __restrict__ slots,
                     long long num_rows, int num_heads, int block_size, long long num_slots,
                     unsigned* err) {
  constexpr int LPR = D / kElems;
  const int sub = threadIdx.x % LPR;
  const long long stride = static_cast<long long>(gridDim.x) * (kThreads / LPR);
  // every lane of a warp runs the same number of iterations: the shuffles are warp-wide
  const long long first = static_cast<long long>(blockIdx.x) * (kThreads / LPR);
  for (long long base = first; base < num_rows; base += stride) {
    const long long row = base + threadIdx.x / LPR;
    const bool in = row < num_rows;
    const long long r = in ? row : num_rows - 1;
    const long long token = r / num_heads;
    const int head = static_cast<int>(r - token * num_heads);
    const long long slot = __ldg(&slots[token]);
    float xk[kElems], xv[kElems];
    load8(k + r * D + sub * kElems, xk);
    load8(v + r * D + sub * kElems, xv);
    __nv_bfloat16 sk, sv;
    const uint32_t ck = quantise<D>(xk, sk), cv = quantise<D>(xv, sv);
    if (!in || slot < 0) continue;  // past the last row, or padding
    if (slot >= num_slots) {
      if (head == 0 && sub == 0) raise_error(err, PKV_DERR_SLOT);
      continue;
    }
    const long long at = slot * num_heads + head;
    *reinterpret_cast<uint32_t*>(kc + at * (D / 2) + sub * 4) = ck;
    *reinterpret_cast<uint32_t*>(vc + at * (D / 2) + sub * 4) = cv;
    if (sub == 0) {
      const long long block = slot / block_size;
      const long long place = (block * num_heads + head) * block_size + (slot - block * block_size);
      ks[place] = sk;
      vs[place] = sv;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    read_fp4_kernel(T* __restrict__ k, T* __restrict__ v, const uint8_t* __restrict__ kc,
                    const uint8_t* __restrict__ vc, const __nv_bfloat16* __restrict__ ks,
                    const __nv_bfloat16* __restrict__ vs, const int64_t* __restrict__ slots,
                    long long num_rows, int num_heads, int block_size, long long num_slots,
                    unsigned* err) {
  constexpr int LPR = D / kElems;
  const long long total = num_rows * LPR;
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += stride) {
    const long long r = i / LPR;
    const int sub = static_cast<int>(i - r * LPR);
    const long long token = r / num_heads;
    const int head = static_cast<int>(r - token * num_heads);
    const long long slot = __ldg(&slots[token]);
    if (slot < 0) continue;
    if (slot >= num_slots) {
      if (head == 0 && sub == 0) raise_error(err, PKV_DERR_SLOT);
      continue;
    }
    const long long at = slot * num_heads + head;
    const long long block = slot / block_size;
    const long long place = (block * num_heads + head) * block_size + (slot - block * block_size);
    const uint32_t ck = __ldg(reinterpret_cast<const uint32_t*>(kc + at * (D / 2)) + sub);
    const uint32_t cv = __ldg(reinterpret_cast<const uint32_t*>(vc + at * (D / 2)) + sub);
    const float sk = __bfloat162float(ks[place]), sv = __bfloat162float(vs[place]);
    float x[kElems];
    decode8(ck, sk, x);
    store8(k + i * kElems, x);
    decode8(cv, sv, x);
    store8(v + i * kElems, x);
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
  const long long per_cta = kThreads / (D / kElems);
  const int grid = static_cast<int>(
      std::max(1LL, std::min((rows + per_cta - 1) / per_cta, 8LL * sm_count())));
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
