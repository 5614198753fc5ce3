// Element types and small device helpers of the operators around the FFN.
#pragma once

#include <cuda_bf16.h>

#include "pi_internal.cuh"

namespace pi {

// Device status bits of a cache (pi_kv_cache::status).
enum : unsigned { kKvBadPage = 1u, kKvBadRange = 2u, kKvBadRows = 4u, kKvTimeout = 8u };

inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool dtype_ok(int dt) { return dt == PI_DT_F16 || dt == PI_DT_BF16 || dt == PI_DT_F32; }
inline int dtype_size(int dt) { return dt == PI_DT_F32 ? 4 : 2; }

// SMs of the current device (cached per device; 0 if the runtime has no device).
int current_sms();

}  // namespace pi

namespace pidev {

template <int DT>
struct Elem;
template <>
struct Elem<PI_DT_F16> {
  using T = __half;
  static __device__ __forceinline__ float to(T v) { return __half2float(v); }
  static __device__ __forceinline__ T from(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<PI_DT_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float to(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T from(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<PI_DT_F32> {
  using T = float;
  static __device__ __forceinline__ float to(T v) { return v; }
  static __device__ __forceinline__ T from(float v) { return v; }
};

// N elements as one aligned load or store.
template <int DT, int N>
struct alignas(N * sizeof(typename Elem<DT>::T)) Pack {
  typename Elem<DT>::T v[N];
};

// Element i of a tensor whose type is only known at run time (small tensors: norm weights, added rows).
__device__ __forceinline__ float load_any(const void *p, int dt, size_t i) {
  if (dt == PI_DT_F16) return __half2float(static_cast<const __half *>(p)[i]);
  if (dt == PI_DT_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  return static_cast<const float *>(p)[i];
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sum over the CTA (every thread gets it); red: NT/32 floats of shared memory,
// free for reuse after the next __syncthreads().
template <int NT>
__device__ __forceinline__ float cta_sum(float v, float *red) {
  v = warp_sum(v);
  if constexpr (NT == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = threadIdx.x % 32 < NT / 32 ? red[threadIdx.x % 32] : 0.f;
  return warp_sum(t);
}

}  // namespace pidev
