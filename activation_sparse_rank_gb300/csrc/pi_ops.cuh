// Element types and small device helpers of the operators around the FFN.
#pragma once

#include <cuda_bf16.h>

#include <atomic>

#include "pi_internal.cuh"

namespace pi {

// Device status bits of a cache (pi_kv_cache::status).
enum : unsigned { kKvBadPage = 1u, kKvBadRange = 2u, kKvBadRows = 4u, kKvTimeout = 8u };

inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool dtype_ok(int dt) { return dt == PI_DT_F16 || dt == PI_DT_BF16 || dt == PI_DT_F32; }
inline int dtype_size(int dt) { return dt == PI_DT_F32 ? 4 : 2; }

// SMs of the current device (cached per device; 0 if the runtime has no device).
int current_sms();

// Let kernel k use `bytes` of dynamic shared memory, of which it never uses more
// than `most`: asked of the runtime once per device and kernel (`done`: a bit a
// device, each instantiation has its own).
template <typename Kern>
cudaError_t allow_smem(Kern *k, size_t bytes, size_t most, std::atomic<uint64_t> &done) {
  if (bytes <= 40 * 1024) return cudaSuccess;        // with the static part still below the default limit
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

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

// Two binary32 values in one register pair: sm_100 and later add,
// multiply and fuse both in one instruction, each half rounded as the scalar
// operation rounds.
using f2 = float2;
__device__ __forceinline__ f2 f2_of(float lo, float hi) { return make_float2(lo, hi); }
__device__ __forceinline__ float2 f2_get(f2 a) { return a; }
__device__ __forceinline__ float f2_sum(f2 a) { return a.x + a.y; }
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) { return __ffma2_rn(a, b, c); }
// A 32-bit word of two 16-bit elements, and back (each rounded to nearest even).
template <int DT>
__device__ __forceinline__ f2 f2_widen(unsigned w) {
  if constexpr (DT == PI_DT_F16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return f2_of(f.x, f.y);
  } else {
    return f2_of(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
}
template <int DT>
__device__ __forceinline__ unsigned f2_narrow(f2 a) {
  const float2 f = f2_get(a);
  if constexpr (DT == PI_DT_F16) {
    const __half2 h = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const unsigned *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const unsigned *>(&h);
  }
}
// Pair j of the 16 bytes w (8 or 4 elements), and its opposite.
template <int DT>
__device__ __forceinline__ f2 f2_from16(const uint4 &w, int j) {
  if constexpr (DT == PI_DT_F32)
    return j ? f2_of(__uint_as_float(w.z), __uint_as_float(w.w)) : f2_of(__uint_as_float(w.x), __uint_as_float(w.y));
  else
    return f2_widen<DT>(j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w);
}
template <int DT>
__device__ __forceinline__ uint4 f2_to16(const f2 *v) {
  if constexpr (DT == PI_DT_F32) {
    const float2 a = f2_get(v[0]), b = f2_get(v[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  } else {
    return make_uint4(f2_narrow<DT>(v[0]), f2_narrow<DT>(v[1]), f2_narrow<DT>(v[2]), f2_narrow<DT>(v[3]));
  }
}

template <int I>
struct Int {
  static constexpr int v = I;
};
// f(Int<0>) .. f(Int<N - 1>), written out: arrays that f indexes stay in registers.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (I < N) {
    f(Int<I>{});
    each<N, I + 1>(f);
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Barrier of group g of NT threads of a CTA of CT.
template <int NT, int CT>
__device__ __forceinline__ void group_sync(int g) {
  if constexpr (NT == CT) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(NT) : "memory");
}
// Sum over group g (every thread gets it); red: CT/32 floats of shared memory,
// free for reuse after the group's next barrier.
template <int NT, int CT>
__device__ __forceinline__ float group_sum(float v, float *red, int g) {
  v = warp_sum(v);
  if constexpr (NT == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  group_sync<NT, CT>(g);
  float t = threadIdx.x % 32 < NT / 32 ? red[g * (NT / 32) + threadIdx.x % 32] : 0.f;
  return warp_sum(t);
}

}  // namespace pidev
