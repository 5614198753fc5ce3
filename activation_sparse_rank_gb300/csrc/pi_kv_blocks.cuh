// Blocks of the 8-bit cache as the copies see them (pi_kv.cu: write and read;
// pi_append.cu: write of rotated keys): where a warp's 16 tokens are, codes and scales.
#pragma once

#include "pi_kv.cuh"
#include "pi_ops.cuh"

namespace kv {

using namespace pidev;

struct KvCopyParams {
  pi_kv_cache c;
  pi_kv_tokens tok;
  const int32_t *start;
  const void *src[2];     // k, v (write)
  void *dst[2];           // k, v (read)
  int64_t st[2], sh[2];   // elements between tokens / heads of src
  int n_slots, per_warp;  // per_warp: (head, key or value) units of a slot that one warp does
};

// Where a warp's 16 tokens are: rows row0 .. row0+n-1 of the packed arrays are
// offsets off .. off+n-1 of block `blk` of page `page`.
struct KvPlace {
  int row0, n, off, page, blk;
  int64_t pos;            // position of row row0 in its sequence
};

// Slot i of a call.  A sequence with n rows from cu on touches at most
// n / 16 + 2 blocks, so sequence s owns the slots from cu[s] / 16 + 2 s on and
// no prefix sum is needed.
__device__ __forceinline__ bool kv_place(const KvCopyParams &p, int slot, KvPlace *o, bool *readable) {
  const int lane = threadIdx.x & 31;
  int lo = 0;                                         // last s with base(s) <= slot: 32 probes a step
  for (int n = p.tok.n_seqs; n > 1;) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool below = lane * step < n && (int64_t)p.tok.cu[at] / PI_KV_BLOCK + 2 * (int64_t)at <= slot;
    const int last = max(0, __popc(__ballot_sync(0xffffffffu, below)) - 1);
    n = min(step, n - last * step);
    lo += last * step;
  }
  const int s = lo, r0 = p.tok.cu[s], r1 = p.tok.cu[s + 1];
  if (r0 < 0 || r1 < r0 || r1 > p.tok.n_tokens) return false;      // flagged by kv_check_cu
  const int64_t first = p.start[s], j = slot - (r0 / PI_KV_BLOCK + 2 * (int64_t)s);
  if (r1 == r0 || j < 0) return false;
  if (first < 0) {
    *readable = false;
    // rows of a negative start: handed out 16 at a time, none readable
    if (j * PI_KV_BLOCK >= r1 - r0) return false;
    *o = KvPlace{r0 + (int)j * PI_KV_BLOCK, min(PI_KV_BLOCK, r1 - r0 - (int)j * PI_KV_BLOCK), 0, 0, 0, first + j * PI_KV_BLOCK};
    return true;
  }
  const int64_t b = first / PI_KV_BLOCK + j, end = first + (r1 - r0);
  const int64_t from = max(b * PI_KV_BLOCK, first), to = min((b + 1) * PI_KV_BLOCK, end);
  if (from >= to) return false;
  o->row0 = r0 + (int)(from - first);
  o->n = (int)(to - from);
  o->pos = from;
  o->off = (int)(from - b * PI_KV_BLOCK);
  const int per = p.c.page_size / PI_KV_BLOCK;
  const int64_t pg = b / per;
  o->blk = (int)(b - pg * per);
  *readable = pg < p.tok.table_pages;
  o->page = *readable ? p.tok.page_table[(int64_t)s * p.tok.table_stride + pg] : 0;
  if (*readable && (o->page < 0 || o->page >= p.c.n_pages)) {
    if ((threadIdx.x & 31) == 0) atomicOr(p.c.status, pi::kKvBadPage);
    *readable = false;
  } else if (!*readable && (threadIdx.x & 31) == 0) {
    atomicOr(p.c.status, pi::kKvBadRange);
  }
  return true;
}

// Every thread looks at one sequence's row range and start.
__device__ __forceinline__ void kv_check_cu(const KvCopyParams &p) {
  for (int64_t s = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; s < p.tok.n_seqs; s += (int64_t)gridDim.x * blockDim.x)
    if (p.tok.cu[s] < 0 || p.tok.cu[s + 1] < p.tok.cu[s] || p.tok.cu[s + 1] > p.tok.n_tokens)
      atomicOr(p.c.status, pi::kKvBadRows);
    else if (p.start[s] < 0 && p.tok.cu[s + 1] > p.tok.cu[s])
      atomicOr(p.c.status, pi::kKvBadRange);
}

// 8 values (four pairs) times inv as E4M3 codes.
__device__ __forceinline__ uint2 encode8(const f2 *v, f2 inv) {
  __nv_fp8x2_storage_t q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = __nv_cvt_float2_to_fp8x2(f2_get(f2_mul(v[e], inv)), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(q[0] | (unsigned)q[1] << 16, q[2] | (unsigned)q[3] << 16);
}

// Largest finite magnitude of 16 bytes of elements: NaN and infinities set no scale.
template <int DT>
__device__ __forceinline__ float amax16(const uint4 &w, float a) {
#pragma unroll
  for (int j = 0; j < 16 / (int)sizeof(typename Elem<DT>::T) / 2; ++j) {
    const float2 f = f2_get(f2_from16<DT>(w, j));
    const float x = fabsf(f.x), y = fabsf(f.y);
    a = fmaxf(a, fmaxf(x < INFINITY ? x : 0.f, y < INFINITY ? y : 0.f));
  }
  return a;
}

__device__ __forceinline__ void decode8(f2 *v, uint2 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const unsigned w = e < 2 ? c.x : c.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(e & 1 ? w >> 16 : w & 0xffff), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[e] = f2_of(f.x, f.y);
  }
}

// Exponent of the smallest power of two s >= 2^PI_KV_MIN_EXP with a <= 448 s
// (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exp(float a) {
  const unsigned b = __float_as_uint(a);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);
  return max(e, PI_KV_MIN_EXP);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }

}  // namespace kv

namespace pi {

// The checks that copies in and out of a cache share; fills all but the arrays.
pi_status check_copy(const pi_kv_cache *c, const pi_kv_tokens *t, const int32_t *start, int dtype, kv::KvCopyParams *p);

}  // namespace pi
