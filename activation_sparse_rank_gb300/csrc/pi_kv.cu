// The 8-bit key/value cache: quantising new tokens into it and reading them back.
//
// A block is PI_KV_BLOCK tokens of one head; its codes are contiguous and it
// has one scale, a power of two.  E4M3 is a floating format, so a power of two
// costs no relative precision against amax / 448, x / s is exact (a code is x
// rounded once, the same in any precision), and raising a scale re-encodes the
// codes it covers exactly unless they turn subnormal.
//
// Both directions are copies with a conversion: bound by HBM for prompts, by
// one load's latency for the single tokens of a decode step.  One warp per
// (block, head, key or value): it alone reads and writes that block, so the
// scale needs no atomics and no second pass.
//
// Measured: prompts of 30005 tokens in all x 8 heads x 128, bf16, 34 us (4.6 TB/s,
// 69% of the copy rate: a warp's chain of place, rows, maximum, codes is longer
// than 16 warps an SM with two blocks each hide); 60015 tokens x 8 x 64 read back 26 us (5.6 TB/s, 83%);
// one token of 32 sequences x 32 heads 5.2 us.
#include "pi_ops.cuh"
#include "pi_kv.cuh"

#include <algorithm>

using namespace pidev;

namespace {

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
    *o = KvPlace{r0 + (int)j * PI_KV_BLOCK, min(PI_KV_BLOCK, r1 - r0 - (int)j * PI_KV_BLOCK), 0, 0, 0};
    return true;
  }
  const int64_t b = first / PI_KV_BLOCK + j, end = first + (r1 - r0);
  const int64_t from = max(b * PI_KV_BLOCK, first), to = min((b + 1) * PI_KV_BLOCK, end);
  if (from >= to) return false;
  o->row0 = r0 + (int)(from - first);
  o->n = (int)(to - from);
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

// A warp's block: 16 rows of D elements as 16 D / 8 vectors of 8, vector
// lane + 32 i to a lane.
// AHEAD: a warp with several units loads the next one while it quantises one, at two
// CTAs an SM (write of the prompts above: 34 us, 38 without it at four, 57 at two).
// Otherwise registers for four CTAs (five: 50 us; 256 dims hold twice as many rows a
// lane).  Those of 64 dims do not spill; of more dims 16-bit rows spill up to 152 bytes
// a thread, binary32 rows up to 540.
template <int DT, int D, bool VEC, bool AHEAD>
__global__ void __launch_bounds__(256, D <= 128 && !AHEAD ? 4 : 2) k_kv_write(const KvCopyParams p) {
  using E = Elem<DT>;
  constexpr int VR = D / 8, NV = PI_KV_BLOCK * VR / 32, WPV = 8 * sizeof(typename E::T) / 16;
  kv_check_cu(p);
  const int lane = threadIdx.x & 31, parts = (2 * p.c.heads + 8 * p.per_warp - 1) / (8 * p.per_warp);
  KvPlace at;
  bool ok;
  if (!kv_place(p, blockIdx.x / parts, &at, &ok) || !ok) return;
  int unit = blockIdx.x % parts * 8 * p.per_warp + (threadIdx.x >> 5);
  const int units = min(2 * p.c.heads, unit + 8 * p.per_warp);
  uint4 x[NV][WPV], next[AHEAD ? NV : 1][WPV];
  auto load = [&](uint4 (*x)[WPV], int unit) {
    const int kv = unit >= p.c.heads, h = unit - kv * p.c.heads;
    const typename E::T *src = static_cast<const typename E::T *>(p.src[kv]) + (int64_t)at.row0 * p.st[kv] + h * p.sh[kv];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < WPV; ++c) x[i][c] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + 32 * i, r = v / VR - at.off;
      if (r >= 0 && r < at.n) {
        const typename E::T *row = src + (int64_t)r * p.st[kv] + v % VR * 8;
        if constexpr (VEC) {
#pragma unroll
          for (int c = 0; c < WPV; ++c) x[i][c] = reinterpret_cast<const uint4 *>(row)[c];
        } else {
          alignas(16) typename E::T e8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) e8[e] = row[e];
#pragma unroll
          for (int c = 0; c < WPV; ++c) x[i][c] = reinterpret_cast<const uint4 *>(e8)[c];
        }
      }
    }
  };
  if constexpr (AHEAD)
    if (unit < units) load(x, unit);
#pragma unroll 1
  for (; unit < units; unit += 8) {
    const int kv = unit >= p.c.heads, h = unit - kv * p.c.heads;
    if constexpr (!AHEAD) load(x, unit);
    else if (unit + 8 < units) load(next, unit + 8);
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < WPV; ++c) a = amax16<DT>(x[i][c], a);
    float s = pow2(scale_exp(warp_max(a)));
    const int64_t page_head = (int64_t)at.page * p.c.heads + h;
    float *scale = (kv ? p.c.v_scales : p.c.k_scales) + page_head * (p.c.page_size / PI_KV_BLOCK) + at.blk;
    uint2 *codes = reinterpret_cast<uint2 *>((kv ? p.c.v_codes : p.c.k_codes) +
                                             (page_head * p.c.page_size + at.blk * PI_KV_BLOCK) * D);
    if (at.off > 0) {
      const float old = *scale;
      if (old < s) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = lane + 32 * i;
          if (v / VR < at.off) {
            f2 f[4];
            decode8(f, codes[v]);
            codes[v] = encode8(f, f2_of(old / s, old / s));
          }
        }
      } else if (old > s) {
        s = old;
      }
    }
    const float inv = 1.0f / s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + 32 * i, r = v / VR - at.off;
      if (r >= 0 && r < at.n) {
        f2 f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = f2_from16<DT>(x[i][WPV == 2 ? e / 2 : 0], WPV == 2 ? e % 2 : e);
        codes[v] = encode8(f, f2_of(inv, inv));
      }
    }
    __syncwarp();                                    // every lane has read the old scale
    if (lane == 0) *scale = s;
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < WPV; ++c) x[i][c] = next[i][c];
    }
  }
}

template <int DT, int D>
__global__ void __launch_bounds__(256) k_kv_read(const KvCopyParams p) {
  using E = Elem<DT>;
  constexpr int VR = D / 8, NV = PI_KV_BLOCK * VR / 32, W = 16 / sizeof(typename E::T);
  kv_check_cu(p);
  // rows of no sequence: below every entry of cu, and from the largest on
  int r0 = p.tok.n_seqs ? p.tok.cu[0] : p.tok.n_tokens, r1 = p.tok.n_seqs ? p.tok.cu[p.tok.n_seqs] : p.tok.n_tokens;
  if (p.tok.n_seqs && (r0 > 0 || r1 < p.tok.n_tokens)) {             // the ends alone do not say so where cu does not ascend
    __shared__ int least, most;
    if (threadIdx.x == 0) least = r0, most = r1;
    __syncthreads();
    for (int s = threadIdx.x; s <= p.tok.n_seqs; s += blockDim.x) r0 = min(r0, p.tok.cu[s]), r1 = max(r1, p.tok.cu[s]);
    r0 = __reduce_min_sync(0xffffffffu, r0), r1 = __reduce_max_sync(0xffffffffu, r1);
    if ((threadIdx.x & 31) == 0) atomicMin(&least, r0), atomicMax(&most, r1);
    __syncthreads();
    r0 = least, r1 = most;
  }
  r0 = max(0, min(p.tok.n_tokens, r0)), r1 = max(r0, min(p.tok.n_tokens, r1));
  const int64_t per_row = (int64_t)p.c.heads * D / W;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (r0 + (p.tok.n_tokens - r1)) * per_row;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t at = i < r0 * per_row ? i : i + (r1 - r0) * per_row;
    for (int kv = 0; kv < 2; ++kv)
      if (p.dst[kv]) static_cast<uint4 *>(p.dst[kv])[at] = make_uint4(0, 0, 0, 0);
  }
  if (p.tok.n_seqs == 0) return;
  const int lane = threadIdx.x & 31, parts = (2 * p.c.heads + 8 * p.per_warp - 1) / (8 * p.per_warp);
  KvPlace at;
  bool ok;
  if (!kv_place(p, blockIdx.x / parts, &at, &ok)) return;
  for (int i_unit = 0, unit = blockIdx.x % parts * 8 * p.per_warp + (threadIdx.x >> 5);
       i_unit < p.per_warp && unit < 2 * p.c.heads; ++i_unit, unit += 8) {
    const int kv = unit >= p.c.heads, h = unit - kv * p.c.heads;
    if (!p.dst[kv]) continue;
    const int64_t page_head = (int64_t)at.page * p.c.heads + h;
    const uint2 *codes = reinterpret_cast<const uint2 *>((kv ? p.c.v_codes : p.c.k_codes) +
                                                         (page_head * p.c.page_size + at.blk * PI_KV_BLOCK) * D);
    uint2 c[NV];
    float s = 0.f;
    if (ok) {
      s = ((kv ? p.c.v_scales : p.c.k_scales) + page_head * (p.c.page_size / PI_KV_BLOCK))[at.blk];
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] = codes[lane + 32 * i];
    }
    typename E::T *dst = static_cast<typename E::T *>(p.dst[kv]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + 32 * i, r = v / VR - at.off;
      if (r < 0 || r >= at.n) continue;
      f2 f[4] = {};
      if (ok) {
        decode8(f, c[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = f2_mul(f[e], f2_of(s, s));
      }
      uint4 *row = reinterpret_cast<uint4 *>(dst + ((int64_t)(at.row0 + r) * p.c.heads + h) * D + v % VR * 8);
      row[0] = f2_to16<DT>(f);
      if constexpr (DT == PI_DT_F32) row[1] = f2_to16<DT>(f + 2);
    }
  }
}

template <int DT, int D>
cudaError_t launch_copy(KvCopyParams p, bool write, bool vec, cudaStream_t s) {
  const int units = 2 * p.c.heads;
  // finding a block's place takes three loads one after another: with enough
  // blocks to fill the GPU a warp uses it for several heads (read of the prefixes above:
  // 26 us, 29 with one)
  p.per_warp = std::max<int64_t>(1, std::min<int64_t>(4, (int64_t)p.n_slots * units / (64 * std::max(1, pi::current_sms()))));
  const unsigned grid = (unsigned)((int64_t)std::max(1, p.n_slots) * ((units + 8 * p.per_warp - 1) / (8 * p.per_warp)));
  constexpr bool kAhead = D <= 128 && DT != PI_DT_F32;         // twice a unit's registers fit
  if (write && vec && kAhead && p.per_warp > 1)
    k_kv_write<DT, D, true, kAhead><<<grid, 256, 0, s>>>(p);
  else if (write && vec)
    k_kv_write<DT, D, true, false><<<grid, 256, 0, s>>>(p);
  else if (write)
    k_kv_write<DT, D, false, false><<<grid, 256, 0, s>>>(p);
  else
    k_kv_read<DT, D><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <int DT>
cudaError_t copy_by_dim(const KvCopyParams &p, bool write, bool vec, cudaStream_t s) {
  switch (p.c.head_dim) {
    case 64: return launch_copy<DT, 64>(p, write, vec, s);
    case 96: return launch_copy<DT, 96>(p, write, vec, s);
    case 128: return launch_copy<DT, 128>(p, write, vec, s);
    default: return launch_copy<DT, 256>(p, write, vec, s);
  }
}

cudaError_t run_copy(const KvCopyParams &p, bool write, bool vec, int dtype, cudaStream_t s) {
  return dtype == PI_DT_F16    ? copy_by_dim<PI_DT_F16>(p, write, vec, s)
         : dtype == PI_DT_BF16 ? copy_by_dim<PI_DT_BF16>(p, write, vec, s)
                               : copy_by_dim<PI_DT_F32>(p, write, vec, s);
}

}  // namespace

namespace pi {

pi_status check_cache(const pi_kv_cache *c) {
  if (!c) return fail(PI_ERR_INVALID_ARG, "cache is NULL");
  if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128 && c->head_dim != 256)
    return fail(PI_ERR_UNSUPPORTED, "head_dim=%d: 64, 96, 128 or 256", c->head_dim);
  if (c->page_size < PI_KV_BLOCK || c->page_size > PI_KV_MAX_PAGE || c->page_size % PI_KV_BLOCK)
    return fail(PI_ERR_UNSUPPORTED, "page_size=%d: a multiple of %d up to %d", c->page_size, PI_KV_BLOCK, PI_KV_MAX_PAGE);
  if (c->n_pages < 1 || c->heads < 1 || c->heads > 65535)
    return fail(PI_ERR_INVALID_ARG, "n_pages=%d, heads=%d: need at least 1 (heads up to 65535)", c->n_pages, c->heads);
  if (!c->k_codes || !c->v_codes || !aligned_to(c->k_codes, 16) || !aligned_to(c->v_codes, 16))
    return fail(PI_ERR_INVALID_ARG, "k_codes and v_codes must be non-NULL and 16-byte aligned");
  if (!c->k_scales || !c->v_scales || !c->status || !aligned_to(c->k_scales, 4) || !aligned_to(c->v_scales, 4) ||
      !aligned_to(c->status, 4))
    return fail(PI_ERR_INVALID_ARG, "k_scales, v_scales and status must be non-NULL and 4-byte aligned");
  return PI_OK;
}

pi_status check_tokens(const pi_kv_tokens *t) {
  if (!t) return fail(PI_ERR_INVALID_ARG, "tokens is NULL");
  if (t->n_seqs < 0 || t->n_tokens < 0 || t->n_seqs > (1 << 20) || t->n_tokens > (1 << 28))
    return fail(PI_ERR_INVALID_ARG, "n_seqs=%d or n_tokens=%d out of range", t->n_seqs, t->n_tokens);
  if (t->n_seqs && (!t->cu || !t->page_table || !aligned_to(t->cu, 4) || !aligned_to(t->page_table, 4)))
    return fail(PI_ERR_INVALID_ARG, "cu and page_table must be non-NULL and 4-byte aligned");
  if (t->n_seqs && (t->table_stride < 1 || t->table_pages < 0))
    return fail(PI_ERR_INVALID_ARG, "table_stride=%d, table_pages=%d", t->table_stride, t->table_pages);
  return PI_OK;
}

}  // namespace pi

namespace {

pi_status check_copy(const pi_kv_cache *c, const pi_kv_tokens *t, const int32_t *start, int dtype, KvCopyParams *p) {
  pi::clear_error();
  pi_status st = pi::check_cache(c);
  if (st == PI_OK) st = pi::check_tokens(t);
  if (st != PI_OK) return st;
  if (!pi::dtype_ok(dtype)) return pi::fail(PI_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (t->n_seqs && (!start || !pi::aligned_to(start, 4)))
    return pi::fail(PI_ERR_INVALID_ARG, "start must be non-NULL and 4-byte aligned");
  *p = KvCopyParams{*c, pi::with_pages(*t), start, {}, {}, {}, {}, t->n_tokens / PI_KV_BLOCK + 2 * t->n_seqs, 1};
  if ((int64_t)(p->n_slots + 1) * (2 * c->heads / 8 + 1) >= (int64_t)1 << 31)
    return pi::fail(PI_ERR_UNSUPPORTED, "n_tokens=%d with heads=%d is too large for one call", t->n_tokens, c->heads);
  return PI_OK;
}

}  // namespace

extern "C" {

pi_status pi_kv_write(const pi_kv_cache *cache, const pi_kv_tokens *tokens, const int32_t *start, const void *k,
                      const int64_t *k_stride, const void *v, const int64_t *v_stride, int32_t dtype, void *stream) {
  KvCopyParams p;
  const pi_status st = check_copy(cache, tokens, start, dtype, &p);
  if (st != PI_OK) return st;
  if (tokens->n_tokens == 0 || tokens->n_seqs == 0) return PI_OK;
  const int e = pi::dtype_size(dtype), V = 16 / e;
  if (!k || !v || !k_stride || !v_stride || !pi::aligned_to(k, e) || !pi::aligned_to(v, e))
    return pi::fail(PI_ERR_INVALID_ARG, "k, v and their strides must be non-NULL, k and v aligned to their type");
  p.src[0] = k, p.src[1] = v;
  bool vec = pi::aligned_to(k, 16) && pi::aligned_to(v, 16);
  for (int i = 0; i < 2; ++i) {
    const int64_t *s = i ? v_stride : k_stride;
    if (s[0] < 0 || s[1] < 0) return pi::fail(PI_ERR_INVALID_ARG, "strides must not be negative");
    p.st[i] = s[0], p.sh[i] = s[1];
    vec = vec && s[0] % V == 0 && s[1] % V == 0;
  }
  PI_TRY_CUDA(run_copy(p, true, vec, dtype, static_cast<cudaStream_t>(stream)));
  return PI_OK;
}

pi_status pi_kv_read(const pi_kv_cache *cache, const pi_kv_tokens *tokens, const int32_t *start, void *k, void *v,
                     int32_t dtype, void *stream) {
  KvCopyParams p;
  const pi_status st = check_copy(cache, tokens, start, dtype, &p);
  if (st != PI_OK) return st;
  if (tokens->n_tokens == 0) return PI_OK;
  if ((!k && !v) || !pi::aligned_to(k, 16) || !pi::aligned_to(v, 16))
    return pi::fail(PI_ERR_INVALID_ARG, "k or v must be non-NULL, both 16-byte aligned");
  p.dst[0] = k, p.dst[1] = v;
  PI_TRY_CUDA(run_copy(p, false, true, dtype, static_cast<cudaStream_t>(stream)));
  return PI_OK;
}

pi_status pi_kv_status(const pi_kv_cache *cache, void *stream) {
  pi::clear_error();
  const pi_status st = pi::check_cache(cache);
  if (st != PI_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned v = 0;
  PI_TRY_CUDA(cudaMemcpyAsync(&v, cache->status, sizeof(v), cudaMemcpyDeviceToHost, s));
  PI_TRY_CUDA(cudaStreamSynchronize(s));
  if (v) {
    PI_TRY_CUDA(cudaMemsetAsync(cache->status, 0, sizeof(v), s));
    PI_TRY_CUDA(cudaStreamSynchronize(s));
    return pi::fail(PI_ERR_DEVICE_CHECK, "cache check failed:%s%s%s%s", (v & pi::kKvBadPage) ? " page out of range" : "",
                    (v & pi::kKvBadRange) ? " position out of range" : "",
                    (v & pi::kKvBadRows) ? " token rows out of range" : "",
                    (v & pi::kKvTimeout) ? " a wait ran out" : "");
  }
  return PI_OK;
}

}  // extern "C"
