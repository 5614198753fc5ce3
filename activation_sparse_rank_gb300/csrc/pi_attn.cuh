// What the attention kernels share (pi_attn.cu: few query rows a head;
// pi_attn_tc.cu: many): parameters, the line of tiles that is cut over the CTAs,
// the tensor maps of the codes and the sum of parts.
#pragma once

#include "pi_kv.cuh"
#include "pi_ops.cuh"
#include "pi_ptx.cuh"

#include <algorithm>

namespace attn {

using namespace pidev;

// The second product's weights 2^(x + ev - R) reach 2^(kBoost + kSlack), inside
// fp16, and are subnormal only below 2^-(14 + kBoost) of the largest.  kSlack:
// m and R follow a score only where it passes them by that much; the sums do
// not depend on m and R, and most steps then leave the accumulators alone.
constexpr float kBoost = 6.f, kSlack = 8.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
  pi_kv_cache c;
  pi_kv_tokens tok;
  const int32_t *length;
  const void *q;
  int64_t qt, qh;
  void *out;
  float *lse;
  int4 *plan;              // [grid] the unit that share i has to add up: sequence, head, row tile, parts + (rows << 16); 0: none
  float *part;             // [2 grid] partials of [ROWS, D] sums, then [ROWS, 2] (m, l)
  float scale;             // sm_scale log2(e)
  int q_heads, group, max_q, causal, row_tiles, grid;
  int wide;                // q, out, part: bits 0, 1, 2 set where 32-byte accesses are aligned
};

// 32 bytes at once, for a row a thread: half the transactions of 16 bytes (prompts of
// 85 tokens x 5 heads over 182 keys, 16 sequences x 22 heads: 111 -> 98 us).
__device__ __forceinline__ void load32(const uint4 *p, uint4 &a, uint4 &b) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w) : "l"(p));
}
__device__ __forceinline__ void store32(uint4 *p, const uint4 &a, const uint4 &b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x),
               "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// sum + l 2^by, by <= 0 or not by much more: a part's l may be so large (its values
// had the smallest scales) that it counts where 2^by alone would be 0.
__device__ __forceinline__ float add_scaled(float sum, float l, float by) {
  if (by < -120.f) {
    const float h = ex2(0.5f * by);
    return sum + l * h * h;
  }
  return fmaf(l, ex2(by), sum);
}

// Four codes as two fp16 pairs: one instruction each.
__device__ __forceinline__ void widen4(unsigned w, unsigned &lo, unsigned &hi) {
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}" : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ unsigned pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const unsigned *>(&h);
}

// Sequence s as the kernels see it: lengths made safe, faults flagged by flag_seq.
struct Seq {
  int row0, n, rows, len, first;    // packed row, query tokens used, query rows, keys, position of the first token
  int left;                         // tokens past max_q
};
__device__ __forceinline__ Seq load_seq(const AttnParams &p, int s) {
  Seq q;
  const int r0 = p.tok.cu[s], r1 = p.tok.cu[s + 1];
  const int n = r0 < 0 || r1 < r0 || r1 > p.tok.n_tokens ? 0 : r1 - r0;
  const int64_t cap = min((int64_t)p.tok.table_pages * p.c.page_size, (int64_t)1 << 30);
  const int len = p.length[s];
  q.row0 = r0, q.n = min(n, p.max_q), q.rows = q.n * p.group, q.left = n - q.n;
  q.len = len < 0 ? 0 : (int)min((int64_t)len, cap);
  q.first = (len < 0 ? 0 : len) - n;
  return q;
}
__device__ __forceinline__ void flag_seq(const AttnParams &p, int s) {
  const int r0 = p.tok.cu[s], r1 = p.tok.cu[s + 1], len = p.length[s];
  if (r0 < 0 || r1 < r0 || r1 > p.tok.n_tokens || r1 - r0 > p.max_q) atomicOr(p.c.status, pi::kKvBadRows);
  if (len < 0 || len > (int64_t)p.tok.table_pages * p.c.page_size || len > 1 << 30) atomicOr(p.c.status, pi::kKvBadRange);
}
// Keys that any row of a row tile (ROWS rows) sees, and the tiles (TILE keys) that hold them.
template <int ROWS>
__device__ __forceinline__ int unit_keys(const AttnParams &p, const Seq &q, int rt) {
  if (rt * ROWS >= q.rows) return 0;
  if (!p.causal) return q.len;
  const int last = min(q.rows, (rt + 1) * ROWS) - 1;
  return max(0, min(q.len, q.first + last / p.group + 1));
}
template <int ROWS, int TILE>
__device__ __forceinline__ int unit_tiles(const AttnParams &p, const Seq &q, int rt) {
  return (unit_keys<ROWS>(p, q, rt) + TILE - 1) / TILE;
}
// Exclusive sum over the CTA's first 128 threads (the others pass 0); *total gets the whole sum.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t *sm, int64_t *total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31 && w < 4) sm[w] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < w) before += sm[i];
    all += sm[i];
  }
  *total = all;
  return before + x - v;
}

__device__ __forceinline__ int64_t cta_begin(int64_t c, int64_t total, int shares) { return c * total / shares; }
__device__ __forceinline__ int64_t cta_owner(int64_t tile, int64_t total, int shares) { return ((tile + 1) * shares - 1) / total; }

// One CTA's share of the line of tiles and its place in it.  A unit is a
// (sequence, head, row tile); units without keys take no place.
struct Share {
  int64_t begin, end;      // tiles
  int64_t total;           // of the line
  int shares;              // that it is cut into
  int s, h, rt;            // the unit that `begin` lies in
  int64_t u0;              // where that unit begins
  Seq sq;
};
struct ShareShared {
  int64_t scan[4], at;
  int s, rt;
};
// Share `cta` of p.grid; false if there is none.  Every thread of the CTA calls it.
// The line is ordered by sequence, head, row tile; a sequence's row tiles have
// the same keys for every head, so the sums run over (sequence, row tile) pairs,
// times the heads.
template <int ROWS, int TILE>
__device__ __forceinline__ bool find_share(const AttnParams &p, ShareShared &sm, int cta, Share *o) {
  const int64_t pairs = (int64_t)p.tok.n_seqs * p.row_tiles, per = (pairs + 127) / 128, k0 = threadIdx.x * per;
  auto tiles_of = [&](int64_t k) {
    const int s = (int)(k / p.row_tiles);
    return unit_tiles<ROWS, TILE>(p, load_seq(p, s), (int)(k - (int64_t)s * p.row_tiles));
  };
  int64_t mine = 0, total;
  if (threadIdx.x < 128)
    for (int64_t k = k0; k < k0 + per && k < pairs; ++k) mine += tiles_of(k);
  int64_t at = cta_scan(mine, sm.scan, &total);
  const int heads = p.c.heads;
  total *= heads;
  const int shares = (int)min((int64_t)p.grid, total);       // every share has a tile, so every part between two of a unit is written
  o->total = total, o->shares = shares;
  if (cta >= shares) return false;
  o->begin = cta_begin(cta, total, shares), o->end = cta_begin(cta + 1, total, shares);
  if (at * heads <= o->begin && o->begin < (at + mine) * heads)
    for (int64_t k = k0;; ++k) {                     // the pair there is of the right sequence
      const int n = tiles_of(k);
      if (o->begin < (at + n) * heads) {
        sm.s = (int)(k / p.row_tiles), sm.rt = (int)(k % p.row_tiles), sm.at = at;
        break;
      }
      at += n;
    }
  __syncthreads();
  // in that sequence: its tiles of one head, then the head and the row tile
  const int lane = threadIdx.x & 31;
  o->s = sm.s;
  o->sq = load_seq(p, o->s);
  int64_t before = 0, all = 0;
  for (int r0 = 0; r0 < p.row_tiles; r0 += 32) {
    const int n = r0 + lane < p.row_tiles ? unit_tiles<ROWS, TILE>(p, o->sq, r0 + lane) : 0;
    all += __reduce_add_sync(0xffffffffu, n);
    before += __reduce_add_sync(0xffffffffu, r0 + lane < sm.rt ? n : 0);
  }
  const int64_t start = (sm.at - before) * heads;
  o->h = (int)((o->begin - start) / all);
  int64_t u0 = start + o->h * all;
  for (int r0 = 0; r0 < p.row_tiles; r0 += 32) {
    const int n = r0 + lane < p.row_tiles ? unit_tiles<ROWS, TILE>(p, o->sq, r0 + lane) : 0;
    int sum = n;                                     // inclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += y;
    }
    const unsigned past = __ballot_sync(0xffffffffu, u0 + sum > o->begin);
    if (past) {
      const int l = __ffs(past) - 1;
      o->rt = r0 + l;
      o->u0 = u0 + __shfl_sync(0xffffffffu, sum - n, l);
      break;
    }
    u0 += __shfl_sync(0xffffffffu, sum, 31);
  }
  return true;
}
// To the next unit with keys; false after the last.
template <int ROWS, int TILE>
__device__ __forceinline__ bool next_unit(const AttnParams &p, Share *o) {
  o->u0 += unit_tiles<ROWS, TILE>(p, o->sq, o->rt);
  do {
    if (++o->rt >= p.row_tiles || o->rt * ROWS >= o->sq.rows) {
      o->rt = 0;
      if (++o->h >= p.c.heads) {
        o->h = 0;
        if (++o->s >= p.tok.n_seqs) return false;
        o->sq = load_seq(p, o->s);
      }
    }
  } while (unit_tiles<ROWS, TILE>(p, o->sq, o->rt) == 0);
  return true;
}

// Parts of a unit are added by the first share whose begin lies inside it (the
// part before its begin is its neighbour's): thread 0 of that share's CTA says so.
template <int ROWS, int TILE>
__device__ __forceinline__ void write_plan(const AttnParams &p, bool any, const Share &at) {
  int4 plan = make_int4(0, 0, 0, 0);
  if (any && at.begin > at.u0) {
    const int64_t c0 = cta_owner(at.u0, at.total, at.shares);
    if (c0 == (int64_t)blockIdx.x - 1) {
      const int parts = (int)(cta_owner(at.u0 + unit_tiles<ROWS, TILE>(p, at.sq, at.rt) - 1, at.total, at.shares) - c0) + 1;
      plan = make_int4(at.s, at.h, at.rt, parts | min(ROWS, at.sq.rows - at.rt * ROWS) << 16);
    }
  }
  p.plan[blockIdx.x] = plan;
}

struct AttnMaps {          // [n_pages heads][page_size][D] codes, boxes of 64 or 16 tokens and up to 128 bytes
  CUtensorMap k, v;
};

// Units cut between CTAs: their parts added in CTA order.  A row's parts come at
// the latency of L2, so of more than eight parts (a long cache with few heads: up
// to one a CTA) four or sixteen warps take a row, a run of parts each.  A pass of
// 16 warps over rows of a unit is an item; a few CTAs an SM take all items, which
// the plan's prefix sums find (a CTA for each share and four rows instead: 60 us
// for attention of 128 query heads over 130001 keys, 48 so, as most had no work).
// Rows of units without keys, and of tokens past max_q: 0 and -inf.
constexpr int kCombineThreads = 512, kMostShares = 1024;
constexpr int combine_ctas(int D) { return D <= 128 ? 3 : 2; }     // that an SM holds
__host__ __device__ constexpr int combine_split(int parts) { return parts > 64 ? 16 : parts > 8 ? 4 : 1; }
template <int DT, int D, int ROWS, int TILE>
__global__ void __launch_bounds__(kCombineThreads, combine_ctas(D)) k_attn_combine(const AttnParams p) {
  using E = Elem<DT>;
  constexpr int LANES = D / 4 <= 16 ? 16 : 32;     // lanes across a row (D = 64: half a warp per part)
  constexpr int VECS = D / 4 <= 32 ? 1 : D / 4 / 32;
  constexpr int WARPS = kCombineThreads / 32;
  __shared__ float4 sums[WARPS][D / 4];
  __shared__ float2 stats[WARPS];
  __shared__ int upto[kMostShares], warp_items[WARPS];       // items of the shares up to each
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int s0 = 0; s0 < p.tok.n_seqs; s0 += kCombineThreads) {       // the leading row tiles of a sequence may see nothing
    auto blank = [&](const Seq &sq) {              // rows of them
      int rows = 0;
      for (int rt = 0; rt < p.row_tiles && rt * ROWS < sq.rows && unit_tiles<ROWS, TILE>(p, sq, rt) == 0; ++rt) rows = min(sq.rows, (rt + 1) * ROWS);
      return rows;
    };
    auto any = [&](const Seq &sq) { return sq.left > 0 || blank(sq) > 0; };
    if (!__syncthreads_or(s0 + (int)threadIdx.x < p.tok.n_seqs && any(load_seq(p, s0 + threadIdx.x)))) continue;
    for (int s = s0; s < min(p.tok.n_seqs, s0 + kCombineThreads); ++s) {
      const Seq sq = load_seq(p, s);
      const int rows = blank(sq);
      const int64_t first = (int64_t)sq.row0 * p.q_heads, n = (int64_t)(rows / p.group) * p.q_heads;
      const int rest = rows % p.group;             // a row tile may end inside a token's heads
      for (int64_t i = blockIdx.x * kCombineThreads + threadIdx.x; i < (n + (rest ? p.q_heads : 0)) * (D / 8); i += gridDim.x * kCombineThreads) {
        const int64_t r = i / (D / 8);
        if (r >= n && (r - n) % p.group >= rest) continue;
        reinterpret_cast<uint4 *>(p.out)[(first + r) * (D / 8) + i % (D / 8)] = make_uint4(0, 0, 0, 0);
        if (p.lse && i % (D / 8) == 0) p.lse[first + r] = -INFINITY;
      }
      const int64_t past = first + (int64_t)sq.n * p.q_heads;
      for (int64_t i = blockIdx.x * kCombineThreads + threadIdx.x; i < (int64_t)sq.left * p.q_heads * (D / 8); i += gridDim.x * kCombineThreads) {
        reinterpret_cast<uint4 *>(p.out)[past * (D / 8) + i] = make_uint4(0, 0, 0, 0);
        if (p.lse && i % (D / 8) == 0) p.lse[past + i / (D / 8)] = -INFINITY;
      }
    }
  }
  griddep_wait();                                  // on every path: this grid does not end before the main kernel's
  {
    int n[2], at = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = 2 * threadIdx.x + k, w = i < p.grid ? p.plan[i].w : 0, per = WARPS / combine_split(w & 0xffff);
      n[k] = w ? ((w >> 16) + per - 1) / per : 0;
    }
    int x = n[0] + n[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_items[warp] = x;
    __syncthreads();
    for (int i = 0; i < warp; ++i) at += warp_items[i];
    upto[2 * threadIdx.x] = at + x - n[1], upto[2 * threadIdx.x + 1] = at + x;
    __syncthreads();
  }
  for (int item = blockIdx.x; item < upto[kMostShares - 1]; item += gridDim.x) {
    int share = 0;                                   // the first with more items up to it
#pragma unroll
    for (int o = kMostShares / 2; o > 0; o >>= 1)
      if (upto[share + o - 1] <= item) share += o;
    const int4 plan = p.plan[share];
    const int parts = plan.w & 0xffff, h = plan.y, rt = plan.z;
    const Seq sq = load_seq(p, plan.x);
    const int64_t c0 = (int64_t)share - 1;
    const int split = combine_split(parts), sub = warp % split, rows = WARPS / split;
    const int per = (parts + split - 1) / split, p0 = min(parts, sub * per), p1 = min(parts, p0 + per);
    auto part = [&](int i) { return p.part + (2 * (c0 + i) + (i == 0)) * ROWS * (D + 2); };
    const int row = (item - (share ? upto[share - 1] : 0)) * rows + warp / split, gr = rt * ROWS + row;
    const bool in = row < ROWS && gr < sq.rows;
    float M = -INFINITY, L = 0.f;
    float4 o[VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      for (int i = p0 + lane; i < p1; i += 32) M = fmaxf(M, part(i)[ROWS * D + 2 * row]);
      M = warp_max(M);
      const float ms = M == -INFINITY ? 0.f : M;
      for (int b = p0; b < p1; b += 32) {          // 32 parts at a time: a lane per weight, then all lanes along the row
        const int n = min(32, p1 - b);
        float w = 0.f;
        if (lane < n) {
          const float *ml = part(b + lane) + ROWS * D + 2 * row;
          w = ex2(ml[0] - ms);
          L = add_scaled(L, ml[1], ml[0] - ms);
        }
#pragma unroll 8
        for (int i = lane / LANES; i < (n + 32 / LANES - 1) / (32 / LANES) * (32 / LANES); i += 32 / LANES) {
          const float wi = __shfl_sync(0xffffffffu, w, i);           // 0 past n
          const float *src = part(b + min(i, n - 1)) + row * D;
#pragma unroll
          for (int k = 0; k < VECS; ++k) {
            const int d = (lane % LANES + k * 32) * 4;
            if (d >= D) continue;
            const float4 x = *reinterpret_cast<const float4 *>(src + d);
            if (i < n) o[k].x = fmaf(x.x, wi, o[k].x), o[k].y = fmaf(x.y, wi, o[k].y), o[k].z = fmaf(x.z, wi, o[k].z), o[k].w = fmaf(x.w, wi, o[k].w);
          }
        }
      }
      L = warp_sum(L);
      if constexpr (LANES == 16) {
        o[0].x += __shfl_xor_sync(0xffffffffu, o[0].x, 16), o[0].y += __shfl_xor_sync(0xffffffffu, o[0].y, 16);
        o[0].z += __shfl_xor_sync(0xffffffffu, o[0].z, 16), o[0].w += __shfl_xor_sync(0xffffffffu, o[0].w, 16);
      }
    }
    if (split > 1) {                               // uniform over the CTA
      __syncthreads();                             // the quarters of the rows before have been read
#pragma unroll
      for (int k = 0; k < VECS; ++k)
        if (lane < LANES && lane + k * 32 < D / 4) sums[warp][lane + k * 32] = o[k];
      if (lane == 0) stats[warp] = make_float2(M, L);
      __syncthreads();
      if (sub) continue;
      float ms = M;
      for (int i = 1; i < split; ++i) ms = fmaxf(ms, stats[warp + i].x);
      M = ms, ms = M == -INFINITY ? 0.f : M;
      L = 0.f;
#pragma unroll
      for (int k = 0; k < VECS; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < split; ++i) {
        const float w = ex2(stats[warp + i].x - ms);
        L = add_scaled(L, stats[warp + i].y, stats[warp + i].x - ms);
#pragma unroll
        for (int k = 0; k < VECS; ++k)
          if (lane % LANES + k * 32 < D / 4) {
            const float4 x = sums[warp + i][lane % LANES + k * 32];
            o[k].x = fmaf(x.x, w, o[k].x), o[k].y = fmaf(x.y, w, o[k].y), o[k].z = fmaf(x.z, w, o[k].z), o[k].w = fmaf(x.w, w, o[k].w);
          }
      }
    }
    if (!in) continue;
    const float ms = M == -INFINITY ? 0.f : M;
    const int64_t orow = (int64_t)(sq.row0 + gr / p.group) * p.q_heads + h * p.group + gr % p.group;
    const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
    for (int k = 0; k < VECS; ++k) {
      const int d = (lane % LANES + k * 32) * 4;
      if (d >= D || lane >= LANES) continue;
      Pack<DT, 4> y;
      y.v[0] = E::from(o[k].x * inv), y.v[1] = E::from(o[k].y * inv), y.v[2] = E::from(o[k].z * inv), y.v[3] = E::from(o[k].w * inv);
      *reinterpret_cast<Pack<DT, 4> *>(static_cast<typename E::T *>(p.out) + orow * D + d) = y;
    }
    if (p.lse && lane == 0) p.lse[orow] = L == 0.f ? -INFINITY : (ms + log2f(L)) * kLn2;
  }
}

// Its CTAs: no more than there can be items.
inline unsigned combine_grid(const AttnParams &p, int D, int rows) {
  return (unsigned)std::min<int64_t>((int64_t)p.tok.n_seqs * p.c.heads * p.row_tiles * rows, combine_ctas(D) * std::max(1, pi::current_sms()));
}

// The driver's tensor-map encoder, looked up through the runtime so that the
// library does not link libcuda.
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeFn encoder() {
  static EncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Codes as [n_pages heads][page_size][D]: a page of a head is one z, so every
// coordinate stays small in a cache of any size.
template <int D>
inline bool encode_codes(CUtensorMap *m, const pi_kv_cache &c, uint8_t *base) {
  const EncodeFn enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)c.page_size, (cuuint64_t)c.n_pages * c.heads};
  const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * c.page_size};
  const cuuint32_t box[3] = {(cuuint32_t)(D < 128 ? D : 128), c.page_size % 64 ? 16u : 64u, 1}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : D == 96 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// pi_attn_tc.cu: head_dim up to 128, row_tiles and grid are its own.
cudaError_t run_tc(const AttnParams &p, int dtype, cudaStream_t s);
constexpr int kTcRows = 256;     // query rows of a unit there

}  // namespace attn
