// Attention over the 8-bit cache for many query rows of a key/value head (a
// prompt in chunks), on tcgen05.
//
// A unit is 256 query rows of a (sequence, head), two row tiles of 128; a tile of
// keys has 128.  Per tile and row tile
//   S = Q K^T       128 x 128, fp16 operands in shared memory, sums in TMEM
//   P = 2^(S f - b) fp16, written over S
//   O += P V        P from TMEM, V from shared memory ([token][dim], N-major)
// E4M3 codes are exact in fp16: converter warps widen each tile once for the 256
// rows.  The scales stay out of the operands: a block's K scale is part of the
// factor f of its 16 columns, its V scale 2^ev of their exponent, so
//   P_j = 2^(x_j + ev_j - R),  acc = sum P_j c_j = sum 2^(x_j - R) v_j,
//   L = sum 2^-ev_j P_j = sum 2^(x_j - R),  out = acc / L
// with R + kBoost near the running maximum of x_j + ev_j (within kSlack): no
// multiplication per element of K or V.  L has the range for any two scales (2^-64
// to 2^120): its terms lie between 2^-149 and 2^80.  P_j does not: where a block's
// scale is far below the largest so far (kFar), a pass of its own adds to L the terms
// of those P_j that are 0.
//
// Roles (16 warps, one CTA an SM): 0-3 and 4-7 softmax of the two row tiles, a row
// a thread; 8-11 converters, a token a thread; 12 tile copies and scales; 13 issues
// the products.  One row tile's products run under the other's softmax; K in fp16
// is double-buffered, codes have three stages.
//
// The line of tiles is cut evenly over the CTAs as in pi_attn.cu.
//
// Measured: chunks of up to 512 tokens over caches of up to 8190, 64 bf16 heads of 128
// on 8: 377 us (895 TFLOP/s, 45% of the dense bf16 rate; 128 dims of bf16 spill 162 bytes
// a thread, fp16 132).  A pair of row tiles takes
// 4650 clocks a tile of keys, of which the products hold the tensor pipe for 3230; a
// row tile's softmax, a row a thread, takes 2760.  Tried and slower: one pass of the
// softmax over registers (538 us), both groups on one row tile's tiles of keys in turn
// (435), K of the next tile widened before V of this one (470).
#include "pi_attn.cuh"

using namespace attn;

namespace {

constexpr int kRows = kTcRows, kHalf = 128, kKeys = 128, kBlocks = kKeys / PI_KV_BLOCK;
constexpr int kThreads = 512;      // four warpgroups: register shares are set for each
constexpr int kStages = 3;         // of codes, K and V of a tile in turn
// From P_j = 0, so x_j + ev_j < R - 126, and ev_j >= ev - kFar for every ev so far it
// follows that x_j is 38 or more below the largest x: its weight is nothing.
constexpr int kFar = 94;
// Tiles whose scales and NaN are kept.  Copies run at most 5 tiles ahead of the first
// softmax group, which every unit waits for; the second has no part in units of one
// row tile, so the copies wait until it has read what it needs of a unit's last three.
constexpr int kScaleRing = 8;

// Shared-memory matrix descriptor, 128-byte swizzle: its low word holds the
// address (and lbo), so a step of `bytes` adds bytes / 16 to it.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr & 0x3FFFF) >> 4 | ((lbo >> 4) & 0x3FFF) << 16; }
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;        // groups of 8 rows 1024 bytes apart
// kind::f16, fp16 operands, binary32 sums, M = 128
__device__ __forceinline__ uint32_t idesc(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kHalf >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n mov.b64 y, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHi));
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
// The loads above are complete; v's uses stay behind this.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(float *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int j = 0; j < N; ++j) asm volatile("" : "+f"(v[j]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

template <int D>
struct Smem {                       // byte offsets from a 1024-byte boundary
  static constexpr int SLABS = (D + 63) / 64, SLAB = 128 * 128, TILE = SLABS * SLAB;   // a slab: 64 fp16 dims of 128 rows
  static constexpr int Q = 0, K = Q + 2 * TILE, V = K + 2 * TILE, C = V + TILE, BYTES = C + kStages * 128 * D;
};
struct Bars {
  unsigned long long c_full[kStages], c_empty[kStages];                // codes: copied, widened
  unsigned long long k_full[2], k_empty[2], v_full, v_empty;           // fp16 tiles: written, used
  unsigned long long s_full[2], p_full[2], o_done[2], q_full[2];       // of a row tile: S ready, P ready, O of a tile done, Q of a unit written
  unsigned long long read[2];                                          // the second row tile's group is done with a unit (in turn)
  unsigned long long drain;                                            // after a failure
};

// 16-byte chunk c of 128-byte row r in a 128-byte-swizzled slab.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
// Chunk c (16 codes) of row r of a tile of codes, as the tile copies swizzle it (rows of 96 are not).
template <int D>
__device__ __forceinline__ uint32_t code_at(int r, int c) {
  return D == 64 ? (uint32_t)(r * 64 + ((c ^ (r >> 1 & 3)) << 4)) : D == 96 ? (uint32_t)(r * 96 + c * 16) : sw128(r, c);
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 1) k_attn_tc(const AttnParams p, const __grid_constant__ AttnMaps maps) {
  using E = Elem<DT>;
  using L = Smem<D>;
  extern __shared__ char smem_raw[];
  char *sm = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ Bars bars;
  __shared__ ShareShared share_sm;
  __shared__ float scales[kScaleRing][2][kBlocks];     // K and V scales of a tile's blocks; below 0: no block
  __shared__ int nan_at[kScaleRing][D];                // first position of a tile with a NaN among its values, by dim
  __shared__ int nan_any[kScaleRing], tile_bad[kScaleRing];   // a block is absent
  __shared__ uint32_t tmem_s;
  __shared__ volatile int failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch();
  for (int s = blockIdx.x * kThreads + tid; s < p.tok.n_seqs; s += gridDim.x * kThreads) flag_seq(p, s);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(smem_addr(&bars.c_full[i]), 33);        // the bytes' arrival, and each lane's scale copies
      bar_init(smem_addr(&bars.c_empty[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&bars.k_full[i]), 4);
      bar_init(smem_addr(&bars.k_empty[i]), 1);
      bar_init(smem_addr(&bars.s_full[i]), 1);
      bar_init(smem_addr(&bars.p_full[i]), 4);
      bar_init(smem_addr(&bars.o_done[i]), 1);
      bar_init(smem_addr(&bars.q_full[i]), 4);
      bar_init(smem_addr(&bars.read[i]), 4);
    }
    bar_init(smem_addr(&bars.v_full), 4);
    bar_init(smem_addr(&bars.v_empty), 1);
    bar_init(smem_addr(&bars.drain), 1);
    bar_init_fence();
    failed = 0;
  }
  Share at;
  const bool any = find_share<kRows, kKeys>(p, share_sm, blockIdx.x, &at);
  if (tid == 0) write_plan<kRows, kKeys>(p, any, at);
  if (!any) return;
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_s)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_s;                        // S of the two row tiles, then O of the two

  // A wait that gives up makes every role leave its loop.
  auto wait = [&](unsigned long long *bar, uint32_t parity) {
    const uint32_t a = smem_addr(bar);
    if (__any_sync(0xffffffffu, bar_try(a, parity & 1))) return true;    // one answer for the warp
    const long long from = clock64();
    do {
      if (__any_sync(0xffffffffu, bar_try(a, parity & 1))) return true;
    } while (!__any_sync(0xffffffffu, failed || clock64() - from >= kWaitClocks));
    failed = 1;
    return false;
  };

  // The CTA's units, for each role: work(unit) until it returns false.
  struct Unit {
    uint32_t g, index;       // tiles and units of this CTA before: buffers and phases follow from them
    uint32_t g1, index1;     // of those, the ones with a second row tile
    int s, h, row0, keys, tiles, t0, t1;
    bool two;                // the unit has a second row tile
    int least;               // keys that the unit's first row sees: below, no row masks anything
    Seq sq;
  };
  bool ok = true;
  int copied = -1;                                     // the last stage use whose copies were issued (warp 12)
  auto units = [&](auto work) {
    Unit u;
    u.g = u.index = u.g1 = u.index1 = 0;
    for (int64_t pos = at.begin; pos < at.end; ++u.index) {
      u.sq = at.sq;
      u.s = at.s, u.h = at.h, u.row0 = at.rt * kRows;
      u.keys = unit_keys<kRows>(p, u.sq, at.rt), u.tiles = (u.keys + kKeys - 1) / kKeys;
      u.t0 = (int)(pos - at.u0), u.t1 = (int)min((int64_t)u.tiles, at.end - at.u0);
      u.least = p.causal ? max(0, min(u.sq.len, u.sq.first + u.row0 / p.group + 1)) : u.sq.len;
      u.two = u.row0 + kHalf < u.sq.rows;
      work(u);
      if (!ok) break;
      u.g += u.t1 - u.t0;
      if (u.two) u.g1 += u.t1 - u.t0, ++u.index1;
      pos = at.u0 + u.t1;
      if (pos < at.end && !next_unit<kRows, kKeys>(p, &at)) break;
    }
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int rt = warp >> 2, row = tid & 127;           // row tile, row of it
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, ts = tmem + lanes + rt * 128, to = tmem + lanes + 256 + rt * 128;
    units([&](const Unit &u) {
      // ================= softmax: row u.row0 + 128 rt + row =================
      if (rt && !u.two) return;
      const Seq &sq = u.sq;
      const int h = u.h, t0 = u.t0, t1 = u.t1;
      const uint32_t first = rt ? u.g1 : u.g;            // phases of this row tile's barriers
      const int r = u.row0 + kHalf * rt + row;
      const bool in = r < sq.rows;
      const int i = in ? r / p.group : 0, hq = h * p.group + (in ? r % p.group : 0);
      const int lim = in && p.causal ? max(0, min(sq.len, sq.first + i + 1)) : sq.len;
      const int min_lim = __reduce_min_sync(0xffffffffu, lim);
      float f = fabsf(p.scale);
      {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const typename E::T *>(p.q) +
                                                           (int64_t)(sq.row0 + i) * p.qt + hq * p.qh);
        uint4 raw[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) raw[c] = make_uint4(0, 0, 0, 0);
        if (in) {
          if (p.wide & 1) {
#pragma unroll
            for (int c = 0; c < D / 8; c += 2) load32(src + c, raw[c], raw[c + 1]);
          } else {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) raw[c] = src[c];
          }
        }
        float up = p.scale < 0.f ? -1.f : 1.f;
        if constexpr (DT == PI_DT_BF16) {                // as in pi_attn.cu: the largest finite magnitude to [2^13, 2^14)
          float mx = 0.f;
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 v = f2_get(f2_from16<DT>(raw[c], j));
              mx = fmaxf(mx, fmaxf(fabsf(v.x) < INFINITY ? fabsf(v.x) : 0.f, fabsf(v.y) < INFINITY ? fabsf(v.y) : 0.f));
            }
          const int ex = max((int)(__float_as_uint(mx) >> 23), 27) - 127 - 13;
          if (mx > 0.f) up *= __uint_as_float((unsigned)(127 - ex) << 23), f *= __uint_as_float((unsigned)(127 + ex) << 23);
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          f2 v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = f2_mul(f2_from16<DT>(raw[c], j), f2_of(up, up));
          *reinterpret_cast<uint4 *>(sm + L::Q + rt * L::TILE + c / 8 * L::SLAB + sw128(row, c % 8)) = f2_to16<PI_DT_F16>(v);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars.q_full[rt]));
      }
      float R = -INFINITY, sum = 0.f;
      int largest = 0;                                   // exponent of the V scales so far (biased)
      for (int t = t0; t < t1; ++t) {
        const uint32_t n = first + (t - t0), ring = (u.g + (t - t0)) % kScaleRing;
        const int k0 = t * kKeys;
        if (!wait(&bars.s_full[rt], n)) {
          ok = false;
          return;
        }
        fence_after();
        // Columns of half a tile as they are, masked ones -inf; absent blocks
        // (a bad page, past the sequence) are masked too.
        const float *ks = scales[ring][0], *vs = scales[ring][1];
        const bool masked = k0 + kKeys > min_lim || tile_bad[ring];
        const int own = (int)(__float_as_uint(vs[lane & 7]) >> 23 & 255);
        largest = max(largest, __reduce_max_sync(0xffffffffu, own));
        const bool far = __any_sync(0xffffffffu, own < largest - kFar);      // rare
        auto load = [&](float *x, int half) {
          tmem_ld32(ts + half * 64, x);
          tmem_ld32(ts + half * 64 + 32, x + 32);
          tmem_wait_ld<64>(x);
          if (masked) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int cols = ks[half * 4 + b] < 0.f ? 0 : lim - k0 - half * 64 - 16 * b;
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (j >= cols) x[16 * b + j] = -INFINITY;
            }
          }
        };
        // not negative, and not 0, so that a masked column stays -inf
        auto factor = [&](int b) { return fmaxf(f * fabsf(ks[b]), 1e-37f); };
        auto exponent = [&](int b) { return (float)((int)(__float_as_uint(vs[b]) >> 23 & 255) - 127); };
        float top = -INFINITY;                           // of x + ev
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          float x[64];
          load(x, half);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            float m = x[16 * b];
#pragma unroll
            for (int j = 1; j < 16; ++j) m = fmaxf(m, x[16 * b + j]);
            top = fmaxf(top, fmaf(m, factor(half * 4 + b), exponent(half * 4 + b)));
          }
        }
        const bool over = top - kBoost > R + kSlack;
        if (__any_sync(0xffffffffu, over)) {
          const float Rn = over ? fmaxf(R, top - kBoost) : R;
          const float by = R == Rn ? 0.f : R - Rn, c = ex2(by);
          R = Rn;
          sum = add_scaled(0.f, sum, by);
          if (t > t0) {                                  // O is the products' until the tile before is done
            if (!wait(&bars.o_done[rt], n - 1)) {
              ok = false;
              return;
            }
            fence_after();
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              float o[32];
              tmem_ld32(to + q * 32, o);
              tmem_wait_ld<32>(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] *= c;
              tmem_st32(to + q * 32, reinterpret_cast<const uint32_t *>(o));
            }
            tmem_wait_st();
          }
        }
        const float Rs = R == -INFINITY ? 0.f : R;
        if (far) {
#pragma unroll 1
          for (int b = 0; b < kBlocks; b += 2) {
            float x[32];
            tmem_ld32(ts + b * 16, x);
            tmem_wait_ld<32>(x);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float fb = factor(b + e), ev = exponent(b + e), bias = ev - Rs;
              const int cols = ks[b + e] < 0.f ? 0 : lim - k0 - 16 * (b + e);
              float part = 0.f;
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float z = fmaf(x[16 * e + j], fb, bias);       // as below, where 2^z is 0 from -126 down
                part += j < cols && z < -126.f ? ex2(z + 100.f) : 0.f;
              }
              if (ev < (float)(largest - 127 - kFar)) sum = fmaf(part, ex2(-ev - 100.f), sum);
            }
          }
        }
        // P takes the first 64 columns of S: its second half is written there only after S's is read
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          float x[64];
          load(x, half);
          uint32_t w[32];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float fb = factor(half * 4 + b), ev = exponent(half * 4 + b), bias = ev - Rs;
            f2 part = f2_of(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const f2 z = f2_fma(f2_of(x[16 * b + 2 * j], x[16 * b + 2 * j + 1]), f2_of(fb, fb), f2_of(bias, bias));
              const f2 e = f2_of(ex2(z.x), ex2(z.y));
              part = f2_add(part, e);
              w[b * 8 + j] = f2_narrow<PI_DT_F16>(e);
            }
            sum = fmaf(f2_sum(part), ex2(-ev), sum);
          }
          tmem_st32(ts + half * 32, w);
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars.p_full[rt]));
      }
      // ---- the unit's result, or this CTA's part of it ----
      if (!wait(&bars.o_done[rt], first + (t1 - t0) - 1)) {
        ok = false;
        return;
      }
      fence_after();
      const bool whole = t0 == 0 && t1 == u.tiles;
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
      const int64_t orow = (int64_t)(sq.row0 + i) * p.q_heads + hq;
      float *part = p.part + (int64_t)(2 * blockIdx.x + (t0 == 0)) * kRows * (D + 2);
      const int pr = kHalf * rt + row;
      bool nan = false;                                  // some tile has NaN that some rows do not see
      for (int t = max(t0, u.least / kKeys); t < t1; ++t) nan |= nan_any[(u.g + (t - t0)) % kScaleRing] != 0;
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        tmem_ld32(to + q * 32, o);
        tmem_wait_ld<32>(o);
        if (nan) {
          for (int t = max(t0, u.least / kKeys); t < t1; ++t) {
            const int ring = (u.g + (t - t0)) % kScaleRing;
            if (!nan_any[ring]) continue;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (nan_at[ring][q * 32 + j] < lim) o[j] = __uint_as_float(0x7fffffffu);
          }
        }
        if (whole) {
          if (in) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<typename E::T *>(p.out) + orow * D + q * 32);
            uint4 y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              f2 v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = f2_mul(f2_of(o[8 * c + 2 * j], o[8 * c + 2 * j + 1]), f2_of(inv, inv));
              y[c] = f2_to16<DT>(v);
            }
            if (p.wide & 2) {
              store32(dst, y[0], y[1]), store32(dst + 2, y[2], y[3]);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c) dst[c] = y[c];
            }
          }
        } else {
          uint4 *dst = reinterpret_cast<uint4 *>(part + pr * D + q * 32);
          const uint32_t *y = reinterpret_cast<const uint32_t *>(o);
#pragma unroll
          for (int c = 0; c < 8; c += 2) {
            const uint4 a = make_uint4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
            const uint4 b = make_uint4(y[4 * c + 4], y[4 * c + 5], y[4 * c + 6], y[4 * c + 7]);
            if (p.wide & 4) store32(dst + c, a, b);
            else dst[c] = a, dst[c + 1] = b;
          }
        }
      }
      fence_before();
      if (!whole) {
        part[kRows * D + 2 * pr] = R, part[kRows * D + 2 * pr + 1] = sum;
      } else if (in && p.lse) {
        p.lse[orow] = sum == 0.f ? -INFINITY : ((R == -INFINITY ? 0.f : R) + log2f(sum)) * kLn2;
      }
      if (rt) {
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars.read[u.index1 & 1]));
      }
    });
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    const int r = tid - 256;
    units([&](const Unit &u) {
      // ================= converters: token r of each tile =================
      const Seq &sq = u.sq;
      for (int t = u.t0; t < u.t1; ++t) {
        const uint32_t gt = u.g + (t - u.t0), b = gt & 1, ring = gt % kScaleRing;
        const int k0 = t * kKeys;
        uint4 c[D / 16];
        bool there = false;
        auto store = [&](char *tile) {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint4 lo, hi;
            widen4(c[j].x, lo.x, lo.y);
            widen4(c[j].y, lo.z, lo.w);
            widen4(c[j].z, hi.x, hi.y);
            widen4(c[j].w, hi.z, hi.w);
            *reinterpret_cast<uint4 *>(tile + j / 4 * L::SLAB + sw128(r, j % 4 * 2)) = lo;
            *reinterpret_cast<uint4 *>(tile + j / 4 * L::SLAB + sw128(r, j % 4 * 2 + 1)) = hi;
          }
          fence_async_smem();
          __syncwarp();
        };
        auto codes = [&](uint32_t use) {                 // of stage use `use`; the stage is free again
          const uint32_t st = use % kStages;
          if (!wait(&bars.c_full[st], use / kStages)) return false;
          const char *src = sm + L::C + st * 128 * D;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) c[j] = *reinterpret_cast<const uint4 *>(src + code_at<D>(r, j));
          there = k0 + r < sq.len && scales[ring][0][r / PI_KV_BLOCK] >= 0.f;
          __syncwarp();
          if (lane == 0) bar_arrive(smem_addr(&bars.c_empty[st]));
          return true;
        };
        // K
        if (!codes(2 * gt) || (gt >= 2 && !wait(&bars.k_empty[b], (gt >> 1) - 1))) {
          ok = false;
          return;
        }
        store(sm + L::K + b * L::TILE);
        if (lane == 0) bar_arrive(smem_addr(&bars.k_full[b]));
        // V
        if (!codes(2 * gt + 1)) {
          ok = false;
          return;
        }
        if (!there) {                                    // whatever the page held before, or nothing
#pragma unroll
          for (int j = 0; j < D / 16; ++j) c[j] = make_uint4(0, 0, 0, 0);
        }
        if (k0 + kKeys > u.least) {
          // A NaN among tokens that only some rows see would reach the others as
          // 0 * NaN: it is taken out, and each dim's first position with one noted.
          bool nan = false;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const unsigned w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) nan |= __vcmpeq4(w[e] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
          }
          if (nan) {
            nan_any[ring] = 1;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              unsigned w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const unsigned is = __vcmpeq4(w[e] & 0x7f7f7f7fu, 0x7f7f7f7fu);
#pragma unroll 1
                for (unsigned left = is; left;) {
                  const int k = (__ffs(left) - 1) / 8;
                  left &= ~(255u << (8 * k));
                  atomicMin(&nan_at[ring][16 * j + 4 * e + k], k0 + r);
                }
                w[e] &= ~is;
              }
              c[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
        }
        if (gt >= 1 && !wait(&bars.v_empty, gt - 1)) {
          ok = false;
          return;
        }
        store(sm + L::V);
        if (lane == 0) bar_arrive(smem_addr(&bars.v_full));
      }
    });
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 12) {
      uint32_t end1 = 0;                                 // tiles up to the end of the last unit with two row tiles
      units([&](const Unit &u) {
        // ================= tile copies; lane l looks after block l % 8 =================
        const int32_t *table = p.tok.page_table + (int64_t)u.s * p.tok.table_stride;
        const int P = p.c.page_size, blocks = P / PI_KV_BLOCK, limit = min(u.keys, u.t1 * kKeys);
        const int step = P % 64 ? 1 : 4;                 // boxes of 64 tokens where pages hold whole ones, else of 16
        for (int t = u.t0; t < u.t1; ++t) {
          const uint32_t gt = u.g + (t - u.t0), ring = gt % kScaleRing;
          // Of the units with two row tiles before this one, all but the last are done with their tiles
          // (a barrier for every other one, so that none is a phase ahead); the last with its last three
          // where this tile takes their places.
          if ((t == u.t0 && u.index1 >= 2 && !wait(&bars.read[u.index1 & 1], (u.index1 >> 1) - 1)) ||
              (u.index1 >= 1 && gt == end1 + kScaleRing - 3 && !wait(&bars.read[(u.index1 - 1) & 1], (u.index1 - 1) >> 1))) {
            ok = false;
            return;
          }
          const int k = t * kKeys + (lane & 7) * 16, cp = k / P, co = k - cp * P;
          const bool has = k < limit;
          const int page = has ? table[cp] : -1;
          const bool good = page >= 0 && page < p.c.n_pages;
          if (has && !good && lane < 8) atomicOr(p.c.status, pi::kKvBadPage);
          const unsigned mask = __ballot_sync(0xffffffffu, good) & 255u;
          int n_boxes = 0;
          for (int b = 0; b < kBlocks; b += step) n_boxes += mask >> b & 1;
          auto copy = [&](const CUtensorMap *map, uint32_t use, bool with_scales) {
            const uint32_t st = use % kStages, bar = smem_addr(&bars.c_full[st]);
            if (use >= kStages && !wait(&bars.c_empty[st], use / kStages - 1)) return false;
            if (with_scales) {
              if (lane < 16) {
                float *dst = &scales[ring][lane >> 3][lane & 7];
                if (good)
                  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)),
                               "l"((lane >> 3 ? p.c.v_scales : p.c.k_scales) + ((int64_t)page * p.c.heads + u.h) * blocks + co / PI_KV_BLOCK)
                               : "memory");
                else
                  *dst = -1.f;
              }
              if (lane == 0) tile_bad[ring] = mask != 255u;
            } else if (t * kKeys + kKeys > u.least) {    // a tile whose NaN are noted
              for (int d = lane; d < D; d += 32) nan_at[ring][d] = 0x7fffffff;
              if (lane == 0) nan_any[ring] = 0;
            }
            __syncwarp();
            if (elect_one()) bar_expect(bar, (uint32_t)n_boxes * step * 16 * D);
            __syncwarp();
#pragma unroll 1
            for (int b = 0; b < kBlocks; b += step) {
              const int z = __shfl_sync(0xffffffffu, page, b) * p.c.heads + u.h, y = __shfl_sync(0xffffffffu, co, b);
              if ((mask >> b & 1) && elect_one()) tile_copy(smem_addr(sm + L::C + st * 128 * D + b * 16 * D), map, 0, y, z, bar);
              __syncwarp();
            }
            if (with_scales && lane < 16 && good) bar_arrive_copies(bar); else bar_arrive(bar);
            copied = (int)use;
            return true;
          };
          if (!copy(&maps.k, 2 * gt, true) || !copy(&maps.v, 2 * gt + 1, false)) {
            ok = false;
            return;
          }
        }
        if (u.two) end1 = u.g + (u.t1 - u.t0);
      });
    } else if (warp == 13) {
      const uint32_t id_s = idesc(kKeys, false), id_o = idesc(D, true);
      const uint32_t q_lo = desc_lo(smem_addr(sm + L::Q), 16), k_lo = desc_lo(smem_addr(sm + L::K), 16), v_lo = desc_lo(smem_addr(sm + L::V), L::SLAB);
      units([&](const Unit &u) {
        // ================= products =================
        const int n_rt = u.two ? 2 : 1;
        auto issue_s = [&](int rt, uint32_t gt) {        // S of a row tile; K's buffer is free after the last row tile's
          if (rt == 0 && !wait(&bars.k_full[gt & 1], gt >> 1)) return false;
          fence_after();
          if (elect_one()) {
            const uint32_t q = q_lo + rt * (L::TILE >> 4), k = k_lo + (gt & 1) * (L::TILE >> 4);
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
              const uint32_t o = (e / 4 * L::SLAB + e % 4 * 32) >> 4;
              mma_ss(tmem + rt * 128, q + o, k + o, id_s, e > 0);
            }
            if (rt == n_rt - 1) mma_commit(smem_addr(&bars.k_empty[gt & 1]));
            mma_commit(smem_addr(&bars.s_full[rt]));
          }
          __syncwarp();
          return true;
        };
        for (int rt = 0; ok && rt < n_rt; ++rt) ok = wait(&bars.q_full[rt], rt ? u.index1 : u.index) && issue_s(rt, u.g);
        for (int t = u.t0; ok && t < u.t1; ++t) {
          const uint32_t gt = u.g + (t - u.t0);
          ok = wait(&bars.v_full, gt);
          for (int rt = 0; ok && rt < n_rt; ++rt) {
            if (!wait(&bars.p_full[rt], (rt ? u.g1 : u.g) + (t - u.t0))) {
              ok = false;
              break;
            }
            fence_after();
            if (elect_one()) {
#pragma unroll
              for (int e = 0; e < kKeys / 16; ++e)
                mma_ts(tmem + 256 + rt * 128, tmem + rt * 128 + e * 8, v_lo + e * (2048 >> 4), id_o, t > u.t0 || e > 0);
              if (rt == n_rt - 1) mma_commit(smem_addr(&bars.v_empty));
              mma_commit(smem_addr(&bars.o_done[rt]));
            }
            __syncwarp();
            if (t + 1 < u.t1) ok = issue_s(rt, gt + 1);
          }
        }
      });
    }
  }
  // Copies and products on their way land before the CTA leaves (bounded).
  if (!ok) {
    failed = 1;
    if (lane == 0) atomicOr(p.c.status, pi::kKvTimeout);
    if (warp == 12 && copied >= 0)                       // stages fill in order, up to kStages of them on their way
      for (int use = max(0, copied - kStages + 1); use <= copied; ++use)
        bar_wait(smem_addr(&bars.c_full[use % kStages]), use / kStages & 1);
    if (warp == 13) {                                  // a commit follows every product before it
      if (elect_one()) mma_commit(smem_addr(&bars.drain));
      __syncwarp();
      bar_wait(smem_addr(&bars.drain), 0);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 13) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int DT, int D>
cudaError_t launch(AttnParams p, cudaStream_t s) {
  constexpr int smem = Smem<D>::BYTES + 1024;
  AttnMaps maps;
  if (!encode_codes<D>(&maps.k, p.c, p.c.k_codes) || !encode_codes<D>(&maps.v, p.c, p.c.v_codes)) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = pi::allow_smem(k_attn_tc<DT, D>, smem, smem, done);
  if (e != cudaSuccess) return e;
  p.row_tiles = (int)(((int64_t)p.max_q * p.group + kRows - 1) / kRows);
  p.grid = std::min(kMostShares, std::max(1, pi::current_sms()));
  k_attn_tc<DT, D><<<p.grid, kThreads, smem, s>>>(p, maps);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return pi::launch_pdl(k_attn_combine<DT, D, kRows, kKeys>, dim3(combine_grid(p, D, kRows)), dim3(kCombineThreads), 0, s, p);
}

}  // namespace

namespace attn {

cudaError_t run_tc(const AttnParams &p, int dtype, cudaStream_t s) {
  if (p.c.head_dim == 64) return dtype == PI_DT_F16 ? launch<PI_DT_F16, 64>(p, s) : launch<PI_DT_BF16, 64>(p, s);
  if (p.c.head_dim == 96) return dtype == PI_DT_F16 ? launch<PI_DT_F16, 96>(p, s) : launch<PI_DT_BF16, 96>(p, s);
  return dtype == PI_DT_F16 ? launch<PI_DT_F16, 128>(p, s) : launch<PI_DT_BF16, 128>(p, s);
}

}  // namespace attn
