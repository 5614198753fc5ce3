// Attention over the 8-bit cache for many query rows of a key/value head (a
// prompt in chunks), on tcgen05.
//
// A unit is 128 query rows of a (sequence, head); a tile 128 keys.  Per tile
//   S = Q K^T       128 x 128, fp16 operands in shared memory, sums in TMEM
//   P = 2^(S f - b) fp16, written over S
//   O += P V        P from TMEM, V from shared memory ([token][dim], N-major)
// E4M3 codes are exact in fp16: converter warps widen each tile once for the 128
// rows.  The scales stay out of the operands: a block's K scale is part of the
// factor f of its 16 columns, its V scale 2^ev of their exponent, so
//   P_j = 2^(x_j + ev_j - R),  acc = sum P_j c_j = sum 2^(x_j - R) v_j,
//   L = sum 2^-ev_j P_j = sum 2^(x_j - R),  out = acc / L
// with R + kBoost near the running maximum of x_j + ev_j (within kSlack): no
// multiplication per element of K or V, and scales of any range.
//
// Bound by the tensor cores where the softmax keeps up: a tile is 4 x 128 x 128 x D
// operations there, and 128 exponentials and about 450 instructions of each of
// the 128 softmax threads.  Roles (12 warps, one CTA an SM): 0-3 softmax, a row a
// thread; 4-7 converters, a token a thread; 8 tile copies and scales; 9 issues the
// products.  K and V are double-buffered in fp16, S in TMEM, so the next S and the
// conversion run under a tile's softmax.
//
// The line of tiles is cut evenly over the CTAs as in pi_attn.cu.
#include "pi_attn.cuh"

using namespace attn;

namespace {

constexpr int kRows = kTcRows, kKeys = 128, kBlocks = kKeys / PI_KV_BLOCK;
constexpr int kThreads = 384;      // three warpgroups: register shares are set for each
constexpr int kScaleRing = 8;    // tiles whose scales are kept: copies run at most 5 tiles ahead of the softmax

__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  // shared-memory matrix descriptor, 128-byte swizzle
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFF) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFF) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// kind::f16, fp16 operands, binary32 sums, M = 128
__device__ __forceinline__ uint32_t idesc(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
               "l"(a), "l"(b), "r"(id), "r"(acc));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
               "r"(a), "l"(b), "r"(id), "r"(acc));
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
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

template <int D>
struct Smem {                       // byte offsets from a 1024-byte boundary
  static constexpr int SLABS = D / 64, SLAB = 128 * 128;               // 64 fp16 dims of 128 rows
  static constexpr int Q = 0, K = Q + SLABS * SLAB, V = K + 2 * SLABS * SLAB, CK = V + 2 * SLABS * SLAB, CV = CK + 128 * D;
  static constexpr int BYTES = CV + 128 * D;
};
struct Bars {
  unsigned long long ck_full, ck_empty, cv_full, cv_empty;             // codes of a tile: copied, widened
  unsigned long long k_full[2], k_empty[2], v_full[2], v_empty[2];     // fp16 tiles: written, used
  unsigned long long s_full[2], p_full[2], o_done, q_full, drain;      // S ready, P ready, a tile's O done, Q of a unit written; after a failure
};

// 16-byte chunk c of 128-byte row r in a 128-byte-swizzled slab.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
// Chunk c (16 codes) of row r of a tile of codes, as the tile copies swizzle it.
template <int D>
__device__ __forceinline__ uint32_t code_at(int r, int c) {
  return D == 64 ? (uint32_t)(r * 64 + ((c ^ (r >> 1 & 3)) << 4)) : sw128(r, c);
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
  __shared__ int nan_any[kScaleRing];
  __shared__ uint32_t tmem_s;
  __shared__ volatile int failed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch();
  for (int s = blockIdx.x * kThreads + tid; s < p.tok.n_seqs; s += gridDim.x * kThreads) flag_seq(p, s);
  if (tid == 0) {
    bar_init(smem_addr(&bars.ck_full), 33);            // the bytes' arrival, and each lane's scale copies
    bar_init(smem_addr(&bars.ck_empty), 4);
    bar_init(smem_addr(&bars.cv_full), 1);
    bar_init(smem_addr(&bars.cv_empty), 4);
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&bars.k_full[i]), 4);
      bar_init(smem_addr(&bars.k_empty[i]), 1);
      bar_init(smem_addr(&bars.v_full[i]), 4);
      bar_init(smem_addr(&bars.v_empty[i]), 1);
      bar_init(smem_addr(&bars.s_full[i]), 1);
      bar_init(smem_addr(&bars.p_full[i]), 4);
    }
    bar_init(smem_addr(&bars.o_done), 1);
    bar_init(smem_addr(&bars.q_full), 4);
    bar_init(smem_addr(&bars.drain), 1);
    bar_init_fence();
    failed = 0;
  }
  Share at;
  if (!find_share<kRows, kKeys>(p, share_sm, &at)) return;
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_s)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_s, tmem_o = tmem + 256;

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
    int s, h, row0, keys, tiles, t0, t1;
    int least;               // keys that the unit's first row sees: below, no row masks anything
    Seq sq;
  };
  bool ok = true;
  int ck_tile = -1, cv_tile = -1;                      // last tiles whose copies were issued (warp 8)
  auto units = [&](auto work) {
    Unit u;
    u.g = u.index = 0;
    for (int64_t pos = at.begin; pos < at.end; ++u.index) {
      u.sq = at.sq;
      u.s = at.s, u.h = at.h, u.row0 = at.rt * kRows;
      u.keys = unit_keys<kRows>(p, u.sq, at.rt), u.tiles = (u.keys + kKeys - 1) / kKeys;
      u.t0 = (int)(pos - at.u0), u.t1 = (int)min((int64_t)u.tiles, at.end - at.u0);
      u.least = p.causal ? max(0, min(u.sq.len, u.sq.first + u.row0 / p.group + 1)) : u.sq.len;
      work(u);
      if (!ok) break;
      u.g += u.t1 - u.t0;
      pos = at.u0 + u.t1;
      if (pos < at.end && !next_unit<kRows, kKeys>(p, &at)) break;
    }
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
    units([&](const Unit &u) {
      // ================= softmax: row row0 + tid =================
      const Seq &sq = u.sq;
      const uint32_t g = u.g;
      const int h = u.h, t0 = u.t0, t1 = u.t1;
      const int row0 = u.row0, tiles = u.tiles, least = u.least;
      const int r = row0 + tid;
      const bool in = r < sq.rows;
      const int i = in ? r / p.group : 0, hq = h * p.group + (in ? r % p.group : 0);
      const int lim = in && p.causal ? max(0, min(sq.len, sq.first + i + 1)) : sq.len;
      float f = fabsf(p.scale);
      {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const typename E::T *>(p.q) +
                                                           (int64_t)(sq.row0 + i) * p.qt + hq * p.qh);
        uint4 raw[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) raw[c] = make_uint4(0, 0, 0, 0);
        if (in) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) raw[c] = src[c];
        }
        float up = p.scale < 0.f ? -1.f : 1.f;         // the factor f is never negative
        if constexpr (DT == PI_DT_BF16) {              // as in pi_attn.cu: the largest finite magnitude to [2^13, 2^14)
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
          *reinterpret_cast<uint4 *>(sm + L::Q + c / 8 * L::SLAB + sw128(tid, c % 8)) = f2_to16<PI_DT_F16>(v);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars.q_full));
      }
      float R = -INFINITY, sum = 0.f;
      const uint32_t lanes = (uint32_t)(warp * 32) << 16;
      uint32_t gt = g;
      for (int t = t0; t < t1; ++t, ++gt) {
        const uint32_t tb = tmem + lanes + (gt & 1) * 128;
        if (!wait(&bars.s_full[gt & 1], gt >> 1)) {
          ok = false;
          break;
        }
        fence_after();
        float x[kKeys];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tb + c * 32, x + 32 * c);
        tmem_wait_ld();
        const float(*sc)[kBlocks] = scales[gt % kScaleRing];
        const int k0 = t * kKeys;
        float fb[kBlocks], ev[kBlocks];
        float top = -INFINITY;                         // of x + ev
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const float ks = sc[0][b];
          // absent blocks (a bad page, past the sequence) are masked with the columns
          const int cols = ks < 0.f ? 0 : lim - (k0 + 16 * b);
          fb[b] = f * ks;
          ev[b] = (float)((int)(__float_as_uint(sc[1][b]) >> 23 & 255) - 127);
          float m = -INFINITY;
          if (cols >= 16) {
#pragma unroll
            for (int j = 0; j < 16; ++j) m = fmaxf(m, x[16 * b + j]);
            m = m * fb[b];
          } else {
            fb[b] = 1.f;                               // scaled here, so that a masked column is -inf whatever the factor
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              x[16 * b + j] = j < cols ? x[16 * b + j] * (f * ks) : -INFINITY;
              m = fmaxf(m, x[16 * b + j]);
            }
            if (cols <= 0) ev[b] = 0.f;
          }
          top = fmaxf(top, m + ev[b]);
        }
        const bool over = top - kBoost > R + kSlack;
        if (__any_sync(0xffffffffu, over)) {
          const float Rn = over ? fmaxf(R, top - kBoost) : R;
          const float c = R == Rn || Rn == -INFINITY ? 1.f : ex2(R - Rn);
          R = Rn;
          sum *= c;
          if (t > t0) {                                // O is the products' until the tile before is done
            if (!wait(&bars.o_done, gt - 1)) {
              ok = false;
              break;
            }
            fence_after();
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              float o[32];
              tmem_ld32(tmem_o + lanes + q * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] *= c;
              tmem_st32(tmem_o + lanes + q * 32, reinterpret_cast<const uint32_t *>(o));
            }
            tmem_wait_st();
          }
        }
        const float Rs = R == -INFINITY ? 0.f : R;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[32];
#pragma unroll
          for (int bb = 0; bb < 4; ++bb) {
            const int b = half * 4 + bb;
            const float bias = ev[b] - Rs;
            f2 part = f2_of(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const f2 z = f2_fma(f2_of(x[16 * b + 2 * j], x[16 * b + 2 * j + 1]), f2_of(fb[b], fb[b]), f2_of(bias, bias));
              const f2 e = f2_of(ex2(z.x), ex2(z.y));
              part = f2_add(part, e);
              w[bb * 8 + j] = f2_narrow<PI_DT_F16>(e);
            }
            sum = fmaf(f2_sum(part), ex2(-ev[b]), sum);
          }
          tmem_st32(tb + half * 32, w);
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars.p_full[gt & 1]));
      }
      // ---- the unit's result, or this CTA's part of it ----
      if (ok && !wait(&bars.o_done, gt - 1)) ok = false;
      if (ok) {
        fence_after();
        const bool whole = t0 == 0 && t1 == tiles;
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
        const int64_t orow = (int64_t)(sq.row0 + i) * p.q_heads + hq;
        float *part = p.part + (int64_t)(2 * blockIdx.x + (t0 == 0)) * kRows * (D + 2);
        int first_nan = -1;                            // ring place of the first tile with a NaN that some rows do not see
        for (int t = max(t0, least / kKeys); t < t1; ++t)
          if (nan_any[(g + t - t0) % kScaleRing]) {
            first_nan = t;
            break;
          }
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          float o[32];
          tmem_ld32(tmem_o + lanes + q * 32, o);
          tmem_wait_ld();
          if (first_nan >= 0) {
            for (int t = first_nan; t < t1; ++t) {
              if (!nan_any[(g + t - t0) % kScaleRing]) continue;
              const int *n = nan_at[(g + t - t0) % kScaleRing] + q * 32;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (n[j] < lim) o[j] = __uint_as_float(0x7fffffffu);
            }
          }
          if (whole) {
            if (in) {
              uint4 *dst = reinterpret_cast<uint4 *>(static_cast<typename E::T *>(p.out) + orow * D + q * 32);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                f2 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = f2_mul(f2_of(o[8 * c + 2 * j], o[8 * c + 2 * j + 1]), f2_of(inv, inv));
                dst[c] = f2_to16<DT>(v);
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<float4 *>(part + tid * D + q * 32 + 4 * c) = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
        }
        fence_before();
        if (!whole) {
          part[kRows * D + 2 * tid] = R, part[kRows * D + 2 * tid + 1] = sum;
        } else if (in && p.lse) {
          p.lse[orow] = sum == 0.f ? -INFINITY : ((R == -INFINITY ? 0.f : R) + log2f(sum)) * kLn2;
        }
      }
    });
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    units([&](const Unit &u) {
      // ================= converters: token tid - 128 of each tile =================
      const Seq &sq = u.sq;
      const uint32_t g = u.g;
      const int t0 = u.t0, t1 = u.t1, least = u.least;
      const int r = tid - 128;
      uint32_t gt = g;
      for (int t = t0; t < t1; ++t, ++gt) {
        const int b = gt & 1, k0 = t * kKeys, ring = gt % kScaleRing;
        // K
        if (!wait(&bars.ck_full, gt) || (gt >= 2 && !wait(&bars.k_empty[b], (gt >> 1) - 1))) {
          ok = false;
          break;
        }
        const bool there = k0 + r < sq.len && scales[ring][0][r / PI_KV_BLOCK] >= 0.f;
        uint4 c[D / 16];
#pragma unroll
        for (int j = 0; j < D / 16; ++j) c[j] = *reinterpret_cast<const uint4 *>(sm + L::CK + code_at<D>(r, j));
        auto store = [&](int base) {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint4 lo, hi;
            widen4(c[j].x, lo.x, lo.y);
            widen4(c[j].y, lo.z, lo.w);
            widen4(c[j].z, hi.x, hi.y);
            widen4(c[j].w, hi.z, hi.w);
            char *slab = sm + base + (b * L::SLABS + j / 4) * L::SLAB;
            *reinterpret_cast<uint4 *>(slab + sw128(r, j % 4 * 2)) = lo;
            *reinterpret_cast<uint4 *>(slab + sw128(r, j % 4 * 2 + 1)) = hi;
          }
        };
        store(L::K);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars.ck_empty)), bar_arrive(smem_addr(&bars.k_full[b]));
        // V
        if (!wait(&bars.cv_full, gt) || (gt >= 2 && !wait(&bars.v_empty[b], (gt >> 1) - 1))) {
          ok = false;
          break;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) c[j] = *reinterpret_cast<const uint4 *>(sm + L::CV + code_at<D>(r, j));
        if (!there) {                                  // whatever the page held before, or nothing
#pragma unroll
          for (int j = 0; j < D / 16; ++j) c[j] = make_uint4(0, 0, 0, 0);
        }
        if (k0 + kKeys > least) {
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
#pragma unroll 1
            for (int d = 0; d < D; ++d) {
              const int j = d / 16, e = d % 16 / 4, sh = d % 4 * 8;
              unsigned v = 0;
#pragma unroll
              for (int jj = 0; jj < D / 16; ++jj)
                if (jj == j) v = e == 0 ? c[jj].x : e == 1 ? c[jj].y : e == 2 ? c[jj].z : c[jj].w;
              if ((v >> sh & 0x7f) == 0x7f) atomicMin(&nan_at[ring][d], k0 + r);
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              c[j].x &= ~__vcmpeq4(c[j].x & 0x7f7f7f7fu, 0x7f7f7f7fu);
              c[j].y &= ~__vcmpeq4(c[j].y & 0x7f7f7f7fu, 0x7f7f7f7fu);
              c[j].z &= ~__vcmpeq4(c[j].z & 0x7f7f7f7fu, 0x7f7f7f7fu);
              c[j].w &= ~__vcmpeq4(c[j].w & 0x7f7f7f7fu, 0x7f7f7f7fu);
            }
          }
        }
        store(L::V);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars.cv_empty)), bar_arrive(smem_addr(&bars.v_full[b]));
      }
    });
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == 8) {
    units([&](const Unit &u) {
      // ================= tile copies; lane l looks after block l % 8 =================
      const uint32_t g = u.g;
      const int s = u.s, h = u.h, t0 = u.t0, t1 = u.t1, keys = u.keys, least = u.least;
      const int32_t *table = p.tok.page_table + (int64_t)s * p.tok.table_stride;
      const int P = p.c.page_size, blocks = P / PI_KV_BLOCK, limit = min(keys, t1 * kKeys);
      const bool by16 = P % 64 != 0;
      uint32_t gt = g;
      for (int t = t0; t < t1; ++t, ++gt) {
        const int k = t * kKeys + (lane & 7) * 16, cp = k / P, co = k - cp * P;
        const bool has = k < limit;
        const int page = has ? table[cp] : -1;
        const bool good = page >= 0 && page < p.c.n_pages;
        if (has && !good && lane < 8) atomicOr(p.c.status, pi::kKvBadPage);
        const unsigned mask = __ballot_sync(0xffffffffu, good) & 255u;
        const int ring = gt % kScaleRing;
        if (gt >= 1 && !wait(&bars.ck_empty, gt - 1)) {
          ok = false;
          break;
        }
        if (lane < 16) {
          float *dst = &scales[ring][lane >> 3][lane & 7];
          if (good)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)),
                         "l"((lane >> 3 ? p.c.v_scales : p.c.k_scales) + ((int64_t)page * p.c.heads + h) * blocks + co / PI_KV_BLOCK)
                         : "memory");
          else
            *dst = -1.f;
        }
        // boxes of 64 tokens where pages hold whole ones, else of 16
        const int step = by16 ? 1 : 4;
        int n_boxes = 0;
        for (int b = 0; b < kBlocks; b += step) n_boxes += mask >> b & 1;
        const uint32_t bytes = (uint32_t)n_boxes * step * 16 * D;
        auto copy = [&](const CUtensorMap *map, int base, unsigned long long *bar) {
          if (elect_one()) bar_expect(smem_addr(bar), bytes);
          __syncwarp();
#pragma unroll 1
          for (int b = 0; b < kBlocks; b += step) {
            const int z = __shfl_sync(0xffffffffu, page, b) * p.c.heads + h, y = __shfl_sync(0xffffffffu, co, b);
            if ((mask >> b & 1) && elect_one()) tile_copy(smem_addr(sm + base + b * 16 * D), map, 0, y, z, smem_addr(bar));
            __syncwarp();
          }
        };
        copy(&maps.k, L::CK, &bars.ck_full);
        ck_tile = gt;
        if (lane < 16 && good) bar_arrive_copies(smem_addr(&bars.ck_full)); else bar_arrive(smem_addr(&bars.ck_full));
        if (gt >= 1 && !wait(&bars.cv_empty, gt - 1)) {
          ok = false;
          break;
        }
        if (t * kKeys + kKeys > least) {               // a tile whose NaN are noted
          for (int d = lane; d < D; d += 32) nan_at[ring][d] = 0x7fffffff;
          if (lane == 0) nan_any[ring] = 0;
          __syncwarp();
        }
        copy(&maps.v, L::CV, &bars.cv_full);
        cv_tile = gt;
      }
    });
    } else if (warp == 9) {
    units([&](const Unit &u) {
      // ================= products =================
      const uint32_t g = u.g;
      const int t0 = u.t0, t1 = u.t1;
      const uint32_t id_s = idesc(kKeys, false), id_o = idesc(D, true);
      auto issue_s = [&](uint32_t gt) {
        if (!wait(&bars.k_full[gt & 1], gt >> 1)) return false;
        fence_after();
        if (elect_one()) {
          const uint32_t q = smem_addr(sm + L::Q), k = smem_addr(sm + L::K + (gt & 1) * L::SLABS * L::SLAB);
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint32_t o = e / 4 * L::SLAB + e % 4 * 32;
            mma_ss(tmem + (gt & 1) * 128, sdesc(q + o, 16, 1024), sdesc(k + o, 16, 1024), id_s, e > 0);
          }
          mma_commit(smem_addr(&bars.k_empty[gt & 1]));
          mma_commit(smem_addr(&bars.s_full[gt & 1]));
        }
        __syncwarp();
        return true;
      };
      ok = wait(&bars.q_full, u.index) && issue_s(g);
      uint32_t gt = g;
      for (int t = t0; ok && t < t1; ++t, ++gt) {
        if (t + 1 < t1) ok = issue_s(gt + 1);
        ok = ok && wait(&bars.v_full[gt & 1], gt >> 1) && wait(&bars.p_full[gt & 1], gt >> 1);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          const uint32_t v = smem_addr(sm + L::V + (gt & 1) * L::SLABS * L::SLAB);
#pragma unroll
          for (int e = 0; e < kKeys / 16; ++e)
            mma_ts(tmem_o, tmem + (gt & 1) * 128 + e * 8, sdesc(v + e * 2048, L::SLAB, 1024), id_o, t > t0 || e > 0);
          mma_commit(smem_addr(&bars.v_empty[gt & 1]));
          mma_commit(smem_addr(&bars.o_done));
        }
        __syncwarp();
      }
    });
    }
  }
  // Copies and products on their way land before the CTA leaves (bounded).
  if (!ok) {
    failed = 1;
    if (lane == 0) atomicOr(p.c.status, pi::kKvTimeout);
    if (warp == 8) {
      if (ck_tile >= 0) bar_wait(smem_addr(&bars.ck_full), ck_tile & 1);
      if (cv_tile >= 0) bar_wait(smem_addr(&bars.cv_full), cv_tile & 1);
    }
    if (warp == 9) {                                   // a commit follows every product before it
      if (elect_one()) mma_commit(smem_addr(&bars.drain));
      __syncwarp();
      bar_wait(smem_addr(&bars.drain), 0);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
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
  p.grid = pi::current_sms();
  k_attn_tc<DT, D><<<p.grid, kThreads, smem, s>>>(p, maps);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return pi::launch_pdl(k_attn_combine<DT, D, kRows, kKeys>, dim3((unsigned)p.tok.n_seqs * p.c.heads, 4), dim3(128), 0, s, p);
}

}  // namespace

namespace attn {

cudaError_t run_tc(const AttnParams &p, int dtype, cudaStream_t s) {
  if (p.c.head_dim == 64) return dtype == PI_DT_F16 ? launch<PI_DT_F16, 64>(p, s) : launch<PI_DT_BF16, 64>(p, s);
  return dtype == PI_DT_F16 ? launch<PI_DT_F16, 128>(p, s) : launch<PI_DT_BF16, 128>(p, s);
}

}  // namespace attn
