// Attention for trees of drafted tokens over the 8-bit cache with many query rows of a
// key/value head (nodes x query heads of it), on tcgen05.
//
// The mathematics, operands and scales are those of pi_attn_tc.cu: S = Q K^T in TMEM,
// P = 2^(S f - b) fp16 over S, O += P V; a unit is up to 256 query rows of a (sequence,
// head).  A row sees the cache before the new tokens and the nodes whose bits its row
// has; only keys from the first new token on look at the bits.
//
// What differs: trees are small, so most units have one row tile and nothing to hide its
// chain S -> softmax -> P V behind.  There both softmax groups have it and take tiles of
// keys in turn, each with its own S, O and running maximum; the two sums are put together
// at the unit's end (each group a share of the dims).  The second half of Q's place holds
// a second tile of values meanwhile, so that the converters do not wait for a product.
// Masks and scores past kHuge are rare: a pass of its own rewrites such an S in TMEM, and
// the main passes know nothing of them.
//
// Roles (16 warps, one CTA an SM): 0-3 and 4-7 softmax, a row a thread; 8-11 converters,
// a token a thread; 12 and 14 copies of keys, with all scales, and of values; 13 issues the
// products (of both groups: the order keeps their softmaxes apart, whose exponentials would
// meet otherwise: two row tiles 171 us, 202 with a warp for each group).
//
// Measured: 16 sequences of 20 to 8191 tokens, trees of 13 to 26, 64 bf16 heads of 128 on 8: 109 us
// (445 TFLOP/s; causal attention of as many rows 136); the same, all of 8191 tokens, trees of up to 16: 111 us
// (134); 60011 tokens under a tree of 64, 128 fp16 heads of 64 on 8: 201 us (625 TFLOP/s).  A row tile's chain
// bounds it, of 3700 clocks a tile of keys at 64 dims, 4900 at 128: 2500 in the softmax, the rest the issue of
// its 16 products and their latency; the tensor pipe is busy for a third, the exponentials' for a fifth.
// Of 128 dims 164 to 206 bytes a thread are spilled, of 64 and 96 dims 16.
// Tried and slower: half tiles of keys as items with S of 64 columns (two row tiles 207 us), weights
// relative to the last maximum in one pass (225), a warp for each group's products (202); 64 dims with P beside
// S in TMEM and the next S issued before P V (213).
#include "pi_attn_tc.cuh"

using namespace attn;

namespace {

constexpr float kHuge = 0x1p22f;
// A tree's tokens lie in three tiles at most, whose NaN are looked at when the unit ends.
// Copies run at most seven tiles ahead of what either group still reads.
static_assert(PI_MAX_TREE <= 2 * kKeys);
constexpr int kRing = 16;
// A unit's beginning and end in tiles of keys: queries in, results or parts out, the first S and the last P V, all
// of it by code that is not in the instruction cache (16 sequences of 20 to 8191 tokens, 64 heads of 128 on 8: trees of
// 8 to 16 140 us without, 106 with 2, 90 with 4, 80 with 6; trees of 13 to 26 154 without, 109).
constexpr int kExtra = 6;
// Columns of S that a pass has at a time.  Short loops where the other roles' are long: four
// roles share the instruction cache (16 sequences of 8191 tokens, one row tile, 128 dims:
// 117 us with 64 columns, 111 with 32; 64 dims, two row tiles: 201 and 219).
constexpr int cols_of(int D) { return D <= 64 ? 64 : 32; }

struct Bars {
  unsigned long long c_full[kStages], c_empty[kStages];                // codes: copied, widened
  unsigned long long k_full[2], k_empty[2], v_full[2], v_empty[2];     // fp16 tiles: written, used
  unsigned long long s_full[2], p_full[2], o_done[2];                  // of a group: S ready, P ready, O of a tile done
  unsigned long long q_full[2];                                        // Q of a row tile written
  unsigned long long pair[2], merged[2];                               // of a group: its sums are there, and put together
  unsigned long long drain;                                            // after a failure
};

__device__ __forceinline__ void tmem_ld16(uint32_t addr, float *v) {
  uint32_t r[16];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
               "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}

template <int N>
__device__ __forceinline__ void load_cols(uint32_t addr, float *x) {
#pragma unroll
  for (int c = 0; c < N; c += 32) tmem_ld32(addr + c, x + c);
  tmem_wait_ld<N>(x);
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Which of the dims d .. d + 31 are NaN in a value at positions k0 .. k1 - 1 that a row of a tree sees.
template <int D>
__device__ __noinline__ unsigned nan_of_seen(const AttnParams &p, int s, int h, int k0, int k1, int first, const int32_t *tree, int d) {
  unsigned is = 0;
  for (int k = k0; k < k1; ++k) {
    const int j = k - first;
    if (j >= 0 && !(tree[j >> 5] >> (j & 31) & 1)) continue;           // j is at most the row's own place: inside its words
    const int page = p.tok.page_table[(int64_t)s * p.tok.table_stride + k / p.c.page_size];
    if (page < 0 || page >= p.c.n_pages) continue;
    const uint8_t *c = p.c.v_codes + (((int64_t)page * p.c.heads + h) * p.c.page_size + k % p.c.page_size) * D + d;
    for (int e = 0; e < 32; ++e) is |= ((c[e] & 0x7f) == 0x7f ? 1u : 0u) << e;
  }
  return is;
}

// ---- what few tiles need, out of the loops' way ----

// Columns of S that a row does not see, -inf: absent blocks (a bad page, past the sequence), columns from `cols` on,
// and of the new tokens (column 0 is new token j0) those whose bits `tree` has not.
__device__ __noinline__ void mask_columns(uint32_t ts, const float *ks, int cols, const int32_t *tree, int words, int j0) {
#pragma unroll 1
  for (int b = 0; b < kBlocks; ++b) {
    float x[16];
    tmem_ld16(ts + b * 16, x);
    tmem_wait_ld<16>(x);
    const int n = ks[b] < 0.f ? 0 : cols - 16 * b;
    const unsigned m = (n <= 0 ? 0u : n >= 16 ? 0xffffu : (1u << n) - 1) & tree_sees(tree, words, j0 + 16 * b);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (!(m >> j & 1)) x[j] = -INFINITY;
    tmem_st16(ts + b * 16, reinterpret_cast<const uint32_t *>(x));
  }
  tmem_wait_st();
}
// O times c.
template <int D>
__device__ __noinline__ void scale_columns(uint32_t to, float c) {
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
// A tile of a warp that has scores past kHuge, or blocks whose value scale is far below another's (kFar): everything
// from the rows' largest exponents `top` on.  ks: K scales, V scales 8 further.  Returns R and the sum.
//
// Scores so large that their last place counts: a fused difference from R would be off by as much, and 2^z not
// finite.  Rounded as the largest is, its own difference is exact.
template <int D>
__device__ __noinline__ float2 rare_tile(uint32_t ts, uint32_t to, const float *ks, float f, float2 rs, float top, int largest, bool begun) {
  float R = rs.x, sum = rs.y;
  const float *vs = ks + kBlocks;
  auto factor = [&](int b) { return fmaxf(f * fabsf(ks[b]), 1e-37f); };
  auto exponent = [&](int b) { return (float)((int)(__float_as_uint(vs[b]) >> 23 & 255) - 127); };
  auto two_steps = [&](float x, int b) { return __fadd_rn(__fmul_rn(x, factor(b)), exponent(b)); };
  const float most = fmaxf(fabsf(top), R == -INFINITY ? 0.f : fabsf(R));
  const bool mine = most > kHuge && most < INFINITY;
  float rough = -INFINITY;
#pragma unroll 1
  for (int b = 0; b < kBlocks; ++b) {
    float x[16];
    tmem_ld16(ts + b * 16, x);
    tmem_wait_ld<16>(x);
#pragma unroll
    for (int j = 0; j < 16; ++j) rough = fmaxf(rough, two_steps(x[j], b));
  }
  if (mine) top = rough;
  const bool over = top - kBoost > R + kSlack;
  if (__any_sync(0xffffffffu, over)) {
    const float Rn = over ? fmaxf(R, top - kBoost) : R, by = R == Rn ? 0.f : R - Rn;
    R = Rn;
    sum = add_scaled(0.f, sum, by);
    if (begun) scale_columns<D>(to, ex2(by));
  }
  const float Rs = R == -INFINITY ? 0.f : R;
#pragma unroll 1
  for (int b = 0; b < kBlocks; ++b) {
    const float fb = factor(b), ev = exponent(b), bias = ev - Rs;
    float x[16];
    tmem_ld16(ts + b * 16, x);
    tmem_wait_ld<16>(x);
    if (ev < (float)(largest - 127 - kFar)) {
      float part = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float z = fmaf(x[j], fb, bias);            // as below, where 2^z is 0 from -126 down
        part += z < -126.f ? ex2(z + 100.f) : 0.f;
      }
      sum = fmaf(part, ex2(-ev - 100.f), sum);
    }
    uint32_t w[8];
    f2 part = f2_of(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f2 z = f2_fma(f2_of(x[2 * j], x[2 * j + 1]), f2_of(fb, fb), f2_of(bias, bias));
      if (mine) z = f2_of(two_steps(x[2 * j], b) - Rs, two_steps(x[2 * j + 1], b) - Rs);
      const f2 y = f2_of(ex2(z.x), ex2(z.y));
      part = f2_add(part, y);
      w[j] = f2_narrow<PI_DT_F16>(y);
    }
    sum = fmaf(f2_sum(part), ex2(-ev), sum);
    tmem_st8(ts + b * 8, w);                             // columns that have been read
  }
  tmem_wait_st();
  return make_float2(R, sum);
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 1) k_attn_tree(const AttnParams p, const __grid_constant__ AttnMaps maps) {
  using E = Elem<DT>;
  using L = Smem<D>;
  constexpr int COLS = cols_of(D);
  extern __shared__ char smem_raw[];
  char *sm = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ Bars bars;
  __shared__ ShareShared share_sm;
  __shared__ float scales[kRing][2][kBlocks];          // K and V scales of a tile's blocks; below 0: no block
  __shared__ int nan_any[kRing], tile_bad[kRing];      // a tile's values have NaN that not all rows see; a block is absent
  __shared__ float2 sums[2][kHalf];                    // one row tile: R and the sum of each group's rows
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
      bar_init(smem_addr(&bars.pair[i]), 4);
      bar_init(smem_addr(&bars.merged[i]), 4);
      bar_init(smem_addr(&bars.v_full[i]), 4);
      bar_init(smem_addr(&bars.v_empty[i]), 1);
    }
    bar_init(smem_addr(&bars.drain), 1);
    bar_init_fence();
    failed = 0;
  }
  Share at;
  const bool any = find_share<kRows, kKeys, kExtra>(p, share_sm, blockIdx.x, &at);
  if (tid == 0) write_plan<kRows, kKeys, kExtra>(p, any, at);
  if (!any) return;
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_s)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_s;                        // S of the two groups, then O of the two

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
    uint32_t n[2], v[2];     // tiles of each group, and in each place for values, before
    uint32_t index1;         // of the units before, the ones with two row tiles
    int s, h, row0, keys, tiles, t0, t1;
    bool two;                // the unit has a second row tile
    int least;               // keys that every row sees: below, no row masks anything
    Seq sq;
    // group g's tiles: every one, or those in turn
    __device__ __forceinline__ int count(int g) const { return two ? t1 - t0 : (t1 - t0 + 1 - g) >> 1; }
    __device__ __forceinline__ int tile(int g, int a) const { return two ? a : 2 * a + g; }        // from t0 on
  };
  bool ok = true;
  int copied = -1;                                     // the last stage use whose copies were issued (warps 12 and 14)
  auto units = [&](auto work) {
    Unit u;
    u.g = u.index = u.index1 = u.n[0] = u.n[1] = u.v[0] = u.v[1] = 0;
    for (int64_t pos = at.begin; pos < at.end; ++u.index) {
      u.sq = at.sq;
      u.s = at.s, u.h = at.h, u.row0 = at.rt * kRows;
      u.keys = unit_keys<kRows>(p, u.sq, at.rt), u.tiles = (u.keys + kKeys - 1) / kKeys;
      u.t0 = (int)max((int64_t)0, pos - at.u0 - kExtra), u.t1 = (int)min((int64_t)u.tiles, at.end - at.u0 - kExtra);
      if (u.t1 <= u.t0) break;                           // what is left of the share is this unit's extra
      u.least = max(0, min(u.sq.len, u.sq.first));
      u.two = u.row0 + kHalf < u.sq.rows;
      work(u);
      if (!ok) break;
      u.g += u.t1 - u.t0;
      u.n[0] += u.count(0), u.n[1] += u.count(1);
      u.v[0] += u.count(0), u.v[1] += u.two ? 0 : u.count(1);
      if (u.two) ++u.index1;
      pos = at.u0 + kExtra + u.t1;
      if (pos < at.end && !next_unit<kRows, kKeys, kExtra>(p, &at)) break;
    }
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int grp = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, ts = tmem + lanes + grp * 128, to = tmem + lanes + 256;
    units([&](const Unit &u) {
      // ================= softmax: row u.row0 + 128 rt + row =================
      const Seq &sq = u.sq;
      const int h = u.h, rt = u.two ? grp : 0;
      const int r = u.row0 + kHalf * rt + row;
      const bool in = r < sq.rows;
      const int i = in ? r / p.group : 0, hq = h * p.group + (in ? r % p.group : 0);
      const int lim = in ? max(0, min(sq.len, sq.first + i + 1)) : sq.len;
      const int min_lim = min(__reduce_min_sync(0xffffffffu, lim), max(0, sq.first));
      const int32_t *tree = in ? p.tree + (int64_t)(sq.row0 + i) * p.words : nullptr;      // the row's bits
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
        if (u.two || grp == 0) {                         // one row tile: the second group has only looked for its factors
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
      }
      float R = -INFINITY, sum = 0.f;
      int largest = 0;                                   // exponent of the V scales so far (biased)
      const uint32_t before = grp ? u.n[1] : u.n[0];
      const int count = u.count(grp);
#pragma unroll 1
      for (int a = 0; a < count; ++a) {
        const int t = u.t0 + u.tile(grp, a), k0 = t * kKeys;
        const uint32_t n = before + a, ring = (u.g + (t - u.t0)) % kRing;
        if (!wait(&bars.s_full[grp], n)) {
          ok = false;
          return;
        }
        fence_after();
        const float *ks = scales[ring][0], *vs = scales[ring][1];
        const int own = (int)(__float_as_uint(vs[lane & 7]) >> 23 & 255);
        largest = max(largest, __reduce_max_sync(0xffffffffu, own));
        const bool far = __any_sync(0xffffffffu, own < largest - kFar);      // rare
        // not negative, and not 0, so that a masked column stays -inf
        auto factor = [&](int b) { return fmaxf(f * fabsf(ks[b]), 1e-37f); };
        auto exponent = [&](int b) { return (float)((int)(__float_as_uint(vs[b]) >> 23 & 255) - 127); };
        if (k0 + kKeys > min_lim || tile_bad[ring]) mask_columns(ts, ks, lim - k0, tree, p.words, k0 - sq.first);
        float top = -INFINITY;                           // of x + ev
#pragma unroll 1
        for (int b = 0; b < kBlocks; b += COLS / 16) {
          float x[COLS];
          load_cols<COLS>(ts + b * 16, x);
#pragma unroll
          for (int e = 0; e < COLS / 16; ++e) {
            float m = x[16 * e];
#pragma unroll
            for (int j = 1; j < 16; ++j) m = fmaxf(m, x[16 * e + j]);
            top = fmaxf(top, fmaf(m, factor(b + e), exponent(b + e)));
          }
        }
        const float most = fmaxf(fabsf(top), R == -INFINITY ? 0.f : fabsf(R));
        const bool mine = most > kHuge && most < INFINITY;
        const bool over = top - kBoost > R + kSlack;
        if (__any_sync(0xffffffffu, over || mine || far)) {
          if (a > 0) {                                   // O is the products' until the group's tile before is done
            if (!wait(&bars.o_done[grp], n - 1)) {
              ok = false;
              return;
            }
            fence_after();
          }
          if (__any_sync(0xffffffffu, mine || far)) {    // all of it out of line
            const float2 rs = rare_tile<D>(ts, to + grp * 128, ks, f, make_float2(R, sum), top, largest, a > 0);
            R = rs.x, sum = rs.y;
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&bars.p_full[grp]));
            continue;
          }
          const float Rn = over ? fmaxf(R, top - kBoost) : R, by = R == Rn ? 0.f : R - Rn;
          R = Rn;
          sum = add_scaled(0.f, sum, by);
          if (a > 0) scale_columns<D>(to + grp * 128, ex2(by));
        }
        const float Rs = R == -INFINITY ? 0.f : R;
        // P takes the first 64 columns of S: what it overwrites has been read
#pragma unroll 1
        for (int b = 0; b < kBlocks; b += COLS / 16) {
          float x[COLS];
          load_cols<COLS>(ts + b * 16, x);
          uint32_t w[COLS / 2];
#pragma unroll
          for (int e = 0; e < COLS / 16; ++e) {
            const float fb = factor(b + e), ev = exponent(b + e), bias = ev - Rs;
            f2 part = f2_of(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const f2 z = f2_fma(f2_of(x[16 * e + 2 * j], x[16 * e + 2 * j + 1]), f2_of(fb, fb), f2_of(bias, bias));
              const f2 y = f2_of(ex2(z.x), ex2(z.y));
              part = f2_add(part, y);
              w[e * 8 + j] = f2_narrow<PI_DT_F16>(y);
            }
            sum = fmaf(f2_sum(part), ex2(-ev), sum);
          }
          if constexpr (COLS == 64) tmem_st32(ts + b * 8, w);
          else tmem_st16(ts + b * 8, w);
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars.p_full[grp]));
      }
      // ---- the unit's result, or this CTA's part of it ----
      const uint32_t one = u.index - u.index1;           // units of one row tile before
      if (count && !wait(&bars.o_done[grp], before + count - 1)) {
        ok = false;
        return;
      }
      const int other_n = u.count(grp ^ 1);
      float mine = 1.f, theirs = 0.f;                    // factors of this group's O and of the other's
      if (!u.two) {
        sums[grp][row] = make_float2(R, sum);
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars.pair[grp]));
        if (!wait(&bars.pair[grp ^ 1], one) || (other_n && !wait(&bars.o_done[grp ^ 1], (grp ? u.n[0] : u.n[1]) + other_n - 1))) {
          ok = false;
          return;
        }
        const float2 other = sums[grp ^ 1][row];
        const float Rn = fmaxf(R, other.x), by = R - Rn, to_it = other.x - Rn;
        mine = R == -INFINITY ? 0.f : ex2(by), theirs = other.x == -INFINITY ? 0.f : ex2(to_it);
        // without a maximum a group's sum is 0, or NaN of NaN scores, which counts
        const float a = R == -INFINITY ? sum : add_scaled(0.f, sum, by), b = other.x == -INFINITY ? other.y : add_scaled(0.f, other.y, to_it);
        sum = grp ? b + a : a + b, R = Rn;
      }
      fence_after();
      const bool whole = u.t0 == 0 && u.t1 == u.tiles;
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
      const int64_t orow = (int64_t)(sq.row0 + i) * p.q_heads + hq;
      float *part = p.part + (int64_t)(2 * blockIdx.x + (u.t0 == 0)) * kRows * (D + 2);
      const int pr = kHalf * rt + row;
      bool nan = false;                                  // some tile has NaN that some rows do not see
      for (int t = max(u.t0, u.least / kKeys); t < u.t1; ++t) nan |= nan_any[(u.g + (t - u.t0)) % kRing] != 0;
#pragma unroll 1
      for (int q = u.two ? 0 : grp; q < D / 32; q += u.two ? 1 : 2) {
        float o[32];
        tmem_ld32(to + grp * 128 + q * 32, o);
        if (!u.two) {
          float o2[32];
          tmem_ld32(to + (grp ^ 1) * 128 + q * 32, o2);
          tmem_wait_ld<32>(o);
          tmem_wait_ld<32>(o2);
          // a group without tiles, or whose rows saw nothing, has no O: whatever is there does not count
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float m = count ? o[j] * mine : 0.f, w = other_n ? o2[j] * theirs : 0.f;
            o[j] = grp ? w + m : m + w;
          }
        } else {
          tmem_wait_ld<32>(o);
        }
        if (nan) {
          for (int t = max(u.t0, u.least / kKeys); t < u.t1; ++t) {
            if (!nan_any[(u.g + (t - u.t0)) % kRing]) continue;
            // which of the tokens it is says the cache itself (rare)
            const unsigned is = in ? nan_of_seen<D>(p, u.s, h, t * kKeys, min(lim, (t + 1) * kKeys), sq.first, tree, q * 32) : 0;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (is >> j & 1) o[j] = __uint_as_float(0x7fffffffu);
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
        if (u.two || grp == 0) part[kRows * D + 2 * pr] = R, part[kRows * D + 2 * pr + 1] = sum;
      } else if (in && p.lse && (u.two || grp == 0)) {
        p.lse[orow] = sum == 0.f ? -INFINITY : ((R == -INFINITY ? 0.f : R) + log2f(sum)) * kLn2;
      }
      if (!u.two) {                                      // neither goes on while the other reads its O and sums
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars.merged[grp]));
        if (!wait(&bars.merged[grp ^ 1], one)) ok = false;
      }
    });
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    const int r = tid - 256;
    units([&](const Unit &u) {
      // ================= converters: token r of each tile =================
      const Seq &sq = u.sq;
      for (int t = u.t0; t < u.t1; ++t) {
        const uint32_t gt = u.g + (t - u.t0), b = gt & 1, ring = gt % kRing;
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
          // 0 * NaN: it is taken out, and noted.
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
              c[j].x &= ~__vcmpeq4(c[j].x & 0x7f7f7f7fu, 0x7f7f7f7fu), c[j].y &= ~__vcmpeq4(c[j].y & 0x7f7f7f7fu, 0x7f7f7f7fu);
              c[j].z &= ~__vcmpeq4(c[j].z & 0x7f7f7f7fu, 0x7f7f7f7fu), c[j].w &= ~__vcmpeq4(c[j].w & 0x7f7f7f7fu, 0x7f7f7f7fu);
            }
          }
          __syncwarp();
        }
        const int place = u.two ? 0 : (t - u.t0) & 1;    // one row tile: the second half of Q's place in turn
        const uint32_t use = (place ? u.v[1] : u.v[0]) + (u.two ? t - u.t0 : (t - u.t0) >> 1);
        if (use >= 1 && !wait(&bars.v_empty[place], use - 1)) {
          ok = false;
          return;
        }
        store(sm + (place ? L::Q + L::TILE : L::V));
        if (lane == 0) bar_arrive(smem_addr(&bars.v_full[place]));
      }
    });
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 12 || warp == 14) {
      const bool values = warp == 14;
      units([&](const Unit &u) {
        // ================= tile copies; lane l looks after block l % 8 =================
        const int32_t *table = p.tok.page_table + (int64_t)u.s * p.tok.table_stride;
        const int P = p.c.page_size, blocks = P / PI_KV_BLOCK, limit = min(u.keys, u.t1 * kKeys);
        const int step = P % 64 ? 1 : 4;                 // boxes of 64 tokens where pages hold whole ones, else of 16
        auto page_of = [&](int t) {
          const int k = t * kKeys + (lane & 7) * 16;
          return k < limit ? table[k / P] : -1;
        };
        int next = page_of(u.t0);                        // looked up a tile ahead
        for (int t = u.t0; t < u.t1; ++t) {
          const uint32_t gt = u.g + (t - u.t0), ring = gt % kRing;
          const int k = t * kKeys + (lane & 7) * 16, co = k % P, page = next;
          const bool has = k < limit;
          next = page_of(t + 1);
          const bool good = page >= 0 && page < p.c.n_pages;
          if (has && !good && lane < 8) atomicOr(p.c.status, pi::kKvBadPage);
          const unsigned mask = __ballot_sync(0xffffffffu, good) & 255u;
          int n_boxes = 0;
          for (int b = 0; b < kBlocks; b += step) n_boxes += mask >> b & 1;
          const uint32_t use = 2 * gt + values, st = use % kStages, bar = smem_addr(&bars.c_full[st]);
          if (use >= kStages && !wait(&bars.c_empty[st], use / kStages - 1)) {
            ok = false;
            return;
          }
          if (!values) {
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
            if (lane == 0) nan_any[ring] = 0;
          }
          __syncwarp();
          if (elect_one()) bar_expect(bar, (uint32_t)n_boxes * step * 16 * D);
          __syncwarp();
#pragma unroll 1
          for (int b = 0; b < kBlocks; b += step) {
            const int z = __shfl_sync(0xffffffffu, page, b) * p.c.heads + u.h, y = __shfl_sync(0xffffffffu, co, b);
            if ((mask >> b & 1) && elect_one()) tile_copy(smem_addr(sm + L::C + st * 128 * D + b * 16 * D), values ? &maps.v : &maps.k, 0, y, z, bar);
            __syncwarp();
          }
          if (!values && lane < 16 && good) bar_arrive_copies(bar); else bar_arrive(bar);
          copied = (int)use;
        }
      });
    } else if (warp == 13) {
      const uint32_t id_s = idesc(kKeys, false), id_o = idesc(D, true);
      const uint32_t q_lo = desc_lo(smem_addr(sm + L::Q), 16), k_lo = desc_lo(smem_addr(sm + L::K), 16);
      const uint32_t v_lo = desc_lo(smem_addr(sm + L::V), L::SLAB), v2_lo = desc_lo(smem_addr(sm + L::Q + L::TILE), L::SLAB);
      units([&](const Unit &u) {
        // ================= products =================
        auto issue_s = [&](int grp, int a) {             // S of a group's a-th tile
          const uint32_t gt = u.g + u.tile(grp, a);
          if (!wait(&bars.k_full[gt & 1], gt >> 1)) return false;
          fence_after();
          if (elect_one()) {
            const uint32_t q = q_lo + (u.two ? grp : 0) * (L::TILE >> 4), k = k_lo + (gt & 1) * (L::TILE >> 4);
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
              const uint32_t o = (e / 4 * L::SLAB + e % 4 * 32) >> 4;
              mma_ss(tmem + grp * 128, q + o, k + o, id_s, e > 0);
            }
            if (!u.two || grp) mma_commit(smem_addr(&bars.k_empty[gt & 1]));       // its last use
            mma_commit(smem_addr(&bars.s_full[grp]));
          }
          __syncwarp();
          return true;
        };
        auto issue_o = [&](int grp, int a) {             // its P V
          const int place = u.two ? 0 : grp;
          if (!wait(&bars.v_full[place], (place ? u.v[1] : u.v[0]) + a) || !wait(&bars.p_full[grp], (grp ? u.n[1] : u.n[0]) + a)) return false;
          fence_after();
          if (elect_one()) {
            const uint32_t v = place ? v2_lo : v_lo;
#pragma unroll
            for (int e = 0; e < kKeys / 16; ++e)
              mma_ts(tmem + 256 + grp * 128, tmem + grp * 128 + e * 8, v + e * (2048 >> 4), id_o, a > 0 || e > 0);
            if (!u.two || grp) mma_commit(smem_addr(&bars.v_empty[place]));
            mma_commit(smem_addr(&bars.o_done[grp]));
          }
          __syncwarp();
          return true;
        };
        ok = wait(&bars.q_full[0], u.index) && (!u.two || wait(&bars.q_full[1], u.index1));
        for (int grp = 0; ok && grp < 2; ++grp) ok = !u.count(grp) || issue_s(grp, 0);
        for (int a = 0; ok && a < u.count(0); ++a)       // the second group has as many, or one less
          for (int grp = 0; ok && grp < 2; ++grp)
            if (a < u.count(grp)) ok = issue_o(grp, a) && (a + 1 >= u.count(grp) || issue_s(grp, a + 1));
      });
    }
  }
  // Copies and products on their way land before the CTA leaves (bounded).
  if (!ok) {
    failed = 1;
    if (lane == 0) atomicOr(p.c.status, pi::kKvTimeout);
    if (warp == 12 || warp == 14)                        // stages fill in order: of the last kStages uses every other one is this warp's
      for (int use = copied; use >= 0 && use > copied - kStages; use -= 2) bar_wait(smem_addr(&bars.c_full[use % kStages]), use / kStages & 1);
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
  cudaError_t e = pi::allow_smem(k_attn_tree<DT, D>, smem, smem, done);
  if (e != cudaSuccess) return e;
  p.row_tiles = (int)(((int64_t)p.max_q * p.group + kRows - 1) / kRows);
  p.grid = std::min(kMostShares, std::max(1, pi::current_sms()));
  k_attn_tree<DT, D><<<p.grid, kThreads, smem, s>>>(p, maps);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return pi::launch_pdl(k_attn_combine<DT, D, kRows, kKeys>, dim3(combine_grid(p, D, kRows)), dim3(kCombineThreads), 0, s, p);
}

}  // namespace

namespace attn {

cudaError_t run_tree(const AttnParams &p, int dtype, cudaStream_t s) {
  if (p.c.head_dim == 64) return dtype == PI_DT_F16 ? launch<PI_DT_F16, 64>(p, s) : launch<PI_DT_BF16, 64>(p, s);
  if (p.c.head_dim == 96) return dtype == PI_DT_F16 ? launch<PI_DT_F16, 96>(p, s) : launch<PI_DT_BF16, 96>(p, s);
  return dtype == PI_DT_F16 ? launch<PI_DT_F16, 128>(p, s) : launch<PI_DT_BF16, 128>(p, s);
}

}  // namespace attn
