// Attention of a sequence's newest tokens over its 8-bit key/value cache.
//
//   x_j = log2(e) sm_scale q.k_j,  p_j = 2^(x_j - m),  out = sum p_j v_j / sum p_j
//
// in one pass over the cache with a running maximum m.  For a single token the
// work is bound by HBM: each code is used by q_heads / heads rows only.
//
// Rows and products.  The query rows of one key/value head (n_s tokens x
// q_heads / heads) are columns of mma.sync m16n8k16 (fp16 operands, binary32
// sums); E4M3 codes are exact in fp16, so q.k has no rounding but that of the
// sums.  bf16 rows are scaled by a power of two per row to fit fp16.  The order of
// the head_dim in a product and of the rows of V^T is free as long as both
// operands agree, so a lane's operands are contiguous bytes of a token's row: it
// reads them from the tile that a tensor-map copy left in a shared-memory ring,
// several tiles ahead, without transposition.
//
// Scales.  A 16-token step of a warp is one block of the cache: its K scale is
// one factor of x, its V scale 2^ev is folded into the weights: acc holds
// sum 2^(x_j + ev_j - R) c_j with R + kBoost the running maximum of x_j + ev_j, so
// neither very large nor very small scales leave fp16's range, while
// l = sum 2^(x_j - m) runs on m.  out = acc 2^(R - m) / l.
//
// Split.  The tiles (64 keys of one unit = sequence, head, row tile) of all
// units form one line that is cut evenly over the CTAs, so a batch of very
// different lengths keeps every SM busy to the end.  A unit cut between CTAs
// leaves partial sums, which k_attn_combine adds in CTA order.
//
// Measured: 64 sequences of up to 8191 tokens, 64 bf16 heads of 128 on 8: 113 us (4.9
// TB/s, 73% of the copy rate; 100 us of it are left without any arithmetic: launch,
// units' beginnings and ends); 128 fp16 heads of 64 on 8 over 130001 tokens: 48 us (41%;
// 380 instructions for 16 tokens x 16 rows, issue slots half full; the variant of 16 rows
// of 64 dims spills 48 bytes at four CTAs an SM, that of 8 rows of 128 dims 36); 16 heads of 64 over
// 513 tokens: 11 us, the latency of two launches and one pass.
#include "pi_attn.cuh"

using namespace attn;

namespace {

constexpr int kTile = 64;                 // keys of a tile

__device__ __forceinline__ void mma16816(float *c, const unsigned *a, unsigned b0, unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A tile (64 tokens) in shared memory, K then V, as the tile copies leave it:
// boxes of min(D, 128) bytes by 64 rows, 16-byte chunks swizzled so that the
// loads below meet no bank twice (D = 96 is not swizzled; D = 64 meets two).
// Of a block (16 rows) lane (g = lane / 4, q = lane % 4) takes of K rows g and
// 8 + g its share of the k-steps, of V rows 2 q, 2 q + 1, 8 + 2 q, 9 + 2 q its dims.
template <int D>
struct Frag {
  static constexpr int BOX = D < 128 ? D : 128, BOXES = D / BOX;
  static constexpr int BOX_BYTES = kTile * BOX, V_AT = kTile * D, BYTES = 2 * V_AT;
  // dims of k-step k (two k indices, and the two 8 further): 4 from here on
  static __device__ __forceinline__ int kdim(int k, int q) {
    if constexpr (D == 96) return k >= 4 ? 64 + q * 8 + (k - 4) * 4 : q * 16 + k * 4;
    return k / (BOX / 16) * BOX + q * (BOX / 4) + k % (BOX / 16) * 4;
  }
  // dim of column c of n-tile j; 4 tiles in a row are 4 dims in a row
  static __device__ __forceinline__ int vdim(int j, int c) {
    if constexpr (D >= 128) return j / 16 * 128 + c * 16 + j % 16;
    return j < 8 ? c * 8 + j : 64 + c * 4 + j - 8;
  }
  static __device__ __forceinline__ uint4 ld16(const char *p) { return *reinterpret_cast<const uint4 *>(p); }
  static __device__ __forceinline__ uint2 ld8(const char *p) { return *reinterpret_cast<const uint2 *>(p); }
  // words of row 8 j + g of the block at src: k-step k's codes are word k
  static __device__ __forceinline__ void load_k(unsigned *w, const char *src, int j, int g, int q) {
    if constexpr (D == 64) {
      *reinterpret_cast<uint4 *>(w) = ld16(src + (8 * j + g) * 64 + ((q ^ (g >> 1 & 3)) << 4));
    } else if constexpr (D == 96) {
      const char *row = src + (8 * j + g) * 96;
      *reinterpret_cast<uint4 *>(w) = ld16(row + q * 16);
      *reinterpret_cast<uint2 *>(w + 4) = ld8(row + 64 + q * 8);
    } else {
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        *reinterpret_cast<uint4 *>(w + 4 * i) = ld16(src + i / 2 * BOX_BYTES + (8 * j + g) * 128 + (((2 * q + i % 2) ^ g) << 4));
    }
  }
  // words of row 2 q + (r & 1) + 8 (r >> 1): byte j is dim vdim(j, g)
  static __device__ __forceinline__ void load_v(unsigned *w, const char *src, int r, int g, int q) {
    const int row = 2 * q + (r & 1), h = r >> 1;
    src += V_AT;
    if constexpr (D == 64) {
      *reinterpret_cast<uint2 *>(w) = ld8(src + (8 * h + row) * 64 + (((g >> 1) ^ q) << 4) + (g & 1) * 8);
    } else if constexpr (D == 96) {
      *reinterpret_cast<uint2 *>(w) = ld8(src + (8 * h + row) * 96 + g * 8);
      w[2] = *reinterpret_cast<const unsigned *>(src + (8 * h + row) * 96 + 64 + g * 4);
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i)
        *reinterpret_cast<uint4 *>(w + 4 * i) = ld16(src + i * BOX_BYTES + (8 * h + row) * 128 + ((g ^ row) << 4));
    }
  }
};

// CTAs of 128 threads that an SM holds, by the registers of the variant (96 for
// 8 rows of 64, 128 for 8 of 128, 255 for 16 of 128); the grid is one wave of them.
constexpr int attn_ctas(int D, int nb) { return nb == 1 ? (D == 64 ? 5 : D <= 128 ? 4 : 2) : D == 64 ? 4 : D == 96 ? 3 : 2; }
// Ring stages of a CTA (a stage: a tile's four blocks) in its share of 224 KB.
template <int D, int NB>
constexpr int attn_stages() {
  const int n = (224 / attn_ctas(D, NB) - 2) * 1024 / Frag<D>::BYTES;   // 2 KB: alignment, barriers
  return n < 8 ? n : 8;
}

// NB: eights of query rows of a warp.  The four warps are WARPS_M groups of rows
// by 4 / WARPS_M groups of a tile's blocks: a warp goes over WARPS_M of them.
//
// Both products have the codes as the 16-row operand and the query rows as the
// 8 columns: S^T = K Q^T and O^T = V^T P^T.  Eight rows (or fewer) then cost
// half the products and registers of a 16-row tile of queries; P^T comes from
// S^T's registers by one 8 x 8 transposition (movmatrix) of each half.
//
// TREE: the new tokens are nodes of trees, of which a row sees what its bits say.
// Only blocks from the first new token on look at them.
template <int DT, int D, int NB, int WARPS_M, bool TREE>
__global__ void __launch_bounds__(128, attn_ctas(D, NB)) k_attn(const AttnParams p, const __grid_constant__ AttnMaps maps) {
  using E = Elem<DT>;
  constexpr int WROWS = 8 * NB, ROWS = WROWS * WARPS_M, KW = 4 / WARPS_M, KS = D / 16, MT = D / 16, STAGES = attn_stages<D, NB>();
  using F = Frag<D>;
  extern __shared__ char smem_raw[];
  // stages; then, KW > 1, a unit's [KW][ROWS][D] sums, [KW][ROWS][3] (m, l, R)
  char *ring = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float *sm = reinterpret_cast<float *>(ring);
  __shared__ ShareShared share_sm;
  __shared__ __align__(8) unsigned long long full[STAGES], empty[STAGES];   // a tile's copies have landed; all warps have read it
  __shared__ float scales[STAGES][2][4];           // K and V scale of its blocks; K below 0: no block
  __shared__ int failed;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wm = warp % WARPS_M, wk = warp / WARPS_M, g = lane >> 2, q4 = lane & 3;
  griddep_launch();                                // every CTA of this grid is resident: the next one may take what is left
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      bar_init(smem_addr(&full[i]), 33);           // the bytes' arrival, and each lane's scale copies
      bar_init(smem_addr(&empty[i]), 4);
    }
    bar_init_fence();
    failed = 0;
  }
  for (int s = blockIdx.x * 128 + threadIdx.x; s < p.tok.n_seqs; s += gridDim.x * 128) flag_seq(p, s);

  Share at;
  const bool any = find_share<ROWS, kTile>(p, share_sm, blockIdx.x, &at);
  if (threadIdx.x == 0) write_plan<ROWS, kTile>(p, any, at);
  if (!any) return;
  bool dead = false;                               // a wait ran out: nothing more is copied or computed
  const bool by16 = p.c.page_size % kTile != 0;    // a tile may lie in several pages: blocks are copied one by one
  const int page_size = p.c.page_size, blocks = page_size / PI_KV_BLOCK;
  const int turn_pages = 4 * kTile / page_size, turn_rest = 4 * kTile - turn_pages * page_size;
  // Tile n of this CTA uses stage n % STAGES for the n / STAGES-th time and is
  // fetched by warp n % 4, STAGES - 1 tiles ahead: what a fetch needs is kept up
  // by that warp alone, once in four tiles.
  int done = 0, stage = 0, phase = 0;              // tiles read; the next one's stage and parity
  int last_fetch = -1;                             // the last tile this warp fetched
  for (int64_t pos = at.begin; pos < at.end;) {
    const Seq &sq = at.sq;
    const int s = at.s, h = at.h, rt = at.rt;
    const int keys = unit_keys<ROWS>(p, sq, rt), tiles = (keys + kTile - 1) / kTile;
    const int t0 = (int)(pos - at.u0), t1 = (int)min((int64_t)tiles, at.end - at.u0);

    // ---- fetches; lane l looks after block l % 4 of the tile ----
    const int32_t *table = p.tok.page_table + (int64_t)s * p.tok.table_stride;
    const float *sc_head = ((lane & 4) ? p.c.v_scales : p.c.k_scales) + (int64_t)h * blocks;
    const int copies = min(keys, t1 * kTile);
    int next = done + ((warp - done) & 3);           // the tile this warp fetches next, and of this lane's block:
    int ck = (t0 + next - done) * kTile + (lane & 3) * 16;       // the first key,
    int cp = ck / page_size, co = ck - cp * page_size;           // the page's place in the table and the offset in it
    int page = ck < copies ? table[cp] : -1;
    auto fetch = [&] {                               // tile `next`
      const int st = next % STAGES, use = next / STAGES;
      if (use > 0 && !dead && !bar_wait(smem_addr(&empty[st]), (use - 1) & 1)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      if (!dead) {
        const bool in = ck < copies, ok = in && page >= 0 && page < p.c.n_pages;
        if (in && !ok && lane < 4) atomicOr(p.c.status, pi::kKvBadPage);
        const uint32_t bar = smem_addr(&full[st]), dst = smem_addr(ring + st * F::BYTES);
        if (lane < 8) {
          float *sc = &scales[st][lane >> 2][lane & 3];
          if (ok)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(sc)),
                         "l"(sc_head + (int64_t)page * p.c.heads * blocks + co / PI_KV_BLOCK) : "memory");
          else
            *sc = -1.f;
        }
        const unsigned good = __ballot_sync(0xffffffffu, ok) & 15u;
        if (!by16) {
          const int z = __shfl_sync(0xffffffffu, page, 0) * p.c.heads + h, y = __shfl_sync(0xffffffffu, co, 0);
          if (elect_one()) {
            if (good & 1) {
              bar_expect(bar, F::BYTES);
#pragma unroll
              for (int i = 0; i < F::BOXES; ++i) {
                tile_copy(dst + i * F::BOX_BYTES, &maps.k, i * 128, y, z, bar);
                tile_copy(dst + F::V_AT + i * F::BOX_BYTES, &maps.v, i * 128, y, z, bar);
              }
            } else {
              bar_arrive(bar);
            }
          }
        } else {
          if (elect_one()) bar_expect(bar, __popc(good) * (F::BYTES / 4));
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            const int z = __shfl_sync(0xffffffffu, page, b) * p.c.heads + h, y = __shfl_sync(0xffffffffu, co, b);
            if ((good >> b & 1) && elect_one()) {
#pragma unroll
              for (int i = 0; i < F::BOXES; ++i) {
                tile_copy(dst + b * 16 * F::BOX + i * F::BOX_BYTES, &maps.k, i * 128, y, z, bar);
                tile_copy(dst + F::V_AT + b * 16 * F::BOX + i * F::BOX_BYTES, &maps.v, i * 128, y, z, bar);
              }
            }
            __syncwarp();
          }
        }
        __syncwarp();
        if (lane < 8 && ok) bar_arrive_copies(bar); else bar_arrive(bar);
        last_fetch = next;
      }
      next += 4, ck += 4 * kTile, cp += turn_pages, co += turn_rest;
      if (co >= page_size) co -= page_size, ++cp;
      page = ck < copies ? table[cp] : -1;
    };
    const int unit_end = done + (t1 - t0);
    while (next < min(unit_end, done + STAGES - 1)) fetch();

    // ---- the rows of this unit: Q^T in registers, row nb * 8 + g of the warp to this lane ----
    const int base_row = rt * ROWS + wm * WROWS;
    unsigned bq[NB][KS][2];
    int lim[NB][2];                                // of the lane's columns: rows nb * 8 + 2 q4 + e
    float fac[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = base_row + nb * 8 + g;
      const bool in = r < sq.rows;
      const int i = in ? r / p.group : 0, hq = h * p.group + (in ? r % p.group : 0);
      const typename E::T *src = static_cast<const typename E::T *>(p.q) + (int64_t)(sq.row0 + i) * p.qt + hq * p.qh;
      f2 x[KS][2];                                 // this lane's four dims of each k-step
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint2 w = make_uint2(0, 0);
        if (in) w = *reinterpret_cast<const uint2 *>(src + F::kdim(k, q4));
        x[k][0] = f2_widen<DT>(w.x), x[k][1] = f2_widen<DT>(w.y);
      }
      float up = 1.f, down = p.scale;
      if constexpr (DT == PI_DT_BF16) {
        // the row's largest finite magnitude to [2^13, 2^14): exact, and fp16 then loses only what is 2^-27 of it
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float2 f = f2_get(x[k][c]);
            mx = fmaxf(mx, fmaxf(fabsf(f.x) < INFINITY ? fabsf(f.x) : 0.f, fabsf(f.y) < INFINITY ? fabsf(f.y) : 0.f));
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = max((int)(__float_as_uint(mx) >> 23), 27) - 127 - 13;    // up = 2^-ex stays normal
        if (mx > 0.f) up = __uint_as_float((unsigned)(127 - ex) << 23), down = p.scale * __uint_as_float((unsigned)(127 + ex) << 23);
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        bq[nb][k][0] = f2_narrow<PI_DT_F16>(f2_mul(x[k][0], f2_of(up, up)));
        bq[nb][k][1] = f2_narrow<PI_DT_F16>(f2_mul(x[k][1], f2_of(up, up)));
      }
      // a padding row masks what every row masks
      const int sees = in && p.causal ? max(0, min(sq.len, sq.first + i + 1)) : sq.len;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        lim[nb][e] = __shfl_sync(0xffffffffu, sees, (2 * q4 + e) * 4);
        fac[nb][e] = __shfl_sync(0xffffffffu, down, (2 * q4 + e) * 4);
      }
    }
    int min_lim = lim[0][0];                       // below it no row of the warp masks anything
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) min_lim = min(min_lim, min(lim[nb][0], lim[nb][1]));
    min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 1));
    min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 2));
    const int32_t *tree[NB][2];                    // the columns' bits
    if constexpr (TREE) {
      min_lim = min(min_lim, max(0, sq.first));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = base_row + nb * 8 + 2 * q4 + e;
          tree[nb][e] = r < sq.rows ? p.tree + (int64_t)(sq.row0 + r / p.group) * p.words : nullptr;
        }
    }

    float acc[NB][MT][4], m[NB][2], l[NB][2], R[NB][2];      // m is 0 and R -inf while no key has been seen
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[nb][i][0] = acc[nb][i][1] = acc[nb][i][2] = acc[nb][i][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        m[nb][e] = l[nb][e] = 0.f, R[nb][e] = -INFINITY;
    }

    for (int t = t0; t < t1; ++t) {
      const int st = stage;
      if (!dead && !bar_wait(smem_addr(&full[st]), phase)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
      phase ^= stage == 0;
      const char *tile = ring + st * F::BYTES;
#pragma unroll 1
      for (int blk = wk * WARPS_M; blk < (wk + 1) * WARPS_M; ++blk) {
        const int k0 = t * kTile + blk * 16;
        const char *src = tile + blk * 16 * F::BOX;
        if (k0 >= keys || dead) break;
        const float ks = scales[st][0][blk], vs = scales[st][1][blk];
        if (ks < 0.f) continue;
        // ---- x = q.k: tokens g and 8 + g, rows 2 q4 and 2 q4 + 1 of each eight ----
        float x[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) x[nb][0] = x[nb][1] = x[nb][2] = x[nb][3] = 0.f;
        {
          unsigned w0[KS], w1[KS];
          F::load_k(w0, src, 0, g, q4);
          F::load_k(w1, src, 1, g, q4);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            unsigned a[4];
            widen4(w0[k], a[0], a[2]);
            widen4(w1[k], a[1], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816(x[nb], a, bq[nb][k][0], bq[nb][k][1]);
          }
        }
        // ---- running maximum, taken up only where a score passes it by kSlack ----
        const bool ragged = k0 + 16 > min_lim;
        unsigned sees[NB][2];                      // TREE: the block's tokens, bit by bit
        if constexpr (TREE) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) sees[nb][e] = ragged ? tree_sees(tree[nb][e], p.words, k0 - sq.first) : 0xffffu;
        }
        const float ev = (float)((int)(__float_as_uint(vs) >> 23) - 127);
        bool over = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float fk = fac[nb][e] * ks, most = fminf(kSlack, R[nb][e] - m[nb][e] + (kBoost + kSlack - ev));
#pragma unroll
            for (int j = e; j < 4; j += 2) {
              x[nb][j] = fmaf(x[nb][j], fk, -m[nb][e]);                // relative to m
              if (ragged && k0 + g + 8 * (j >> 1) >= lim[nb][e]) x[nb][j] = -INFINITY;
              if (TREE && !(sees[nb][e] >> (g + 8 * (j >> 1)) & 1)) x[nb][j] = -INFINITY;
              over |= x[nb][j] > most;
            }
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float bm = fmaxf(x[nb][e], x[nb][2 + e]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
              if (bm == -INFINITY) continue;           // every row of these keys is masked
              const bool none = R[nb][e] == -INFINITY;
              const float mn = none ? bm : m[nb][e] + fmaxf(bm, 0.f), Rn = fmaxf(R[nb][e], bm + m[nb][e] + ev - kBoost);
              const float by = m[nb][e] - mn, c = ex2(R[nb][e] - Rn);
              if (!none) l[nb][e] *= ex2(by);
              x[nb][e] += by, x[nb][2 + e] += by;
              m[nb][e] = mn, R[nb][e] = Rn;
#pragma unroll
              for (int i = 0; i < MT; ++i) acc[nb][i][e] *= c, acc[nb][i][2 + e] *= c;
            }
        }
        // ---- weights, transposed into the second product's operand ----
        unsigned pb[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // x <= 14 - shift, and shift <= 198 once a key has been seen (before that x is -inf and shift inf):
            // of its own exponent, since 2^x is 0 where a weight of 2^(x + shift) still counts
            const float shift = fminf(m[nb][e] - R[nb][e] + ev, 200.f);
            l[nb][e] += ex2(x[nb][e]) + ex2(x[nb][2 + e]);
            w[e] = ex2(x[nb][e] + shift), w[2 + e] = ex2(x[nb][2 + e] + shift);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
            asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pb[nb][j]) : "r"(pack_half2(w[2 * j], w[2 * j + 1])));
        }
        // ---- acc += v p ----
        unsigned v[4][D / 32];
#pragma unroll
        for (int r = 0; r < 4; ++r) F::load_v(v[r], src, r, g, q4);
        if (ragged) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (k0 + 2 * q4 + (r & 1) + 8 * (r >> 1) >= sq.len) {    // past the sequence: whatever the page held before
#pragma unroll
              for (int c = 0; c < D / 32; ++c) v[r][c] = 0;
            }
          // A NaN among tokens that only some rows see would reach the others as
          // 0 * NaN: it is taken out here and given to the rows that see it.
          bool nan = false;
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) nan |= __vcmpeq4(v[r][c] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
          if (__any_sync(0xffffffffu, nan)) {
            unsigned see[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
                             : "=r"(see[nb][j])
                             : "r"(pack_half2(k0 + 8 * j + g < lim[nb][0] && (!TREE || (sees[nb][0] >> (8 * j + g) & 1)),
                                              k0 + 8 * j + g < lim[nb][1] && (!TREE || (sees[nb][1] >> (8 * j + g) & 1)))));
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              unsigned n[4];
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const unsigned is = __vcmpeq4(v[r][c] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                n[r] = is & 0x38383838u;           // the code of 1
                v[r][c] &= ~is;
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                unsigned a[4];
                widen4(__byte_perm(n[0], n[1], i ? 0x7362 : 0x5140), a[0], a[1]);
                widen4(__byte_perm(n[2], n[3], i ? 0x7362 : 0x5140), a[2], a[3]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                  float cnt[4] = {0.f, 0.f, 0.f, 0.f};
                  mma16816(cnt, a, see[nb][0], see[nb][1]);
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    if (cnt[k] > 0.f) acc[nb][2 * c + i][k] = __uint_as_float(0x7fffffffu);
                }
              }
            }
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c)           // dims 4 c .. 4 c + 3 of the lane, two tokens side by side
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            unsigned a[4];
            widen4(__byte_perm(v[0][c], v[1][c], i ? 0x7362 : 0x5140), a[0], a[1]);
            widen4(__byte_perm(v[2][c], v[3][c], i ? 0x7362 : 0x5140), a[2], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816(acc[nb][2 * c + i], a, pb[nb][0], pb[nb][1]);
          }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&empty[st]));
      // one stage is kept behind: the tile before this one has been read, or nearly, by every warp
      if (next == done + STAGES - 1 && next < unit_end) fetch();
      ++done;
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], o);

#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (R[nb][e] == -INFINITY) m[nb][e] = -INFINITY;
    // ---- the unit's result, or this CTA's part of it ----
    // Lane (g, q4) has, of rows 2 q4 + e of each eight, the dims vdim(j, g), j = 2 i + (k >> 1) of acc[i][k], k & 1 == e.
    const bool whole = t0 == 0 && t1 == tiles;
    float *part = p.part + (int64_t)(2 * blockIdx.x + (t0 == 0)) * ROWS * (D + 2);
    if (dead) {                                    // copies may still be on their way: give them time, then leave
      for (int n = max(0, last_fetch - STAGES); n <= last_fetch; ++n)
        if ((n & 3) == warp) bar_wait(smem_addr(&full[n % STAGES]), n / STAGES & 1);
      if (lane == 0) atomicOr(p.c.status, pi::kKvTimeout);
      failed = 1;
    }
    __syncthreads();                               // every warp is done with the ring
    if (failed) return;
    if constexpr (KW > 1) {
      float *st = sm + KW * ROWS * D;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = wm * WROWS + nb * 8 + 2 * q4 + e;
          float *o = st + (wk * ROWS + row) * 3;
          if (g == 0) o[0] = m[nb][e], o[1] = l[nb][e], o[2] = R[nb][e];
          o = sm + (wk * ROWS + row) * D;
#pragma unroll
          for (int i = 0; i < MT; i += 2)
            *reinterpret_cast<float4 *>(o + F::vdim(2 * i, g)) =
                make_float4(acc[nb][i][e], acc[nb][i][2 + e], acc[nb][i + 1][e], acc[nb][i + 1][2 + e]);
        }
      __syncthreads();
      for (int i = threadIdx.x; i < ROWS * (D / 4); i += 128) {
        const int row = i / (D / 4), d = i % (D / 4) * 4;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) M = fmaxf(M, st[(w * ROWS + row) * 3]);
        const float ms = M == -INFINITY ? 0.f : M;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const float *t = st + (w * ROWS + row) * 3;
          L += t[1] * ex2(t[0] - ms);
          const float c = t[2] == -INFINITY ? 0.f : ex2(t[2] - ms);
          const float4 x = *reinterpret_cast<const float4 *>(sm + (w * ROWS + row) * D + d);
          o.x = fmaf(x.x, c, o.x), o.y = fmaf(x.y, c, o.y), o.z = fmaf(x.z, c, o.z), o.w = fmaf(x.w, c, o.w);
        }
        if (whole) {
          const int r = rt * ROWS + row;
          if (r >= sq.rows) continue;
          const int64_t orow = (int64_t)(sq.row0 + r / p.group) * p.q_heads + h * p.group + r % p.group;
          const float inv = L == 0.f ? 0.f : 1.0f / L;
          Pack<DT, 4> y;
          y.v[0] = E::from(o.x * inv), y.v[1] = E::from(o.y * inv), y.v[2] = E::from(o.z * inv), y.v[3] = E::from(o.w * inv);
          *reinterpret_cast<Pack<DT, 4> *>(static_cast<typename E::T *>(p.out) + orow * D + d) = y;
          if (p.lse && d == 0) p.lse[orow] = L == 0.f ? -INFINITY : (ms + log2f(L)) * kLn2;
        } else {
          *reinterpret_cast<float4 *>(part + row * D + d) = o;
          if (d == 0) part[ROWS * D + 2 * row] = M, part[ROWS * D + 2 * row + 1] = L;
        }
      }
      fence_async_smem();
      __syncthreads();                             // the sums have been read: the ring is free again
    } else {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = warp * WROWS + nb * 8 + 2 * q4 + e, gr = rt * ROWS + row;
          if (whole && gr >= sq.rows) continue;
          const float L = l[nb][e], ms = m[nb][e] == -INFINITY ? 0.f : m[nb][e];
          const float c = (R[nb][e] == -INFINITY ? 0.f : ex2(R[nb][e] - ms)) * (whole ? (L == 0.f ? 0.f : 1.0f / L) : 1.f);
          const int64_t orow = (int64_t)(sq.row0 + gr / p.group) * p.q_heads + h * p.group + gr % p.group;
#pragma unroll
          for (int i = 0; i < MT; i += 2) {
            const int d = F::vdim(2 * i, g);
            const float4 o = make_float4(acc[nb][i][e] * c, acc[nb][i][2 + e] * c, acc[nb][i + 1][e] * c, acc[nb][i + 1][2 + e] * c);
            if (whole) {
              Pack<DT, 4> y;
              y.v[0] = E::from(o.x), y.v[1] = E::from(o.y), y.v[2] = E::from(o.z), y.v[3] = E::from(o.w);
              *reinterpret_cast<Pack<DT, 4> *>(static_cast<typename E::T *>(p.out) + orow * D + d) = y;
            } else {
              *reinterpret_cast<float4 *>(part + row * D + d) = o;
            }
          }
          if (g == 0) {
            if (whole) {
              if (p.lse) p.lse[orow] = L == 0.f ? -INFINITY : (ms + log2f(L)) * kLn2;
            } else {
              part[ROWS * D + 2 * row] = m[nb][e], part[ROWS * D + 2 * row + 1] = L;
            }
          }
        }
    }

    pos = at.u0 + t1;
    if (pos >= at.end || !next_unit<ROWS, kTile>(p, &at)) break;
  }
}

struct AttnShape {
  int nb, warps_m;
};
// Rows of a row tile: the fewest eights that hold all query rows of a head
// while a warp's registers can (16 rows, 8 of 256 dims); above, two warps of that
// share a tile of keys (32 rows with two instead of four: 105 -> 66 us at 8 x 8192
// keys x 8 heads of 128), of 256 dims up to four.
AttnShape attn_shape(int D, int64_t max_rows) {
  const int nb_max = D <= 128 ? 2 : 1;
  const int nb = max_rows <= 8 ? 1 : nb_max;
  return AttnShape{nb, max_rows <= 8 * nb ? 1 : max_rows <= 16 * nb ? 2 : 4};
}

int attn_grid(int D, int nb) { return std::min(kMostShares, attn_ctas(D, nb) * std::max(1, pi::current_sms())); }

template <int DT, int D, int NB, int WARPS_M, bool TREE>
cudaError_t launch_attn(const AttnParams &p, cudaStream_t s) {
  constexpr int ROWS = 8 * NB * WARPS_M;
  constexpr int kRing = attn_stages<D, NB>() * Frag<D>::BYTES, kSums = WARPS_M < 4 ? 4 / WARPS_M * ROWS * (D + 3) * 4 : 0;
  constexpr int smem = (kRing > kSums ? kRing : kSums) + 1024;
  static_assert(attn_stages<D, NB>() >= 2 && attn_stages<D, NB>() <= 8);
  AttnMaps maps;
  if (!encode_codes<D>(&maps.k, p.c, p.c.k_codes) || !encode_codes<D>(&maps.v, p.c, p.c.v_codes)) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = pi::allow_smem(k_attn<DT, D, NB, WARPS_M, TREE>, smem, smem, done);
  if (e != cudaSuccess) return e;
  k_attn<DT, D, NB, WARPS_M, TREE><<<p.grid, 128, smem, s>>>(p, maps);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // its prefix sums overlap the main kernel's end
  return pi::launch_pdl(k_attn_combine<DT, D, ROWS, kTile>, dim3(combine_grid(p, D, ROWS)), dim3(kCombineThreads), 0, s, p);
}

template <int DT, int D, int NB, int WARPS_M>
cudaError_t launch_attn(const AttnParams &p, cudaStream_t s) {
  return p.tree ? launch_attn<DT, D, NB, WARPS_M, true>(p, s) : launch_attn<DT, D, NB, WARPS_M, false>(p, s);
}

template <int DT, int D>
cudaError_t attn_by_rows(const AttnParams &p, cudaStream_t s) {
  const AttnShape k = attn_shape(D, (int64_t)p.max_q * p.group);
  if constexpr (D <= 128) {
    if (k.nb == 1) return launch_attn<DT, D, 1, 1>(p, s);
    return k.warps_m == 1 ? launch_attn<DT, D, 2, 1>(p, s) : launch_attn<DT, D, 2, 2>(p, s);
  } else {
    return k.warps_m == 1 ? launch_attn<DT, D, 1, 1>(p, s) : k.warps_m == 2 ? launch_attn<DT, D, 1, 2>(p, s) : launch_attn<DT, D, 1, 4>(p, s);
  }
}

// From how many query rows a head on the tcgen05 kernel (row tiles of 128, each
// tile of keys widened once for them) is taken.  48 rows of 8 sequences x 8192 keys
// x 8 heads of 128: 79 us there, 105 us with four warps of 16 rows here; of one
// sequence of 3000 keys 24 and 32 us; of 64 sequences of 300 keys 68 and 58 us.
// 32 rows with two warps of 16 rows here: 66, 21 and 48 us (there 79, 23 and 68).
bool many_rows(int D, int64_t rows) { return D <= 128 && rows > 32; }
// A tree's kernel of many rows (pi_attn_tree.cu) is ahead from 17 rows on where caches are long: 24 to 32 rows, 8 heads of
// 128, 16 sequences of 20 to 8191 keys 73 us there, 93 to 98 here; 8 of 8192 65 and 70; one of 30000 39 and 40; of 64
// dims 51 and 63, 47 and 55, 32 and 33.  8 of 4000: 45 either way.  One of 3000: 24 and 21; 64 of 300: 61 and 45 to 47.
// Lengths are known on the device alone; the page table says how long a cache may be, so short caches under a wide
// one pay those differences (the header says so).
bool many_nodes(int D, int64_t rows, int64_t most_keys) { return D <= 128 && rows > 16 && most_keys >= 4096; }

template <int DT>
cudaError_t attn_by_dim(const AttnParams &p, cudaStream_t s) {
  switch (p.c.head_dim) {
    case 64: return attn_by_rows<DT, 64>(p, s);
    case 96: return attn_by_rows<DT, 96>(p, s);
    case 128: return attn_by_rows<DT, 128>(p, s);
    default: return attn_by_rows<DT, 256>(p, s);
  }
}

}  // namespace

namespace pi {

int current_sms() {
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms[dev];
}

}  // namespace pi

namespace {

pi_status attend(const pi_kv_cache *cache, const pi_kv_tokens *tokens, const int32_t *length, int32_t max_q, const int32_t *mask,
                 int32_t words, const void *q, const int64_t *q_stride, int32_t q_heads, int32_t dtype, float sm_scale,
                 int32_t causal, void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
  pi::clear_error();
  pi_status st = pi::check_cache(cache);
  if (st == PI_OK) st = pi::check_tokens(tokens);
  if (st != PI_OK) return st;
  if (dtype != PI_DT_F16 && dtype != PI_DT_BF16) return pi::fail(PI_ERR_INVALID_ARG, "q must be fp16 or bf16");
  if (q_heads < 1 || q_heads % cache->heads)
    return pi::fail(PI_ERR_INVALID_ARG, "q_heads=%d is not a multiple of the cache's %d heads", q_heads, cache->heads);
  if (max_q < 0) return pi::fail(PI_ERR_INVALID_ARG, "max_q=%d is negative", max_q);
  if (!(fabsf(sm_scale) < INFINITY)) return pi::fail(PI_ERR_INVALID_ARG, "sm_scale must be finite");
  if (tokens->n_tokens == 0 || tokens->n_seqs == 0 || max_q == 0) return PI_OK;
  if (!q || !q_stride || !out || !length || !pi::aligned_to(q, 16) || !pi::aligned_to(out, 16))
    return pi::fail(PI_ERR_INVALID_ARG, "q, q_stride, out and length must be non-NULL, q and out 16-byte aligned");
  if (q_stride[0] < 0 || q_stride[1] < 0 || q_stride[0] % 8 || q_stride[1] % 8)
    return pi::fail(PI_ERR_INVALID_ARG, "q's strides must be multiples of 8 elements");
  if (!pi::aligned_to(length, 4) || !pi::aligned_to(lse, 4))
    return pi::fail(PI_ERR_INVALID_ARG, "length and lse must be 4-byte aligned");
  max_q = std::min(max_q, tokens->n_tokens);
  if (mask && max_q > PI_MAX_TREE) return pi::fail(PI_ERR_UNSUPPORTED, "max_q=%d: up to %d with a mask", max_q, PI_MAX_TREE);
  if (mask && (int64_t)words * 32 < max_q)
    return pi::fail(PI_ERR_INVALID_ARG, "mask_words=%d hold no bits for max_q=%d", words, max_q);
  if ((int64_t)cache->n_pages * cache->heads >= (int64_t)1 << 31 ||
      (int64_t)tokens->n_seqs * cache->heads >= (int64_t)1 << 31 || (int64_t)max_q * (q_heads / cache->heads) >= 1 << 30)
    return pi::fail(PI_ERR_UNSUPPORTED, "n_pages x heads, n_seqs x heads or max_q x q_heads / heads is too large");
  const size_t need = pi_kv_attention_workspace_bytes(cache, q_heads, tokens->n_tokens, tokens->n_seqs);
  if (!ws || !pi::aligned_to(ws, 16) || ws_bytes < need)
    return pi::fail(PI_ERR_INVALID_ARG, "ws must be 16-byte aligned and hold %zu bytes, has %zu", need, ws_bytes);
  const int group = q_heads / cache->heads;
  const AttnShape shape = attn_shape(cache->head_dim, (int64_t)max_q * group);
  const int rows = 8 * shape.nb * shape.warps_m;
  const AttnParams p{*cache, pi::with_pages(*tokens), length, q, q_stride[0], q_stride[1], out, lse, static_cast<int4 *>(ws),
                     reinterpret_cast<float *>(static_cast<int4 *>(ws) + attn_grid(cache->head_dim, 1)),
                     sm_scale * kLog2e, q_heads, group, max_q, causal != 0,
                     (int)(((int64_t)max_q * group + rows - 1) / rows), attn_grid(cache->head_dim, shape.nb),
                     (pi::aligned_to(q, 32) && q_stride[0] % 16 == 0 && q_stride[1] % 16 == 0 ? 1 : 0) |
                         (pi::aligned_to(out, 32) ? 2 : 0) |
                         (pi::aligned_to(static_cast<int4 *>(ws) + attn_grid(cache->head_dim, 1), 32) ? 4 : 0),
                     mask, words};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t q_rows = (int64_t)max_q * group;
  if (many_rows(cache->head_dim, q_rows) || (mask && many_nodes(cache->head_dim, q_rows, (int64_t)p.tok.table_pages * cache->page_size)))
    PI_TRY_CUDA(mask ? run_tree(p, dtype, s) : run_tc(p, dtype, s));
  else
    PI_TRY_CUDA(dtype == PI_DT_F16 ? attn_by_dim<PI_DT_F16>(p, s) : attn_by_dim<PI_DT_BF16>(p, s));
  return PI_OK;
}

}  // namespace

extern "C" {

size_t pi_kv_attention_workspace_bytes(const pi_kv_cache *c, int32_t q_heads, int32_t n_tokens, int32_t n_seqs) {
  pi::clear_error();
  if (pi::check_cache(c) != PI_OK || q_heads < 1 || n_tokens < 0 || n_seqs < 0) return 0;
  const int D = c->head_dim;
  const size_t rows = D <= 128 ? std::max({(size_t)attn_grid(D, 1) * 8, (size_t)attn_grid(D, 2) * 32, (size_t)std::max(1, pi::current_sms()) * kTcRows}) : (size_t)attn_grid(D, 1) * 32;
  return sizeof(int4) * attn_grid(D, 1) + sizeof(float) * 2 * rows * (size_t)(D + 2);
}

pi_status pi_kv_attention(const pi_kv_cache *cache, const pi_kv_tokens *tokens, const int32_t *length, int32_t max_q,
                          const void *q, const int64_t *q_stride, int32_t q_heads, int32_t dtype, float sm_scale,
                          int32_t causal, void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
  return attend(cache, tokens, length, max_q, nullptr, 0, q, q_stride, q_heads, dtype, sm_scale, causal, out, lse, ws, ws_bytes, stream);
}

pi_status pi_kv_tree_attention(const pi_kv_cache *cache, const pi_kv_tokens *tokens, const int32_t *length, int32_t max_q,
                               const int32_t *mask, int32_t mask_words, const void *q, const int64_t *q_stride, int32_t q_heads,
                               int32_t dtype, float sm_scale, void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
  pi::clear_error();
  if (!mask || !pi::aligned_to(mask, 4) || mask_words < 1)
    return pi::fail(PI_ERR_INVALID_ARG, "mask must be non-NULL and 4-byte aligned, mask_words=%d at least 1", mask_words);
  return attend(cache, tokens, length, max_q, mask, mask_words, q, q_stride, q_heads, dtype, sm_scale, 1, out, lse, ws, ws_bytes, stream);
}

}  // extern "C"
