// New keys, turned by their positions, and values into the 8-bit cache, and the
// same tokens' queries turned, in one launch.
//
// As the cache write (pi_kv.cu) a warp has a block's 16 tokens of one head of the
// keys or the values, and here of the queries too: those it stores turned instead
// of quantised.  A CTA works on one block, so the cosines and sines of its tokens
// are computed once, into shared memory, for all its heads.  Turned keys are not
// rounded before they are quantised: a code is the binary32 result rounded once.
// A key is turned twice, for the block's largest element and for its codes, which
// costs less than the registers that would keep it.  A warp loads its next head while it
// turns one (16-bit types up to 128 dims, whose registers hold both).
//
// Measured: prompts of 24003 tokens, 64 query heads on 8 of 128, bf16: 156 us (6.3 TB/s, 93% of
// the copy rate; 172 without loading ahead); one token of 32 sequences 7.2 us, the latency of a block's
// place, its rows and its old scale.  Five prompts of 24003 tokens in all, the same heads: 145 us in 16 bits,
// 293 in binary32 (95% and 91%); 32 heads on 4 of 256: bf16 152, fp16 191, binary32 400 (90%, 72%, 67%).  At 256
// dims a lane's part of a head is more than its 128 registers hold beside the sums: fp16 spills 788 to 820
// bytes a thread and binary32 292 to 1404, bf16 nothing, 128 dims 4 to 28.
#include "pi_kv_blocks.cuh"
#include "pi_rope.cuh"

#include <algorithm>

using namespace kv;

namespace {

struct AppendParams {
  KvCopyParams kv;
  pi_rotary r;
  const int32_t *pos;       // or NULL: positions in the sequence
  const void *q;
  void *q_out;
  int64_t qt, qh;
  int q_heads;
};

template <int DT, int D, bool VEC, bool HALF, bool AHEAD>
__global__ void __launch_bounds__(256, 2) k_kv_append(const AppendParams a) {
  using E = Elem<DT>;
  using T = typename E::T;
  const KvCopyParams &p = a.kv;
  constexpr int VR = D / 8, NP = VR / 4, W = 8 * sizeof(T) / 16;     // vectors of 8 a row, pairs of them a lane, accesses a vector
  __shared__ float4 table[PI_KV_BLOCK * D / 4];
  kv_check_cu(p);
  const int lane = threadIdx.x & 31, all = 2 * p.c.heads + a.q_heads, parts = (all + 8 * p.per_warp - 1) / (8 * p.per_warp);
  KvPlace at;
  bool ok;
  if (!kv_place(p, blockIdx.x / parts, &at, &ok)) return;            // the same for the whole CTA
  int unit = blockIdx.x % parts * 8 * p.per_warp + (threadIdx.x >> 5);
  const int units = min(all, unit + 8 * p.per_warp);
  const int rp = a.r.dim / 16;                                       // turned pairs of vectors a row

  // pair t of a row: its two vectors
  auto col = [&](int t, bool turned, int second) {
    return HALF && turned && t < rp ? t + second * rp : 2 * t + second;
  };
  uint4 x[NP][2][W], next[AHEAD ? NP : 1][2][W];
  auto load = [&](uint4 (*x)[2][W], int unit) {
    const int kind = unit < p.c.heads ? 0 : unit < 2 * p.c.heads ? 1 : 2;
    const int h = unit - kind * p.c.heads;
    const int64_t st = kind == 2 ? a.qt : p.st[kind], sh = kind == 2 ? a.qh : p.sh[kind];
    const T *src = static_cast<const T *>(kind == 2 ? a.q : p.src[kind]) + (int64_t)at.row0 * st + h * sh;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int e = lane + 32 * i, r = e / (VR / 2) - at.off, t = e % (VR / 2);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int c = 0; c < W; ++c) x[i][s][c] = make_uint4(0, 0, 0, 0);
        if (r >= 0 && r < at.n) {
          const T *row = src + (int64_t)r * st + col(t, kind != 1, s) * 8;
          if constexpr (VEC) {
#pragma unroll
            for (int c = 0; c < W; ++c) x[i][s][c] = reinterpret_cast<const uint4 *>(row)[c];
          } else {
            alignas(16) T e8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) e8[k] = row[k];
#pragma unroll
            for (int c = 0; c < W; ++c) x[i][s][c] = reinterpret_cast<const uint4 *>(e8)[c];
          }
        }
      }
    }
  };
  // the pair's 16 elements, turned where they are to be
  auto values = [&](f2 *v, int i, bool turned) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * s + k] = f2_from16<DT>(x[i][s][W == 2 ? k / 2 : 0], W == 2 ? k % 2 : k);
    const int e = lane + 32 * i, row = e / (VR / 2) - at.off, t = e % (VR / 2);
    if (turned && t < rp && row >= 0 && row < at.n) rope_turn<8, HALF>(v, table + row * 4 * rp + t, rp);
  };

  if (unit < units) load(x, unit);
  const int freqs = a.r.dim / 2;
  for (int i = threadIdx.x; i < at.n * freqs; i += 256) {
    const int r = i / freqs, f = i % freqs;
    rope_put<8>(table + r * 4 * rp, rp, f, rope_angle(a.r.turns[f], a.pos ? a.pos[at.row0 + r] : at.pos + r, a.r.magnitude));
  }
  __syncthreads();
  auto advance = [&] {
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int c = 0; c < W; ++c) x[i][s][c] = next[i][s][c];
    } else if (unit + 8 < units) {
      load(x, unit + 8);
    }
  };
#pragma unroll 1
  for (; unit < units; advance(), unit += 8) {
    if constexpr (AHEAD)
      if (unit + 8 < units) load(next, unit + 8);
    if (unit >= 2 * p.c.heads) {
      const int h = unit - 2 * p.c.heads;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int e = lane + 32 * i, r = e / (VR / 2) - at.off, t = e % (VR / 2);
        if (r < 0 || r >= at.n) continue;
        f2 v[8];
        values(v, i, true);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint4 *row = reinterpret_cast<uint4 *>(static_cast<T *>(a.q_out) + ((int64_t)(at.row0 + r) * a.q_heads + h) * D + col(t, true, s) * 8);
          row[0] = f2_to16<DT>(v + 4 * s);
          if constexpr (DT == PI_DT_F32) row[1] = f2_to16<DT>(v + 4 * s + 2);
        }
      }
      continue;
    }
    if (!ok) continue;
    const int kv = unit >= p.c.heads, h = unit - kv * p.c.heads;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      f2 v[8];
      values(v, i, !kv);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float b = fabsf(v[k].x), c = fabsf(v[k].y);
        amax = fmaxf(amax, fmaxf(b < INFINITY ? b : 0.f, c < INFINITY ? c : 0.f));
      }
    }
    float s = pow2(scale_exp(warp_max(amax)));
    const int64_t page_head = (int64_t)at.page * p.c.heads + h;
    float *scale = (kv ? p.c.v_scales : p.c.k_scales) + page_head * (p.c.page_size / PI_KV_BLOCK) + at.blk;
    uint2 *codes = reinterpret_cast<uint2 *>((kv ? p.c.v_codes : p.c.k_codes) +
                                             (page_head * p.c.page_size + at.blk * PI_KV_BLOCK) * D);
    if (at.off > 0) {
      const float old = *scale;
      if (old < s) {
        for (int v = lane; v < at.off * VR; v += 32) {
          f2 f[4];
          decode8(f, codes[v]);
          codes[v] = encode8(f, f2_of(old / s, old / s));
        }
      } else if (old > s) {
        s = old;
      }
    }
    const float inv = 1.0f / s;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int e = lane + 32 * i, row = e / (VR / 2), t = e % (VR / 2), r = row - at.off;
      if (r < 0 || r >= at.n) continue;
      f2 v[8];
      values(v, i, !kv);
#pragma unroll
      for (int c = 0; c < 2; ++c) codes[row * VR + col(t, !kv, c)] = encode8(v + 4 * c, f2_of(inv, inv));
    }
    __syncwarp();                                    // every lane has read the old scale
    if (lane == 0) *scale = s;
  }
}

template <int DT, int D>
cudaError_t launch(AppendParams a, bool vec, cudaStream_t s) {
  const int units = 2 * a.kv.c.heads + a.q_heads;
  // as in the cache write: with enough blocks to fill the GPU a warp does several heads of one
  a.kv.per_warp = std::max<int64_t>(1, std::min<int64_t>((units + 7) / 8, (int64_t)a.kv.n_slots * units / (64 * std::max(1, pi::current_sms()))));
  const unsigned grid = (unsigned)((int64_t)std::max(1, a.kv.n_slots) * ((units + 8 * a.kv.per_warp - 1) / (8 * a.kv.per_warp)));
  constexpr bool kAhead = D <= 128 && DT != PI_DT_F32;             // twice a unit's registers fit
  if (a.r.interleaved)
    vec ? k_kv_append<DT, D, true, false, kAhead><<<grid, 256, 0, s>>>(a) : k_kv_append<DT, D, false, false, false><<<grid, 256, 0, s>>>(a);
  else
    vec ? k_kv_append<DT, D, true, true, kAhead><<<grid, 256, 0, s>>>(a) : k_kv_append<DT, D, false, true, false><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <int DT>
cudaError_t by_dim(const AppendParams &a, bool vec, cudaStream_t s) {
  switch (a.kv.c.head_dim) {
    case 64: return launch<DT, 64>(a, vec, s);
    case 96: return launch<DT, 96>(a, vec, s);
    case 128: return launch<DT, 128>(a, vec, s);
    default: return launch<DT, 256>(a, vec, s);
  }
}

}  // namespace

extern "C" pi_status pi_kv_append(const pi_kv_cache *cache, const pi_kv_tokens *tokens, const int32_t *start,
                                  const pi_rotary *rotary, const int32_t *positions, const void *k, const int64_t *k_stride,
                                  const void *v, const int64_t *v_stride, const void *q, const int64_t *q_stride,
                                  int32_t q_heads, void *q_out, int32_t dtype, void *stream) {
  AppendParams a;
  pi_status st = pi::check_copy(cache, tokens, start, dtype, &a.kv);
  if (st == PI_OK) st = pi::check_rotary(rotary, cache->head_dim);
  if (st != PI_OK) return st;
  if (rotary->dim % 16) return pi::fail(PI_ERR_UNSUPPORTED, "rotary dim=%d: a multiple of 16 here", rotary->dim);
  if (q_heads < 0 || q_heads > 65535 || (q_heads > 0) != (q != nullptr) || (q != nullptr) != (q_out != nullptr))
    return pi::fail(PI_ERR_INVALID_ARG, "q_heads=%d: q and q_out both with it, or neither", q_heads);
  if (tokens->n_tokens == 0 || tokens->n_seqs == 0) return PI_OK;
  const int e = pi::dtype_size(dtype), V = 16 / e;
  if (!k || !v || !k_stride || !v_stride || !pi::aligned_to(k, e) || !pi::aligned_to(v, e))
    return pi::fail(PI_ERR_INVALID_ARG, "k, v and their strides must be non-NULL, k and v aligned to their type");
  if (q && (!q_stride || !pi::aligned_to(q, e) || !pi::aligned_to(q_out, 16)))
    return pi::fail(PI_ERR_INVALID_ARG, "q_stride must be non-NULL, q aligned to its type, q_out 16-byte aligned");
  if (!pi::aligned_to(positions, 4)) return pi::fail(PI_ERR_INVALID_ARG, "positions must be 4-byte aligned");
  if ((int64_t)(a.kv.n_slots + 1) * ((2 * cache->heads + q_heads) / 8 + 1) >= (int64_t)1 << 31)
    return pi::fail(PI_ERR_UNSUPPORTED, "n_tokens=%d with heads=%d and q_heads=%d is too large for one call", tokens->n_tokens,
                    cache->heads, q_heads);
  bool vec = true;
  const void *src[3] = {k, v, q};
  const int64_t *stride[3] = {k_stride, v_stride, q_stride};
  for (int i = 0; i < (q ? 3 : 2); ++i) {
    const int64_t *s = stride[i];
    if (s[0] < 0 || s[1] < 0) return pi::fail(PI_ERR_INVALID_ARG, "strides must not be negative");
    vec = vec && pi::aligned_to(src[i], 16) && s[0] % V == 0 && s[1] % V == 0;
  }
  for (int i = 0; i < 2; ++i) a.kv.src[i] = src[i], a.kv.st[i] = stride[i][0], a.kv.sh[i] = stride[i][1];
  a.r = *rotary, a.pos = positions, a.q = q, a.q_out = q_out, a.q_heads = q ? q_heads : 0;
  a.qt = q ? q_stride[0] : 0, a.qh = q ? q_stride[1] : 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PI_TRY_CUDA(dtype == PI_DT_F16    ? by_dim<PI_DT_F16>(a, vec, s)
              : dtype == PI_DT_BF16 ? by_dim<PI_DT_BF16>(a, vec, s)
                                    : by_dim<PI_DT_F32>(a, vec, s));
  return PI_OK;
}
