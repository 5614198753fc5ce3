// Layer norm, forward (with an optional addition before it) and backward.
//
//   y  = (t - mean) rstd w + b          t = x, or the stored sum x + add
//   dx = rstd (g - mean_j(g) - h mean_j(g h)) + d_sum,  h = (t - mean) rstd, g = dy w
//   dw = sum_rows dy h,  db = sum_rows dy
//
// Bound by HBM: a handful of operations per element read.  A row is read once
// and stays in registers between its reductions, so the variance is the mean
// square about the mean (no cancellation) at no extra traffic.
//
// Measured: 16384 x 8192 bf16 84 us (6.4 TB/s, 95% of the copy rate); its gradient
// with d_sum, 16001 x 4096 bf16, 111 us (4.7 TB/s, 70%; binary32 161 us, 97%: the 16-bit
// rows' chain of two passes and a reduction is not hidden by 16 warps an SM, which
// its sums' registers allow); 8 x 4096 with an addition 3 us.
#include "pi_ops.cuh"

#include <algorithm>
#include <type_traits>

using namespace pidev;

namespace {

// Which columns a thread has: NP pairs.  VEC: NV packs of 16 bytes (V
// elements), pack t + i NT; pair j is half of pack j / (V / 2).  Otherwise
// pair j is the two columns t + 2 j NT and t + (2 j + 1) NT.
template <int X, bool VEC, int NT, int NV>
struct Cols {
  static constexpr int V = 16 / sizeof(typename Elem<X>::T), PP = V / 2, NP = VEC ? NV * PP : NV;
};

// Pairs of a row of another tensor (a weight, an added row) at this thread's
// columns, of a type known at run time; `one` where absent or past the row.
template <int V>
__device__ __forceinline__ void load_pack(f2 *o, const void *p, int dt, int k) {
  if (dt == PI_DT_F32) {
#pragma unroll
    for (int c = 0; c < V / 4; ++c) {
      const uint4 w = static_cast<const uint4 *>(p)[k * (V / 4) + c];
      o[2 * c] = f2_from16<PI_DT_F32>(w, 0), o[2 * c + 1] = f2_from16<PI_DT_F32>(w, 1);
    }
  } else {
    uint4 w = make_uint4(0, 0, 0, 0);
    if constexpr (V == 8) {
      w = static_cast<const uint4 *>(p)[k];
    } else {
      const uint2 h = static_cast<const uint2 *>(p)[k];
      w.x = h.x, w.y = h.y;
    }
#pragma unroll
    for (int j = 0; j < V / 2; ++j) o[j] = dt == PI_DT_F16 ? f2_from16<PI_DT_F16>(w, j) : f2_from16<PI_DT_BF16>(w, j);
  }
}
template <int X, bool VEC, int NT, int NV>
__device__ __forceinline__ void load_cols(f2 *o, const void *p, int dt, int t, int d, float one) {
  using C = Cols<X, VEC, NT, NV>;
  const f2 fill = f2_of(one, one);
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < C::PP; ++j) o[i * C::PP + j] = fill;
      if (p && t + i * NT < d / C::V) load_pack<C::V>(o + i * C::PP, p, dt, t + i * NT);
    }
  } else {
    auto load = [&](auto type) {                     // all loads of one type, so that they are under way together
      constexpr int Y = decltype(type)::value;
      typename Elem<Y>::T raw[2 * C::NP];
#pragma unroll
      for (int j = 0; j < 2 * C::NP; ++j)
        if (t + j * NT < d) raw[j] = static_cast<const typename Elem<Y>::T *>(p)[t + j * NT];
#pragma unroll
      for (int j = 0; j < C::NP; ++j) {
        const int c0 = t + 2 * j * NT;
        o[j] = f2_of(c0 < d ? Elem<Y>::to(raw[2 * j]) : one, c0 + NT < d ? Elem<Y>::to(raw[2 * j + 1]) : one);
      }
    };
    if (!p) {
#pragma unroll
      for (int j = 0; j < C::NP; ++j) o[j] = fill;
    } else if (dt == PI_DT_F32) {
      load(std::integral_constant<int, PI_DT_F32>());
    } else if (dt == PI_DT_F16) {
      load(std::integral_constant<int, PI_DT_F16>());
    } else {
      load(std::integral_constant<int, PI_DT_BF16>());
    }
  }
}
// Pairs of a row of X, 0 past its end; and their store.
template <int X, int NT, int NP>
__device__ __forceinline__ void load_scalar(f2 *o, const typename Elem<X>::T *row, int t, int d) {
  typename Elem<X>::T raw[2 * NP];
#pragma unroll
  for (int j = 0; j < 2 * NP; ++j) raw[j] = Elem<X>::from(0.f);
#pragma unroll
  for (int j = 0; j < 2 * NP; ++j)
    if (t + j * NT < d) raw[j] = row[t + j * NT];
#pragma unroll
  for (int j = 0; j < NP; ++j) o[j] = f2_of(Elem<X>::to(raw[2 * j]), Elem<X>::to(raw[2 * j + 1]));
}
template <int X, bool VEC, int NT, int NV>
__device__ __forceinline__ void store_cols(typename Elem<X>::T *row, const f2 *v, int t, int d) {
  using C = Cols<X, VEC, NT, NV>;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t + i * NT < d / C::V) reinterpret_cast<uint4 *>(row)[t + i * NT] = f2_to16<X>(v + i * C::PP);
  } else {
#pragma unroll
    for (int j = 0; j < C::NP; ++j) {
      const float2 f = f2_get(v[j]);
      const int c0 = t + 2 * j * NT, c1 = c0 + NT;
      if (c0 < d) row[c0] = Elem<X>::from(f.x);
      if (c1 < d) row[c1] = Elem<X>::from(f.y);
    }
  }
}
// 1 where pair j's halves are columns of the row, 0 past its end (scalar
// columns; a pack is all in or all out).
template <int NT>
__device__ __forceinline__ f2 in_row(int j, int t, int d) {
  return f2_of(t + 2 * j * NT < d ? 1.f : 0.f, t + (2 * j + 1) * NT < d ? 1.f : 0.f);
}

// A thread's 16-byte pieces of the rows that its group works on next, in
// shared memory: it copies them there itself (cp.async) and is the only one to
// read them, so a stage needs no barrier and no wait but its own.  The copies
// in flight take no registers, and a row's load is hidden behind the rows
// before it.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *dst, const void *src) {
  const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most n of the newest groups are in flight (n < 4).
__device__ __forceinline__ void copy_wait(int n) {
  if (n >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

struct NormParams {
  const void *x, *add, *w, *b;
  void *y, *sum;
  float *mean, *rstd;
  int64_t x_stride;
  int rows, d, add_dt, w_dt;
  float eps;
  int stages, stage_bytes;   // ring of one CTA
};

// CTAs of NT threads (128 at least) that an SM holds.  Rows through the ring have
// their loads in flight without a thread's registers: 512 threads, of 128
// registers, do (16384 x 8192 bf16: 85 us, 155 us with 1024); plain loads need more.
constexpr int norm_ctas(int NT, bool VEC) { return std::max(1, (VEC ? 512 : 1024) / std::max(NT, 128)); }
// The same of the gradient kernel (256 threads at least), by columns of a thread.
constexpr int grad_ctas_sm(int NT, int cols) { return NT > 256 ? 1 : cols <= 8 ? 3 : 2; }

// Group of NT threads per row (a CTA has 128 at least: four groups of one warp,
// two of two).
// VEC: rows come through the ring, one after another to each group; otherwise
// (odd widths, unaligned rows) plain loads, a group for each row.
// WREG: weight and bias have x's type (or are absent) and stay in registers.
template <int X, bool VEC, int NT, int NV, bool WREG>
__global__ void __launch_bounds__(NT < 128 ? 128 : NT, norm_ctas(NT, VEC)) k_norm(const NormParams p) {
  using E = Elem<X>;
  using T = typename E::T;
  using C = Cols<X, VEC, NT, NV>;
  constexpr int V = C::V, PP = C::PP, NP = C::NP;
  constexpr int GROUPS = NT < 128 ? 128 / NT : 1, CT = NT * GROUPS;
  extern __shared__ __align__(16) char ring[];
  __shared__ float red[2][2][32];
  const int t = threadIdx.x % NT, g = threadIdx.x / NT;
  const int nv = p.d / V;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  const int64_t row0 = (int64_t)blockIdx.x * GROUPS + g;

  // a stage: the groups' rows of x, then of what is added (its packs' halves apart)
  const int add_bytes = !VEC || !p.add ? 0 : V * (p.add_dt == PI_DT_F32 ? 4 : 2);   // per pack: 8, 16 or 32
  auto x_slot = [&](int stage, int i) { return ring + (size_t)stage * p.stage_bytes + (g * nv + t + i * NT) * 16; };
  auto a_slot = [&](int stage, int i, int half) {
    return ring + (size_t)stage * p.stage_bytes + ((GROUPS * (1 + half) + g) * nv + t + i * NT) * 16;
  };
  auto fetch = [&](int64_t row, int stage) {
    if constexpr (VEC) {
      if (row < p.rows) {
        const T *x = static_cast<const T *>(p.x) + row * p.x_stride;
        const char *a = static_cast<const char *>(p.add) + (size_t)row * nv * add_bytes;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int k = t + i * NT;
          if (k >= nv) continue;
          copy_async<16>(x_slot(stage, i), x + (size_t)k * V);
          if (add_bytes == 8) copy_async<8>(a_slot(stage, i, 0), a + (size_t)k * 8);
          if (add_bytes >= 16) copy_async<16>(a_slot(stage, i, 0), a + (size_t)k * add_bytes);
          if (add_bytes == 32) copy_async<16>(a_slot(stage, i, 1), a + (size_t)k * 32 + 16);
        }
      }
      copy_commit();
    }
  };
  for (int s = 0; s < p.stages - 1; ++s) fetch(row0 + s * step, s);

  uint4 rw[WREG ? NV : 1], rb[WREG ? NV : 1];
  if constexpr (WREG) {
    f2 one[PP];
#pragma unroll
    for (int j = 0; j < PP; ++j) one[j] = f2_of(1.f, 1.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = t + i * NT;
      rw[i] = f2_to16<X>(one), rb[i] = make_uint4(0, 0, 0, 0);
      if (k < nv && p.w) rw[i] = static_cast<const uint4 *>(p.w)[k];
      if (k < nv && p.b) rb[i] = static_cast<const uint4 *>(p.b)[k];
    }
  }

  f2 ww[WREG ? 1 : NP], bb[WREG ? 1 : NP];           // plain loads: a row a group, so these come beside x's
  if constexpr (!WREG && !VEC) {
    load_cols<X, VEC, NT, NV>(ww, p.w, p.w_dt, t, p.d, 1.f);
    load_cols<X, VEC, NT, NV>(bb, p.b, p.w_dt, t, p.d, 0.f);
  }
  int turn = 0, at = 0, next = p.stages - 1;
  for (int64_t row = row0; row < p.rows; row += step, turn ^= 1) {
    f2 v[NP];
    if constexpr (VEC) {
      fetch(row + (p.stages - 1) * step, next);
      copy_wait(p.stages - 1);
      next = next + 1 == p.stages ? 0 : next + 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (t + i * NT < nv) w = *reinterpret_cast<const uint4 *>(x_slot(at, i));
#pragma unroll
        for (int j = 0; j < PP; ++j) v[i * PP + j] = f2_from16<X>(w, j);
      }
    } else {
      load_scalar<X, NT, NP>(v, static_cast<const T *>(p.x) + row * p.x_stride, t, p.d);
    }
    if (p.add) {
      T *sum = static_cast<T *>(p.sum) + (size_t)row * p.d;
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (t + i * NT >= nv) continue;
          f2 a[PP];
          if (p.add_dt == PI_DT_F32) {
#pragma unroll
            for (int c = 0; c < V / 4; ++c) {
              const uint4 w = *reinterpret_cast<const uint4 *>(a_slot(at, i, c));
              a[2 * c] = f2_from16<PI_DT_F32>(w, 0), a[2 * c + 1] = f2_from16<PI_DT_F32>(w, 1);
            }
          } else {
            load_pack<V>(a, a_slot(at, i, 0), p.add_dt, 0);
          }
#pragma unroll
          for (int j = 0; j < PP; ++j) a[j] = f2_add(v[i * PP + j], a[j]);
          const uint4 w = f2_to16<X>(a);
          reinterpret_cast<uint4 *>(sum)[t + i * NT] = w;
#pragma unroll
          for (int j = 0; j < PP; ++j) v[i * PP + j] = f2_from16<X>(w, j);
        }
      } else {
        f2 a[NP];
        load_cols<X, false, NT, NV>(a, static_cast<const char *>(p.add) + (size_t)row * p.d * (p.add_dt == PI_DT_F32 ? 4 : 2),
                                    p.add_dt, t, p.d, 0.f);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const float2 f = f2_get(f2_add(v[j], a[j]));
          v[j] = f2_of(E::to(E::from(f.x)), E::to(E::from(f.y)));
        }
        store_cols<X, false, NT, NV>(sum, v, t, p.d);
      }
    }
    at = at + 1 == p.stages ? 0 : at + 1;
    f2 s = f2_of(0.f, 0.f), q = s;
#pragma unroll
    for (int j = 0; j < NP; ++j) s = f2_add(s, v[j]);
    const float mean = group_sum<NT, CT>(f2_sum(s), red[turn][0], g) / (float)p.d;
    const f2 minus = f2_of(-mean, -mean);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      v[j] = f2_add(v[j], minus);
      if constexpr (VEC) {
        if (t + j / PP * NT < nv) q = f2_fma(v[j], v[j], q);
      } else {
        q = f2_fma(f2_mul(v[j], in_row<NT>(j, t, p.d)), v[j], q);
      }
    }
    const float rstd = 1.0f / sqrtf(group_sum<NT, CT>(f2_sum(q), red[turn][1], g) / (float)p.d + p.eps);
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    const f2 scale = f2_of(rstd, rstd);
    T *y = static_cast<T *>(p.y) + (size_t)row * p.d;
    if constexpr (WREG) {
#pragma unroll
      for (int j = 0; j < NP; ++j)
        v[j] = f2_fma(f2_mul(v[j], scale), f2_from16<X>(rw[j / PP], j % PP), f2_from16<X>(rb[j / PP], j % PP));
    } else {
      if constexpr (VEC) {
        load_cols<X, VEC, NT, NV>(ww, p.w, p.w_dt, t, p.d, 1.f);
        load_cols<X, VEC, NT, NV>(bb, p.b, p.w_dt, t, p.d, 0.f);
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) v[j] = f2_fma(f2_mul(v[j], scale), ww[j], bb[j]);
    }
    store_cols<X, VEC, NT, NV>(y, v, t, p.d);
  }
}

struct NormGradParams {
  const void *dy, *x, *w, *dsum;
  const float *mean, *rstd;
  void *dx;
  float *part;          // [CTAs, 2, d]: dweight, dbias over the rows of one CTA
  int64_t x_stride;
  int rows, d, w_dt;
  int stages, stage_bytes;
};

// Each group of NT threads takes the rows g, g + groups, ...; a thread keeps
// its columns over all of them, so dweight and dbias add up in its registers.
// HOLD: h and g of a row stay in registers between the passes; without it
// (the widest rows, whose threads have 64 registers) they are formed again.
template <int X, bool VEC, int NT, int NV>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT, grad_ctas_sm(NT, 2 * Cols<X, VEC, NT, NV>::NP)) k_norm_grad(const NormGradParams p) {
  using E = Elem<X>;
  using T = typename E::T;
  using C = Cols<X, VEC, NT, NV>;
  constexpr int V = C::V, PP = C::PP, NP = C::NP;
  constexpr int GROUPS = NT < 256 ? 256 / NT : 1, CT = NT * GROUPS;
  constexpr bool HOLD = NT <= 512;
  extern __shared__ __align__(16) char ring[];       // stages, then (GROUPS > 1) [2, d] sums
  __shared__ float red[2][2][32];
  const int t = threadIdx.x % NT, g = threadIdx.x / NT;
  const int nv = p.d / V;
  const float inv = 1.0f / (float)p.d;
  const int64_t step = (int64_t)gridDim.x * GROUPS, row0 = (int64_t)blockIdx.x * GROUPS + g;
  const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy), *ds = static_cast<const T *>(p.dsum);

  auto slot = [&](int stage, int which, int i) {
    return reinterpret_cast<uint4 *>(ring + (size_t)stage * p.stage_bytes + ((which * GROUPS + g) * nv + t + i * NT) * 16);
  };
  auto fetch = [&](int64_t row, int stage) {
    if constexpr (VEC) {
      if (row < p.rows) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int k = t + i * NT;
          if (k >= nv) continue;
          copy_async<16>(slot(stage, 0, i), x + row * p.x_stride + (size_t)k * V);
          copy_async<16>(slot(stage, 1, i), dy + (size_t)row * p.d + (size_t)k * V);
          if (ds) copy_async<16>(slot(stage, 2, i), ds + (size_t)row * p.d + (size_t)k * V);
        }
      }
      copy_commit();
    }
  };
  for (int s = 0; s < p.stages; ++s) fetch(row0 + s * step, s);
  griddep_launch();                                  // the column sums' CTAs take the places that this grid leaves

  f2 dw[NP], db[NP], w[HOLD ? NP : 1];
#pragma unroll
  for (int j = 0; j < NP; ++j) dw[j] = db[j] = f2_of(0.f, 0.f);
  if constexpr (HOLD) load_cols<X, VEC, NT, NV>(w, p.w, p.w_dt, t, p.d, 1.f);

  int turn = 0, at = 0;
  for (int64_t row = row0; row < p.rows; row += step, turn ^= 1) {
    const float mean = p.mean[row], rstd = p.rstd[row];
    const f2 minus = f2_of(-mean, -mean), scale = f2_of(rstd, rstd);
    if constexpr (VEC) copy_wait(p.stages - 1);
    // pass 1: h and g (0 past the row's end, where dy is read as 0), the column sums and the row's two sums
    f2 h[NP], gg[NP], s1 = f2_of(0.f, 0.f), s2 = s1;
    auto form = [&](f2 *ho, f2 *go, bool sums) {
      f2 xs[VEC ? 1 : NP], ys[VEC ? 1 : NP];
      f2 wl[HOLD ? 1 : NP];
      if constexpr (!HOLD) load_cols<X, VEC, NT, NV>(wl, p.w, p.w_dt, t, p.d, 1.f);
      if constexpr (!VEC) {
        load_scalar<X, NT, NP>(xs, x + row * p.x_stride, t, p.d);
        load_scalar<X, NT, NP>(ys, dy + (size_t)row * p.d, t, p.d);
      }
#pragma unroll
      for (int i = 0; i < NP / (VEC ? PP : 1); ++i) {
        uint4 rx = make_uint4(0, 0, 0, 0), ry = make_uint4(0, 0, 0, 0);
        if constexpr (VEC)
          if (t + i * NT < nv) rx = *slot(at, 0, i), ry = *slot(at, 1, i);
#pragma unroll
        for (int c = 0; c < (VEC ? PP : 1); ++c) {
          const int j = i * (VEC ? PP : 1) + c;
          const f2 xv = VEC ? f2_from16<X>(rx, c) : xs[VEC ? 0 : j], yv = VEC ? f2_from16<X>(ry, c) : ys[VEC ? 0 : j];
          ho[j] = f2_mul(f2_add(xv, minus), scale);
          go[j] = f2_mul(yv, HOLD ? w[HOLD ? j : 0] : wl[HOLD ? 0 : j]);
          if (sums) {
            dw[j] = f2_fma(yv, ho[j], dw[j]);
            db[j] = f2_add(db[j], yv);
            s1 = f2_add(s1, go[j]);
            s2 = f2_fma(go[j], ho[j], s2);
          }
        }
      }
    };
    form(h, gg, true);
    float a = warp_sum(f2_sum(s1)), b = warp_sum(f2_sum(s2));
    if constexpr (NT > 32) {
      if ((threadIdx.x & 31) == 0) red[turn][0][threadIdx.x >> 5] = a, red[turn][1][threadIdx.x >> 5] = b;
      group_sync<NT, CT>(g);
      const int l = threadIdx.x & 31;
      a = warp_sum(l < NT / 32 ? red[turn][0][g * (NT / 32) + l] : 0.f);
      b = warp_sum(l < NT / 32 ? red[turn][1][g * (NT / 32) + l] : 0.f);
    }
    const f2 m1 = f2_of(-a * inv, -a * inv), m2 = f2_of(-b * inv, -b * inv);
    if constexpr (!HOLD) form(h, gg, false);
    // pass 2: rstd (g - mean(g) - h mean(g h)) + d_sum
#pragma unroll
    for (int j = 0; j < NP; ++j) h[j] = f2_add(f2_fma(h[j], m2, gg[j]), m1);
    if (ds) {
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          uint4 rs = make_uint4(0, 0, 0, 0);
          if (t + i * NT < nv) rs = *slot(at, 2, i);
#pragma unroll
          for (int c = 0; c < PP; ++c) h[i * PP + c] = f2_fma(h[i * PP + c], scale, f2_from16<X>(rs, c));
        }
      } else {
        load_scalar<X, NT, NP>(gg, ds + (size_t)row * p.d, t, p.d);
#pragma unroll
        for (int j = 0; j < NP; ++j) h[j] = f2_fma(h[j], scale, gg[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j) h[j] = f2_mul(h[j], scale);
    }
    store_cols<X, VEC, NT, NV>(static_cast<T *>(p.dx) + (size_t)row * p.d, h, t, p.d);
    fetch(row + p.stages * step, at);                // after the stage's last read
    at = at + 1 == p.stages ? 0 : at + 1;
  }
  if (!p.part) return;
  float *part = p.part + (size_t)blockIdx.x * 2 * p.d;
  auto each = [&](auto put) {                        // put(column, dweight, dbias)
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c0 = VEC ? (t + j / PP * NT) * V + j % PP * 2 : t + 2 * j * NT, c1 = VEC ? c0 + 1 : c0 + NT;
      const float2 fw = f2_get(dw[j]), fb = f2_get(db[j]);
      if (c0 < p.d) put(c0, fw.x, fb.x);
      if (c1 < p.d) put(c1, fw.y, fb.y);
    }
  };
  if constexpr (GROUPS == 1) {
    each([&](int c, float fw, float fb) { part[c] = fw, part[p.d + c] = fb; });
  } else {                                           // the CTA's groups one after another
    float *acc = reinterpret_cast<float *>(ring + (size_t)p.stages * p.stage_bytes);
    for (int k = 0; k < GROUPS; ++k) {
      if (g == k)
        each([&](int c, float fw, float fb) {
          acc[c] = (k ? acc[c] : 0.f) + fw;
          acc[p.d + c] = (k ? acc[p.d + c] : 0.f) + fb;
        });
      __syncthreads();
    }
    for (int j = threadIdx.x; j < 2 * p.d; j += blockDim.x) part[j] = acc[j];
  }
}

// Column sums of part [n, 2 d]: 32 columns a CTA, 8 row classes added in order.
__global__ void __launch_bounds__(256) k_norm_colsum(const float *part, int n, int d, float *dw, float *db) {
  __shared__ float red[8][32];
  griddep_wait();
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float s = 0.f;
  if (col < 2 * d)
#pragma unroll 4
    for (int i = r; i < n; i += 8) s += part[(size_t)i * 2 * d + col];
  red[r][c] = s;
  __syncthreads();
  if (r == 0 && col < 2 * d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][c];
    if (col < d) {
      if (dw) dw[col] = s;
    } else if (db) {
      db[col - d] = s;
    }
  }
}

// Stages of a ring in what a CTA may have of an SM's 224 KB: up to four forward.
// The gradient has three rows to copy for one and two stages do (30000 x 760
// binary32: 67 us, 95 with four, which leave L1 nothing).
constexpr size_t kRingMost = 224 * 1024;
int ring_stages(int stage_bytes, int ctas_per_sm, int most) { return std::max(1, std::min(most, 224 * 1024 / ctas_per_sm / stage_bytes)); }

template <int X, bool VEC, int NT, int NV, bool WREG>
cudaError_t launch_norm(NormParams p, cudaStream_t s) {
  constexpr int GROUPS = NT < 128 ? 128 / NT : 1, CT = NT * GROUPS, V = Cols<X, VEC, NT, NV>::V;
  const int per_sm = norm_ctas(NT, VEC);
  unsigned grid = (unsigned)((p.rows + GROUPS - 1) / GROUPS);
  p.stages = 1, p.stage_bytes = 0;
  size_t smem = 0;
  if (VEC) {
    grid = std::min(grid, (unsigned)(per_sm * std::max(1, pi::current_sms())));
    const int per_pack = 16 * (1 + (!p.add ? 0 : V * pi::dtype_size(p.add_dt) > 16 ? 2 : 1));
    p.stage_bytes = GROUPS * (p.d / V) * per_pack;
    p.stages = std::min(ring_stages(p.stage_bytes, per_sm, 4), (p.rows - 1) / (int)(grid * GROUPS) + 1);
    smem = (size_t)p.stages * p.stage_bytes;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = pi::allow_smem(k_norm<X, VEC, NT, NV, WREG>, smem, kRingMost, done);
    if (e != cudaSuccess) return e;
  }
  k_norm<X, VEC, NT, NV, WREG><<<grid, CT, smem, s>>>(p);
  return cudaGetLastError();
}

template <int X, bool VEC, int NT, int NV>
cudaError_t norm_by_weight(const NormParams &p, cudaStream_t s) {
  if constexpr (VEC)
    if (p.w_dt == X || (!p.w && !p.b)) return launch_norm<X, VEC, NT, NV, true>(p, s);
  return launch_norm<X, VEC, NT, NV, false>(p, s);
}

// Smallest group that holds a row.
template <int X, bool VEC, int NV>
cudaError_t norm_by_width(const NormParams &p, cudaStream_t s) {
  constexpr int C = 2 * Cols<X, VEC, 32, NV>::NP;    // columns of a thread
  if (p.d <= 32 * C) return norm_by_weight<X, VEC, 32, NV>(p, s);
  if (p.d <= 64 * C) return norm_by_weight<X, VEC, 64, NV>(p, s);
  if (p.d <= 128 * C) return norm_by_weight<X, VEC, 128, NV>(p, s);
  if (p.d <= 256 * C) return norm_by_weight<X, VEC, 256, NV>(p, s);
  if constexpr (1024 * C <= PI_MAX_D)                // (the caller has chosen NV such that a row fits)
    if (p.d > 512 * C) return norm_by_weight<X, VEC, 1024, NV>(p, s);
  return norm_by_weight<X, VEC, 512, NV>(p, s);
}

template <int X>
cudaError_t norm_by_type(const NormParams &p, bool vec, cudaStream_t s) {
  // plain loads: a warp a row while 16 columns a thread hold it (40000 x 301 bf16: 40 us,
  // 57 with two warps and 8 columns); wider rows 8 columns (30000 x 805: 56 us, 89 with 16)
  if (!vec) return p.d > 512 && p.d <= 4096 ? norm_by_width<X, false, 4>(p, s) : norm_by_width<X, false, 8>(p, s);
  return norm_by_width<X, true, 4>(p, s);
}

// Columns of the gradient kernel up to which a warp takes a row, and up to which
// half a CTA of 256 threads does, with 8 and with 16 columns a thread.
constexpr int kGradWarpD = 256, kGradHalfD = 1024, kGradHalfD16 = 2048;
// CTAs of the gradient kernel: a function of rows and d alone, because the order
// in which dweight's rows are added follows from it; as many as the GPU's 152 SMs hold.
int grad_ctas(int rows, int d) {
  const int groups = d <= kGradWarpD ? 8 : d <= kGradHalfD16 ? 2 : 1;
  return std::max(1, std::min((rows + groups - 1) / groups, 152 * (d <= kGradHalfD ? 3 : d <= 256 * 16 ? 2 : 1)));
}

template <int X, bool VEC, int NT, int COLS>
cudaError_t launch_grad(NormGradParams p, cudaStream_t s) {
  constexpr int CT = NT < 256 ? 256 : NT, GROUPS = CT / NT, V = 16 / (int)sizeof(typename Elem<X>::T), NV = VEC ? COLS * (int)sizeof(typename Elem<X>::T) / 16 : COLS / 2;
  const int grid = grad_ctas(p.rows, p.d);
  p.stages = 0, p.stage_bytes = 0;
  if (VEC) {
    p.stage_bytes = (p.dsum ? 3 : 2) * GROUPS * (p.d / V) * 16;
    p.stages = ring_stages(p.stage_bytes, grad_ctas_sm(NT, COLS), 2);
  }
  const size_t smem = (size_t)p.stages * p.stage_bytes + (GROUPS > 1 ? 2 * p.d * sizeof(float) : 0);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = pi::allow_smem(k_norm_grad<X, VEC, NT, NV>, smem, kRingMost, done);
  if (e != cudaSuccess) return e;
  k_norm_grad<X, VEC, NT, NV><<<grid, CT, smem, s>>>(p);
  return cudaGetLastError();
}

template <int X, bool VEC>
cudaError_t grad_by_width(const NormGradParams &p, cudaStream_t s) {
  // columns of a thread: 16 at most, two accumulators each
  if (p.d <= kGradWarpD) return launch_grad<X, VEC, 32, 8>(p, s);
  if (p.d <= kGradHalfD) return launch_grad<X, VEC, 128, 8>(p, s);
  if (p.d <= kGradHalfD16) return launch_grad<X, VEC, 128, 16>(p, s);
  if (p.d <= 256 * 16) return launch_grad<X, VEC, 256, 16>(p, s);
  if (p.d <= 512 * 16) return launch_grad<X, VEC, 512, 16>(p, s);
  return launch_grad<X, VEC, 1024, 16>(p, s);
}

template <int X>
cudaError_t grad_by_type(const NormGradParams &p, bool vec, cudaStream_t s) {
  return vec ? grad_by_width<X, true>(p, s) : grad_by_width<X, false>(p, s);
}

pi_status check_shape(int rows, int d, int dtype, int64_t x_stride) {
  if (rows < 0) return pi::fail(PI_ERR_INVALID_ARG, "rows=%d is negative", rows);
  if (d < 1 || d > PI_MAX_D) return pi::fail(PI_ERR_UNSUPPORTED, "d=%d outside [1, %d]", d, PI_MAX_D);
  if (!pi::dtype_ok(dtype)) return pi::fail(PI_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (rows > 1 && x_stride < d) return pi::fail(PI_ERR_INVALID_ARG, "x_stride is less than d=%d", d);
  return PI_OK;
}

}  // namespace

extern "C" {

pi_status pi_layer_norm(const void *x, int64_t x_stride, const void *add, int32_t add_dtype, const void *weight,
                        const void *bias, int32_t w_dtype, int32_t rows, int32_t d, int32_t dtype, float eps, void *y,
                        void *sum, float *mean, float *rstd, void *stream) {
  pi::clear_error();
  pi_status st = check_shape(rows, d, dtype, x_stride);
  if (st != PI_OK) return st;
  if ((add && !pi::dtype_ok(add_dtype)) || ((weight || bias) && !pi::dtype_ok(w_dtype)))
    return pi::fail(PI_ERR_INVALID_ARG, "unknown add_dtype %d or w_dtype %d", add_dtype, w_dtype);
  if (!(eps >= 0.f)) return pi::fail(PI_ERR_INVALID_ARG, "eps must be 0 or more");
  if ((add != nullptr) != (sum != nullptr)) return pi::fail(PI_ERR_INVALID_ARG, "add and sum go together");
  if (rows == 0) return PI_OK;
  const int e = pi::dtype_size(dtype);
  if (!x || !y || !pi::aligned_to(x, e) || !pi::aligned_to(y, e) || !pi::aligned_to(sum, e))
    return pi::fail(PI_ERR_INVALID_ARG, "x and y must be non-NULL, x, y and sum aligned to their type");
  if ((add && !pi::aligned_to(add, pi::dtype_size(add_dtype))) ||
      ((weight || bias) && (!pi::aligned_to(weight, pi::dtype_size(w_dtype)) || !pi::aligned_to(bias, pi::dtype_size(w_dtype)))))
    return pi::fail(PI_ERR_INVALID_ARG, "add, weight and bias must be aligned to their type");
  if (!pi::aligned_to(mean, 4) || !pi::aligned_to(rstd, 4))
    return pi::fail(PI_ERR_INVALID_ARG, "mean and rstd must be 4-byte aligned");
  if (sum == x && rows > 1 && x_stride != d) return pi::fail(PI_ERR_INVALID_ARG, "sum may be x only where x is contiguous");
  const int V = 16 / e;
  const bool vec = d % V == 0 && (rows == 1 || x_stride % V == 0) && pi::aligned_to(x, 16) && pi::aligned_to(y, 16) &&
                   pi::aligned_to(sum, 16) && pi::aligned_to(add, 16) && pi::aligned_to(weight, 16) &&
                   pi::aligned_to(bias, 16);
  const NormParams p{x, add, weight, bias, y, sum, mean, rstd, x_stride, rows, d, add_dtype, w_dtype, eps};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PI_TRY_CUDA(dtype == PI_DT_F16    ? norm_by_type<PI_DT_F16>(p, vec, s)
              : dtype == PI_DT_BF16 ? norm_by_type<PI_DT_BF16>(p, vec, s)
                                    : norm_by_type<PI_DT_F32>(p, vec, s));
  return PI_OK;
}

size_t pi_layer_norm_backward_workspace_bytes(int32_t rows, int32_t d) {
  if (rows < 0 || d < 1 || d > PI_MAX_D) return 0;
  return sizeof(float) * 2 * (size_t)d * (size_t)grad_ctas(rows, d);
}

pi_status pi_layer_norm_backward(const void *dy, const void *x, int64_t x_stride, const void *weight, int32_t w_dtype,
                                 const float *mean, const float *rstd, const void *d_sum, int32_t rows, int32_t d,
                                 int32_t dtype, void *dx, float *dweight, float *dbias, void *ws, size_t ws_bytes,
                                 void *stream) {
  pi::clear_error();
  pi_status st = check_shape(rows, d, dtype, x_stride);
  if (st != PI_OK) return st;
  if (weight && !pi::dtype_ok(w_dtype)) return pi::fail(PI_ERR_INVALID_ARG, "unknown w_dtype %d", w_dtype);
  if (!pi::aligned_to(dweight, 4) || !pi::aligned_to(dbias, 4))
    return pi::fail(PI_ERR_INVALID_ARG, "dweight and dbias must be 4-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dweight) PI_TRY_CUDA(cudaMemsetAsync(dweight, 0, sizeof(float) * d, s));
    if (dbias) PI_TRY_CUDA(cudaMemsetAsync(dbias, 0, sizeof(float) * d, s));
    return PI_OK;
  }
  const int e = pi::dtype_size(dtype);
  if (!dy || !x || !dx || !pi::aligned_to(dy, e) || !pi::aligned_to(x, e) || !pi::aligned_to(dx, e) ||
      !pi::aligned_to(d_sum, e))
    return pi::fail(PI_ERR_INVALID_ARG, "dy, x and dx must be non-NULL, dy, x, dx and d_sum aligned to their type");
  if (!mean || !rstd || !pi::aligned_to(mean, 4) || !pi::aligned_to(rstd, 4))
    return pi::fail(PI_ERR_INVALID_ARG, "mean and rstd must be non-NULL and 4-byte aligned");
  if (weight && !pi::aligned_to(weight, pi::dtype_size(w_dtype)))
    return pi::fail(PI_ERR_INVALID_ARG, "weight must be aligned to its type");
  const bool want = dweight || dbias;
  if (want && (!ws || !pi::aligned_to(ws, 16) || ws_bytes < pi_layer_norm_backward_workspace_bytes(rows, d)))
    return pi::fail(PI_ERR_INVALID_ARG, "ws must be 16-byte aligned and hold %zu bytes, has %zu",
                    pi_layer_norm_backward_workspace_bytes(rows, d), ws_bytes);
  const int V = 16 / e;
  const bool vec = d % V == 0 && (rows == 1 || x_stride % V == 0) && pi::aligned_to(dy, 16) && pi::aligned_to(x, 16) &&
                   pi::aligned_to(dx, 16) && pi::aligned_to(d_sum, 16) && pi::aligned_to(weight, 16);
  float *part = want ? static_cast<float *>(ws) : nullptr;
  const NormGradParams p{dy, x, weight, d_sum, mean, rstd, dx, part, x_stride, rows, d, w_dtype};
  PI_TRY_CUDA(dtype == PI_DT_F16    ? grad_by_type<PI_DT_F16>(p, vec, s)
              : dtype == PI_DT_BF16 ? grad_by_type<PI_DT_BF16>(p, vec, s)
                                    : grad_by_type<PI_DT_F32>(p, vec, s));
  if (want) {
    PI_TRY_CUDA(pi::launch_pdl(k_norm_colsum, dim3((unsigned)(2 * d + 31) / 32), dim3(256), 0, s, part, grad_ctas(rows, d), d, dweight, dbias));
  }
  return PI_OK;
}

}  // extern "C"
