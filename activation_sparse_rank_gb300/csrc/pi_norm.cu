// Layer norm, forward (with an optional addition before it) and backward.
//
//   y  = (t - mean) rstd w + b          t = x, or the stored sum x + add
//   dx = rstd (g - mean_j(g) - h mean_j(g h)) + d_sum,  h = (t - mean) rstd, g = dy w
//   dw = sum_rows dy h,  db = sum_rows dy
//
// Bound by HBM: a handful of operations per element read.  A row is read once
// and stays in registers between its reductions, so the variance is the mean
// square about the mean (no cancellation) at no extra traffic.
#include "pi_ops.cuh"

#include <algorithm>

using namespace pidev;

namespace {

// N consecutive elements of a tensor whose type is a run-time value, as
// binary32.  For N > 1 the address is a multiple of 4 elements and the base
// 16-byte aligned.
template <int N>
__device__ __forceinline__ void load_n(float *o, const void *p, int dt, size_t i) {
  if constexpr (N == 1) {
    o[0] = load_any(p, dt, i);
  } else if (dt == PI_DT_F32) {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + c);
      o[c] = f.x, o[c + 1] = f.y, o[c + 2] = f.z, o[c + 3] = f.w;
    }
  } else if (dt == PI_DT_F16) {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const Pack<PI_DT_F16, 4> f = *reinterpret_cast<const Pack<PI_DT_F16, 4> *>(static_cast<const __half *>(p) + i + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c + e] = __half2float(f.v[e]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const Pack<PI_DT_BF16, 4> f =
          *reinterpret_cast<const Pack<PI_DT_BF16, 4> *>(static_cast<const __nv_bfloat16 *>(p) + i + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c + e] = __bfloat162float(f.v[e]);
    }
  }
}

struct NormParams {
  const void *x, *add, *w, *b;
  void *y, *sum;
  float *mean, *rstd;
  int64_t x_stride;
  int rows, d, add_dt, w_dt;
  float eps;
};

// One row for each group of NT threads (NT == 32: four rows a CTA, no CTA
// barrier); thread t of the group holds the NV packs t, t + NT, ... of V elements.
template <int X, int V, int NT, int NV>
__global__ void __launch_bounds__(NT < 128 ? 128 : NT) k_norm(const NormParams p) {
  using P = Pack<X, V>;
  using E = Elem<X>;
  constexpr int GROUPS = NT < 128 ? 128 / NT : 1;
  __shared__ float red[2][32];
  const int t = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * GROUPS + threadIdx.x / NT;
  if (row >= p.rows) return;
  const int nv = p.d / V;
  const typename E::T *x = static_cast<const typename E::T *>(p.x) + row * p.x_stride;
  P raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (t + i * NT < nv) raw[i] = reinterpret_cast<const P *>(x)[t + i * NT];
  float v[NV][V];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = t + i * NT < nv;
    if (in && p.add) {
      float a[V];
      const size_t at = (size_t)row * p.d + (size_t)(t + i * NT) * V;
      load_n<V>(a, p.add, p.add_dt, at);
#pragma unroll
      for (int e = 0; e < V; ++e) raw[i].v[e] = E::from(E::to(raw[i].v[e]) + a[e]);
      *reinterpret_cast<P *>(static_cast<typename E::T *>(p.sum) + at) = raw[i];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      v[i][e] = in ? E::to(raw[i].v[e]) : 0.f;
      s += v[i][e];
    }
  }
  const float mean = cta_sum<NT>(s, red[0]) / (float)p.d;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      v[i][e] -= mean;
      if (t + i * NT < nv) q = fmaf(v[i][e], v[i][e], q);
    }
  const float rstd = 1.0f / sqrtf(cta_sum<NT>(q, red[1]) / (float)p.d + p.eps);
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  typename E::T *y = static_cast<typename E::T *>(p.y) + (size_t)row * p.d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int k = t + i * NT;
    if (k >= nv) continue;
    float w[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = 1.f, b[e] = 0.f;
    if (p.w) load_n<V>(w, p.w, p.w_dt, (size_t)k * V);
    if (p.b) load_n<V>(b, p.b, p.w_dt, (size_t)k * V);
    P o;
#pragma unroll
    for (int e = 0; e < V; ++e) o.v[e] = E::from(fmaf(v[i][e] * rstd, w[e], b[e]));
    reinterpret_cast<P *>(y)[k] = o;
  }
}

struct NormGradParams {
  const void *dy, *x, *w, *dsum;
  const float *mean, *rstd;
  void *dx;
  float *part;          // [groups, 2, d]: dweight, dbias over the rows of one CTA
  int64_t x_stride;
  int rows, d, w_dt;
};

// Each group of NT threads takes the rows g, g + groups, ...; a thread keeps
// its columns over all of them, so dweight and dbias add up in its registers.
template <int X, int V, int NT, int NV>
__global__ void __launch_bounds__(NT < 128 ? 128 : NT) k_norm_grad(const NormGradParams p) {
  using P = Pack<X, V>;
  using E = Elem<X>;
  constexpr int GROUPS = NT < 128 ? 128 / NT : 1;
  __shared__ float red[2][2][32];
  extern __shared__ float acc[];                     // GROUPS > 1: [2, d]
  const int t = threadIdx.x % NT, g = threadIdx.x / NT;
  const int nv = p.d / V;
  const float inv = 1.0f / (float)p.d;
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[i][e] = 0.f, db[i][e] = 0.f;

  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * GROUPS + g; row < p.rows; row += (int64_t)gridDim.x * GROUPS, turn ^= 1) {
    const typename E::T *x = static_cast<const typename E::T *>(p.x) + row * p.x_stride;
    const typename E::T *dy = static_cast<const typename E::T *>(p.dy) + row * p.d;
    const typename E::T *ds = static_cast<const typename E::T *>(p.dsum) + row * p.d;
    P rx[NV], ry[NV], rs[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = t + i * NT;
      if (k < nv) {
        rx[i] = reinterpret_cast<const P *>(x)[k];
        ry[i] = reinterpret_cast<const P *>(dy)[k];
        if (p.dsum) rs[i] = reinterpret_cast<const P *>(ds)[k];
      }
    }
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = t + i * NT;
      if (k >= nv) continue;
      float w[V];
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = 1.f;
      if (p.w) load_n<V>(w, p.w, p.w_dt, (size_t)k * V);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float h = (E::to(rx[i].v[e]) - mean) * rstd, y = E::to(ry[i].v[e]);
        dw[i][e] = fmaf(y, h, dw[i][e]);
        db[i][e] += y;
        s1 = fmaf(y, w[e], s1);
        s2 = fmaf(y * w[e], h, s2);
      }
    }
    if constexpr (NT == 32) {
      s1 = warp_sum(s1), s2 = warp_sum(s2);
    } else {
      s1 = warp_sum(s1), s2 = warp_sum(s2);
      if ((threadIdx.x & 31) == 0) red[turn][0][threadIdx.x >> 5] = s1, red[turn][1][threadIdx.x >> 5] = s2;
      __syncthreads();
      const int l = threadIdx.x & 31;
      s1 = warp_sum(l < NT / 32 ? red[turn][0][l] : 0.f);
      s2 = warp_sum(l < NT / 32 ? red[turn][1][l] : 0.f);
    }
    s1 *= inv, s2 *= inv;
    typename E::T *dx = static_cast<typename E::T *>(p.dx) + row * p.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = t + i * NT;
      if (k >= nv) continue;
      float w[V];
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = 1.f;
      if (p.w) load_n<V>(w, p.w, p.w_dt, (size_t)k * V);
      P o;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float h = (E::to(rx[i].v[e]) - mean) * rstd;
        float r = rstd * (E::to(ry[i].v[e]) * w[e] - s1 - h * s2);
        if (p.dsum) r += E::to(rs[i].v[e]);
        o.v[e] = E::from(r);
      }
      reinterpret_cast<P *>(dx)[k] = o;
    }
  }
  if (!p.part) return;
  float *part = p.part + (size_t)blockIdx.x * 2 * p.d;
  if constexpr (GROUPS == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = t + i * NT;
      if (k >= nv) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) part[k * V + e] = dw[i][e], part[p.d + k * V + e] = db[i][e];
    }
  } else {                                           // the CTA's groups one after another
    for (int turn_g = 0; turn_g < GROUPS; ++turn_g) {
      if (g == turn_g) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int k = t + i * NT;
          if (k >= nv) continue;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            float &a = acc[k * V + e], &b = acc[p.d + k * V + e];
            a = (turn_g ? a : 0.f) + dw[i][e];
            b = (turn_g ? b : 0.f) + db[i][e];
          }
        }
      }
      __syncthreads();
    }
    for (int j = threadIdx.x; j < 2 * p.d; j += blockDim.x) part[j] = acc[j];
  }
}

// Column sums of part [n, 2 d]: 32 columns a CTA, 8 row classes added in order.
__global__ void __launch_bounds__(256) k_norm_colsum(const float *__restrict__ part, int n, int d, float *dw, float *db) {
  __shared__ float red[8][32];
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

template <int X, int V, int NT, int NV>
cudaError_t launch_norm(const NormParams &p, cudaStream_t s) {
  constexpr int GROUPS = NT < 128 ? 128 / NT : 1;
  k_norm<X, V, NT, NV><<<(p.rows + GROUPS - 1) / GROUPS, NT < 128 ? 128 : NT, 0, s>>>(p);
  return cudaGetLastError();
}

// Smallest group that holds a row: C elements a thread.
template <int X, int V, int C>
cudaError_t norm_by_width(const NormParams &p, cudaStream_t s) {
  if (p.d <= 32 * C) return launch_norm<X, V, 32, C / V>(p, s);
  if (p.d <= 128 * C) return launch_norm<X, V, 128, C / V>(p, s);
  if (p.d <= 256 * C) return launch_norm<X, V, 256, C / V>(p, s);
  if (p.d <= 512 * C) return launch_norm<X, V, 512, C / V>(p, s);
  return launch_norm<X, V, 1024, C / V>(p, s);
}

template <int X>
cudaError_t norm_by_type(const NormParams &p, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(typename Elem<X>::T);
  return vec ? norm_by_width<X, V, 16>(p, s) : norm_by_width<X, 1, 16>(p, s);
}

// CTAs of the gradient kernel: a function of rows and d alone, because the
// order in which dweight's rows are added follows from it.
constexpr int kGradCtas = 304;
int grad_ctas(int rows, int d) {
  const int groups = d <= 512 ? 4 : 1;
  return std::max(1, std::min((rows + groups - 1) / groups, kGradCtas));
}

template <int X, int V, int NT, int NV>
cudaError_t launch_grad(const NormGradParams &p, cudaStream_t s) {
  k_norm_grad<X, V, NT, NV><<<grad_ctas(p.rows, p.d), NT < 128 ? 128 : NT, NT < 128 ? 2 * p.d * sizeof(float) : 0, s>>>(p);
  return cudaGetLastError();
}

template <int X, int V, int C>
cudaError_t grad_by_width(const NormGradParams &p, cudaStream_t s) {
  if (p.d <= 32 * C) return launch_grad<X, V, 32, C / V>(p, s);
  if (p.d <= 128 * C) return launch_grad<X, V, 128, C / V>(p, s);
  if (p.d <= 256 * C) return launch_grad<X, V, 256, C / V>(p, s);
  if (p.d <= 512 * C) return launch_grad<X, V, 512, C / V>(p, s);
  return launch_grad<X, V, 1024, C / V>(p, s);
}

template <int X>
cudaError_t grad_by_type(const NormGradParams &p, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(typename Elem<X>::T);
  return vec ? grad_by_width<X, V, 16>(p, s) : grad_by_width<X, 1, 16>(p, s);
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
    k_norm_colsum<<<(2 * d + 31) / 32, 256, 0, s>>>(part, grad_ctas(rows, d), d, dweight, dbias);
    PI_TRY_CUDA(cudaGetLastError());
  }
  return PI_OK;
}

}  // extern "C"
