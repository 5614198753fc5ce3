// Rotary positions: queries and keys turned by the angles of their positions.
//
// A copy with arithmetic: bound by HBM for a prompt, by one load's latency for the
// single tokens of a decode step.  The angles of a token are the same for all of
// its heads, so a CTA takes whole tokens (or many heads of one), computes their
// cosines and sines once, into shared memory, while its first rows are on their
// way, and every thread then turns units of two vectors, one access each.
#include "pi_rope.cuh"

#include <algorithm>

using namespace pidev;

namespace {

constexpr int kThreads = 256;
constexpr int kMostTokens = 32;     // of a CTA

struct RotaryParams {
  pi_rotary r;
  const int32_t *pos;
  const void *x;
  void *y;
  int64_t xt, xh, yt, yh;
  int tokens, heads, dim;
  int per_tokens, per_heads;        // of a CTA
  int copy;                         // elements past the turned ones are copied
  float sign;
};

// V: elements of a vector; units of two of them, V pairs.
template <int DT, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) k_rotary(const RotaryParams p) {
  using E = Elem<DT>;
  using T = typename E::T;
  extern __shared__ float4 table[];                  // [tokens of the CTA][max(1, V / 2)][units]
  constexpr int CHUNKS = V >= 2 ? V / 2 : 1;
  const int t0 = blockIdx.x * p.per_tokens, nt = min(p.per_tokens, p.tokens - t0);
  const int h0 = blockIdx.y * p.per_heads, nh = min(p.per_heads, p.heads - h0);
  const int units = p.r.dim / (2 * V), n = nt * nh * units;
  const T *x = static_cast<const T *>(p.x) + t0 * p.xt + h0 * p.xh;
  T *y = static_cast<T *>(p.y) + t0 * p.yt + h0 * p.yh;

  struct Unit {
    int t, h, j;
    Pack<DT, V> a, b;
  };
  auto ia = [&](int j) { return HALF ? j * V : 2 * j * V; };
  auto ib = [&](int j) { return HALF ? p.r.dim / 2 + j * V : 2 * j * V + V; };
  auto load = [&](Unit &u, int i) {
    if (i >= n) return;
    u.j = i % units;
    const int r = i / units;
    u.h = r % nh, u.t = r / nh;
    const T *row = x + u.t * p.xt + u.h * p.xh;
    u.a = *reinterpret_cast<const Pack<DT, V> *>(row + ia(u.j));
    u.b = *reinterpret_cast<const Pack<DT, V> *>(row + ib(u.j));
  };
  auto turn = [&](const Unit &u, int i) {
    if (i >= n) return;
    T *row = y + u.t * p.yt + u.h * p.yh;
    Pack<DT, V> a, b;
    if constexpr (V == 1) {
      const float2 cs = reinterpret_cast<const float2 *>(table)[u.t * units + u.j];
      const float xa = E::to(u.a.v[0]), xb = E::to(u.b.v[0]);
      a.v[0] = E::from(fmaf(xa, cs.x, -cs.y * xb)), b.v[0] = E::from(fmaf(xa, cs.y, cs.x * xb));
    } else {
      f2 v[V];
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        v[k] = f2_of(E::to(u.a.v[2 * k]), E::to(u.a.v[2 * k + 1]));
        v[V / 2 + k] = f2_of(E::to(u.b.v[2 * k]), E::to(u.b.v[2 * k + 1]));
      }
      rope_turn<V, HALF>(v, table + (int64_t)u.t * CHUNKS * units + u.j, units);
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        a.v[2 * k] = E::from(v[k].x), a.v[2 * k + 1] = E::from(v[k].y);
        b.v[2 * k] = E::from(v[V / 2 + k].x), b.v[2 * k + 1] = E::from(v[V / 2 + k].y);
      }
    }
    *reinterpret_cast<Pack<DT, V> *>(row + ia(u.j)) = a;
    *reinterpret_cast<Pack<DT, V> *>(row + ib(u.j)) = b;
  };

  Unit u0, u1;
  load(u0, threadIdx.x), load(u1, threadIdx.x + kThreads);
  const int freqs = p.r.dim / 2;
  for (int i = threadIdx.x; i < nt * freqs; i += kThreads) {
    const int t = i / freqs, f = i % freqs;
    float2 cs = rope_angle(p.r.turns[f], p.pos[t0 + t], p.r.magnitude);
    cs.y *= p.sign;
    if constexpr (V == 1) reinterpret_cast<float2 *>(table)[t * units + f] = cs;
    else rope_put<V>(table + t * CHUNKS * units, units, f, cs);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 2 * kThreads) {
    turn(u0, i), turn(u1, i + kThreads);
    load(u0, i + 2 * kThreads), load(u1, i + 3 * kThreads);
  }
  if (p.copy) {
    const int rest = (p.dim - p.r.dim) / V, m = nt * nh * rest;
    for (int i = threadIdx.x; i < m; i += kThreads) {
      const int j = i % rest, r = i / rest, h = r % nh, t = r / nh;
      *reinterpret_cast<Pack<DT, V> *>(y + t * p.yt + h * p.yh + p.r.dim + j * V) =
          *reinterpret_cast<const Pack<DT, V> *>(x + t * p.xt + h * p.xh + p.r.dim + j * V);
    }
  }
}

template <int DT, int V>
cudaError_t launch(RotaryParams p, cudaStream_t s) {
  // about four units a thread where there is enough work to fill the SMs, else one
  const int64_t units = p.r.dim / (2 * V), row = p.heads * units, all = row * p.tokens;
  const int64_t want = kThreads * std::max<int64_t>(1, std::min<int64_t>(4, all / (kThreads * 8 * (int64_t)std::max(1, pi::current_sms()))));
  p.per_tokens = (int)std::max<int64_t>(1, std::min<int64_t>(kMostTokens, want / std::max<int64_t>(1, row)));
  const int64_t parts = std::min<int64_t>(p.heads, std::max<int64_t>(1, row / want));
  p.per_heads = (int)((p.heads + parts - 1) / parts);
  const dim3 grid((p.tokens + p.per_tokens - 1) / p.per_tokens, (p.heads + p.per_heads - 1) / p.per_heads);
  const size_t smem = (size_t)p.per_tokens * p.r.dim / 2 * sizeof(float2);
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = p.r.interleaved ? pi::allow_smem(k_rotary<DT, V, false>, smem, kMostTokens * PI_MAX_ROTARY / 2 * sizeof(float2), done[0])
                                        : pi::allow_smem(k_rotary<DT, V, true>, smem, kMostTokens * PI_MAX_ROTARY / 2 * sizeof(float2), done[1]);
  if (e != cudaSuccess) return e;
  if (p.r.interleaved)
    k_rotary<DT, V, false><<<grid, kThreads, smem, s>>>(p);
  else
    k_rotary<DT, V, true><<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int DT>
cudaError_t by_vector(const RotaryParams &p, int v, cudaStream_t s) {
  if constexpr (DT != PI_DT_F32)
    if (v == 8) return launch<DT, 8>(p, s);
  return v >= 4 ? launch<DT, 4>(p, s) : launch<DT, 1>(p, s);
}

}  // namespace

namespace pi {

pi_status check_rotary(const pi_rotary *r, int head_dim) {
  if (!r) return fail(PI_ERR_INVALID_ARG, "rotary is NULL");
  if (r->dim < 2 || r->dim % 2 || r->dim > PI_MAX_ROTARY)
    return fail(PI_ERR_UNSUPPORTED, "rotary dim=%d: an even number up to %d", r->dim, PI_MAX_ROTARY);
  if (r->dim > head_dim) return fail(PI_ERR_INVALID_ARG, "rotary dim=%d is above head_dim=%d", r->dim, head_dim);
  if (!(fabsf(r->magnitude) < INFINITY)) return fail(PI_ERR_INVALID_ARG, "magnitude must be finite");
  if (!r->turns || !aligned_to(r->turns, 8)) return fail(PI_ERR_INVALID_ARG, "turns must be non-NULL and 8-byte aligned");
  return PI_OK;
}

}  // namespace pi

extern "C" pi_status pi_rotary_apply(const pi_rotary *rotary, const int32_t *positions, int32_t n_tokens, int32_t heads,
                                     int32_t head_dim, const void *x, const int64_t *x_stride, void *y,
                                     const int64_t *y_stride, int32_t dtype, int32_t inverse, void *stream) {
  pi::clear_error();
  const pi_status st = pi::check_rotary(rotary, head_dim);
  if (st != PI_OK) return st;
  if (!pi::dtype_ok(dtype)) return pi::fail(PI_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (n_tokens < 0 || n_tokens > (1 << 28) || heads < 1 || heads > 65535 || head_dim > PI_MAX_D)
    return pi::fail(PI_ERR_INVALID_ARG, "n_tokens=%d, heads=%d or head_dim=%d out of range", n_tokens, heads, head_dim);
  if (n_tokens == 0) return PI_OK;
  const int e = pi::dtype_size(dtype);
  if (!x || !y || !x_stride || !y_stride || !positions || !pi::aligned_to(x, e) || !pi::aligned_to(y, e) ||
      !pi::aligned_to(positions, 4))
    return pi::fail(PI_ERR_INVALID_ARG, "x, y, their strides and positions must be non-NULL and aligned to their type");
  int64_t all = reinterpret_cast<uintptr_t>(x) / e | reinterpret_cast<uintptr_t>(y) / e;     // elements: what divides it divides every offset
  for (int i = 0; i < 2; ++i) {
    if (x_stride[i] < 0 || y_stride[i] < 0) return pi::fail(PI_ERR_INVALID_ARG, "strides must not be negative");
    all |= x_stride[i] | y_stride[i];
  }
  all |= rotary->dim / 2;                           // where the second vectors are, and whole units of neighbours
  const bool same = x == y && x_stride[0] == y_stride[0] && x_stride[1] == y_stride[1];
  if (!same) all |= head_dim;
  // vectors of 16 bytes where everything is a multiple of them, else of 8 bytes for 16-bit types, else single elements
  const int v = e == 2 && all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 1;
  const RotaryParams p{*rotary, positions, x, y, x_stride[0], x_stride[1], y_stride[0], y_stride[1], n_tokens, heads, head_dim,
                       1, heads, !same && head_dim > rotary->dim, inverse ? -1.f : 1.f};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PI_TRY_CUDA(dtype == PI_DT_F16    ? by_vector<PI_DT_F16>(p, v, s)
              : dtype == PI_DT_BF16 ? by_vector<PI_DT_BF16>(p, v, s)
                                    : by_vector<PI_DT_F32>(p, v, s));
  return PI_OK;
}
