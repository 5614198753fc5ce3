// Rotary positions: queries and keys turned by the angles of their positions.
//
// A copy with arithmetic: bound by HBM for a prompt, by one load's latency for the
// single tokens of a decode step.  The angles of a token are the same for all of
// its heads, so a CTA takes whole tokens (or many heads of one), computes their
// cosines and sines once, into shared memory, while its first rows are on their
// way, and every thread then turns units of two vectors, one access each, at one place
// of several heads.
//
// Measured: 16001 tokens x 72 heads of 128 bf16 out of a packed projection 88 us (6.7 TB/s,
// 99% of the copy rate; binary32 173 us); 40 heads of 32 tokens 2.1 us; 100000 tokens of one head 37 us: there
// the angles, one for two elements with a division and two loads each, take the time.
#include "pi_rope.cuh"

#include <algorithm>

using namespace pidev;

namespace {

constexpr int kMostThreads = 512;
constexpr int kMostTokens = 32;     // of a CTA
constexpr int kMostDim = 2 * kMostThreads;       // a row's units, of single elements, are a CTA's threads at most

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

// V elements as one access.
template <int DT, int V>
struct alignas(V * sizeof(typename Elem<DT>::T)) Vec {
  static constexpr int WORDS = V * (int)sizeof(typename Elem<DT>::T) / 4;
  unsigned w[WORDS];
  __device__ __forceinline__ f2 get(int k) const {   // elements 2 k and 2 k + 1
    if constexpr (DT == PI_DT_F32) return f2_of(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
    else return f2_widen<DT>(w[k]);
  }
  __device__ __forceinline__ void set(int k, f2 v) {
    if constexpr (DT == PI_DT_F32) w[2 * k] = __float_as_uint(v.x), w[2 * k + 1] = __float_as_uint(v.y);
    else w[k] = f2_narrow<DT>(v);
  }
};

// A thread has unit j (two vectors of V elements, V pairs) of every `step`-th row of the
// CTA's tokens x heads.
template <int DT, int V, bool HALF>
__global__ void __launch_bounds__(kMostThreads, 3) k_rotary(const RotaryParams p) {
  using E = Elem<DT>;
  using T = typename E::T;
  extern __shared__ float4 table[];                  // [tokens of the CTA][max(1, V / 2)][units]
  constexpr int CHUNKS = V >= 2 ? V / 2 : 1;
  const int t0 = blockIdx.x * p.per_tokens, nt = min(p.per_tokens, p.tokens - t0);
  const int h0 = blockIdx.y * p.per_heads, nh = min(p.per_heads, p.heads - h0);
  const int units = p.r.dim / (2 * V), all = p.copy ? (p.dim + 2 * V - 1) / (2 * V) : units;    // of a row: turned, and with copied ones
  const int step = blockDim.x / all, rows = nt * nh;
  const int j = threadIdx.x % all, first = threadIdx.x < step * all ? threadIdx.x / all : rows;
  const T *x = static_cast<const T *>(p.x) + t0 * p.xt + h0 * p.xh;
  T *y = static_cast<T *>(p.y) + t0 * p.yt + h0 * p.yh;
  const bool turned = j < units;
  const int ia = HALF && turned ? j * V : 2 * j * V, ib = HALF && turned ? p.r.dim / 2 + j * V : ia + V;

  auto fill = [&] {
    const int freqs = p.r.dim / 2;
    for (int i = threadIdx.x; i < nt * freqs; i += blockDim.x) {
      const int t = i / freqs, f = i - t * freqs;
      float2 cs = rope_angle(p.r.turns[f], p.pos[t0 + t], p.r.magnitude);
      cs.y *= p.sign;
      if constexpr (V == 1) reinterpret_cast<float2 *>(table)[t * units + f] = cs;
      else rope_put<V>(table + t * CHUNKS * units, units, f, cs);
    }
    __syncthreads();
  };
  if constexpr (V == 1) {
    fill();
    for (int r = first; r < rows; r += step) {
      const int t = r / nh, h = r - t * nh;
      const float2 cs = turned ? reinterpret_cast<const float2 *>(table)[t * units + j] : make_float2(1.f, 0.f);
      const T *in = x + t * p.xt + h * p.xh;
      T *out = y + t * p.yt + h * p.yh;
      if (ib >= p.dim) {                             // the last element of an odd number
        out[ia] = in[ia];
        continue;
      }
      const T c = in[ia], d = in[ib];
      const float a = E::to(c), b = E::to(d);
      out[ia] = turned ? E::from(fmaf(a, cs.x, -cs.y * b)) : c, out[ib] = turned ? E::from(fmaf(a, cs.y, cs.x * b)) : d;
    }
  } else {
    using Pair = Vec<DT, V>;
    const bool one = nt == 1;                        // rows are heads
    auto row_of = [&](int r, int64_t st, int64_t sh) {
      if (one) return r * sh;
      const int t = r / nh;
      return t * st + (r - t * nh) * sh;
    };
    auto load = [&](int r, Pair &a, Pair &b) {
      if (r >= rows) return;
      const T *in = x + row_of(r, p.xt, p.xh);
      a = *reinterpret_cast<const Pair *>(in + ia), b = *reinterpret_cast<const Pair *>(in + ib);
    };
    auto turn = [&](int r, Pair &a, Pair &b) {
      if (r >= rows) return;
      if (turned) {
        f2 v[V];
#pragma unroll
        for (int k = 0; k < V / 2; ++k) v[k] = a.get(k), v[V / 2 + k] = b.get(k);
        rope_turn<V, HALF>(v, table + (one ? 0 : r / nh) * CHUNKS * units + j, units);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) a.set(k, v[k]), b.set(k, v[V / 2 + k]);
      }
      T *out = y + row_of(r, p.yt, p.yh);
      *reinterpret_cast<Pair *>(out + ia) = a, *reinterpret_cast<Pair *>(out + ib) = b;
    };
    Pair a0, b0, a1, b1;
    load(first, a0, b0), load(first + step, a1, b1);
    fill();
    for (int r = first; r < rows; r += 2 * step) {
      turn(r, a0, b0), turn(r + step, a1, b1);
      load(r + 2 * step, a0, b0), load(r + 3 * step, a1, b1);
    }
  }
}

template <int DT, int V>
cudaError_t launch(RotaryParams p, cudaStream_t s) {
  // About three units a thread, of which two are loaded before the angles are computed, in CTAs of
  // about 128 threads: of one token's heads, of small tokens several, more heads take several CTAs
  // (8190 tokens x 71 heads of 64, 16 turned: 26 us; with 512 threads and two units 33.  16001 x 72 x
  // 128: 89 and 86).  Little work in all: one unit a thread, in small CTAs.
  const int64_t units = ((p.copy ? p.dim : p.r.dim) + 2 * V - 1) / (2 * V), all = (int64_t)p.heads * units * p.tokens;
  const bool few = all < (int64_t)1024 * std::max(1, pi::current_sms());
  const int64_t most = std::max<int64_t>(1, (few ? 64 : 128) / units), each = few ? 1 : 3;     // rows at once, in turn
  p.per_tokens = (int)std::max<int64_t>(1, std::min<int64_t>(kMostTokens, most * each / p.heads));
  const int64_t parts = std::min<int64_t>(p.heads, (p.heads + most * each - 1) / (most * each));
  p.per_heads = (int)((p.heads + parts - 1) / parts);
  const dim3 grid((p.tokens + p.per_tokens - 1) / p.per_tokens, (p.heads + p.per_heads - 1) / p.per_heads);
  const int64_t rows = std::min(most, ((int64_t)p.per_tokens * p.per_heads + each - 1) / each);
  const int threads = (int)((std::max<int64_t>(rows * units, 64) + 31) / 32 * 32);
  const size_t smem = (size_t)p.per_tokens * p.r.dim / 2 * sizeof(float2);
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = p.r.interleaved ? pi::allow_smem(k_rotary<DT, V, false>, smem, kMostTokens * PI_MAX_ROTARY / 2 * sizeof(float2), done[0])
                                        : pi::allow_smem(k_rotary<DT, V, true>, smem, kMostTokens * PI_MAX_ROTARY / 2 * sizeof(float2), done[1]);
  if (e != cudaSuccess) return e;
  if (p.r.interleaved)
    k_rotary<DT, V, false><<<grid, threads, smem, s>>>(p);
  else
    k_rotary<DT, V, true><<<grid, threads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int DT>
cudaError_t by_vector(const RotaryParams &p, int v, cudaStream_t s) {
  if constexpr (DT != PI_DT_F32)
    if (v == 8) return launch<DT, 8>(p, s);
  return v >= 4 ? launch<DT, 4>(p, s) : v == 2 ? launch<DT, 2>(p, s) : launch<DT, 1>(p, s);
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
  if (n_tokens < 0 || n_tokens > (1 << 28) || heads < 1 || heads > 65535 || head_dim > kMostDim)
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
  const bool copy = !same && head_dim > rotary->dim;
  if (copy) all |= (head_dim - rotary->dim) % 2 ? 1 : (head_dim - rotary->dim) / 2;
  // vectors of up to 16 bytes of which everything is a multiple
  const int v = e == 2 && all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
  const RotaryParams p{*rotary, positions, x, y, x_stride[0], x_stride[1], y_stride[0], y_stride[1], n_tokens, heads, head_dim,
                       1, heads, copy, inverse ? -1.f : 1.f};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PI_TRY_CUDA(dtype == PI_DT_F16    ? by_vector<PI_DT_F16>(p, v, s)
              : dtype == PI_DT_BF16 ? by_vector<PI_DT_BF16>(p, v, s)
                                    : by_vector<PI_DT_F32>(p, v, s));
  return PI_OK;
}
