// Log-probabilities of given tokens, entropy and the most likely tokens.
//
//   m = max_j x_j,  Z = sum_j 2^(log2(e) (x_j - m)),  S = sum_j z_j 2^(z_j),  z_j = log2(e) (x_j - m)
//   lse = m + ln Z,  logprob = x_t - lse,  entropy = ln 2 (log2 Z - S / Z)
//
// The logits are read once, with a running maximum; Z and S move to a new
// maximum as Z' = c Z, S' = c (S + (m - m') log2(e) Z), c = 2^(log2(e)(m - m')).
// Bound by HBM for many rows; by latency for the few of a decode step.
#include "pi_ops.cuh"

#include <algorithm>

using namespace pidev;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct ScoreParams {
  const void *x;
  int64_t stride;
  int rows, vocab, top_k;
  const int32_t *target;
  float *logprob, *entropy, *lse;
  int32_t *top_index;
  float *top_logprob;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Stats {
  float m, Z, S;
};
// Sums a relative to their own maxima, put together.
__device__ __forceinline__ Stats join(Stats a, Stats b) {
  const float m = fmaxf(a.m, b.m), ms = m == -INFINITY ? 0.f : m;
  const float da = (a.m - ms) * kLog2e, db = (b.m - ms) * kLog2e;
  const float ca = ex2(da), cb = ex2(db);
  // a part whose factor is 0 adds nothing (its difference may be -inf)
  const float sa = ca == 0.f ? 0.f : ca * fmaf(da, a.Z, a.S), sb = cb == 0.f ? 0.f : cb * fmaf(db, b.Z, b.S);
  return Stats{m, fmaf(ca, a.Z, cb * b.Z), sa + sb};
}

// Order of the alternatives: larger logit first (NaN above all, -0 as 0), then smaller index.
__device__ __forceinline__ unsigned long long order_key(float x, int j) {
  unsigned b = __float_as_uint(x == 0.f ? 0.f : x);
  b = b & 0x80000000u ? ~b : b | 0x80000000u;
  if (x != x) b = 0xffffffffu;
  return (unsigned long long)b << 32 | (0xffffffffu - (unsigned)j);
}

template <int DT, int V>
__global__ void __launch_bounds__(512) k_score(const ScoreParams p) {
  using E = Elem<DT>;
  using P = Pack<DT, V>;
  __shared__ Stats red[16];
  __shared__ unsigned long long kred[16];
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const typename E::T *x = static_cast<const typename E::T *>(p.x) + row * p.stride;
  const int nv = p.vocab / V;
  Stats st{-INFINITY, 0.f, 0.f};
  for (int i = threadIdx.x; i < nv; i += 512) {
    const P raw = reinterpret_cast<const P *>(x)[i];
    float f[V], m = -INFINITY;
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = E::to(raw.v[e]), m = fmaxf(m, f[e]);
    if (m > st.m) st = join(st, Stats{m, 0.f, 0.f});
    const float ms = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float z = (f[e] - ms) * kLog2e, w = ex2(z);
      st.Z += w;
      if (w > 0.f) st.S = fmaf(w, z, st.S);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    st = join(st, Stats{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.Z, o),
                        __shfl_xor_sync(0xffffffffu, st.S, o)});
  if (lane == 0) red[warp] = st;
  __syncthreads();
  st = red[0];
#pragma unroll
  for (int w = 1; w < 16; ++w) st = join(st, red[w]);
  const float lse = st.m + log2f(st.Z) * kLn2;
  if (threadIdx.x == 0) {
    if (p.lse) p.lse[row] = lse;
    if (p.entropy) p.entropy[row] = kLn2 * (log2f(st.Z) - st.S / st.Z);
    if (p.logprob) {
      const int t = p.target[row];
      p.logprob[row] = t < 0 ? 0.f : t >= p.vocab ? __uint_as_float(0x7fffffffu) : E::to(x[t]) - lse;
    }
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < p.top_k; ++k) {
    unsigned long long best = 0;
    for (int j = threadIdx.x; j < p.vocab; j += 512) {
      const unsigned long long key = order_key(E::to(x[j]), j);
      if (key < last && key > best) best = key;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) kred[warp] = best;
    __syncthreads();
    best = kred[0];
#pragma unroll
    for (int w = 1; w < 16; ++w) best = max(best, kred[w]);
    last = best;
    if (threadIdx.x == 0) {
      const int j = (int)(0xffffffffu - (unsigned)best);
      p.top_index[(int64_t)row * p.top_k + k] = j;
      p.top_logprob[(int64_t)row * p.top_k + k] = E::to(x[j]) - lse;
    }
    __syncthreads();
  }
}

template <int DT>
cudaError_t score_by_type(const ScoreParams &p, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(typename Elem<DT>::T);
  if (vec)
    k_score<DT, V><<<p.rows, 512, 0, s>>>(p);
  else
    k_score<DT, 1><<<p.rows, 512, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

extern "C" pi_status pi_token_logprobs(const void *logits, int64_t row_stride, int32_t dtype, int32_t rows, int32_t vocab,
                                       const int32_t *target, int32_t top_k, float *logprob, float *entropy, float *lse,
                                       int32_t *top_index, float *top_logprob, void *stream) {
  pi::clear_error();
  if (rows < 0) return pi::fail(PI_ERR_INVALID_ARG, "rows=%d is negative", rows);
  if (vocab < 1) return pi::fail(PI_ERR_INVALID_ARG, "vocab=%d: need at least one token", vocab);
  if (!pi::dtype_ok(dtype)) return pi::fail(PI_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (top_k < 0 || top_k > PI_MAX_TOP_K || top_k > vocab)
    return pi::fail(PI_ERR_INVALID_ARG, "top_k=%d outside [0, min(%d, vocab)]", top_k, PI_MAX_TOP_K);
  if (rows == 0) return PI_OK;
  if (!logits || !pi::aligned_to(logits, pi::dtype_size(dtype)))
    return pi::fail(PI_ERR_INVALID_ARG, "logits must be non-NULL and aligned to their type");
  if (rows > 1 && row_stride < vocab) return pi::fail(PI_ERR_INVALID_ARG, "row_stride is less than vocab=%d", vocab);
  if (logprob && !target) return pi::fail(PI_ERR_INVALID_ARG, "logprob needs target");
  if (top_k && (!top_index || !top_logprob)) return pi::fail(PI_ERR_INVALID_ARG, "top_k needs top_index and top_logprob");
  if (!pi::aligned_to(target, 4) || !pi::aligned_to(logprob, 4) || !pi::aligned_to(entropy, 4) ||
      !pi::aligned_to(lse, 4) || !pi::aligned_to(top_index, 4) || !pi::aligned_to(top_logprob, 4))
    return pi::fail(PI_ERR_INVALID_ARG, "target and the outputs must be 4-byte aligned");
  const int V = 16 / pi::dtype_size(dtype);
  const bool vec = pi::aligned_to(logits, 16) && vocab % V == 0 && (rows == 1 || row_stride % V == 0);
  const ScoreParams p{logits, row_stride, rows, vocab, top_k, target, logprob, entropy, lse, top_index, top_logprob};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PI_TRY_CUDA(dtype == PI_DT_F16    ? score_by_type<PI_DT_F16>(p, vec, s)
              : dtype == PI_DT_BF16 ? score_by_type<PI_DT_BF16>(p, vec, s)
                                    : score_by_type<PI_DT_F32>(p, vec, s));
  return PI_OK;
}
