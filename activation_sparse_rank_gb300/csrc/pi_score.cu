// Log-probabilities of given tokens, entropy and the most likely tokens.
//
//   m = max_j x_j,  z_j = log2(e) (x_j - m),  Z = sum_j 2^z_j,  S = sum_j z_j 2^z_j
//   lse = m + ln Z,  logprob = x_t - lse,  entropy = ln 2 (log2 Z - S / Z)
//
// Sums relative to one maximum move to another as Z' = c Z, S' = c (S + d Z)
// with d = log2(e) (m - m'), c = 2^d.  Bound by HBM for many rows; by latency
// for the few of a decode step.
//
// Few rows: a row is read once and kept in registers (up to 256 bytes a thread; a
// cluster of CTAs where one is too small).  Many rows stream through shared memory.
// Each thread's maximum gives its sums their reference and, together, the
// alternatives a bound: the k-th largest of any selection of elements is at most
// the k-th largest of all.  Elements at or above that bound are few; they are
// ranked by counting.
//
// Measured: 2048 x 131072 bf16, 20 alternatives, 107 us (5.0 TB/s, 75% of the copy rate;
// 90 us without alternatives; 608 CTAs take three or four rows each); 16 x 50007
// binary32, 5 alternatives, 7.2 us.
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

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct Stats {
  float m, Z, S;
};
// Sums a relative to their own maxima, put together.
__device__ __forceinline__ Stats join(Stats a, Stats b) {
  const float m = max_nan(a.m, b.m), ms = m == -INFINITY ? 0.f : m;
  const float da = (a.m - ms) * kLog2e, db = (b.m - ms) * kLog2e;
  const float ca = ex2(da), cb = ex2(db);
  // a part whose factor is 0 adds nothing (its difference may be -inf)
  const float sa = ca == 0.f ? 0.f : ca * fmaf(da, a.Z, a.S), sb = cb == 0.f ? 0.f : cb * fmaf(db, b.Z, b.S);
  return Stats{m, fmaf(ca, a.Z, cb * b.Z), sa + sb};
}

// The sums of a warp's 32 lanes, in every lane.
__device__ __forceinline__ Stats warp_join(Stats a) {
  float m = a.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float d = (a.m - (m == -INFINITY ? 0.f : m)) * kLog2e, c = ex2(d);
  const float S = c == 0.f ? 0.f : c * fmaf(d, a.Z, a.S);
  return Stats{m, warp_sum(c * a.Z), warp_sum(S)};
}

// Order of the alternatives: larger logit first (NaN above all, -0 as 0), then smaller index.
__device__ __forceinline__ unsigned long long order_key(float x, int j) {
  unsigned b = __float_as_uint(x == 0.f ? 0.f : x);
  b = b & 0x80000000u ? ~b : b | 0x80000000u;
  if (x != x) b = 0xffffffffu;
  return (unsigned long long)b << 32 | (0xffffffffu - (unsigned)j);
}

__device__ __forceinline__ float logit_of(unsigned long long key) {
  const unsigned b = (unsigned)(key >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
// What the threads of a CTA's warps agree on for one row's outputs.
__device__ __forceinline__ void write_stats(const ScoreParams &p, int row, const Stats &st, float lse, float x_target) {
  if (p.lse) p.lse[row] = lse;
  const bool none = !(fabsf(st.m) < INFINITY);       // NaN, +inf, or nothing but -inf
  if (p.entropy) p.entropy[row] = none ? __uint_as_float(0x7fffffffu) : kLn2 * (log2f(st.Z) - st.S / st.Z);
  if (p.logprob) {
    const int t = p.target[row];
    p.logprob[row] = t < 0 ? 0.f : t >= p.vocab || none ? __uint_as_float(0x7fffffffu) : x_target - lse;
  }
}
__device__ __forceinline__ float lse_of(const Stats &st) {
  return fabsf(st.m) < INFINITY ? st.m + log2f(st.Z) * kLn2 : st.m == -INFINITY ? st.m : __uint_as_float(0x7fffffffu);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Store into the same shared variable of the cluster's CTA 0.
template <typename T>
__device__ __forceinline__ void store_leader(T *p, unsigned long long v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

constexpr int kRegVecs = 16;         // 16-byte pieces of a row a thread holds
constexpr int kSlots = 128;          // runs of pieces that are looked through for alternatives
constexpr int kRuns = 8;             // of a thread and row of k_score_stream, at most
constexpr int kList = 512;           // alternatives ranked by counting
constexpr int kMaxCluster = 8;

// Largest element of a piece, NaN above all.
template <int DT>
__device__ __forceinline__ float piece_max(const uint4 &r) {
  const unsigned w[4] = {r.x, r.y, r.z, r.w};
  if constexpr (DT == PI_DT_F16) {
    __half2 a = __hmax2_nan(*reinterpret_cast<const __half2 *>(&w[0]), *reinterpret_cast<const __half2 *>(&w[1]));
    a = __hmax2_nan(a, __hmax2_nan(*reinterpret_cast<const __half2 *>(&w[2]), *reinterpret_cast<const __half2 *>(&w[3])));
    return max_nan(__low2float(a), __high2float(a));
  } else if constexpr (DT == PI_DT_BF16) {
    __nv_bfloat162 a = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&w[0]), *reinterpret_cast<const __nv_bfloat162 *>(&w[1]));
    a = __hmax2_nan(a, __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&w[2]), *reinterpret_cast<const __nv_bfloat162 *>(&w[3])));
    return max_nan(__low2float(a), __high2float(a));
  } else {
    return max_nan(max_nan(__uint_as_float(w[0]), __uint_as_float(w[1])), max_nan(__uint_as_float(w[2]), __uint_as_float(w[3])));
  }
}
// The piece with nothing below `least` (a finite number, or the rounding of one up to the type's lowest).
template <int DT>
__device__ __forceinline__ uint4 clamp_piece(uint4 r, float least) {
  unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == PI_DT_F16) {
      const __half2 h = __hmax2(*reinterpret_cast<const __half2 *>(&w[k]), __half2half2(__float2half_rd(fmaxf(least, -65504.f))));
      w[k] = *reinterpret_cast<const unsigned *>(&h);
    } else if constexpr (DT == PI_DT_BF16) {
      const __nv_bfloat162 h = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&w[k]), __bfloat162bfloat162(__float2bfloat16_rd(least)));
      w[k] = *reinterpret_cast<const unsigned *>(&h);
    } else {
      w[k] = __float_as_uint(fmaxf(__uint_as_float(w[k]), least));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whether what clamp_piece makes of 140 below m is at least 100 below m, so that its
// weight is 0: not where m - 140 rounds to m, nor where it is past fp16's lowest value.
template <int DT>
__device__ __forceinline__ bool clamps_near(float m) {
  return fabsf(m) < 0x1p24f && (DT != PI_DT_F16 || m > -65400.f);
}
// A piece's sums relative to m = -minus added to Z and S.  NEAR: what is further
// below m than 140 has weight 0 either way, and is clamped before the subtraction,
// in the element's type (one operation for two, and no 0 (-inf)).  Otherwise the
// difference is clamped: then only what is -inf or far below has weight 0.
template <int DT, bool NEAR>
__device__ __forceinline__ void add_piece(const uint4 &raw, float least, f2 minus, f2 &Z, f2 &S) {
  const f2 l2e = f2_of(kLog2e, kLog2e);
  const uint4 r = NEAR ? clamp_piece<DT>(raw, least) : raw;
#pragma unroll
  for (int j = 0; j < 8 / (int)sizeof(typename Elem<DT>::T); ++j) {
    f2 zz = f2_mul(f2_add(f2_from16<DT>(r, j), minus), l2e);
    if constexpr (!NEAR) zz = f2_of(fmaxf(zz.x, -200.f), fmaxf(zz.y, -200.f));
    const float2 z = f2_get(zz);
    const f2 e = f2_of(ex2(z.x), ex2(z.y));
    Z = f2_add(Z, e);
    S = f2_fma(e, zz, S);
  }
}

// keys[0, n) (distinct): the k largest in order, to put(rank, key).
template <typename F>
__device__ __forceinline__ void rank_keys(const unsigned long long *keys, int n, int k, F put) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const unsigned long long mine = keys[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += keys[j] > mine;
    if (rank < k) put(rank, mine);
  }
}

// A row as 16-byte pieces: they start at the last 16-byte boundary at or before
// it, and its first and last one may hold elements of other rows.
template <int DT>
struct Row {
  using T = typename Elem<DT>::T;
  static constexpr int V = 16 / sizeof(T);
  const T *x;
  int off, pieces, vocab;                            // elements of the first piece before the row; pieces; elements
  __device__ __forceinline__ Row(const ScoreParams &p, int r) {
    x = static_cast<const T *>(p.x) + r * p.stride;
    off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    vocab = p.vocab;
    pieces = (int)(((int64_t)vocab + off + V - 1) / V);
  }
  __device__ __forceinline__ const uint4 *base() const { return reinterpret_cast<const uint4 *>(x - off); }
  __device__ __forceinline__ bool inner(int c) const { return c > 0 && c < pieces - 1; }
  // Piece c with -inf for what is not the row's (not read).
  __device__ __forceinline__ uint4 edge(int c) const {
    constexpr unsigned low = DT == PI_DT_F32 ? 0xff800000u : DT == PI_DT_F16 ? 0xfc00fc00u : 0xff80ff80u;
    alignas(16) T e[V];
    *reinterpret_cast<uint4 *>(e) = make_uint4(low, low, low, low);
    if (c < pieces) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int j = c * V + k - off;
        if (j >= 0 && j < vocab) e[k] = x[j];
      }
    }
    return *reinterpret_cast<const uint4 *>(e);
  }
};

template <int NW>
struct TopShared {
  unsigned tops[NW * 32];
  unsigned long long list[kList], best[NW];
  int owner[kSlots], counts[NW];
  int n_list, n_owners;
  unsigned tau;
};

// The k largest keys of pieces [first, last) of a row, in order, to put(rank,
// key); returns how many there are.  mt: the largest element of this thread's
// pieces first + t, first + t + NT, ....  The whole CTA calls it.
//
// The k-th largest of any of the elements is at most the k-th largest of all: the
// thread maxima give a bound, and few threads have anything at or above it.
// Their pieces are read again, by all threads.  A row that has left L2 by then
// costs HBM a sector for each piece, so where `runs` gives the maxima of a thread's
// runs of `span` pieces ([run][thread]), only those at or above the bound are read
// (2048 x 131072 bf16: 113 -> 105 us).
template <int DT, int NT, typename F>
__device__ __forceinline__ int cta_top(const Row<DT> &w, int first, int last, float mt, int K, TopShared<NT / 32> &sh, F put,
                                       const float *runs = nullptr, int span = 0) {
  using E = Elem<DT>;
  constexpr int NW = NT / 32, V = Row<DT>::V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, M = min(32, max(4, (2 * K + NW - 1) / NW));
  const int begin = max(0, first * V - w.off), end = min(w.vocab, last * V - w.off);      // elements
  const unsigned key = first + (int)threadIdx.x < last ? (unsigned)(order_key(mt, 0) >> 32) : 0u;
  unsigned cur = key, kept = 0;                      // 0: no element
#pragma unroll 1
  for (int r = 0; r < M; ++r) {                      // the M largest of each warp
    const unsigned mx = __reduce_max_sync(0xffffffffu, cur);
    if (lane == r) kept = mx;
    if (lane == __ffs(__ballot_sync(0xffffffffu, cur == mx)) - 1) cur = 0;
  }
  if (lane < M) sh.tops[warp * M + lane] = kept;
  if (threadIdx.x == 0) sh.tau = NW * M < K ? 0u : 0xffffffffu, sh.n_list = sh.n_owners = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < NW * M; i += NT) {
    const unsigned t = sh.tops[i];
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < NW * M; ++j) above += sh.tops[j] > t;
    if (above < K) atomicMin(&sh.tau, t);
  }
  __syncthreads();
  const unsigned tau = sh.tau;
  const int each = (last - first + NT - 1) / NT;     // pieces of a thread
  // elements whose key is `low` or more, of the runs whose maximum is, into the list; false if they are too many
  auto collect = [&](unsigned low) {
    if (key && key >= low) {
      for (int k = 0; k < (runs ? (each + span - 1) / span : 1); ++k) {
        if (runs && (unsigned)(order_key(runs[k * NT + threadIdx.x], 0) >> 32) < low) continue;
        const int n = atomicAdd(&sh.n_owners, 1);
        if (n < kSlots) sh.owner[n] = threadIdx.x | k << 16;
      }
    }
    __syncthreads();
    const int n = sh.n_owners, run = runs ? span : each;
    if (n <= kSlots) {
      const float by = 1.f / (float)run;             // i / run, exact: i + 0.5 is at least 0.5 / run from a whole quotient
#pragma unroll 1
      for (int i = threadIdx.x; i < n * run; i += NT) {
        const int o = (int)(((float)i + 0.5f) * by), at = sh.owner[o];
        const int c = first + ((at >> 16) * run + i - o * run) * NT + (at & 0xffff);
        if (c >= last) continue;
        const uint4 r = w.inner(c) ? ld_stream(w.base() + c) : w.edge(c);
        if ((unsigned)(order_key(piece_max<DT>(r), 0) >> 32) < low) continue;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float2 f = f2_get(f2_from16<DT>(r, k / 2));
          const int at = c * V + k - w.off;
          const unsigned long long e = order_key(k & 1 ? f.y : f.x, at);
          if ((unsigned)(e >> 32) < low || at < 0 || at >= w.vocab) continue;
          const int m = atomicAdd(&sh.n_list, 1);
          if (m < kList) sh.list[m] = e;
        }
      }
    }
    __syncthreads();
    return n <= kSlots && sh.n_list <= kList;
  };
  if (collect(tau)) {
    rank_keys(sh.list, sh.n_list, K, put);
    return min(K, sh.n_list);
  }
  // Many equal to the bound (masked rows): those above it, of fewer than K threads, then the equal ones by index.
  __syncthreads();
  if (threadIdx.x == 0) sh.n_list = sh.n_owners = 0;
  __syncthreads();
  if (tau != 0xffffffffu ? collect(tau + 1) : true) {
    int found = min(K, sh.n_list);
    rank_keys(sh.list, sh.n_list, K, put);
#pragma unroll 1
    for (int j0 = begin; j0 < end && found < K; j0 += NT) {
      const int j = j0 + threadIdx.x;
      const unsigned long long e = j < end ? order_key(E::to(w.x[j]), j) : 0;
      const bool hit = j < end && (unsigned)(e >> 32) == tau;
      const unsigned mask = __ballot_sync(0xffffffffu, hit);
      if (lane == 0) sh.counts[warp] = __popc(mask);
      __syncthreads();
      int at = found + __popc(mask & ((1u << lane) - 1)), all = found;
      for (int i = 0; i < NW; ++i) {
        if (i < warp) at += sh.counts[i];
        all += sh.counts[i];
      }
      if (hit && at < K) put(at, e);
      found = min(K, all);
      __syncthreads();
    }
    return found;
  }
  // Many above it in few threads: one after another.
  unsigned long long prev = ~0ull;
  int found = 0;
#pragma unroll 1
  for (; found < min(K, end - begin); ++found) {
    unsigned long long best = 0;
    for (int j = begin + threadIdx.x; j < end; j += NT) {
      const unsigned long long e = order_key(E::to(w.x[j]), j);
      if (e < prev && e > best) best = e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) sh.best[warp] = best;
    __syncthreads();
    prev = sh.best[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) prev = max(prev, sh.best[i]);
    if (threadIdx.x == 0) put(found, prev);
    __syncthreads();
  }
  return found;
}

// One row for a cluster of CTAs; CTA r has the row's pieces [r share, (r + 1)
// share), thread t of it pieces t, t + NT, ..., which it keeps in registers from
// the maximum to the sums.
template <int DT, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) k_score_row(const ScoreParams p, int share) {
  using E = Elem<DT>;
  constexpr int NW = NT / 32;
  __shared__ Stats red[NW];
  __shared__ TopShared<NW> sh;
  __shared__ unsigned long long in_keys[kMaxCluster][PI_MAX_TOP_K];
  __shared__ unsigned long long in_mz[kMaxCluster], in_s[kMaxCluster];
  uint32_t rank, size;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  if (size > 1) cluster_arrive();                    // waited for before the leader's memory is written
  const int row = blockIdx.x / size, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = p.top_k;
  const Row<DT> w(p, row);
  const int first = rank * share, last = min(w.pieces, first + share);

  uint4 raw[kRegVecs];
  const unsigned low = DT == PI_DT_F32 ? 0xff800000u : DT == PI_DT_F16 ? 0xfc00fc00u : 0xff80ff80u;    // -inf
#pragma unroll
  for (int i = 0; i < kRegVecs; ++i) raw[i] = make_uint4(low, low, low, low);
#pragma unroll
  for (int i = 0; i < kRegVecs; ++i) {
    const int c = first + i * NT + threadIdx.x;
    if (c < last && w.inner(c)) raw[i] = ld_stream(w.base() + c);
  }
  if (threadIdx.x == 0 && rank == 0) raw[0] = w.edge(0);
  if (w.pieces > 1 && w.pieces - 1 >= first && w.pieces - 1 < last && (w.pieces - 1 - first) % NT == threadIdx.x) {
    const uint4 r = w.edge(w.pieces - 1);
    const int at = (w.pieces - 1 - first) / NT;
    each<kRegVecs>([&](auto i) {
      if (at == i.v) raw[i.v] = r;
    });
  }

  // ---- this thread's maximum and sums ----
  float mt = -INFINITY;
  each<kRegVecs>([&](auto i) {
    if (i.v == 0 || first + i.v * NT < last) mt = max_nan(mt, piece_max<DT>(raw[i.v]));    // uniform: pieces of no thread
  });
  Stats st{mt, 0.f, 0.f};
  if (mt > -INFINITY) {                              // else nothing, or a NaN that m carries on
    const f2 minus = f2_of(-mt, -mt);
    f2 Z = f2_of(0.f, 0.f), S = Z;
    auto add = [&](auto near) {
      each<kRegVecs>([&](auto i) {
        if (i.v == 0 || first + i.v * NT < last) add_piece<DT, decltype(near)::v>(raw[i.v], mt - 140.f, minus, Z, S);
      });
    };
    if (clamps_near<DT>(mt)) add(Int<1>{}); else add(Int<0>{});
    st.Z = f2_sum(Z), st.S = f2_sum(S);
  }
  __syncwarp();
  st = warp_join(st);
  if (lane == 0) red[warp] = st;
  __syncthreads();
  if (warp == NW - 1) st = warp_join(lane < NW ? red[lane] : Stats{-INFINITY, 0.f, 0.f});     // of the CTA
  if (size > 1) cluster_wait();
  if (K) {
    auto put = [&](int r, unsigned long long key) { store_leader(&in_keys[rank][r], key); };
    const int n = cta_top<DT, NT>(w, first, last, mt, K, sh, put);
    for (int r = n + threadIdx.x; r < K; r += NT) put(r, 0);
  }
  if (threadIdx.x == NT - 1) {
    store_leader(&in_mz[rank], (unsigned long long)__float_as_uint(st.m) << 32 | __float_as_uint(st.Z));
    store_leader(&in_s[rank], __float_as_uint(st.S));
  }
  if (size > 1) {
    cluster_arrive();
    if (rank) return;                                // its memory is nobody's to read
    cluster_wait();
  } else {
    __syncthreads();
  }

  // ---- the leader: the row's statistics and alternatives ----
  st = Stats{-INFINITY, 0.f, 0.f};
  if (lane < (int)size)
    st = Stats{__uint_as_float((unsigned)(in_mz[lane] >> 32)), __uint_as_float((unsigned)in_mz[lane]), __uint_as_float((unsigned)in_s[lane])};
  st = warp_join(st);
  const float lse = lse_of(st);
  if (threadIdx.x == 0) {
    const int t = p.logprob ? p.target[row] : -1;
    write_stats(p, row, st, lse, t >= 0 && t < p.vocab ? E::to(w.x[t]) : 0.f);
  }
  if (K) {
    auto out = [&](int r, unsigned long long key) {
      p.top_index[(int64_t)row * K + r] = (int)(0xffffffffu - (unsigned)key);
      p.top_logprob[(int64_t)row * K + r] = st.m == -INFINITY ? __uint_as_float(0x7fffffffu) : logit_of(key) - lse;
    };
    if (size == 1) {
      for (int r = threadIdx.x; r < K; r += NT) out(r, in_keys[0][r]);
    } else {
      // every CTA's list is sorted: a key's rank is its own place and how many of each other list are above it
      for (int i = threadIdx.x; i < (int)size * K; i += NT) {
        const int c = i / K, r = i % K;
        const unsigned long long key = in_keys[c][r];
        if (!key) continue;
        int above = r;
        for (int o = 0; o < (int)size; ++o) {
          if (o == c) continue;
          int lo = 0, hi = min(K, K - above);        // past K the key is out
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (in_keys[o][mid] > key) lo = mid + 1; else hi = mid;
          }
          above += lo;
          if (above >= K) break;
        }
        if (above < K) out(above, key);
      }
    }
  }
}

// Many rows: a persistent CTA takes whole rows, one after another, in batches of
// stream_batch pieces a thread that come through a ring in shared memory: a thread
// copies its own pieces there (cp.async) and is the only one to read them, so a
// batch needs no barrier, and what is on its way takes no registers.  Copies run
// a batch ahead, into the next row too, so what is done at a row's end costs
// little bandwidth; two batches ahead took 127 us for 2048 x 131072 (116 so), as
// the ring then leaves L1 too little for the pieces that are read again.
constexpr int kStages = 2;
constexpr int stream_batch(int NT) { return NT == 64 ? 2 : 4; }
constexpr int stream_smem(int NT) { return kStages * stream_batch(NT) * NT * 16; }
constexpr int stream_ctas(int NT) { return 1024 / NT; }
template <int DT, int NT>
__global__ void __launch_bounds__(NT, stream_ctas(NT)) k_score_stream(const ScoreParams p) {
  using E = Elem<DT>;
  constexpr int NW = NT / 32, RB = stream_batch(NT);
  extern __shared__ __align__(16) uint4 ring[];      // [stage][piece][thread]
  __shared__ Stats red[NW];
  __shared__ TopShared<NW> sh;
  __shared__ float runs[kRuns][NT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = p.top_k;

  // the next batch to copy
  int crow = blockIdx.x, cb = 0, cstage = 0;
  Row<DT> cw(p, min(crow, p.rows - 1));
  auto copy = [&] {
    if (crow < p.rows) {
      uint4 *dst = ring + cstage * RB * NT + threadIdx.x;
      const int c0 = cb * RB * NT + threadIdx.x;
      const bool inner = cb > 0 && (cb + 1) * RB * NT < cw.pieces;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const int c = c0 + i * NT;
        if (inner || cw.inner(c))
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(dst + i * NT)),
                       "l"(cw.base() + c) : "memory");
      }
      if (!inner) {
#pragma unroll 1
        for (int i = 0; i < RB; ++i)
          if (!cw.inner(c0 + i * NT)) dst[i * NT] = cw.edge(c0 + i * NT);
      }
      if ((cb + 1) * RB * NT >= cw.pieces) {
        cb = 0, crow += gridDim.x;
        if (crow < p.rows) cw = Row<DT>(p, crow);
      } else {
        ++cb;
      }
    }
    cstage = cstage + 1 == kStages ? 0 : cstage + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) copy();

  int stage = 0;
#pragma unroll 1
  for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const Row<DT> w(p, row);
    Stats st{-INFINITY, 0.f, 0.f};
    const int per_run = ((w.pieces + RB * NT - 1) / (RB * NT) + kRuns - 1) / kRuns;    // batches of a run
    float run_max = -INFINITY;
    int run = 0, left = per_run;
#pragma unroll 1
    for (int b = 0; b * RB * NT < w.pieces; ++b) {
      copy();                                        // into the stage that the last batch left
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      const uint4 *raw = ring + stage * RB * NT + threadIdx.x;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const int n = min(RB, (w.pieces - b * RB * NT + NT - 1) / NT);   // pieces of this batch that any thread has
#pragma unroll
      for (int i = 0; i < RB; ++i)
        if (i < n) run_max = max_nan(run_max, piece_max<DT>(raw[i * NT]));
      const float m = max_nan(st.m, run_max);
      if (m > -INFINITY) {
        const float d = (st.m - m) * kLog2e, c = ex2(d);
        f2 Z = f2_of(c * st.Z, 0.f), S = f2_of(c == 0.f ? 0.f : c * fmaf(d, st.Z, st.S), 0.f);
        const f2 minus = f2_of(-m, -m);
        auto add = [&](auto near) {
#pragma unroll
          for (int i = 0; i < RB; ++i)
            if (i < n) add_piece<DT, decltype(near)::v>(raw[i * NT], m - 140.f, minus, Z, S);
        };
        if (clamps_near<DT>(m)) add(Int<1>{}); else add(Int<0>{});
        st.Z = f2_sum(Z), st.S = f2_sum(S);
      }
      st.m = m;
      runs[run][threadIdx.x] = run_max;              // the run so far
      if (--left == 0) ++run, left = per_run, run_max = -INFINITY;
      __syncwarp();
    }

    // ---- the row's results ----
    const float mt = st.m;
    st = warp_join(st);
    if (lane == 0) red[warp] = st;
    __syncthreads();
    st = warp_join(lane < NW ? red[lane] : Stats{-INFINITY, 0.f, 0.f});
    const float lse = lse_of(st);
    if (threadIdx.x == 0) {
      const int t = p.logprob ? p.target[row] : -1;
      write_stats(p, row, st, lse, t >= 0 && t < p.vocab ? E::to(w.x[t]) : 0.f);
    }
    if (K)
      cta_top<DT, NT>(w, 0, w.pieces, mt, K, sh, [&](int k, unsigned long long key) {
        p.top_index[(int64_t)row * K + k] = (int)(0xffffffffu - (unsigned)key);
        p.top_logprob[(int64_t)row * K + k] = st.m == -INFINITY ? __uint_as_float(0x7fffffffu) : logit_of(key) - lse;
      }, &runs[0][0], per_run * RB);
    __syncthreads();                                 // red and sh are free for the next row
  }
}

// Rows wider than a cluster's registers: one CTA a row, the row read once for
// the sums and once for each alternative.
template <int DT>
__global__ void __launch_bounds__(512) k_score_wide(const ScoreParams p) {
  using E = Elem<DT>;
  __shared__ Stats red[16];
  __shared__ unsigned long long kred[16];
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const typename E::T *x = static_cast<const typename E::T *>(p.x) + row * p.stride;
  Stats st{-INFINITY, 0.f, 0.f};
  for (int j = threadIdx.x; j < p.vocab; j += 512) {
    const float f = E::to(x[j]);
    if (!(f <= st.m)) st = join(st, Stats{f, 0.f, 0.f});       // NaN too
    const float z = fmaxf((f - (st.m == -INFINITY ? 0.f : st.m)) * kLog2e, -200.f), w = ex2(z);
    st.Z += w, st.S = fmaf(w, z, st.S);
  }
  st = warp_join(st);
  if (lane == 0) red[warp] = st;
  __syncthreads();
  st = warp_join(lane < 16 ? red[lane] : Stats{-INFINITY, 0.f, 0.f});
  const float lse = lse_of(st);
  if (threadIdx.x == 0) {
    const int t = p.logprob ? p.target[row] : -1;
    write_stats(p, row, st, lse, t >= 0 && t < p.vocab ? E::to(x[t]) : 0.f);
  }
  unsigned long long prev = ~0ull;
  for (int k = 0; k < p.top_k; ++k) {
    unsigned long long best = 0;
    for (int j = threadIdx.x; j < p.vocab; j += 512) {
      const unsigned long long key = order_key(E::to(x[j]), j);
      if (key < prev && key > best) best = key;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) kred[warp] = best;
    __syncthreads();
    prev = kred[0];
#pragma unroll
    for (int w = 1; w < 16; ++w) prev = max(prev, kred[w]);
    if (threadIdx.x == 0) {
      p.top_index[(int64_t)row * p.top_k + k] = (int)(0xffffffffu - (unsigned)prev);
      p.top_logprob[(int64_t)row * p.top_k + k] = st.m == -INFINITY ? __uint_as_float(0x7fffffffu) : logit_of(prev) - lse;
    }
    __syncthreads();
  }
}

template <int DT, int NT>
cudaError_t launch_row(const ScoreParams &p, int pieces, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.rows * cluster);
  cfg.blockDim = dim3(NT);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_score_row<DT, NT>, p, (pieces + cluster - 1) / cluster);
}

template <int DT, int NT>
cudaError_t launch_stream(const ScoreParams &p, cudaStream_t s) {
  static_assert(stream_smem(NT) + kRuns * NT * 4 + sizeof(TopShared<NT / 32>) + 512 <= 48 * 1024);
  k_score_stream<DT, NT><<<std::min(p.rows, stream_ctas(NT) * pi::current_sms()), NT, stream_smem(NT), s>>>(p);
  return cudaGetLastError();
}

template <int DT>
cudaError_t score_by_type(const ScoreParams &p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(typename Elem<DT>::T);
  // elements of a row's first piece before the row: the same for all, or the worst
  const int e = 16 / V, off = p.rows == 1 || p.stride % V == 0 ? (int)((reinterpret_cast<uintptr_t>(p.x) & 15) / e) : V - 1;
  const int64_t pieces64 = ((int64_t)p.vocab + off + V - 1) / V;
  if (pieces64 > (int64_t)512 * kRegVecs * kMaxCluster) {
    k_score_wide<DT><<<p.rows, 512, 0, s>>>(p);
    return cudaGetLastError();
  }
  const int pieces = (int)pieces64;
  auto fit = [&](int threads) {                      // CTAs of a cluster that hold a row
    int c = 1;
    while (c < kMaxCluster && (int64_t)threads * kRegVecs * c < pieces) c *= 2;
    return c;
  };
  // rows enough for every SM: whole rows one after another (620 x 2000 bf16: 6.0 us, a
  // CTA for each row 7.6; 5000 rows 17 and 29; 200 x 50007 binary32 14 us, a cluster for
  // each 21, but 200 x 32000 bf16 10 and 8), by CTAs that suit their width
  // (15630 x 2518 bf16: 50 us with 64 threads, 66 with 128; 2829 x 33510 fp16: 57 us with
  // 128, 65 with 256; 2048 x 131072 bf16: 105 us with 256, 149 with 128)
  if (p.rows >= (pieces > 6144 ? 1 : 2) * pi::current_sms())
    return pieces <= 640 ? launch_stream<DT, 64>(p, s) : pieces <= 6144 ? launch_stream<DT, 128>(p, s) : launch_stream<DT, 256>(p, s);
  // narrow rows: two warps; but the thread maxima of two bound many alternatives loosely
  // (16 x 5000 bf16, 20 of them: 9.3 us, 6.6 with 256 threads), unless most threads of
  // 256 would have no piece (16 x 700: 7.5 and 14.1)
  if (pieces <= 192 || (pieces <= 64 * kRegVecs && p.top_k <= 8)) return launch_row<DT, 64>(p, pieces, 1, s);
  // 256 threads a CTA, so that several are at different stages on an SM, and as many
  // CTAs as hold the row, no more (16 x 50007 binary32: 6.9 us with 4, 8.0 with 8);
  // 512 where eight of those do not (there 7.9)
  int cluster = fit(256);
  if (pieces <= 256 * kRegVecs * cluster) return launch_row<DT, 256>(p, pieces, cluster, s);
  return launch_row<DT, 512>(p, pieces, kMaxCluster, s);
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
  const ScoreParams p{logits, row_stride, rows, vocab, top_k, target, logprob, entropy, lse, top_index, top_logprob};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PI_TRY_CUDA(dtype == PI_DT_F16    ? score_by_type<PI_DT_F16>(p, s)
              : dtype == PI_DT_BF16 ? score_by_type<PI_DT_BF16>(p, s)
                                    : score_by_type<PI_DT_F32>(p, s));
  return PI_OK;
}
