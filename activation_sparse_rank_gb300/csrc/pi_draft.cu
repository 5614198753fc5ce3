// Drafted tokens: the tree they make, and which of them the target accepts.
//
// The tree.  A node's way to its root by doubling: in each round a node takes the
// bits of the node that it points to and then points where that one does, so a
// chain of n takes log2 n rounds.  Bound by latency: a CTA a sequence.
//
// Verification (speculative sampling with several drafts a node).  At a node with
// target p and draft q the children are gone through in turn, with w = p and W = 1:
//   accept child x if u q(x) W < w(x);  else w = max(w - W q, 0), W = sum w
// and the token after the last accepted node is the first i with sum_{j<=i} w_j > u W.
// Nothing that is left was 0 before, so after k rejections w = max(p - A q, 0), A the sum
// of the W before each (1 for the first): one step however many there were.  Without a
// draft w is p without the refused tokens: a pass compares each element with each of them.
//
// Sums are whole numbers of 2^-60: adding them is associative, so the result does
// not depend on how a row is split, and a probability's 24 bits are kept down to
// 2^-37; what is left after a rejection, its sum and both sides of a comparison have 48 bits
// (binary32 pairs: GB300's 64-bit floating point is 64 times slower).  A row is read only where a sum is needed: for a chain once for the whole
// sequence (at the rejection, or after the last token), and there its sums also say
// which warp has the sampled token.  What is needed of the other rows is the drafted
// token's two elements, all fetched at once at the start.
//
// A cluster of CTAs a sequence; they exchange one number each a pass, through
// distributed shared memory.
//
// Measured: 64 sequences with 8 nodes against 131072 tokens, binary32: 28 us; a pass of all of them
// takes 12 us for the target alone (2.7 TB/s), 16 with the draft (4.2), and a second refusal at a node 4 to 5 us
// more for its sequence alone (12 if all have one): latency and the fetch of instructions, 23 of them an element for the
// target alone and the first refusal, 31 for the later ones.  HBM does not bound a pass (18% of it from cold caches): 0.84
// waves of CTAs issue in a third of the cycles, and 40% of the warps' waiting is for instructions, 21% for loads.
// One sequence, a chain of four against 50007: 8.4 us.  Given tokens, all refused, 64 sequences against 131072: 18 us for
// one at a node, 31 for two, 44 for seven (two passes from two on; binary32; bf16 7 to 11% more).
#include "pi_ops.cuh"

#include <algorithm>

using namespace pidev;

namespace {

constexpr int kNodes = PI_MAX_TREE;

struct TreeParams {
  const int32_t *parent, *cu;
  int n_seqs, n_tokens, max_q, words;
  int32_t *mask, *depth;
};

__global__ void __launch_bounds__(kNodes) k_draft_tree(const TreeParams p) {
  __shared__ int to[2][kNodes];
  __shared__ unsigned bits[2][kNodes / 32][kNodes];
  const int s = blockIdx.x, i = threadIdx.x, r0 = p.cu[s], r1 = p.cu[s + 1];
  if (r0 < 0 || r1 < r0 || r1 > p.n_tokens) return;
  const int n = min(r1 - r0, p.max_q);
  int at = -1, now = 0;
  unsigned own[kNodes / 32];
  if (i < n) {
    at = p.parent[r0 + i];
    if (at < 0 || at >= i) at = -1;
  }
  to[0][i] = at;
#pragma unroll
  for (int w = 0; w < kNodes / 32; ++w) {
    own[w] = i < n && i / 32 == w ? 1u << i % 32 : 0u;
    if (w < p.words) bits[0][w][i] = own[w];
  }
  while (__syncthreads_or(at >= 0)) {                // the rows of this round are written
    if (at >= 0) {
#pragma unroll
      for (int w = 0; w < kNodes / 32; ++w)
        if (w < p.words) own[w] |= bits[now][w][at];
      at = to[now][at];
    }
    now ^= 1;
    to[now][i] = at;
#pragma unroll
    for (int w = 0; w < kNodes / 32; ++w)
      if (w < p.words) bits[now][w][i] = own[w];
  }
  if (i < n) {
    int d = -1;
#pragma unroll
    for (int w = 0; w < kNodes / 32; ++w)
      if (w < p.words) d += __popc(own[w]);
    if (p.depth) p.depth[r0 + i] = d;
  }
  if (p.mask)
    for (int k = i; k < n * p.words; k += blockDim.x) p.mask[(int64_t)r0 * p.words + k] = bits[now][k % p.words][k / p.words];
  for (int64_t k = (int64_t)n * p.words + i; k < (int64_t)(r1 - r0) * p.words; k += blockDim.x)       // rows past max_q
    if (p.mask) p.mask[(int64_t)r0 * p.words + k] = 0;
  for (int k = n + i; k < r1 - r0; k += blockDim.x)
    if (p.depth) p.depth[r0 + k] = -1;
}

// ---- verification -----------------------------------------------------------------

constexpr int kMostCluster = 8;
constexpr int kMostVocab = 1 << 21;

struct VerifyParams {
  const void *target, *draft;
  int64_t t_stride, q_stride;
  int vocab, n_seqs, n_tokens, max_q;
  const int32_t *drawn, *parent, *cu;
  const float *accept, *sample;
  int32_t *accepted, *path, *token;
};

using u64 = unsigned long long;

// A probability: NaN and what is below 0 count as 0, what is above 1 as 1.
__device__ __forceinline__ float unit(float p) { return __saturatef(p); }

// What is left of a probability, h + l in binary32 with |l| at most half a last place of h
// (48 bits; for whole steps of 2^-24 and the like exact).
struct Left {
  f2 h, l;                                           // of two elements
};
__device__ __forceinline__ f2 minus(f2 a, f2 b) { return f2_fma(b, f2_of(-1.f, -1.f), a); }
// max(p - q, 0)
__device__ __forceinline__ Left first_left(f2 p, f2 q) {
  const f2 m = f2_of(fminf(p.x, q.x), fminf(p.y, q.y)), d = minus(p, m);
  return Left{d, minus(minus(p, d), m)};             // p >= m: what d lost
}
// max(p - A q, 0), A = a.x + a.y
__device__ __forceinline__ Left later_left(f2 p, f2 q, float2 a) {
  const f2 big = f2_of(-a.x, -a.x), n = f2_mul(q, big);
  const f2 nl = f2_fma(q, f2_of(-a.y, -a.y), f2_fma(q, big, f2_mul(q, f2_of(a.x, a.x))));
  const f2 s = f2_add(p, n), t = minus(s, p);        // s + what it lost = p + n
  const f2 tail = f2_add(f2_add(minus(p, minus(s, t)), minus(n, t)), nl);
  const f2 h = f2_add(s, tail), l = minus(tail, minus(h, s));
  return Left{f2_of(fmaxf(h.x, 0.f), fmaxf(h.y, 0.f)), f2_of(h.x > 0.f ? l.x : 0.f, h.y > 0.f ? l.y : 0.f)};
}

// Sums of what is left in whole 2^-60: each is cut into three numbers of 22 bits or less,
// read off the last bits of a sum with a constant whose last place is 2^-22, 2^-44 and
// 2^-60; what such a sum rounds away is exact and goes on to the next (l with it, to 2^-48).
constexpr float kTo22 = 2.f, kTo44 = 0x1.8p-21f, kTo60 = 0x1.8p-37f;
constexpr float kTiny = 0x1p-61f;                    // up to here, what is not 0 would round to 0 (a tie, to even): 1 more
struct Parts {
  unsigned a, b, c;
};
__device__ __forceinline__ void add_left(Parts &s, const Left &w) {
  const f2 t = f2_add(w.h, f2_of(kTo22, kTo22)), r = f2_add(minus(w.h, f2_add(t, f2_of(-kTo22, -kTo22))), w.l);
  const f2 u = f2_add(r, f2_of(kTo44, kTo44)), q = minus(r, f2_add(u, f2_of(-kTo44, -kTo44)));
  const f2 v = f2_add(q, f2_of(kTo60, kTo60));
  s.a += __float_as_uint(t.x) + __float_as_uint(t.y);
  s.b += __float_as_uint(u.x) + __float_as_uint(u.y);
  s.c += __float_as_uint(v.x) + __float_as_uint(v.y);
  s.c += (w.h.x > 0.f && w.h.x <= kTiny) + (w.h.y > 0.f && w.h.y <= kTiny);
}
// The sum of n elements, less the constants' bits.
__device__ __forceinline__ u64 joined(const Parts &s, unsigned n) {
  return ((u64)(s.a - n * __float_as_uint(kTo22)) << 38) + (u64)((int64_t)(int)(s.b - n * __float_as_uint(kTo44)) << 16) +
         (u64)(int64_t)(int)(s.c - n * __float_as_uint(kTo60));
}

// A sum of whole 2^-60 in two parts.
__device__ __forceinline__ float2 in_two(u64 s) {
  const float h = __ull2float_rz(s);
  return make_float2(h * 0x1p-60f, (float)(s - __float2ull_rz(h)) * 0x1p-60f);
}
// a b in two parts
__device__ __forceinline__ float2 product(float a, float b) {
  const float h = a * b;
  return make_float2(h, fmaf(a, b, -h));
}
constexpr float kUp = 0x1p60f;                       // keeps the parts of small products above binary32's least

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// A value into the same shared variable of the cluster's CTA `rank`.
__device__ __forceinline__ void store_in(u64 *at, int rank, u64 v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(at)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <int DT, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_verify(const VerifyParams p, const int size) {
  using E = Elem<DT>;
  using T = typename E::T;
  constexpr int V = 16 / sizeof(T), kWarps = NT / 32;
  constexpr int kMostChunks = kMostVocab / 4 / 32 / kWarps + 1;      // pieces of 32 vectors that a warp's share of a row has
  constexpr int kAtOnce = V == 4 ? 4 : 2;            // pieces of a row that a warp loads together, as registers allow
  constexpr int kRun = 512 / V;                      // pieces whose parts, added, stay within 32 bits
  __shared__ int s_parent[kNodes], s_drawn[kNodes], s_path[kNodes];
  __shared__ float s_u[kNodes], s_p[kNodes], s_q[kNodes];
  __shared__ int gone[kNodes];                       // drafted tokens rejected there (no draft)
  __shared__ u64 warp_total[2][kWarps], cta_total[2][kMostCluster], chunk[kMostChunks];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % size, s = blockIdx.x / size;
  if (size > 1) cluster_arrive();                    // waited for before another CTA's memory is written
  const int r0 = p.cu[s], r1 = p.cu[s + 1];
  const int n = r0 < 0 || r1 < r0 || r1 > p.n_tokens ? 0 : min(r1 - r0, p.max_q);
  const T *target = static_cast<const T *>(p.target), *draft = static_cast<const T *>(p.draft);
  if (tid < n) {
    const int up = p.parent[r0 + tid], x = p.drawn[r0 + tid];
    const bool hangs = tid > 0 && up >= 0 && up < tid, in = hangs && x >= 0 && x < p.vocab;
    s_parent[tid] = hangs ? up : -1, s_drawn[tid] = x;
    s_u[tid] = p.accept[r0 + tid];
    s_p[tid] = in ? unit(E::to(target[(r0 + up) * p.t_stride + x])) : 0.f;
    s_q[tid] = !in ? 0.f : draft ? unit(E::to(draft[(r0 + up) * p.q_stride + x])) : 1.f;
  }
  if (rank == 0)
    for (int i = tid; i < p.max_q; i += NT) p.path[(int64_t)s * p.max_q + i] = i || n == 0 ? -1 : 0;
  __syncthreads();
  if (size > 1) cluster_wait();
  if (n == 0) {
    if (rank == 0 && tid == 0) p.accepted[s] = 0, p.token[s] = -1;
    return;
  }

  int cur = 0, count = 0, j = 0, passes = 0;
  int no = 0;                                        // rejections at this node
  float2 taken = make_float2(0.f, 0.f);              // the W before each of them, added up, in two parts
  const T *prow = target + (int64_t)r0 * p.t_stride, *qrow = draft ? draft + (int64_t)r0 * p.q_stride : nullptr;
  // What the target has left of elements i and i + 1 after `no` rejections.
  auto left = [&](f2 pi, f2 qi, int i) {
    Left w{pi, f2_of(0.f, 0.f)};
    if (no == 0) return w;
    if (draft) {
      w = no == 1 ? first_left(pi, qi) : later_left(pi, qi, taken);
    } else {
      for (int k = 0; k < no; ++k) {
        if (gone[k] == i) w.h.x = 0.f;
        if (gone[k] == i + 1) w.h.y = 0.f;
      }
    }
    return w;
  };
  auto left_of = [&](float pi, float qi, int i) {    // one element, in whole 2^-60
    Parts s = {0, 0, 0};
    add_left(s, left(f2_of(pi, 0.f), f2_of(qi, 0.f), i));
    return joined(s, 2);
  };
  // Element i of the row is element i + shift of a line whose vectors of V are aligned.
  int shift = 0, per_warp = 0;
  bool both = true;                                  // the two rows are aligned alike
  auto load = [&](const T *row, int i, bool vec, float *x) {         // V elements from i on, 0 where there are none
    if (vec && i >= 0 && i + V <= p.vocab) {
      const Pack<DT, V> v = *reinterpret_cast<const Pack<DT, V> *>(row + i);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = unit(E::to(v.v[e]));
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = i + e >= 0 && i + e < p.vocab ? unit(E::to(row[i + e])) : 0.f;
    }
  };
  auto line = [&] {
    shift = (int)(reinterpret_cast<uintptr_t>(prow) / sizeof(T) % V);
    both = !qrow || (reinterpret_cast<uintptr_t>(prow) - reinterpret_cast<uintptr_t>(qrow)) % 16 == 0;
    const int chunks = ((p.vocab + shift + V - 1) / V + 31) / 32;
    per_warp = (chunks + size * kWarps - 1) / (size * kWarps);
  };
  // Sum of what is left over this lane's part of piece c.
  auto sum_of = [&](int c) {
    const int i = (c * 32 + lane) * V - shift;
    float x[V], y[V];
    load(prow, i, true, x);
    if (no && draft) load(qrow, i, both, y);
    Parts s = {0, 0, 0};
#pragma unroll
    for (int e = 0; e < V; e += 2) add_left(s, left(f2_of(x[e], x[e + 1]), no && draft ? f2_of(y[e], y[e + 1]) : f2_of(0.f, 0.f), i + e));
    return joined(s, V);
  };
  // The same over pieces c0 .. c1 - 1.  drawn: 1 with a draft and one rejection, 2 with more.
  auto sum_run = [&](int c0, int c1, auto drawn) {
    constexpr bool DRAWN = decltype(drawn)::v > 0, MANY = decltype(drawn)::v > 1;
    // pieces of whole vectors: their loads go out together, without a look at the row's ends
    const int i0 = both ? min(c1, max(c0, shift ? 1 : 0)) : c1, i1 = max(i0, min(c1, (p.vocab + shift) / (32 * V)));
    u64 all = 0;
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      if (c == i0) c = i1;
      if (c < c1) all += sum_of(c);
    }
    const Pack<DT, V> *pv = reinterpret_cast<const Pack<DT, V> *>(prow - shift) + lane;
    const Pack<DT, V> *qv = DRAWN ? reinterpret_cast<const Pack<DT, V> *>(qrow - shift) + lane : nullptr;
#pragma unroll 1
    for (int from = i0; from < i1; from += kRun) {
      const int to = min(i1, from + kRun);
      Parts s = {0, 0, 0};
      auto add = [&](int c, const Pack<DT, V> &x, const Pack<DT, V> &y) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const f2 pi = f2_of(unit(E::to(x.v[e])), unit(E::to(x.v[e + 1])));
          if constexpr (DRAWN) {
            const f2 qi = f2_of(unit(E::to(y.v[e])), unit(E::to(y.v[e + 1])));
            add_left(s, MANY ? later_left(pi, qi, taken) : first_left(pi, qi));
          } else {
            add_left(s, left(pi, f2_of(0.f, 0.f), (c * 32 + lane) * V - shift + e));
          }
        }
      };
      // one body for all: what a code this size costs is its fetch into the instruction cache
#pragma unroll 1
      for (int c = from; c < to; c += kAtOnce) {
        Pack<DT, V> x[kAtOnce], y[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          x[k] = y[k] = Pack<DT, V>{};
          if (c + k < to) {
            x[k] = pv[(c + k) * 32];
            if constexpr (DRAWN) y[k] = qv[(c + k) * 32];
          }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) add(c + k, x[k], y[k]);
      }
      all += joined(s, (unsigned)((to - from + kAtOnce - 1) / kAtOnce * kAtOnce) * V);
    }
    return all;
  };
  // A pass over the row: every CTA gets the whole sum.
  auto pass = [&] {
    line();
    const int b = passes++ & 1, c0 = (rank * kWarps + warp) * per_warp;
    u64 t = !no || !draft ? sum_run(c0, c0 + per_warp, Int<0>{}) : no == 1 ? sum_run(c0, c0 + per_warp, Int<1>{}) : sum_run(c0, c0 + per_warp, Int<2>{});
    t = warp_sum64(t);
    if (lane == 0) warp_total[b][warp] = t;
    __syncthreads();
    if (warp == 0) {
      const u64 mine = warp_sum64(lane < kWarps ? warp_total[b][lane] : 0);
      if (lane < size) store_in(&cta_total[b][rank], lane, mine);
      __syncwarp();
    }
    if (size > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    u64 all = 0;
    for (int k = 0; k < size; ++k) all += cta_total[b][k];
    return all;
  };
  auto next_child = [&] {                            // of cur, after j; n if there is none
    for (int k = (j + 1) & ~31; k < n; k += 32) {
      const unsigned is = __ballot_sync(0xffffffffu, k + lane > j && k + lane < n && s_parent[k + lane] == cur);
      if (is) return k + __ffs(is) - 1;
    }
    return n;
  };

  u64 all = 0;                                       // sum of what is left, where `no` > 0
  float2 whole_mass = make_float2(1.f, 0.f);         // the same, in two parts
  bool behind = false;                               // the last pass's parts are not those of `all`
  while ((j = next_child()) < n) {
    // u q W < w; both sides in two parts, exact before the first rejection (W = 1 and w = p)
    const float2 uq = product(s_u[j], s_q[j] * kUp);
    float2 need = uq, has = make_float2(s_p[j] * kUp, 0.f);
    if (no) {
      const Left w = left(f2_of(s_p[j], 0.f), f2_of(s_q[j], 0.f), s_drawn[j]);
      has = make_float2(w.h.x * kUp, w.l.x * kUp);
      need = product(uq.x, whole_mass.x);
      need.y += uq.x * whole_mass.y + uq.y * whole_mass.x;
      const float up = need.x + need.y;
      need = make_float2(up, need.y - (up - need.x));
    }
    if (need.x < has.x || (need.x == has.x && need.y < has.y)) {
      cur = j, ++count, no = 0, behind = false, whole_mass = make_float2(1.f, 0.f), taken = make_float2(0.f, 0.f);
      if (tid == 0) s_path[count] = j;
      prow = target + (int64_t)(r0 + cur) * p.t_stride;
      if (draft) qrow = draft + (int64_t)(r0 + cur) * p.q_stride;
      continue;
    }
    const u64 was = no && !draft ? left_of(s_p[j], s_q[j], s_drawn[j]) : 0;
    if (draft) {
      const float h = taken.x + whole_mass.x, z = h - taken.x;       // two parts added, then put in order
      const float l = (taken.x - (h - z)) + (whole_mass.x - z) + (taken.y + whole_mass.y);
      taken = make_float2(h + l, l - ((h + l) - h));
    } else {
      __syncthreads();                               // the list of the node before has been read
      if (tid == 0) gone[no] = s_drawn[j];
      __syncthreads();
    }
    if (no++ == 0 || draft) all = pass();
    else all -= was, behind = true;                  // a given token takes its own share along
    whole_mass = in_two(all);
  }
  if (no == 0 || behind) all = pass();
  if (all == 0 && no) {                              // nothing is left: the target itself
    no = 0;
    all = pass();
  }
  if (rank == 0) {
    if (tid == 0) p.accepted[s] = count;
    for (int i = 1 + tid; i <= count; i += NT) p.path[(int64_t)s * p.max_q + i] = s_path[i];
  }
  if (all == 0) {
    if (rank == 0 && tid == 0) p.token[s] = -1;
    return;
  }
  // ---- the first element whose sum up to it is above u times the whole ----
  const float u = p.sample[s];
  const u64 part = !(u > 0.f) ? 0 : u >= 1.f ? ~0ull : __float2ull_rz(u * 0x1p64f);
  u64 rest = __umul64hi(part, all);                  // below `all`
  const int b = (passes - 1) & 1;
  for (int k = 0; k < rank; ++k) {
    const u64 t = cta_total[b][k];
    if (rest < t) return;                            // in a CTA before this one
    rest -= t;
  }
  if (rest >= cta_total[b][rank]) return;
  int w = 0;
  while (w < kWarps - 1 && rest >= warp_total[b][w]) rest -= warp_total[b][w++];
  const int c0 = (rank * kWarps + w) * per_warp;
  for (int k = warp; k < per_warp; k += kWarps) {
    const u64 t = warp_sum64(sum_of(c0 + k));
    if (lane == 0) chunk[k] = t;
  }
  __syncthreads();
  if (warp) return;
  int k = 0;
  while (k < per_warp - 1 && rest >= chunk[k]) rest -= chunk[k++];
  const u64 own = sum_of(c0 + k);
  u64 upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  const int first = __ffs(__ballot_sync(0xffffffffu, upto > rest)) - 1;
  if (lane == first) {
    rest -= upto - own;
    const int i = ((c0 + k) * 32 + lane) * V - shift;
    float x[V], y[V];
    load(prow, i, true, x);
    if (no && draft) load(qrow, i, both, y);
    int e = 0;
#pragma unroll
    for (int m = 0; m < V; ++m) {
      const u64 t = left_of(x[m], no && draft ? y[m] : 0.f, i + m);
      if (e == m && rest >= t) rest -= t, ++e;
    }
    p.token[s] = min(i + e, p.vocab - 1);
  }
}

template <int DT, int NT>
cudaError_t launch_verify(const VerifyParams &p, int size, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.n_seqs * size));
  cfg.blockDim = dim3(NT);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_verify<DT, NT>, p, size);
}

// CTAs of a sequence: while all are on the SMs at once and a warp has two pieces of a row.
// 512 threads where that leaves SMs free, else 256, of which an SM holds four.
template <int DT>
cudaError_t launch_verify(const VerifyParams &p, cudaStream_t s) {
  const int sms = std::max(1, pi::current_sms());
  const int64_t pieces = ((int64_t)p.vocab * (int)sizeof(typename Elem<DT>::T) + 511) / 512;
  int size = 1;
  while (size < kMostCluster && (int64_t)p.n_seqs * size * 2 <= 4 * sms && pieces >= 4 * size * 8) size *= 2;
  return (int64_t)p.n_seqs * size <= sms && pieces >= 2 * size * 16 ? launch_verify<DT, 512>(p, size, s) : launch_verify<DT, 256>(p, size, s);
}

pi_status check_nodes(int n_seqs, int n_tokens, int max_q, const int32_t *parent, const int32_t *cu) {
  if (n_seqs < 0 || n_tokens < 0 || n_seqs > (1 << 20) || n_tokens > (1 << 28))
    return pi::fail(PI_ERR_INVALID_ARG, "n_seqs=%d or n_tokens=%d out of range", n_seqs, n_tokens);
  if (max_q < 1 || max_q > PI_MAX_TREE) return pi::fail(PI_ERR_UNSUPPORTED, "max_q=%d: 1 to %d", max_q, PI_MAX_TREE);
  if (n_seqs && (!cu || !pi::aligned_to(cu, 4))) return pi::fail(PI_ERR_INVALID_ARG, "cu must be non-NULL and 4-byte aligned");
  if (n_seqs && n_tokens && (!parent || !pi::aligned_to(parent, 4)))
    return pi::fail(PI_ERR_INVALID_ARG, "parent must be non-NULL and 4-byte aligned");
  return PI_OK;
}

}  // namespace

extern "C" {

pi_status pi_draft_tree(const int32_t *parent, const int32_t *cu, int32_t n_seqs, int32_t n_tokens, int32_t max_q,
                        int32_t *mask, int32_t *depth, void *stream) {
  pi::clear_error();
  const pi_status st = check_nodes(n_seqs, n_tokens, max_q, parent, cu);
  if (st != PI_OK) return st;
  if (!pi::aligned_to(mask, 4) || !pi::aligned_to(depth, 4))
    return pi::fail(PI_ERR_INVALID_ARG, "mask and depth must be 4-byte aligned");
  if (n_seqs == 0 || n_tokens == 0 || (!mask && !depth)) return PI_OK;
  const TreeParams p{parent, cu, n_seqs, n_tokens, max_q, (max_q + 31) / 32, mask, depth};
  k_draft_tree<<<n_seqs, p.words * 32, 0, static_cast<cudaStream_t>(stream)>>>(p);
  PI_TRY_CUDA(cudaGetLastError());
  return PI_OK;
}

pi_status pi_verify_draft(const void *target, int64_t target_stride, const void *draft, int64_t draft_stride, int32_t dtype,
                          int32_t vocab, const int32_t *drawn, const int32_t *parent, const int32_t *cu, int32_t n_seqs,
                          int32_t n_tokens, int32_t max_q, const float *accept, const float *sample, int32_t *accepted,
                          int32_t *path, int32_t *token, void *stream) {
  pi::clear_error();
  const pi_status st = check_nodes(n_seqs, n_tokens, max_q, parent, cu);
  if (st != PI_OK) return st;
  if (!pi::dtype_ok(dtype)) return pi::fail(PI_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (vocab < 1) return pi::fail(PI_ERR_INVALID_ARG, "vocab=%d: at least 1", vocab);
  if (vocab > kMostVocab) return pi::fail(PI_ERR_UNSUPPORTED, "vocab=%d: up to %d", vocab, kMostVocab);
  if (n_seqs == 0) return PI_OK;
  const int e = pi::dtype_size(dtype);
  if (!accepted || !path || !token || !sample || !pi::aligned_to(accepted, 4) || !pi::aligned_to(path, 4) ||
      !pi::aligned_to(token, 4) || !pi::aligned_to(sample, 4))
    return pi::fail(PI_ERR_INVALID_ARG, "accepted, path, token and sample must be non-NULL and 4-byte aligned");
  if (n_tokens && (!target || !drawn || !accept || !pi::aligned_to(target, e) || !pi::aligned_to(draft, e) ||
                   !pi::aligned_to(drawn, 4) || !pi::aligned_to(accept, 4)))
    return pi::fail(PI_ERR_INVALID_ARG, "target, drawn and accept must be non-NULL, arrays aligned to their type");
  if (target_stride < vocab || (draft && draft_stride < vocab))
    return pi::fail(PI_ERR_INVALID_ARG, "rows lie in one another: strides %lld and %lld, vocab %d", (long long)target_stride,
                    (long long)draft_stride, vocab);
  const VerifyParams p{target, draft, target_stride, draft_stride, vocab, n_seqs, n_tokens, max_q, drawn, parent, cu, accept, sample,
                       accepted, path, token};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PI_TRY_CUDA(dtype == PI_DT_F16    ? launch_verify<PI_DT_F16>(p, s)
              : dtype == PI_DT_BF16 ? launch_verify<PI_DT_BF16>(p, s)
                                    : launch_verify<PI_DT_F32>(p, s));
  return PI_OK;
}

}  // extern "C"
