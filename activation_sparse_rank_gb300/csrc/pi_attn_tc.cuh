// Pieces that the tcgen05 kernels of attention share (pi_attn_tc.cu, pi_attn_tree.cu):
// tiles, descriptors, products, accesses to TMEM.
#pragma once

#include "pi_attn.cuh"

namespace attn {

constexpr int kRows = kTcRows, kHalf = 128, kKeys = 128, kBlocks = kKeys / PI_KV_BLOCK;
constexpr int kThreads = 512;      // four warpgroups: register shares are set for each
constexpr int kStages = 3;         // of codes, K and V of a tile in turn
// From P_j = 0, so x_j + ev_j < R - 126, and ev_j >= ev - kFar for every ev so far it
// follows that x_j is 38 or more below the largest x: its weight is nothing.
constexpr int kFar = 94;
// Tiles whose scales and NaN are kept.  Copies run at most 5 tiles ahead of the first
// softmax group, which every unit waits for; the second has no part in units of one
// row tile, so the copies wait until it has read what it needs of a unit's last three.
constexpr int kScaleRing = 8;

// Shared-memory matrix descriptor, 128-byte swizzle: its low word holds the
// address (and lbo), so a step of `bytes` adds bytes / 16 to it.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr & 0x3FFFF) >> 4 | ((lbo >> 4) & 0x3FFF) << 16; }
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;        // groups of 8 rows 1024 bytes apart
// kind::f16, fp16 operands, binary32 sums, M = 128
__device__ __forceinline__ uint32_t idesc(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kHalf >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n mov.b64 y, {%2, %5};\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHi));
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
        "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
// The loads above are complete; v's uses stay behind this.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(float *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int j = 0; j < N; ++j) asm volatile("" : "+f"(v[j]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16-byte chunk c of 128-byte row r in a 128-byte-swizzled slab.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
// Chunk c (16 codes) of row r of a tile of codes, as the tile copies swizzle it (rows of 96 are not).
template <int D>
__device__ __forceinline__ uint32_t code_at(int r, int c) {
  return D == 64 ? (uint32_t)(r * 64 + ((c ^ (r >> 1 & 3)) << 4)) : D == 96 ? (uint32_t)(r * 96 + c * 16) : sw128(r, c);
}

template <int D>
struct Smem {                       // byte offsets from a 1024-byte boundary
  static constexpr int SLABS = (D + 63) / 64, SLAB = 128 * 128, TILE = SLABS * SLAB;   // a slab: 64 fp16 dims of 128 rows
  static constexpr int Q = 0, K = Q + 2 * TILE, V = K + 2 * TILE, C = V + TILE, BYTES = C + kStages * 128 * D;
};

}  // namespace attn
