// Rotation of pairs of a head's elements by a position's angles (pi_rope.cu,
// pi_append.cu).
//
//   a' = m (a cos t - b sin t),  b' = m (a sin t + b cos t),  t = position * frequency
//
// Angles.  A frequency is kept as a whole number of 2^-64 turns a position, so the
// product with a position modulo 2^64 is the angle modulo a turn, exactly, however
// far the position; what is left of it beside the nearest quarter turn, 1/4 of a half turn at
// most, is cut to whole 2^-31 half turns (1.5e-9 of an angle, however small) and rounded to
// binary32 (2^-27 half turns at most: 2.4e-8).
#pragma once

#include "pi_ops.cuh"

namespace pi {

pi_status check_rotary(const pi_rotary *r, int head_dim);

}  // namespace pi

namespace pidev {

// m cos t and m sin t.
__device__ __forceinline__ float2 rope_angle(uint64_t turn, int64_t pos, float m) {
  const uint64_t t = turn * (uint64_t)pos;
  const uint64_t q = (t + (1ull << 61)) >> 62;                       // the nearest quarter
  const float r = (float)(int)((int64_t)(t - (q << 62)) >> 32) * 0x1p-31f;     // half turns, up to 1/4
  float s, c;
  sincospif(r, &s, &c);
  s *= m, c *= m;
  switch ((int)q & 3) {
    case 0: return make_float2(c, s);
    case 1: return make_float2(-s, c);
    case 2: return make_float2(-c, -s);
    default: return make_float2(s, -c);
  }
}

// Cosines and sines of a unit of 2 V elements (V pairs), as the lanes load them:
// two pairs to a float4 (cos, cos, sin, sin), the float4s of one place in their
// units side by side, so that neighbouring lanes meet neighbouring banks.
template <int V>
__device__ __forceinline__ void rope_put(float4 *table, int units, int freq, float2 cs) {
  float *at = reinterpret_cast<float *>(table + (freq % V / 2) * units + freq / V) + freq % 2;
  at[0] = cs.x, at[2] = cs.y;
}
// v: 2 V elements; the first V and the last V make pairs, or neighbours do.
template <int V, bool HALF>
__device__ __forceinline__ void rope_turn(f2 *v, const float4 *at, int units) {
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    const float4 cs = at[k * units];
    if constexpr (HALF) {
      const f2 a = v[k], b = v[V / 2 + k], c = f2_of(cs.x, cs.y), s = f2_of(cs.z, cs.w);
      v[k] = f2_fma(a, c, f2_mul(b, f2_of(-cs.z, -cs.w)));
      v[V / 2 + k] = f2_fma(a, s, f2_mul(b, c));
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const f2 x = v[2 * k + e];
        const float c = e ? cs.y : cs.x, s = e ? cs.w : cs.z;
        v[2 * k + e] = f2_fma(f2_of(x.x, x.x), f2_of(c, s), f2_mul(f2_of(x.y, x.y), f2_of(-s, c)));
      }
    }
  }
}

}  // namespace pidev
