// Rotation of a head's channels by their position's angles: four channels a lane, a
// head of 128 channels a warp.
#pragma once

#include "quant_common.cuh"

namespace kattn {
namespace {

// The angles of a lane's channels 4 lane .. 4 lane + 3, for one position.
//   half layout: channel i < half turns with channel i + half, by angle i.  half is a
//     multiple of 4, so the partner's four channels are those of one lane.
//   interleaved: channels 2i and 2i + 1 turn by angle i.
struct Turn {
  float c[4], s[4];
  int partner;                    // lane of the partner's channels (half layout)
  bool turns;                     // these channels are rotated
};
template <bool kInter>
__device__ __forceinline__ Turn load_turn(const float* __restrict__ table, int position, int half, int lane) {
  Turn t;
  const int lanes = half >> 2;                    // that hold the first of each pair (half layout)
  t.turns = lane < 2 * lanes;
  t.partner = lane;
  const float* at = table + (int64_t)position * half * 2;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    t.c[e] = 1.0f;
    t.s[e] = 0.0f;
  }
  if (!t.turns) return t;
  if constexpr (kInter) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(at) + lane);
    t.c[0] = t.c[1] = a.x;
    t.c[2] = t.c[3] = a.z;
    t.s[0] = -a.y;
    t.s[1] = a.y;
    t.s[2] = -a.w;
    t.s[3] = a.w;
  } else {
    const bool first = lane < lanes;
    t.partner = first ? lane + lanes : lane - lanes;
    const float4* v = reinterpret_cast<const float4*>(at) + 2 * (first ? lane : lane - lanes);
    const float4 a = __ldg(v), b = __ldg(v + 1);
    t.c[0] = a.x;
    t.c[1] = a.z;
    t.c[2] = b.x;
    t.c[3] = b.z;
    t.s[0] = first ? -a.y : a.y;
    t.s[1] = first ? -a.w : a.w;
    t.s[2] = first ? -b.y : b.y;
    t.s[3] = first ? -b.w : b.w;
  }
  return t;
}

// f: the lane's channels, turned in place.  Each product and sum is rounded on its
// own (a - b s is a + b (-s) to the bit), so that the result, and the 8-bit codes
// made of it, are those of the formula in float32.
template <bool kInter>
__device__ __forceinline__ void turn(const Turn& t, float (&f)[4]) {
  float o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = kInter ? f[e ^ 1] : __shfl_sync(0xffffffffu, f[e], t.partner);
  if (!t.turns) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = __fadd_rn(__fmul_rn(f[e], t.c[e]), __fmul_rn(o[e], t.s[e]));
}

}  // namespace
}  // namespace kattn
