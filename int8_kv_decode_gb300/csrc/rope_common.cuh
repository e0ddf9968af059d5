// Rotation of a head's channels by their position's angles: sixteen lanes a head, eight
// channels a lane in two runs of four, so that both channels of a pair are the lane's.
#pragma once

#include "decode_split.cuh"      // programmatic launches
#include "quant_common.cuh"

namespace kattn {
namespace {

// A load, after griddep_wait, of what a kernel before may have written while this one had
// started: a plain one, as the read-only path takes its data for constant since the start.
template <typename T>
__device__ __forceinline__ T ld_fresh(const T* p) {
  return *p;
}

// Where the two runs of lane l (of 16) begin, and whether its channels are rotated.
//   half layout: channel i < half turns with channel i + half, by angle i: the runs are
//     4l and 4l + half.  half is a multiple of 4; the lanes past the last pair hold the
//     channels behind 2 half.
//   interleaved: channels 2i and 2i + 1 turn by angle i: eight channels in a row.
// In both layouts the lane's angles are 4l .. 4l + 3.
struct Runs {
  int a, b;
  bool turns;
};
template <bool kInter>
__device__ __forceinline__ Runs lane_runs(int half, int l) {
  const int lanes = half >> 2;
  Runs r;
  r.turns = l < lanes;
  r.a = kInter || !r.turns ? 8 * l : 4 * l;       // (8 lanes + 8 (l - lanes) behind the last pair)
  r.b = kInter || !r.turns ? 8 * l + 4 : 4 * l + half;
  return r;
}

struct Angles {
  float2 a[4];                                    // (cos, sin)
};
__device__ __forceinline__ Angles load_angles(const float* table, int position, int half, int l) {
  const float4* at = reinterpret_cast<const float4*>(table + (int64_t)position * half * 2) + 2 * l;
  const float4 x = ld_fresh(at), y = ld_fresh(at + 1);
  return {{make_float2(x.x, x.y), make_float2(x.z, x.w), make_float2(y.x, y.y), make_float2(y.z, y.w)}};
}

// A pair (x, y) turned.  Each product and sum is rounded on its own, so that the result,
// and the 8-bit codes made of it, are those of the formula in float32.
__device__ __forceinline__ void turn_pair(float& x, float& y, float2 a) {
  const float u = __fsub_rn(__fmul_rn(x, a.x), __fmul_rn(y, a.y));
  y = __fadd_rn(__fmul_rn(y, a.x), __fmul_rn(x, a.y));
  x = u;
}
template <bool kInter>
__device__ __forceinline__ void turn(const Angles& t, float (&a)[4], float (&b)[4]) {
  if constexpr (kInter) {
    turn_pair(a[0], a[1], t.a[0]);
    turn_pair(a[2], a[3], t.a[1]);
    turn_pair(b[0], b[1], t.a[2]);
    turn_pair(b[2], b[3], t.a[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) turn_pair(a[e], b[e], t.a[e]);
  }
}

// Heads of one row, turned by a warp: the heads 2 i + (lane / 16) below n, all loaded
// before the first is turned.  x, y: the row's first of these heads.  know: its position
// has angles (else NaN).
constexpr int kTurnHeads = 8;
template <typename T, typename O, bool kInter, typename Position>
__device__ __forceinline__ void turn_heads(const T* x, O* y, int n, const float* table, int half, int lane,
                                           Position position) {
  const int l = lane & 15, side = lane >> 4;
  const Runs r = lane_runs<kInter>(half, l);
  Vec<T, 4> ra[kTurnHeads / 2], rb[kTurnHeads / 2];
#pragma unroll
  for (int i = 0; i < kTurnHeads / 2; ++i)
    if (2 * i + side < n) {
      ra[i] = *reinterpret_cast<const Vec<T, 4>*>(x + (2 * i + side) * kD + r.a);
      rb[i] = *reinterpret_cast<const Vec<T, 4>*>(x + (2 * i + side) * kD + r.b);
    }
  bool know;
  const int at = position(know);                  // (its loads go beside those of the row)
  if (at < 0) return;
  Angles t;
  if (r.turns) t = load_angles(table, at, half, l);
#pragma unroll
  for (int i = 0; i < kTurnHeads / 2; ++i) {
    if (2 * i + side >= n) break;
    float a[4], b[4];
    unpack(ra[i], a);
    unpack(rb[i], b);
    if (r.turns) turn<kInter>(t, a, b);
    if (!know) a[0] = a[1] = a[2] = a[3] = b[0] = b[1] = b[2] = b[3] = __int_as_float(0x7fc00000);
    *reinterpret_cast<Vec<O, 4>*>(y + (2 * i + side) * kD + r.a) = pack<O, 4>(a);
    *reinterpret_cast<Vec<O, 4>*>(y + (2 * i + side) * kD + r.b) = pack<O, 4>(b);
  }
}

}  // namespace
}  // namespace kattn
