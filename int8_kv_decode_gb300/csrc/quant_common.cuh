// Rows of 32- or 16-bit elements in vectors, and their 8-bit codes under a scale.
#pragma once

#include <type_traits>

#include "device_common.cuh"

namespace kattn {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
}

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T v[VEC];
};
template <int VEC>
struct alignas(VEC) Codes {
  uint8_t v[VEC];
};

// Two elements at a time: a 16-bit pair takes one instruction to pack, and one each
// to unpack.
__device__ __forceinline__ float2 pair_f32(__nv_bfloat162 v) {
  const uint32_t b = *reinterpret_cast<const uint32_t*>(&v);
  return make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_f32(__half2 v) { return __half22float2(v); }
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Vec<T, VEC>& v, float (&f)[VEC]) {
  if constexpr (sizeof(T) == 4 || VEC == 1) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = to_f32(v.v[e]);
  } else {
    using P = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 x = pair_f32(reinterpret_cast<const P*>(v.v)[e / 2]);
      f[e] = x.x;
      f[e + 1] = x.y;
    }
  }
}
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> pack(const float (&f)[VEC]) {
  Vec<T, VEC> v;
  if constexpr (sizeof(T) == 4 || VEC == 1) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v.v[e] = from_f32<T>(f[e]);
  } else if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2)
      reinterpret_cast<__half2*>(v.v)[e / 2] = __floats2half2_rn(f[e], f[e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 2)
      reinterpret_cast<__nv_bfloat162*>(v.v)[e / 2] = __floats2bfloat162_rn(f[e], f[e + 1]);
  }
  return v;
}

// The largest of values >= 0 over the warp: their bits are ordered as integers.
__device__ __forceinline__ float warp_max_abs(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// Low bytes of four words as one word.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040u), __byte_perm(c, d, 0x0040u), 0x5410u);
}

__device__ __forceinline__ uint8_t code_of(float z, float s0, bool e4m3) {
  if (s0 == 0.0f) return 0;
  const float u = __fdiv_rn(z, s0);
  if (e4m3) return __nv_cvt_float_to_fp8(u, __NV_SATFINITE, __NV_E4M3);
  return (uint8_t)(int8_t)max(-127, min(127, __float2int_rn(u)));
}

// Codes of VEC elements without a division each.  t = z * (1 / s0) differs from the
// quotient z / s0, rounded to float32, by at most 2 float32 steps (1 / s0 and the
// product are off by half a step of theirs each, the quotient by half a step), so
// the code of t is the quotient's unless a rounding border lies that near:
//   int8  borders n + 1/2: 2 steps of |t| <= 127 are below 1.6e-5, so |t - rint(t)|
//         up to 0.4999 is safe;
//   e4m3  borders at the middle of two values of 4 significant bits: the low 20
//         bits of t's mantissa are then 0x80000; further than 4 steps is safe.
//         Below 2^-6 the grid is coarser: those divide.
// Elements near a border divide, and all of them where `divide` is true: with s0 whose
// reciprocal may overflow, and with elements that are not finite, which become +-127 (NaN: 0)
// or saturate (NaN: NaN).
__device__ __forceinline__ bool scale_divides(float s0) { return !(s0 > 1e-30f); }
template <int VEC>
__device__ __forceinline__ Codes<VEC> codes_of(const float (&z)[VEC], float s0, float inv, bool e4m3, bool divide) {
  Codes<VEC> c;
  bool near = divide;
  if (!e4m3) {
    const float magic = 12582912.0f;              // 1.5 * 2^23: the sum's low byte is rint(t)
    float far = 0.0f;
    uint32_t y[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float t = __fmul_rn(z[e], inv), u = __fadd_rn(t, magic);
      far = fmaxf(far, fabsf(__fsub_rn(t, __fsub_rn(u, magic))));
      y[e] = __float_as_uint(u);
    }
    if constexpr (VEC >= 4) {
#pragma unroll
      for (int e = 0; e < VEC; e += 4)
        reinterpret_cast<uint32_t*>(c.v)[e / 4] = low_bytes(y[e], y[e + 1], y[e + 2], y[e + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) c.v[e] = (uint8_t)y[e];
    }
    near |= !(far <= 0.4999f);
  } else {
    float t[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      t[e] = __fmul_rn(z[e], inv);
      near |= ((__float_as_uint(t[e]) & 0xfffffu) - 0x7fffcu) <= 8u;
      near |= fabsf(t[e]) < 0.015625f && t[e] != 0.0f;
    }
    if constexpr (VEC >= 4) {
#pragma unroll
      for (int e = 0; e < VEC; e += 2)
        reinterpret_cast<__nv_fp8x2_storage_t*>(c.v)[e / 2] =
            __nv_cvt_float2_to_fp8x2(make_float2(t[e], t[e + 1]), __NV_SATFINITE, __NV_E4M3);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) c.v[e] = __nv_cvt_float_to_fp8(t[e], __NV_SATFINITE, __NV_E4M3);
    }
  }
  if (near) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) c.v[e] = code_of(z[e], s0, e4m3);
  }
  return c;
}

}  // namespace
}  // namespace kattn
