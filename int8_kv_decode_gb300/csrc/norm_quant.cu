// Residual addition, root-mean-square norm and 8-bit quantization of rows.
//
//   h = x (+ residual, rounded to its type),  z = h * weight
//   codes = round(z / s0),  s0 = max |z| / 127 (or 448)
//   scale = s0 / sqrt(mean(h^2) + eps)
// The factor 1 / rms is the same for the whole row, so it goes into the scale:
// the codes depend on z alone, and one pass gives both max |z| and sum h^2.
//
// Bound by memory: an element is read once (twice with a residual), written once
// to the residual and once as a byte.  A row stays in registers between the pass
// that reduces it and the codes.  8192 rows of 4096 bf16 with a residual (235 MB,
// 35 us at the measured copy rate) take 47 us, 5.0 TB/s; what keeps it from the
// rest is issue (65% busy, 31 instructions an element).  A thread holds two vectors
// of 16 bytes (one: 61 us, four: 63 us).  16 rows of 2048 take 3.3 us: latency.
#include <algorithm>
#include <type_traits>

#include "device_common.cuh"
#include "ops_internal.cuh"

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
// Elements near a border, and s0 whose reciprocal may overflow, divide.
template <int VEC>
__device__ __forceinline__ Codes<VEC> codes_of(const float (&z)[VEC], float s0, float inv, bool e4m3) {
  Codes<VEC> c;
  bool near = !(s0 > 1e-30f);
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

constexpr int kMaxThreads = 512;                  // 128 registers a thread

// TPR threads hold a row, NV vectors of VEC elements each; a block of at least 256
// threads takes blockDim / TPR rows at a time, in a grid stride, and keeps its part
// of the weight.  TPR and NV go by d and VEC, and VEC by d and the alignment of pointers
// and strides (launch_type): a row's codes depend on nothing else, and its scale, whose sum
// of squares has an order that follows them, not on how many rows there are.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormParams p, const int tpr, const bool e4m3) {
  __shared__ float s_sum[2][32], s_max[2][32];
  using V = Vec<T, VEC>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
  const int rows_here = blockDim.x / tpr, warps_row = tpr / 32, warp0 = sub * warps_row;
  const bool grouped = p.group != p.d;
  const float top = e4m3 ? 448.0f : 127.0f;
  // (elements past d are zero throughout, and so is the weight's part of them)
  V w[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * tpr + t) * VEC;
    w[v] = V{};
    if (c < p.d) w[v] = *reinterpret_cast<const V*>(static_cast<const T*>(p.weight) + c);
  }
  int par = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rows_here; row0 < p.rows;
       row0 += (int64_t)gridDim.x * rows_here, par ^= 1) {
    const int64_t row = row0 + sub;
    const bool in = row < p.rows;
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
    const T* res = static_cast<const T*>(p.residual) + row * p.res_stride;
    T* res_out = static_cast<T*>(p.residual_out) + row * p.res_out_stride;
    V xv[NV], rv[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * tpr + t) * VEC;
      xv[v] = V{};
      if (in && c < p.d) xv[v] = *reinterpret_cast<const V*>(x + c);
      if (p.residual) {
        rv[v] = V{};
        if (in && c < p.d) rv[v] = *reinterpret_cast<const V*>(res + c);
      }
    }
    float z[NV][VEC], sum = 0.0f, amax = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * tpr + t) * VEC;
      float h[VEC], f[VEC];
      unpack(xv[v], h);
      if (p.residual) {
        unpack(rv[v], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = __fadd_rn(h[e], f[e]);
        rv[v] = pack<T, VEC>(h);
        if (in && c < p.d) *reinterpret_cast<V*>(res_out + c) = rv[v];
        unpack(rv[v], h);
      }
      unpack(w[v], f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        sum = __fmaf_rn(h[e], h[e], sum);
        z[v][e] = __fmul_rn(h[e], f[e]);
        amax = fmaxf(amax, fabsf(z[v][e]));
      }
    }
    sum = warp_sum(sum);
    if (!grouped) amax = warp_max_abs(amax);
    // the factor 1 / rms is needed where a scale is written: the row's first warp, or
    // all of them (grouped)
    const bool scales_here = grouped || t < 32;
    if (warps_row > 1) {
      if (lane == 0) {
        s_sum[par][warp] = sum;
        s_max[par][warp] = amax;
      }
      __syncthreads();                            // (the other parity's values are read by then)
      if (scales_here) sum = warp_sum(lane < warps_row ? s_sum[par][warp0 + lane] : 0.0f);
      if (!grouped) amax = warp_max_abs(lane < warps_row ? s_max[par][warp0 + lane] : 0.0f);
    }
    float r = 0.0f;
    if (scales_here)
      r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)p.d), p.eps)));
    float s0 = 0.0f, inv = 0.0f;
    if (!grouped) {
      s0 = __fdiv_rn(amax, top);
      inv = __frcp_rn(s0);
      if (in && t == 0) p.scales[row] = __fmul_rn(s0, r);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * tpr + t) * VEC;
      if (grouped) {                              // 128 / VEC lanes share a scale (VEC = 1: 4 warps)
        constexpr int kLanes = VEC == 1 ? 32 : 128 / VEC;
        float a = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) a = fmaxf(a, fabsf(z[v][e]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        s0 = __fdiv_rn(a, top);
        inv = __frcp_rn(s0);
        if (in && c < p.d && c % 128 == 0) p.scales[row * (p.d / 128) + c / 128] = __fmul_rn(s0, r);
      }
      const Codes<VEC> out = codes_of<VEC>(z[v], s0, inv, e4m3);
      if (in && c < p.d) *reinterpret_cast<Codes<VEC>*>(p.codes + row * p.d + c) = out;
    }
  }
}

constexpr int kThreads = 256;

// Rows that norm_kernel's registers cannot hold, and 128-channel groups that its
// vectors do not line up with: one block per row, read again for the codes, with loads of
// single elements.  8192 rows of 4096 bf16 with a residual, an odd stride and 128-channel
// groups 108 us (53 us for aligned rows with one scale, 62 us with groups, each from a cold
// L2; an odd stride without groups, norm_kernel with VEC = 1, 115 us); 1677 rows of 20000
// 152 us (35 us of bytes).  Bound by those loads.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_long_kernel(const NormParams p, const bool e4m3) {
  __shared__ float s_sum[kThreads / 32], s_max[kThreads / 32];
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.res_stride : nullptr;
  T* res_out = p.residual ? static_cast<T*>(p.residual_out) + row * p.res_out_stride : nullptr;
  const T* w = static_cast<const T*>(p.weight);
  const T* h = res ? res_out : x;
  const bool grouped = p.group != p.d;
  float sum = 0.0f, amax = 0.0f;
  for (int c = threadIdx.x; c < p.d; c += kThreads) {
    float v = to_f32(x[c]);
    if (res) {
      const T t = from_f32<T>(__fadd_rn(v, to_f32(res[c])));
      res_out[c] = t;
      v = to_f32(t);
    }
    sum = __fmaf_rn(v, v, sum);
    amax = fmaxf(amax, fabsf(__fmul_rn(v, to_f32(w[c]))));
  }
  sum = warp_sum(sum);
  amax = warp_max(amax);
  if (lane == 0) {
    s_sum[warp] = sum;
    s_max[warp] = amax;
  }
  __syncthreads();                                // (and residual_out is written)
  sum = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) {
    sum += s_sum[i];
    amax = fmaxf(amax, s_max[i]);
  }
  const float top = e4m3 ? 448.0f : 127.0f;
  const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)p.d), p.eps)));
  if (!grouped) {
    const float s0 = __fdiv_rn(amax, top);
    for (int c = threadIdx.x; c < p.d; c += kThreads)
      p.codes[row * p.d + c] = code_of(__fmul_rn(to_f32(h[c]), to_f32(w[c])), s0, e4m3);
    if (threadIdx.x == 0) p.scales[row] = __fmul_rn(s0, r);
    return;
  }
  for (int g = warp; g < p.d / 128; g += kThreads / 32) {   // a warp per group
    float z[4], a = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = g * 128 + 32 * e + lane;
      z[e] = __fmul_rn(to_f32(h[c]), to_f32(w[c]));
      a = fmaxf(a, fabsf(z[e]));
    }
    const float s0 = __fdiv_rn(warp_max(a), top);
#pragma unroll
    for (int e = 0; e < 4; ++e) p.codes[row * p.d + g * 128 + 32 * e + lane] = code_of(z[e], s0, e4m3);
    if (lane == 0) p.scales[row * (p.d / 128) + g] = __fmul_rn(s0, r);
  }
}

int multiprocessors() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    sms = 1;
  return sms;
}

template <typename T, int VEC>
cudaError_t launch_vec(const NormParams& p, bool e4m3, cudaStream_t stream) {
  constexpr int kShare = 2;                       // vectors a thread, as far as a block reaches
  const int vecs = (p.d + VEC - 1) / VEC;
  int tpr = 32;
  while (tpr < kMaxThreads && kShare * tpr < vecs) tpr *= 2;
  const int nv = (vecs + tpr - 1) / tpr;
  const int threads = std::max(tpr, kThreads), rows_here = threads / tpr;
  const int64_t blocks = (p.rows + rows_here - 1) / rows_here;
  const unsigned grid =
      (unsigned)std::min<int64_t>(blocks, (int64_t)multiprocessors() * (2048 / threads));   // (as many as fit)
  if (nv <= 1) norm_kernel<T, VEC, 1><<<grid, threads, 0, stream>>>(p, tpr, e4m3);
  else if (nv <= 2) norm_kernel<T, VEC, 2><<<grid, threads, 0, stream>>>(p, tpr, e4m3);
  else if (nv <= 4 || VEC == 8) norm_kernel<T, VEC, 4><<<grid, threads, 0, stream>>>(p, tpr, e4m3);
  else norm_kernel<T, VEC, VEC == 8 ? 4 : 8><<<grid, threads, 0, stream>>>(p, tpr, e4m3);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const NormParams& p, bool e4m3, cudaStream_t stream) {
  constexpr int kVec = 16 / (int)sizeof(T);
  auto fits = [](const void* q, int64_t stride) {
    return (uintptr_t)q % 16 == 0 && stride % kVec == 0;
  };
  const bool vec = p.d % kVec == 0 && fits(p.x, p.x_stride) && fits(p.weight, 0) &&
                   (uintptr_t)p.codes % kVec == 0 &&
                   (!p.residual || (fits(p.residual, p.res_stride) && fits(p.residual_out, p.res_out_stride)));
  constexpr int kMost = kMaxThreads * 32;         // 32 elements a thread (8 without vectors)
  if (vec && p.d <= kMost) return launch_vec<T, kVec>(p, e4m3, stream);
  if (p.group == p.d && p.d <= kMost / 4) return launch_vec<T, 1>(p, e4m3, stream);
  norm_long_kernel<T><<<(unsigned)p.rows, kThreads, 0, stream>>>(p, e4m3);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm_quant(const NormParams& p, int x_type, int code_type,
                                  cudaStream_t stream) {
  const bool e4m3 = code_type == KATTN_E4M3;
  if (x_type == KATTN_F32) return launch_type<float>(p, e4m3, stream);
  if (x_type == KATTN_BF16) return launch_type<__nv_bfloat16>(p, e4m3, stream);
  return launch_type<__half>(p, e4m3, stream);
}

}  // namespace kattn
