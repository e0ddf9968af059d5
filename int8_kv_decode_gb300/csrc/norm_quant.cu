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

#include "ops_internal.cuh"
#include "quant_common.cuh"

namespace kattn {
namespace {

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
      const Codes<VEC> out = codes_of<VEC>(z[v], s0, inv, e4m3, scale_divides(s0));
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
