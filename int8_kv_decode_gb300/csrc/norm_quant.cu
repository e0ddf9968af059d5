// Residual addition, root-mean-square norm and 8-bit quantization of rows.
//
//   h = x (+ residual, rounded to its type),  z = h * weight
//   codes = round(z / s0),  s0 = max |z| / 127 (or 448)
//   scale = s0 / sqrt(mean(h^2) + eps)
// The factor 1 / rms is the same for the whole row, so it goes into the scale:
// the codes depend on z alone, and one pass gives both max |z| and sum h^2.
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

__device__ __forceinline__ uint8_t code_of(float z, float s0, bool e4m3) {
  if (s0 == 0.0f) return 0;
  const float u = __fdiv_rn(z, s0);
  if (e4m3) return __nv_cvt_float_to_fp8(u, __NV_SATFINITE, __NV_E4M3);
  return (uint8_t)(int8_t)max(-127, min(127, __float2int_rn(u)));
}

constexpr int kThreads = 256;

// One block per row; the row is read again (from L2) for the codes.
template <typename T, bool kE4m3>
__global__ void __launch_bounds__(kThreads) norm_row_kernel(const NormParams p) {
  __shared__ float s_sum[kThreads / 32], s_max[kThreads / 32];
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.res_stride : nullptr;
  T* res_out = p.residual ? static_cast<T*>(p.residual_out) + row * p.res_out_stride : nullptr;
  const T* w = static_cast<const T*>(p.weight);
  const T* h = res ? res_out : x;
  float sum = 0.0f;
  for (int c = threadIdx.x; c < p.d; c += kThreads) {
    float v = to_f32(x[c]);
    if (res) {
      const T t = from_f32<T>(__fadd_rn(v, to_f32(res[c])));
      res_out[c] = t;
      v = to_f32(t);
    }
    sum = __fmaf_rn(v, v, sum);
  }
  sum = warp_sum(sum);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int i = 0; i < kThreads / 32; ++i) sum += s_sum[i];
  const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)p.d), p.eps)));
  const int groups = p.d / p.group;
  for (int gi = 0; gi < groups; ++gi) {
    const int c0 = gi * p.group, c1 = c0 + p.group;
    float a = 0.0f;
    for (int c = c0 + threadIdx.x; c < c1; c += kThreads)
      a = fmaxf(a, fabsf(__fmul_rn(to_f32(h[c]), to_f32(w[c]))));
    a = warp_max(a);
    __syncthreads();
    if (lane == 0) s_max[warp] = a;
    __syncthreads();
    for (int i = 0; i < kThreads / 32; ++i) a = fmaxf(a, s_max[i]);
    const float s0 = __fdiv_rn(a, kE4m3 ? 448.0f : 127.0f);
    for (int c = c0 + threadIdx.x; c < c1; c += kThreads)
      p.codes[row * p.d + c] = code_of(__fmul_rn(to_f32(h[c]), to_f32(w[c])), s0, kE4m3);
    if (threadIdx.x == 0) p.scales[row * groups + gi] = __fmul_rn(s0, r);
  }
}

template <typename T>
cudaError_t launch_type(const NormParams& p, int code_type, cudaStream_t stream) {
  if (code_type == KATTN_E4M3) norm_row_kernel<T, true><<<(unsigned)p.rows, kThreads, 0, stream>>>(p);
  else norm_row_kernel<T, false><<<(unsigned)p.rows, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm_quant(const NormParams& p, int x_type, int code_type,
                                  cudaStream_t stream) {
  if (x_type == KATTN_F32) return launch_type<float>(p, code_type, stream);
  if (x_type == KATTN_BF16) return launch_type<__nv_bfloat16>(p, code_type, stream);
  return launch_type<__half>(p, code_type, stream);
}

}  // namespace kattn
