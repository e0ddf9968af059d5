// Rotary positions of query and key heads, and the table of their angles.
//
// A warp takes four heads of a row: the row's angles are loaded once for them, a lane
// holds four channels of each.  Bound by memory: an element is read and written once,
// for three operations.
#include <algorithm>

#include "blocks_internal.cuh"
#include "rope_common.cuh"

namespace kattn {
namespace {

constexpr int kWarps = 8, kHeads = 4;             // heads a warp takes

template <typename T, typename O, bool kInter>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31, groups = (p.heads + kHeads - 1) / kHeads;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int row = (int)(item / groups), h0 = (int)(item - (int64_t)row * groups) * kHeads;
  if (row >= p.rows) return;
  const int n = min(kHeads, p.heads - h0);
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride + h0 * kD + 4 * lane;
  O* y = static_cast<O*>(p.out) + row * p.out_stride + h0 * kD + 4 * lane;
  const int position = __ldg(p.positions + row);
  Vec<T, 4> raw[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (i < n) raw[i] = *reinterpret_cast<const Vec<T, 4>*>(x + i * kD);
  if (position < 0) return;                       // a padding row
  const bool known = position < p.n_positions;
  const Turn t = load_turn<kInter>(p.table, known ? position : 0, p.half, lane);
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (i >= n) break;
    float f[4];
    unpack(raw[i], f);
    turn<kInter>(t, f);
    if (!known) f[0] = f[1] = f[2] = f[3] = __int_as_float(0x7fc00000);
    *reinterpret_cast<Vec<O, 4>*>(y + i * kD) = pack<O, 4>(f);
  }
}

// One thread per angle, in float64: a float32 product of a position of some 10^5 and
// its frequency is off by hundredths of a radian.
__global__ void __launch_bounds__(256) table_kernel(const double* freq, int64_t n, int half, float2* table) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t position = i / half;
    double s, c;
    sincos((double)position * __ldg(freq + (i - position * half)), &s, &c);
    table[i] = make_float2((float)c, (float)s);
  }
}

template <typename T, typename O>
cudaError_t launch_types(const RopeParams& p, cudaStream_t stream) {
  const int64_t items = (int64_t)p.rows * ((p.heads + kHeads - 1) / kHeads);
  const unsigned blocks = (unsigned)((items + kWarps - 1) / kWarps);
  if (p.interleaved) rope_kernel<T, O, true><<<blocks, kWarps * 32, 0, stream>>>(p);
  else rope_kernel<T, O, false><<<blocks, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int x_type, int out_type, cudaStream_t stream) {
  const bool wide = out_type == KATTN_F32;
  switch (x_type) {
    case KATTN_F32: return launch_types<float, float>(p, stream);
    case KATTN_BF16:
      return wide ? launch_types<__nv_bfloat16, float>(p, stream)
                  : launch_types<__nv_bfloat16, __nv_bfloat16>(p, stream);
    default:
      return wide ? launch_types<__half, float>(p, stream) : launch_types<__half, __half>(p, stream);
  }
}

cudaError_t launch_rope_table(const double* freq, int n_positions, int half, float* table,
                              cudaStream_t stream) {
  const int64_t n = (int64_t)n_positions * half;
  table_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 152 * 16), 256, 0, stream>>>(
      freq, n, half, reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

}  // namespace kattn
