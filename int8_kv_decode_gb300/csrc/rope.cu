// Rotary positions of query and key heads, and the table of their angles.
//
// A warp takes eight heads of a row, two at a time: the row's angles are loaded once for
// them.  Bound by memory: an element is read and written once, for three operations.  8192
// rows of 36 bf16 heads to float32 (231 MB, 34.0 us at the measured copy rate): 34.6 us; 16 rows:
// 1.7 us, a launch.
#include <algorithm>

#include "blocks_internal.cuh"
#include "rope_common.cuh"

namespace kattn {
namespace {

constexpr int kWarps = 8;

template <typename T, typename O, bool kInter>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31, groups = (p.heads + kTurnHeads - 1) / kTurnHeads;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int row = (int)(item / groups), h0 = (int)(item - (int64_t)row * groups) * kTurnHeads;
  griddep_wait();                                 // what the kernels before wrote is in place
  if (row >= p.rows) return;
  turn_heads<T, O, kInter>(static_cast<const T*>(p.x) + row * p.x_stride + h0 * kD,
                           static_cast<O*>(p.out) + row * p.out_stride + h0 * kD, min(kTurnHeads, p.heads - h0),
                           p.table, p.half, lane, [&](bool& know) {
                             const int position = ld_fresh(p.positions + row);      // below 0: a padding row
                             know = position < p.n_positions;
                             return know ? position : 0;
                           });
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
  const int64_t items = (int64_t)p.rows * ((p.heads + kTurnHeads - 1) / kTurnHeads);
  const unsigned blocks = (unsigned)((items + kWarps - 1) / kWarps);
  return launch_pdl(p.interleaved ? rope_kernel<T, O, true> : rope_kernel<T, O, false>, dim3(blocks),
                    dim3(kWarps * 32), 0, stream, p);
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
