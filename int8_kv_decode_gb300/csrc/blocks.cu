// Rows written into a block-scaled cache and read back.
//
// A block of R = 32, 64 or 128 rows of one head shares a scale: codes = round(x / s),
// s = max |x| / 127 (int8) or / 448 (e4m3) over the block's rows.  Rows come in over
// time: where new rows need a larger scale than the block has, the rows that stay are
// coded again under the new one, code' = round(code * (s_old / s)).
#include <algorithm>

#include "blocks_internal.cuh"
#include "rope_common.cuh"

namespace kattn {
namespace {

// The last b in [0, n) whose key(b) is <= t, for keys that rise (0 if there is none),
// by a whole warp: 32 keys a step.
template <typename Key>
__device__ __forceinline__ int warp_find(int n, int64_t t, int lane, Key key) {
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < n && key(lo + at) <= t);
    const int k = max(__popc(le) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Keys that a row of the block table can hold (fewer than 2^30: key numbers are 32-bit).
__device__ __forceinline__ int64_t table_keys(const BlockCache& c) {
  return min((int64_t)c.max_pages << c.page_shift, (int64_t)1 << 30);
}
// Whether sequence b's rows lie in the call's and its keys in the table's pages.
__device__ __forceinline__ bool span_valid(const SpanParams& s, int b, int64_t most) {
  const int c0 = __ldg(s.cu + b), c1 = __ldg(s.cu + b + 1), st = __ldg(s.start + b);
  return c0 >= 0 && c0 <= c1 && c1 <= s.rows && st >= 0 && (int64_t)st + (c1 - c0) <= most;
}
__device__ __forceinline__ void flag_bad_spans(const SpanParams& s, int64_t most) {
  for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < s.B; b += (int64_t)gridDim.x * blockDim.x)
    if (!span_valid(s, (int)b, most)) atomicOr(s.err, KATTN_DEVERR_BAD_SEQUENCE);
}

// Row in its plane of key `key` of sequence b; -1 (flagged) where its page is not one.
__device__ __forceinline__ int row_of_key(const BlockCache& c, uint32_t* err, int b, int key) {
  const int page = __ldg(c.block_table + (int64_t)b * c.max_pages + (key >> c.page_shift));
  if ((unsigned)page >= (unsigned)c.n_pages) {
    atomicOr(err, KATTN_DEVERR_BAD_PAGE);
    return -1;
  }
  return (page << c.page_shift) | (key & ((1 << c.page_shift) - 1));
}

// ----------------------------------------------------------------- append
// One block of threads per (block of rows that a sequence touches, head, K or V): a
// warp holds 8 of its rows in registers, a lane four channels of each.  The blocks
// that sequence b touches are the units floor(cu[b] / R) + 2 b + j: at most floor(n / R)
// + 2 for its n rows, so units of different sequences never meet, and the grid is known
// without the lengths.  Queries, if any, are turned by further blocks of threads.
constexpr int kRowsPerWarp = 8, kQHeads = 4;

template <typename T, int kBlock, bool kE4m3, bool kInter>
__global__ void __launch_bounds__(kBlock * 4) append_kernel(const AppendParams p, const unsigned kv_blocks) {
  constexpr int kWarps = kBlock / kRowsPerWarp;
  __shared__ float s_max[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int R = kBlock;
  int64_t most = table_keys(p.c);
  if (p.table) most = min(most, (int64_t)p.n_positions);
  flag_bad_spans(p.s, most);

  if (blockIdx.x >= kv_blocks) {                  // ---- queries: a warp takes four heads of a row
    const int groups = (p.Hq + kQHeads - 1) / kQHeads;
    const int64_t item = (int64_t)(blockIdx.x - kv_blocks) * kWarps + warp;
    const int row = (int)(item / groups), h0 = (int)(item - (int64_t)row * groups) * kQHeads;
    if (row >= p.s.rows) return;
    const int n = min(kQHeads, p.Hq - h0);
    const T* x = static_cast<const T*>(p.q) + row * p.q_stride + h0 * kD + 4 * lane;
    T* y = static_cast<T*>(p.q_out) + row * p.q_out_stride + h0 * kD + 4 * lane;
    Vec<T, 4> raw[kQHeads];
#pragma unroll
    for (int i = 0; i < kQHeads; ++i)
      if (i < n) raw[i] = *reinterpret_cast<const Vec<T, 4>*>(x + i * kD);
    const int b = warp_find(p.s.B, row, lane, [&](int i) { return (int64_t)__ldg(p.s.cu + i); });
    if (row < __ldg(p.s.cu + b) || row >= __ldg(p.s.cu + b + 1)) return;     // no sequence's row
    const bool ok = span_valid(p.s, b, most);
    const int position = ok ? __ldg(p.s.start + b) + row - __ldg(p.s.cu + b) : 0;
    const Turn t = load_turn<kInter>(p.table, position, p.half, lane);
#pragma unroll
    for (int i = 0; i < kQHeads; ++i) {
      if (i >= n) break;
      float f[4];
      unpack(raw[i], f);
      turn<kInter>(t, f);
      if (!ok) f[0] = f[1] = f[2] = f[3] = __int_as_float(0x7fc00000);
      *reinterpret_cast<Vec<T, 4>*>(y + i * kD) = pack<T, 4>(f);
    }
    return;
  }

  // ---- the unit: sequence b, its j-th touched block, head h of K or V
  const int64_t unit = blockIdx.x / (2 * p.c.Hkv);
  const int plane = blockIdx.x - (unsigned)unit * (2 * p.c.Hkv);
  const bool is_k = plane < p.c.Hkv;
  const int h = is_k ? plane : plane - p.c.Hkv;
  const int b = warp_find(p.s.B, unit, lane, [&](int i) { return (int64_t)(__ldg(p.s.cu + i) / R) + 2 * i; });
  if (!span_valid(p.s, b, most)) return;
  const int c0 = __ldg(p.s.cu + b), n = __ldg(p.s.cu + b + 1) - c0, st = __ldg(p.s.start + b);
  const int64_t j = unit - (c0 / R + 2 * (int64_t)b);
  if (n == 0 || j < 0 || j > (st + n - 1) / R - st / R) return;
  const int key0 = (st / R + (int)j) * R;         // the block's keys: [key0, key0 + R)
  const int row0 = row_of_key(p.c, p.s.err, b, key0);
  if (row0 < 0) return;
  const int lo = max(st - key0, 0), hi = min(st + n - key0, R);    // its new rows: [lo, hi)
  uint8_t* codes = (is_k ? p.c.k : p.c.v) + ((int64_t)h * p.c.cap_rows + row0) * kD + 4 * lane;
  float* scale = (is_k ? p.c.k_scale : p.c.v_scale) + (((int64_t)h * p.c.cap_rows + row0) >> p.c.block_shift);
  const float was = lo > 0 ? *scale : 0.0f;       // (read by every thread before the barrier below)

  const int64_t stride = is_k ? p.k_stride : p.v_stride;
  const T* x = static_cast<const T*>(is_k ? p.k_new : p.v_new) + (int64_t)h * kD + 4 * lane;
  const int r0 = warp * kRowsPerWarp;
  Vec<T, 4> raw[kRowsPerWarp];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    raw[i] = Vec<T, 4>{};
    if (r0 + i >= lo && r0 + i < hi)
      raw[i] = *reinterpret_cast<const Vec<T, 4>*>(x + (int64_t)(c0 + key0 - st + r0 + i) * stride);
  }
  float f[kRowsPerWarp][4], amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    unpack(raw[i], f[i]);
    if (is_k && p.table && r0 + i >= lo && r0 + i < hi)
      turn<kInter>(load_turn<kInter>(p.table, key0 + r0 + i, p.half, lane), f[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(f[i][e]));
  }
  amax = warp_max_abs(amax);
  if (lane == 0) s_max[warp] = amax;
  __syncthreads();
  amax = warp_max_abs(lane < kWarps ? s_max[lane] : 0.0f);
  const float own = __fdiv_rn(amax, kE4m3 ? 448.0f : 127.0f);
  const float s = fmaxf(own, was);
  if (threadIdx.x == 0) *scale = s;
  const float inv = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    if (r0 + i < lo || r0 + i >= hi) continue;
    const Codes<4> c = codes_of(f[i], s, inv, kE4m3);
    *reinterpret_cast<Codes<4>*>(codes + (r0 + i) * kD) = c;
  }
  if (r0 < lo && s > was) {                       // the rows that stay, under the larger scale
    const float by = __fdiv_rn(was, s);
    uint32_t old[kRowsPerWarp];
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i)
      old[i] = r0 + i < lo ? *reinterpret_cast<const uint32_t*>(codes + (r0 + i) * kD) : 0u;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
      if (r0 + i >= lo) break;
      uint32_t w = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint8_t byte = (uint8_t)(old[i] >> (8 * e));
        uint8_t again;
        if constexpr (kE4m3) {
          const __half_raw v = __nv_cvt_fp8_to_halfraw(byte, __NV_E4M3);
          again = __nv_cvt_float_to_fp8(__fmul_rn(__half2float(__half(v)), by), __NV_SATFINITE, __NV_E4M3);
        } else {
          again = (uint8_t)(int8_t)__float2int_rn(__fmul_rn((float)(int8_t)byte, by));
        }
        w |= (uint32_t)again << (8 * e);
      }
      *reinterpret_cast<uint32_t*>(codes + (r0 + i) * kD) = w;
    }
  }
}

// ------------------------------------------------------------------- read
// A warp takes 32 rows of one head of K or V: eight lanes a row, 16 codes a lane, in
// steps of four rows; lane i looks row i up first.
template <typename O, bool kE4m3>
__global__ void __launch_bounds__(256) read_kernel(const ReadParams p) {
  const int lane = threadIdx.x & 31;
  const int planes = 2 * p.c.Hkv;
  const int64_t most = table_keys(p.c);
  flag_bad_spans(p.s, most);
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int tile = (int)(item / planes), plane = (int)(item - (int64_t)tile * planes);
  const int64_t first = (int64_t)tile * 32;
  if (first >= p.s.rows) return;
  const bool is_k = plane < p.c.Hkv;
  const int h = is_k ? plane : plane - p.c.Hkv;
  O* out = static_cast<O*>(is_k ? p.out_k : p.out_v);
  if (!out) return;
  const int64_t base = (int64_t)h * p.c.cap_rows;
  int row = -1;
  float sc = 0.0f;
  {
    const int64_t r = first + lane;
    int b = warp_find(p.s.B, first, lane, [&](int i) { return (int64_t)__ldg(p.s.cu + i); });
    while (b + 1 < p.s.B && r >= __ldg(p.s.cu + b + 1)) ++b;
    if (r < p.s.rows && r >= __ldg(p.s.cu + b) && r < __ldg(p.s.cu + b + 1) && span_valid(p.s, b, most)) {
      row = row_of_key(p.c, p.s.err, b, __ldg(p.s.start + b) + (int)r - __ldg(p.s.cu + b));
      if (row >= 0) sc = __ldg((is_k ? p.c.k_scale : p.c.v_scale) + ((base + row) >> p.c.block_shift));
    }
  }
  const uint8_t* codes = (is_k ? p.c.k : p.c.v) + base * kD + 16 * (lane & 7);
  uint4 raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = __shfl_sync(0xffffffffu, row, 4 * i + (lane >> 3));
    raw[i] = make_uint4(0, 0, 0, 0);
    if (at >= 0) raw[i] = __ldg(reinterpret_cast<const uint4*>(codes + (int64_t)at * kD));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int src = 4 * i + (lane >> 3);
    const float s = __shfl_sync(0xffffffffu, sc, src);
    const bool in = __shfl_sync(0xffffffffu, row, src) >= 0;
    O* y = out + ((first + src) * p.c.Hkv + h) * kD + 16 * (lane & 7);
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    constexpr int kPer = 16 / sizeof(O);          // values of a 16-byte store
#pragma unroll
    for (int v = 0; v < 16; v += kPer) {
      float f[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const uint8_t byte = (uint8_t)(w[(v + e) / 4] >> (8 * ((v + e) % 4)));
        float c;
        if constexpr (kE4m3) c = __half2float(__half(__nv_cvt_fp8_to_halfraw(byte, __NV_E4M3)));
        else c = (float)(int8_t)byte;
        f[e] = __fmul_rn(c, s);
      }
      if (in) *reinterpret_cast<Vec<O, kPer>*>(y + v) = pack<O, kPer>(f);
    }
  }
}

template <typename T, int kBlock, bool kE4m3>
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream) {
  const int64_t kv = ((int64_t)p.s.rows / kBlock + 2 * (int64_t)p.s.B) * 2 * p.c.Hkv;
  int64_t blocks = kv;
  if (p.q) {
    constexpr int kWarps = kBlock / kRowsPerWarp;
    const int64_t items = (int64_t)p.s.rows * ((p.Hq + kQHeads - 1) / kQHeads);
    blocks += (items + kWarps - 1) / kWarps;
  }
  if (p.interleaved) append_kernel<T, kBlock, kE4m3, true><<<(unsigned)blocks, kBlock * 4, 0, stream>>>(p, (unsigned)kv);
  else append_kernel<T, kBlock, kE4m3, false><<<(unsigned)blocks, kBlock * 4, 0, stream>>>(p, (unsigned)kv);
  return cudaGetLastError();
}
template <typename T, bool kE4m3>
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream) {
  switch (p.c.block_shift) {
    case 5: return launch_append<T, 32, kE4m3>(p, stream);
    case 6: return launch_append<T, 64, kE4m3>(p, stream);
    default: return launch_append<T, 128, kE4m3>(p, stream);
  }
}
template <typename T>
cudaError_t launch_append(const AppendParams& p, int code_type, cudaStream_t stream) {
  return code_type == KATTN_E4M3 ? launch_append<T, true>(p, stream) : launch_append<T, false>(p, stream);
}
template <typename O>
cudaError_t launch_read(const ReadParams& p, int code_type, cudaStream_t stream) {
  const int64_t items = ((int64_t)p.s.rows + 31) / 32 * 2 * p.c.Hkv;
  const unsigned blocks = (unsigned)((items + 7) / 8);
  if (code_type == KATTN_E4M3) read_kernel<O, true><<<blocks, 256, 0, stream>>>(p);
  else read_kernel<O, false><<<blocks, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_blocks(const AppendParams& p, int x_type, int code_type, cudaStream_t stream) {
  switch (x_type) {
    case KATTN_F32: return launch_append<float>(p, code_type, stream);
    case KATTN_BF16: return launch_append<__nv_bfloat16>(p, code_type, stream);
    default: return launch_append<__half>(p, code_type, stream);
  }
}

cudaError_t launch_read_blocks(const ReadParams& p, int code_type, int out_type, cudaStream_t stream) {
  switch (out_type) {
    case KATTN_F32: return launch_read<float>(p, code_type, stream);
    case KATTN_BF16: return launch_read<__nv_bfloat16>(p, code_type, stream);
    default: return launch_read<__half>(p, code_type, stream);
  }
}

}  // namespace kattn
