// Rows written into a block-scaled cache and read back.
//
// A block of R = 32, 64 or 128 rows of one head shares a scale: codes = round(x / s),
// s = max |x| / 127 (int8) or / 448 (e4m3) over the block's rows.  Rows come in over
// time: where new rows need a larger scale than the block has, the rows that stay are
// coded again under the new one, code' = round(code * (s_old / s)).
//
// What bounds them.  Writing 7 prompts of 300 to 2500 rows (7851 in all; 32 query and 4 kv
// heads, bf16; 157 MB, 23 us at the measured copy rate): 28 us, 5.5 TB/s, by issue (70%):
// unpacking, turning and coding are some 30 instructions an element and lane.  A row for each
// of 64 sequences: 5 us, the chain of loads span, page, scale.  Reading 150k rows of 4 heads as
// bf16 (463 MB, 68 us): 75 us, 6.2 TB/s; 700 rows: 2.5 us, latency.
#include <algorithm>
#include <type_traits>

#include "blocks_internal.cuh"
#include "rope_common.cuh"

namespace kattn {
namespace {

// Keys that a row of the block table can hold (fewer than 2^30: key numbers are 32-bit).
__device__ __forceinline__ int64_t table_keys(const BlockCache& c) {
  return min((int64_t)c.max_pages << c.page_shift, (int64_t)1 << 30);
}
// The rows of a sequence and its first key; whether the rows lie in the call's and the
// keys in the table's row.
struct RowSpan {
  int b, c0, c1, n, start;                        // n: its rows, none where they leave the call's
  bool valid;
};
__device__ __forceinline__ RowSpan make_span(const SpanParams& s, int b, int c0, int c1, int start, int64_t most) {
  const bool rises = c0 >= 0 && c0 <= c1 && c1 <= s.rows;
  return {b, c0, c1, rises ? c1 - c0 : 0, start, rises && start >= 0 && (int64_t)start + (c1 - c0) <= most};
}
__device__ __forceinline__ RowSpan span_of(const SpanParams& s, int b, int64_t most) {
  return make_span(s, b, ld_fresh(s.cu + b), ld_fresh(s.cu + b + 1), ld_fresh(s.start + b), most);
}
__device__ __forceinline__ void flag_bad_spans(const SpanParams& s, int64_t most) {
  for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < s.B; b += (int64_t)gridDim.x * blockDim.x)
    if (!span_of(s, (int)b, most).valid) atomicOr(s.err, KATTN_DEVERR_BAD_SEQUENCE);
}

// The last sequence b whose key(b, cu[b]) is <= t, for keys that rise (0 if there is
// none), by a whole warp: 64 of them a step.  The last step's loads hold its span too, so
// that a call of up to 64 sequences goes to memory once.
template <typename Key>
__device__ __forceinline__ RowSpan find_span(const SpanParams& s, int64_t t, int64_t most, int lane, Key key) {
  int lo = 0, n = s.B;
  auto count = [&](int step, int x, int y) {      // those of lo + i step, i < 64, i step < n; x, y: cu of lane, lane + 32
    const int i = lane * step, j = (lane + 32) * step;
    return __popc(__ballot_sync(0xffffffffu, i < n && key(lo + i, x) <= t)) +
           __popc(__ballot_sync(0xffffffffu, j < n && key(lo + j, y) <= t));
  };
  while (n > 64) {
    const int step = (n + 63) >> 6;
    const int x = ld_fresh(s.cu + min(lo + lane * step, s.B)), y = ld_fresh(s.cu + min(lo + (lane + 32) * step, s.B));
    const int k = max(count(step, x, y) - 1, 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  const int x = ld_fresh(s.cu + min(lo + lane, s.B)), y = ld_fresh(s.cu + min(lo + lane + 32, s.B));
  const int sx = ld_fresh(s.start + min(lo + lane, s.B - 1)), sy = ld_fresh(s.start + min(lo + lane + 32, s.B - 1));
  const int k = max(count(1, x, y) - 1, 0);
  auto pick = [&](int u, int v, int i) { return i < 32 ? __shfl_sync(0xffffffffu, u, i) : __shfl_sync(0xffffffffu, v, i - 32); };
  const int c1 = k < 63 ? pick(x, y, k + 1) : ld_fresh(s.cu + lo + 64);
  return make_span(s, lo + k, pick(x, y, k), c1, pick(sx, sy, k), most);
}

// Row in its plane of key `key`, by its page; -1 (flagged) where that is not one.
__device__ __forceinline__ int page_of_key(const BlockCache& c, int b, int key) {
  return ld_fresh(c.block_table + (int64_t)b * c.max_pages + (key >> c.page_shift));
}
__device__ __forceinline__ int row_of_key(const BlockCache& c, uint32_t* err, int page, int key) {
  if ((unsigned)page >= (unsigned)c.n_pages) {
    atomicOr(err, KATTN_DEVERR_BAD_PAGE);
    return -1;
  }
  return (page << c.page_shift) | (key & ((1 << c.page_shift) - 1));
}

// The four codes of a word as float32 values, exact.
template <bool kE4m3>
__device__ __forceinline__ void code_values(uint32_t w, float* f) {
  if constexpr (kE4m3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
      const float2 v = __half22float2(__half2(h));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
    w ^= 0x80808080u;                             // code + 128 as the low mantissa bits of 2^23
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[e] = __fsub_rn(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440u | e)), 8388736.0f);
  }
}

// ----------------------------------------------------------------- append
// One block of threads per (block of rows that a sequence touches, head, K or V): a
// warp holds 8 of its rows in registers, two at a time, a lane eight channels of each.  The
// blocks that sequence b touches are the units floor(cu[b] / R) + 2 b + j: at most floor(n /
// R) + 2 for its n rows, so units of different sequences never meet, and the grid is known
// without the lengths.  Queries, if any, are turned by further blocks of threads.
// The maximum keeps a NaN, so a block of rows that are not all finite is known by it: its
// scale is then taken again from the finite elements, as an infinite scale would code every
// row of the block to 0, those that stay among them.
constexpr int kRowsPerWarp = 8;

// The largest absolute value, or NaN.
__device__ __forceinline__ float max_abs_or_nan(float x, float y, float z) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

template <typename T, int kBlock, bool kE4m3, bool kInter>
__global__ void __launch_bounds__(kBlock * 4) append_kernel(const AppendParams p, const unsigned kv_blocks) {
  constexpr int kWarps = kBlock / kRowsPerWarp;
  __shared__ float s_max[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int R = kBlock;
  // (The kernel that follows is not let in early: its blocks would take the place of this
  // one's.  A row for each of 64 sequences written and read back 10.0 us, with it 13 us.)
  griddep_wait();                                 // what the kernels before wrote is in place
  int64_t most = table_keys(p.c);
  if (p.table) most = min(most, (int64_t)p.n_positions);
  if ((int64_t)blockIdx.x * blockDim.x < p.s.B) flag_bad_spans(p.s, most);

  if (blockIdx.x >= kv_blocks) {                  // ---- queries: a warp takes heads of a row
    const int groups = (p.Hq + kTurnHeads - 1) / kTurnHeads;
    const int64_t item = (int64_t)(blockIdx.x - kv_blocks) * kWarps + warp;
    const int row = (int)(item / groups), h0 = (int)(item - (int64_t)row * groups) * kTurnHeads;
    if (row >= p.s.rows) return;
    turn_heads<T, T, kInter>(static_cast<const T*>(p.q) + row * p.q_stride + h0 * kD,
                             static_cast<T*>(p.q_out) + row * p.q_out_stride + h0 * kD,
                             min(kTurnHeads, p.Hq - h0), p.table, p.half, lane, [&](bool& know) {
      const RowSpan s = find_span(p.s, row, most, lane, [](int, int cu) { return (int64_t)cu; });
      know = s.valid;
      return row < s.c0 || row >= s.c1 ? -1 : know ? s.start + row - s.c0 : 0;   // (-1: no sequence's row)
    });
    return;
  }

  // ---- the unit: sequence b, its j-th touched block, head h of K or V
  const unsigned unit = blockIdx.x / (2u * p.c.Hkv);
  const int plane = (int)(blockIdx.x - unit * (2u * p.c.Hkv));
  const bool is_k = plane < p.c.Hkv;
  const int h = is_k ? plane : plane - p.c.Hkv;
  const RowSpan span = find_span(p.s, unit, most, lane, [](int i, int cu) { return (int64_t)(cu / R) + 2 * i; });
  if (!span.valid || span.n == 0) return;
  const int b = span.b;
  const int st = span.start, n = span.n;
  const int64_t j = (int64_t)unit - (span.c0 / R + 2 * (int64_t)b);
  if (j < 0 || j > (st + n - 1) / R - st / R) return;
  const int key0 = (st / R + (int)j) * R;         // the block's keys: [key0, key0 + R)
  const int page = page_of_key(p.c, b, key0);     // (looked at after the rows' loads)
  const int lo = max(st - key0, 0), hi = min(st + n - key0, R);    // its new rows: [lo, hi)

  const int64_t stride = is_k ? p.k_stride : p.v_stride;
  const bool turns_k = is_k && p.table != nullptr;
  const int l = lane & 15, side = lane >> 4;
  const Runs run = lane_runs<kInter>(turns_k ? p.half : 0, l);
  const T* x = static_cast<const T*>(is_k ? p.k_new : p.v_new) + (int64_t)(span.c0 + key0 - st) * stride + h * kD;
  const int r0 = warp * kRowsPerWarp;             // row r0 + 2 i + side of the block in step i
  Vec<T, 4> ra[kRowsPerWarp / 2], rb[kRowsPerWarp / 2];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp / 2; ++i) {
    const int r = r0 + 2 * i + side;
    ra[i] = rb[i] = Vec<T, 4>{};
    if (r >= lo && r < hi) {
      ra[i] = *reinterpret_cast<const Vec<T, 4>*>(x + r * stride + run.a);
      rb[i] = *reinterpret_cast<const Vec<T, 4>*>(x + r * stride + run.b);
    }
  }
  const int row0 = row_of_key(p.c, p.s.err, page, key0);
  if (row0 < 0) return;
  uint8_t* codes = (is_k ? p.c.k : p.c.v) + ((int64_t)h * p.c.cap_rows + row0) * kD;
  float* scale = (is_k ? p.c.k_scale : p.c.v_scale) + (((int64_t)h * p.c.cap_rows + row0) >> p.c.block_shift);
  const float was = lo > 0 ? *scale : 0.0f;       // (read by every thread before the barrier below)
  float fa[kRowsPerWarp / 2][4], fb[kRowsPerWarp / 2][4], amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kRowsPerWarp / 2; ++i) {
    const int r = r0 + 2 * i + side;
    unpack(ra[i], fa[i]);
    unpack(rb[i], fb[i]);
    if (turns_k && run.turns && r >= lo && r < hi)
      turn<kInter>(load_angles(p.table, key0 + r, p.half, l), fa[i], fb[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) amax = max_abs_or_nan(amax, fa[i][e], fb[i][e]);
  }
  auto block_max = [&](float v) {                 // (a NaN is the largest: warp_max_abs goes by the bits)
    v = warp_max_abs(v);
    if (lane == 0) s_max[warp] = v;
    __syncthreads();
    return warp_max_abs(lane < kWarps ? s_max[lane] : 0.0f);
  };
  amax = block_max(amax);
  const bool odd = !(amax < INFINITY);            // elements that are not finite
  if (odd) {
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp / 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = fabsf(fa[i][e]), y = fabsf(fb[i][e]);
        amax = fmaxf(amax, fmaxf(x < INFINITY ? x : 0.0f, y < INFINITY ? y : 0.0f));
      }
    __syncthreads();                              // (the maxima are read)
    amax = block_max(amax);
    if (threadIdx.x == 0) atomicOr(p.s.err, KATTN_DEVERR_NOT_FINITE);
  }
  const float own = __fdiv_rn(amax, kE4m3 ? 448.0f : 127.0f);
  const float s = fmaxf(own, was);
  if (threadIdx.x == 0) *scale = s;
  const float inv = __frcp_rn(s);
  const bool divide = odd || scale_divides(s);
#pragma unroll
  for (int i = 0; i < kRowsPerWarp / 2; ++i) {
    const int r = r0 + 2 * i + side;
    if (r < lo || r >= hi) continue;
    const Codes<4> ca = codes_of(fa[i], s, inv, kE4m3, divide), cb = codes_of(fb[i], s, inv, kE4m3, divide);
    *reinterpret_cast<Codes<4>*>(codes + r * kD + run.a) = ca;
    *reinterpret_cast<Codes<4>*>(codes + r * kD + run.b) = cb;
  }
  if (r0 < lo && s > was) {                       // the rows that stay, under the larger scale
    const float by = __fdiv_rn(was, s);
    uint32_t old[kRowsPerWarp];
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i)
      old[i] = r0 + i < lo ? *reinterpret_cast<const uint32_t*>(codes + (r0 + i) * kD + 4 * lane) : 0u;
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
      *reinterpret_cast<uint32_t*>(codes + (r0 + i) * kD + 4 * lane) = w;
    }
  }
}

// ------------------------------------------------------------------- read
// A warp looks 8 or 16 rows up, one a lane, and takes them from one of the 2 Hkv planes of K
// and V: all their codes are loaded before the first become values.  A lane takes as many codes
// of a row as make a 16-byte store, so that loads and stores of a row are whole.  The warps
// of a block take the planes of the same rows, whose values lie side by side.
template <typename O, bool kE4m3, int kTile>
__global__ void __launch_bounds__(256, 4) read_kernel(const ReadParams p) {
  constexpr int kPer = 16 / sizeof(O), kLanes = kD / kPer;       // codes a lane, lanes a row
  constexpr int kRows = 32 / kLanes, kLoads = kTile / kRows;     // rows a load, loads
  using Raw = typename std::conditional<kPer == 8, uint2, uint32_t>::type;
  const int lane = threadIdx.x & 31;
  griddep_wait();
  const int64_t most = table_keys(p.c);
  if ((int64_t)blockIdx.x * blockDim.x < p.s.B) flag_bad_spans(p.s, most);
  const int planes = (p.out_k ? p.c.Hkv : 0) + (p.out_v ? p.c.Hkv : 0);
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int tile = (int)(item / planes), plane = (int)(item - (int64_t)tile * planes);
  const int64_t first = (int64_t)tile * kTile;
  if (first >= p.s.rows) return;
  const bool is_k = p.out_k && plane < p.c.Hkv;
  const int h = plane - (p.out_k && plane >= p.c.Hkv ? p.c.Hkv : 0);
  const int64_t base = (int64_t)h * p.c.cap_rows;

  // ---- lane i: row first + i.  Its sequence is that of row `first` or one of those that
  // follow; 32 of them are looked at together.
  int row = -1;
  {
    const int b0 = find_span(p.s, first, most, lane, [](int, int cu) { return (int64_t)cu; }).b;
    const int r = (int)min(first + lane, (int64_t)INT32_MAX);
    const int at = min(b0 + lane, p.s.B - 1);
    const int begins = ld_fresh(p.s.cu + at), starts = ld_fresh(p.s.start + at);
    const int ends = b0 + lane < p.s.B ? ld_fresh(p.s.cu + b0 + lane + 1) : INT32_MAX;
    int k = 0;                                    // the ends up to the row, by halving
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const int e = __shfl_sync(0xffffffffu, ends, k + d - 1);
      if (e <= r) k += d;
    }
    const int c0 = __shfl_sync(0xffffffffu, begins, k), c1 = __shfl_sync(0xffffffffu, ends, k);
    const int st = __shfl_sync(0xffffffffu, starts, k);
    RowSpan s = make_span(p.s, b0 + k, c0, c1, st, most);
    if (c1 <= r) {                                // (k = 31: further on)
      int b = b0 + k;
      while (b + 1 < p.s.B && r >= ld_fresh(p.s.cu + b + 1)) ++b;
      s = span_of(p.s, b, most);
    }
    if (s.b < p.s.B && lane < kTile && first + lane < p.s.rows && s.valid && r >= s.c0 && r < s.c0 + s.n) {
      const int key = s.start + r - s.c0;
      row = row_of_key(p.c, p.s.err, page_of_key(p.c, s.b, key), key);
    }
  }
  const int col = (lane % kLanes) * kPer, sub = lane / kLanes;
  const uint8_t* codes = (is_k ? p.c.k : p.c.v) + base * kD + col;
  Raw raw[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = __shfl_sync(0xffffffffu, row, i * kRows + sub);
    raw[i] = Raw{};
    if (at >= 0) raw[i] = ld_fresh(reinterpret_cast<const Raw*>(codes + (int64_t)at * kD));
  }
  const float sc = row >= 0 ? ld_fresh((is_k ? p.c.k_scale : p.c.v_scale) + ((base + row) >> p.c.block_shift)) : 0.0f;
  O* y = static_cast<O*>(is_k ? p.out_k : p.out_v) + (first * p.c.Hkv + h) * kD + col;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int src = i * kRows + sub;
    const float s = __shfl_sync(0xffffffffu, sc, src);
    const bool in = __shfl_sync(0xffffffffu, row, src) >= 0;
    float f[kPer];
    if constexpr (kPer == 8) {
      code_values<kE4m3>(raw[i].x, f);
      code_values<kE4m3>(raw[i].y, f + 4);
    } else {
      code_values<kE4m3>(raw[i], f);
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) f[e] = __fmul_rn(f[e], s);
    if (in) *reinterpret_cast<Vec<O, kPer>*>(y + (int64_t)src * p.c.Hkv * kD) = pack<O, kPer>(f);
  }
}

template <typename T, int kBlock, bool kE4m3>
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream) {
  const int64_t kv = ((int64_t)p.s.rows / kBlock + 2 * (int64_t)p.s.B) * 2 * p.c.Hkv;
  int64_t blocks = kv;
  if (p.q) {
    constexpr int kWarps = kBlock / kRowsPerWarp;
    const int64_t items = (int64_t)p.s.rows * ((p.Hq + kTurnHeads - 1) / kTurnHeads);
    blocks += (items + kWarps - 1) / kWarps;
  }
  return launch_pdl(p.interleaved ? append_kernel<T, kBlock, kE4m3, true> : append_kernel<T, kBlock, kE4m3, false>,
                    dim3((unsigned)blocks), dim3(kBlock * 4), 0, stream, p, (unsigned)kv);
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
// Rows a warp: few where there are few, so that their warps share the multiprocessors and a
// warp's chain is short (us a call with 8 / 16 / 32; bf16 rows of 4 heads: 1 row for each of 64
// sequences 2.6 / 3.3 / 4.3, 2000 2.9 / 3.1 / 4.2, 8000 5.6 / 5.4 / 5.4, 16000 9.7 / 7.9 / 8.5,
// 144000 78 / 72 / 71; with 4, one row 2.2 as with 8, 8000 7.7).  float32 rows fill a warp's
// stores one by one: 8 are always best (8000 rows 7.2 / 8.0 / 8.1, 144000 112 / 116 / 118).
template <typename O, int kTile>
cudaError_t launch_read(const ReadParams& p, int code_type, int planes, cudaStream_t stream) {
  const int64_t items = ((int64_t)p.s.rows + kTile - 1) / kTile * planes;
  return launch_pdl(code_type == KATTN_E4M3 ? read_kernel<O, true, kTile> : read_kernel<O, false, kTile>,
                    dim3((unsigned)((items + 7) / 8)), dim3(256), 0, stream, p);
}
template <typename O>
cudaError_t launch_read(const ReadParams& p, int code_type, cudaStream_t stream) {
  const int planes = (p.out_k ? p.c.Hkv : 0) + (p.out_v ? p.c.Hkv : 0);
  if constexpr (sizeof(O) == 2)
    if ((int64_t)p.s.rows * planes > 32768) return launch_read<O, 16>(p, code_type, planes, stream);
  return launch_read<O, 8>(p, code_type, planes, stream);
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
