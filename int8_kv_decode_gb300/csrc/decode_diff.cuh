// What the kernels of the differential attention share: the windows of a sequence,
// the work units over a batch, and the arithmetic of a row, so that a row has the
// same bytes whichever of them takes it.
#pragma once

#include <type_traits>

#include "decode_split.cuh"
#include "ops_internal.cuh"

namespace kattn {
namespace {

// Windows sit at fixed key positions, so the bytes of a row depend on its own keys
// alone.
constexpr int kWindow = 256;
// The first kShortKeys keys lie in shorter windows: a short sequence is then spread
// over more warps, and a long one has only these.  (One sequence of 257 keys: 14.7
// us a call, 18.8 with one window for them; the first 512 or 1024 keys in windows of
// 128, or the first 256 in windows of 64, leave that as it is and slow the verify
// case from 62 to 66, 75 and 75 us.)
constexpr int kShortWindow = 128, kShortKeys = 256, kShortWindows = kShortKeys / kShortWindow;
constexpr int kWinBlocks = kWindow / kBlockBk;    // 8: lane e < 8 holds the row of block e
constexpr int kMaxGroups = 256;                   // entries of the prefix over sequences
constexpr int kQStride = kD + 16;                 // bytes between query rows (spread over banks)
// The running maximum that the weights refer to moves only when a block's maximum
// exceeds it by more than kLag: most blocks then rescale nothing.  Weights stay
// below e^kLag < 2^6.
constexpr float kLag = 4.0f;

__host__ __device__ inline int diff_windows(int keys) {
  return keys <= kShortKeys ? (keys + kShortWindow - 1) / kShortWindow
                            : kShortWindows + (keys - kShortKeys + kWindow - 1) / kWindow;
}
__device__ __forceinline__ int window_start(int w) {
  return w < kShortWindows ? w * kShortWindow : kShortKeys + (w - kShortWindows) * kWindow;
}
__device__ __forceinline__ int window_keys(int w) { return w < kShortWindows ? kShortWindow : kWindow; }
__host__ __device__ inline int diff_stride(int R) { return 2 * R * (2 * kD + 2); }   // floats

struct DiffItem {
  int b, pair, w, rg, ctx, row0;                  // b < 0: none
  int fresh;                                      // other queries than the item before
};

__device__ __forceinline__ bool diff_valid(const DiffParams& p, int b, int ctx) {
  if (p.block_table == nullptr) return sequence_ok(p.row_start[b], ctx, p.M, p.cap_rows, p.max_ctx);
  if (ctx < 1 || ctx > p.max_ctx) return false;
  const int64_t keys = (int64_t)ctx + p.M - 1;
  return ((keys + (1 << p.page_shift) - 1) >> p.page_shift) <= (int64_t)p.max_pages;
}

// Row (in a plane) of block e = lane of the item's window, in two steps: the
// table entry is loaded well before it is looked at.  Lanes past the window hold 0.
__device__ __forceinline__ int row_entry(const DiffParams& p, const DiffItem& it, int lane) {
  const int key = window_start(it.w) + lane * kBlockBk;
  if (it.b < 0 || lane * kBlockBk >= window_keys(it.w) || key >= it.ctx + p.M - 1) return 0;
  if (p.block_table == nullptr) return it.row0 + key;
  return __ldg(p.block_table + (int64_t)it.b * p.max_pages + (key >> p.page_shift));
}
__device__ __forceinline__ int row_of_entry(const DiffParams& p, const DiffItem& it, int page, int lane) {
  if (p.block_table == nullptr) return page;
  const int key = window_start(it.w) + lane * kBlockBk;
  if ((unsigned)page >= (unsigned)p.n_pages) {
    atomicOr(p.err_word, KATTN_DEVERR_BAD_PAGE);
    page = 0;
  }
  return (page << p.page_shift) | (key & ((1 << p.page_shift) - 1));
}

// warp_quantize_row's result for a row already loaded (lane: elements 4 lane ..),
// without its four divisions: x * (1 / s) is off by less than 3.1e-5 (|x / s| <=
// 127; 1/s, the product and the quotient's own rounding 2^-24 each), so its
// nearest integer is that of the division unless it lies closer than 1e-4 to a
// half; those, and scales whose reciprocal may overflow, divide.
__device__ __forceinline__ uint32_t quantize_loaded_row(float4 x, float* scale_out) {
  const float amax = warp_max(fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
  const float s = quant_scale(amax);
  *scale_out = s;
  const float inv = __frcp_rn(s);
  const float magic = 12582912.0f;                // 1.5 * 2^23: the sum's low byte is the integer
  const float t[4] = {__fmul_rn(x.x, inv), __fmul_rn(x.y, inv), __fmul_rn(x.z, inv), __fmul_rn(x.w, inv)};
  uint32_t r[4];
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = __fadd_rn(t[i], magic);
    far = fmaxf(far, fabsf(__fsub_rn(t[i], __fsub_rn(y, magic))));
    r[i] = __float_as_uint(y);
  }
  if (far > 0.4999f || !(s > 1e-30f))
    return pack_i8x4(quant_one(x.x, s), quant_one(x.y, s), quant_one(x.z, s), quant_one(x.w, s));
  return __byte_perm(__byte_perm(r[0], r[1], 0x0040u), __byte_perm(r[2], r[3], 0x0040u), 0x5410u);
}

// Shared memory by 32-bit address and immediate offset: the block loop's addresses
// are lane constants plus a stage or buffer offset.
template <int kOff>
__device__ __forceinline__ uint4 lds128a(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4+%5];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr), "n"(kOff)
               : "memory");
  return v;
}
template <int kOff>
__device__ __forceinline__ float2 lds64a(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2+%3];\n"
               : "=f"(v.x), "=f"(v.y)
               : "r"(addr), "n"(kOff)
               : "memory");
  return v;
}
template <int kOff>
__device__ __forceinline__ float lds32a(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1+%2];\n" : "=f"(v) : "r"(addr), "n"(kOff) : "memory");
  return v;
}
template <int kOff>
__device__ __forceinline__ void sts32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0+%1], %2;\n" ::"r"(addr), "n"(kOff), "f"(v) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, float2 v) {
  asm volatile("st.shared.v2.f32 [%0], {%1,%2};\n" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}

// Four 8 x 8 matrices of 16-bit elements, transposed: thread (g, c) gets elements
// [rows 2c, 2c + 1][column g] of matrix i in r[i]; lane 8 i + r gives the address
// of row r of matrix i.
template <int kOff>
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4+%5];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(kOff)
               : "memory");
}

// The first of a chain of products: nothing to add to.
__device__ __forceinline__ void mma_i8_first(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7},"
      " {%8,%9}, {%10,%10,%10,%10};\n"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}

__device__ __forceinline__ bool bar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// Whether the stage's copy landed, for the whole warp; the wait is bounded.
__device__ __noinline__ bool stage_wait(uint32_t bar, uint32_t parity) {
  for (uint32_t it = 0; it < kSpinLimit; ++it)
    if (__all_sync(0xffffffffu, bar_try_wait(bar, parity))) return true;
  return false;
}
__device__ __forceinline__ bool stage_ready(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, bar_try_wait(bar, parity)) || stage_wait(bar, parity);
}

// The row's reference moves to the block's maximum bm where that exceeds its
// threshold; alpha: the factor of what is summed up so far.
__device__ __forceinline__ void move_reference(float bm, float& m_run, float& m_move, float& alpha) {
  if (bm > m_move) {
    // (nothing is summed up yet where the threshold was -inf)
    if (m_move != -INFINITY) alpha = exp_diff(m_run, bm);
    m_run = bm;
    m_move = __fadd_rd(bm, kLag);                 // (no more than kLag above, however large the scores)
  }
}

// out = o_0 / l_0 - lam * (o_1 / l_1), each operation rounded on its own, here and
// in the merge alike.
__device__ __forceinline__ float diff_out(float o0, float l0, float o1, float l1, float lam) {
  return __fsub_rn(__fdiv_rn(o0, l0), __fmul_rn(lam, __fdiv_rn(o1, l1)));
}

// Q.K of 32 keys and 8 rows on the int8 MMA: acc[half] of keys 16 half + g (+ 8), rows
// 2c + e.  k0: address of row g, chunk 2c of the keys (rows g, g + 8, ... share the
// swizzle); q: bytes 32c .. 32c + 31 of row g.
__device__ __forceinline__ void key_products(uint32_t k0, uint4 qlo, uint4 qhi, int (&acc)[2][4]) {
#pragma unroll
  for (int part = 0; part < 2; ++part) {          // 64 channels each, both halves side by side
    const uint32_t k = part ? k0 ^ 16u : k0;
    const uint4 a0 = lds128a<0>(k), b0 = lds128a<8 * kD>(k);
    const uint4 a1 = lds128a<16 * kD>(k), b1 = lds128a<24 * kD>(k);
    const uint4 q = part ? qhi : qlo;
    if (part == 0) {
      mma_i8_first(acc[0], a0.x, b0.x, a0.y, b0.y, q.x, q.y);
      mma_i8_first(acc[1], a1.x, b1.x, a1.y, b1.y, q.x, q.y);
    } else {
      mma_i8(acc[0], a0.x, b0.x, a0.y, b0.y, q.x, q.y);
      mma_i8(acc[1], a1.x, b1.x, a1.y, b1.y, q.x, q.y);
    }
    mma_i8(acc[0], a0.z, b0.z, a0.w, b0.w, q.z, q.w);
    mma_i8(acc[1], a1.z, b1.z, a1.w, b1.w, q.z, q.w);
  }
}
// Scores s = (S * (qs * ks)) * sm_scale, rounded as written: sc[half][key g | g + 8] of
// rows 2c, 2c + 1; ks4[q]: k_scale of key g + 8q.
__device__ __forceinline__ void scores_of(const int (&acc)[2][4], const float (&ks4)[4], float2 qs,
                                          float sm_scale, float2 (&sc)[2][2]) {
#pragma unroll
  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) {
      const float ks = ks4[2 * hf + k2];
      const float2 qk = f2_mul(qs, make_float2(ks, ks));
      const float2 S = make_float2(__int2float_rn(acc[hf][2 * k2]), __int2float_rn(acc[hf][2 * k2 + 1]));
      sc[hf][k2] = f2_mul(f2_mul(S, qk), make_float2(sm_scale, sm_scale));
    }
}
// Keys at or past a row's own; key0: the thread's first.
__device__ __forceinline__ void hide_keys(float2 (&sc)[2][2], int key0, int keys_x, int keys_y) {
#pragma unroll
  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) {
      const int key = key0 + 16 * hf + 8 * k2;
      if (key >= keys_x) sc[hf][k2].x = -INFINITY;
      if (key >= keys_y) sc[hf][k2].y = -INFINITY;
    }
}
// Weights e^(s - m) in place of the scores, the difference first: exact near the largest,
// where the weights matter, however large the scores are.  A row's reference moves, to the
// block's maximum, only where a score exceeds it by more than kLag; only then are the
// maxima of the row's 32 keys put together.  l_run: this thread's weights so far.
// Returns (to the warp) whether what is summed up so far has to be scaled by alpha.
__device__ __forceinline__ bool block_weights(float2 (&sc)[2][2], float2& m_run, float2& m_move,
                                              float2& l_run, float2& alpha) {
  bool moved = false;
  float2 bm = make_float2(fmaxf(fmaxf(sc[0][0].x, sc[0][1].x), fmaxf(sc[1][0].x, sc[1][1].x)),
                          fmaxf(fmaxf(sc[0][0].y, sc[0][1].y), fmaxf(sc[1][0].y, sc[1][1].y)));
  if (__any_sync(0xffffffffu, bm.x > m_move.x || bm.y > m_move.y)) {
#pragma unroll
    for (int o2 = 4; o2 <= 16; o2 <<= 1) {
      bm.x = fmaxf(bm.x, __shfl_xor_sync(0xffffffffu, bm.x, o2));
      bm.y = fmaxf(bm.y, __shfl_xor_sync(0xffffffffu, bm.y, o2));
    }
    move_reference(bm.x, m_run.x, m_move.x, alpha.x);
    move_reference(bm.y, m_run.y, m_move.y, alpha.y);
    moved = __any_sync(0xffffffffu, alpha.x != 1.0f || alpha.y != 1.0f);
  }
  const float2 l2e = make_float2(kLog2e, kLog2e);
#pragma unroll
  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) {
      const float2 x2 = f2_mul(f2_sub(sc[hf][k2], m_run), l2e);
      // (a key the row does not see: 2^-inf = 0)
      sc[hf][k2] = make_float2(fast_exp2(x2.x), fast_exp2(x2.y));
    }
  l_run = f2_fma(l_run, alpha, f2_add(f2_add(sc[0][0], sc[0][1]), f2_add(sc[1][0], sc[1][1])));
  return moved;
}
// The row sum of a thread's weights over the threads that share its rows.
__device__ __forceinline__ float row_total(float v) {
  v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
// The operand of the second product is weight * v_scale * 2^E as f16 hi + lo: 22 bits,
// or steps of 2^-24 below 2^-3.  E per row and plane, for the window:
//   * the largest v_scale among the keys that the row sees, times 2^E, lies in [2^8,
//     2^9), so that with weights below 2^6 no product reaches 2^15.  The largest product
//     is at least the smallest v_scale (the weight of the largest score is 1 or more),
//     so with scales within a factor of 2^6 a product is held to 22 bits or 2^-27 of
//     the row's largest;
//   * where the scales differ by more (or one is 0) the largest scale may belong to a key
//     of no weight, and the steps would swallow the others.  E then follows the largest
//     product so far, per map (follow_products), which lies in [2^14, 2^15): 22 bits or
//     2^-39 of it.
// Which of them goes by the row's own keys.  (Where every window is of the second kind the
// calls take 141 us instead of 122, 64 sequences of 512 to 32768 keys, one column, and 183
// instead of 144, 64 x 1k..4k, 5 columns; one such key per sequence costs 1%.)
constexpr float kSpread = 0.015625f;              // 2^-6
__device__ __forceinline__ float power_scale(int top, float v) {    // 2^E: v 2^E in [2^top, 2^(top + 1))
  const int bexp = min(max(254 + top - (int)((__float_as_uint(v) >> 23) & 0xffu), 1), 253);
  return __uint_as_float((uint32_t)bexp << 23);
}
__device__ __forceinline__ float operand_scale(float vmax) { return power_scale(8, vmax); }
__device__ __forceinline__ float inverse_scale(float up) {
  return __uint_as_float((254u << 23) - __float_as_uint(up));
}
// E that follows the products: 2^E for the largest so far.
__device__ __forceinline__ float product_scale(float mag) { return power_scale(14, mag); }
// A block of such a row: m, its largest product; alpha, the factor of what is summed up so
// far as its reference moved; mag, the largest product so far.  Returns the factor with
// the step to the new E, a power of two.  (An E that rises makes up for an alpha, so what
// is summed up stays below 2^31; after alpha = 0 nothing is left of it.)
__device__ __forceinline__ float follow_products(float m, float alpha, float& mag) {
  const float was = inverse_scale(product_scale(mag));
  mag = fmaxf(__fmul_rn(mag, alpha), m);
  return alpha == 0.0f ? 0.0f : __fmul_rn(alpha, __fmul_rn(product_scale(mag), was));
}
// Products weight * v_scale of keys that a row may not see: their weight is 0, but 2^E
// goes by the keys that the row sees, and with a larger scale 2^E may leave float32, where
// 0 * inf is no number.
__device__ __forceinline__ void hide_products(float2& y, float2 w) {
  if (w.x == 0.0f) y.x = 0.0f;
  if (w.y == 0.0f) y.y = 0.0f;
}
// What the scales of a row's keys in the window are: of those it sees the largest and
// the smallest, and the largest of all (no number counts as the largest).
struct ScaleRange {
  float most, least, all;
  __device__ __forceinline__ void add(float v, bool seen) {
    if (seen) {
      most = fmaxf(most, v);
      least = fminf(least, v);
    }
    all = __uint_as_float(max(__float_as_uint(all), __float_as_uint(v)));
  }
  __device__ __forceinline__ bool spread() const { return least < __fmul_rn(most, kSpread); }
  // (times 2^E: 1 where E follows the products, and then a factor of its own)
  __device__ __forceinline__ float scale() const { return spread() ? 1.0f : operand_scale(most); }
  // Whether the blocks need care: an E that follows the products, or hidden keys whose
  // scale times 2^E is not finite.  Such units take an instantiation of the block loop of
  // their own, so that the others pay nothing.
  __device__ __forceinline__ bool care() const { return spread() || !(__fmul_rn(all, scale()) < INFINITY); }
};
// Over the warp, from each lane's largest and smallest (values >= 0 are ordered as their
// bits are).
__device__ __forceinline__ ScaleRange warp_range(float most, float least) {
  const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
  return {m, __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(least))), m};
}
// Bytes (XOR 0x80) of two keys of two channels into the mantissa of 1024, less 1152:
// exact f16.  vw: words of the transposing load; af: the operand's rows g and g + 8,
// keys 2c, 2c + 1 and 2c + 8, 2c + 9.
__device__ __forceinline__ void value_operand(uint32_t w0, uint32_t w1, uint32_t (&af)[4]) {
  const uint32_t t0 = w0 ^ 0x80808080u, t1 = w1 ^ 0x80808080u;
  af[0] = i8pair_to_h2(t0, 0x4240u);
  af[1] = i8pair_to_h2(t0, 0x4341u);
  af[2] = i8pair_to_h2(t1, 0x4240u);
  af[3] = i8pair_to_h2(t1, 0x4341u);
}

// The units of a batch: per sequence its windows, for each plane pair and row group.
// Units follow one another window by window within a row group, then row group by row
// group, so that its queries are read and quantized once for a run of windows.  A
// worker takes the units that start in its share of the batch's cost: one for each of a
// sequence's short windows, `longer` for the others.
struct DiffUnits {
  const DiffParams& p;
  const int* prefix;                              // cost before each group of gs sequences
  int gs, ng, nrg, longer;
  __device__ __forceinline__ DiffUnits(const DiffParams& params, const int* sums, int row_groups, int cost)
      : p(params), prefix(sums), nrg(row_groups), longer(cost) {
    gs = (p.B + kMaxGroups - 1) / kMaxGroups;
    ng = (p.B + gs - 1) / gs;
  }
  __device__ __forceinline__ int windows(int ctx) const { return diff_windows(ctx + p.M - 1); }
  __device__ __forceinline__ int cost(int w) const { return w < kShortWindows ? 1 : longer; }
  __device__ __forceinline__ int before(int w) const {        // of the windows before w
    return min(w, kShortWindows) + max(w - kShortWindows, 0) * longer;
  }
  __device__ __forceinline__ int of(int b, int ctx) const {
    return diff_valid(p, b, ctx) ? before(windows(ctx)) * p.pairs * nrg : 0;
  }
  // Fills sums[kMaxGroups + 1] (with scratch for 4 warps); for the whole block, of at
  // least 128 threads.
  __device__ __forceinline__ void count(int* sums, int* scratch) const {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kMaxGroups; i += blockDim.x) {
      int n = 0;
      if (i < ng)
        for (int b = i * gs; b < min(p.B, i * gs + gs); ++b) n += of(b, p.ctx_len[b]);
      sums[i] = n;
    }
    __syncthreads();
    constexpr int kPer = kMaxGroups / 128;
    int n[kPer], run = 0, incl = 0;
    if (tid < 128) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        n[i] = sums[tid * kPer + i];
        run += n[i];
      }
      incl = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) scratch[warp] = incl;
    }
    __syncthreads();
    if (tid < 128) {
      int base = incl - run;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (w < warp) base += scratch[w];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        sums[tid * kPer + i] = base;
        base += n[i];
      }
      if (tid == 127) sums[kMaxGroups] = base;
    }
  }
  __device__ __forceinline__ void at_sequence(DiffItem& it, int b) const {
    it.b = b;
    it.ctx = p.ctx_len[b];
    it.row0 = p.block_table ? 0 : (int)p.row_start[b];
  }
  // The first unit that starts in [*at, end), and where; false: none.
  __device__ __forceinline__ bool find(int* at, int end, DiffItem* unit) const {
    if (*at >= end) return false;
    DiffItem it{};
    int lo = 0, hi = ng;                          // prefix[lo] <= *at < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= *at) lo = mid;
      else hi = mid;
    }
    int i = *at - prefix[lo], b = lo * gs;
    for (int n; gs > 1 && i >= (n = of(b, p.ctx_len[b])); ++b) i -= n;
    at_sequence(it, b);
    const int nw = windows(it.ctx), all = before(nw), run = i / all;
    i -= run * all;                               // into the run of a row group
    it.w = i <= kShortWindows ? i : kShortWindows + (i - kShortWindows + longer - 1) / longer;
    it.pair = run / nrg;
    it.rg = run - it.pair * nrg;
    it.fresh = 1;
    *at += min(before(it.w), all) - i;
    if (*at >= end) return false;
    if (it.w >= nw) {                             // the next run's first (there is one)
      it.w = nw - 1;
      it = after(it);
    }
    *unit = it;
    return true;
  }
  __device__ __forceinline__ DiffItem after(DiffItem it) const {   // the unit after it (there is one)
    it.fresh = 0;
    if (++it.w < windows(it.ctx)) return it;
    it.w = 0;
    it.fresh = 1;
    if (++it.rg < nrg) return it;
    it.rg = 0;
    if (++it.pair < p.pairs) return it;
    it.pair = 0;
    int b = it.b + 1;
    while (of(b, p.ctx_len[b]) == 0) ++b;
    at_sequence(it, b);
    return it;
  }
  __device__ __forceinline__ int blocks(const DiffItem& it) const {
    const int n = min(window_keys(it.w), it.ctx + p.M - 1 - window_start(it.w));
    return (n + kBlockBk - 1) / kBlockBk;
  }
};

// The rows of sequences that break the rules: NaN and the error bit.
__device__ __forceinline__ void mark_bad_sequences(const DiffParams& p) {
  const int64_t n = (int64_t)p.M * (p.Hq / 2) * 2 * kD;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (diff_valid(p, b, p.ctx_len[b])) continue;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) p.out[b * n + i] = __int_as_float(0x7fc00000);
    if (threadIdx.x == 0) atomicOr(p.err_word, KATTN_DEVERR_BAD_SEQUENCE);
  }
}

// 2-D view [rows][128] of an 8-bit cache; kBlockBk-row boxes, 128-byte swizzle.
inline bool encode_plane_map(CUtensorMap* map, const void* base, int64_t rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 enc = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kD};
  const cuuint32_t box[2] = {(cuuint32_t)kD, (cuuint32_t)kBlockBk};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace kattn
