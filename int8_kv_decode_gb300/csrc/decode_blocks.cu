// Decode attention over a paged cache whose 8-bit rows share a scale per block of R =
// 32, 64 or 128 rows and head:
//   out = softmax(q K^T sm_scale) V,  K = k_scale[block] k8,  V = v_scale[block] v8
//
// Two launches: split_kernel reduces windows of the keys, merge_kernel joins the windows
// of a row.  A sequence of one window is finished by the first.
//
// A warp takes a unit: sequence, window, kv head and up to 16 of the rows (query heads x
// draft columns) that read the head.  It streams the window in steps of 32 keys through
// its own ring in shared memory (TMA, two stages), and per step
//   * S^T = K Q^T on f16 MMAs: the codes are exact in f16, and so are bf16 and f16
//     queries scaled by a power of two per row (float32 queries as f16 hi + lo, 22 bits),
//     so the products are exact and the sums float32;
//   * all 32 keys share a scale, so a score is one product and one sum: x = S c - m, with
//     c = k_scale * row factor, in base 2;
//   * weights 2^x; the reference m of a row moves only where a weight would pass 2^15;
//   * the weights go to f16 (float32 queries: hi + lo) and, through a transposition of
//     8 x 8 blocks in registers, to the second product, whose row sums take the weights
//     as rounded: a weight's rounding then cancels where it dominates;
//   * O = O + v_scale (V^T P^T): the product of a step starts at zero and enters the
//     float32 sum with the block's scale, so scales of any range need no care.
// The K and V codes are converted once for all rows of the unit.
#include "blocks_internal.cuh"
#include "decode_diff.cuh"

namespace kattn {
namespace {

constexpr int kWarpsB = 4, kThreadsB = kWarpsB * 32;
constexpr int kStages = 2;
constexpr float kTop = 9.0f;                      // weights are 2^9 at the reference
constexpr float kMoveAt = 15.0f;                  // and reach 2^15 before it moves

// Windows sit at fixed key positions, so that a row's bytes depend on its own keys
// alone: the first kNear keys in windows of 128, the others in windows of 256.
constexpr int kNearKeys = 128, kFarKeys = 256, kNear = 1024;
static_assert(kFarKeys / kBlockBk <= 32, "a lane holds the row and scales of each block of a window");
__host__ __device__ inline int block_windows(int keys) {
  return keys <= kNear ? (keys + kNearKeys - 1) / kNearKeys
                       : kNear / kNearKeys + (keys - kNear + kFarKeys - 1) / kFarKeys;
}
__host__ __device__ inline int block_window_start(int w) {
  return w < kNear / kNearKeys ? w * kNearKeys : kNear + (w - kNear / kNearKeys) * kFarKeys;
}
__host__ __device__ inline int block_stride(int R) { return R * kD + (2 * R + 3) / 4 * 4; }   // floats

struct BlockItem {
  int b, kh, w, rg, ctx;                          // b < 0: none
};

__device__ __forceinline__ bool context_valid(const BlockDecodeParams& p, int ctx) {
  const int64_t keys = (int64_t)ctx + p.M - 1;
  return ctx >= 1 && ctx <= p.max_ctx &&
         ((keys + (1 << p.c.page_shift) - 1) >> p.c.page_shift) <= (int64_t)p.c.max_pages;
}

// The units of a batch: per sequence, head and row group its windows.  Cost is counted
// in steps of 128 keys, and a worker takes the units that start in its share of it.
struct BlockUnits {
  const BlockDecodeParams& p;
  const int* prefix;                              // cost before each group of gs sequences
  int gs, ng, nrg;
  __device__ __forceinline__ BlockUnits(const BlockDecodeParams& params, const int* sums, int row_groups)
      : p(params), prefix(sums), nrg(row_groups) {
    gs = (p.B + kMaxGroups - 1) / kMaxGroups;
    ng = (p.B + gs - 1) / gs;
  }
  __device__ __forceinline__ int steps(int ctx) const { return (ctx + p.M - 1 + kNearKeys - 1) / kNearKeys; }
  __device__ __forceinline__ int of(int ctx) const {
    return context_valid(p, ctx) ? steps(ctx) * p.c.Hkv * nrg : 0;
  }
  // Fills sums[kMaxGroups + 1], for a block of kThreadsB threads.
  __device__ __forceinline__ void count(int* sums, int* scratch) const {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kPer = kMaxGroups / kThreadsB;
    int n[kPer], run = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = tid * kPer + i;
      n[i] = 0;
      if (at < ng)
        for (int b = at * gs; b < min(p.B, at * gs + gs); ++b) n[i] += of(__ldg(p.ctx_len + b));
      run += n[i];
    }
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int base = incl - run;
#pragma unroll
    for (int w = 0; w < kWarpsB; ++w)
      if (w < warp) base += scratch[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      sums[tid * kPer + i] = base;
      base += n[i];
    }
    if (tid == kThreadsB - 1) sums[kMaxGroups] = base;
  }
  // The first unit that starts in [*at, end) of the cost; b < 0: none.
  __device__ __forceinline__ BlockItem find(int* at, int end) const {
    BlockItem it{-1, 0, 0, 0, 0};
    if (*at >= end) return it;
    int lo = 0, hi = ng;                          // prefix[lo] <= *at < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= *at) lo = mid;
      else hi = mid;
    }
    int i = *at - prefix[lo], b = lo * gs, ctx = __ldg(p.ctx_len + b);
    for (int n; i >= (n = of(ctx));) {
      i -= n;
      ctx = __ldg(p.ctx_len + ++b);
    }
    const int all = steps(ctx), run = i / all;
    i -= run * all;
    const int key = i * kNearKeys;
    it.w = key <= kNear ? i : kNear / kNearKeys + (key - kNear + kFarKeys - 1) / kFarKeys;
    it.b = b;
    it.ctx = ctx;
    it.kh = run / nrg;
    it.rg = run - it.kh * nrg;
    *at += min(block_window_start(it.w) / kNearKeys, all) - i;
    if (*at >= end) it.b = -1;
    else if (it.w >= block_windows(ctx + p.M - 1)) it = after(it);
    return it;
  }
  // The unit that follows `it` (there is one), without a look at the order of lengths.
  __device__ __forceinline__ BlockItem after(BlockItem it) const {
    if (++it.w < block_windows(it.ctx + p.M - 1)) return it;
    it.w = 0;
    if (++it.rg < nrg) return it;
    it.rg = 0;
    if (++it.kh < p.c.Hkv) return it;
    it.kh = 0;
    do {
      it.ctx = __ldg(p.ctx_len + ++it.b);
    } while (!context_valid(p, it.ctx));
    return it;
  }
  // Cost of the unit, and its blocks of 32 keys.
  __device__ __forceinline__ int cost(const BlockItem& it) const {
    return min(block_window_start(it.w + 1) / kNearKeys, steps(it.ctx)) - block_window_start(it.w) / kNearKeys;
  }
  __device__ __forceinline__ int blocks(const BlockItem& it) const {
    const int s0 = block_window_start(it.w);
    return (min(block_window_start(it.w + 1), it.ctx + p.M - 1) - s0 + kBlockBk - 1) / kBlockBk;
  }
};

template <int T, bool kPrecise>
struct __align__(1024) BlockSmem {
  uint8_t ring[kWarpsB][kStages][2][kBlockBytes];         // [stage][K | V]
  // f16 queries (hi, and lo): row r's 16-byte chunk of channels 8 i at chunk
  // 4 (i % 4) + i / 4, XOR 4 in odd rows: a lane's loads of its 32 channels spread
  // over the banks
  uint4 q[kWarpsB][T][kPrecise ? 2 : 1][8][kD / 8];
  float factor[kWarpsB][T][8];                            // scores' factor of each row
  uint64_t full[kWarpsB][kStages];
  int prefix[kMaxGroups + 1];
  int scratch[kWarpsB];
};

// K and V rows of 32 keys into a stage, by one lane (predicated).
__device__ __forceinline__ void load_block(uint32_t dst, const TmaMaps& maps, int row, uint32_t bar,
                                           uint64_t policy) {
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n"
      " @p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%5], %7;\n"
      " @p cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%5], %6;\n"
      " @p cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%8], [%2, {%3, %4}], [%5], %6;\n}\n" ::"r"(dst),
      "l"(&maps.k), "l"(&maps.v), "r"(0), "r"(row), "r"(bar), "l"(policy), "r"((uint32_t)(2 * kBlockBytes)),
      "r"(dst + kBlockBytes)
      : "memory");
}

// Two codes of a word as f16x2, exact: bytes 0 and 1, or 2 and 3 (kPairs), or 0 and 2,
// then 1 and 3.
__device__ __forceinline__ uint32_t e4m3_h2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
template <bool kE4m3, bool kAlternate>
__device__ __forceinline__ void codes_h2(uint32_t w, uint32_t& a, uint32_t& b) {
  if constexpr (kE4m3) {
    if (kAlternate) w = __byte_perm(w, 0, 0x3120u);
    a = e4m3_h2(w);
    b = e4m3_h2(w >> 16);
  } else {
    w ^= 0x80808080u;
    a = i8pair_to_h2(w, kAlternate ? 0x4240u : 0x4140u);
    b = i8pair_to_h2(w, kAlternate ? 0x4341u : 0x4342u);
  }
}
// e4m3 codes that are no numbers as 0 (0 * NaN would reach rows that do not see the key).
__device__ __forceinline__ uint32_t numbers_only(uint32_t w) {
  return w & ~__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma_zero(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7},"
      " {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(0.0f));
}

// Four elements of a query row as float32.
__device__ __forceinline__ float4 load_query4(const void* q, int type, int64_t at) {
  if (type == KATTN_F32) return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(q) + at));
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + at));
  if (type == KATTN_BF16)
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
// Two neighbouring channels of the output, rounded once to its type.
__device__ __forceinline__ void store_out2(void* out, int type, int64_t at, float x, float y) {
  if (type == KATTN_F32) {
    *reinterpret_cast<float2*>(static_cast<float*>(out) + at) = make_float2(x, y);
  } else if (type == KATTN_BF16) {
    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(out) + at) = __floats2bfloat162_rn(x, y);
  } else {
    *reinterpret_cast<__half2*>(static_cast<__half*>(out) + at) = __floats2half2_rn(x, y);
  }
}

// Rows of sequences without keys are 0; of those that break the rules NaN, and flagged.
__device__ __forceinline__ void fill_other_rows(const BlockDecodeParams& p) {
  const int64_t n = (int64_t)p.M * p.Hq * kD;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int ctx = __ldg(p.ctx_len + b);
    if (context_valid(p, ctx)) continue;
    const float v = ctx == 0 ? 0.0f : __int_as_float(0x7fc00000);
    for (int64_t i = 2 * threadIdx.x; i < n; i += 2 * blockDim.x) store_out2(p.out, p.q_type, b * n + i, v, v);
    if (ctx != 0 && threadIdx.x == 0) atomicOr(p.err_word, KATTN_DEVERR_BAD_SEQUENCE);
  }
}

template <int T, bool kE4m3, bool kPrecise>
__global__ void __launch_bounds__(kThreadsB, T == 1 ? 3 : 2)
block_split_kernel(const BlockDecodeParams p, const __grid_constant__ TmaMaps maps) {
  using Smem = BlockSmem<T, kPrecise>;
  constexpr int kUnitRows = 8 * T, kParts = kPrecise ? 2 : 1;
  extern __shared__ unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + (0u - smem_u32(smem_raw)) % 1024u);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int g = lane >> 2, c = lane & 3;
  const int M = p.M, R = p.R;
  const int nrg = (R + kUnitRows - 1) / kUnitRows;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&sm.full[warp][i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  const BlockUnits units(p, sm.prefix, nrg);
  units.count(sm.prefix, sm.scratch);
  fill_other_rows(p);
  __syncthreads();
  griddep_launch_dependents();
  const int total = sm.prefix[kMaxGroups];
  // (blocks s, s + sms, ... start on the same multiprocessor: their warps are numbered one
  // after the other, so that the work of each multiprocessor is the same)
  const int G = gridDim.x * kWarpsB;
  const int per_sm = gridDim.x / p.sms, more = gridDim.x - per_sm * p.sms, on = blockIdx.x % p.sms;
  const int worker = (on * per_sm + min(on, more) + blockIdx.x / p.sms) * kWarpsB + warp;
  int u = (int)((int64_t)worker * total / G);
  const int u_end = (int)((int64_t)(worker + 1) * total / G);
  BlockItem it = units.find(&u, u_end);
  if (it.b < 0) return;

  const uint32_t ginv = 65536u / (uint32_t)p.g + 1u;      // rr / g for rr < 64
  auto column = [&](int rr) -> int { return (int)(((uint32_t)rr * ginv) >> 16); };
  // What lane e holds of block e of an item: the table's entry, then the row in the 2-D
  // view of all planes, and the scales of K and V.
  auto entry_of = [&](const BlockItem& x) -> int {
    const int key = block_window_start(x.w) + lane * kBlockBk;
    if (x.b < 0 || lane >= units.blocks(x)) return 0;
    return __ldg(p.c.block_table + (int64_t)x.b * p.c.max_pages + (key >> p.c.page_shift));
  };
  auto row_of = [&](const BlockItem& x, int page) -> int {
    const int key = block_window_start(x.w) + lane * kBlockBk;
    if (x.b < 0 || lane >= units.blocks(x)) return 0;
    if ((unsigned)page >= (unsigned)p.c.n_pages) {
      atomicOr(p.err_word, KATTN_DEVERR_BAD_PAGE);
      page = 0;
    }
    return x.kh * p.c.cap_rows + ((page << p.c.page_shift) | (key & ((1 << p.c.page_shift) - 1)));
  };
  auto next_of = [&](const BlockItem& x) -> BlockItem {
    u += units.cost(x);
    if (u < u_end) return units.after(x);
    return BlockItem{-1, 0, 0, 0, 0};
  };
  const uint32_t ring = smem_u32(sm.ring[warp]), bars = smem_u32(sm.full[warp]);
  const uint64_t policy = nrg > 1 ? l2_evict_normal() : l2_evict_first();

  // the current item and the next
  int row = row_of(it, entry_of(it));
  float ks = __ldg(p.c.k_scale + (row >> p.c.block_shift)), vs = __ldg(p.c.v_scale + (row >> p.c.block_shift));
  BlockItem nx = next_of(it);
  int entry = entry_of(nx), row_n = 0;
  float ks_n = 0.0f, vs_n = 0.0f;
  int nb = units.blocks(it), nb_n = nx.b >= 0 ? units.blocks(nx) : 0;

  // copies: block `ahead` of the current item (blocks past its last are the next's) is
  // the next to be issued; `issued` and `taken` count them
  uint32_t issued = 0, taken = 0;
  int ahead = 0;
  auto issue = [&](bool next_known) {
    while (issued - taken < kStages && (ahead < nb || (next_known && ahead - nb < nb_n))) {
      const int r = ahead < nb ? __shfl_sync(0xffffffffu, row, ahead) : __shfl_sync(0xffffffffu, row_n, ahead - nb);
      const uint32_t st = issued % kStages;
      load_block(ring + st * 2 * kBlockBytes, maps, r, bars + 8 * st, policy);
      ++issued;
      ++ahead;
    }
  };
  issue(false);
  int fresh_b = -1, fresh_kh = -1, fresh_rg = -1;

  for (;;) {
    const int s0 = block_window_start(it.w);
    // ---- the unit's queries
    if (it.b != fresh_b || it.kh != fresh_kh || it.rg != fresh_rg) {
      fresh_b = it.b;
      fresh_kh = it.kh;
      fresh_rg = it.rg;
      __syncwarp();
#pragma unroll 1
      for (int n = 0; n < T; ++n) {
        float4 x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int rr = it.rg * kUnitRows + 8 * n + r, j = column(min(rr, R - 1));
          x[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (rr < R)
            x[r] = load_query4(p.q, p.q_type,
                               (((int64_t)it.b * M + j) * p.Hq + it.kh * p.g + rr - j * p.g) * kD + 4 * lane);
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          // scaled so that the row's largest lies in [2^14, 2^15): then bf16 elements down to
          // 2^-28 of it are exact, and f16 sums of products cannot overflow float32
          const float own = fmaxf(fmaxf(fabsf(x[r].x), fabsf(x[r].y)), fmaxf(fabsf(x[r].z), fabsf(x[r].w)));
          const float big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(own)));
          const float up = power_scale(14, big);
          const float4 y = make_float4(x[r].x * up, x[r].y * up, x[r].z * up, x[r].w * up);
          uint2 hi, lo;
          split_f16x2(y.x, y.y, hi.x, lo.x);
          split_f16x2(y.z, y.w, hi.y, lo.y);
          const int chunk = lane >> 1, at = (4 * (chunk & 3) + (chunk >> 2)) ^ (4 * (r & 1));
          reinterpret_cast<uint2*>(&sm.q[warp][n][0][r][at])[lane & 1] = hi;
          if constexpr (kPrecise) reinterpret_cast<uint2*>(&sm.q[warp][n][kParts - 1][r][at])[lane & 1] = lo;
          if (lane == 0) sm.factor[warp][n][r] = __fmul_rn(__fmul_rn(p.sm_scale, kLog2e), inverse_scale(up));
        }
      }
      __syncwarp();
    }
    // keys that the thread's rows 2c, 2c + 1 of each tile see
    int keys[T][2];
#pragma unroll
    for (int n = 0; n < T; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        keys[n][e] = it.ctx + column(min(it.rg * kUnitRows + 8 * n + 2 * c + e, R - 1));

    float2 m[T], l[T];                            // references and row sums of rows 2c, 2c + 1
    float o[8][T][4];                             // [16 channels][tile]
#pragma unroll
    for (int n = 0; n < T; ++n) {
      m[n] = make_float2(-INFINITY, -INFINITY);
      l[n] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int md = 0; md < 8; ++md)
#pragma unroll
        for (int v = 0; v < 4; ++v) o[md][n][v] = 0.0f;
    }

#pragma unroll 1
    for (int i = 0; i < nb; ++i) {
      const int t0 = s0 + i * kBlockBk;
      const float ksb = __shfl_sync(0xffffffffu, ks, i), vsb = __shfl_sync(0xffffffffu, vs, i);
      const uint32_t st = taken % kStages, kbuf = ring + st * 2 * kBlockBytes, vbuf = kbuf + kBlockBytes;
      const bool edge = t0 + kBlockBk > it.ctx;   // keys that some row does not see
      if (!stage_ready(bars + 8 * st, (taken / kStages) & 1u)) {
        // a copy never arrived: flag it, give the others in flight a bounded chance, leave
        if (lane == 0) {
          atomicOr(p.err_word, KATTN_DEVERR_TIMEOUT);
          for (uint32_t k = taken + 1; k < issued; ++k)
            mbar_wait_bounded(&sm.full[warp][k % kStages], (k / kStages) & 1u);
        }
        return;
      }
      // ---- S^T = K Q^T: keys 16 half + g (+ 8), rows 2c, 2c + 1 of tile n
      float s[T][2][4];
#pragma unroll
      for (int part = 0; part < 2; ++part) {      // 64 channels: chunks 2c + part of the rows
        const uint32_t ka = kbuf + (uint32_t)swz(g, 2 * c + part);
        const uint4 kw[4] = {lds128a<0>(ka), lds128a<8 * kD>(ka), lds128a<16 * kD>(ka), lds128a<24 * kD>(ka)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 qw[T][kParts];
#pragma unroll
          for (int n = 0; n < T; ++n)
#pragma unroll
            for (int w = 0; w < kParts; ++w)
              qw[n][w] = sm.q[warp][n][w][g][(4 * (2 * part + h) + c) ^ (4 * (g & 1))];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t a[2][4];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint4 w0 = kw[2 * hf], w1 = kw[2 * hf + 1];
              codes_h2<kE4m3, false>(h == 0 ? (x == 0 ? w0.x : w0.y) : (x == 0 ? w0.z : w0.w), a[hf][0], a[hf][2]);
              codes_h2<kE4m3, false>(h == 0 ? (x == 0 ? w1.x : w1.y) : (x == 0 ? w1.z : w1.w), a[hf][1], a[hf][3]);
            }
#pragma unroll
            for (int n = 0; n < T; ++n)
#pragma unroll
              for (int w = 0; w < kParts; ++w) {
                const uint2 b = x == 0 ? make_uint2(qw[n][w].x, qw[n][w].y) : make_uint2(qw[n][w].z, qw[n][w].w);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                  if (part == 0 && h == 0 && x == 0 && w == 0) mma_zero(s[n][hf], a[hf], b);
                  else mma_f16(s[n][hf], a[hf], b);
                }
              }
          }
        }
      }
      // ---- weights
      uint2 pf[T][2][kParts];                     // the second product's operand: [half]
      float2 gain[T];                             // v_scale, for the rows that see a key of the block
#pragma unroll
      for (int n = 0; n < T; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(&sm.factor[warp][n][2 * c]);
        const float2 cf = f2_mul(f, make_float2(ksb, ksb));
        float2 x[2][2];                           // [half][key g | g + 8]
        auto scores = [&](float2 ref) {
          const float2 down = make_float2(-ref.x, -ref.y);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2)
              x[hf][k2] = f2_fma(make_float2(s[n][hf][2 * k2], s[n][hf][2 * k2 + 1]), cf, down);
          if (edge) hide_keys(x, t0 + g, keys[n][0], keys[n][1]);
        };
        scores(m[n]);                             // (a reference of -inf: +inf, above the limit)
        auto largest = [&]() -> float2 {
          return make_float2(fmaxf(fmaxf(x[0][0].x, x[0][1].x), fmaxf(x[1][0].x, x[1][1].x)),
                             fmaxf(fmaxf(x[0][0].y, x[0][1].y), fmaxf(x[1][0].y, x[1][1].y)));
        };
        const float2 most = largest();
        if (__any_sync(0xffffffffu, most.x > kMoveAt || most.y > kMoveAt)) {
          // A row's reference moves, to where its largest score has the weight 2^kTop.  (Which
          // rows move goes by the sums that asked for it, so it depends on the row alone.)
          auto row_most = [&](float2 v) -> float2 {
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
              v.x = fmaxf(v.x, __shfl_xor_sync(0xffffffffu, v.x, d));
              v.y = fmaxf(v.y, __shfl_xor_sync(0xffffffffu, v.y, d));
            }
            return v;
          };
          const float2 over = row_most(most);
          scores(make_float2(0.0f, 0.0f));
          const float2 top = row_most(largest());
          auto move = [&](float over, float top, float& ref) -> float {    // the factor of what is summed up
            if (!(over > kMoveAt)) return 1.0f;
            const float to = __fsub_rn(top, kTop);
            const float by = ref == -INFINITY ? 0.0f : fast_exp2(__fsub_rn(ref, to));
            ref = to;
            return by;
          };
          const float2 al = make_float2(move(over.x, top.x, m[n].x), move(over.y, top.y, m[n].y));
          l[n] = f2_mul(l[n], al);
#pragma unroll
          for (int md = 0; md < 8; ++md) {
            const float2 a0 = f2_mul(make_float2(o[md][n][0], o[md][n][1]), al);
            const float2 a1 = f2_mul(make_float2(o[md][n][2], o[md][n][3]), al);
            o[md][n][0] = a0.x; o[md][n][1] = a0.y; o[md][n][2] = a1.x; o[md][n][3] = a1.y;
          }
          scores(m[n]);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float2 w0 = make_float2(fast_exp2(x[hf][0].x), fast_exp2(x[hf][0].y));
          const float2 w1 = make_float2(fast_exp2(x[hf][1].x), fast_exp2(x[hf][1].y));
          if constexpr (kPrecise) {
            uint32_t h0, l0, h1, l1;
            split_f16x2(w0.x, w0.y, h0, l0);
            split_f16x2(w1.x, w1.y, h1, l1);
            pf[n][hf][0] = make_uint2(transpose8(h0), transpose8(h1));
            pf[n][hf][kParts - 1] = make_uint2(transpose8(l0), transpose8(l1));
          } else {
            const __half2 h0 = __floats2half2_rn(w0.x, w0.y), h1 = __floats2half2_rn(w1.x, w1.y);
            pf[n][hf][0] = make_uint2(transpose8(*reinterpret_cast<const uint32_t*>(&h0)),
                                      transpose8(*reinterpret_cast<const uint32_t*>(&h1)));
          }
        }
        gain[n] = make_float2(vsb, vsb);
        if (edge) gain[n] = make_float2(t0 < keys[n][0] ? vsb : 0.0f, t0 < keys[n][1] ? vsb : 0.0f);
        // row sums: a product with ones
        const uint32_t ones[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
        float r[4];
        mma_zero(r, ones, pf[n][0][0]);
        mma_f16(r, ones, pf[n][1][0]);
        if constexpr (kPrecise) {
          mma_f16(r, ones, pf[n][0][kParts - 1]);
          mma_f16(r, ones, pf[n][1][kParts - 1]);
        }
        l[n] = f2_add(l[n], make_float2(r[0], r[1]));
      }
      // ---- O += v_scale V^T P^T.  Row g of m-tile q is channel 16q + 2g, row g + 8 the next
      // one: a 16-bit element of the buffer is two channels of a key, so that the transposing
      // load pairs the keys 2c, 2c + 1 of both channels in a register.
      const uint32_t va = vbuf + (uint32_t)((lane & 15) * kD + (((lane >> 4) ^ (lane & 7)) << 4));
#pragma unroll
      for (int q = 0; q < 8; q += 2) {
        uint32_t vw[2][4];
        ldsm_x4_trans<0>(vw[0], va ^ (uint32_t)(q << 4));
        ldsm_x4_trans<2048>(vw[1], va ^ (uint32_t)(q << 4));
        if (kE4m3 && edge) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int k = 0; k < 4; ++k) vw[hf][k] = numbers_only(vw[hf][k]);
        }
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          uint32_t a[2][4];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            codes_h2<kE4m3, true>(vw[hf][2 * d], a[hf][0], a[hf][1]);
            codes_h2<kE4m3, true>(vw[hf][2 * d + 1], a[hf][2], a[hf][3]);
          }
#pragma unroll
          for (int n = 0; n < T; ++n) {
            float y[4];
            mma_zero(y, a[0], pf[n][0][0]);
            mma_f16(y, a[1], pf[n][1][0]);
            if constexpr (kPrecise) {
              mma_f16(y, a[0], pf[n][0][kParts - 1]);
              mma_f16(y, a[1], pf[n][1][kParts - 1]);
            }
            float* to = o[q + d][n];
            const float2 r0 = f2_fma(make_float2(y[0], y[1]), gain[n], make_float2(to[0], to[1]));
            const float2 r1 = f2_fma(make_float2(y[2], y[3]), gain[n], make_float2(to[2], to[3]));
            to[0] = r0.x; to[1] = r0.y; to[2] = r1.x; to[3] = r1.y;
          }
        }
      }
      ++taken;
      if (i == 0) {                               // the next item's rows and scales
        row_n = row_of(nx, entry);
        ks_n = nx.b >= 0 ? __ldg(p.c.k_scale + (row_n >> p.c.block_shift)) : 0.0f;
        vs_n = nx.b >= 0 ? __ldg(p.c.v_scale + (row_n >> p.c.block_shift)) : 0.0f;
      }
      __syncwarp();
      issue(true);
    }

    // ---- the window's result
    const bool whole = block_windows(it.ctx + M - 1) == 1;
    float* part = p.partials + (((size_t)it.b * p.nwin_max + it.w) * p.c.Hkv + it.kh) * block_stride(R);
#pragma unroll
    for (int n = 0; n < T; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = it.rg * kUnitRows + 8 * n + 2 * c + e;
        if (rr >= R) continue;
        const float lr = e ? l[n].y : l[n].x;
        if (whole) {
          const int j = column(rr);
          const int64_t at = (((int64_t)it.b * M + j) * p.Hq + it.kh * p.g + rr - j * p.g) * kD + 2 * g;
#pragma unroll
          for (int md = 0; md < 8; ++md)
            store_out2(p.out, p.q_type, at + 16 * md, __fdiv_rn(o[md][n][e], lr), __fdiv_rn(o[md][n][2 + e], lr));
        } else {
          float* dst = part + (size_t)rr * kD + 2 * g;
#pragma unroll
          for (int md = 0; md < 8; ++md)
            *reinterpret_cast<float2*>(dst + 16 * md) = make_float2(o[md][n][e], o[md][n][2 + e]);
          if (g == 0) {
            part[(size_t)R * kD + 2 * rr] = e ? m[n].y : m[n].x;
            part[(size_t)R * kD + 2 * rr + 1] = lr;
          }
        }
      }

    // ---- next item
    if (nx.b < 0) return;
    ahead -= nb;
    it = nx;
    row = row_n;
    ks = ks_n;
    vs = vs_n;
    nb = nb_n;
    nx = next_of(it);
    nb_n = nx.b >= 0 ? units.blocks(nx) : 0;
    entry = entry_of(nx);
    issue(false);
  }
}

// ------------------------------------------------------------------ merge
// Joins the windows of a row: W warps; the windows k, k + 8, ... are summed with the
// weights 2^(m_s - max m), for k = 0 .. 7, and the eight sums are added in order, so the
// order depends on neither W nor other rows.  A window in which a draft column's row sees
// no key has m = -inf and weight 0.
constexpr int kSums = 8, kBatchB = 4;

template <int W>
__global__ void __launch_bounds__(32 * W) block_merge_kernel(const BlockDecodeParams p) {
  constexpr int kOwn = kSums / W;
  __shared__ float4 s_o[kSums][kD / 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
  const int ctx = __ldg(p.ctx_len + b), R = p.R;
  const int kh = head / p.g, rr = j * p.g + head - kh * p.g;
  const size_t stride = (size_t)p.c.Hkv * block_stride(R);
  const float* base = p.partials + ((size_t)b * p.nwin_max * p.c.Hkv + kh) * block_stride(R);
  const float2* mlcol = reinterpret_cast<const float2*>(base + (size_t)R * kD) + rr;
  const float* ocol = base + (size_t)rr * kD + 4 * lane;
  const bool valid = context_valid(p, ctx) && block_windows(ctx + p.M - 1) > 1;
  griddep_wait();                                 // every partial is in place
  if (!valid) return;
  const int ns = block_windows(ctx + j);

  float4 v[kBatchB];
  auto load = [&](int s0) {
#pragma unroll
    for (int n = 0; n < kBatchB; ++n) {
      const int s = s0 + W * n + warp;
      v[n] = s < ns ? __ldcg(reinterpret_cast<const float4*>(ocol + s * stride)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  };
  auto stats = [&](int s) {                       // m, l of window s
    return s < ns ? __ldcg(reinterpret_cast<const float2*>(reinterpret_cast<const float*>(mlcol) + s * stride))
                  : make_float2(-INFINITY, 0.0f);
  };
  load(0);
  const float2 st0 = stats(lane);
  float mx = st0.x;
  for (int s = lane + 32; s < ns; s += 32) mx = fmaxf(mx, stats(s).x);
  mx = warp_max(mx);

  float4 acc[kOwn];
#pragma unroll
  for (int k = 0; k < kOwn; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f;
  for (int s0 = 0; s0 < ns; s0 += 32) {           // lane n weighs window s0 + n
    const float2 st = s0 ? stats(s0 + lane) : st0;
    const float w = fast_exp2(__fsub_rn(st.x, mx));       // (-inf: 0)
    l = __fmaf_rn(w, st.y, l);
#pragma unroll 1
    for (int at = 0; at < 32 && s0 + at < ns; at += W * kBatchB) {
      if (s0 + at > 0) load(s0 + at);
#pragma unroll
      for (int n = 0; n < kBatchB; ++n) {
        const float wn = __shfl_sync(0xffffffffu, w, at + W * n + warp);
        float4& x = acc[n % kOwn];
        x = make_float4(__fmaf_rn(wn, v[n].x, x.x), __fmaf_rn(wn, v[n].y, x.y), __fmaf_rn(wn, v[n].z, x.z),
                        __fmaf_rn(wn, v[n].w, x.w));
      }
    }
  }
  l = warp_sum(l);
#pragma unroll
  for (int k = 0; k < kOwn; ++k) s_o[k * W + warp][lane] = acc[k];
  __syncthreads();
  if (warp != 0) return;
  float4 O = s_o[0][lane];
#pragma unroll
  for (int k = 1; k < kSums; ++k) {
    const float4 x = s_o[k][lane];
    O = make_float4(__fadd_rn(O.x, x.x), __fadd_rn(O.y, x.y), __fadd_rn(O.z, x.z), __fadd_rn(O.w, x.w));
  }
  const int64_t at = (((int64_t)b * p.M + j) * p.Hq + head) * kD + 4 * lane;
  store_out2(p.out, p.q_type, at, __fdiv_rn(O.x, l), __fdiv_rn(O.y, l));
  store_out2(p.out, p.q_type, at + 2, __fdiv_rn(O.z, l), __fdiv_rn(O.w, l));
}

// ------------------------------------------------------------------- host
template <int T, bool kE4m3, bool kPrecise>
cudaError_t launch_split(BlockDecodeParams p, const TmaMaps& maps, cudaStream_t stream) {
  const auto kern = block_split_kernel<T, kE4m3, kPrecise>;
  const int smem = (int)sizeof(BlockSmem<T, kPrecise>) + 1024;     // + alignment slack
  // per device: the blocks that the GPU holds at once; the shared-memory limit is raised
  // with the first call
  static std::atomic<int> slots_cache[kMaxDevices], sms_cache[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  int slots = cached ? slots_cache[dev].load() : 0, sms = cached ? sms_cache[dev].load() : 0;
  if (slots <= 0 || sms <= 0) {
    int per_sm = 0;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreadsB, smem)) != cudaSuccess) return e;
    slots = sms * (per_sm > 0 ? per_sm : 1);
    if (cached) {
      slots_cache[dev].store(slots);
      sms_cache[dev].store(sms);
    }
  }
  p.sms = sms;
  kern<<<(unsigned)std::min<int64_t>(block_decode_units(p), slots), kThreadsB, smem, stream>>>(p, maps);
  return cudaGetLastError();
}
template <bool kE4m3>
cudaError_t launch_split(const BlockDecodeParams& p, const TmaMaps& maps, cudaStream_t stream) {
  const bool precise = p.q_type == KATTN_F32;
  if (p.R <= 8) return precise ? launch_split<1, kE4m3, true>(p, maps, stream) : launch_split<1, kE4m3, false>(p, maps, stream);
  return precise ? launch_split<2, kE4m3, true>(p, maps, stream) : launch_split<2, kE4m3, false>(p, maps, stream);
}

template <int W>
cudaError_t launch_merge(const BlockDecodeParams& p, cudaStream_t stream) {
  return launch_pdl(block_merge_kernel<W>, dim3((unsigned)p.Hq, (unsigned)p.M, (unsigned)p.B), dim3(32 * W), 0, stream, p);
}

}  // namespace

int64_t block_decode_units(const BlockDecodeParams& p) {
  const int rows = p.R <= 8 ? 8 : 16;
  return (int64_t)p.B * block_windows(p.max_ctx + p.M - 1) * p.c.Hkv * ((p.R + rows - 1) / rows);
}

size_t block_decode_workspace_bytes(int B, int M, int Hq, int max_ctx) {
  // Hkv * block_stride(R) <= Hq * (M * (d + 2) + 3) whatever Hkv is
  return 256 + (size_t)B * block_windows(max_ctx + M - 1) * Hq * (M * (kD + 2) + 3) * sizeof(float);
}

void set_block_decode_workspace(BlockDecodeParams& p, void* workspace) {
  p.err_word = static_cast<uint32_t*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  p.nwin_max = block_windows(p.max_ctx + p.M - 1);
}

cudaError_t launch_decode_blocks(const BlockDecodeParams& p, int code_type, cudaStream_t stream) {
  TmaMaps maps;
  const int64_t rows = (int64_t)p.c.Hkv * p.c.cap_rows;
  if (!encode_plane_map(&maps.k, p.c.k, rows) || !encode_plane_map(&maps.v, p.c.v, rows))
    return cudaErrorInvalidValue;
  const cudaError_t e = code_type == KATTN_E4M3 ? launch_split<true>(p, maps, stream)
                                                : launch_split<false>(p, maps, stream);
  if (e != cudaSuccess || p.nwin_max <= 1) return e;
  if (p.nwin_max <= 32) return launch_merge<2>(p, stream);
  if (p.nwin_max <= 256) return launch_merge<4>(p, stream);
  return launch_merge<8>(p, stream);
}

}  // namespace kattn
