// Decode attention over a paged cache whose 8-bit rows share a scale per block of R =
// 32, 64 or 128 rows and head:
//   out = softmax(q K^T sm_scale) V,  K = k_scale[block] k8,  V = v_scale[block] v8
//
// Two launches: split_kernel reduces windows of the keys, merge_kernel joins the windows
// of a row.  A sequence of one window is finished by the first.
//
// A block of four warps takes a unit: sequence, window of 512 keys, kv head and T tiles of 8
// of the rows (query heads x draft columns) that read the head; T = 1 to 5 (unit_tiles).
// Warp w takes the steps of 32 keys w, w + 4, ..., so a short window is shared by all four as
// well, and the warps' sums come together in shared memory: one partial a window.  (A warp
// per window of 256 keys took 122 us where this takes 97, 64 sequences of 512 to 32768 keys:
// more partials, larger shares of work per warp.)  A warp's K and V rows come by TMA into a
// buffer each, refilled for the step that follows as soon as its products are issued.  Per step
//   * S^T = K Q^T on f16 MMAs: the codes are exact in f16, and so are bf16 and f16
//     queries scaled by a power of two per row (float32 queries as f16 hi + lo, 22 bits),
//     so the products are exact and the sums float32;
//   * all 32 keys share a scale, so a score is one product and one sum: x = S c - m, with
//     c = k_scale * row factor, in base 2;
//   * weights 2^x; the reference m of a row moves only where a weight would pass 2^15;
//   * the weights go to f16 (float32 queries: hi + lo) and, through a transposition of
//     8 x 8 blocks in registers, to the second product, whose row sums take the weights
//     as rounded: a weight's rounding then cancels where it dominates.  11 bits, as hi + lo
//     doubles that product's MMAs: beside the output's own rounding they add nothing to see in
//     bf16 (1.68e-3 relative on 64 long contexts, where float32 weights give 1.67e-3), and a
//     third in f16 (2.7e-4, 2.1e-4); a call that wants more takes float32 queries;
//   * O = O + v_scale (V^T P^T): the product of a step starts at zero and enters the
//     float32 sum with the block's scale (a row that sees a huge one: kHuge).  From three
//     tiles on O lies in tensor memory, each lane's columns its own store, read and written
//     once a step: so the codes are converted once for up to 40 rows, the order of every
//     row's operations stays that of one tile, and three blocks still fit a multiprocessor.
//
// What bounds it.  Up to 8 rows a head, HBM: 64 sequences of 512 to 32768 keys over 64-row
// pages, 32 query and 4 kv heads (544 MB, 80 us at the measured copy rate): 97 us a call, the
// split alone 90 (6.0 TB/s), issue 42%.  2 sequences of 128k keys with float32 queries (267
// MB, 39 us): 56 us, split 49, of which the second MMAs for hi + lo take tensor pipe to 34%.
// With more rows, issue and the latency of a step's chain at 12 warps a multiprocessor (920
// instructions a step at T = 2, 330 of them to make f16 of the codes; 1620 at T = 5): 16
// sequences of 1k to 4k keys, 40 rows a head, 34 us; 64 of them 78 us.  One sequence of 257
// keys: 6.2 us, latency alone.
#include <cmath>

#include "blocks_internal.cuh"
#include "decode_diff.cuh"
#include "tcgen05_common.cuh"

namespace kattn {
namespace {

constexpr int kWarpsB = 4, kThreadsB = kWarpsB * 32;
constexpr float kTop = 9.0f;                      // weights are 2^9 at the reference
constexpr float kMoveAt = 15.0f;                  // and reach 2^15 before it moves
// A row whose reference is larger than this takes its scores as they are rounded, x = (S c)
// - m: x = S c - m in one rounding may be far off at the largest, whose own rounding made m.
// (Every step of a unit with such a row goes the way of a step that moves references.)
constexpr float kLarge = 1048576.0f;
// A warp's sums O of a row are up to 2^22 times the values (128 keys of weights up to 2^15),
// those of a long context up to 2^45 times.  So where a row sees a step of the warp's window
// with a v_scale of kHuge or more (values up to 2^128), its sums there are taken by kDown, a
// power of two: what it costs lies 2^126 below such values.  The sign of the row sum says so
// where sums are joined, which bring all of them to the same side.  A row goes by the steps
// that it sees itself, so its bytes stay its own, and those of a row with none are as they are.
// (Looking for such scales: 0.4% of 64 sequences of 512 to 32768 keys, 1.6% of 64 of 1k to 4k
// with 5 columns; a scale for each row in the loop took 3%.)
constexpr float kHuge = 0x1p64f, kDown = 0x1p-64f, kUp = 0x1p64f;
__device__ __forceinline__ bool is_down(float l) { return (int)__float_as_uint(l) < 0; }
__device__ __forceinline__ float mark_down(float l, bool down) {
  return down ? __uint_as_float(__float_as_uint(l) | 0x80000000u) : l;
}

// Windows of 512 keys sit at fixed positions, so that a row's bytes depend on its own keys
// alone.  (Windows of 1024 from key 4096 on: 103 us instead of 99, 64 sequences of 512 to
// 32768 keys, as fewer units spread less well.)
constexpr int kKeys = 512;
static_assert(kKeys / kBlockBk / kWarpsB <= 32, "a lane holds the row and scales of each of a warp's steps");
__host__ __device__ inline int block_windows(int keys) { return (keys + kKeys - 1) / kKeys; }
__host__ __device__ inline int block_stride(int R) { return R * kD + (2 * R + 3) / 4 * 4; }   // floats

struct BlockItem {
  int b, kh, w, rg, ctx;                          // b < 0: none
};

__device__ __forceinline__ bool context_valid(const BlockDecodeParams& p, int ctx) {
  const int64_t keys = (int64_t)ctx + p.M - 1;
  return ctx >= 1 && ctx <= p.max_ctx &&
         ((keys + (1 << p.c.page_shift) - 1) >> p.c.page_shift) <= (int64_t)p.c.max_pages;
}

// The units of a batch: per sequence, head and row group its windows.
struct BlockUnits {
  const BlockDecodeParams& p;
  const int* prefix;                              // units before each group of gs sequences
  int gs, ng, nrg;
  __device__ __forceinline__ BlockUnits(const BlockDecodeParams& params, const int* sums, int row_groups)
      : p(params), prefix(sums), nrg(row_groups) {
    gs = (p.B + kMaxGroups - 1) / kMaxGroups;
    ng = (p.B + gs - 1) / gs;
  }
  __device__ __forceinline__ int windows(int ctx) const { return block_windows(ctx + p.M - 1); }
  __device__ __forceinline__ int of(int ctx) const {
    return context_valid(p, ctx) ? windows(ctx) * p.c.Hkv * nrg : 0;
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
        for (int b = at * gs; b < min(p.B, at * gs + gs); ++b) n[i] += of(__ldcg(p.ctx_len + b));
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
  // Unit `at` (below `end`; b < 0: none).
  __device__ __forceinline__ BlockItem find(int at, int end) const {
    BlockItem it{-1, 0, 0, 0, 0};
    if (at >= end) return it;
    int lo = 0, hi = ng;                          // prefix[lo] <= at < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= at) lo = mid;
      else hi = mid;
    }
    int i = at - prefix[lo];
    it.b = lo * gs;
    it.ctx = __ldcg(p.ctx_len + it.b);
    for (int n; i >= (n = of(it.ctx));) {
      i -= n;
      it.ctx = __ldcg(p.ctx_len + ++it.b);
    }
    const int nw = windows(it.ctx), run = i / nw;
    it.w = i - run * nw;
    it.kh = run / nrg;
    it.rg = run - it.kh * nrg;
    return it;
  }
  // The unit that follows `it` (there is one).
  __device__ __forceinline__ BlockItem after(BlockItem it) const {
    if (++it.w < windows(it.ctx)) return it;
    it.w = 0;
    if (++it.rg < nrg) return it;
    it.rg = 0;
    if (++it.kh < p.c.Hkv) return it;
    it.kh = 0;
    do {
      it.ctx = __ldcg(p.ctx_len + ++it.b);
    } while (!context_valid(p, it.ctx));
    return it;
  }
  // Its blocks of 32 keys.
  __device__ __forceinline__ int blocks(const BlockItem& it) const {
    return (min(kKeys, it.ctx + p.M - 1 - it.w * kKeys) + kBlockBk - 1) / kBlockBk;
  }
};

// Where the sums O of a unit's T tiles of 8 rows are kept: in registers (32 a tile) for one
// or two tiles, else in tensor memory, a lane's own columns as its own store: per 16
// channels the first kLow columns of the tiles side by side, then the others.
template <int T>
struct Sums {
  static constexpr bool kTensor = T > 2;
  static constexpr int kLow = T == 3 ? 8 : 16, kHigh = 4 * T - kLow;
  // columns allocated, powers of two (with 256 for T = 5 two blocks would have room)
  enum : int { kFirst = 128, kSecond = T == 5 ? 32 : 0 };
  static constexpr int kJoin = kTensor ? 1 : T;           // tiles that the warps join at a time
};
constexpr int kPerSm = 3;                         // blocks a multiprocessor holds

template <int T, bool kPrecise>
struct __align__(1024) BlockSmem {
  uint8_t ring[kWarpsB][2][kBlockBytes];                  // [K | V] of each warp
  // the warps' sums of a unit's tiles, in the order of the MMA's registers; their
  // references and row sums
  float4 o[kWarpsB][Sums<T>::kJoin][8][32];
  float2 ml[kWarpsB][T][8];
  // f16 queries (hi, and lo): row r's 16-byte chunk of channels 8 i at chunk
  // 4 (i % 4) + i / 4, XOR 4 in odd rows: a lane's loads of its 32 channels spread
  // over the banks
  uint4 q[T][kPrecise ? 2 : 1][8][kD / 8];
  float factor[T][8];                                     // scores' factor of each row
  uint64_t full[kWarpsB][2];
  int prefix[kMaxGroups + 1];
  int scratch[kWarpsB];
  int failed;                                             // a warp's copy never arrived
  uint32_t tensor[2];                                     // tensor memory
};

// 4, 8 or 16 columns of this warp's lanes of tensor memory.  Loads are in place after
// tensor_loaded, stores after tc_wait_st.
template <int N>
__device__ __forceinline__ void tensor_load(uint32_t at, uint32_t* v) {
  if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at));
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(at));
  } else {
    static_assert(N == 16);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at));
  }
}
template <int N>
__device__ __forceinline__ void tensor_store(uint32_t at, const uint32_t* v) {
  if constexpr (N == 4) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3])
                 : "memory");
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(at), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_assert(N == 16);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n"
        ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
  }
}
template <int N>
__device__ __forceinline__ void tensor_loaded(uint32_t (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));    // (no use of it comes before)
}
__device__ __forceinline__ float2 as_float2(uint32_t x, uint32_t y) {
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}

// Rows of 32 keys of a plane into a buffer, by one lane (predicated).
__device__ __forceinline__ void load_block(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar,
                                           uint64_t policy) {
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n"
      " @p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%4], %6;\n"
      " @p cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;\n}\n" ::"r"(dst),
      "l"(map), "r"(0), "r"(row), "r"(bar), "l"(policy), "r"((uint32_t)kBlockBytes)
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

// The smaller; NaN if x is.  (fminf gives the other one.)
__device__ __forceinline__ float min_or_nan(float x, float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(x), "f"(y));
  return r;
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
__device__ __forceinline__ float4 query_values(float4 x, int) { return x; }
__device__ __forceinline__ float4 query_values(uint2 w, int type) {
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
    const int ctx = __ldcg(p.ctx_len + b);
    if (context_valid(p, ctx)) continue;
    const float v = ctx == 0 ? 0.0f : __int_as_float(0x7fc00000);
    for (int64_t i = 2 * threadIdx.x; i < n; i += 2 * blockDim.x) store_out2(p.out, p.q_type, b * n + i, v, v);
    if (ctx != 0 && threadIdx.x == 0) atomicOr(p.err_word, KATTN_DEVERR_BAD_SEQUENCE);
  }
}

// (Blocks a multiprocessor holds: with 4, 128 registers a thread, and T = 1, 99 us instead
// of 96, 64 sequences of 512 to 32768 keys; float32 queries, 2 of 120k to 131k keys, 60
// instead of 55; one sequence as before.)
template <int T, bool kE4m3, bool kPrecise>
__global__ void __launch_bounds__(kThreadsB, kPerSm)
block_split_kernel(const BlockDecodeParams p, const __grid_constant__ TmaMaps maps) {
  using Smem = BlockSmem<T, kPrecise>;
  using S = Sums<T>;
  constexpr int kUnitRows = 8 * T, kParts = kPrecise ? 2 : 1;
  extern __shared__ unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + (0u - smem_u32(smem_raw)) % 1024u);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int g = lane >> 2, c = lane & 3;
  const int M = p.M, R = p.R;
  const int nrg = (R + kUnitRows - 1) / kUnitRows;
  if (lane == 0) {
    mbar_init(&sm.full[warp][0], 1);
    mbar_init(&sm.full[warp][1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid == 0) sm.failed = 0;
  griddep_wait();                                 // what the kernels before wrote is in place
  const BlockUnits units(p, sm.prefix, nrg);
  units.count(sm.prefix, sm.scratch);
  fill_other_rows(p);
  __syncthreads();
  griddep_launch_dependents();
  const int total = sm.prefix[kMaxGroups];
  // Each block of threads takes a run of units that follow one another.  (Blocks s, s + sms,
  // ... start on the same multiprocessor: they are numbered one after the other, so that the
  // work of each multiprocessor is the same.)
  const int G = gridDim.x;
  const int per_sm = G / p.sms, more = G - per_sm * p.sms, on = blockIdx.x % p.sms;
  const int worker = on * per_sm + min(on, more) + blockIdx.x / p.sms;
  int u = (int)((int64_t)worker * total / G);
  const int u_end = (int)((int64_t)(worker + 1) * total / G);
  BlockItem it = units.find(u, u_end);
  if (it.b < 0) return;
  if constexpr (S::kTensor) {
    if (warp == 0) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sm.tensor[0])),
                   "r"((int)S::kFirst));
      if constexpr (S::kSecond > 0)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n"
                     ::"r"(smem_u32(&sm.tensor[1])), "r"((int)S::kSecond));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    tc_fence_before();
  }

  const uint32_t ginv = 65536u / (uint32_t)p.g + 1u;      // rr / g for rr < 64
  auto column = [&](int rr) -> int { return (int)(((uint32_t)rr * ginv) >> 16); };
  // The warp's steps of an item: blocks warp, warp + 4, ... of its window.  What lane e holds
  // of step e: the table's entry, then the row in the 2-D view of all planes, and the scales.
  auto steps_of = [&](const BlockItem& x) -> int {
    return x.b < 0 ? 0 : (units.blocks(x) - warp + kWarpsB - 1) / kWarpsB;
  };
  auto key_of = [&](const BlockItem& x) -> int {
    return x.w * kKeys + (lane * kWarpsB + warp) * kBlockBk;
  };
  auto entry_of = [&](const BlockItem& x, int steps) -> int {
    if (lane >= steps) return 0;
    return __ldcg(p.c.block_table + (int64_t)x.b * p.c.max_pages + (key_of(x) >> p.c.page_shift));
  };
  auto row_of = [&](const BlockItem& x, int steps, int page) -> int {
    if (lane >= steps) return 0;
    if ((unsigned)page >= (unsigned)p.c.n_pages) {
      atomicOr(p.err_word, KATTN_DEVERR_BAD_PAGE);
      page = 0;
    }
    return x.kh * p.c.cap_rows + ((page << p.c.page_shift) | (key_of(x) & ((1 << p.c.page_shift) - 1)));
  };
  auto next_of = [&](const BlockItem& x) -> BlockItem {
    if (++u < u_end) return units.after(x);
    return BlockItem{-1, 0, 0, 0, 0};
  };
  // Queries of an item's rows, by the four warps together: 2 T rows each.  A row is scaled so
  // that its largest lies in [2^14, 2^15): bf16 elements down to 2^-28 of it are then exact,
  // and sums of products stay in float32.
  auto convert_queries = [&](const BlockItem& x) {
    using Raw = typename std::conditional<kPrecise, float4, uint2>::type;
    Raw v[2 * T];                                 // (all of them on their way at once)
#pragma unroll
    for (int i = 0; i < 2 * T; ++i) {
      const int rr = x.rg * kUnitRows + warp * 2 * T + i, j = column(min(rr, R - 1));
      v[i] = Raw{};
      if (rr < R) {
        const int64_t at = (((int64_t)x.b * M + j) * p.Hq + x.kh * p.g + rr - j * p.g) * kD + 4 * lane;
        v[i] = __ldcg(reinterpret_cast<const Raw*>(static_cast<const char*>(p.q) + at * (kPrecise ? 4 : 2)));
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * T; ++i) {
      const int n = (warp * 2 * T + i) >> 3, r = (warp * 2 * T + i) & 7;
      const float4 y = query_values(v[i], p.q_type);
      const float own = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
      const float big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(own)));
      const float up = power_scale(14, big);
      uint2 hi, lo;
      split_f16x2(y.x * up, y.y * up, hi.x, lo.x);
      split_f16x2(y.z * up, y.w * up, hi.y, lo.y);
      const int chunk = lane >> 1, at = (4 * (chunk & 3) + (chunk >> 2)) ^ (4 * (r & 1));
      reinterpret_cast<uint2*>(&sm.q[n][0][r][at])[lane & 1] = hi;
      if constexpr (kPrecise) reinterpret_cast<uint2*>(&sm.q[n][kParts - 1][r][at])[lane & 1] = lo;
      if (lane == 0) sm.factor[n][r] = __fmul_rn(__fmul_rn(p.sm_scale, kLog2e), inverse_scale(up));
    }
  };
  const uint32_t kbuf = smem_u32(sm.ring[warp][0]), vbuf = kbuf + kBlockBytes;
  const uint32_t kbar = smem_u32(&sm.full[warp][0]), vbar = kbar + 8;
  const uint64_t policy = nrg > 1 ? l2_evict_normal() : l2_evict_first();

  // the current item and the next
  int nb = steps_of(it);
  int row = row_of(it, nb, entry_of(it, nb));
  bool ahead = false;                             // the item's first step is on its way
  if (nb > 0) {
    const int r = __shfl_sync(0xffffffffu, row, 0);
    load_block(kbuf, &maps.k, r, kbar, policy);
    load_block(vbuf, &maps.v, r, vbar, policy);
    ahead = true;
  }
  float ks = __ldcg(p.c.k_scale + (row >> p.c.block_shift)), vs = __ldcg(p.c.v_scale + (row >> p.c.block_shift));
  BlockItem nx = next_of(it);
  int nb_n = steps_of(nx);
  int entry = entry_of(nx, nb_n);
  uint32_t ph = 0;                                // parity of the step's copies
  convert_queries(it);
  __syncthreads();
  uint32_t low = 0, high = 0;                     // this warp's lanes of tensor memory
  if constexpr (S::kTensor) {
    tc_fence_after();
    low = sm.tensor[0] + ((uint32_t)(32 * warp) << 16);
    high = S::kSecond > 0 ? sm.tensor[1] + ((uint32_t)(32 * warp) << 16) : low + 8 * S::kLow;
  }
  // tile n's four columns of the channels 16 md ..
  auto columns_of = [&](int md, int n) -> uint32_t {
    return n < S::kLow / 4 ? low + md * S::kLow + 4 * n : high + md * S::kHigh + 4 * (n - S::kLow / 4);
  };
#ifdef KATTN_BLOCKS_STAGE_LIMIT
  // Test builds only: the warps KATTN_BLOCKS_STAGE_WARPS (a bit each) take this many
  // copies, then find none ready.
  int copies = 0;
  auto ready = [&](uint32_t bar, uint32_t parity) {
    return !((KATTN_BLOCKS_STAGE_WARPS >> warp & 1) && copies++ >= KATTN_BLOCKS_STAGE_LIMIT) && stage_ready(bar, parity);
  };
#else
  auto ready = [&](uint32_t bar, uint32_t parity) { return stage_ready(bar, parity); };
#endif
  auto leave = [&]() {                            // by every warp: the tensor memory is given back
    if constexpr (S::kTensor) {
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      if (warp == 0) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(sm.tensor[0]), "r"((int)S::kFirst));
        if constexpr (S::kSecond > 0)
          asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(sm.tensor[1]), "r"((int)S::kSecond));
      }
    }
  };

  for (;;) {
    const int s0 = it.w * kKeys;
    if (nb > 0 && !ahead) {
      const int r = __shfl_sync(0xffffffffu, row, 0);
      load_block(kbuf, &maps.k, r, kbar, policy);
      load_block(vbuf, &maps.v, r, vbar, policy);
    }
    // the next item's rows and scales
    const int row_n = row_of(nx, nb_n, entry);
    const float ks_n = __ldcg(p.c.k_scale + (row_n >> p.c.block_shift));
    const float vs_n = __ldcg(p.c.v_scale + (row_n >> p.c.block_shift));
    const int first_n = __shfl_sync(0xffffffffu, row_n, 0);
    ahead = nb > 0 && nb_n > 0;
    // keys that the thread's row 2c + e of tile n sees
    auto keys_of = [&](int n, int e) -> int {
      return it.ctx + column(min(it.rg * kUnitRows + 8 * n + 2 * c + e, R - 1));
    };

    float2 m[T], l[T];                            // references and row sums of rows 2c, 2c + 1
    float o[S::kTensor ? 1 : 8][S::kTensor ? 1 : T][4];   // [16 channels][tile]
#pragma unroll
    for (int n = 0; n < T; ++n) {
      m[n] = make_float2(-INFINITY, -INFINITY);
      l[n] = make_float2(0.0f, 0.0f);
      if constexpr (!S::kTensor) {
#pragma unroll
        for (int md = 0; md < 8; ++md)
#pragma unroll
          for (int v = 0; v < 4; ++v) o[md][n][v] = 0.0f;
      }
    }
    if constexpr (S::kTensor) {
      uint32_t z[S::kLow];
#pragma unroll
      for (int i = 0; i < S::kLow; ++i) z[i] = 0u;
#pragma unroll
      for (int md = 0; md < 8; ++md) {
        tensor_store<S::kLow>(low + md * S::kLow, z);
        if constexpr (S::kHigh > 0) tensor_store<S::kHigh>(high + md * S::kHigh, z);
      }
      tc_wait_st();
    }
    // A copy never arrived: flag it; the block of threads leaves at the next barrier.
    auto give_up = [&]() {
      if (lane == 0) {
        atomicOr(p.err_word, KATTN_DEVERR_TIMEOUT);
        sm.failed = 1;
      }
    };
    int first_huge = INT32_MAX;                   // first key of the warp's first step with a huge scale
    auto goes_down = [&](int n, int e) { return first_huge < keys_of(n, e); };
    bool large = false;                           // some row's reference passes kLarge
    int flying = 0;                               // after giving up: copies on their way (1: K, 2: V, by parity)

#pragma unroll 1
    for (int i = 0; i < nb; ++i) {
      const int t0 = s0 + (i * kWarpsB + warp) * kBlockBk;
      const float ksb = __shfl_sync(0xffffffffu, ks, i);
      const int next = i + 1 < nb ? __shfl_sync(0xffffffffu, row, i + 1) : nb_n > 0 ? first_n : -1;
      const bool edge = t0 + kBlockBk > it.ctx;   // keys that some row does not see
      // Every row sees the steps that begin before ctx.  Behind it there is one at most, the
      // warp's last: the rows that see it go down there if its scale is the first huge one.
      const bool lowers = t0 >= it.ctx && t0 == first_huge;
      if (!ready(kbar, ph)) {
        give_up();
        flying = 3;
        break;
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
              qw[n][w] = sm.q[n][w][g][(4 * (2 * part + h) + c) ^ (4 * (g & 1))];
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
      __syncwarp();                               // (every lane's loads of the buffer have returned)
      if (next >= 0) load_block(kbuf, &maps.k, next, kbar, policy);
      // ---- weights
      uint2 pf[T][2][kParts];                     // the second product's operand: [half]
#pragma unroll
      for (int n = 0; n < T; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(&sm.factor[n][2 * c]);
        const float2 cf = f2_mul(f, make_float2(ksb, ksb));
        float2 x[2][2];                           // [half][key g | g + 8]
        auto scores = [&](float2 ref, bool rounded) {
          const float2 down = make_float2(-ref.x, -ref.y);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2)
              x[hf][k2] = f2_fma(make_float2(s[n][hf][2 * k2], s[n][hf][2 * k2 + 1]), cf, down);
          if (rounded) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int k2 = 0; k2 < 2; ++k2) {
                if (fabsf(ref.x) > kLarge) x[hf][k2].x = __fsub_rn(__fmul_rn(s[n][hf][2 * k2], cf.x), ref.x);
                if (fabsf(ref.y) > kLarge) x[hf][k2].y = __fsub_rn(__fmul_rn(s[n][hf][2 * k2 + 1], cf.y), ref.y);
              }
          }
          if (edge) hide_keys(x, t0 + g, keys_of(n, 0), keys_of(n, 1));
        };
        scores(m[n], false);                      // (a reference of -inf: +inf, above the limit)
        auto largest = [&]() -> float2 {
          return make_float2(fmaxf(fmaxf(x[0][0].x, x[0][1].x), fmaxf(x[1][0].x, x[1][1].x)),
                             fmaxf(fmaxf(x[0][0].y, x[0][1].y), fmaxf(x[1][0].y, x[1][1].y)));
        };
        const float2 most = largest();
        if (__any_sync(0xffffffffu, most.x > kMoveAt || most.y > kMoveAt) || large || lowers) {
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
          scores(m[n], true);
          const float2 over = row_most(largest());
          scores(make_float2(0.0f, 0.0f), false);
          const float2 top = row_most(largest());
          auto move = [&](float over, float top, float& ref) -> float {    // the factor of what is summed up
            if (!(over > kMoveAt)) return 1.0f;
            const float to = __fsub_rn(top, kTop);
            const float by = ref == -INFINITY ? 0.0f : fast_exp2(__fsub_rn(ref, to));
            ref = to;
            return by;
          };
          const float2 al = make_float2(move(over.x, top.x, m[n].x), move(over.y, top.y, m[n].y));
          large |= __any_sync(0xffffffffu, (fabsf(m[n].x) > kLarge && m[n].x > -INFINITY) ||
                                               (fabsf(m[n].y) > kLarge && m[n].y > -INFINITY));
          l[n] = f2_mul(l[n], al);
          float2 alo = al;                        // (of O)
          if (lowers && goes_down(n, 0)) alo.x = __fmul_rn(al.x, kDown);
          if (lowers && goes_down(n, 1)) alo.y = __fmul_rn(al.y, kDown);
          if (i == 0) {                           // (nothing is summed up yet)
          } else if constexpr (S::kTensor) {
            uint32_t v[32];
#pragma unroll
            for (int md = 0; md < 8; ++md) tensor_load<4>(columns_of(md, n), v + 4 * md);
            tensor_loaded(v);
#pragma unroll
            for (int i2 = 0; i2 < 32; i2 += 2) {
              const float2 a0 = f2_mul(as_float2(v[i2], v[i2 + 1]), alo);
              v[i2] = __float_as_uint(a0.x);
              v[i2 + 1] = __float_as_uint(a0.y);
            }
#pragma unroll
            for (int md = 0; md < 8; ++md) tensor_store<4>(columns_of(md, n), v + 4 * md);
            tc_wait_st();
          } else {
#pragma unroll
            for (int md = 0; md < 8; ++md) {
              const float2 a0 = f2_mul(make_float2(o[md][n][0], o[md][n][1]), alo);
              const float2 a1 = f2_mul(make_float2(o[md][n][2], o[md][n][3]), alo);
              o[md][n][0] = a0.x; o[md][n][1] = a0.y; o[md][n][2] = a1.x; o[md][n][3] = a1.y;
            }
          }
          scores(m[n], true);
          // (a reference past 2^27 may lie 16 below the largest; a score that is no number stays
          // one, as in a step that moves none)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2)
              x[hf][k2] = make_float2(min_or_nan(x[hf][k2].x, kMoveAt), min_or_nan(x[hf][k2].y, kMoveAt));
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
      if (i == 0) {                               // (the scales are here by now)
        if (const uint32_t huge = __ballot_sync(0xffffffffu, lane < nb && fabsf(vs) >= kHuge)) {
          first_huge = s0 + ((__ffs(huge) - 1) * kWarpsB + warp) * kBlockBk;
          if (first_huge < it.ctx || (huge >> lane & 1u)) vs = __fmul_rn(vs, kDown);
        }
      }
      float vsb = __shfl_sync(0xffffffffu, vs, i);
      if (edge && !(fabsf(vsb) < INFINITY)) vsb = 0.0f;    // (0 * inf would reach rows that see none of them)
      // ---- O += v_scale V^T P^T.  Row g of m-tile q is channel 16q + 2g, row g + 8 the next
      // one: a 16-bit element of the buffer is two channels of a key, so that the transposing
      // load pairs the keys 2c, 2c + 1 of both channels in a register.
      if (!ready(vbar, ph)) {
        give_up();
        flying = next >= 0 ? 6 : 2;
        break;
      }
      const float2 gain = make_float2(vsb, vsb);
      const uint32_t va = vbuf + (uint32_t)((lane & 15) * kD + (((lane >> 4) ^ (lane & 7)) << 4));
      constexpr int kUnrollV = S::kTensor ? 1 : 4;        // (fewer instructions to fetch: 1%)
#pragma unroll kUnrollV
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
          uint32_t ot[S::kTensor ? 4 * T : 1];    // (on their way beside the products)
          if constexpr (S::kTensor) {
            tensor_load<S::kLow>(low + (q + d) * S::kLow, ot);
            if constexpr (S::kHigh > 0) tensor_load<S::kHigh>(high + (q + d) * S::kHigh, ot + S::kLow);
          }
          float y[T][4];
#pragma unroll
          for (int n = 0; n < T; ++n) {
            mma_zero(y[n], a[0], pf[n][0][0]);
            mma_f16(y[n], a[1], pf[n][1][0]);
            if constexpr (kPrecise) {
              mma_f16(y[n], a[0], pf[n][0][kParts - 1]);
              mma_f16(y[n], a[1], pf[n][1][kParts - 1]);
            }
          }
          if constexpr (S::kTensor) tensor_loaded(ot);
#pragma unroll
          for (int n = 0; n < T; ++n)
#pragma unroll
            for (int v = 0; v < 4; v += 2) {
              if constexpr (S::kTensor) {
                uint32_t* to = ot + 4 * n + v;
                const float2 r = f2_fma(make_float2(y[n][v], y[n][v + 1]), gain, as_float2(to[0], to[1]));
                to[0] = __float_as_uint(r.x);
                to[1] = __float_as_uint(r.y);
              } else {
                float* to = o[q + d][n] + v;
                const float2 r = f2_fma(make_float2(y[n][v], y[n][v + 1]), gain, make_float2(to[0], to[1]));
                to[0] = r.x;
                to[1] = r.y;
              }
            }
          if constexpr (S::kTensor) {
            tensor_store<S::kLow>(low + (q + d) * S::kLow, ot);
            if constexpr (S::kHigh > 0) tensor_store<S::kHigh>(high + (q + d) * S::kHigh, ot + S::kLow);
          }
        }
      }
      if constexpr (S::kTensor) tc_wait_st();     // (the next step loads them)
      __syncwarp();
      if (next >= 0) load_block(vbuf, &maps.v, next, vbar, policy);
      ph ^= 1u;
    }

    // ---- the warps' sums come together, some tiles at a time
    const bool whole = block_windows(it.ctx + M - 1) == 1;
    float* part = p.partials + (((size_t)it.b * p.nwin_max + it.w) * p.c.Hkv + it.kh) * block_stride(R);
#pragma unroll
    for (int n = 0; n < T; ++n)
      if (g == 0) {
        if (first_huge != INT32_MAX)
          l[n] = make_float2(mark_down(l[n].x, goes_down(n, 0)), mark_down(l[n].y, goes_down(n, 1)));
        sm.ml[warp][n][2 * c] = make_float2(m[n].x, l[n].x);
        sm.ml[warp][n][2 * c + 1] = make_float2(m[n].y, l[n].y);
      }
    bool special = false;                         // a warp of the block has huge scales, or found no copy
#pragma unroll 1
    for (int n0 = 0; n0 < T; n0 += S::kJoin) {
      if constexpr (S::kTensor) {
        uint32_t v[32];
#pragma unroll
        for (int md = 0; md < 8; ++md) tensor_load<4>(columns_of(md, n0), v + 4 * md);
        tensor_loaded(v);
        if (n0 > 0) __syncthreads();              // (the tile before is read)
#pragma unroll
        for (int md = 0; md < 8; ++md) {
          const float2 x = as_float2(v[4 * md], v[4 * md + 1]), y = as_float2(v[4 * md + 2], v[4 * md + 3]);
          sm.o[warp][0][md][lane] = make_float4(x.x, x.y, y.x, y.y);
        }
      } else {
#pragma unroll
        for (int n = 0; n < T; ++n)
#pragma unroll
          for (int md = 0; md < 8; ++md)
            sm.o[warp][n][md][lane] = make_float4(o[md][n][0], o[md][n][1], o[md][n][2], o[md][n][3]);
      }
      if (n0 == 0) special = __syncthreads_or(flying != 0 || first_huge != INT32_MAX);
      else __syncthreads();
      if (special) {
        if (sm.failed) {                          // give the copies on their way a bounded chance, and leave
          if (lane == 0) {
            if (flying == 0 && ahead) flying = 3;
            if (flying & 1) mbar_wait_bounded(&sm.full[warp][0], ph);
            if (flying & 2) mbar_wait_bounded(&sm.full[warp][1], ph);
            if (flying & 4) mbar_wait_bounded(&sm.full[warp][0], ph ^ 1u);
          }
          __syncwarp();
          leave();
          return;
        }
        // a row that goes down in one warp goes down in all
#pragma unroll 1
        for (int t = 0; t < S::kJoin; ++t) {
          bool down[2] = {false, false}, own[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            for (int w = 0; w < kWarpsB; ++w) down[e] |= is_down(sm.ml[w][n0 + t][2 * c + e].y);
            own[e] = is_down(sm.ml[warp][n0 + t][2 * c + e].y);
          }
          const float fx = down[0] && !own[0] ? kDown : 1.0f, fy = down[1] && !own[1] ? kDown : 1.0f;
          for (int md = 0; md < 8; ++md) {
            float4& x = sm.o[warp][t][md][lane];
            x = make_float4(__fmul_rn(x.x, fx), __fmul_rn(x.y, fy), __fmul_rn(x.z, fx), __fmul_rn(x.w, fy));
          }
          __syncthreads();                        // (every sign is read)
          if (g == 0)
            for (int e = 0; e < 2; ++e) {
              float& sum = sm.ml[warp][n0 + t][2 * c + e].y;
              sum = mark_down(sum, down[e]);
            }
        }
        __syncthreads();
      }
#pragma unroll
      for (int t = 0; t < S::kJoin; ++t) {
        const int n = n0 + t;
        // weights 2^(m_w - m) of the warps, for rows 2c and 2c + 1
        float4 st[kWarpsB];                       // m, l of both rows
#pragma unroll
        for (int w = 0; w < kWarpsB; ++w) st[w] = *reinterpret_cast<const float4*>(&sm.ml[w][n][2 * c]);
        float mr[2], lr[2], wt[2][kWarpsB];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          auto ref = [&](int w) { return e ? st[w].z : st[w].x; };
          auto sum = [&](int w) { return e ? st[w].w : st[w].y; };
          mr[e] = fmaxf(fmaxf(ref(0), ref(1)), fmaxf(ref(2), ref(3)));
#pragma unroll
          for (int w = 0; w < kWarpsB; ++w)
            wt[e][w] = mr[e] == -INFINITY ? 0.0f : fast_exp2(__fsub_rn(ref(w), mr[e]));
          lr[e] = __fadd_rn(__fmaf_rn(wt[e][1], sum(1), __fmul_rn(wt[e][0], sum(0))),
                            __fmaf_rn(wt[e][3], sum(3), __fmul_rn(wt[e][2], sum(2))));
        }
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const int md = 2 * warp + d;
          float4 x[kWarpsB];
#pragma unroll
          for (int w = 0; w < kWarpsB; ++w) x[w] = sm.o[w][t][md][lane];
          auto join = [&](const float (&wt)[kWarpsB], float a0, float a1, float a2, float a3) {
            return __fadd_rn(__fmaf_rn(wt[1], a1, __fmul_rn(wt[0], a0)), __fmaf_rn(wt[3], a3, __fmul_rn(wt[2], a2)));
          };
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rr = it.rg * kUnitRows + 8 * n + 2 * c + e;
            if (rr >= R) continue;
            const float y0 = e ? join(wt[1], x[0].y, x[1].y, x[2].y, x[3].y) : join(wt[0], x[0].x, x[1].x, x[2].x, x[3].x);
            const float y1 = e ? join(wt[1], x[0].w, x[1].w, x[2].w, x[3].w) : join(wt[0], x[0].z, x[1].z, x[2].z, x[3].z);
            if (whole) {
              const int j = column(rr);
              const int64_t at = (((int64_t)it.b * M + j) * p.Hq + it.kh * p.g + rr - j * p.g) * kD + 16 * md + 2 * g;
              const float by = is_down(lr[e]) ? __fmul_rn(lr[e], -kDown) : lr[e];
              store_out2(p.out, p.q_type, at, __fdiv_rn(y0, by), __fdiv_rn(y1, by));
            } else {
              *reinterpret_cast<float2*>(part + (size_t)rr * kD + 16 * md + 2 * g) = make_float2(y0, y1);
              if (warp == 0 && d == 0 && g == 0)
                *reinterpret_cast<float2*>(part + (size_t)R * kD + 2 * rr) = make_float2(mr[e], lr[e]);
            }
          }
        }
      }
    }

    // ---- next item
    if (nx.b < 0) {
      leave();
      return;
    }
    if (nx.b != it.b || nx.kh != it.kh || nx.rg != it.rg) convert_queries(nx);
    it = nx;
    row = row_n;
    ks = ks_n;
    vs = vs_n;
    nb = nb_n;
    nx = next_of(it);
    nb_n = steps_of(nx);
    entry = entry_of(nx, nb_n);
    __syncthreads();                              // the sums are read, the queries in place
  }
}

// ------------------------------------------------------------------ merge
// Joins the windows of a row: W warps; the windows k, k + 16, ... are summed with the
// weights 2^(m_s - max m), for k = 0 .. 15, and the sixteen sums are added in order, so the
// order depends on neither W nor other rows.  A window in which a draft column's row sees
// no key has m = -inf and weight 0.  From the first 64 windows on of which one went down, all
// sums are on that side.  Bound by the trips to L2 that depend on one another (references,
// then 4 W windows a trip).
constexpr int kSums = 16, kBatchB = 4, kChunk = 64;

template <int W>
__global__ void __launch_bounds__(32 * W) block_merge_kernel(const BlockDecodeParams p) {
  constexpr int kOwn = kSums / W;
  static_assert(kBatchB % kOwn == 0 || kOwn % kBatchB == 0, "a batch holds whole rounds of the sums, or part of one");
  __shared__ float4 s_o[kSums][kD / 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
  const int ctx = __ldcg(p.ctx_len + b), R = p.R;
  const int kh = head / p.g, rr = j * p.g + head - kh * p.g;
  const size_t stride = (size_t)p.c.Hkv * block_stride(R);
  const float* base = p.partials + ((size_t)b * p.nwin_max * p.c.Hkv + kh) * block_stride(R);
  const float* mlcol = base + (size_t)R * kD + 2 * rr;
  const float* ocol = base + (size_t)rr * kD + 4 * lane;
  const bool valid = context_valid(p, ctx) && block_windows(ctx + p.M - 1) > 1;
  griddep_wait();                                 // every partial is in place
  if (!valid) return;
  const int ns = block_windows(ctx + j);

  float4 v[kBatchB];
  auto load = [&](int s0) {                       // the warp's windows s0 + warp + W n
#pragma unroll
    for (int n = 0; n < kBatchB; ++n) {
      const int s = s0 + W * n + warp;
      v[n] = s < ns ? __ldcg(reinterpret_cast<const float4*>(ocol + s * stride)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  };
  auto stats = [&](int s) {                       // m, l of window s
    return s < ns ? __ldcg(reinterpret_cast<const float2*>(mlcol + s * stride)) : make_float2(-INFINITY, 0.0f);
  };
  load(0);
  const float2 st0 = stats(lane), st1 = stats(lane + 32);
  float mx = fmaxf(st0.x, st1.x);
  for (int s = lane + kChunk; s < ns; s += 8 * 32) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = stats(s + 32 * i).x;
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, r[i]);
  }
  mx = warp_max(mx);

  float4 acc[kOwn];
#pragma unroll
  for (int k = 0; k < kOwn; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f, up = 1.0f;
  float2 a = st0, c = st1;
  for (int s0 = 0; s0 < ns; s0 += kChunk) {       // lane n weighs windows s0 + n and s0 + 32 + n
    float w0 = fast_exp2(__fsub_rn(a.x, mx)), w1 = fast_exp2(__fsub_rn(c.x, mx));   // (-inf: 0)
    l = __fmaf_rn(w1, fabsf(c.y), __fmaf_rn(w0, fabsf(a.y), l));
    if (up != 1.0f || __any_sync(0xffffffffu, is_down(a.y) || is_down(c.y))) {
      if (up == 1.0f) {
        up = kUp;
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
          acc[k] = make_float4(__fmul_rn(acc[k].x, kDown), __fmul_rn(acc[k].y, kDown), __fmul_rn(acc[k].z, kDown),
                               __fmul_rn(acc[k].w, kDown));
      }
      if (!is_down(a.y)) w0 = __fmul_rn(w0, kDown);
      if (!is_down(c.y)) w1 = __fmul_rn(w1, kDown);
    }
    a = stats(s0 + kChunk + lane);                // the next chunk's
    c = stats(s0 + kChunk + 32 + lane);
#pragma unroll
    for (int at = 0; at < kChunk; at += W * kBatchB) {
      if (s0 + at >= ns) break;
      float4 x[kBatchB];
#pragma unroll
      for (int n = 0; n < kBatchB; ++n) x[n] = v[n];
      load(s0 + at + W * kBatchB);                // the next batch, on its way meanwhile
#pragma unroll
      for (int n = 0; n < kBatchB; ++n) {
        const int k = at + W * n;                 // (+ warp: the window in the chunk)
        const float wn = __shfl_sync(0xffffffffu, k < 32 ? w0 : w1, (k & 31) + warp);
        float4& y = acc[(at / W + n) % kOwn];
        y = make_float4(__fmaf_rn(wn, x[n].x, y.x), __fmaf_rn(wn, x[n].y, y.y), __fmaf_rn(wn, x[n].z, y.z),
                        __fmaf_rn(wn, x[n].w, y.w));
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
  store_out2(p.out, p.q_type, at, __fmul_rn(__fdiv_rn(O.x, l), up), __fmul_rn(__fdiv_rn(O.y, l), up));
  store_out2(p.out, p.q_type, at + 2, __fmul_rn(__fdiv_rn(O.z, l), up), __fmul_rn(__fdiv_rn(O.w, l), up));
}

// Rows of at most kSums windows: a warp each, all its windows on their way at once.  The same
// sums: each of the sixteen has one window.
constexpr int kRowsOfMerge = 4;
__global__ void __launch_bounds__(32 * kRowsOfMerge) block_merge_short_kernel(const BlockDecodeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kRowsOfMerge + (threadIdx.x >> 5);
  const int b = (int)(row / (p.M * p.Hq)), at = (int)(row - (int64_t)b * p.M * p.Hq), j = at / p.Hq, head = at - j * p.Hq;
  if (b >= p.B) return;
  const int ctx = __ldcg(p.ctx_len + b), R = p.R;
  const int kh = head / p.g, rr = j * p.g + head - kh * p.g;
  const size_t stride = (size_t)p.c.Hkv * block_stride(R);
  const float* base = p.partials + ((size_t)b * p.nwin_max * p.c.Hkv + kh) * block_stride(R);
  const float* mlcol = base + (size_t)R * kD + 2 * rr;
  const float* ocol = base + (size_t)rr * kD + 4 * lane;
  const bool valid = context_valid(p, ctx) && block_windows(ctx + p.M - 1) > 1;
  griddep_wait();                                 // every partial is in place
  if (!valid) return;
  const int ns = block_windows(ctx + j);
  float4 v[kSums];
#pragma unroll
  for (int s = 0; s < kSums; ++s)
    v[s] = s < ns ? __ldcg(reinterpret_cast<const float4*>(ocol + s * stride)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float2 st = lane < ns ? __ldcg(reinterpret_cast<const float2*>(mlcol + lane * stride))
                              : make_float2(-INFINITY, 0.0f);
  float w = fast_exp2(__fsub_rn(st.x, warp_max(st.x)));
  const float l = warp_sum(__fmul_rn(w, fabsf(st.y)));
  const bool low_side = __any_sync(0xffffffffu, is_down(st.y));
  if (low_side && !is_down(st.y)) w = __fmul_rn(w, kDown);
  const float up = low_side ? kUp : 1.0f;
  float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int s = 0; s < kSums; ++s) {
    const float wn = __shfl_sync(0xffffffffu, w, s);
    const float4 x = make_float4(__fmul_rn(wn, v[s].x), __fmul_rn(wn, v[s].y), __fmul_rn(wn, v[s].z), __fmul_rn(wn, v[s].w));
    O = s == 0 ? x : make_float4(__fadd_rn(O.x, x.x), __fadd_rn(O.y, x.y), __fadd_rn(O.z, x.z), __fadd_rn(O.w, x.w));
  }
  const int64_t to = row * kD + 4 * lane;
  store_out2(p.out, p.q_type, to, __fmul_rn(__fdiv_rn(O.x, l), up), __fmul_rn(__fdiv_rn(O.y, l), up));
  store_out2(p.out, p.q_type, to + 2, __fmul_rn(__fdiv_rn(O.z, l), up), __fmul_rn(__fdiv_rn(O.w, l), up));
}

// ------------------------------------------------------------------- host
// Units of T tiles that a call has at most.
int64_t units_of(const BlockDecodeParams& p, int T) {
  return (int64_t)p.B * block_windows(p.max_ctx + p.M - 1) * p.c.Hkv * ((p.R + 8 * T - 1) / (8 * T));
}

// Tiles of 8 rows in a unit (1 to 5; float32 queries: to 4), the rows that read a head being
// dealt into groups of as many.  Large units convert the codes for more rows at once; small
// ones are more, for the multiprocessors to share.  The choice is the least of an estimate,
// units a multiprocessor (in thirds, three at a time) times the cost of a unit, 7, 11, 15, 20
// and 24 us with three of them there (two thirds of that alone), from this table (us a call,
// bf16 queries, int8 codes, 32 query and 4 kv heads; in brackets what the rule takes):
//   sequences x keys, columns    at most 1      2       3       4       5 tiles
//    1 x 100, 8                    [5.2]      6.9     8.9    10.1
//    1 x 512, 5                    [8.8]     10.9    13.6             18.0
//    1 x 4096, 5                  [10.6]     12.0    14.9             19.1
//    4 x 1k..4k, 5                 14.5     [16.6]   19.1             20.2
//   16 x 1k..4k, 3                 25.9      27.2   [25.0]
//   16 x 1k..4k, 5                 33.9      35.7    37.7            [33.7]
//   16 x 1k..4k, 8                 46.9     [38.0]   48.9    44.4
//   64 x 1k..4k, 2                 51.6     [40.4]
//   64 x 1k..4k, 3                 72.9      71.8   [53.3]
//   64 x 1k..4k, 5                115       103      94              [77]
//   64 x 1k..4k, 8                177       137     136    [118]
//   16 x 16k..32k, 5              280       215     190             [154]
//    1 x 64k, 8                    73       [66]     68      64
//   90 x 100..500, 8               47        41      46     [40]
// (All 64 rows as one unit of 8 tiles, two blocks a multiprocessor: 143 us for 64 x 1k..4k, 8,
// when 4 tiles took 130.)
// The costs are those of bf16 queries and int8 codes.  e4m3 takes as long (16 x 1k..4k, 5:
// 34.3 us); with float32 queries, whose MMAs are twice as many, they were not taken one by one
// (16 x 1k..4k, 5: 47.5; 64 of them 125).  The scales that kHuge looks for came later: up to
// 2% more than here.
// Units are counted from max_ctx, as the host does not know the lengths.  With a limit of
// 131072, in brackets with the batch's own: 1 x 4096 keys, 5 columns 26.6 us [11.1]; 16 x
// 1k..4k, 5 61 [34]; 64 x 1k..4k, 1, 2 and 5 columns 55 [33], 85 [41] and 190 [78].
int unit_tiles(const BlockDecodeParams& p) {
  const int tiles = (p.R + 7) / 8, most = std::min(tiles, p.q_type == KATTN_F32 ? 4 : 5);
  static const int cost[5] = {7, 11, 15, 20, 24};
  int best = 1;
  double least = 0.0;
  for (int t = 1; t <= most; ++t) {
    const int groups = (tiles + t - 1) / t;
    if (t > 1 && (tiles + groups - 1) / groups < t) continue;      // smaller units make as many groups
    const double a_sm = (double)units_of(p, t) / p.sms, full = std::floor(a_sm / 3.0), rest = a_sm - 3.0 * full;
    const double time = cost[t - 1] * (full + (rest > 0.0 ? 0.5 + rest / 6.0 : 0.0));
    if (t == 1 || time < least) {
      best = t;
      least = time;
    }
  }
  return best;
}

template <int T, bool kE4m3, bool kPrecise>
cudaError_t raise_limit() {
  return cudaFuncSetAttribute(block_split_kernel<T, kE4m3, kPrecise>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sizeof(BlockSmem<T, kPrecise>) + 1024);
}
// Every kernel loaded and allowed its shared memory, with the first call on a device: a later
// call of other sizes may be captured.
cudaError_t prepare_device() {
  const cudaError_t e[] = {
      raise_limit<1, false, false>(), raise_limit<2, false, false>(), raise_limit<3, false, false>(),
      raise_limit<4, false, false>(), raise_limit<5, false, false>(), raise_limit<1, false, true>(),
      raise_limit<2, false, true>(),  raise_limit<3, false, true>(),  raise_limit<4, false, true>(),
      raise_limit<1, true, false>(),  raise_limit<2, true, false>(),  raise_limit<3, true, false>(),
      raise_limit<4, true, false>(),  raise_limit<5, true, false>(),  raise_limit<1, true, true>(),
      raise_limit<2, true, true>(),   raise_limit<3, true, true>(),   raise_limit<4, true, true>()};
  for (const cudaError_t x : e)
    if (x != cudaSuccess) return x;
  cudaFuncAttributes a;
  cudaError_t x = cudaFuncGetAttributes(&a, block_merge_kernel<2>);
  if (x == cudaSuccess) x = cudaFuncGetAttributes(&a, block_merge_kernel<4>);
  if (x == cudaSuccess) x = cudaFuncGetAttributes(&a, block_merge_short_kernel);
  if (x == cudaSuccess) x = cudaFuncGetAttributes(&a, block_merge_kernel<16>);
  return x;
}

template <int T, bool kE4m3, bool kPrecise>
cudaError_t launch_split(const BlockDecodeParams& p, const TmaMaps& maps, cudaStream_t stream) {
  const auto kern = block_split_kernel<T, kE4m3, kPrecise>;
  const int smem = (int)sizeof(BlockSmem<T, kPrecise>) + 1024;     // + alignment slack
  static_assert((sizeof(BlockSmem<T, kPrecise>) + 2048) * kPerSm <= 228 * 1024,
                "with the slack and the reserve of a block");
  const int64_t units = units_of(p, T), slots = (int64_t)p.sms * kPerSm;
  return launch_pdl(kern, dim3((unsigned)std::min(units, slots)), dim3(kThreadsB), (size_t)smem, stream, p, maps);
}
template <bool kE4m3>
cudaError_t launch_split(const BlockDecodeParams& p, const TmaMaps& maps, cudaStream_t stream) {
  const int tiles = unit_tiles(p);
  if (p.q_type == KATTN_F32) {
    switch (tiles) {
      case 1: return launch_split<1, kE4m3, true>(p, maps, stream);
      case 2: return launch_split<2, kE4m3, true>(p, maps, stream);
      case 3: return launch_split<3, kE4m3, true>(p, maps, stream);
      default: return launch_split<4, kE4m3, true>(p, maps, stream);
    }
  }
  switch (tiles) {
    case 1: return launch_split<1, kE4m3, false>(p, maps, stream);
    case 2: return launch_split<2, kE4m3, false>(p, maps, stream);
    case 3: return launch_split<3, kE4m3, false>(p, maps, stream);
    case 4: return launch_split<4, kE4m3, false>(p, maps, stream);
    default: return launch_split<5, kE4m3, false>(p, maps, stream);
  }
}

template <int W>
cudaError_t launch_merge(const BlockDecodeParams& p, cudaStream_t stream) {
  return launch_pdl(block_merge_kernel<W>, dim3((unsigned)p.Hq, (unsigned)p.M, (unsigned)p.B), dim3(32 * W), 0, stream, p);
}

}  // namespace

int64_t block_decode_units(const BlockDecodeParams& p) { return units_of(p, 1); }

size_t block_decode_workspace_bytes(int B, int M, int Hq, int max_ctx) {
  // Hkv * block_stride(R) <= Hq * (M * (d + 2) + 3) whatever Hkv is
  return 256 + (size_t)B * block_windows(max_ctx + M - 1) * Hq * (M * (kD + 2) + 3) * sizeof(float);
}

void set_block_decode_workspace(BlockDecodeParams& p, void* workspace) {
  p.err_word = static_cast<uint32_t*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  p.nwin_max = block_windows(p.max_ctx + p.M - 1);
}

cudaError_t launch_decode_blocks(const BlockDecodeParams& params, int code_type, cudaStream_t stream) {
  BlockDecodeParams p = params;
  static std::atomic<int> sms_cache[kMaxDevices];
  int dev = 0;
  cudaError_t dev_error = cudaGetDevice(&dev);
  if (dev_error != cudaSuccess) return dev_error;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  p.sms = cached ? sms_cache[dev].load() : 0;
  if (p.sms <= 0) {
    dev_error = cudaDeviceGetAttribute(&p.sms, cudaDevAttrMultiProcessorCount, dev);
    if (dev_error == cudaSuccess) dev_error = prepare_device();
    if (dev_error != cudaSuccess) return dev_error;
    if (cached) sms_cache[dev].store(p.sms);
  }
  TmaMaps maps;
  const int64_t rows = (int64_t)p.c.Hkv * p.c.cap_rows;
  if (!encode_plane_map(&maps.k, p.c.k, rows) || !encode_plane_map(&maps.v, p.c.v, rows))
    return cudaErrorInvalidValue;
  const cudaError_t e = code_type == KATTN_E4M3 ? launch_split<true>(p, maps, stream)
                                                : launch_split<false>(p, maps, stream);
  if (e != cudaSuccess || p.nwin_max <= 1) return e;
  // Warps a row, by the windows that it may have: 64 sequences of 1k to 4k keys, 5 columns 77
  // us a call with one (the short form), 86 with 2; 16 sequences 34 and 36; 2 of 120k to 131k
  // keys, 8 rows on each of 4 heads, 56 us with 16 and 63 with 4; 64 of 512 to 32768 keys 96
  // us with 2, 4 or 8.
  if (p.nwin_max <= kSums) {
    const int64_t rows = (int64_t)p.B * p.M * p.Hq;
    return launch_pdl(block_merge_short_kernel, dim3((unsigned)((rows + kRowsOfMerge - 1) / kRowsOfMerge)),
                      dim3(32 * kRowsOfMerge), 0, stream, p);
  }
  if (p.nwin_max <= 32) return launch_merge<2>(p, stream);
  if (p.nwin_max <= 128) return launch_merge<4>(p, stream);
  return launch_merge<16>(p, stream);
}

}  // namespace kattn
