// Differential decode attention over the int8 cache:
//   out = softmax(s_0) V - lam softmax(s_1) V
// for a pair of query heads (2i, 2i + 1), the key planes 2p and 2p + 1 and the
// 256 value channels of both planes.
//
// Two launches: diff_split_kernel, or diff_tc_kernel for many rows per map and
// enough windows, reduces windows of the keys; diff_merge_kernel joins the windows
// of a row and takes the difference.  A sequence of one window is finished by the
// first.
//
// What bounds it: 528 bytes per key and plane pair must come from HBM, for
// 2 * 128 products per query row and map on the key side and 2 * 256 on the value
// side, so with up to 8 rows per map the stream of the cache is the floor, and the
// split reads each byte once for both maps.  Measured, 64 sequences of 512 to
// 32768 keys over 64-row pages, 32 query and 4 kv heads (554 MB, 82 us at the
// measured copy rate): 8 rows per map, split 105 us (5.3 TB/s), the call 122 us; 4
// rows per map, the call 104 us.  The split at 8 rows is bound by the chain of a
// block's steps at 12 warps a multiprocessor, no single pipe: tensor 50% busy,
// issue 37%; with the cache in L2, or without the int8 products, it takes 7% less.
// With more rows each group of 8 rows streams the window again, from L2: bound by
// the steps alone (2 draft columns, 16 rows per map, 64 sequences of 1k to 4k keys:
// the call 82 us).  A single short sequence is bound by latency: about 9 us, and 1.6
// us for each of a window's 4 or 8 blocks.
#include "decode_diff_tc.cuh"

namespace kattn {
namespace {

// ------------------------------------------------------------------ split
// Two warps work on a unit (sequence, window, plane pair, row group).  Warp a
// owns map a and plane a: it streams the rows of key plane 2p + a and value
// plane 2p + a through its own ring, scores its key plane and takes the softmax
// weights of map a; the two exchange their weights through shared memory, once
// per block; then each sums its 128 value channels for both maps, so every
// value is converted to f16 once.  The pairs do not wait for one another.
// Measured alternatives on the serving case: one warp for both planes (255
// registers, 8 warps a multiprocessor) took 193 us a call; windows of 128 keys 151
// us (twice the partials and item starts), of 512 keys the same as 256, with fewer
// units to spread.
constexpr int kPairs = 2;                         // pairs of warps in a block
constexpr int kThreads = kPairs * 64;

// What the warps of a pair hand over per block: the weights of both maps, as the
// second product's operand takes them (two keys of a row side by side), and the
// factors of the rows where a reference moved (kMoved).
template <int T>
struct Exchange {
  float w[T][kBlockBk / 2][8][2];
  float alpha[2][8];                              // of each map's rows
  int info[2];                                    // per warp: kFailed | kMoved
};
constexpr int kFailed = 1, kMoved = 2;

// What a warp needs once per block or item is kept here, not in registers (the
// accumulators take a good part of the 168 that three blocks leave a thread).
struct __align__(16) WarpState {
  float vs[kBlockBk];                             // v_scale of the block
  float qs[8];
  float up[8];                                    // 2^E of the operand's rows (1: it follows the products)
  float mag[2][8], post[2][8], factor[2][8];      // then, per tile: largest product (-1: no such row), 2^E, rescaling
  float row_sum[8];                               // of a sequence that ends in its window
  uint8_t q[8 * kQStride];
  int rows[2][kWinBlocks + 2];                    // rows of the blocks, by item slot
  DiffItem item[2];                               // the current and the next
};

template <int T>
struct __align__(1024) DiffSmem {
  static constexpr int kExBytes = (int)sizeof(Exchange<T>);
  uint8_t ring[kPairs][2][2][kBlockBytes];        // [K|V] of each warp
  WarpState ws[kPairs][2];
  alignas(16) Exchange<T> ex[kPairs][2];          // by block parity
  uint64_t full[kPairs][2][2];
  int prefix[kMaxGroups + 1];
  int warp_total[kThreads / 32];
};

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p));
}

// kBlockBk rows of a plane into a stage, 128-byte swizzle, by one lane of the warp
// (predicated, so that the warp does not branch).  The stage was read by every lane
// before: their loads have returned, as products that took them were issued.
__device__ __forceinline__ void load_stage(uint32_t dst, const CUtensorMap* map, int row,
                                           uint32_t bar, uint64_t policy) {
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n"
      " @p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%4], %6;\n"
      " @p cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;\n}\n" ::"r"(dst), "l"(map), "r"(0), "r"(row), "r"(bar),
      "l"(policy), "r"((uint32_t)kBlockBytes)
      : "memory");
}

// T: tiles of 8 query rows on the value side.  T = 2: 8 rows of each map, a tile
// per map.  T = 1: 4 rows of each map in one tile, map 0 in rows 0..3.
// (Blocks a multiprocessor holds: T = 2 has 64 accumulators a thread; at 4 blocks,
// 128 registers, the serving call takes 128 us instead of 125.  T = 1 gains: 106
// us instead of 108.)
template <int T>
__global__ void __launch_bounds__(kThreads, T == 1 ? 4 : 3)
diff_split_kernel(const DiffParams p, const __grid_constant__ TmaMaps maps) {
  using Smem = DiffSmem<T>;
  constexpr int kUnitRows = T == 1 ? 4 : 8;       // rows of each map in a unit
  extern __shared__ unsigned char smem_raw[];
  // (offset, not masked: the compiler goes on knowing that this is shared memory)
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + (0u - smem_u32(smem_raw)) % 1024u);
  // (broadcast, so that what follows from the warp's number is known to be uniform)
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int wp = warp >> 1, a = warp & 1;         // the pair of warps; the warp's map and plane
  const int g = lane >> 2, c = lane & 3;
  const int M = p.M, R = p.R, H = p.Hq / 2;
  const int nrg = (R + kUnitRows - 1) / kUnitRows;
  if (lane == 0) {
    mbar_init(&sm.full[wp][a][0], 1);
    mbar_init(&sm.full[wp][a][1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }

  const DiffUnits units(p, sm.prefix, nrg, 1);
  units.count(sm.prefix, sm.warp_total);
  mark_bad_sequences(p);
  __syncthreads();
  griddep_launch_dependents();
  const int total = sm.prefix[kMaxGroups];
  // Each pair of warps takes a run of units that follow one another.
  // Blocks s, s + sms, ... start on the same multiprocessor: their pairs are
  // numbered one after the other, so that the runs, whose lengths differ by one
  // unit, add up to the same work on each.  (A numbering by block alone can give one
  // multiprocessor all the longer runs; with 4 heads per pair 111 us, 109 us so.)
  const int G = gridDim.x * kPairs;
  const int per_sm = gridDim.x / p.sms, more = gridDim.x - per_sm * p.sms, on = blockIdx.x % p.sms;
  const int worker = (on * per_sm + min(on, more) + blockIdx.x / p.sms) * kPairs + wp;
  int u = (int)((int64_t)worker * total / G);
  const int u_end = (int)((int64_t)(worker + 1) * total / G);
  DiffItem unit;
  if (!units.find(&u, u_end, &unit)) return;

  // rr / g and the query head of unit row rr (rr < 64, g <= 64: exact)
  const uint32_t ginv = 65536u / (uint32_t)p.g + 1u;
  auto column = [&](int rr) -> int { return (int)(((uint32_t)rr * ginv) >> 16); };

  WarpState& ws = sm.ws[wp][a];
  int ipar = 0;                                   // slot of the current item
  auto put = [&](int slot, const DiffItem& it) {
    __syncwarp();
    if (lane == 0) ws.item[slot] = it;
    __syncwarp();
  };
  auto put_next = [&](int slot) {                 // the unit after the other slot's
    DiffItem it = ws.item[slot ^ 1];
    if (u + 1 < u_end) it = units.after(it);
    else it.b = -1;
    put(slot, it);
  };
  // The rows of an item's blocks (in the 2-D view of all planes, which is also the
  // index of their scales), and after the last its successor's first, or -1.
  auto put_rows = [&](int slot, int entry) {
    const DiffItem& it = ws.item[slot];
    const int row = row_of_entry(p, it, entry, lane) + (2 * it.pair + a) * p.cap_rows;
    const bool in = it.b >= 0 && lane < units.blocks(it);
    __syncwarp();
    if (lane < kWinBlocks) ws.rows[slot][lane] = in ? row : -1;
    if (in) {                                     // its scales, read at its start
      prefetch_l2(p.k_scale + row);
      prefetch_l2(p.v_scale + row);
    }
    __syncwarp();
  };
  put(0, unit);
  put_next(1);
  put_rows(0, row_entry(p, ws.item[0], lane));
  int entry = row_entry(p, ws.item[1], lane);     // the next item's, not looked at yet

  // ---- copies: the K rows of a block into one buffer, its V rows into another; a
  // buffer is refilled with the next block's as soon as its products are issued.
  const uint32_t lws = smem_u32(&ws), kbuf = smem_u32(sm.ring[wp][a][0]), vbuf = kbuf + kBlockBytes;
  const uint32_t kbar = smem_u32(sm.full[wp][a]), vbar = kbar + 8;
  const uint64_t policy = nrg > 1 ? l2_evict_normal() : l2_evict_first();
  load_stage(kbuf, &maps.k, ws.rows[0][0], kbar, policy);
  load_stage(vbuf, &maps.v, ws.rows[0][0], vbar, policy);
  uint32_t ph = 0;                                // parity of the block's copies
  bool k_ahead = false;                           // the next block's K copy is under way
  // ---- shared-memory addresses of this lane
  const uint32_t exbase = smem_u32(&sm.ex[wp][0]);
  uint32_t lex = exbase;                          // exchange buffer of the next block
  constexpr int kExAlpha = T * 1024, kExInfo = kExAlpha + 64;
  constexpr int kVs = offsetof(WarpState, vs), kQs = offsetof(WarpState, qs);
  constexpr int kUp = offsetof(WarpState, up), kQ = offsetof(WarpState, q);
  const uint32_t lww = (T == 1 ? 0 : 1024 * a) + ((g >> 1) * 8 + (T == 1 ? 4 * a : 0) + 2 * c) * 8 + (g & 1) * 4;
  const uint32_t lwr = (c * 8 + g) * 8;

#ifdef KATTN_DIFF_STAGE_LIMIT
  // Test builds only: a warp of the maps KATTN_DIFF_STAGE_MAPS (a bit each) takes this
  // many copies, then finds none ready.
  int taken = 0;
  auto ready = [&](uint32_t bar) {
    return !((KATTN_DIFF_STAGE_MAPS >> a & 1) && taken++ >= KATTN_DIFF_STAGE_LIMIT) && stage_ready(bar, ph);
  };
#else
  auto ready = [&](uint32_t bar) { return stage_ready(bar, ph); };
#endif
  // Before a warp leaves early: a bounded chance for its copies in flight to land
  // (the block's V copy, and its K copy or the next block's).
  auto drain = [&](bool k_taken) {
    if (lane != 0) return;
    mbar_wait_bounded(&sm.full[wp][a][1], ph);
    if (!k_taken) mbar_wait_bounded(&sm.full[wp][a][0], ph);
    else if (k_ahead) mbar_wait_bounded(&sm.full[wp][a][0], ph ^ 1u);
  };
  // A copy of this warp never arrived: tell the other warp at its next exchange
  // (the buffer that it reads then), flag it, and leave.
  auto give_up = [&](bool k_taken) {
    if (lane == 0) {
      sts32(lex + kExInfo + 4 * a, (uint32_t)kFailed);
      atomicOr(p.err_word, KATTN_DEVERR_TIMEOUT);
    }
    named_sync(1 + wp, 64);
    drain(k_taken);
  };

  for (;;) {
    const DiffItem& it0 = ws.item[ipar];
    const int nb = units.blocks(it0);
    const int s0 = window_start(it0.w);           // the unit's keys: [s0, s1)
    const int s1 = min(s0 + window_keys(it0.w), it0.ctx + M - 1);
    // ---- the unit's queries of map a, quantized per row
    if (it0.fresh) {
      float4 x[kUnitRows];
#pragma unroll
      for (int r = 0; r < kUnitRows; ++r) {
        const int rr = min(it0.rg * kUnitRows + r, R - 1);
        const int j = column(rr), head = 2 * (it0.pair * p.g + rr - j * p.g) + a;
        x[r] = __ldg(reinterpret_cast<const float4*>(
                         p.q + (((int64_t)it0.b * M + j) * p.Hq + head) * kD) + lane);
      }
#pragma unroll
      for (int r = 0; r < kUnitRows; ++r) {
        float s;
        const uint32_t w = quantize_loaded_row(x[r], &s);
        const bool in = it0.rg * kUnitRows + r < R;
        *reinterpret_cast<uint32_t*>(&ws.q[r * kQStride + 4 * lane]) = in ? w : 0u;
        if (lane == 0) ws.qs[r] = in ? s : 0.0f;
      }
    }
    // Keys that unit row r of the tile sees (T = 1: rows 4..7 are those of map 1).
    auto keys_of = [&](int r) -> int {
      return it0.ctx + column(min(it0.rg * kUnitRows + (T == 1 ? r & 3 : r), R - 1));
    };
    // ---- the plane's scales: those of block 0, and the largest v_scale among the
    // keys that every row sees
    float nk, nv;                                 // scales of the next block's key `lane`
    bool care;                                    // see ScaleRange
    {
      const int own = min(it0.ctx, s1), d0 = max(it0.ctx, s0), drafts = s1 - d0;
      float most = 0.0f, least = INFINITY;
#pragma unroll
      for (int e = 0; e < kWinBlocks; ++e) {
        const int key = s0 + 32 * e + lane, at = ws.rows[ipar][e] + lane;
        const float v = key < s1 ? __ldg(p.v_scale + at) : 0.0f;
        if (key < own) {
          most = fmaxf(most, v);
          least = fminf(least, v);
        }
        if (e == 0) {
          nv = v;
          nk = key < s1 ? __ldg(p.k_scale + at) : 0.0f;
        }
      }
      float draft = 0.0f;
      if (lane < drafts) draft = __ldg(p.v_scale + ws.rows[ipar][(d0 + lane - s0) >> 5] + ((d0 + lane - s0) & 31));
      const int r = lane & 7, keys = keys_of(r);  // lane r < 8: row r
      ScaleRange range = warp_range(most, least);
      for (int i = 0; i < drafts; ++i) range.add(__shfl_sync(0xffffffffu, draft, i), d0 + i < keys);
      if (lane < 8) ws.up[r] = range.scale();
      care = __any_sync(0xffffffffu, range.care());
      if (care && lane < 8) {
#pragma unroll
        for (int n = 0; n < T; ++n) ws.mag[n][r] = range.spread() ? 0.0f : -1.0f;
      }
    }
    __syncwarp();

    // Of rows 2c + e: the reference (m), the score above which it moves,
    // and the sum of this thread's weights.
    float2 m_run = make_float2(0.0f, 0.0f), m_move = make_float2(-INFINITY, -INFINITY);
    float2 l_run = make_float2(0.0f, 0.0f);
    float o[8][T][4];                             // [m-tile of 16 channels][tile]
#pragma unroll
    for (int md = 0; md < 8; ++md)
#pragma unroll
      for (int n = 0; n < T; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v) o[md][n][v] = 0.0f;

    // The blocks of the unit; false: a copy never arrived, and the warp leaves.
    auto blocks = [&](auto careful) __attribute__((always_inline)) -> bool {
      constexpr bool kCare = decltype(careful)::value;
      for (int i = 0; i < nb; ++i) {
        if (i + 1 == nb) {                          // the next item's rows, its first after this one's last
          put_rows(ipar ^ 1, entry);
          if (lane == 0) ws.rows[ipar][nb] = ws.rows[ipar ^ 1][0];
          __syncwarp();
        }
        const int t0 = s0 + i * kBlockBk;
        const int next = ws.rows[ipar][i + 1];      // row of the block after this one, or -1
        float ks4[4];                               // k_scale of keys g + 8q
#pragma unroll
        for (int q = 0; q < 4; ++q) ks4[q] = __shfl_sync(0xffffffffu, nk, g + 8 * q);
        sts32<kVs>(lws + 4 * lane, nv);
        {
          const bool in = t0 + kBlockBk + lane < s1;
          nk = in ? __ldg(p.k_scale + next + lane) : 0.0f;
          nv = in ? __ldg(p.v_scale + next + lane) : 0.0f;
        }
        // ---- Q.K: keys 16 half + g (+ 8), rows 2c + e
        int acc[2][4];
        {
          uint4 qlo = make_uint4(0, 0, 0, 0), qhi = qlo;
          if (T == 2 || g < 4) {
            const uint32_t lq = lws + g * kQStride + 32 * c;
            qlo = lds128a<kQ>(lq);
            qhi = lds128a<kQ + 16>(lq);
          }
          if (!ready(kbar)) {
            give_up(false);
            return false;
          }
          key_products(kbuf + (uint32_t)swz(g, 2 * c), qlo, qhi, acc);
          __syncwarp();
          k_ahead = next >= 0;
          if (next >= 0) load_stage(kbuf, &maps.k, next, kbar, policy);
        }
        // ---- scores s = (S * (qs * ks)) * sm_scale, rounded as written
        float2 sc[2][2];                            // [half][key g | g + 8], rows 2c, 2c + 1
        {
          float2 qsr = make_float2(0.0f, 0.0f);
          if (T == 2 || c < 2) qsr = lds64a<kQs>(lws + 8 * c);
          scores_of(acc, ks4, qsr, p.sm_scale, sc);
        }
        if (t0 + kBlockBk > it0.ctx)                // keys that some row does not see
          hide_keys(sc, t0 + g, keys_of(2 * c), keys_of(2 * c + 1));
        float2 alpha = make_float2(1.0f, 1.0f);
        int info = 0;
        if (block_weights(sc, m_run, m_move, l_run, alpha)) {
          info = kMoved;
          if (g == 0) sts64(lex + kExAlpha + 32 * a + 8 * c, alpha);
        }
        // ---- hand the weights over
        if (T == 2 || c < 2) {
          const uint32_t w = lex + lww;
          sts32<0>(w, sc[0][0].x);
          sts32<8>(w, sc[0][0].y);
          sts32<256>(w, sc[0][1].x);
          sts32<264>(w, sc[0][1].y);
          sts32<512>(w, sc[1][0].x);
          sts32<520>(w, sc[1][0].y);
          sts32<768>(w, sc[1][1].x);
          sts32<776>(w, sc[1][1].y);
        }
        if (lane == 0) sts32(lex + kExInfo + 4 * a, (uint32_t)info);
        named_sync(1 + wp, 64);
        const float2 both = lds64a<kExInfo>(lex);
        const int info0 = __float_as_int(both.x), info1 = __float_as_int(both.y);
        const uint32_t lexr = lex + lwr, exa = lex + kExAlpha;
        lex = exbase + exbase + Smem::kExBytes - lex;      // the other buffer
        if (kCare || (info0 | info1)) {
          if ((info0 | info1) & kFailed) {        // the other warp has left
            drain(true);
            return false;
          }
          if constexpr (kCare) {                  // row g of each tile: its largest product, and E
#pragma unroll
            for (int n = 0; n < T; ++n) {
              const uint32_t w = lexr + 1024 * n, v = lws + 8 * c;
              float m = 0.0f;
              auto take = [&](float2 w2, float2 v2) {
                float2 y = f2_mul(w2, v2);
                hide_products(y, w2);
                m = fmaxf(m, fmaxf(y.x, y.y));
              };
              take(lds64a<0>(w), lds64a<kVs>(v));
              take(lds64a<256>(w), lds64a<kVs + 32>(v));
              take(lds64a<512>(w), lds64a<kVs + 64>(v));
              take(lds64a<768>(w), lds64a<kVs + 96>(v));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
              if (c == 0) {
                const int map = T == 1 ? g >> 2 : n, r = T == 1 ? g & 3 : g;
                const float al = (map ? info1 : info0) & kMoved ? lds32a<0>(exa + 32 * map + 4 * r) : 1.0f;
                float mag = ws.mag[n][g];
                ws.factor[n][g] = mag < 0.0f ? al : follow_products(m, al, mag);
                ws.post[n][g] = mag < 0.0f ? 1.0f : product_scale(mag);
                ws.mag[n][g] = mag;
              }
            }
            __syncwarp();
          }
#pragma unroll
          for (int n = 0; n < T; ++n) {
            // the tile's rows 2c, 2c + 1: map n, or (T = 1) map c / 2
            const int map = T == 1 ? c >> 1 : n, r0 = T == 1 ? 2 * (c & 1) : 2 * c;
            float2 al;
            if constexpr (kCare) {
              al = *reinterpret_cast<const float2*>(&ws.factor[n][2 * c]);
            } else {
              al = lds64a<0>(exa + 32 * map + 4 * r0);
              if (!((map ? info1 : info0) & kMoved)) al = make_float2(1.0f, 1.0f);
            }
#pragma unroll
            for (int md = 0; md < 8; ++md) {
              const float2 lo = f2_mul(make_float2(o[md][n][0], o[md][n][1]), al);
              const float2 hi = f2_mul(make_float2(o[md][n][2], o[md][n][3]), al);
              o[md][n][0] = lo.x; o[md][n][1] = lo.y; o[md][n][2] = hi.x; o[md][n][3] = hi.y;
            }
          }
        }
        // ---- P.V: the operand w * v_scale * 2^E as f16 hi + lo (22 bits), V exact
        const float up = lds32a<kUp>(lws + 4 * g);
        const float2 up2 = make_float2(up, up);
        if (!ready(vbar)) {
          give_up(true);
          return false;
        }
        // A = V^T.  Row g of m-tile q is channel 16q + 2g, row g + 8 the next one; a
        // 16-bit element of the buffer is two channels of a key, so the transposing
        // load pairs the keys 2c, 2c + 1 of both channels in a register.  Lane 8i + r
        // addresses key r (+ 8 if i is odd) of the half, 16-byte chunk q + i / 2.
        const uint32_t va = vbuf + (uint32_t)((lane & 15) * kD + (((lane >> 4) ^ (lane & 7)) << 4));
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float2 v0 = f2_mul(hf ? lds64a<kVs + 64>(lws + 8 * c) : lds64a<kVs>(lws + 8 * c), up2);
          const float2 v1 = f2_mul(hf ? lds64a<kVs + 96>(lws + 8 * c) : lds64a<kVs + 32>(lws + 8 * c), up2);
          uint2 bhi[T], blo[T];
#pragma unroll
          for (int n = 0; n < T; ++n) {
            const uint32_t w = lexr + 1024 * n;
            const float2 w0 = hf ? lds64a<512>(w) : lds64a<0>(w), w1 = hf ? lds64a<768>(w) : lds64a<256>(w);
            float2 y0 = f2_mul(w0, v0), y1 = f2_mul(w1, v1);
            if constexpr (kCare) {
              hide_products(y0, w0);
              hide_products(y1, w1);
              const float post = ws.post[n][g];
              y0 = f2_mul(y0, make_float2(post, post));
              y1 = f2_mul(y1, make_float2(post, post));
            }
            split_f16x2(y0.x, y0.y, bhi[n].x, blo[n].x);
            split_f16x2(y1.x, y1.y, bhi[n].y, blo[n].y);
          }
#pragma unroll
          for (int q = 0; q < 8; q += 2) {
            uint32_t vw[4];                         // keys 2c.. and 2c+8.. of tile q, then of tile q + 1
            if (hf) ldsm_x4_trans<2048>(vw, va ^ (uint32_t)(q << 4));
            else ldsm_x4_trans<0>(vw, va ^ (uint32_t)(q << 4));
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              uint32_t af[4];
              value_operand(vw[2 * d], vw[2 * d + 1], af);
#pragma unroll
              for (int n = 0; n < T; ++n) mma_f16(o[q + d][n], af, bhi[n]);
#pragma unroll
              for (int n = 0; n < T; ++n) mma_f16(o[q + d][n], af, blo[n]);
            }
          }
        }
        __syncwarp();
        if (next >= 0) load_stage(vbuf, &maps.v, next, vbar, policy);
        ph ^= 1u;
      }
      return true;
    };
    if (!(!care ? blocks(std::false_type{}) : blocks(std::true_type{}))) return;
    const bool whole = diff_windows(it0.ctx + M - 1) == 1;
    const int b = it0.b, pair = it0.pair;

    // ---- the window's result
    float down[T][2];                             // 2^-E of rows 2c + e
#pragma unroll
    for (int n = 0; n < T; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float up = ws.up[2 * c + e];
        if (care) up = __fmul_rn(up, ws.post[n][2 * c + e]);
        down[n][e] = inverse_scale(up);
      }
    l_run = make_float2(row_total(l_run.x), row_total(l_run.y));
    if (whole) {                                  // the other map's row sums
      if (lane == 0) sts32(lex + kExInfo + 4 * a, 0u);
      if (g == 0) {
        ws.row_sum[2 * c] = l_run.x;
        ws.row_sum[2 * c + 1] = l_run.y;
      }
      named_sync(1 + wp, 64);
      const float2 both = lds64a<kExInfo>(lex);
      lex = exbase + exbase + Smem::kExBytes - lex;      // (a warp that runs ahead writes the other)
      if (__float_as_int(both.x) | __float_as_int(both.y)) {
        // the other warp gave up at the last block's V copy: both K and V of the next
        // block are under way here, if there is one
        if (lane == 0 && k_ahead) {
          mbar_wait_bounded(&sm.full[wp][a][0], ph);
          mbar_wait_bounded(&sm.full[wp][a][1], ph);
        }
        return;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = T == 1 ? (2 * c + e) & 3 : 2 * c + e, rr = it0.rg * kUnitRows + r;
        const bool in = rr < R && (T == 2 || c < 2);
        const int j = column(min(rr, R - 1)), i = pair * p.g + min(rr, R - 1) - j * p.g;
        const int64_t row = ((int64_t)b * M + j) * H + i;
        const float lam = in ? p.lam[p.lam_per_row ? row : i] : 0.0f;
        const float l0 = sm.ws[wp][0].row_sum[r], l1 = sm.ws[wp][1].row_sum[r];
#pragma unroll
        for (int md = 0; md < 8; ++md) {
          const float x0 = __fmul_rn(o[md][0][e], down[0][e]);
          const float x1 = __fmul_rn(o[md][0][2 + e], down[0][e]);
          const float y0 = T == 2 ? __fmul_rn(o[md][T - 1][e], down[T - 1][e])
                                  : __shfl_xor_sync(0xffffffffu, x0, 2);
          const float y1 = T == 2 ? __fmul_rn(o[md][T - 1][2 + e], down[T - 1][e])
                                  : __shfl_xor_sync(0xffffffffu, x1, 2);
          if (in)
            *reinterpret_cast<float2*>(p.out + row * 2 * kD + a * kD + 16 * md + 2 * g) =
                make_float2(diff_out(x0, l0, y0, l1, lam), diff_out(x1, l0, y1, l1, lam));
        }
      }
    } else {
      float* part = p.partials + (((size_t)b * p.nwin_max + it0.w) * p.pairs + pair) * diff_stride(R);
#pragma unroll
      for (int n = 0; n < T; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 2 * c + e, map = T == 1 ? r >> 2 : n;
          const int rr = it0.rg * kUnitRows + (T == 1 ? r & 3 : r);
          if (rr >= R) continue;
          float* dst = part + (size_t)(map * R + rr) * 2 * kD + a * kD + 2 * g;
#pragma unroll
          for (int md = 0; md < 8; ++md)
            *reinterpret_cast<float2*>(dst + 16 * md) =
                make_float2(__fmul_rn(o[md][n][e], down[n][e]), __fmul_rn(o[md][n][2 + e], down[n][e]));
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = it0.rg * kUnitRows + 2 * c + e;
        if (g == 0 && rr < R && (T == 2 || c < 2)) {
          float* ml = part + (size_t)2 * R * 2 * kD + 4 * rr;    // m_0, m_1, l_0, l_1
          ml[a] = e ? m_run.y : m_run.x;
          ml[2 + a] = e ? l_run.y : l_run.x;
        }
      }
    }

    // ---- next item
    if (++u >= u_end) {
      named_sync(1 + wp, 64);                     // (for a warp that gave up at the last V copy)
      return;
    }
    ipar ^= 1;
    put_next(ipar ^ 1);
    entry = row_entry(p, ws.item[ipar ^ 1], lane);
    if (ws.item[ipar ^ 1].b >= 0 && ws.item[ipar ^ 1].fresh) {   // its queries (lane: a line of a row)
      const DiffItem& nx = ws.item[ipar ^ 1];
      const int rr = min(nx.rg * kUnitRows + min(lane >> 2, kUnitRows - 1), R - 1), j = column(rr);
      prefetch_l2(p.q + (((int64_t)nx.b * M + j) * p.Hq + 2 * (nx.pair * p.g + rr - j * p.g) + a) * kD +
                  32 * (lane & 3));
    }
  }
}

// Joins the windows of a row: W warps take a half of its channels.  The windows
// k, k + 8, ... are summed with the weights e^(m_s - max m), for k = 0 .. 7; the
// eight sums are added in order, and the two maps are subtracted.  The order depends
// on neither W nor other rows.  Bound by the partials' way out of L2 and the trips
// there that depend on one another (statistics, then 4 W windows a trip): a warp has
// to have enough windows for its lifetime, and a long row enough warps.  Measured, the
// call with W = 2, 4, 8: 16 sequences of 1k to 4k keys, 5 columns 56, 58, 62 us (64
// sequences 183, 191, 210); 64 of up to 32k keys 123, 121, 125 us; 4 of 128k keys
// 163, 145, 136 us.
constexpr int kClasses = 8, kBatch = 4;
template <int W>
constexpr int merge_halves = W == 8 ? 1 : 2;      // of a row, in a block

template <int W>
__global__ void __launch_bounds__(32 * W * merge_halves<W>) diff_merge_kernel(const DiffParams p) {
  constexpr int kOwn = kClasses / W;              // sums of a warp: k = warp, warp + W, ...
  static_assert(kBatch % kOwn == 0 && W * kBatch <= 32, "a batch holds whole rounds of the sums");
  __shared__ float4 s_o[merge_halves<W>][kClasses][2][kD / 4];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W, side = (threadIdx.x >> 5) / W;
  const int i = blockIdx.x * merge_halves<W> >> 1, j = blockIdx.y, b = blockIdx.z;
  const int half = merge_halves<W> == 2 ? side : blockIdx.x & 1;
  const int ctx = p.ctx_len[b], H = p.Hq / 2, R = p.R;
  const bool valid = diff_valid(p, b, ctx);
  const int64_t row = ((int64_t)b * p.M + j) * H + i;
  const float lam = p.lam[p.lam_per_row ? row : i];
  const int ns = diff_windows(ctx + j);
  const int pair = i / p.g, rr = j * p.g + i % p.g;
  const size_t stride = (size_t)p.pairs * diff_stride(R);
  const float* base = p.partials + ((size_t)b * p.nwin_max * p.pairs + pair) * diff_stride(R);
  const float* mlcol = base + (size_t)2 * R * 2 * kD + 4 * rr;
  const float* ocol = base + (size_t)rr * 2 * kD + half * kD + 4 * lane;
  const size_t map1 = (size_t)R * 2 * kD;
  griddep_wait();                                 // every partial is in place
  if (!valid || diff_windows(ctx + p.M - 1) == 1) return;

  float4 v[kBatch][2];
  // The warp's n-th window after s0 (s0 a multiple of 4 W): W n + warp.
  auto load = [&](int s0) {
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int s = s0 + W * n + warp;
#pragma unroll
      for (int a = 0; a < 2; ++a)
        v[n][a] = s < ns ? __ldcg(reinterpret_cast<const float4*>(ocol + s * stride + a * map1))
                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  };
  auto stats = [&](int s) {                       // m_0, m_1, l_0, l_1 of window s
    return s < ns ? __ldcg(reinterpret_cast<const float4*>(mlcol + s * stride))
                  : make_float4(-INFINITY, -INFINITY, 0.0f, 0.0f);
  };
  load(0);
  const float4 st0 = stats(lane);
  float mx[2] = {st0.x, st0.y};                   // the row's maxima
  for (int s = lane + 32; s < ns; s += 32) {
    const float4 st = stats(s);
    mx[0] = fmaxf(mx[0], st.x);
    mx[1] = fmaxf(mx[1], st.y);
  }
  mx[0] = warp_max(mx[0]);
  mx[1] = warp_max(mx[1]);

  float4 acc[kOwn][2];
#pragma unroll
  for (int k = 0; k < kOwn; ++k)
#pragma unroll
    for (int a = 0; a < 2; ++a) acc[k][a] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l[2] = {0.0f, 0.0f};
  for (int s0 = 0; s0 < ns; s0 += 32) {           // lane n weighs window s0 + n
    float w[2];
    {
      const float4 st = s0 ? stats(s0 + lane) : st0;
      w[0] = exp_diff(st.x, mx[0]);               // (-inf past the last window: 0)
      w[1] = exp_diff(st.y, mx[1]);
      l[0] = __fmaf_rn(w[0], st.z, l[0]);
      l[1] = __fmaf_rn(w[1], st.w, l[1]);
    }
#pragma unroll 1
    for (int at = 0; at < 32 && s0 + at < ns; at += W * kBatch) {
      if (s0 + at > 0) load(s0 + at);
#pragma unroll
      for (int n = 0; n < kBatch; ++n)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const float wn = __shfl_sync(0xffffffffu, w[a], at + W * n + warp);
          float4& x = acc[n % kOwn][a];
          x = make_float4(__fmaf_rn(wn, v[n][a].x, x.x), __fmaf_rn(wn, v[n][a].y, x.y),
                          __fmaf_rn(wn, v[n][a].z, x.z), __fmaf_rn(wn, v[n][a].w, x.w));
        }
    }
  }
  l[0] = warp_sum(l[0]);
  l[1] = warp_sum(l[1]);

#pragma unroll
  for (int k = 0; k < kOwn; ++k)
#pragma unroll
    for (int a = 0; a < 2; ++a) s_o[side][k * W + warp][a][lane] = acc[k][a];
  __syncthreads();
  if (warp != 0) return;
  float4 O[2];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    O[a] = s_o[side][0][a][lane];
#pragma unroll
    for (int k = 1; k < kClasses; ++k) {
      const float4 x = s_o[side][k][a][lane];
      O[a] = make_float4(__fadd_rn(O[a].x, x.x), __fadd_rn(O[a].y, x.y), __fadd_rn(O[a].z, x.z),
                         __fadd_rn(O[a].w, x.w));
    }
  }
  *reinterpret_cast<float4*>(p.out + row * 2 * kD + half * kD + 4 * lane) =
      make_float4(diff_out(O[0].x, l[0], O[1].x, l[1], lam), diff_out(O[0].y, l[0], O[1].y, l[1], lam),
                  diff_out(O[0].z, l[0], O[1].z, l[1], lam), diff_out(O[0].w, l[0], O[1].w, l[1], lam));
}

// ------------------------------------------------------------------- host
// 2-D view [rows][128] of an int8 cache; kBlockBk-row boxes, 128-byte swizzle.
bool encode_plane_map(CUtensorMap* map, const int8_t* base, int64_t rows) {
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
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int T>
cudaError_t launch_split(DiffParams p, const TmaMaps& maps, cudaStream_t stream) {
  const auto kern = diff_split_kernel<T>;
  const int smem = (int)sizeof(DiffSmem<T>) + 1024;     // + alignment slack
  // per device: the CTAs that the GPU holds at once; the shared-memory limit is
  // raised with the first call
  static std::atomic<int> slots_cache[kMaxDevices], sms_cache[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  int slots = cached ? slots_cache[dev].load() : 0, sms = cached ? sms_cache[dev].load() : 0;
  if (slots <= 0 || sms <= 0) {
    int per_sm = 0;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) !=
        cudaSuccess)
      return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, smem)) !=
        cudaSuccess)
      return e;
    slots = sms * (per_sm > 0 ? per_sm : 1);
    if (cached) {
      slots_cache[dev].store(slots);
      sms_cache[dev].store(sms);
    }
  }
  p.sms = sms;
  kern<<<(unsigned)std::min<int64_t>(diff_units(p), slots), kThreads, smem, stream>>>(p, maps);
  return cudaGetLastError();
}

// Whether diff_tc_kernel takes the call: more than 16 rows per map, and enough windows
// for the multiprocessors to have several at once.  One window alone takes it longer,
// and short sequences have more unit starts than blocks.  The call in us, diff_tc_kernel |
// row groups (in brackets: the side that the rule takes where it is the slower):
//   32 query and 4 kv heads
//   sequences x keys, columns       3             5             8
//    1 x 100                       23 | 16       24 | 16       34 | 16
//    4 x 1k..4k                    26 | 28       29 | 30       38 | 30
//    8 x 1k..4k                    33 | 30       39 | 31       56 | 51
//   12 x 1k..4k                    41 | 31 (tc)  42 | 52       59 | 70
//   16 x 1k..4k                    43 | 44       54 | 53 (tc)  75 | 76
//   24 x 1k..4k                    45 | 52       71 | 74      102 | 100 (tc)
//   64 x 1k..4k                   103 | 121     144 | 177     218 | 279
//   16 x 16k..32k                 228 | 254     308 | 399     473 | 622
//    1 x 64k                       76 | 65 (tc)  76 | 88      112 | 124
//   90 x 100..500                  49 | 49       76 | 70      112 | 100
//   256 x 100..500                122 | 110     186 | 179     262 | 280 (groups)
//   5 columns, other heads       16q / 2kv     48q / 6kv     64q / 8kv
//   16 x 1k..4k                    40 | 32       71 | 76       81 | 98
//   64 x 1k..4k                    82 | 99      202 | 264     260 | 339
//   90 x 100..500                  44 | 44      103 | 98      121 | 126 (groups)
// (With 16 rows, two groups: 64 x 1k..4k 80 | 84, 16 x 1k..4k 37 | 33.)  The windows are
// counted from max_ctx, as the host does not know the lengths: a limit far above them
// (131072, as a server's graph may pass) brings short batches here too, and a wider join.
// Then, 32q / 4kv: 1 x 100, 8 columns 37 us instead of 16; 16 x 1k..4k, 5 columns 60
// instead of 54 (groups 60); 64 x 1k..4k, 5 columns 170 instead of 144; 90 x 100..500, 8
// columns 169 instead of 100 (groups 156).
bool many_rows(const DiffParams& p) {
  static std::atomic<int> sms_cache[kMaxDevices];
  if (p.R <= 16 || p.nwin_max < 4) return false;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  int sms = cached ? sms_cache[dev].load() : 0;
  if (sms <= 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return false;
    if (cached) sms_cache[dev].store(sms);
  }
  return 2 * (int64_t)p.B * p.nwin_max * p.pairs >= 5 * (int64_t)sms;
}

template <int W>
cudaError_t launch_merge(const DiffParams& p, cudaStream_t stream) {
  constexpr int kHalves = merge_halves<W>;
  return launch_pdl(diff_merge_kernel<W>, dim3((unsigned)(p.Hq / kHalves), (unsigned)p.M, (unsigned)p.B),
                    dim3(32 * W * kHalves), 0, stream, p);
}

}  // namespace

int64_t diff_units(const DiffParams& p) {
  const int rows = p.R <= 4 ? 4 : 8;
  return (int64_t)p.B * diff_windows(p.max_ctx + p.M - 1) * p.pairs * ((p.R + rows - 1) / rows);
}

size_t diff_workspace_bytes(int B, int M, int Hq, int max_ctx) {
  // pairs * diff_stride(R) = Hq * M * (2 d + 2) whatever Hkv is
  return 256 + (size_t)B * diff_windows(max_ctx + M - 1) * Hq * M * (2 * kD + 2) * sizeof(float);
}

void set_diff_workspace(DiffParams& p, void* workspace) {
  p.err_word = static_cast<uint32_t*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  p.nwin_max = diff_windows(p.max_ctx + p.M - 1);
}

cudaError_t launch_decode_diff(const DiffParams& p, cudaStream_t stream) {
  TmaMaps maps;
  const int64_t rows = (int64_t)p.Hkv * p.cap_rows;
  if (!encode_plane_map(&maps.k, p.k, rows) || !encode_plane_map(&maps.v, p.v, rows))
    return cudaErrorInvalidValue;
  const cudaError_t e = many_rows(p) ? launch_tc_rows(p, maps, stream)
                        : p.R <= 4   ? launch_split<1>(p, maps, stream)
                                     : launch_split<2>(p, maps, stream);
  if (e != cudaSuccess || p.nwin_max <= 1) return e;
  if (p.nwin_max <= 32) return launch_merge<2>(p, stream);
  if (p.nwin_max <= 256) return launch_merge<4>(p, stream);
  return launch_merge<8>(p, stream);
}

}  // namespace kattn
