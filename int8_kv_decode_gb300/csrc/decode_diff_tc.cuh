// The windows of the differential attention for more than 16 rows per map, with P.V
// on the fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// A block takes a unit (sequence, window, plane pair) with all rows: one warp per 8
// rows of a map, and one that issues copies and MMAs.  Per 32 keys, copied by TMA into
// a ring of stages, a warp scores its rows on the int8 MMA, takes their weights, and
// writes them times the v_scales of either plane as f16 hi + lo; the warps share the
// conversion of the values to f16, so every value is converted once for all rows.
// After a barrier one thread issues, for both planes,
//   D[channel][row] += V^T[channel][key] P[row][key]
// (M = 128, N = the rows of both maps, K = 16), hi and lo of the first 16 keys, then of
// the second: the order of the mma.sync kernel, whose bits a step of tcgen05
// reproduces, so a row has the same bytes in either.  The MMAs run beside the next
// block's scores.
//
// What bounds it: the instructions of a block (660 per warp of 8 rows) in the chain
// scores, weights, operands, with the warps that tensor memory leaves a
// multiprocessor (2 blocks of 11 at 40 rows): issue 48%, int8 MMA 38% busy.  16
// sequences of 16k to 32k keys, 5 draft columns, 32 query and 4 kv heads: the call 308
// us (405 MB, 60 us at the measured copy rate; this kernel 256 us), row groups on
// mma.sync 399 us.  Tried:
// mbarriers in place of the block's barrier, so that warps run up to a block apart,
// the same to 5% slower; one block a multiprocessor with 6 stages 19% slower; the cache
// in L2, or another L2 policy, the same.
#pragma once

#include "decode_diff.cuh"
#include "tcgen05_common.cuh"

namespace kattn {
namespace {

constexpr int kTcStageBytes = 4 * kBlockBytes;    // K of both planes, V of both

// Of a block with W warps of 8 rows (W / 2 per map).
template <int W>
struct TcShape {
  static constexpr int kRows = 8 * W, kTiles = W / 2;
  static constexpr int kThreads = 32 * (W + 1);   // and the warp that issues copies and MMAs
  static constexpr int kOperand = 32 * kRows;     // bytes of P: 16 keys, hi or lo
  // tensor-memory columns: the rows of either plane's product, a power of two in all
  static constexpr int kColumns = W <= 4 ? 64 : W <= 8 ? 128 : 256, kPlane = kColumns / 2;
  static constexpr int kStages = W <= 8 ? 2 : 3;
  static constexpr int kPerSm = W <= 8 ? 3 : 2;   // blocks a multiprocessor holds
  static constexpr int kReaders = W >= 8 ? 8 : 4; // warps that read the accumulators
};

template <int W>
struct __align__(1024) DiffTcSmem {
  uint8_t ring[TcShape<W>::kStages][kTcStageBytes];
  uint8_t vt[2][2][kBlockBytes];                  // [plane][16 keys]: V^T as f16, K-major
  uint8_t pb[2][2][2][TcShape<W>::kOperand];      // [plane][16 keys][hi | lo]: P, K-major
  float ks[2][2][kWindow], vs[2][2][kWindow];     // [item slot][plane]: the window's scales
  float down[2][2][8 * W];                        // [item slot][plane][row]: 2^-E (minus the largest product
                                                  // while E follows it)
  float alpha[2][8 * W];                          // [plane] where E follows the products, else [0]
  float row_sum[8 * W];                           // of a sequence that ends in its window
  int rows[2][kWinBlocks];                        // [item slot]: rows of the blocks in a plane
  uint64_t full[TcShape<W>::kStages], done;       // a stage's copies landed; the MMAs are done
  int fail[2];                                    // the block (+ 1) at which a wait ran out
  uint32_t tmem;
};

__device__ __forceinline__ void tc_mma_n(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, 1, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc));
}
__device__ __forceinline__ void copy_word_async(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src),
               "r"(in ? 4 : 0)
               : "memory");
}

template <int W>
__global__ void __launch_bounds__(TcShape<W>::kThreads, TcShape<W>::kPerSm)
diff_tc_kernel(const DiffParams p, const __grid_constant__ TmaMaps maps) {
  using S = TcShape<W>;
  static_assert((sizeof(DiffTcSmem<W>) + 2048) * S::kPerSm <= 228 * 1024, "with the slack and the reserve of a block");
  constexpr int kStages = S::kStages, kTiles = S::kTiles, kReaders = S::kReaders;
  extern __shared__ unsigned char smem_raw[];
  DiffTcSmem<W>& sm = *reinterpret_cast<DiffTcSmem<W>*>(smem_raw + (0u - smem_u32(smem_raw)) % 1024u);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const bool issuer = warp == W;
  const int a = warp >= kTiles, rg = a ? warp - kTiles : warp;   // a warp's map (and key plane), and tile
  const int g = lane >> 2, c = lane & 3, odd = g & 1;
  const int M = p.M, R = p.R, H = p.Hq / 2;

  // (the sums over the batch are needed at the start alone)
  int* const prefix = reinterpret_cast<int*>(sm.vt);
  DiffUnits units(p, prefix, 1, 1);
  units.count(prefix, prefix + kMaxGroups + 1);
  mark_bad_sequences(p);
  __syncthreads();
  griddep_launch_dependents();
  // A block each, if there are enough; else shares by their blocks: where the units are
  // just more than the blocks, two short ones go together, not two long ones.
  if (prefix[kMaxGroups] > (int)gridDim.x) {
    units.longer = kWindow / kShortWindow;
    __syncthreads();
    units.count(prefix, prefix + kMaxGroups + 1);
    __syncthreads();
  }
  const int total = prefix[kMaxGroups], G = gridDim.x;
  // (blocks that start on one multiprocessor are numbered one after the other)
  const int per_sm = G / p.sms, more = G - per_sm * p.sms, on = blockIdx.x % p.sms;
  const int worker = on * per_sm + min(on, more) + blockIdx.x / p.sms;
  int at = (int)((int64_t)worker * total / G);    // where the unit starts in the batch's cost
  const int end = (int)((int64_t)(worker + 1) * total / G);
  DiffItem it;
  if (!units.find(&at, end, &it)) return;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[s], 1);
    mbar_init(&sm.done, 1);
    sm.fail[0] = sm.fail[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (issuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n"
                 ::"r"(smem_u32(&sm.tmem)), "r"(S::kColumns));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  auto after = [&](const DiffItem& x, int at) {   // the unit after x, which starts at `at`
    DiffItem n = x;
    n.b = -1;
    if (at + units.cost(x.w) < end) n = units.after(x);
    return n;
  };
  DiffItem nxt = after(it, at);
  // rows of an item's blocks from the table's entries (one warp)
  auto put_rows = [&](int slot, const DiffItem& x, int entry) {
    const int row = row_of_entry(p, x, entry, lane);
    if (lane < kWinBlocks) sm.rows[slot][lane] = x.b >= 0 && lane < units.blocks(x) ? row : 0;
    __syncwarp();
  };
  // an item's scales, one word per thread and copy; keys past the last are 0
  auto copy_scales = [&](int slot, const DiffItem& x) {
    const int n = min(window_keys(x.w), x.ctx + M - 1 - window_start(x.w));
    for (int i = tid; i < 2 * kWindow; i += S::kThreads) {
      const int key = i & (kWindow - 1), pl = i / kWindow;
      const bool in = key < n;
      const int64_t at = in ? (int64_t)sm.rows[slot][key >> 5] + (key & 31) + (2 * x.pair + pl) * p.cap_rows : 0;
      copy_word_async(smem_u32(&sm.ks[slot][pl][key]), p.k_scale + at, in);
      copy_word_async(smem_u32(&sm.vs[slot][pl][key]), p.v_scale + at, in);
    }
  };
  if (issuer) put_rows(0, it, row_entry(p, it, lane));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  copy_scales(0, it);
  asm volatile("cp.async.wait_all;\n" ::: "memory");
  __syncthreads();

  const uint64_t policy = l2_evict_first();
  int commits = 0, waited = 0;                    // MMA groups committed / waited for
  int gb = 0, st = 0;                             // the block, its stage and the parity of its copies
  uint32_t ph = 0;
  int slot = 0, nb = units.blocks(it), nb_next = nxt.b >= 0 ? units.blocks(nxt) : 0;
  // Copies (the issuing warp): block `ahead` of this item, or of the next one, into the
  // next stage.  A stage is refilled once every warp has passed the block in it.
  int ahead = 0, put_st = 0, issued = 0;
  auto produce = [&]() -> bool {
    const bool mine = ahead < nb;
    if (!mine && ahead - nb >= nb_next) return false;
    const int row = mine ? sm.rows[slot][ahead] : sm.rows[slot ^ 1][ahead - nb];
    const int plane = 2 * (mine ? it.pair : nxt.pair);
    uint8_t* dst = sm.ring[put_st];
    uint64_t* bar = &sm.full[put_st];
    if (lane == 0) {
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      mbar_expect_tx(bar, kTcStageBytes);
#pragma unroll
      for (int pl = 0; pl < 2; ++pl) {
        tma_load_block(dst + pl * kBlockBytes, &maps.k, row + (plane + pl) * p.cap_rows, bar, policy);
        tma_load_block(dst + (2 + pl) * kBlockBytes, &maps.v, row + (plane + pl) * p.cap_rows, bar, policy);
      }
    }
    __syncwarp();
    ++ahead;
    ++issued;
    put_st = put_st + 1 == kStages ? 0 : put_st + 1;
    return true;
  };
#ifdef KATTN_DIFF_STAGE_LIMIT
  // Test builds only: the warps of the maps KATTN_DIFF_STAGE_MAPS (a bit each) take
  // this many copies, then find none ready.
  int taken = 0;
  auto ready = [&](uint64_t* bar, uint32_t parity) {
    return !((KATTN_DIFF_STAGE_MAPS >> a & 1) && taken++ >= KATTN_DIFF_STAGE_LIMIT) &&
           stage_ready(smem_u32(bar), parity);
  };
#else
  auto ready = [&](uint64_t* bar, uint32_t parity) { return stage_ready(smem_u32(bar), parity); };
#endif
  // rr / g and the query head of unit row rr (rr < 64, g <= 64: exact)
  const uint32_t ginv = 65536u / (uint32_t)p.g + 1u;
  auto column = [&](int rr) -> int { return (int)(((uint32_t)rr * ginv) >> 16); };

  // Accumulators: a warp sees the lanes (channels) 32 (warp mod 4) ...; the first
  // kReaders warps divide the quarters of both planes.
  const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)W << 17) | ((128u >> 4) << 24);   // N = 8 W
  // this lane's place in the operands: P (row 2c + odd, keys g & ~1 ...) and V^T (row g)
  const int lane_p = warp * 256 + (2 * c + odd) * 16 + (g & 6) * 2, lane_v = g * 16 + c * 4;
  uint4 qlo = make_uint4(0, 0, 0, 0), qhi = qlo;  // bytes 32c .. 32c + 31 of row g
  float2 qs = make_float2(0.0f, 0.0f);            // scales of rows 2c, 2c + 1
  bool failed = false;

  for (;;) {
    const int s0 = window_start(it.w), s1 = min(s0 + window_keys(it.w), it.ctx + M - 1);
    int pentry = 0;
    if (issuer) {
      pentry = row_entry(p, nxt, lane);
      if (gb == 0)
        for (int n = 0; n < kStages && n < nb; ++n) produce();
    }
    // every accumulator starts at +0
    if (warp < kReaders) {
      float z[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = 0.0f;
#pragma unroll
      for (int x = 0; x < 8 / kReaders; ++x)
#pragma unroll
        for (int n = 0; n < S::kRows; n += 16)
          tc_st16(tlane + (kReaders == 4 ? x : warp >> 2) * S::kPlane + n, z);
      tc_wait_st();
    }
    // ---- the queries of the warp's 8 rows, quantized per row
    if (it.fresh && !issuer) {
      float4 x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int rr = min(rg * 8 + r, R - 1), j = column(rr);
        const int head = 2 * (it.pair * p.g + rr - j * p.g) + a;
        x[r] = __ldg(reinterpret_cast<const float4*>(p.q + (((int64_t)it.b * M + j) * p.Hq + head) * kD) + lane);
      }
      uint32_t q[8];
      float sc[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const bool in = rg * 8 + r < R;
        uint32_t w = quantize_loaded_row(x[r], &sc[r]);
        w = in ? w : 0u;
        if (!in) sc[r] = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t v = __shfl_sync(0xffffffffu, w, 8 * c + k);
          if (g == r) q[k] = v;
        }
        if (r == 2 * c) qs.x = sc[r];
        if (r == 2 * c + 1) qs.y = sc[r];
      }
      qlo = make_uint4(q[0], q[1], q[2], q[3]);
      qhi = make_uint4(q[4], q[5], q[6], q[7]);
    }
    auto keys_of = [&](int r) -> int { return it.ctx + column(min(rg * 8 + r, R - 1)); };
    // ---- 2^E of the row 2c + odd, for either plane's scales (with a minus: it follows the
    // products).  Lane j takes column j, so that every warp finds the same `care` (see
    // ScaleRange): they go through the blocks together.
    float up[2];
    bool care = false;
#pragma unroll
    for (int pl = 0; pl < 2; ++pl) {
      float most = 0.0f, least = INFINITY;
#pragma unroll
      for (int e = 0; e < kWinBlocks; ++e)
        if (s0 + 32 * e + lane < min(it.ctx, s1)) {
          const float v = sm.vs[slot][pl][32 * e + lane];
          most = fmaxf(most, v);
          least = fminf(least, v);
        }
      ScaleRange range = warp_range(most, least);
      const int keys = it.ctx + min(lane & 7, M - 1);
      for (int key = max(it.ctx, s0); key < s1; ++key) range.add(sm.vs[slot][pl][key - s0], key < keys);
      care |= range.care();
      const float u = range.spread() ? -1.0f : range.scale();
      up[pl] = __shfl_sync(0xffffffffu, u, column(min(rg * 8 + 2 * c + odd, R - 1)));
      if (g < 2 && !issuer)
        sm.down[slot][pl][8 * warp + 2 * c + g] = up[pl] < 0.0f ? -0.0f : inverse_scale(up[pl]);
    }
    care = __any_sync(0xffffffffu, care);
    __syncwarp();
    float2 m_run = make_float2(0.0f, 0.0f), m_move = make_float2(-INFINITY, -INFINITY);
    float2 l_run = make_float2(0.0f, 0.0f);

    const float* const ks0 = &sm.ks[slot][a][g];
    auto blocks = [&](auto careful) __attribute__((always_inline)) {
      constexpr bool kCare = decltype(careful)::value;
      for (int i = 0; i < nb; ++i, ++gb) {
        const int t0 = s0 + i * kBlockBk;
        bool moved = false;
        if (!issuer) {
          bool ok = ready(&sm.full[st], ph);
          const uint32_t ring = smem_u32(sm.ring[st]);
          int acc[2][4];
          key_products(ring + a * kBlockBytes + (uint32_t)swz(g, 2 * c), qlo, qhi, acc);
          float ks4[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) ks4[q] = ks0[32 * i + 8 * q];
          float2 sc[2][2];
          scores_of(acc, ks4, qs, p.sm_scale, sc);
          if (t0 + kBlockBk > it.ctx) hide_keys(sc, t0 + g, keys_of(2 * c), keys_of(2 * c + 1));
          float2 alpha = make_float2(1.0f, 1.0f);
          moved = block_weights(sc, m_run, m_move, l_run, alpha);
          // ---- the weights of two keys of a row side by side: keys 8q + (g & ~1) and the
          // next, row 2c + odd
          float2 w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 x = sc[q >> 1][q & 1];
            const float other = __shfl_xor_sync(0xffffffffu, odd ? x.x : x.y, 4);
            w[q] = odd ? make_float2(other, x.y) : make_float2(x.x, other);
          }
          // ---- the MMAs of the block before have read the operands
          if (commits > waited) {
            const bool ok_m = stage_ready(smem_u32(&sm.done), (uint32_t)(commits - 1) & 1u);
            if (ok_m) waited = commits;             // else the exit waits again
            ok = ok && ok_m;
            tc_fence_after();
          }
          if (!ok) {
            sm.fail[gb & 1] = gb + 1;
          } else {
            uint8_t* const dst = &sm.pb[0][0][0][0] + lane_p;
            const float* const vs0 = &sm.vs[0][0][0] + slot * 2 * kWindow + 32 * i + (g & 6);
            auto put = [&](float2 y, int pl, int q) {
              uint32_t hi, lo;
              split_f16x2(y.x, y.y, hi, lo);
              uint8_t* const to = dst + (pl * 4 + (q >> 1) * 2) * S::kOperand + (q & 1) * 128;
              *reinterpret_cast<uint32_t*>(to) = hi;
              *reinterpret_cast<uint32_t*>(to + S::kOperand) = lo;
            };
            if constexpr (kCare) {                // (state in shared memory: the other loop needs the registers)
#pragma unroll 1
              for (int pl = 0; pl < 2; ++pl) {
                const int row = 8 * warp + 2 * c + odd;
                const float u = pl ? up[1] : up[0];
                float mag = -sm.down[slot][pl][row], m = 0.0f;
                float2 y[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float2 vs = *reinterpret_cast<const float2*>(vs0 + pl * kWindow + 8 * q);
                  y[q] = f2_mul(w[q], f2_mul(vs, make_float2(fabsf(u), fabsf(u))));
                  hide_products(y[q], w[q]);
                  m = fmaxf(m, fmaxf(y[q].x, y[q].y));
                }
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                float f = odd ? alpha.y : alpha.x, post = 1.0f;
                if (u < 0.0f) {
                  f = follow_products(m, f, mag);
                  post = product_scale(mag);
                }
                moved = __any_sync(0xffffffffu, moved || f != 1.0f);
                __syncwarp();                     // (every lane has read the row's state)
                if (g < 2) {
                  sm.alpha[pl][row] = f;
                  sm.down[slot][pl][row] = -mag;
                }
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 4; ++q) put(f2_mul(y[q], make_float2(post, post)), pl, q);
              }
            } else {
#pragma unroll
              for (int pl = 0; pl < 2; ++pl)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float2 vs = *reinterpret_cast<const float2*>(vs0 + pl * kWindow + 8 * q);
                  put(f2_mul(w[q], f2_mul(vs, make_float2(up[pl], up[pl]))), pl, q);
                }
              if (g == 0) *reinterpret_cast<float2*>(&sm.alpha[0][8 * warp + 2 * c]) = alpha;
            }
            // ---- V^T: item x = (plane, 16 keys, 32 channels).  Row 16q + g holds channel
            // 16q + 2g, row 16q + 8 + g the next one.
            const uint32_t va = ring + 2 * kBlockBytes +
                                (uint32_t)((lane & 15) * kD + (((lane >> 4) ^ (lane & 7)) << 4));
#pragma unroll
            for (int x0 = 0; x0 < 16; x0 += W) {
              const int x = x0 + warp;              // 8 plane + 4 half + chunk pair
              if (x0 + W > 16 && x >= 16) break;
              uint32_t vw[4];
              ldsm_x4_trans<0>(vw, (va ^ (uint32_t)((x & 3) << 5)) + (x >> 3) * kBlockBytes + ((x >> 2) & 1) * 2048);
              uint8_t* const to = &sm.vt[0][0][0] + lane_v + x * 1024;
#pragma unroll
              for (int d = 0; d < 2; ++d) {
                uint32_t af[4];
                value_operand(vw[2 * d], vw[2 * d + 1], af);
                *reinterpret_cast<uint32_t*>(to + d * 512) = af[0];
                *reinterpret_cast<uint32_t*>(to + d * 512 + 256) = af[1];
                *reinterpret_cast<uint32_t*>(to + d * 512 + 128) = af[2];
                *reinterpret_cast<uint32_t*>(to + d * 512 + 384) = af[3];
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        } else if (i == 0) {                        // the next item's rows
          put_rows(slot ^ 1, nxt, pentry);
        }
        tc_fence_before();
        const bool rescale = __syncthreads_or(moved) != 0;
        if (sm.fail[gb & 1] == gb + 1) {
          failed = true;
          return;
        }
        if (rescale) {                              // D *= alpha where a reference moved
          if (warp < kReaders) {
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 8 / kReaders; ++x)
#pragma unroll 1
              for (int n = 0; n < S::kRows; n += 16) {
                const int pl = kReaders == 4 ? x : warp >> 2;
                const uint32_t at = tlane + pl * S::kPlane + n;
                float v[16];
                tc_ld16(at, v);
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                  const float2 y = f2_mul(make_float2(v[j], v[j + 1]),
                                          *reinterpret_cast<const float2*>(&sm.alpha[kCare ? pl : 0][n + j]));
                  v[j] = y.x;
                  v[j + 1] = y.y;
                }
                tc_st16(at, v);
              }
            tc_wait_st();
            tc_fence_before();
          }
          __syncthreads();
        }
        if (issuer) {
          if (lane == 0) {
            tc_fence_after();
#pragma unroll
            for (int pl = 0; pl < 2; ++pl)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const uint64_t v = smem_desc(sm.vt[pl][hf]);
                tc_mma_n(tmem + pl * S::kPlane, v, smem_desc(sm.pb[pl][hf][0]), kIdesc);
                tc_mma_n(tmem + pl * S::kPlane, v, smem_desc(sm.pb[pl][hf][1]), kIdesc);
              }
            tc_commit(&sm.done);
          }
          __syncwarp();
          while (issued <= gb + kStages && produce()) {}
        }
        ++commits;
        if (++st == kStages) {
          st = 0;
          ph ^= 1u;
        }
        if (i == 0 && nxt.b >= 0) copy_scales(slot ^ 1, nxt);
      }
    };
    if (!care) {
      blocks(std::false_type{});
    } else {
      blocks(std::true_type{});
#pragma unroll
      for (int pl = 0; pl < 2; ++pl)
        if (up[pl] < 0.0f && g < 2 && !issuer) {
          float& x = sm.down[slot][pl][8 * warp + 2 * c + g];
          x = inverse_scale(product_scale(-x));
        }
    }
    if (failed) break;

    // ---- the window's row sums and references
    const bool whole = units.windows(it.ctx) == 1;
    float* part = p.partials + (((size_t)it.b * p.nwin_max + it.w) * p.pairs + it.pair) * diff_stride(R);
    l_run = make_float2(row_total(l_run.x), row_total(l_run.y));
    if (g == 0 && !issuer) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = rg * 8 + 2 * c + e;
        if (whole) {
          sm.row_sum[8 * warp + 2 * c + e] = e ? l_run.y : l_run.x;
        } else if (rr < R) {
          float* ml = part + (size_t)2 * R * 2 * kD + 4 * rr;        // m_0, m_1, l_0, l_1
          ml[a] = e ? m_run.y : m_run.x;
          ml[2 + a] = e ? l_run.y : l_run.x;
        }
      }
    }
    // ---- the last MMAs land; the next item's scales have
    bool ok = true;
    if (commits > waited) {
      ok = stage_ready(smem_u32(&sm.done), (uint32_t)(commits - 1) & 1u);
      if (ok) waited = commits;
      tc_fence_after();
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    if (__syncthreads_or(!ok)) {
      failed = true;
      break;
    }
    if (warp < kReaders) {
      // lane l of a quarter is row l of V^T: channel 16 (l / 16) + 2 (l mod 8) + (l / 8) mod 2
      const int ch0 = 32 * (warp & 3) + (lane & 16) + 2 * (lane & 7) + ((lane >> 3) & 1);
#pragma unroll 1
      for (int x = 0; x < 8 / kReaders; ++x) {
        const int pl = kReaders == 4 ? x : warp >> 2;
        const uint32_t at = tlane + pl * S::kPlane;
        float* dst0 = part + pl * kD + ch0;
        float* dst1 = dst0 + (size_t)R * 2 * kD;
#pragma unroll 1
        for (int t = 0; t < kTiles; ++t) {        // rows 8t .. 8t + 7 of both maps
          float o[2][8];
          tc_ld8(at + 8 * t, o[0]);
          tc_ld8(at + 8 * (kTiles + t), o[1]);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
              const float4 d = *reinterpret_cast<const float4*>(&sm.down[slot][pl][8 * (m * kTiles + t) + j]);
              o[m][j] = __fmul_rn(o[m][j], d.x);
              o[m][j + 1] = __fmul_rn(o[m][j + 1], d.y);
              o[m][j + 2] = __fmul_rn(o[m][j + 2], d.z);
              o[m][j + 3] = __fmul_rn(o[m][j + 3], d.w);
            }
          const int n = R - 8 * t;                // rows that there are
          if (!whole) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j < n) {
                dst0[j * 2 * kD] = o[0][j];
                dst1[j * 2 * kD] = o[1][j];
              }
            dst0 += 8 * 2 * kD;
            dst1 += 8 * 2 * kD;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j < n) {
                const int r = 8 * t + j, col = column(r), i = it.pair * p.g + r - col * p.g;
                const int64_t row = ((int64_t)it.b * M + col) * H + i;
                p.out[row * 2 * kD + pl * kD + ch0] =
                    diff_out(o[0][j], sm.row_sum[r], o[1][j], sm.row_sum[8 * kTiles + r],
                             p.lam[p.lam_per_row ? row : i]);
              }
          }
        }
      }
    }
    at += units.cost(it.w);
    if (nxt.b < 0) break;
    ahead -= nb;                                  // (blocks of the next item copied already)
    it = nxt;
    nb = nb_next;
    nxt = after(it, at);
    nb_next = nxt.b >= 0 ? units.blocks(nxt) : 0;
    slot ^= 1;
  }

  // ---- leave: every copy and MMA in flight lands (bounded) before the tensor memory
  // is given back.  The copies of blocks gb .. issued - 1 are under way.
  if (issuer && lane == 0) {
    for (int k = gb; k < issued; ++k) {
      mbar_wait_bounded(&sm.full[st], ph);
      if (++st == kStages) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (failed) atomicOr(p.err_word, KATTN_DEVERR_TIMEOUT);
  }
  if (commits > waited) mbar_wait_bounded(&sm.done, (uint32_t)(commits - 1) & 1u);
  asm volatile("cp.async.wait_all;\n" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (issuer)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(S::kColumns));
}

template <int W>
cudaError_t launch_tc(DiffParams p, const TmaMaps& maps, cudaStream_t stream) {
  const auto kern = diff_tc_kernel<W>;
  const int smem = (int)sizeof(DiffTcSmem<W>) + 1024;         // + alignment slack
  // per device: the multiprocessors; the shared-memory limit is raised with the first call
  static std::atomic<int> sms_cache[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kMaxDevices;
  int sms = cached ? sms_cache[dev].load() : 0;
  if (sms <= 0) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return e;
    if (cached) sms_cache[dev].store(sms);
  }
  p.sms = sms;
  const int64_t units = (int64_t)p.B * p.nwin_max * p.pairs;
  kern<<<(unsigned)std::min<int64_t>(units, (int64_t)sms * TcShape<W>::kPerSm), TcShape<W>::kThreads, smem,
         stream>>>(p, maps);
  return cudaGetLastError();
}

inline cudaError_t launch_tc_rows(const DiffParams& p, const TmaMaps& maps, cudaStream_t stream) {
  switch ((p.R + 7) / 8) {
    case 3: return launch_tc<6>(p, maps, stream);
    case 4: return launch_tc<8>(p, maps, stream);
    case 5: return launch_tc<10>(p, maps, stream);
    case 6: return launch_tc<12>(p, maps, stream);
    case 7: return launch_tc<14>(p, maps, stream);
    default: return launch_tc<16>(p, maps, stream);
  }
}

}  // namespace
}  // namespace kattn
