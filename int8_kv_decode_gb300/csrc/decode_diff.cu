// Differential decode attention over the int8 cache:
//   out = softmax(s_0) V - lam softmax(s_1) V
// for a pair of query heads (2i, 2i + 1), the key planes 2p and 2p + 1 and the
// 256 value channels of both planes.
//
// Two launches: diff_split_kernel reduces windows of kWindow keys, and
// diff_merge_kernel joins the windows of a row and takes the difference.  A
// sequence of one window is finished by the first.
//
// What bounds it: 528 bytes per key and plane pair must come from HBM, for
// 2 * 128 products per query row and map on the key side and 2 * 256 on the value
// side, so with up to 8 rows per map the stream of the cache is the bound.  The
// split reads each byte once for both maps.
#include "decode_split.cuh"
#include "ops_internal.cuh"

namespace kattn {
namespace {

// Every warp works on its own: it takes a unit (sequence, window, plane pair,
// row group), streams the window's rows through its own ring and writes the
// window's partial.  No warp waits for another, so a stall of one is covered by
// the others.  Windows sit at fixed key positions, so the bytes of a row depend
// on its own keys alone.
constexpr int kWindow = 256;
constexpr int kWinBlocks = kWindow / kBlockBk;    // 8: lane e < 8 holds the row of block e
constexpr int kWarps = 4;
constexpr int kStageBytes = 2 * kBlockBytes;      // the K (or V) rows of both planes of a block
constexpr int kMaxGroups = 512;                   // entries of the prefix over sequences
constexpr int kQStride = kD + 16;                 // bytes between query rows (spread over banks)

__host__ __device__ inline int diff_windows(int keys) { return (keys + kWindow - 1) / kWindow; }
__host__ __device__ inline int diff_stride(int R) { return 2 * R * (2 * kD + 2); }   // floats

// Tiles of 8 query rows: T = 2, one tile per map; T = 1, up to 4 rows, those of
// map 0 in rows 0..3 of the tile and those of map 1 in rows 4..7.
template <int T>
struct __align__(1024) DiffSmem {
  static constexpr int kStages = T == 1 ? 2 : 3;
  uint8_t ring[kWarps][kStages][kStageBytes];
  float scale[kWarps][4][kBlockBk];               // ks of both planes, vs of both planes
  uint8_t q[kWarps][T * 8 * kQStride];
  float qs[kWarps][T * 8];
  uint64_t full[kWarps][kStages];
  int prefix[kMaxGroups + 1];
  int warp_total[kWarps];
};

__device__ __forceinline__ bool diff_valid(const DiffParams& p, int b, int ctx) {
  if (p.block_table == nullptr) return sequence_ok(p.row_start[b], ctx, p.M, p.cap_rows, p.max_ctx);
  if (ctx < 1 || ctx > p.max_ctx) return false;
  const int64_t keys = (int64_t)ctx + p.M - 1;
  return ((keys + (1 << p.page_shift) - 1) >> p.page_shift) <= (int64_t)p.max_pages;
}

struct DiffItem {
  int b, pair, w, rg, ctx, row0;                  // b < 0: none
};

// Row (in a plane) of block e = lane of the item's window; lanes past the window hold 0.
__device__ __forceinline__ int block_row(const DiffParams& p, const DiffItem& it, int lane) {
  const int key = it.w * kWindow + lane * kBlockBk;
  if (it.b < 0 || lane >= kWinBlocks || key >= it.ctx + p.M - 1) return 0;
  if (p.block_table == nullptr) return it.row0 + key;
  int page = __ldg(p.block_table + (int64_t)it.b * p.max_pages + (key >> p.page_shift));
  if ((unsigned)page >= (unsigned)p.n_pages) {
    atomicOr(p.err_word, KATTN_DEVERR_BAD_PAGE);
    page = 0;
  }
  return (page << p.page_shift) | (key & ((1 << p.page_shift) - 1));
}

// Online-softmax update of one tile over a block; s0 / s1 hold the scores of the
// two 16-key halves in the MMA layout and return the weights.
__device__ __forceinline__ void diff_softmax(float (&s0)[4], float (&s1)[4], float (&m_run)[2],
                                             float (&l_run)[2], float (&alpha)[2], bool& rescale) {
  float mnew[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float bm = fmaxf(fmaxf(s0[e], s0[2 + e]), fmaxf(s1[e], s1[2 + e]));
    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
    mnew[e] = fmaxf(m_run[e], bm);
  }
  const float2 l2e = make_float2(kLog2e, kLog2e);
  const float2 mn = make_float2(mnew[0], mnew[1]);
  const bool live0 = mnew[0] != -INFINITY, live1 = mnew[1] != -INFINITY;
  const float2 da = f2_mul(f2_sub(make_float2(m_run[0], m_run[1]), mn), l2e);
  alpha[0] = live0 ? fast_exp2(da.x) : 1.0f;
  alpha[1] = live1 ? fast_exp2(da.y) : 1.0f;
  rescale |= (alpha[0] != 1.0f) | (alpha[1] != 1.0f);
  m_run[0] = mnew[0];
  m_run[1] = mnew[1];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2 d0 = f2_mul(f2_sub(make_float2(s0[2 * k], s0[2 * k + 1]), mn), l2e);
    const float2 d1 = f2_mul(f2_sub(make_float2(s1[2 * k], s1[2 * k + 1]), mn), l2e);
    s0[2 * k] = live0 ? fast_exp2(d0.x) : 0.0f;
    s0[2 * k + 1] = live1 ? fast_exp2(d0.y) : 0.0f;
    s1[2 * k] = live0 ? fast_exp2(d1.x) : 0.0f;
    s1[2 * k + 1] = live1 ? fast_exp2(d1.y) : 0.0f;
  }
  const float2 sum = f2_add(f2_add(make_float2(s0[0], s0[1]), make_float2(s0[2], s0[3])),
                            f2_add(make_float2(s1[0], s1[1]), make_float2(s1[2], s1[3])));
  const float2 l = f2_fma(make_float2(l_run[0], l_run[1]), make_float2(alpha[0], alpha[1]), sum);
  l_run[0] = l.x;
  l_run[1] = l.y;
}

// out = o_0 / l_0 - lam * (o_1 / l_1), each operation rounded on its own, here and
// in the merge alike.
__device__ __forceinline__ float diff_out(float o0, float l0, float o1, float l1, float lam) {
  return __fsub_rn(__fdiv_rn(o0, l0), __fmul_rn(lam, __fdiv_rn(o1, l1)));
}

template <int T>
__global__ void __launch_bounds__(kWarps * 32, T == 1 ? 3 : 2)
diff_split_kernel(const DiffParams p, const __grid_constant__ TmaMaps maps) {
  using Smem = DiffSmem<T>;
  constexpr int kStages = Smem::kStages;
  constexpr int kRows = T * 8;
  constexpr int kUnitRows = T == 1 ? 4 : 8;       // rows of each map in a unit
  extern __shared__ unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int M = p.M, R = p.R, H = p.Hq / 2;
  const int nrg = (R + kUnitRows - 1) / kUnitRows;
  uint64_t* full = sm.full[warp];
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }

  // ---- units of the sequences before each group of gs sequences
  const int gs = (p.B + kMaxGroups - 1) / kMaxGroups;
  const int ng = (p.B + gs - 1) / gs;
  const int per_win = p.pairs * nrg;
  auto units_of = [&](int b) -> int {
    const int ctx = p.ctx_len[b];
    return diff_valid(p, b, ctx) ? diff_windows(ctx + M - 1) * per_win : 0;
  };
  for (int i = tid; i < kMaxGroups; i += kWarps * 32) {
    int n = 0;
    if (i < ng)
      for (int b = i * gs; b < min(p.B, i * gs + gs); ++b) n += units_of(b);
    sm.prefix[i] = n;
  }
  __syncthreads();
  {
    constexpr int kPer = kMaxGroups / (kWarps * 32);
    int n[kPer], run = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      n[i] = sm.prefix[tid * kPer + i];
      run += n[i];
    }
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sm.warp_total[warp] = incl;
    __syncthreads();
    int base = incl - run;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (w < warp) base += sm.warp_total[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      sm.prefix[tid * kPer + i] = base;
      base += n[i];
    }
    if (tid == kWarps * 32 - 1) sm.prefix[kMaxGroups] = base;
  }
  // ---- the rows of sequences that break the rules
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (diff_valid(p, b, p.ctx_len[b])) continue;
    float* o = p.out + (int64_t)b * M * H * 2 * kD;
    for (int64_t i = tid; i < (int64_t)M * H * 2 * kD; i += kWarps * 32)
      o[i] = __int_as_float(0x7fc00000);
    if (tid == 0) atomicOr(p.err_word, KATTN_DEVERR_BAD_SEQUENCE);
  }
  __syncthreads();
  griddep_launch_dependents();
  const int total = sm.prefix[kMaxGroups];
  const int G = gridDim.x * kWarps;
  int t = warp * gridDim.x + blockIdx.x;          // neighbouring units on different SMs
  if (t >= total) return;

  auto find = [&](int u) -> DiffItem {
    DiffItem it{-1, 0, 0, 0, 0, 0};
    if (u >= total) return it;
    int lo = 0, hi = ng;                          // prefix[lo] <= u < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sm.prefix[mid] <= u) lo = mid;
      else hi = mid;
    }
    int r = u - sm.prefix[lo], b = lo * gs;
    if (gs > 1)
      for (int n; r >= (n = units_of(b)); ++b) r -= n;
    it.b = b;
    it.w = r / per_win;
    r -= it.w * per_win;
    it.pair = r / nrg;
    it.rg = r - it.pair * nrg;
    it.ctx = p.ctx_len[b];
    it.row0 = p.block_table ? 0 : (int)p.row_start[b];
    return it;
  };
  auto blocks_of = [&](const DiffItem& it) -> int {
    const int n = min(kWindow, it.ctx + M - 1 - it.w * kWindow);
    return (n + kBlockBk - 1) / kBlockBk;
  };

  DiffItem it0 = find(t), it1 = find(t + G);
  int row0 = block_row(p, it0, lane), row1 = block_row(p, it1, lane);

  // ---- producer: lane 0 issues, every lane keeps the same counters.  Stages
  // go K, V, K, V, ... over this item's blocks, then the next item's.
  int pnext = 0, pblk = 0, pv = 0, ist = 0, inflight = 0;
  int pn = blocks_of(it0);
  const uint64_t policy = nrg > 1 ? l2_evict_normal() : l2_evict_first();
  auto produce = [&]() {
    while (inflight < kStages) {
      if (pblk >= pn) {
        if (pnext || it1.b < 0) break;
        pnext = 1;
        pblk = 0;
        pn = blocks_of(it1);
      }
      const int pair = pnext ? it1.pair : it0.pair;
      const int row = __shfl_sync(0xffffffffu, pnext ? row1 : row0, pblk) + 2 * pair * p.cap_rows;
      if (lane == 0) {
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        mbar_expect_tx(&full[ist], kStageBytes);
        const CUtensorMap* map = pv ? &maps.v : &maps.k;
        tma_load_block(sm.ring[warp][ist], map, row, &full[ist], policy);
        tma_load_block(sm.ring[warp][ist] + kBlockBytes, map, row + p.cap_rows, &full[ist], policy);
      }
      pblk += pv;
      pv ^= 1;
      ++inflight;
      ist = ist + 1 == kStages ? 0 : ist + 1;
    }
  };
  int cst = 0;
  uint32_t cph = 0;
  auto consumed = [&]() {
    __syncwarp();
    --inflight;
    if (++cst == kStages) {
      cst = 0;
      cph ^= 1u;
    }
    produce();
  };
  produce();

  for (;;) {
    const int ctx = it0.ctx, s0 = it0.w * kWindow, s1 = min(s0 + kWindow, ctx + M - 1);
    const int64_t plane = (int64_t)2 * it0.pair * p.cap_rows;
    const float* ksp = p.k_scale + plane;
    const float* vsp = p.v_scale + plane;
    // scales of the window: the values of block 0, and the largest v_scale of
    // each plane over the keys that every row sees
    float nx[4], vm[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < kWinBlocks; ++e) {
      const int row = __shfl_sync(0xffffffffu, row0, e) + lane, key = s0 + 32 * e + lane;
      if (key < s1) {
        const float a = __ldg(vsp + row), b = __ldg(vsp + p.cap_rows + row);
        if (key < ctx) {
          vm[0] = fmaxf(vm[0], a);
          vm[1] = fmaxf(vm[1], b);
        }
        if (e == 0) {
          nx[2] = a;
          nx[3] = b;
        }
      } else if (e == 0) {
        nx[2] = nx[3] = 0.0f;
      }
      if (e == 0) {
        nx[0] = key < s1 ? __ldg(ksp + row) : 0.0f;
        nx[1] = key < s1 ? __ldg(ksp + p.cap_rows + row) : 0.0f;
      }
    }
    // ---- the unit's queries, quantized per row
    __syncwarp();
#pragma unroll 4
    for (int r = 0; r < kRows; ++r) {
      const int a = T == 1 ? r >> 2 : r >> 3;
      const int rr = it0.rg * kUnitRows + (T == 1 ? r & 3 : r & 7);
      uint32_t w = 0;
      float s = 0.0f;
      if (rr < R) {
        const int j = rr / p.g, head = 2 * (it0.pair * p.g + rr % p.g) + a;
        w = warp_quantize_row(p.q + (((int64_t)it0.b * M + j) * p.Hq + head) * kD, &s);
      }
      *reinterpret_cast<uint32_t*>(&sm.q[warp][r * kQStride + 4 * lane]) = w;
      if (lane == 0) sm.qs[warp][r] = s;
    }
    __syncwarp();
    uint32_t qw[T][8];
    float qsr[T][2];
#pragma unroll
    for (int n = 0; n < T; ++n) {
      const uint4* src = reinterpret_cast<const uint4*>(&sm.q[warp][(n * 8 + g) * kQStride + 32 * c]);
      const uint4 lo = src[0], hi = src[1];
      qw[n][0] = lo.x; qw[n][1] = lo.y; qw[n][2] = lo.z; qw[n][3] = lo.w;
      qw[n][4] = hi.x; qw[n][5] = hi.y; qw[n][6] = hi.z; qw[n][7] = hi.w;
      qsr[n][0] = sm.qs[warp][n * 8 + 2 * c];
      qsr[n][1] = sm.qs[warp][n * 8 + 2 * c + 1];
    }
    // Draft column of tile rows 2c + e; the rows of both maps share it.
    int L[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = it0.rg * kUnitRows + (T == 1 ? (2 * c + e) & 3 : 2 * c + e);
      L[e] = ctx + min(rr / p.g, M - 1);
    }
    // Power of two 2^E per plane and row: the largest v_scale among the window's
    // keys that the row sees, times 2^E, lies in [2^14, 2^15), so that a = p *
    // v_scale * 2^E stays in f16's normal range down to weights that do not
    // matter.  upb: of row g (the operand's row); down: 2^-E of rows 2c + e.
    float upb[2], down[2][2];
    {
      float vmax[2][2];
#pragma unroll
      for (int pl = 0; pl < 2; ++pl) vmax[pl][0] = vmax[pl][1] = warp_max(vm[pl]);
      for (int key = max(ctx, s0); key < s1; ++key) {    // draft keys
        const int row = __shfl_sync(0xffffffffu, row0, (key - s0) >> 5) + ((key - s0) & 31);
#pragma unroll
        for (int pl = 0; pl < 2; ++pl) {
          const float v = __ldg(vsp + pl * (int64_t)p.cap_rows + row);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (key < L[e]) vmax[pl][e] = fmaxf(vmax[pl][e], v);
        }
      }
#pragma unroll
      for (int pl = 0; pl < 2; ++pl) {
        float up[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int bexp = min(max(268 - (int)((__float_as_uint(vmax[pl][e]) >> 23) & 0xffu), 1), 253);
          up[e] = __uint_as_float((uint32_t)bexp << 23);
          down[pl][e] = __uint_as_float((uint32_t)(254 - bexp) << 23);
        }
        const float u0 = __shfl_sync(0xffffffffu, up[0], g >> 1);
        const float u1 = __shfl_sync(0xffffffffu, up[1], g >> 1);
        upb[pl] = (g & 1) ? u1 : u0;
      }
    }

    float m_run[T][2], l_run[T][2];
    float o[2][8][T][4];                          // [plane][m-tile][tile]
#pragma unroll
    for (int n = 0; n < T; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_run[n][e] = -INFINITY;
        l_run[n][e] = 0.0f;
      }
#pragma unroll
    for (int pl = 0; pl < 2; ++pl)
#pragma unroll
      for (int md = 0; md < 8; ++md)
#pragma unroll
        for (int n = 0; n < T; ++n)
#pragma unroll
          for (int u = 0; u < 4; ++u) o[pl][md][n][u] = 0.0f;

    const int nb = blocks_of(it0);
    bool failed = false;
    for (int i = 0; i < nb; ++i) {
      const int t0 = s0 + i * kBlockBk;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) sm.scale[warp][k][lane] = nx[k];
      {
        const int row = __shfl_sync(0xffffffffu, row0, min(i + 1, kWinBlocks - 1)) + lane;
        const bool in = i + 1 < nb && t0 + kBlockBk + lane < s1;
        nx[0] = in ? __ldg(ksp + row) : 0.0f;
        nx[1] = in ? __ldg(ksp + p.cap_rows + row) : 0.0f;
        nx[2] = in ? __ldg(vsp + row) : 0.0f;
        nx[3] = in ? __ldg(vsp + p.cap_rows + row) : 0.0f;
      }
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[cst], cph))) {
        failed = true;
        break;
      }
      // ---- scores of both maps: sc[tile][half], keys 16 half + g (+ 8), rows 2c + e
      float sc[T][2][4];
      {
        const uint8_t* Kt = sm.ring[warp][cst];
        int acc[T][2][4];
#pragma unroll
        for (int n = 0; n < T; ++n)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[n][hf][u] = 0;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int ra = 16 * hf + g, rb = ra + 8;
            const uint8_t* B = Kt + a * kBlockBytes;
            const uint4 a_lo = lds128(B + swz(ra, 2 * c)), a_hi = lds128(B + swz(ra, 2 * c + 1));
            const uint4 b_lo = lds128(B + swz(rb, 2 * c)), b_hi = lds128(B + swz(rb, 2 * c + 1));
            const uint32_t wa[8] = {a_lo.x, a_lo.y, a_lo.z, a_lo.w, a_hi.x, a_hi.y, a_hi.z, a_hi.w};
            const uint32_t wb[8] = {b_lo.x, b_lo.y, b_lo.z, b_lo.w, b_hi.x, b_hi.y, b_hi.z, b_hi.w};
            // T = 1: the rows of the other map are zero, so both planes add up in one tile
            const bool mine = T == 2 || (g >> 2) == a;
            constexpr int kTile1 = T - 1;
            const int n = T == 1 ? 0 : a;
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_i8(acc[T == 1 ? 0 : (a ? kTile1 : 0)][hf], wa[2 * s], wb[2 * s], wa[2 * s + 1],
                     wb[2 * s + 1], mine ? qw[n][2 * s] : 0u, mine ? qw[n][2 * s + 1] : 0u);
          }
        consumed();
        // s = (S * (qs * ks)) * sm_scale; a tile row's map picks the plane of ks
#pragma unroll
        for (int n = 0; n < T; ++n) {
          const float* kss = sm.scale[warp][T == 1 ? c >> 1 : n];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
              const float ks = kss[16 * hf + 8 * k2 + g];
              const float2 qk = f2_mul(make_float2(qsr[n][0], qsr[n][1]), make_float2(ks, ks));
              float2 s2 = f2_mul(make_float2(__int2float_rn(acc[n][hf][2 * k2]),
                                             __int2float_rn(acc[n][hf][2 * k2 + 1])), qk);
              s2 = f2_mul(s2, make_float2(p.sm_scale, p.sm_scale));
              sc[n][hf][2 * k2] = s2.x;
              sc[n][hf][2 * k2 + 1] = s2.y;
            }
        }
      }
      if (t0 + kBlockBk > ctx) {                  // keys that some row does not see
#pragma unroll
        for (int n = 0; n < T; ++n)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (t0 + 16 * hf + g + 8 * (u >> 1) >= L[u & 1]) sc[n][hf][u] = -INFINITY;
      }
      float alpha[T][2];
      bool rescale = false;
#pragma unroll
      for (int n = 0; n < T; ++n)
        diff_softmax(sc[n][0], sc[n][1], m_run[n], l_run[n], alpha[n], rescale);
      if (rescale) {
#pragma unroll
        for (int pl = 0; pl < 2; ++pl)
#pragma unroll
          for (int md = 0; md < 8; ++md)
#pragma unroll
            for (int n = 0; n < T; ++n) {
              const float2 a2 = make_float2(alpha[n][0], alpha[n][1]);
              const float2 lo = f2_mul(make_float2(o[pl][md][n][0], o[pl][md][n][1]), a2);
              const float2 hi = f2_mul(make_float2(o[pl][md][n][2], o[pl][md][n][3]), a2);
              o[pl][md][n][0] = lo.x; o[pl][md][n][1] = lo.y;
              o[pl][md][n][2] = hi.x; o[pl][md][n][3] = hi.y;
            }
      }
      // ---- the weights in the operand's layout: keys 2c, 2c+1, 2c+8, 2c+9 of the
      // half, row g
      float pb[T][2][4];
#pragma unroll
      for (int n = 0; n < T; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int srcA = 8 * c + (g >> 1), srcB = srcA + 4;
          float fA[4], fB[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            fA[u] = __shfl_sync(0xffffffffu, sc[n][hf][u], srcA);
            fB[u] = __shfl_sync(0xffffffffu, sc[n][hf][u], srcB);
          }
          const bool odd = g & 1;
          pb[n][hf][0] = odd ? fA[1] : fA[0];
          pb[n][hf][1] = odd ? fB[1] : fB[0];
          pb[n][hf][2] = odd ? fA[3] : fA[2];
          pb[n][hf][3] = odd ? fB[3] : fB[2];
        }
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[cst], cph))) {
        failed = true;
        break;
      }
      // ---- P.V: the operand a = p * v_scale * 2^E as f16 hi + lo (22 bits), V exact
#pragma unroll
      for (int pl = 0; pl < 2; ++pl)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint8_t* Vt = sm.ring[warp][cst] + pl * kBlockBytes;
          const float* vss = sm.scale[warp][2 + pl] + 16 * hf + 2 * c;
          const float2 v0 = *reinterpret_cast<const float2*>(vss);
          const float2 v1 = *reinterpret_cast<const float2*>(vss + 8);
          const float2 up2 = make_float2(upb[pl], upb[pl]);
          uint2 bhi[T], blo[T];
#pragma unroll
          for (int n = 0; n < T; ++n) {
            const float2 x = f2_mul(f2_mul(make_float2(pb[n][hf][0], pb[n][hf][1]), v0), up2);
            const float2 y = f2_mul(f2_mul(make_float2(pb[n][hf][2], pb[n][hf][3]), v1), up2);
            split_f16x2(x.x, x.y, bhi[n].x, blo[n].x);
            split_f16x2(y.x, y.y, bhi[n].y, blo[n].y);
          }
          const int kr = 16 * hf + 2 * c;
          const uint4 vw0 = lds128(Vt + swz(kr, g)), vw1 = lds128(Vt + swz(kr + 1, g));
          const uint4 vw2 = lds128(Vt + swz(kr + 8, g)), vw3 = lds128(Vt + swz(kr + 9, g));
          const uint32_t w0[4] = {vw0.x, vw0.y, vw0.z, vw0.w}, w1[4] = {vw1.x, vw1.y, vw1.z, vw1.w};
          const uint32_t w2[4] = {vw2.x, vw2.y, vw2.z, vw2.w}, w3[4] = {vw3.x, vw3.y, vw3.z, vw3.w};
#pragma unroll
          for (int md = 0; md < 8; ++md) {
            const int wi = md >> 1;
            const uint32_t sel = (md & 1) ? 0x7362u : 0x5140u;
            const uint32_t t01 = __byte_perm(w0[wi], w1[wi], sel) ^ 0x80808080u;
            const uint32_t t23 = __byte_perm(w2[wi], w3[wi], sel) ^ 0x80808080u;
            const uint32_t af[4] = {i8pair_to_h2(t01, 0x4140u), i8pair_to_h2(t01, 0x4342u),
                                    i8pair_to_h2(t23, 0x4140u), i8pair_to_h2(t23, 0x4342u)};
#pragma unroll
            for (int n = 0; n < T; ++n) {
              mma_f16(o[pl][md][n], af, bhi[n]);
              mma_f16(o[pl][md][n], af, blo[n]);
            }
          }
        }
      consumed();
    }
    if (failed) {
      // A copy never arrived: flag it, give the copies in flight a bounded chance
      // to land, then leave.
      if (lane == 0) {
        atomicOr(p.err_word, KATTN_DEVERR_TIMEOUT);
        for (int k = 0; k < inflight; ++k) {
          mbar_wait_bounded(&full[cst], cph);
          if (++cst == kStages) {
            cst = 0;
            cph ^= 1u;
          }
        }
      }
      return;
    }

    // ---- the window's result
#pragma unroll
    for (int n = 0; n < T; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l_run[n][e];
        v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 8));
        l_run[n][e] = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 16));
      }
    const bool whole = diff_windows(ctx + M - 1) == 1;
    const int b = it0.b, pair = it0.pair;
    if (whole) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = it0.rg * kUnitRows + (T == 1 ? (2 * c + e) & 3 : 2 * c + e);
        const bool in = rr < R && (T == 2 || c < 2);
        const int j = rr / p.g, i = pair * p.g + rr % p.g;
        const int64_t row = ((int64_t)b * M + j) * H + i;
        const float lam = in ? p.lam[p.lam_per_row ? row : i] : 0.0f;
        const float l0 = l_run[0][e];
        const float l1 = T == 2 ? l_run[T - 1][e] : __shfl_xor_sync(0xffffffffu, l_run[0][e], 2);
#pragma unroll
        for (int pl = 0; pl < 2; ++pl)
#pragma unroll
          for (int md = 0; md < 8; ++md) {
            const float x0 = __fmul_rn(o[pl][md][0][e], down[pl][e]);
            const float x1 = __fmul_rn(o[pl][md][0][2 + e], down[pl][e]);
            const float y0 = T == 2 ? __fmul_rn(o[pl][md][T - 1][e], down[pl][e])
                                    : __shfl_xor_sync(0xffffffffu, x0, 2);
            const float y1 = T == 2 ? __fmul_rn(o[pl][md][T - 1][2 + e], down[pl][e])
                                    : __shfl_xor_sync(0xffffffffu, x1, 2);
            if (in)
              *reinterpret_cast<float2*>(p.out + row * 2 * kD + pl * kD + 16 * g + 2 * md) =
                  make_float2(diff_out(x0, l0, y0, l1, lam), diff_out(x1, l0, y1, l1, lam));
          }
      }
    } else {
      float* part = p.partials + (((size_t)b * p.nwin_max + it0.w) * p.pairs + pair) * diff_stride(R);
#pragma unroll
      for (int n = 0; n < T; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 2 * c + e, a = T == 1 ? r >> 2 : n;
          const int rr = it0.rg * kUnitRows + (T == 1 ? r & 3 : r);
          if (rr >= R) continue;
          float* dst = part + (size_t)(a * R + rr) * 2 * kD + 16 * g;
#pragma unroll
          for (int pl = 0; pl < 2; ++pl)
#pragma unroll
            for (int md = 0; md < 8; md += 2)
              *reinterpret_cast<float4*>(dst + pl * kD + 2 * md) =
                  make_float4(__fmul_rn(o[pl][md][n][e], down[pl][e]),
                              __fmul_rn(o[pl][md][n][2 + e], down[pl][e]),
                              __fmul_rn(o[pl][md + 1][n][e], down[pl][e]),
                              __fmul_rn(o[pl][md + 1][n][2 + e], down[pl][e]));
          if (g == 0) {
            part[(size_t)2 * R * 2 * kD + a * R + rr] = m_run[n][e];
            part[(size_t)2 * R * 2 * kD + 2 * R + a * R + rr] = l_run[n][e];
          }
        }
    }

    // ---- next item
    t += G;
    if (t >= total) break;
    it0 = it1;
    row0 = row1;
    it1 = find(t + G);
    row1 = block_row(p, it1, lane);
    if (pnext) {
      pnext = 0;                                  // the producer is already on this item
    } else {
      pblk = 0;                                   // it had nothing left to read ahead
      pn = blocks_of(it0);
    }
    produce();
  }
}

// Joins the windows of a row, one block per (sequence, column, head): warp k sums
// the windows k, k + 8, ... of both maps with the weights e^(m_s - max m), the
// eight sums are added in order, and the two maps are subtracted.  The order
// depends on the row's own window count alone.
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(kMergeWarps * 32, 4) diff_merge_kernel(const DiffParams p) {
  __shared__ float4 s_o[kMergeWarps][2][2 * kD / 4];
  __shared__ float s_m[kMergeWarps][2], s_l[kMergeWarps][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
  const int ctx = p.ctx_len[b], H = p.Hq / 2, R = p.R;
  griddep_wait();                                 // every partial is in place
  if (!diff_valid(p, b, ctx) || diff_windows(ctx + p.M - 1) == 1) return;
  const int ns = diff_windows(ctx + j);
  const int pair = i / p.g, rr = j * p.g + i % p.g;
  const size_t stride = (size_t)p.pairs * diff_stride(R);
  const float* base = p.partials + ((size_t)b * p.nwin_max * p.pairs + pair) * diff_stride(R);
  const float* mcol = base + (size_t)2 * R * 2 * kD + rr;
  const float* lcol = mcol + 2 * R;
  const float* ocol = base + (size_t)rr * 2 * kD + 4 * lane;
  const size_t map1 = (size_t)R * 2 * kD;
  // the row's maxima
  float mx[2] = {-INFINITY, -INFINITY};
  for (int s = threadIdx.x; s < ns; s += kMergeWarps * 32) {
    mx[0] = fmaxf(mx[0], __ldcg(mcol + s * stride));
    mx[1] = fmaxf(mx[1], __ldcg(mcol + s * stride + R));
  }
  mx[0] = warp_max(mx[0]);
  mx[1] = warp_max(mx[1]);
  if (lane == 0) {
    s_m[warp][0] = mx[0];
    s_m[warp][1] = mx[1];
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    mx[0] = fmaxf(mx[0], s_m[w][0]);
    mx[1] = fmaxf(mx[1], s_m[w][1]);
  }
  float4 acc[2][2];                               // [map][128-channel half]
  float l[2] = {0.0f, 0.0f};                      // of the windows this lane weighs
  const int nw = (ns - warp + kMergeWarps - 1) / kMergeWarps;   // windows of this warp
  for (int n0 = 0; n0 < nw; n0 += 32) {
    // lane n weighs window warp + 8 (n0 + n)
    const int s = warp + kMergeWarps * (n0 + lane);
    float w[2] = {0.0f, 0.0f};
    if (s < ns) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        w[a] = merge_weight(__ldcg(mcol + s * stride + a * R), mx[a]);
        l[a] = __fmaf_rn(w[a], __ldcg(lcol + s * stride + a * R), l[a]);
      }
    }
#pragma unroll 4
    for (int n = 0; n < min(32, nw - n0); ++n) {
      const float* src = ocol + (size_t)(warp + kMergeWarps * (n0 + n)) * stride;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const float wn = __shfl_sync(0xffffffffu, w[a], n);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(src + a * map1 + h * kD));
          if (n0 + n == 0)
            acc[a][h] = make_float4(__fmul_rn(wn, v.x), __fmul_rn(wn, v.y), __fmul_rn(wn, v.z),
                                    __fmul_rn(wn, v.w));
          else
            acc[a][h] = make_float4(__fmaf_rn(wn, v.x, acc[a][h].x), __fmaf_rn(wn, v.y, acc[a][h].y),
                                    __fmaf_rn(wn, v.z, acc[a][h].z), __fmaf_rn(wn, v.w, acc[a][h].w));
        }
      }
    }
  }
  if (nw > 0) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      s_o[warp][a][lane] = acc[a][0];
      s_o[warp][a][32 + lane] = acc[a][1];
      const float v = warp_sum(l[a]);
      if (lane == 0) s_l[warp][a] = v;
    }
  }
  __syncthreads();
  const int ch = threadIdx.x;                     // one channel per thread
  float O[2], Ls[2];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    O[a] = reinterpret_cast<const float*>(s_o[0][a])[ch];
    Ls[a] = s_l[0][a];
    for (int w = 1; w < min(ns, kMergeWarps); ++w) {
      O[a] = __fadd_rn(O[a], reinterpret_cast<const float*>(s_o[w][a])[ch]);
      Ls[a] = __fadd_rn(Ls[a], s_l[w][a]);
    }
  }
  const int64_t row = ((int64_t)b * p.M + j) * H + i;
  p.out[row * 2 * kD + ch] = diff_out(O[0], Ls[0], O[1], Ls[1], p.lam[p.lam_per_row ? row : i]);
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
cudaError_t launch_split(const DiffParams& p, const TmaMaps& maps, cudaStream_t stream) {
  const auto kern = diff_split_kernel<T>;
  const int smem = (int)sizeof(DiffSmem<T>) + 1024;     // + alignment slack
  // per device: the CTAs that the GPU holds at once; the shared-memory limit is
  // raised with the first call
  static std::atomic<int> slots_cache[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int slots = (dev >= 0 && dev < kMaxDevices) ? slots_cache[dev].load() : 0;
  if (slots <= 0) {
    int sms = 0, per_sm = 0;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) !=
        cudaSuccess)
      return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kWarps * 32, smem)) !=
        cudaSuccess)
      return e;
    slots = sms * (per_sm > 0 ? per_sm : 1);
    if (dev >= 0 && dev < kMaxDevices) slots_cache[dev].store(slots);
  }
  kern<<<(unsigned)std::min<int64_t>(diff_units(p), slots), kWarps * 32, smem, stream>>>(p, maps);
  return cudaGetLastError();
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
  const cudaError_t e = p.R <= 4 ? launch_split<1>(p, maps, stream) : launch_split<2>(p, maps, stream);
  if (e != cudaSuccess || p.nwin_max <= 1) return e;
  return launch_pdl(diff_merge_kernel, dim3((unsigned)(p.Hq / 2), (unsigned)p.M, (unsigned)p.B),
                    dim3(kMergeWarps * 32), 0, stream, p);
}

}  // namespace kattn
