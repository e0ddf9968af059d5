// The pages of a paged cache: reserving, freeing, forking, compacting, copying.
//
// reserve, fork and compact are each one cluster of kCluster blocks: the
// phases below depend on one another over the whole pool, and the barrier of a
// cluster costs a fraction of a microsecond where a second launch costs
// several.  What the blocks hand over goes through the workspace in L2.
#include <algorithm>

#include "device_common.cuh"
#include "ops_internal.cuh"

namespace kattn {
namespace {

constexpr int kCluster = 8;                       // blocks of a plan (the portable cluster size)
constexpr int kThreads = 1024;
constexpr int kWarpsPerBlock = kThreads / 32;
constexpr int kUnroll = 8;                        // pages a thread looks at per tile
constexpr int kTile = kThreads * kUnroll;
static_assert(kUnroll * kWarpsPerBlock == 256, "one counter per thread of the first 8 warps");

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return (int)r;
}

__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xffffffffu, v); }

struct BlockScratch {
  int warp[kWarpsPerBlock];
  int count[256];
  int total;
};

// Sum of v over the block, to every thread.
__device__ __forceinline__ int block_sum(int v, BlockScratch& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum_int(v);
  __syncthreads();
  if (lane == 0) s.warp[warp] = v;
  __syncthreads();
  return warp_sum_int(s.warp[lane]);
}

// Exclusive prefix of v over the block's threads; *total: the sum.
__device__ __forceinline__ int block_prefix(int v, BlockScratch& s, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();
  if (lane == 31) s.warp[warp] = incl;
  __syncthreads();
  int w = s.warp[lane];
  const int all = warp_sum_int(w);
  w = warp_sum_int(lane < warp ? w : 0);
  *total = all;
  return w + incl - v;
}

// The pages of block `rank`: [lo, hi).
struct Chunk {
  int per, lo, hi;
};
__device__ __forceinline__ Chunk chunk_of(int n_pages, int rank) {
  Chunk c;
  c.per = (n_pages + kCluster - 1) / kCluster;
  c.lo = min(n_pages, rank * c.per);
  c.hi = min(n_pages, c.lo + c.per);
  return c;
}

// Ranks of the pages of [lo, hi) for which pick(page, count) holds, in
// ascending order: put(rank, page, count) is called for each.  Returns how many
// there are (to every thread).  Per tile, each warp's ballot gives the ranks
// within 32 pages and a scan over the tile's 256 ballots those between them.
template <typename Pick, typename Put>
__device__ __forceinline__ int rank_pages(const int32_t* refs, int lo, int hi, BlockScratch& s,
                                          Pick pick, Put put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int t0 = lo; t0 < hi; t0 += kTile) {
    int c[kUnroll];
    unsigned bal[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int p = t0 + u * kThreads + (int)threadIdx.x;
      c[u] = p < hi ? __ldcg(refs + p) : 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int p = t0 + u * kThreads + (int)threadIdx.x;
      bal[u] = __ballot_sync(0xffffffffu, p < hi && pick(p, c[u]));
    }
    __syncthreads();                              // the last tile's counters are read
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (lane == 0) s.count[u * kWarpsPerBlock + warp] = __popc(bal[u]);
    __syncthreads();
    const int mine = threadIdx.x < 256 ? s.count[threadIdx.x] : 0;
    int total;
    const int before = block_prefix(mine, s, &total);
    if (threadIdx.x < 256) s.count[threadIdx.x] = before;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (bal[u] >> lane & 1u)
        put(base + s.count[u * kWarpsPerBlock + warp] + __popc(bal[u] & ((1u << lane) - 1u)),
            t0 + u * kThreads + (int)threadIdx.x, c[u]);
    base += total;
  }
  return base;
}

// Where the entry of rank k lies in a list that each block wrote from its
// chunk's start on: block c's ranks begin at the sum of the counts before it.
struct Places {
  int start[kCluster + 1];
  int per;
};
__device__ __forceinline__ Places places_of(const int* chunk, int per) {
  Places p;
  p.per = per;
  p.start[0] = 0;
#pragma unroll
  for (int c = 0; c < kCluster; ++c) p.start[c + 1] = p.start[c] + __ldcg(chunk + c);
  return p;
}
__device__ __forceinline__ int place(const Places& p, int k) {
  int at = k;
#pragma unroll
  for (int c = 1; c < kCluster; ++c)
    if (k >= p.start[c]) at = c * p.per + k - p.start[c];
  return at;
}

// One reference less on page e of a row (an entry below 0 is unused).
__device__ __forceinline__ void drop_page(const PageParams& p, int e) {
  if (e < 0) return;
  if (e >= p.n_pages) {
    atomicOr(p.ws.err, KATTN_DEVERR_BAD_PAGE);
    return;
  }
  if (atomicSub(p.refs + e, 1) <= 0) {
    atomicAdd(p.refs + e, 1);
    atomicOr(p.ws.err, KATTN_DEVERR_BAD_PAGE);
  }
}

// Rows a length covers, and whether it is one (0 <= len <= max_pages * page).
__device__ __forceinline__ bool len_ok(const PageParams& p, int len) {
  return len >= 0 && (int64_t)len <= ((int64_t)p.max_pages << p.page_shift);
}
__device__ __forceinline__ int pages_for(const PageParams& p, int len) {
  return (int)(((int64_t)len + (1 << p.page_shift) - 1) >> p.page_shift);
}

// List entries [lo, hi) of block `rank`.
__device__ __forceinline__ void list_range(int n, int rank, int& lo, int& hi) {
  const int per = (n + kCluster - 1) / kCluster;
  lo = min(n, rank * per);
  hi = min(n, lo + per);
}

// The first list entry that names a slot wins it: claim holds n - i.
__device__ __forceinline__ void claim_slots(const PageParams& p, int rank) {
  for (int i = rank * kThreads + threadIdx.x; i < p.n; i += kCluster * kThreads) {
    const int s = p.seqs[i];
    if ((unsigned)s < (unsigned)p.n_slots) atomicMax(p.ws.claim + s, p.n - i);
  }
}
__device__ __forceinline__ bool slot_mine(const PageParams& p, int i, int s) {
  return (unsigned)s < (unsigned)p.n_slots && __ldcg(p.ws.claim + s) == p.n - i;
}

// ---------------------------------------------------------------- reserve
//   1. claims;  2. per list entry the missing pages (one warp each), and the
//   free pages of the block's chunk in order;  3. the entries' first ranks (a
//   scan over the list) and the pages of those ranks into the table.
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
reserve_kernel(const PageParams p) {
  __shared__ BlockScratch s;
  __shared__ int first[kThreads];
  const int rank = cluster_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  claim_slots(p, rank);
  cluster_sync();
  int lo, hi;
  list_range(p.n, rank, lo, hi);
  for (int i = lo + warp; i < hi; i += kWarpsPerBlock) {
    const int slot = p.seqs[i], len = p.lens[i];
    int miss = 0;
    if (slot_mine(p, i, slot) && len_ok(p, len)) {
      const int need = pages_for(p, len);
      const int32_t* row = p.table + (int64_t)slot * p.max_pages;
      for (int c = lane; c < need; c += 32) miss += __ldcg(row + c) < 0;
      miss = warp_sum_int(miss);
    } else if (lane == 0) {
      atomicOr(p.ws.err, KATTN_DEVERR_BAD_SEQUENCE);
    }
    if (lane == 0) p.ws.flag[i] = miss;
  }
  const Chunk ch = chunk_of(p.n_pages, rank);
  int* list = p.ws.list + ch.lo;
  const int free_here = rank_pages(
      p.refs, ch.lo, ch.hi, s, [](int, int c) { return c == 0; },
      [&](int r, int page, int) { list[r] = page; });
  if (threadIdx.x == 0) p.ws.chunk[rank] = free_here;
  cluster_sync();
  const Places pl = places_of(p.ws.chunk, ch.per);
  // pages wanted before this block's entries, and by the whole list
  int64_t before = 0, all = 0;
  for (int i = threadIdx.x; i < p.n; i += kThreads) {
    const int m = __ldcg(p.ws.flag + i);
    all += m;
    if (i < lo) before += m;
  }
  // (a list wants at most what the pool holds, or it gets nothing: the sums are
  // compared in 64 bits, capped well above any pool)
  const int cap = 1 << 20;
  const int all_hi = block_sum((int)(all >> 20), s), all_lo = block_sum((int)(all & (cap - 1)), s);
  const int bef_hi = block_sum((int)(before >> 20), s), bef_lo = block_sum((int)(before & (cap - 1)), s);
  const int64_t want = (int64_t)all_hi * cap + all_lo;
  const bool enough = want <= (int64_t)pl.start[kCluster];
  if (!enough && rank == 0 && threadIdx.x == 0) atomicOr(p.ws.err, KATTN_DEVERR_NO_PAGES);
  if (enough) {
    int base = (int)((int64_t)bef_hi * cap + bef_lo);
    for (int i0 = lo; i0 < hi; i0 += kThreads) {
      const int i = i0 + threadIdx.x;
      int total;
      const int mine = block_prefix(i < hi ? __ldcg(p.ws.flag + i) : 0, s, &total);
      __syncthreads();
      first[threadIdx.x] = base + mine;
      __syncthreads();
      for (int k = warp; k < min(kThreads, hi - i0); k += kWarpsPerBlock) {
        const int slot = p.seqs[i0 + k];
        if (__ldcg(p.ws.flag + i0 + k) == 0) continue;
        const int need = pages_for(p, p.lens[i0 + k]);
        int32_t* row = p.table + (int64_t)slot * p.max_pages;
        int at = first[k];
        for (int c0 = 0; c0 < need; c0 += 32) {
          const int c = c0 + lane;
          const bool miss = c < need && __ldcg(row + c) < 0;
          const unsigned bal = __ballot_sync(0xffffffffu, miss);
          if (miss) {
            const int page = __ldcg(p.ws.list + place(pl, at + __popc(bal & ((1u << lane) - 1u))));
            row[c] = page;
            p.refs[page] = 1;
          }
          at += __popc(bal);
        }
      }
      base += total;
    }
  }
  // the claims go back to zero for the next call
  for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
    const int slot = p.seqs[i];
    if ((unsigned)slot < (unsigned)p.n_slots) p.ws.claim[slot] = 0;
  }
}

// ------------------------------------------------------------------- free
// One block per list entry.  The exchange takes an entry out of the table once,
// so a slot named twice loses its pages once.
__global__ void __launch_bounds__(256) free_kernel(const PageParams p) {
  const int slot = p.seqs[blockIdx.x];
  if ((unsigned)slot >= (unsigned)p.n_slots) {
    if (threadIdx.x == 0) atomicOr(p.ws.err, KATTN_DEVERR_BAD_SEQUENCE);
    return;
  }
  int32_t* row = p.table + (int64_t)slot * p.max_pages;
  for (int c = threadIdx.x; c < p.max_pages; c += blockDim.x) {
    if (__ldcg(row + c) == -1) continue;
    drop_page(p, atomicExch(row + c, -1));
  }
}

// ------------------------------------------------------------------- fork
//   1. claims of the children, marks of the parents;  2. per pair (one warp
//   each) the checks, and the release of what a valid child held;  3. the free
//   pages in order;  4. the ranks of the pairs that need a page of their own,
//   and the children's rows.
// flag: 0 skipped, 1 valid, 2 valid with a page of its own.
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
fork_kernel(const PageParams p) {
  __shared__ BlockScratch s;
  __shared__ int first[kThreads];
  const int rank = cluster_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  claim_slots(p, rank);
  for (int i = rank * kThreads + threadIdx.x; i < p.n; i += kCluster * kThreads) {
    const int s2 = p.parents[i];
    if ((unsigned)s2 < (unsigned)p.n_slots) p.ws.mark[s2] = 1;
  }
  cluster_sync();
  int lo, hi;
  list_range(p.n, rank, lo, hi);
  const int page_mask = (1 << p.page_shift) - 1;
  for (int i = lo + warp; i < hi; i += kWarpsPerBlock) {
    const int child = p.seqs[i], parent = p.parents[i], len = p.lens[i];
    bool ok = slot_mine(p, i, child) && (unsigned)parent < (unsigned)p.n_slots && len_ok(p, len);
    if (ok) ok = __ldcg(p.ws.mark + child) == 0;
    unsigned err = ok ? 0u : KATTN_DEVERR_BAD_SEQUENCE;
    if (ok) {
      const int need = pages_for(p, len);
      const int32_t* row = p.table + (int64_t)parent * p.max_pages;
      bool absent = false, outside = false;
      for (int c = lane; c < need; c += 32) {
        const int e = __ldcg(row + c);
        absent |= e < 0;
        outside |= e >= p.n_pages;
      }
      if (__any_sync(0xffffffffu, absent)) err |= KATTN_DEVERR_BAD_SEQUENCE;
      if (__any_sync(0xffffffffu, outside)) err |= KATTN_DEVERR_BAD_PAGE;
      ok = err == 0;
    }
    if (ok) {
      const int32_t* row = p.table + (int64_t)child * p.max_pages;
      for (int c = lane; c < p.max_pages; c += 32) drop_page(p, __ldcg(row + c));
    } else if (lane == 0) {
      atomicOr(p.ws.err, err);
    }
    if (lane == 0) p.ws.flag[i] = !ok ? 0 : (len & page_mask) ? 2 : 1;
  }
  cluster_sync();
  const Chunk ch = chunk_of(p.n_pages, rank);
  int* list = p.ws.list + ch.lo;
  const int free_here = rank_pages(
      p.refs, ch.lo, ch.hi, s, [](int, int c) { return c == 0; },
      [&](int r, int page, int) { list[r] = page; });
  if (threadIdx.x == 0) p.ws.chunk[rank] = free_here;
  cluster_sync();
  const Places pl = places_of(p.ws.chunk, ch.per);
  const int supply = pl.start[kCluster];
  int before = 0;
  for (int i = threadIdx.x; i < lo; i += kThreads) before += __ldcg(p.ws.flag + i) == 2;
  int base = block_sum(before, s);
  for (int i0 = lo; i0 < hi; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    int total;
    const int mine = block_prefix(i < hi && __ldcg(p.ws.flag + i) == 2 ? 1 : 0, s, &total);
    __syncthreads();
    first[threadIdx.x] = base + mine;
    __syncthreads();
    for (int k = warp; k < min(kThreads, hi - i0); k += kWarpsPerBlock) {
      const int flag = __ldcg(p.ws.flag + i0 + k);
      int from = -1, to = -1;
      if (flag != 0) {
        const int child = p.seqs[i0 + k], parent = p.parents[i0 + k], len = p.lens[i0 + k];
        int full = len >> p.page_shift;
        int32_t* row = p.table + (int64_t)child * p.max_pages;
        const int32_t* src = p.table + (int64_t)parent * p.max_pages;
        if (flag == 2) {
          if (first[k] < supply) {
            from = __ldcg(src + full);
            to = __ldcg(p.ws.list + place(pl, first[k]));
            if (lane == 0) p.refs[to] = 1;
          } else {                                // no page left: the child stays empty
            if (lane == 0) atomicOr(p.ws.err, KATTN_DEVERR_NO_PAGES);
            full = 0;
          }
        }
        for (int c = lane; c < p.max_pages; c += 32) {
          int e = -1;
          if (c < full) {
            e = __ldcg(src + c);
            atomicAdd(p.refs + e, 1);
          } else if (c == full && to >= 0) {
            e = to;
          }
          row[c] = e;
        }
      }
      if (lane == 0) {
        p.src[i0 + k] = from;
        p.dst[i0 + k] = to;
      }
    }
    base += total;
  }
  for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
    const int child = p.seqs[i], parent = p.parents[i];
    if ((unsigned)child < (unsigned)p.n_slots) p.ws.claim[child] = 0;
    if ((unsigned)parent < (unsigned)p.n_slots) p.ws.mark[parent] = 0;
  }
}

// ---------------------------------------------------------------- compact
//   1. live pages per chunk;  2. with their sum n_live, the free pages below it
//   and the live pages at or above it, in order;  3. the moves, the counts
//   after them, and the map of the pages that move.  rewrite_kernel then takes
//   the table through the map.
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
compact_kernel(const PageParams p) {
  __shared__ BlockScratch s;
  const int rank = cluster_rank();
  const Chunk ch = chunk_of(p.n_pages, rank);
  int live = 0;
  for (int t0 = ch.lo; t0 < ch.hi; t0 += kTile) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int at = t0 + u * kThreads + (int)threadIdx.x;
      live += at < ch.hi && __ldcg(p.refs + at) > 0;
    }
  }
  live = block_sum(live, s);
  if (threadIdx.x == 0) p.ws.chunk[rank] = live;
  cluster_sync();
  int n_live = 0;
#pragma unroll
  for (int c = 0; c < kCluster; ++c) n_live += __ldcg(p.ws.chunk + c);
  int* holes = p.ws.list + ch.lo;
  int2* movers = p.ws.list2 + ch.lo;
  const int n_holes = rank_pages(
      p.refs, ch.lo, min(ch.hi, n_live), s, [](int, int c) { return c <= 0; },
      [&](int r, int page, int) { holes[r] = page; });
  const int n_movers = rank_pages(
      p.refs, max(ch.lo, n_live), ch.hi, s,
      [&](int page, int c) {
        if (c <= 0) p.ws.to[page] = -1;           // no table entry may name it
        return c > 0;
      },
      [&](int r, int page, int c) { movers[r] = make_int2(page, c); });
  if (threadIdx.x == 0) {
    p.ws.chunk[kCluster + rank] = n_holes;
    p.ws.chunk[2 * kCluster + rank] = n_movers;
  }
  cluster_sync();
  const Places ph = places_of(p.ws.chunk + kCluster, ch.per);
  const Places pm = places_of(p.ws.chunk + 2 * kCluster, ch.per);
  const int moves = pm.start[kCluster];           // as many as holes
  const int slots = max(1, p.n_pages / 2);
  for (int k = rank * kThreads + threadIdx.x; k < slots; k += kCluster * kThreads) {
    int from = -1, to = -1;
    if (k < moves) {
      const int2 m = __ldcg(p.ws.list2 + place(pm, k));
      from = m.x;
      to = __ldcg(p.ws.list + place(ph, k));
      p.ws.to[from] = to;
      p.ref_out[to] = m.y;
    }
    p.src[k] = from;
    p.dst[k] = to;
  }
  // the other counts: a live page below n_live keeps its own, none is left above
  for (int at = max(ch.lo, n_live) + threadIdx.x; at < ch.hi; at += kThreads) p.ref_out[at] = 0;
  if (p.ref_out != p.refs)
    for (int at = ch.lo + threadIdx.x; at < min(ch.hi, n_live); at += kThreads) {
      const int c = __ldcg(p.refs + at);
      if (c > 0) p.ref_out[at] = c;
    }
  if (rank == 0 && threadIdx.x == 0) {
    p.counts[0] = n_live;
    p.counts[1] = moves;
  }
}


__global__ void __launch_bounds__(256) rewrite_kernel(const PageParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");   // the moves
  const int n_live = __ldcg(p.counts);
  const int64_t all = (int64_t)p.n_slots * p.max_pages;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all;
       i += (int64_t)gridDim.x * blockDim.x) {
    int e = p.table[i];
    if (e >= n_live) {
      const int to = e < p.n_pages ? __ldcg(p.ws.to + e) : -1;
      if (to < 0) atomicOr(p.ws.err, KATTN_DEVERR_BAD_PAGE);
      else e = to;
    }
    p.table_out[i] = e;
  }
}

// ------------------------------------------------------------------- copy
// One block per (list entry, plane, K or V), in a grid stride.
__global__ void __launch_bounds__(256) copy_kernel(const CopyParams p) {
  const int n = p.count ? min(p.n, max(0, *p.count)) : p.n;
  const int64_t units = (int64_t)n * p.Hkv * 2;
  const int vecs = p.page_rows * kD / 16;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int which = (int)(u & 1);
    const int64_t ih = u >> 1;
    const int i = (int)(ih / p.Hkv), h = (int)(ih - (int64_t)i * p.Hkv);
    const int from = p.src[i], to = p.dst[i];
    if (from < 0 || to < 0) continue;
    if (from >= p.n_pages || to >= p.n_pages) {
      if (threadIdx.x == 0) atomicOr(p.err, KATTN_DEVERR_BAD_PAGE);
      continue;
    }
    const int64_t plane = (int64_t)h * p.cap_rows;
    const int64_t a = plane + (int64_t)from * p.page_rows, b = plane + (int64_t)to * p.page_rows;
    int8_t* x = which ? p.v : p.k;
    float* y = which ? p.v_scale : p.k_scale;
    const uint4* xs = reinterpret_cast<const uint4*>(x + a * kD);
    uint4* xd = reinterpret_cast<uint4*>(x + b * kD);
    for (int c = threadIdx.x; c < vecs; c += blockDim.x) xd[c] = xs[c];
    for (int c = threadIdx.x; c < p.page_rows; c += blockDim.x) y[b + c] = y[a + c];
  }
}

struct PageLayout {
  size_t claim, mark, flag, chunk, list, to, list2, total;
};
PageLayout page_layout(int n_slots, int n_pages) {
  PageLayout w{};
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t s = up((size_t)n_slots * sizeof(int)), g = up((size_t)n_pages * sizeof(int));
  w.claim = 256;
  w.mark = w.claim + s;
  w.flag = w.mark + s;
  w.chunk = w.flag + s;
  w.list = w.chunk + 256;
  w.to = w.list + g;
  w.list2 = w.to + g;
  w.total = w.list2 + 2 * g;
  return w;
}

}  // namespace

size_t page_workspace_bytes(int n_slots, int n_pages) { return page_layout(n_slots, n_pages).total; }

void set_page_workspace(PageParams& p, void* workspace) {
  const PageLayout w = page_layout(p.n_slots, p.n_pages);
  char* ws = static_cast<char*>(workspace);
  p.ws.err = reinterpret_cast<uint32_t*>(ws);
  p.ws.claim = reinterpret_cast<int*>(ws + w.claim);
  p.ws.mark = reinterpret_cast<int*>(ws + w.mark);
  p.ws.flag = reinterpret_cast<int*>(ws + w.flag);
  p.ws.chunk = reinterpret_cast<int*>(ws + w.chunk);
  p.ws.list = reinterpret_cast<int*>(ws + w.list);
  p.ws.to = reinterpret_cast<int*>(ws + w.to);
  p.ws.list2 = reinterpret_cast<int2*>(ws + w.list2);
}

cudaError_t launch_reserve_pages(const PageParams& p, cudaStream_t stream) {
  reserve_kernel<<<kCluster, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_free_sequences(const PageParams& p, cudaStream_t stream) {
  free_kernel<<<(unsigned)p.n, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_fork_sequences(const PageParams& p, cudaStream_t stream) {
  fork_kernel<<<kCluster, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_compact_pages(const PageParams& p, cudaStream_t stream) {
  compact_kernel<<<kCluster, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t all = (int64_t)p.n_slots * p.max_pages;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((all + 255) / 256, 152 * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rewrite_kernel, p);
}

cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t stream) {
  const int64_t units = (int64_t)p.n * p.Hkv * 2;
  copy_kernel<<<(unsigned)std::min<int64_t>(units, 152 * 8), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kattn
