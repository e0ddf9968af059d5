// The pages of a paged cache: reserving, freeing, forking, compacting, copying.
//
// reserve, fork and compact each plan over the whole pool in phases that depend on
// one another.  A small pool is planned by one block; a large one by a cluster of
// kCluster blocks, whose barrier costs a fraction of a microsecond where another
// launch costs several.  What the blocks hand over goes through the workspace in
// L2.  Bound by latency: a phase is one or two dependent trips to L2.  Measured:
// reserving for 8 slots of a 4096-page pool 5.9 us, for 512 slots of a 262144-page
// pool (65k pages taken) 14.5 us; 8 forks 6.5 us, 512 forks of rows up to 512 pages
// 15.8 us; planning the compaction of 4096 pages 5.2 us, of 32768 pages 9.4 us, and
// 4 us to take a 512 x 512 table through it.
#include <algorithm>
#include <climits>

#include "device_common.cuh"
#include "ops_internal.cuh"

namespace kattn {
namespace {

// Blocks of a large plan: the barrier of a wider cluster costs more, and spreads
// rows and lists over more warps (512 forks: 8 blocks 21.2 us, 16 blocks 15.8 us;
// the compaction of 32768 pages, which has neither: 9.4 and 14.5 us).
constexpr int kCluster = 16, kCompactCluster = 8;
constexpr int kThreads = 1024;
constexpr int kWarpsPerBlock = kThreads / 32;
static_assert(kWarpsPerBlock == 32, "the sums over a block's warps take one per lane");
constexpr int kAhead = 8;                         // loads a lane has in flight

// CL: blocks of the plan, 1 or kCluster.
template <int CL>
__device__ __forceinline__ void plan_sync() {
  if constexpr (CL == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release;\n" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;\n" ::: "memory");
  }
}
template <int CL>
__device__ __forceinline__ int plan_rank() {
  return CL == 1 ? 0 : (int)blockIdx.x;           // the grid is one cluster
}

__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xffffffffu, v); }

struct BlockScratch {
  int warp[kWarpsPerBlock];
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
template <int CL>
__device__ __forceinline__ Chunk chunk_of(int n_pages, int rank) {
  Chunk c;
  c.per = (n_pages + CL - 1) / CL;
  c.lo = min(n_pages, rank * c.per);
  c.hi = min(n_pages, c.lo + c.per);
  return c;
}

// Ranks of the pages of [lo, hi) for which pick(page, count) holds, in ascending
// order: put(rank, page, count) is called for each.  Returns how many there are (to
// every thread).  Each warp has a run of pages, counts with ballots, and gives the
// ranks after a scan over the warps.  A run of up to 32 kHeld pages stays in
// registers in between; a longer one is read again (kHeld 4, 8, 16: the compaction of
// 32768 pages 9.4, 9.4, 9.7 us, reserving in a pool of 262144 15.1, 14.5, 13.9 us,
// 512 forks 15.8, 15.8, 16.1 us).
constexpr int kHeld = 8;

template <typename Pick, typename Put>
__device__ __forceinline__ int rank_pages(const int32_t* refs, int lo, int hi, BlockScratch& s,
                                          Pick pick, Put put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = max(0, hi - lo), run = (n + kThreads - 1) / kThreads * 32;
  const int w0 = min(n, warp * run) + lo, w1 = min(n, warp * run + run) + lo;
  int c[kHeld];
  auto load = [&](int p0) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int p = p0 + 32 * u + lane;
      c[u] = p < w1 ? __ldcg(refs + p) : 0;
    }
  };
  auto over = [&](int p0, auto&& each) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      if (p0 + 32 * u >= w1) break;               // (the same for the whole warp)
      const int p = p0 + 32 * u + lane;
      const bool take = p < w1 && pick(p, c[u]);
      each(p, c[u], take, __ballot_sync(0xffffffffu, take));
    }
  };
  int mine = 0;
  for (int p0 = w0; p0 < w1; p0 += 32 * kHeld) {
    load(p0);
    over(p0, [&](int, int, bool, unsigned bal) { mine += __popc(bal); });
  }
  __syncthreads();
  if (lane == 0) s.warp[warp] = mine;
  __syncthreads();
  const int v = s.warp[lane], total = warp_sum_int(v);
  int at = warp_sum_int(lane < warp ? v : 0);
  for (int p0 = w0; p0 < w1; p0 += 32 * kHeld) {
    if (w1 - w0 > 32 * kHeld) load(p0);
    over(p0, [&](int p, int count, bool take, unsigned bal) {
      if (take) put(at + __popc(bal & ((1u << lane) - 1u)), p, count);
      at += __popc(bal);
    });
  }
  return total;
}

// Where the entry of rank k lies in a list that each block wrote from its
// chunk's start on: block c's ranks begin at the sum of the counts before it.
template <int CL>
struct Places {
  int start[CL + 1];
  int per;
};
template <int CL>
__device__ __forceinline__ Places<CL> places_of(const int* chunk, int per) {
  Places<CL> p;
  p.per = per;
  int v[CL];
#pragma unroll
  for (int c = 0; c < CL; ++c) v[c] = __ldcg(chunk + c);
  p.start[0] = 0;
#pragma unroll
  for (int c = 0; c < CL; ++c) p.start[c + 1] = p.start[c] + v[c];
  return p;
}
template <int CL>
__device__ __forceinline__ int place(const Places<CL>& p, int k) {
  int at = k;
#pragma unroll
  for (int c = 1; c < CL; ++c)
    if (k >= p.start[c]) at = c * p.per + k - p.start[c];
  return at;
}

// One reference less on each of a lane's pages of a row (an entry below 0 is
// unused): the subtractions go out together, then their results are looked at.
template <int N>
__device__ __forceinline__ void drop_pages(const PageParams& p, const int (&e)[N]) {
  int before[N];
  bool outside = false;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const bool in = (unsigned)e[u] < (unsigned)p.n_pages;
    outside |= e[u] >= p.n_pages;
    before[u] = in ? atomicSub(p.refs + e[u], 1) : 1;
  }
#pragma unroll
  for (int u = 0; u < N; ++u)
    if (before[u] <= 0) {                         // it had none: put it back
      atomicAdd(p.refs + e[u], 1);
      outside = true;
    }
  if (outside) atomicOr(p.ws.err, KATTN_DEVERR_BAD_PAGE);
}
// Entries c0 + 32 u + lane of a row, -1 past the end.
__device__ __forceinline__ void load_entries(const int32_t* row, int c0, int end, int (&e)[kAhead]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int c = c0 + 32 * u + lane;
    e[u] = c < end ? __ldcg(row + c) : -1;
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
template <int CL>
__device__ __forceinline__ void list_range(int n, int rank, int& lo, int& hi) {
  const int per = (n + CL - 1) / CL;
  lo = min(n, rank * per);
  hi = min(n, lo + per);
}

// A slot that a list names again, and a child that is also a parent.  Lists of up to
// kThreads entries are looked through in shared memory; longer ones leave marks in
// the workspace, which costs a trip to L2 and a barrier (512 slots reserved: 15.3 us
// instead of 13.1, the scan over the list below included): the first entry that names
// a slot wins its claim, n - i.
struct Lists {
  int seq[kThreads], parent[kThreads];
};
__device__ __forceinline__ bool short_list(const PageParams& p) {
  return p.n <= kThreads && (int64_t)p.n * p.max_pages < INT32_MAX;
}
template <int CL>
__device__ __forceinline__ void take_lists(const PageParams& p, int rank, Lists& l) {
  if (short_list(p)) {
    if ((int)threadIdx.x < p.n) {
      l.seq[threadIdx.x] = p.seqs[threadIdx.x];
      if (p.parents) l.parent[threadIdx.x] = p.parents[threadIdx.x];
    }
    __syncthreads();
    return;
  }
  for (int i = rank * kThreads + threadIdx.x; i < p.n; i += CL * kThreads) {
    const int s = p.seqs[i];
    if ((unsigned)s < (unsigned)p.n_slots) atomicMax(p.ws.claim + s, p.n - i);
    if (p.parents && (unsigned)p.parents[i] < (unsigned)p.n_slots) p.ws.mark[p.parents[i]] = 1;
  }
  plan_sync<CL>();
}
// Whether entry i may have slot s (for the whole warp).
__device__ __forceinline__ bool slot_mine(const PageParams& p, const Lists& l, int i, int s) {
  if ((unsigned)s >= (unsigned)p.n_slots) return false;
  if (!short_list(p))
    return __ldcg(p.ws.claim + s) == p.n - i && !(p.parents && __ldcg(p.ws.mark + s) != 0);
  const int lane = threadIdx.x & 31;
  bool taken = false;
  for (int j = lane; j < i; j += 32) taken |= l.seq[j] == s;
  if (p.parents)
    for (int j = lane; j < p.n; j += 32) taken |= l.parent[j] == s;
  return !__any_sync(0xffffffffu, taken);
}
// The marks of this block's entries go back to zero for the next call.
__device__ __forceinline__ void return_marks(const PageParams& p, int lo, int hi) {
  if (short_list(p)) return;
  for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
    const int s = p.seqs[i];
    if ((unsigned)s < (unsigned)p.n_slots) p.ws.claim[s] = 0;
    if (p.parents && (unsigned)p.parents[i] < (unsigned)p.n_slots) p.ws.mark[p.parents[i]] = 0;
  }
}

// The pages that the list entries want: value(i) of entry i.  Calls each(i, rank of
// its first page) for this block's entries [lo, hi), a warp each, once enough(all
// wanted) has said to.
template <typename Value, typename Enough, typename Each>
__device__ __forceinline__ void over_wants(const PageParams& p, int lo, int hi, BlockScratch& s,
                                           int* first, Value value, Enough enough, Each each) {
  const int warp = threadIdx.x >> 5;
  if (short_list(p)) {                            // one scan over the whole list
    int total;
    const int mine = block_prefix((int)threadIdx.x < p.n ? value(threadIdx.x) : 0, s, &total);
    first[threadIdx.x] = mine;
    __syncthreads();
    if (!enough((int64_t)total)) return;
    for (int i = lo + warp; i < hi; i += kWarpsPerBlock) each(i, first[i]);
    return;
  }
  // the sums before this block's entries and of the whole list, in 64 bits: 20 low
  // bits and the rest
  int64_t before = 0, all = 0;
  for (int i = threadIdx.x; i < p.n; i += kThreads) {
    const int m = value(i);
    all += m;
    if (i < lo) before += m;
  }
  const int low = (1 << 20) - 1;
  const int64_t want = ((int64_t)block_sum((int)(all >> 20), s) << 20) + block_sum((int)(all & low), s);
  const int64_t start = ((int64_t)block_sum((int)(before >> 20), s) << 20) + block_sum((int)(before & low), s);
  if (!enough(want)) return;
  int base = (int)min(start, (int64_t)INT32_MAX / 2);   // (ranks past the pool are never taken)
  for (int i0 = lo; i0 < hi; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    int total;
    const int mine = block_prefix(i < hi ? value(i) : 0, s, &total);
    __syncthreads();
    first[threadIdx.x] = base + mine;
    __syncthreads();
    for (int k = warp; k < min(kThreads, hi - i0); k += kWarpsPerBlock) each(i0 + k, first[k]);
    base += total;
  }
}

// ---------------------------------------------------------------- reserve
//   1. per list entry the missing pages (one warp each), and the free pages of the
//   block's chunk in order;  2. the entries' first ranks (a scan over the list) and
//   the pages of those ranks into the table.
template <int CL>
__global__ void __launch_bounds__(kThreads) reserve_kernel(const PageParams p) {
  __shared__ BlockScratch s;
  __shared__ Lists lists;
  __shared__ int first[kThreads];
  const int rank = plan_rank<CL>();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  take_lists<CL>(p, rank, lists);
  int lo, hi;
  list_range<CL>(p.n, rank, lo, hi);
  for (int i = lo + warp; i < hi; i += kWarpsPerBlock) {
    const int slot = p.seqs[i], len = p.lens[i];
    int miss = 0;
    if (slot_mine(p, lists, i, slot) && len_ok(p, len)) {
      const int need = pages_for(p, len);
      const int32_t* row = p.table + (int64_t)slot * p.max_pages;
      bool outside = false;
      for (int c0 = 0; c0 < need; c0 += 32 * kAhead) {
        int e[kAhead];
        load_entries(row, c0, need, e);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          miss += c0 + 32 * u + lane < need && e[u] < 0;
          outside |= e[u] >= p.n_pages;
        }
      }
      if (outside) atomicOr(p.ws.err, KATTN_DEVERR_BAD_PAGE);
      miss = warp_sum_int(miss);
    } else if (lane == 0) {
      atomicOr(p.ws.err, KATTN_DEVERR_BAD_SEQUENCE);
    }
    if (lane == 0) p.ws.flag[i] = miss;
  }
  const Chunk ch = chunk_of<CL>(p.n_pages, rank);
  int* list = p.ws.list + ch.lo;
  const int free_here = rank_pages(
      p.refs, ch.lo, ch.hi, s, [](int, int c) { return c == 0; },
      [&](int r, int page, int) { list[r] = page; });
  if (threadIdx.x == 0) p.ws.chunk[rank] = free_here;
  plan_sync<CL>();
  const Places<CL> pl = places_of<CL>(p.ws.chunk, ch.per);
  over_wants(
      p, lo, hi, s, first, [&](int i) { return __ldcg(p.ws.flag + i); },
      [&](int64_t want) {                         // all of them, or none
        const bool enough = want <= (int64_t)pl.start[CL];
        if (!enough && rank == 0 && threadIdx.x == 0) atomicOr(p.ws.err, KATTN_DEVERR_NO_PAGES);
        return enough;
      },
      [&](int i, int at) {
        if (__ldcg(p.ws.flag + i) == 0) return;
        const int need = pages_for(p, p.lens[i]);
        int32_t* row = p.table + (int64_t)p.seqs[i] * p.max_pages;
        for (int c0 = 0; c0 < need; c0 += 32 * kAhead) {
          int e[kAhead];
          load_entries(row, c0, need, e);
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {      // the pages first, then the stores
            const bool miss = c0 + 32 * u + lane < need && e[u] < 0;
            const unsigned bal = __ballot_sync(0xffffffffu, miss);
            e[u] = miss ? __ldcg(p.ws.list + place(pl, at + __popc(bal & ((1u << lane) - 1u)))) : -1;
            at += __popc(bal);
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u)
            if (e[u] >= 0) {
              row[c0 + 32 * u + lane] = e[u];
              p.refs[e[u]] = 1;
            }
        }
      });
  return_marks(p, lo, hi);
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
    const int e[1] = {atomicExch(row + c, -1)};
    drop_pages(p, e);
  }
}

// ------------------------------------------------------------------- fork
//   1. per pair (one warp each) the checks, and the release of what a valid child
//   held;  2. the free pages in order;  3. the ranks of the pairs that need a page of
//   their own, and the children's rows.
// flag: 0 skipped, 1 valid, 2 valid with a page of its own.
template <int CL>
__global__ void __launch_bounds__(kThreads) fork_kernel(const PageParams p) {
  __shared__ BlockScratch s;
  __shared__ Lists lists;
  __shared__ int first[kThreads];
  const int rank = plan_rank<CL>();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  take_lists<CL>(p, rank, lists);
  int lo, hi;
  list_range<CL>(p.n, rank, lo, hi);
  const int page_mask = (1 << p.page_shift) - 1;
  for (int i = lo + warp; i < hi; i += kWarpsPerBlock) {
    const int child = p.seqs[i], parent = p.parents[i], len = p.lens[i];
    bool ok = slot_mine(p, lists, i, child) && (unsigned)parent < (unsigned)p.n_slots && len_ok(p, len);
    unsigned err = ok ? 0u : KATTN_DEVERR_BAD_SEQUENCE;
    if (ok) {
      const int need = pages_for(p, len);
      const int32_t* row = p.table + (int64_t)parent * p.max_pages;
      bool absent = false, outside = false;
      for (int c0 = 0; c0 < need; c0 += 32 * kAhead) {
        int e[kAhead];
        load_entries(row, c0, need, e);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          absent |= c0 + 32 * u + lane < need && e[u] < 0;
          outside |= e[u] >= p.n_pages;
        }
      }
      if (__any_sync(0xffffffffu, absent)) err |= KATTN_DEVERR_BAD_SEQUENCE;
      if (__any_sync(0xffffffffu, outside)) err |= KATTN_DEVERR_BAD_PAGE;
      ok = err == 0;
    }
    if (ok) {
      const int32_t* row = p.table + (int64_t)child * p.max_pages;
      for (int c0 = 0; c0 < p.max_pages; c0 += 32 * kAhead) {
        int e[kAhead];
        load_entries(row, c0, p.max_pages, e);
        drop_pages(p, e);
      }
    } else if (lane == 0) {
      atomicOr(p.ws.err, err);
    }
    if (lane == 0) p.ws.flag[i] = !ok ? 0 : (len & page_mask) ? 2 : 1;
  }
  plan_sync<CL>();
  const Chunk ch = chunk_of<CL>(p.n_pages, rank);
  int* list = p.ws.list + ch.lo;
  const int free_here = rank_pages(
      p.refs, ch.lo, ch.hi, s, [](int, int c) { return c == 0; },
      [&](int r, int page, int) { list[r] = page; });
  if (threadIdx.x == 0) p.ws.chunk[rank] = free_here;
  plan_sync<CL>();
  const Places<CL> pl = places_of<CL>(p.ws.chunk, ch.per);
  const int supply = pl.start[CL];
  over_wants(
      p, lo, hi, s, first, [&](int i) { return (int)(__ldcg(p.ws.flag + i) == 2); },
      [](int64_t) { return true; },
      [&](int i, int at) {
        const int flag = __ldcg(p.ws.flag + i);
        int from = -1, to = -1;
        if (flag != 0) {
          const int child = p.seqs[i], parent = p.parents[i], len = p.lens[i];
          int full = len >> p.page_shift;
          int32_t* row = p.table + (int64_t)child * p.max_pages;
          const int32_t* src = p.table + (int64_t)parent * p.max_pages;
          if (flag == 2) {
            if (at < supply) {
              from = __ldcg(src + full);
              to = __ldcg(p.ws.list + place(pl, at));
            } else {                              // no page left: the child stays empty
              if (lane == 0) atomicOr(p.ws.err, KATTN_DEVERR_NO_PAGES);
              full = 0;
            }
          }
          for (int c0 = 0; c0 < p.max_pages; c0 += 32 * kAhead) {
            int e[kAhead];
            load_entries(src, c0, full, e);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
              const int c = c0 + 32 * u + lane;
              if (c < full) atomicAdd(p.refs + e[u], 1);
              if (c < p.max_pages) row[c] = c == full ? to : e[u];
            }
          }
          if (to >= 0 && lane == 0) p.refs[to] = 1;
        }
        if (lane == 0) {
          p.src[i] = from;
          p.dst[i] = to;
        }
      });
  return_marks(p, lo, hi);
}

// ---------------------------------------------------------------- compact
//   1. live pages per chunk;  2. with their sum n_live, the free pages below it
//   and the live pages at or above it, in order;  3. the moves, the counts
//   after them, and the map of all pages.  rewrite_kernel then takes the table through
//   the map.
template <int CL>
__global__ void __launch_bounds__(kThreads) compact_kernel(const PageParams p) {
  __shared__ BlockScratch s;
  const int rank = plan_rank<CL>();
  const Chunk ch = chunk_of<CL>(p.n_pages, rank);
  int live = 0;
  for (int t0 = ch.lo; t0 < ch.hi; t0 += kThreads * kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = t0 + u * kThreads + (int)threadIdx.x;
      live += at < ch.hi && __ldcg(p.refs + at) > 0;
    }
  }
  live = block_sum(live, s);
  if (threadIdx.x == 0) p.ws.chunk[rank] = live;
  plan_sync<CL>();
  int n_live = 0;
#pragma unroll
  for (int c = 0; c < CL; ++c) n_live += __ldcg(p.ws.chunk + c);
  int* holes = p.ws.list + ch.lo;
  int2* movers = p.ws.list2 + ch.lo;
  const int n_holes = rank_pages(
      p.refs, ch.lo, min(ch.hi, n_live), s,
      [&](int page, int c) {
        p.ws.to[page] = c <= 0 ? -1 : page;       // it stays; no table entry may name a free one
        return c <= 0;
      },
      [&](int r, int page, int) { holes[r] = page; });
  const int n_movers = rank_pages(
      p.refs, max(ch.lo, n_live), ch.hi, s,
      [&](int page, int c) {
        if (c <= 0) p.ws.to[page] = -1;           // no table entry may name it
        return c > 0;
      },
      [&](int r, int page, int c) { movers[r] = make_int2(page, c); });
  if (threadIdx.x == 0) {
    p.ws.chunk[CL + rank] = n_holes;
    p.ws.chunk[2 * CL + rank] = n_movers;
  }
  plan_sync<CL>();
  const Places<CL> ph = places_of<CL>(p.ws.chunk + CL, ch.per);
  const Places<CL> pm = places_of<CL>(p.ws.chunk + 2 * CL, ch.per);
  const int moves = pm.start[CL];           // as many as holes
  const int slots = max(1, p.n_pages / 2);
  for (int k = rank * kThreads + threadIdx.x; k < slots; k += CL * kThreads) {
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
  const int64_t all = (int64_t)p.n_slots * p.max_pages;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all;
       i += (int64_t)gridDim.x * blockDim.x) {
    int e = p.table[i];
    if (e >= 0) {                                 // (a free page has no place: another's rows move there)
      const int to = e < p.n_pages ? __ldcg(p.ws.to + e) : -1;
      if (to < 0) atomicOr(p.ws.err, KATTN_DEVERR_BAD_PAGE);
      else e = to;
    }
    p.table_out[i] = e;
  }
}

// ------------------------------------------------------------------- copy
// One block per (list entry, plane), in a grid stride: the page's rows of K and of V
// are loaded together (four 16-byte loads a thread and step), then stored.  Bound by
// HBM: 7864 pages of 64 rows and 4 planes (1.06 GB moved) take 173 us, 6.1 TB/s.
// Streaming cache hints cost 3% (179 us).
constexpr int kCopyThreads = 256;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyParams p) {
  const int n = p.count ? min(p.n, max(0, *p.count)) : p.n;
  const int64_t units = (int64_t)n * p.Hkv;
  const int vecs = p.page_rows * kD / 16;         // a multiple of 256 (page_rows >= 32)
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = (int)(u / p.Hkv), h = (int)(u - (int64_t)i * p.Hkv);
    const int from = __ldg(p.src + i), to = __ldg(p.dst + i);
    if (from < 0 || to < 0) continue;
    if (from >= p.n_pages || to >= p.n_pages) {
      if (threadIdx.x == 0) atomicOr(p.err, KATTN_DEVERR_BAD_PAGE);
      continue;
    }
    const int64_t plane = (int64_t)h * p.cap_rows;
    const int64_t a = plane + (int64_t)from * p.page_rows, b = plane + (int64_t)to * p.page_rows;
    const uint4* ks = reinterpret_cast<const uint4*>(p.k + a * kD) + threadIdx.x;
    const uint4* vs = reinterpret_cast<const uint4*>(p.v + a * kD) + threadIdx.x;
    uint4* kd = reinterpret_cast<uint4*>(p.k + b * kD) + threadIdx.x;
    uint4* vd = reinterpret_cast<uint4*>(p.v + b * kD) + threadIdx.x;
    // the scales: threads of the first half take K's, of the second V's
    const bool second = threadIdx.x >= kCopyThreads / 2;
    const int r0 = threadIdx.x & (kCopyThreads / 2 - 1);
    float* sc = second ? p.v_scale : p.k_scale;
    for (int r = r0; r < p.page_rows; r += kCopyThreads / 2) sc[b + r] = __ldg(sc + a + r);
    int c = 0;
    for (; c + 2 * kCopyThreads <= vecs; c += 2 * kCopyThreads) {
      const uint4 k0 = __ldg(ks + c), k1 = __ldg(ks + c + kCopyThreads);
      const uint4 v0 = __ldg(vs + c), v1 = __ldg(vs + c + kCopyThreads);
      *(kd + c) = k0;
      *(kd + c + kCopyThreads) = k1;
      *(vd + c) = v0;
      *(vd + c + kCopyThreads) = v1;
    }
    if (c < vecs) {
      const uint4 k0 = __ldg(ks + c), v0 = __ldg(vs + c);
      *(kd + c) = k0;
      *(vd + c) = v0;
    }
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

// A plan by one block, or by one cluster of kCluster blocks (more than the portable
// 8, which every GPU of this kind holds).
template <typename Kernel>
cudaError_t launch_plan(Kernel one, Kernel many, int blocks, bool large, const PageParams& p,
                        cudaStream_t stream) {
  if (!large) {
    one<<<1, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  const cudaError_t e = cudaFuncSetAttribute(many, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, many, p);
}
// Where the cluster starts to pay (one block / the cluster, us): reserving for 8
// slots over 16384 pages 8.4 / 10.1, over 32768 pages 11.2 / 10.5; for 64 slots
// 9.3 / 9.3; compacting 4096 pages 7.0 / 7.5, 8192 pages 8.7 / 7.4.
bool large_plan(const PageParams& p) { return p.n_pages > 16384 || p.n > 64; }
bool large_compaction(const PageParams& p) { return p.n_pages > 4096; }

cudaError_t launch_reserve_pages(const PageParams& p, cudaStream_t stream) {
  return launch_plan(reserve_kernel<1>, reserve_kernel<kCluster>, kCluster, large_plan(p), p, stream);
}

cudaError_t launch_free_sequences(const PageParams& p, cudaStream_t stream) {
  free_kernel<<<(unsigned)p.n, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_fork_sequences(const PageParams& p, cudaStream_t stream) {
  return launch_plan(fork_kernel<1>, fork_kernel<kCluster>, kCluster, large_plan(p), p, stream);
}

cudaError_t launch_compact_pages(const PageParams& p, cudaStream_t stream) {
  const cudaError_t e =
      launch_plan(compact_kernel<1>, compact_kernel<kCompactCluster>, kCompactCluster,
                  large_compaction(p), p, stream);
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
  const int64_t units = (int64_t)p.n * p.Hkv;
  copy_kernel<<<(unsigned)std::min<int64_t>(units, 152 * 8), kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kattn
