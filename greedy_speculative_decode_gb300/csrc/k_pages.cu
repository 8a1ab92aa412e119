// k_pages.cu -- the pages of a cache handed out, shared between sequences,
// packed and copied.
//
// A table's row s holds held[s] pages for its length[s] positions; refs counts
// the rows that hold a page, and whatever else a program counts there.  Both
// plans (fork, compact) are functions of the table and the counts alone: sums
// over rows and pages, no order of arrival.  Each is one launch of one cluster
// of up to eight CTAs, which meet at the cluster's barriers: a table's numbers are few
// (64 rows of 256 pages and 20 thousand pages are 200 KB, in L2), so what bounds
// them is the chain of dependent loads and barriers, not bytes: with the copy of
// its pages a fork of 1 row to 8 takes 8.2 us in a graph (one CTA),
// of 64 rows of up to 4096 positions 15.4 (eight CTAs).  The copy of the pages is a
// kernel of its own behind the plan, queued before that has ended; it is bound by
// memory: 64 x 4096 positions of two layers compacted, 180 MB read and as many
// written, in 73 us (76.5 with loads that stay in L2), 0.71 of the copy rate.
//
// Free pages are found by rank: a warp counts those of its range of pages with
// ballots, the counts are summed over warps and CTAs, and a second look at the
// ranges gives each free page its rank, so that pages are handed out in order,
// lowest first.
#include "pages.h"

#include <algorithm>
#include <cooperative_groups.h>

#include "sv_ptx.cuh"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kPgThreads = 1024, kPgWarps = 32;
// CTAs of a plan's cluster: one where there is little to look through.
constexpr int kPgWide = 8;
static_assert(kPagesMaxSeq == kPgThreads, "a thread a row");

// Exclusive sums over the block's threads; total in `sum`.  (s: a word a warp; two barriers.)
__device__ __forceinline__ int block_scan(int v, int* s, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPgWarps; ++w) {
    const int n = s[w];
    before += w < warp ? n : 0;
    all += n;
  }
  sum = all;
  return before + x - v;
}

// All of the plan's threads meet; what they wrote is seen.
template <int CTAS>
__device__ __forceinline__ void meet() {
  if (CTAS == 1) __syncthreads();
  else cg::this_cluster().sync();
}

// The pages of a warp: 32-page steps a .. b - 1 of the pool, in order of (CTA, warp).
template <int CTAS>
struct PageRange {
  int a, b;
  __device__ __forceinline__ PageRange(int n_pages, int rank) {
    const unsigned steps = (n_pages + 31) / 32, w = rank * kPgWarps + (threadIdx.x >> 5);
    constexpr unsigned kAll = CTAS * kPgWarps;  // (a power of two; below 2^22 steps)
    a = (int)(steps * w / kAll);
    b = (int)(steps * (w + 1) / kAll);
  }
  // Whether a page is in the range of one of a CTA's warps.
  static __device__ __forceinline__ bool has(int n_pages, int rank, int page) {
    const unsigned steps = (n_pages + 31) / 32, step = (unsigned)page / 32;
    return step >= steps * rank / CTAS && step < steps * (rank + 1) / CTAS;
  }
};

// Pages of the range with a count of zero.
template <int CTAS>
__device__ __forceinline__ int count_free(const PageRange<CTAS>& g, const int* refs, int n_pages) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll 1
  for (int s = g.a; s < g.b; s += 4) {
    int x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int page = (s + i) * 32 + lane;
      x[i] = s + i < g.b && page < n_pages ? __ldcg(refs + page) : 1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) n += __popc(__ballot_sync(0xffffffffu, x[i] == 0));
  }
  return n;
}

// Free pages before this warp's range, and of the whole pool (`all`); a cluster barrier.
template <int CTAS>
__device__ __forceinline__ int free_before(int mine, int* s_scan, int* s_total, int& all) {
  cg::cluster_group cluster = cg::this_cluster();
  int sum;
  const int before = block_scan((threadIdx.x & 31) == 0 ? mine : 0, s_scan, sum);
  if (CTAS == 1) {
    all = sum;
    return __shfl_sync(0xffffffffu, before, 0);
  }
  if (threadIdx.x == 0) *s_total = sum;
  cluster.sync();
  int base = 0;
  all = 0;
  const int rank = (int)cluster.block_rank();
#pragma unroll
  for (int c = 0; c < CTAS; ++c) {
    const int n = *cluster.map_shared_rank(s_total, c);
    base += c < rank ? n : 0;
    all += n;
  }
  return base + __shfl_sync(0xffffffffu, before, 0);
}

struct ForkShared {
  int src[kPagesMaxSeq], kept[kPagesMaxSeq], need[kPagesMaxSeq], held[kPagesMaxSeq];
  int last[kPagesMaxSeq];    // a last page that is not full, or -1; below -1: the row gets a copy of page -2 - last
  int offset[kPagesMaxSeq + 1];
  int scan[kPgWarps];
  int total;
};

// New rows.  Every CTA works out the rows' numbers by itself; entries and pages
// are divided among them.
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kPgThreads, 1) k_fork(const ForkParams p) {
  extern __shared__ int s_raw[];
  ForkShared& s = *reinterpret_cast<ForkShared*>(s_raw);
  const int tid = threadIdx.x, lane = tid & 31, rank = CTAS == 1 ? 0 : (int)cg::this_cluster().block_rank();
  pdl_trigger();
  pdl_wait();
  const int S = p.in.n_seq, W = p.in.width, all_threads = CTAS * kPgThreads, me = rank * kPgThreads + tid;
  // ---- the rows: what they keep and need
  int wrong = 0, keep = 0, kept = 0, need = 0, src = -1, held = 0, last = -1;
  if (tid < S) {
    src = p.source ? __ldcg(p.source + tid) : tid;
    const int asked = p.keep ? __ldcg(p.keep + tid) : INT32_MAX, room = p.room ? __ldcg(p.room + tid) : 0;
    held = min(max(__ldcg(p.in.held + tid), 0), W);
    if (src < -1 || src >= S) wrong = ST_BAD_PAGE;
    else if (src >= 0) {
      const int have = min(max(__ldcg(p.in.held + src), 0), W);
      keep = min(min(max(__ldcg(p.in.length + src), 0), max(asked, 0)), (int)min((int64_t)have * kPage, (int64_t)INT32_MAX));
      kept = (int)(((int64_t)keep + kPage - 1) / kPage);
      need = max(kept, (int)(((int64_t)max(room, 0) + kPage - 1) / kPage));
      if (need > W) wrong = ST_BAD_PAGE;
      else if (keep % kPage) {
        last = __ldcg(p.in.table + (int64_t)src * W + kept - 1);
        if ((uint32_t)last >= (uint32_t)p.in.n_pages) last = -1;
      }
    }
    s.src[tid] = src;
    s.kept[tid] = kept;
    s.need[tid] = need;
    s.held[tid] = held;
    s.last[tid] = last;
  }
  // ---- the counts: those of before, ...
  for (int i = me; i < p.in.n_pages; i += all_threads) p.count[i] = __ldcg(p.in.refs + i);
  meet<CTAS>();
  wrong = __syncthreads_or(wrong) ? ST_BAD_PAGE : 0;
  // ... less the old rows' entries, with the new rows'
  const int entries = S * W;  // (at most 2^29)
  if (!wrong) {
    for (int e = me; e < entries; e += all_threads) {
      const int row = (unsigned)e / (unsigned)W, j = e - row * W;
      if (j >= max(s.held[row], s.kept[row])) continue;
      const int old = j < s.held[row] ? __ldcg(p.in.table + e) : -1;
      int now = -1;
      if (j < s.kept[row]) {
        now = s.src[row] == row ? old : __ldcg(p.in.table + (int64_t)s.src[row] * W + j);
        if (p.in_place && s.src[row] != row) p.staged[e] = now;
        if ((uint32_t)now >= (uint32_t)p.in.n_pages && p.status) atomicOr(p.status, ST_BAD_PAGE);
      }
      if (old == now) continue;
      if ((uint32_t)old < (uint32_t)p.in.n_pages) atomicSub(p.count + old, 1);
      if ((uint32_t)now < (uint32_t)p.in.n_pages) atomicAdd(p.count + now, 1);
    }
  }
  meet<CTAS>();
  // ---- last pages that are not full: one row may go on in the page itself
  int copy = 0;
  if (!wrong && last >= 0) {
    const int holders = __ldcg(p.count + last);
    if (holders > 1) {
      int part = 0, lowest = S;
      for (int i = 0; i < S; ++i)
        if (s.last[i] == last) {
          ++part;
          lowest = min(lowest, i);
        }
      copy = holders != part || lowest != tid;
    }
  }
  int wanted;
  const int offset = block_scan(tid < S ? need - kept + copy : 0, s.scan, wanted);
  if (tid < S) {
    s.offset[tid] = offset;
    if (copy) s.last[tid] = -2 - last;  // (every thread has compared: block_scan's barriers)
  }
  // ---- free pages, lowest first
  const PageRange<CTAS> range(p.in.n_pages, rank);
  const int mine = count_free(range, p.count, p.in.n_pages);
  int free_all;
  int at = free_before<CTAS>(mine, s.scan, &s.total, free_all);
  if (!wrong && free_all < wanted) wrong = ST_NO_PAGES;
  if (wrong) {  // nothing changes
    if (me < S) p.moves[me] = make_int2(-1, -1);
    if (me == 0 && p.status) atomicOr(p.status, wrong);
    meet<CTAS>();  // the others read this CTA's total
    return;
  }
  // A copied page has a holder less.  Behind the barrier, for until then the other CTAs
  // may have `holders` still to read; each CTA for the pages that it has below.  (The
  // counts stay above zero: whether a page is free does not change.)
  if (copy && PageRange<CTAS>::has(p.in.n_pages, rank, last)) atomicSub(p.count + last, 1);
  __syncthreads();
  for (int st = range.a; st < range.b; ++st) {
    const int page = st * 32 + lane;
    const int n = page < p.in.n_pages ? __ldcg(p.count + page) : 1;
    const uint32_t free = __ballot_sync(0xffffffffu, n == 0);
    const int r = at + __popc(free & ((1u << lane) - 1u));
    at += __popc(free);
    if (page >= p.in.n_pages) continue;
    const bool given = n == 0 && r < wanted;
    p.out.refs[page] = given ? 1 : n;
    if (!given) continue;
    int lo = 0, hi = S;  // the last row whose new pages begin at or before r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.offset[mid] <= r) lo = mid; else hi = mid;
    }
    const int i = r - s.offset[lo], from = s.last[lo];
    const int j = s.kept[lo] - (from < -1) + i;
    p.out.table[(int64_t)lo * W + j] = page;
    if (from < -1 && i == 0) p.moves[lo] = make_int2(-2 - from, page);
  }
  // ---- the rows' entries and numbers
  for (int e = me; e < entries; e += all_threads) {
    const int row = (unsigned)e / (unsigned)W, j = e - row * W;
    const int kept_here = s.kept[row] - (s.last[row] < -1);
    if (j < kept_here) {
      if (!p.in_place) p.out.table[e] = __ldcg(p.in.table + (int64_t)s.src[row] * W + j);
      else if (s.src[row] != row) p.out.table[e] = p.staged[e];
    } else if (j >= s.need[row] && (!p.in_place || j < s.held[row])) {
      p.out.table[e] = -1;
    }
  }
  if (rank == 0 && tid < S) {
    p.out.length[tid] = keep;
    p.out.held[tid] = need;
    if (!copy) p.moves[tid] = make_int2(-1, -1);
  }
  meet<CTAS>();
}

struct CompactShared {
  int scan[kPgWarps];
  int total;
};

// With U pages in use, the used ones at U and above go to the free ones below:
// the k-th highest to the k-th lowest.
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kPgThreads, 1) k_compact(const CompactParams p) {
  __shared__ CompactShared s;
  const int tid = threadIdx.x, lane = tid & 31, rank = CTAS == 1 ? 0 : (int)cg::this_cluster().block_rank();
  pdl_trigger();
  pdl_wait();
  const int N = p.in.n_pages, W = p.in.width, all_threads = CTAS * kPgThreads, me = rank * kPgThreads + tid;
  const PageRange<CTAS> range(N, rank);
  const int mine = count_free(range, p.in.refs, N);
  int free_all;
  const int free_at = free_before<CTAS>(mine, s.scan, &s.total, free_all);
  const int used = N - free_all;
  for (int k = me; k < p.n_moves; k += all_threads) p.moves[k] = make_int2(-1, -1);
  meet<CTAS>();
  int at = free_at;
  for (int st = range.a; st < range.b; ++st) {
    const int page = st * 32 + lane;
    const bool in = page < N;
    const int n = in ? __ldcg(p.in.refs + page) : 1;
    const uint32_t free = __ballot_sync(0xffffffffu, n == 0);
    const int r = at + __popc(free & ((1u << lane) - 1u));  // free pages below
    at += __popc(free);
    if (!in) continue;
    p.where[page] = n ? page : -1;
    if (n == 0 && page < used && r < p.n_moves) p.moves[r].y = page;
    // used pages above: all used, less those up to this one
    const int k = used - (page - r) - 1;
    if (n != 0 && page >= used && k < p.n_moves) p.moves[k].x = page;
    if (!p.in_place) p.out.refs[page] = n;
  }
  meet<CTAS>();
  // (free pages below `used` and used ones from there on are as many)
  for (int k = me; k < p.n_moves; k += all_threads) {
    const int2 m = __ldcg(p.moves + k);
    if (m.x < 0) break;
    p.where[m.x] = m.y;
    p.out.refs[m.y] = __ldcg(p.in.refs + m.x);
    p.out.refs[m.x] = 0;
  }
  meet<CTAS>();
  const int entries = p.in.n_seq * W;
  for (int e = me; e < entries; e += all_threads) {
    const int row = (unsigned)e / (unsigned)W, j = e - row * W;
    if (j >= __ldcg(p.in.held + row)) {
      if (!p.in_place) p.out.table[e] = -1;
      continue;
    }
    int page = __ldcg(p.in.table + e);
    if ((uint32_t)page < (uint32_t)N) {
      const int to = __ldcg(p.where + page);
      if (to >= 0) page = to;
    } else if (p.status) {
      atomicOr(p.status, ST_BAD_PAGE);
    }
    if (!p.in_place || page != __ldcg(p.in.table + e)) p.out.table[e] = page;
  }
  if (!p.in_place)
    for (int i = me; i < p.in.n_seq; i += all_threads) {
      p.out.length[i] = __ldcg(p.in.length + i);
      p.out.held[i] = __ldcg(p.in.held + i);
    }
}

// 16 bytes that are read once: past L1 (see the wait below), and first to leave L2.
__device__ __forceinline__ uint4 load_once(const uint8_t* p, uint64_t policy) {
  uint4 x;
  asm volatile("ld.global.cg.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p), "l"(policy) : "memory");
  return x;
}

// Pages copied within or between pools: a block a (move, pool, K or V) at a
// time, 16 bytes a thread, four of them on their way before the first is stored.
__global__ void __launch_bounds__(256) k_copy_pages(const __grid_constant__ CopyParams p) {
  const int tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();  // the moves, and whoever wrote the pages
  const uint64_t once = policy_evict_first();
  const int64_t units = (int64_t)p.n_moves * p.n_pools * 2;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int mv = (int)(u / (2 * p.n_pools)), w = (int)(u - (int64_t)mv * 2 * p.n_pools), at = w >> 1;
    const int2 m = __ldcg(p.moves + mv);
    if (m.x == -1 && m.y == -1) continue;
    if ((uint32_t)m.x >= (uint32_t)p.n_from || (uint32_t)m.y >= (uint32_t)p.n_to) {
      if (tid == 0 && p.status) atomicOr(p.status, ST_BAD_PAGE);
      continue;
    }
    const CopyParams::Pool& pool = p.pool[at];
    const uint8_t* src = (w & 1 ? pool.v : pool.k) + (int64_t)m.x * p.page_bytes;
    uint8_t* dst = (w & 1 ? pool.v_to : pool.k_to) + (int64_t)m.y * p.page_bytes;
    for (int i = tid * 16; i < p.page_bytes; i += 4 * 256 * 16) {
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * 4096 < p.page_bytes) x[k] = load_once(src + i + k * 4096, once);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * 4096 < p.page_bytes) __stcs(reinterpret_cast<uint4*>(dst + i + k * 4096), x[k]);
    }
    if (p.exp_bytes) {
      const uint8_t* es = (w & 1 ? pool.v_exp : pool.k_exp) + (int64_t)m.x * p.exp_bytes;
      uint8_t* ed = (w & 1 ? pool.v_exp_to : pool.k_exp_to) + (int64_t)m.y * p.exp_bytes;
      for (int i = tid; i < p.exp_bytes; i += 256) ed[i] = __ldcg(es + i);
    }
  }
}

}  // namespace

cudaError_t prepare_pages() {
  const cudaError_t e = cudaFuncSetAttribute(k_fork<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(ForkShared));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(k_fork<kPgWide>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(ForkShared));
}

// Whether one CTA is enough: it looks through entries and pages 1024 at a time, where
// eight have their barriers.  (Entries and pages, then us of a plan in a graph with one CTA
// and with eight: fork 585 6.1 and 7.8, 3292 8.1 and 9.0, 6740 10.9 and 9.5, 14000 18.2
// and 10.1; compact 567 4.7 and 6.3, 3274 5.8 and 7.2, 6706 7.6 and 7.4, 13934 11.2 and 8.1.)
static bool small_plan(const PageTable& t) { return (int64_t)t.n_seq * t.width + t.n_pages <= 4 * kPgThreads; }

// A kernel that may be launched while the one ahead of it ends (it waits for that
// before it reads anything).
template <class P>
static cudaError_t launch_behind(void (*kernel)(P), const P& p, unsigned grid, unsigned block, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_fork(const ForkParams& p, cudaStream_t s) {
  return small_plan(p.in) ? launch_behind(k_fork<1>, p, 1, kPgThreads, sizeof(ForkShared), s)
                          : launch_behind(k_fork<kPgWide>, p, kPgWide, kPgThreads, sizeof(ForkShared), s);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t s) {
  return small_plan(p.in) ? launch_behind(k_compact<1>, p, 1, kPgThreads, 0, s)
                          : launch_behind(k_compact<kPgWide>, p, kPgWide, kPgThreads, 0, s);
}

cudaError_t launch_copy(const CopyParams& p, int num_sms, cudaStream_t s) {
  const int64_t units = (int64_t)p.n_moves * p.n_pools * 2;
  return launch_behind(k_copy_pages, p, (unsigned)std::min<int64_t>(units, 8 * (int64_t)num_sms), 256, 0, s);
}

}  // namespace sv
