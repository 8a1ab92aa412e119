// attend_dev.cuh -- attention of a ragged batch's rows over a paged cache.
//
// Row i of sequence s stands at position t = first[s] + i and sees the
// positions p <= t, with a window W only those with p > t - W or p < sinks:
//   s_p = scale * q . k_p,  o = sum_p softmax(s)_p v_p,  lse = ln sum_p exp(s_p).
// The cache is read once per tile of 8 N query rows (token rows x the query
// heads of a kv head, packed one behind the other whatever the group size), so
// few rows are bound by its bytes: a CTA streams chunks of four pages by TMA
// into a ring, and four warps share each chunk.
//   Scores, transposed: S^T = K Q^T.  Warp w takes page w: its 16 positions
//     are the 16 rows of an mma, eight query rows its columns, so single-token
//     decode with a group of up to eight heads wastes none of it.  K goes from
//     8 to 16 bits in registers.
//   The query rows' maxima over the chunk meet in shared memory, and each warp
//     leaves its weights there, transposed on the way (stmatrix).
//   O^T += V^T P^T: warp w takes D / 4 columns of every position, so the
//     accumulators need no merge between warps.  A transposing load of bytes
//     makes V's operand (four consecutive positions of a column in a word).
//
// An 8-bit cache's exponents cost an addition each.  The key's scales its
// score; the value's, ev, is added to the score in log2 units, t' = log2(e) s +
// ev, and the weights are p' = 2^(t' - max t'): they already carry the value's
// scale, the largest is 1, and f16 (11 bits, the tensor cores' type that holds
// every e4m3 code) rounds them relative to the largest contribution.  The
// denominator takes p' 2^-ev, unrounded, in fp32.  Queries go to f16 divided
// by a power of two near their row's largest value: exact for elements within
// 2^-17 of it, and below that off by at most 2^-25 of it.  A bf16 cache keeps
// bf16 queries, and the weights are taken as the sum of two bf16 values
// (about 2^-16), since one would shift outputs by up to half a bf16 step.
//
// Splits are ranges of absolute positions (attn_split_start), and a row's
// arithmetic does not depend on the rows, sequences or tiles beside it: a
// chunk a row does not see leaves its maximum, sum and accumulators as they
// are, bit for bit.  So each row's result is the same in every batch.
#pragma once
#include "paged_dev.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace sv {
namespace {

constexpr int kAttendWarps = 4;
constexpr int kAttendThreads = (kAttendWarps + 1) * 32;  // consumers, then the producer warp

// A tile of query rows.
struct AttendTile {
  int row0, f0, nf, kvh;  // the sequence's first row, the tile's first query row, the sequence's query rows
  int first;              // position of the sequence's first row
};
// What the producer tells the consumers of a chunk.
struct alignas(16) AttendDesc {
  int base, loaded, flags, split;  // first position; pages in the ring; kDesc*
  AttendTile tile;
  int pad[3];
};
// kDescTile: the first chunk of another tile; kDescLast: the split's last
// chunk; kDescEdge: some row does not see some position, or a page is not
// there; kDescEnd: no chunk, there are no more
enum : int { kDescTile = 1, kDescLast = 2, kDescEdge = 4, kDescEnd = 8 };

template <int D_, int FMT_, int N_>
struct AttendCfg {
  static constexpr int D = D_, FMT = FMT_, N = N_;  // N: query tiles of 8 rows
  static constexpr bool kBf16 = FMT == SV_KV_BF16;
  static constexpr int RB = D * (kBf16 ? 2 : 1);  // bytes of a position's row
  static constexpr int kPageBytes = kPage * RB;
  static constexpr int CP = kAttendWarps;         // pages per chunk: one a warp
  static constexpr int kChunk = CP * kPage;
  static constexpr int kStageBytes = 2 * CP * kPageBytes;
  static constexpr int kStages = RB == 64 ? 4 : RB == 512 ? 2 : 3;
  // CTAs per SM that registers are cut for (the rings allow 4 at rows of 64
  // and 128 bytes, 2 at 256, 1 at 512)
  static constexpr int kRingSm = RB <= 128 ? 4 : RB == 256 ? 2 : 1;
  static constexpr int kRegSm = N <= 2 ? 4 : N == 4 ? 3 : 2;
  static constexpr int kPerSm = kRingSm < kRegSm ? kRingSm : kRegSm;
  static constexpr int NK = D / 16;               // k16 steps of a score
  static constexpr int DW = D / kAttendWarps;     // output columns per warp
  static constexpr int U = DW / 16;               // their 16-column units
  static constexpr int QR = 8 * N;                // query rows of a tile
  static constexpr bool kQRegs = N * NK <= 8;     // query fragments stay in registers
  // shared memory
  static constexpr int kScaleBytes = kBf16 ? 0 : 2 * CP * kPage;
  static constexpr int kOffScale = kStages * kStageBytes;
  static constexpr int kOffQ = kOffScale + kStages * kScaleBytes;  // query fragments [N][NK][32 lanes][2 words]
  static constexpr int kQBytes = N * NK * 256;
  static constexpr int kPStride = kChunk * 2 + 16;                 // bytes of a query row's weights, padded against
  static constexpr int kOffP = kOffQ + kQBytes;                    // bank conflicts
  static constexpr int kPBytes = QR * kPStride;                    // (bf16: twice, high and low parts)
  static constexpr int kOffMax = kOffP + kPBytes * (kBf16 ? 2 : 1);  // [QR][4] maxima of the warps
  static constexpr int kOffSum = kOffMax + QR * 16;                // [QR][4] sums
  static constexpr int kOffRow = kOffSum + QR * 16;                // [QR] score factors, positions, slots, maxima
  static constexpr int kOffDesc = kOffRow + 4 * QR * 4;            // [stages] chunk descriptors
  static constexpr int kOffBar = kOffDesc + kStages * (int)sizeof(AttendDesc);
  static constexpr int kOffSeq = kOffBar + 2 * kStages * 8;        // [n_seq + 1] chunks before, first, row start
  static constexpr int smem_bytes(int n_seq) { return 1024 + kOffSeq + 4 * (3 * n_seq + 2); }
  static_assert(1024 + kOffSeq + 4 * (3 * kAttendMaxSeq + 2) <= 227 * 1024, "shared memory of a CTA");
};

// Position within a page of score row n (0 .. 15).  A value fragment's
// register holds four consecutive positions of an 8-bit page, two of a bf16
// page; the scores take the same order, so weights need no shuffle.
template <bool kBf16>
__device__ __forceinline__ constexpr int pos_of_row(int n) {
  return kBf16 ? n : 4 * ((n & 7) >> 1) + (n & 1) + ((n >> 3) << 1);
}

// Byte offset of 16-byte unit c of position p in a page's shared-memory image:
// 128-byte boxes of all 16 positions, 128B-swizzled (rows of 64 bytes lie two
// to a box row).
template <int RB>
__device__ __forceinline__ uint32_t page_off(int p, int c) {
  if (RB == 64) return (uint32_t)((p >> 1) * 128 + ((((p & 1) * 4 + c) ^ ((p >> 1) & 7)) << 4));
  return (uint32_t)((c >> 3) * 2048 + p * 128 + (((c & 7) ^ (p & 7)) << 4));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool kBf16>
__device__ __forceinline__ void mma_16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kBf16) mma_bf16(d, a, b0, b1); else mma_f16(d, a, b0, b1);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two 16 x 16 byte matrices, transposed: lane (g, q) gets bytes 4 q .. 4 q + 3
// of columns g (r0) and g + 8 (r1) of the first, r2 and r3 of the second.
__device__ __forceinline__ void ldsm_b8_x2_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Two / four 8 x 8 matrices of 16-bit values, stored transposed.
__device__ __forceinline__ void stsm_x2_trans(uint32_t addr, uint32_t r0, uint32_t r1) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(r0), "r"(r1)
               : "memory");
}
__device__ __forceinline__ void stsm_x4_trans(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0),
               "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}

__device__ __forceinline__ int split_of(int pos, int d) {
  return pos < kAttnRegionA ? pos / kAttnSplitA : kAttnSplitsA + (pos - kAttnRegionA) / attn_split_b(d);
}

// The splits a range of rows t0 .. t1 of one sequence sees some position of:
// 0 .. n_sink - 1 and lo .. hi.
struct SplitRange {
  int n_sink, lo, n;  // n: splits in all
  __device__ __forceinline__ int at(int j) const { return j < n_sink ? j : lo + j - n_sink; }
};
// (limit: positions the block table reaches; those beyond are unseen)
__device__ __forceinline__ SplitRange splits_seen(int t0, int t1, int window, int sinks, int limit, int d) {
  SplitRange r = {0, 0, 0};
  t1 = min(t1, limit - 1);
  if (t1 < 0) return r;
  const int hi = split_of(t1, d);
  const int64_t w0 = (int64_t)t0 - window + 1;
  if (window > 0 && w0 > 0) {
    r.lo = w0 > t1 ? hi + 1 : split_of((int)w0, d);
    if (sinks > 0) r.n_sink = min(r.lo, split_of(min(sinks - 1, t1), d) + 1);
  }
  r.n = r.n_sink + hi - r.lo + 1;
  return r;
}

// The chunks that the rows of a sequence see: 0 .. n_sink - 1 and lo .. (n in
// all).  Consecutive ones of one split are an item, whose partial is one.
struct ChunkList {
  int n_sink, lo, n;
  __device__ __forceinline__ int at(int i) const { return i < n_sink ? i : lo + i - n_sink; }
};
template <class C>
__device__ __forceinline__ ChunkList chunks_seen(int t0, int t1, int window, int sinks, int limit) {
  ChunkList r = {0, 0, 0};
  t1 = min(t1, limit - 1);
  if (t1 < 0) return r;
  const int hi = t1 / C::kChunk;
  const int64_t w0 = (int64_t)t0 - window + 1;
  if (window > 0 && w0 > 0) {
    r.lo = w0 > t1 ? hi + 1 : (int)w0 / C::kChunk;
    if (sinks > 0) r.n_sink = min(r.lo, min(sinks - 1, t1) / C::kChunk + 1);
  }
  r.n = r.n_sink + hi - r.lo + 1;
  return r;
}

// The call's work: for each sequence, kv head and query tile the sequence's
// chunk list, one list behind the other.  CTA c of G takes the items that
// begin among chunks total c / G .. total (c + 1) / G - 1: a contiguous run, so
// that it seldom changes its queries, of nearly equal length for each CTA.
template <class C>
struct AttendWork {
  const AttendParams& p;
  const int *before, *first, *start;  // shared memory, per sequence
  int total, G;
};

// Walks a CTA's chunks in order, past chunks of which the tile sees nothing.
template <class C>
struct AttendWalk {
  AttendTile tile;
  ChunkList list;
  int seq, tiles, x, i;   // x: kv head * tiles + tile of the list; i: place in the list
  int t0, t1;             // positions of the tile's first and last token row
  int u, end;             // the chunk's number; the CTA's last + 1
  int base, split;
  uint32_t mask;          // pages that some row of the tile sees
  bool valid, fresh;      // fresh: the first chunk since the tile changed

  __device__ __forceinline__ void start(const AttendWork<C>& wk) {
    valid = false;
    fresh = true;
    u = (int)((int64_t)wk.total * blockIdx.x / gridDim.x);
    end = (int)((int64_t)wk.total * (blockIdx.x + 1) / gridDim.x);
    if (u >= end) return;
    int lo = 0, hi = wk.p.rows.n_seq;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (wk.before[mid] <= u) lo = mid; else hi = mid;
    }
    seq = lo;
    open_seq(wk);
    x = (u - wk.before[seq]) / list.n;
    i = (u - wk.before[seq]) % list.n;
    open_tile(wk);
    // to the first item that begins here
    if (i > 0)
      while (split_of(list.at(i) * C::kChunk, C::D) == split_of(list.at(i - 1) * C::kChunk, C::D)) {
        ++u;
        if (++i == list.n && !next_list(wk)) return;
        if (i == 0) break;
      }
    settle(wk);
  }
  __device__ __forceinline__ void open_seq(const AttendWork<C>& wk) {
    tile.first = wk.first[seq];
    tile.row0 = wk.start[seq];
    const int n = wk.start[seq + 1] - tile.row0;
    tile.nf = n * wk.G;
    tiles = (tile.nf + C::QR - 1) / C::QR;
    list = chunks_seen<C>(tile.first, tile.first + n - 1, wk.p.window, wk.p.sinks, wk.p.rows.limit());
  }
  __device__ __forceinline__ void open_tile(const AttendWork<C>& wk) {
    tile.kvh = x / tiles;
    tile.f0 = x % tiles * C::QR;
    t0 = tile.first + tile.f0 / wk.G;
    t1 = tile.first + (min(tile.f0 + C::QR, tile.nf) - 1) / wk.G;
    fresh = true;
  }
  // the next list's first chunk (u is its number); false: the CTA's work is done
  __device__ __forceinline__ bool next_list(const AttendWork<C>& wk) {
    if (u >= end) return false;
    i = 0;
    if (++x == tiles * wk.p.n_kv_heads) {
      x = 0;
      do ++seq; while (wk.before[seq + 1] == wk.before[seq]);
      open_seq(wk);
    }
    open_tile(wk);
    return true;
  }
  // from the chunk at u to the next one with a page that is seen
  __device__ __forceinline__ void settle(const AttendWork<C>& wk) {
    valid = false;
    for (;;) {
      base = list.at(i) * C::kChunk;
      const int s = split_of(base, C::D);
      // (past the CTA's share only an item that it has begun is carried on)
      if (u >= end && (i == 0 || split_of(list.at(i - 1) * C::kChunk, C::D) != s)) return;
      split = s;
      mask = 0;
#pragma unroll
      for (int j = 0; j < C::CP; ++j) {
        const int a = base + j * kPage;
        const bool vis = a <= t1 && a < wk.p.rows.limit() &&
                         (wk.p.window <= 0 || a + kPage - 1 > t0 - wk.p.window || a < wk.p.sinks);
        mask |= (vis ? 1u : 0u) << j;
      }
      if (mask) {
        valid = true;
        return;
      }
      if (!step(wk)) return;
    }
  }
  __device__ __forceinline__ bool step(const AttendWork<C>& wk) {
    ++u;
    return ++i < list.n || next_list(wk);
  }
  __device__ __forceinline__ void next(const AttendWork<C>& wk) {
    fresh = false;
    valid = false;
    if (step(wk)) settle(wk);
  }
};

// Chunks of each sequence, as running totals in shared memory (all threads).
template <class C>
__device__ int attend_plan(const AttendParams& p, int G, int* before, int* first, int* start) {
  const int tid = threadIdx.x, S = p.rows.n_seq;
  // (rows outside the call's buffers are left out)
  for (int s = tid; s <= S; s += kAttendThreads)
    start[s] = p.rows.row_start ? min(max(p.rows.row_start[s], 0), p.rows.n_rows) : s * p.rows.rows_each;
  for (int s = tid; s < S; s += kAttendThreads) first[s] = first_of(p.rows, s);
  __syncthreads();
  for (int s = tid; s < S; s += kAttendThreads) {
    const int n = max(0, start[s + 1] - start[s]);
    const int tiles = (n * G + C::QR - 1) / C::QR;
    const ChunkList l = chunks_seen<C>(first[s], first[s] + n - 1, p.window, p.sinks, p.rows.limit());
    before[s] = n > 0 ? tiles * p.n_kv_heads * l.n : 0;
    if (n > 0 && first[s] + n > p.rows.limit() && p.status) atomicOr(p.status, ST_BAD_PAGE);
  }
  __syncthreads();
  if (tid < 32) {  // exclusive running total
    int carry = 0;
    for (int s0 = 0; s0 < S; s0 += 32) {
      const int v = s0 + tid < S ? before[s0 + tid] : 0;
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (tid >= o) x += y;
      }
      if (s0 + tid < S) before[s0 + tid] = carry + x - v;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (tid == 0) before[S] = carry;
  }
  __syncthreads();
  return before[S];
}

// ------------------------------------------------------------------ producer
// One warp: lane l < CP takes page l of K, lane 16 + l that of V.  The next
// chunk's page numbers and exponents are requested while the current one waits
// for its place in the ring.  A descriptor goes with each chunk; the last one
// says that there are no more.
template <class C>
__device__ void attend_produce(const AttendParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const AttendWork<C>& wk, uint8_t* smem, uint64_t* full, uint64_t* empty) {
  const int lane = threadIdx.x & 31, j = lane & 15;
  const bool is_v = lane >= 16;
  const CUtensorMap* map = is_v ? &vmap : &kmap;
  const uint8_t* exps = is_v ? p.v_exp : p.k_exp;
  const uint64_t pol = policy_evict_first();
  AttendDesc* desc = reinterpret_cast<AttendDesc*>(smem + C::kOffDesc);
  auto page_of = [&](const AttendWalk<C>& k) {
    if (!k.valid || j >= C::CP || !((k.mask >> j) & 1)) return -1;
    return find_page(p.rows, p.n_pages, k.seq, k.base + j * kPage, p.status);
  };
  auto exps_of = [&](const AttendWalk<C>& k, int page) {
    uint4 e = make_uint4(0u, 0u, 0u, 0u);
    if (C::kBf16 || page < 0) return e;
    const size_t ph = (size_t)page * p.n_kv_heads + k.tile.kvh;
    if (p.block == 1) return __ldcg(reinterpret_cast<const uint4*>(exps + ph * kPage));
    e.x = e.y = e.z = e.w = 0x01010101u * __ldcg(exps + ph);
    return e;
  };
  AttendWalk<C> cur;
  cur.start(wk);
  int page = page_of(cur);
  uint4 ex = exps_of(cur, page);
  int n = 0;
  for (;; ++n) {
    const int st = n % C::kStages, use = n / C::kStages;
    AttendWalk<C> nxt = cur;
    int npage = -1;
    if (cur.valid) {
      nxt.next(wk);
      npage = page_of(nxt);
    }
    const bool ok = use == 0 || mbar_wait(&empty[st], (use - 1) & 1);
    if (!__all_sync(0xffffffffu, ok)) {
      if (p.status && lane == 0) atomicOr(p.status, ST_TIMEOUT);
      break;
    }
    const uint32_t got = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
    if (lane == 0) {
      AttendDesc& d = desc[st];
      d.base = cur.base;
      d.loaded = (int)got;
      if (cur.valid) {
        const bool last = !nxt.valid || nxt.fresh || nxt.split != cur.split;
        // whether every row of the tile sees every position of the chunk
        const int cend = cur.base + C::kChunk - 1;
        const bool all = got == (1u << C::CP) - 1u && cend <= cur.t0 &&
                         (p.window <= 0 || cur.base > cur.t1 - p.window || cend < p.sinks);
        d.flags = (cur.fresh ? kDescTile : 0) | (last ? kDescLast : 0) | (all ? 0 : kDescEdge);
        d.split = cur.split;
        if (cur.fresh || last) d.tile = cur.tile;
      } else {
        d.flags = kDescEnd;
      }
      mbar_arrive_expect_tx(&full[st], 2 * __popc(got) * C::kPageBytes);
    }
    if (!C::kBf16 && j < C::CP)
      *reinterpret_cast<uint4*>(smem + C::kOffScale + st * C::kScaleBytes + (is_v ? C::CP * kPage : 0) + j * kPage) = ex;
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[st]);  // after the descriptor and the exponents
    if (!cur.valid) return;
    if (page >= 0) {
      uint8_t* dst = smem + st * C::kStageBytes + ((is_v ? C::CP : 0) + j) * C::kPageBytes;
      const int ph = (p.page0 + page) * p.n_kv_heads + cur.tile.kvh;
      if (C::RB == 64) {
        tma_load_2d(dst, map, 0, ph * 8, &full[st], pol);
      } else {
#pragma unroll
        for (int c = 0; c < C::RB / 128; ++c) tma_load_2d(dst + c * 2048, map, c * 128, ph * kPage, &full[st], pol);
      }
    }
    ex = exps_of(nxt, npage);
    page = npage;
    cur = nxt;
  }
  // (after a timeout) what is still on its way into the ring lands before the CTA ends
  for (int k = n > C::kStages ? n - C::kStages : 0; k < n && lane == 0; ++k)
    mbar_wait(&full[k % C::kStages], (k / C::kStages) & 1);
}

// ------------------------------------------------------------------ consumers
// Named barrier over `count` threads; whether any of them says `v`.
__device__ __forceinline__ bool sync_or(int id, int count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// The sums, maxima and accumulators of a tile in the course of an item, and
// what a chunk does to them.  A lane (g, q4) holds positions g and g + 8 of its
// warp's page (in pos_of_row's order) against query rows 2 q4, 2 q4 + 1 of
// each query tile, then columns g and g + 8 of its warp's units against them.
template <class C>
struct AttendRows {
  static constexpr int N = C::N, CP = C::CP, U = C::U, W = kAttendWarps;
  static constexpr bool kBf16 = C::kBf16;
  const AttendParams& p;
  uint8_t* smem;
  int warp, lane, g, q4;
  float o[U][N][4], m_run[N][2], l_run[N][2];
  uint32_t qr[C::kQRegs ? N * C::NK : 1][2];  // query fragments, where they stay in registers

  __device__ __forceinline__ AttendRows(const AttendParams& p_, uint8_t* smem_) : p(p_), smem(smem_) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    g = lane >> 2;
    q4 = lane & 3;
  }
  __device__ __forceinline__ float* s_max() const { return reinterpret_cast<float*>(smem + C::kOffMax); }
  __device__ __forceinline__ float* s_sum() const { return reinterpret_cast<float*>(smem + C::kOffSum); }
  __device__ __forceinline__ float* s_fac() const { return reinterpret_cast<float*>(smem + C::kOffRow); }
  __device__ __forceinline__ int* s_t() const { return reinterpret_cast<int*>(smem + C::kOffRow) + C::QR; }
  __device__ __forceinline__ int* s_slot() const { return reinterpret_cast<int*>(smem + C::kOffRow) + 2 * C::QR; }
  __device__ __forceinline__ float* s_m() const { return reinterpret_cast<float*>(smem + C::kOffRow) + 3 * C::QR; }
  __device__ __forceinline__ const uint2* s_q() const { return reinterpret_cast<const uint2*>(smem + C::kOffQ) + lane; }
  __device__ __forceinline__ bool sees(int t, int pos) const {
    return pos <= t && (p.window <= 0 || pos > t - p.window || pos < p.sinks);
  }

  // A tile's queries as B fragments, the rows' score factors, positions and
  // output slots.  A piece is 8 elements of one query row; they go to the
  // lanes and k16 steps that meet the same elements of K (a lane's 16-byte
  // unit of a key row, four elements a step).
  __device__ __forceinline__ void queries(const AttendTile& it, int G) {
    constexpr int kPieces = C::QR * C::D / 8, T = W * 32;
    constexpr int kPer = (kPieces + T - 1) / T, kBatch = kPer < 4 ? kPer : 4;
#pragma unroll 1
    for (int u0 = 0; u0 < kPer; u0 += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int v = threadIdx.x + (u0 + u) * T, qi = v / (C::D / 8), c8 = v % (C::D / 8), f = it.f0 + qi;
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if ((kPieces % T == 0 || v < kPieces) && f < it.nf)
          x[u] = __ldcg(reinterpret_cast<const uint4*>(p.q + (int64_t)(it.row0 + f / G) * p.q_stride +
                                                       (it.kvh * G + f % G) * C::D + c8 * 8));
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int v = threadIdx.x + (u0 + u) * T, qi = v / (C::D / 8), c8 = v % (C::D / 8), f = it.f0 + qi;
        float fac = p.scale_log2;
        uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        if (!kBf16) {
          uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
          m = max(m & 0xffffu, m >> 16);
#pragma unroll
          for (int o = C::D / 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          // the row's largest exponent E: q / 2^(E - 127) is below 2 (E = 0, and
          // rows of zeros, count as E = 1; an infinity or NaN makes the row NaN)
          const int E = min(max((int)(m >> 7), 1), 253);
          const float down = __uint_as_float((uint32_t)(254 - E) << 23);
          fac = m >= 0x7f80u ? __uint_as_float(0x7fffffffu)
                             : __fmul_rn(p.scale_log2, __uint_as_float((uint32_t)E << 23));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_f16x2(__fmul_rn(__uint_as_float(w[i] << 16), down),
                              __fmul_rn(__uint_as_float(w[i] & 0xffff0000u), down));
        }
        if (kPieces % T != 0 && v >= kPieces) continue;
        // the 16-byte unit of a key row that holds these elements: its lane and steps
        const int c = kBf16 ? c8 : c8 >> 1;
        const int lane_q = C::RB == 64 ? c : (c & 7) >> 1;
        int k0 = C::RB == 64 ? 0 : (c >> 3) * 2 + (c & 1);
        k0 = kBf16 ? k0 * 2 : k0 * 4 + (c8 & 1) * 2;
        uint2* dst = reinterpret_cast<uint2*>(smem + C::kOffQ) + ((qi >> 3) * C::NK + k0) * 32 + (qi & 7) * 4 + lane_q;
        dst[0] = make_uint2(w[0], w[1]);
        dst[32] = make_uint2(w[2], w[3]);
        if (c8 == 0) {
          s_fac()[qi] = fac;
          s_t()[qi] = it.first + f / G;
          s_slot()[qi] = f < it.nf ? (it.row0 + f / G) * p.n_q_heads + it.kvh * G + f % G : -1;
        }
      }
    }
  }

  __device__ __forceinline__ void open() {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      m_run[n][0] = m_run[n][1] = -INFINITY;
      l_run[n][0] = l_run[n][1] = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) o[u][n][0] = o[u][n][1] = o[u][n][2] = o[u][n][3] = 0.0f;
    }
  }
  __device__ __forceinline__ void keep_queries() {
    if constexpr (C::kQRegs) {
#pragma unroll
      for (int k = 0; k < N * C::NK; ++k) {
        const uint2 v = s_q()[k * 32];
        qr[k][0] = v.x;
        qr[k][1] = v.y;
      }
    }
  }

  // Scores of this warp's page, in log2 units with the value's exponent added,
  // -inf where a row does not see them, and their maxima.  iv: 2^-ev.
  template <bool kEdge>
  __device__ __forceinline__ void scores(uint32_t kbase, const uint8_t* sc, int base, uint32_t loaded,
                                         float (&s)[N][4], float (&iv)[2]) {
#pragma unroll
    for (int n = 0; n < N; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
    const bool have = !kEdge || ((loaded >> warp) & 1);
    const int pos = pos_of_row<kBf16>(g), pos8 = pos_of_row<kBf16>(g + 8);
    if (have) {
      const uint32_t kp = kbase + warp * C::kPageBytes;
      constexpr int kUnits = C::RB / 64;      // 16-byte units of a key row per lane
      constexpr int kSteps = C::NK / kUnits;  // k16 steps per unit
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        uint32_t x[2][4];
        const int c = C::RB == 64 ? q4 : (u >> 1) * 8 + 2 * q4 + (u & 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[h][0]), "=r"(x[h][1]), "=r"(x[h][2]), "=r"(x[h][3])
                       : "r"(kp + page_off<C::RB>(h ? pos8 : pos, c)));
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t a[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            a[h] = kBf16 ? x[h][(2 * k) & 3] : f16x2_of_lo(x[h][k & 3]);
            a[2 + h] = kBf16 ? x[h][(2 * k + 1) & 3] : f16x2_of_hi(x[h][k & 3]);
          }
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const int f = n * C::NK + u * kSteps + k;
            if constexpr (C::kQRegs) {
              mma_16<kBf16>(s[n], a, qr[f][0], qr[f][1]);
            } else {
              const uint2 b = s_q()[f * 32];
              mma_16<kBf16>(s[n], a, b.x, b.y);
            }
          }
        }
      }
    }
    float ks[2], ev[2];
    if (!kBf16) {  // positions pos and pos + 2: two bytes of a word of the page's exponents
      const int sh = 8 * (pos & 3);
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(sc + warp * kPage + (pos & ~3)) >> sh;
      const uint32_t vw = *reinterpret_cast<const uint32_t*>(sc + (CP + warp) * kPage + (pos & ~3)) >> sh;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t bk = (kw >> (16 * h)) & 255u, bv = (vw >> (16 * h)) & 255u;
        ks[h] = __uint_as_float(bk << 23);  // (255: infinity, times a score of zero codes: NaN)
        ev[h] = bv == kExpNaN ? __uint_as_float(0x7fffffffu) : (float)((int)bv - 127);
        iv[h] = exp_byte_inverse((int)bv);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float2 f = reinterpret_cast<const float2*>(s_fac())[n * 4 + q4];
      const int2 t = kEdge ? reinterpret_cast<const int2*>(s_t())[n * 4 + q4] : make_int2(0, 0);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float& x = s[n][2 * h + c];
          const float fc = c ? f.y : f.x;
          x = kBf16 ? __fmul_rn(x, fc) : __fmaf_rn(x, __fmul_rn(fc, ks[h]), ev[h]);
          if (kEdge) x = have && sees(c ? t.y : t.x, base + warp * kPage + (h ? pos8 : pos)) ? x : -INFINITY;
        }
        float mx = fmaxf(s[n][c], s[n][2 + c]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        if (g == 0) s_max()[(n * 8 + 2 * q4 + c) * W + warp] = mx;
      }
    }
  }

  // The scores' weights against the rows' running maxima, to shared memory
  // ([query row][position]); accumulators and sums are scaled to the new maxima.
  template <bool kEdge>
  __device__ __forceinline__ void weights(const float (&s)[N][4], const float (&iv)[2], bool last) {
    uint32_t hi[N][2], lo[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float pv[4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int qi = n * 8 + 2 * q4 + c;
        const float4 a = reinterpret_cast<const float4*>(s_max())[qi];
        const float m = fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), m_run[n][c]);
        // a row that has seen nothing yet: every weight is 2^-inf = 0
        const float ref = m == -INFINITY ? 0.0f : m;
        const float alpha = m == m_run[n][c] ? 1.0f : ex2(__fsub_rn(m_run[n][c], ref));
        m_run[n][c] = m;
        float sum = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = s[n][2 * h + c], e = ex2(__fsub_rn(x, ref));
          pv[2 * h + c] = e;
          if (kBf16)
            sum = __fadd_rn(sum, e);
          else if (kEdge)  // (the exponent of a masked place may be anything)
            sum = x == -INFINITY ? sum : __fmaf_rn(e, iv[h], sum);
          else
            sum = __fmaf_rn(e, iv[h], sum);
        }
        l_run[n][c] = __fmaf_rn(l_run[n][c], alpha, sum);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          o[u][n][c] = __fmul_rn(o[u][n][c], alpha);
          o[u][n][2 + c] = __fmul_rn(o[u][n][2 + c], alpha);
        }
        if (last) {
          float l = l_run[n][c];
          l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 4));
          l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 8));
          l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 16));
          if (g == 0) {
            s_sum()[qi * W + warp] = l;
            if (warp == 0) s_m()[qi] = m;
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (kBf16) {
          hi[n][h] = pack_bf16x2(pv[2 * h], pv[2 * h + 1]);
          lo[n][h] = pack_bf16x2(__fsub_rn(pv[2 * h], bf16r(pv[2 * h])), __fsub_rn(pv[2 * h + 1], bf16r(pv[2 * h + 1])));
        } else {
          hi[n][h] = pack_f16x2(pv[2 * h], pv[2 * h + 1]);
        }
      }
    }
    // matrix h: score rows 8 h .. of the page; lane l gives the row address of
    // query row l mod 8, matrix l / 8 (and the next query tile's above 16)
    const uint32_t at = smem_u32(smem + C::kOffP) + (uint32_t)((lane & 7) * C::kPStride + (warp * kPage + ((lane >> 3) & 1) * 8) * 2);
    if constexpr (N == 1) {
      stsm_x2_trans(at, hi[0][0], hi[0][1]);
      if (kBf16) stsm_x2_trans(at + C::kPBytes, lo[0][0], lo[0][1]);
    } else {
#pragma unroll
      for (int n = 0; n < N; n += 2) {
        const uint32_t a2 = at + (uint32_t)((n + (lane >> 4)) * 8 * C::kPStride);
        stsm_x4_trans(a2, hi[n][0], hi[n][1], hi[n + 1][0], hi[n + 1][1]);
        if (kBf16) stsm_x4_trans(a2 + C::kPBytes, lo[n][0], lo[n][1], lo[n + 1][0], lo[n + 1][1]);
      }
    }
  }

  // An infinity or NaN of a bf16 page in a place that some row does not see
  // must not meet that row's weight of zero: it is taken out here and added to
  // the rows that see it.  (a: columns g, g + 8 of unit u, positions 2 q4, 2 q4
  // + 1 and 8 more of page j; the accumulators of these columns are held by
  // the same quad of lanes.)
  __device__ __forceinline__ void set_apart(int base, int j, int u, uint32_t (&a)[4]) {
    auto bad = [](uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; };
    if (!__any_sync(0xffffffffu, bad(a[0]) || bad(a[1]) || bad(a[2]) || bad(a[3]))) return;
    for (int src = 0; src < 4; ++src)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = __shfl_sync(0xffffffffu, a[k], (lane & ~3) | src);
        for (int e = 0; e < 2; ++e) {
          const uint32_t b = e ? w & 0xffff0000u : w << 16;
          if ((b & 0x7f800000u) != 0x7f800000u) continue;
          const int pos = base + j * kPage + (k >> 1) * 8 + 2 * src + e;
#pragma unroll
          for (int n = 0; n < N; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (sees(s_t()[n * 8 + 2 * q4 + c], pos)) {
                float& x = o[u][n][2 * (k & 1) + c];
                x = __fadd_rn(x, __uint_as_float(b));
              }
        }
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if ((a[k] & 0x7f80u) == 0x7f80u) a[k] &= 0xffff0000u;
      if ((a[k] & 0x7f800000u) == 0x7f800000u) a[k] &= 0x0000ffffu;
    }
  }

  // O^T += V^T P^T on this warp's columns.
  template <bool kEdge>
  __device__ __forceinline__ void values(uint32_t vbase, int base, uint32_t loaded) {
    const uint32_t pt = smem_u32(smem + C::kOffP) + (uint32_t)((lane & 7) * C::kPStride + (lane >> 3) * 16);
#pragma unroll
    for (int j = 0; j < CP; j += 2) {
      if (kEdge && !((loaded >> j) & 3u)) continue;
      // the weights of pages j and j + 1: (b0, b1) of each, for every query tile
      uint32_t b[N][4], bl[kBf16 ? N : 1][4];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const uint32_t at = pt + (uint32_t)(n * 8 * C::kPStride + j * kPage * 2);
        ldsm_x4(at, b[n][0], b[n][1], b[n][2], b[n][3]);
        if (kBf16) ldsm_x4(at + C::kPBytes, bl[kBf16 ? n : 0][0], bl[kBf16 ? n : 0][1], bl[kBf16 ? n : 0][2], bl[kBf16 ? n : 0][3]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t r[4];
        if constexpr (!kBf16)
          ldsm_b8_x2_trans(vbase + (j + (lane >> 4)) * C::kPageBytes + page_off<C::RB>(lane & 15, warp * U + u), r);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // page j + h
          if (kEdge && !((loaded >> (j + h)) & 1u)) continue;
          uint32_t a[4];
          if constexpr (!kBf16) {
            a[0] = f16x2_of_lo(r[2 * h]);
            a[1] = f16x2_of_lo(r[2 * h + 1]);
            a[2] = f16x2_of_hi(r[2 * h]);
            a[3] = f16x2_of_hi(r[2 * h + 1]);
            if (kEdge) {
              // what lies in places that a row does not see may be any byte: a
              // NaN code must not meet its weight of zero
              const uint32_t top = 0x5f005f00u;  // 448
#pragma unroll
              for (int k = 0; k < 4; ++k) asm("min.f16x2 %0, %0, %1;" : "+r"(a[k]) : "r"(top));
            }
          } else {
            ldsm_x4_trans(vbase + (j + h) * C::kPageBytes + page_off<C::RB>(lane & 15, (warp * U + u) * 2 + (lane >> 4)),
                          a[0], a[2], a[1], a[3]);
            if (kEdge) set_apart(base, j + h, u, a);
          }
#pragma unroll
          for (int n = 0; n < N; ++n) {
            mma_16<kBf16>(o[u][n], a, b[n][2 * h], b[n][2 * h + 1]);
            if (kBf16) mma_16<kBf16>(o[u][n], a, bl[kBf16 ? n : 0][2 * h], bl[kBf16 ? n : 0][2 * h + 1]);
          }
        }
      }
    }
  }

  // The item's partial: accumulators from every warp, (max, sum) from the first threads.
  __device__ __forceinline__ void partial(int split) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int slot = s_slot()[n * 8 + 2 * q4 + c];
        if (slot < 0) continue;
        float* dst = p.part_o + ((size_t)slot * p.max_splits + split) * C::D + warp * C::DW + g;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          dst[16 * u] = o[u][n][c];
          dst[16 * u + 8] = o[u][n][2 + c];
        }
      }
    const int tid = threadIdx.x;
    if (tid < C::QR && s_slot()[tid] >= 0) {
      const float4 l = reinterpret_cast<const float4*>(s_sum())[tid];
      p.part_ml[(size_t)s_slot()[tid] * p.max_splits + split] =
          make_float2(s_m()[tid], __fadd_rn(__fadd_rn(l.x, l.y), __fadd_rn(l.z, l.w)));
    }
  }
};

template <class C>
__device__ void attend_consume(const AttendParams& p, int G, uint8_t* smem, uint64_t* full, uint64_t* empty) {
  AttendRows<C> rows(p, smem);
  const AttendDesc* desc = reinterpret_cast<const AttendDesc*>(smem + C::kOffDesc);
  constexpr int T = kAttendWarps * 32;
  for (int i = 0;; ++i) {
    const int st = i % C::kStages;
    // A warp whose wait ran out says so at the chunk's first barrier, where all
    // of them then leave.
    const bool ok = mbar_wait(&full[st], (i / C::kStages) & 1);
    const AttendDesc& d = desc[st];
    const int flags = ok ? d.flags : kDescEnd;
    auto timed_out = [&](bool mine) {
      const bool any = sync_or(2, T, mine);
      if (any && p.status && threadIdx.x == 0) atomicOr(p.status, ST_TIMEOUT);
      return any;
    };
    if (flags & kDescEnd) {
      timed_out(!ok);
      return;
    }
    const int base = d.base;
    const uint32_t loaded = (uint32_t)d.loaded;
    const bool last = flags & kDescLast, tile = flags & kDescTile;
    if (tile) {
      if (timed_out(false)) return;  // and every warp is done with the last tile's queries
      rows.queries(d.tile, G);
      named_sync(2, T);
      rows.keep_queries();
      rows.open();
    }
    const uint32_t kbase = smem_u32(smem + st * C::kStageBytes), vbase = kbase + C::CP * C::kPageBytes;
    const uint8_t* sc = smem + C::kOffScale + st * C::kScaleBytes;
    auto chunk = [&](auto edge) {
      constexpr bool kEdge = decltype(edge)::value;
      float s[C::N][4], iv[2];
      rows.template scores<kEdge>(kbase, sc, base, loaded, s, iv);
      if (tile) named_sync(2, T); else if (timed_out(false)) return false;
      rows.template weights<kEdge>(s, iv, last);
      named_sync(2, T);
      rows.template values<kEdge>(vbase, base, loaded);
      return true;
    };
    if (!((flags & kDescEdge) ? chunk(std::true_type{}) : chunk(std::false_type{}))) return;
    fence_proxy_async_smem();  // reads of the stage precede its next TMA write
    __syncwarp();
    const int split = d.split;
    if (rows.lane == 0) mbar_arrive(&empty[st]);
    if (last) {
      rows.partial(split);
      rows.open();
    }
  }
}

template <int D, int FMT, int N>
__global__ void __launch_bounds__(kAttendThreads, AttendCfg<D, FMT, N>::kPerSm)
    k_attend(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const AttendParams p) {
  using C = AttendCfg<D, FMT, N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kStages;
  int* before = reinterpret_cast<int*>(smem + C::kOffSeq);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 2);  // the bytes' announcement, and the mask and exponents
      mbar_init(&empty[i], kAttendWarps);
    }
    fence_barrier_init();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  pdl_trigger();
  pdl_wait();
  const int S = p.rows.n_seq, G = p.n_q_heads / p.n_kv_heads;
  int *first = before + S + 1, *start = first + S;  // (S + 1 starts)
  AttendWork<C> wk{p, before, first, start, 0, G};
  wk.total = attend_plan<C>(p, G, before, first, start);
  if (threadIdx.x >= kAttendWarps * 32)
    attend_produce<C>(p, kmap, vmap, wk, smem, full, empty);
  else
    attend_consume<C>(p, G, smem, full, empty);
}

// The splits of one (row, query head) merged: out = sum_s o_s 2^(m_s - M) /
// sum_s l_s 2^(m_s - M).  Four warps, warp w adding every fourth split from w
// in order, then the warps in order: a fixed order for the splits that the
// row sees, whatever else is in the call.
template <int D>
__global__ void __launch_bounds__(128) k_attend_merge(const AttendParams p) {
  constexpr int V = D / 32;  // elements per lane: columns V * lane ..
  __shared__ float s_m[4], s_l[4];
  __shared__ float s_o[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x / p.n_q_heads, hq = blockIdx.x % p.n_q_heads;
  pdl_trigger();
  pdl_wait();
  int seq, i;
  if (!find_row(p.rows, r, seq, i)) return;
  const int t = first_of(p.rows, seq) + i;
  const SplitRange sr = splits_seen(t, t, p.window, p.sinks, p.rows.limit(), D);
  const size_t base = ((size_t)r * p.n_q_heads + hq) * p.max_splits;
  float M = -INFINITY;
  for (int j = threadIdx.x; j < sr.n; j += 128) M = fmaxf(M, __ldcg(&p.part_ml[base + sr.at(j)].x));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) s_m[warp] = M;
  __syncthreads();
  M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const float ref = M == -INFINITY ? 0.0f : M;
  float l = 0.0f, acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.0f;
#pragma unroll 4
  for (int j = warp; j < sr.n; j += 4) {
    const size_t slot = base + sr.at(j);
    const float2 ml = __ldcg(&p.part_ml[slot]);
    const float* src = p.part_o + slot * D + lane * V;
    float x[V];
    if constexpr (V == 2) {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
      x[0] = v.x; x[1] = v.y;
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(src + e));
        x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
      }
    }
    const float f = ex2(__fsub_rn(ml.x, ref));
    l = __fmaf_rn(ml.y, f, l);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = __fmaf_rn(x[e], f, acc[e]);
  }
  if (lane == 0) s_l[warp] = l;
#pragma unroll
  for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = acc[e];
  __syncthreads();
  l = __fadd_rn(__fadd_rn(s_l[0], s_l[1]), __fadd_rn(s_l[2], s_l[3]));
  const bool none = l == 0.0f;  // a row that sees nothing: zeros
  bf16* out = p.out + (int64_t)r * p.out_stride + hq * D;
  for (int c = threadIdx.x; c < D; c += 128) {
    const float a = __fadd_rn(__fadd_rn(s_o[0][c], s_o[1][c]), __fadd_rn(s_o[2][c], s_o[3][c]));
    out[c] = __float2bfloat16_rn(none ? 0.0f : __fdiv_rn(a, l));
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[(size_t)r * p.n_q_heads + hq] =
        none ? -INFINITY : __fmul_rn(__fadd_rn(M, log2f(l)), 0.6931471805599453f);
  asm volatile("fence.proxy.async.global;" ::: "memory");  // a context reads it next by bulk copies
}

template <int D, int FMT, int N>
cudaError_t attend_launch_t(const CUtensorMap& kmap, const CUtensorMap& vmap, const AttendParams& p, int num_sms,
                            cudaStream_t s, bool pdl) {
  using C = AttendCfg<D, FMT, N>;
  const int smem = C::smem_bytes(p.rows.n_seq);
  // CTAs per SM at this much shared memory: asked once for each size
  static std::atomic<int64_t> known{0};
  int64_t k = known.load(std::memory_order_relaxed);
  cudaError_t e = cudaSuccess;
  if ((int)(k >> 8) != smem) {
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_attend<D, FMT, N>, kAttendThreads, smem);
    if (e != cudaSuccess) return e;
    k = ((int64_t)smem << 8) | n;
    known.store(k, std::memory_order_relaxed);
  }
  const int per_sm = (int)(k & 255);
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  // a bound on the call's chunks (the lengths are known on the device only)
  const int G = p.n_q_heads / p.n_kv_heads;
  const int64_t tiles = (int64_t)p.rows.n_rows * G / C::QR + p.rows.n_seq;
  const int64_t items = tiles * p.n_kv_heads * (p.rows.limit() / C::kChunk + 1);
  const int64_t grid = std::min<int64_t>(items, (int64_t)num_sms * per_sm);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max<int64_t>(1, grid));
  cfg.blockDim = dim3(kAttendThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, k_attend<D, FMT, N>, kmap, vmap, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)((int64_t)p.rows.n_rows * p.n_q_heads));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;  // the merge may be resident before the partials are complete: it waits for them
  return cudaLaunchKernelEx(&cfg, k_attend_merge<D>, p);
}

// Query tiles of 8, 16, 32 or 64 rows (32 at most for heads of 256): the
// smallest that hold a sequence's rows at once, so that its pages are read and
// widened once.  A row's result is the same in each (the columns of an mma do
// not meet).
template <int D, int FMT>
cudaError_t attend_launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const AttendParams& p, int num_sms,
                          cudaStream_t s, bool pdl) {
  const int64_t f = (int64_t)p.rows.max_rows * (p.n_q_heads / p.n_kv_heads);
  if (f <= 8) return attend_launch_t<D, FMT, 1>(kmap, vmap, p, num_sms, s, pdl);
  if (f <= 16) return attend_launch_t<D, FMT, 2>(kmap, vmap, p, num_sms, s, pdl);
  if (f <= 32 || D == 256) return attend_launch_t<D, FMT, 4>(kmap, vmap, p, num_sms, s, pdl);
  return attend_launch_t<D, FMT, D == 256 ? 4 : 8>(kmap, vmap, p, num_sms, s, pdl);
}

template <int D, int FMT, int N>
cudaError_t attend_prepare_t() {
  using C = AttendCfg<D, FMT, N>;
  return cudaFuncSetAttribute(k_attend<D, FMT, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              C::smem_bytes(kAttendMaxSeq));
}
template <int D, int FMT>
cudaError_t attend_prepare() {
  cudaError_t e;
  if ((e = attend_prepare_t<D, FMT, 1>()) != cudaSuccess || (e = attend_prepare_t<D, FMT, 2>()) != cudaSuccess ||
      (e = attend_prepare_t<D, FMT, 4>()) != cudaSuccess)
    return e;
  return attend_prepare_t<D, FMT, D == 256 ? 4 : 8>();
}

}  // namespace
}  // namespace sv
