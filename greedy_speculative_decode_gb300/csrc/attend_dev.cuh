// attend_dev.cuh -- attention of a ragged batch's rows over a paged cache.
//
// Row i of sequence s stands at position t = first[s] + i and sees the
// positions p <= t, with a window W only those with p > t - W or p < sinks:
//   s_p = scale * q . k_p,  o = sum_p softmax(s)_p v_p,  lse = ln sum_p exp(s_p).
// The cache is read once per tile of 16 MT query rows (token rows x the query
// heads of a kv head, packed one behind the other whatever the group size), so
// few rows are bound by its bytes: a CTA streams chunks of CP pages by TMA
// into a ring and eight warps share each chunk.
//   Scores: warp w takes 2 CP of the chunk's positions (a page, or half of
//     one), all query rows; K goes from 8 to 16 bits in registers.
//   The rows' maxima over the chunk meet in shared memory, each warp writes its
//     weights there in the order the second product reads them, and
//   O += P V: warp w takes D / 8 columns of every position, so the
//     accumulators need no merge between warps.
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

constexpr int kAttendWarps = 8;
constexpr int kAttendThreads = (kAttendWarps + 1) * 32;  // consumers, then the producer warp

// What the producer tells the consumers of a chunk (and, with an item's last
// chunk, of the item after it, whose queries they fetch meanwhile).
struct AttendTile {
  int row0, f0, nf, kvh;  // the sequence's first row, the tile's first query row, the sequence's query rows
  int first;              // position of the sequence's first row
};
struct alignas(16) AttendDesc {
  int base, loaded, flags, split;  // first position; pages in the ring; kDesc*
  AttendTile now, next;
  int pad[2];
};
enum : int { kDescLast = 1, kDescNext = 2, kDescEdge = 4, kDescEnd = 8 };

template <int D_, int FMT_, int MT_>
struct AttendCfg {
  static constexpr int D = D_, FMT = FMT_, MT = MT_;
  static constexpr bool kBf16 = FMT == SV_KV_BF16;
  static constexpr int RB = D * (kBf16 ? 2 : 1);  // bytes of a position's row
  static constexpr int kPageBytes = kPage * RB;
  static constexpr int CP = RB <= 128 ? 8 : 4;    // pages per chunk
  static constexpr int kChunk = CP * kPage;
  static constexpr int kStageBytes = 2 * CP * kPageBytes;
  // ring depth: 96 KB a CTA (64 KB at the smallest rows; 128 KB for rows of 512 bytes)
  static constexpr int kStages = RB == 64 ? 4 : RB == 512 ? 2 : 3;
  static constexpr int kPerSm = RB == 512 || MT == 4 ? 1 : 2;  // CTAs per SM the registers are cut for
  static constexpr int NT = CP / 4;               // 8-position score tiles per warp
  static constexpr int NK = D / 16;               // k16 steps of a score
  static constexpr int DW = D / kAttendWarps;     // output columns per warp
  static constexpr int NO = DW / 8;               // their 8-column tiles
  static constexpr int QR = 16 * MT;              // query rows of a tile
  // shared memory
  static constexpr int kScaleBytes = kBf16 ? 0 : 2 * CP * kPage;
  static constexpr int kOffScale = kStages * kStageBytes;
  static constexpr int kOffQ = kOffScale + kStages * kScaleBytes;    // two A-fragment tiles
  static constexpr int kQBytes = MT * NK * 512;
  static constexpr int kOffP = kOffQ + 2 * kQBytes;                  // weights, A fragments
  static constexpr int kPBytes = MT * CP * 512 * (kBf16 ? 2 : 1);
  static constexpr int kOffMax = kOffP + kPBytes;                    // [QR][8] row maxima
  static constexpr int kOffSum = kOffMax + QR * 32;                  // [QR][8] row sums
  static constexpr int kOffRow = kOffSum + QR * 32;                  // [2][QR] score factors, [2][QR] positions, [QR] maxima
  static constexpr int kOffDesc = kOffRow + 5 * QR * 4;              // [stages] chunk descriptors
  static constexpr int kOffBar = kOffDesc + kStages * (int)sizeof(AttendDesc);
  static constexpr int kOffSeq = kOffBar + 2 * kStages * 8;          // [n_seq + 1] items before, first, row start
  static constexpr int smem_bytes(int n_seq) { return 1024 + kOffSeq + 4 * (3 * n_seq + 2); }
  static_assert(1024 + kOffSeq + 4 * (3 * kAttendMaxSeq + 2) <= 227 * 1024, "shared memory of a CTA");
};

// Position within a page of score column n (0 .. 15).  A value fragment's
// register holds four consecutive positions of an 8-bit page, two of a bf16
// page; the scores take the same order, so weights need no shuffle.
template <bool kBf16>
__device__ __forceinline__ constexpr int pos_of_col(int n) {
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

// One unit of work: a split of a kv head for a tile of query rows.
struct AttendItem {
  AttendTile tile;
  int seq, split;
  int t0, t1;  // positions of the tile's first and last token row
};

template <class C>
struct AttendWork {
  const AttendParams& p;
  const int *before, *first, *start;  // shared memory, per sequence
  int total, G;

  // Work item w: query tiles fastest (they share the split's pages in L2),
  // then kv heads, then splits from the last (the longest) to the first.
  __device__ __forceinline__ void decode(int w, AttendItem& it) const {
    int lo = 0, hi = p.rows.n_seq;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= w) lo = mid; else hi = mid;
    }
    it.seq = lo;
    AttendTile& tl = it.tile;
    tl.first = first[lo];
    tl.row0 = start[lo];
    const int n = start[lo + 1] - tl.row0;
    tl.nf = n * G;
    const int tiles = (tl.nf + C::QR - 1) / C::QR;
    int x = w - before[lo];
    const int tile = x % tiles;
    x /= tiles;
    tl.kvh = x % p.n_kv_heads;
    x /= p.n_kv_heads;
    const SplitRange sr = splits_seen(tl.first, tl.first + n - 1, p.window, p.sinks, p.rows.limit(), C::D);
    it.split = sr.at(sr.n - 1 - x);
    tl.f0 = tile * C::QR;
    it.t0 = tl.first + tl.f0 / G;
    it.t1 = tl.first + (min(tl.f0 + C::QR, tl.nf) - 1) / G;
  }
  // Pages of chunk c of the item that some row of the tile sees, as a mask.
  __device__ __forceinline__ uint32_t seen(const AttendItem& it, int base) const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < C::CP; ++j) {
      const int a = base + j * kPage;
      const bool vis = a <= it.t1 && (p.window <= 0 || a + kPage - 1 > it.t0 - p.window || a < p.sinks);
      m |= (vis ? 1u : 0u) << j;
    }
    return m;
  }
  __device__ __forceinline__ int chunk_end(const AttendItem& it) const {
    return min(min(attn_split_start(it.split + 1, C::D), it.t1 + 1), p.rows.limit());
  }
};

// Walks the CTA's chunks in order: items w, w + step, ..., each from the start
// of its split; chunks and items of which nothing is seen are passed over.
template <class C>
struct AttendWalk {
  AttendItem it;
  int w, base, end;
  uint32_t mask;
  bool valid;

  __device__ __forceinline__ void start(const AttendWork<C>& wk, int w0) {
    w = w0;
    valid = false;
    if (w < wk.total) {
      open(wk);
      settle(wk, gridDim.x);
    }
  }
  __device__ __forceinline__ void open(const AttendWork<C>& wk) {
    wk.decode(w, it);
    base = attn_split_start(it.split, C::D);
    end = wk.chunk_end(it);
  }
  // from (w, base) to the next chunk with a page that is seen
  __device__ __forceinline__ void settle(const AttendWork<C>& wk, int step) {
    for (;;) {
      for (; base < end; base += C::kChunk) {
        mask = wk.seen(it, base);
        if (mask) {
          valid = true;
          return;
        }
      }
      w += step;
      if (w >= wk.total) {
        valid = false;
        return;
      }
      open(wk);
    }
  }
  __device__ __forceinline__ void next(const AttendWork<C>& wk) {
    base += C::kChunk;
    settle(wk, gridDim.x);
  }
};

// Items of each sequence, as running totals in shared memory (all threads).
template <class C>
__device__ int attend_plan(const AttendParams& p, int G, int* before, int* first, int* start) {
  const int tid = threadIdx.x, S = p.rows.n_seq;
  for (int s = tid; s <= S; s += kAttendThreads) 
    // (rows outside the call's buffers are left out)
    start[s] = p.rows.row_start ? min(max(p.rows.row_start[s], 0), p.rows.n_rows) : s * p.rows.rows_each;
  for (int s = tid; s < S; s += kAttendThreads) first[s] = first_of(p.rows, s);
  __syncthreads();
  for (int s = tid; s < S; s += kAttendThreads) {
    const int n = max(0, start[s + 1] - start[s]);
    const int tiles = (n * G + C::QR - 1) / C::QR;
    const SplitRange sr = splits_seen(first[s], first[s] + n - 1, p.window, p.sinks, p.rows.limit(), C::D);
    before[s] = n > 0 ? tiles * p.n_kv_heads * sr.n : 0;
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
    return find_page(p.rows, p.n_pages, k.it.seq, k.base + j * kPage, p.status);
  };
  auto exps_of = [&](const AttendWalk<C>& k, int page) {
    uint4 e = make_uint4(0u, 0u, 0u, 0u);
    if (C::kBf16 || page < 0) return e;
    const size_t ph = (size_t)page * p.n_kv_heads + k.it.tile.kvh;
    if (p.block == 1) return __ldcg(reinterpret_cast<const uint4*>(exps + ph * kPage));
    e.x = e.y = e.z = e.w = 0x01010101u * __ldcg(exps + ph);
    return e;
  };
  AttendWalk<C> cur;
  cur.start(wk, blockIdx.x);
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
        const bool last = !nxt.valid || nxt.w != cur.w;
        // whether every row of the tile sees every position of the chunk
        const int cend = cur.base + C::kChunk - 1;
        const bool all = got == (1u << C::CP) - 1u && cend <= cur.it.t0 &&
                         (p.window <= 0 || cur.base > cur.it.t1 - p.window || cend < p.sinks);
        d.flags = (last ? kDescLast : 0) | (last && nxt.valid ? kDescNext : 0) | (all ? 0 : kDescEdge);
        d.split = cur.it.split;
        d.now = cur.it.tile;
        if (last && nxt.valid) d.next = nxt.it.tile;
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
      const int ph = (p.page0 + page) * p.n_kv_heads + cur.it.tile.kvh;
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
// The query tile as A fragments.  Piece v of a tile is 8 elements of one
// query row; its elements go to the lanes and k16 steps that meet the same
// elements of K (a lane's 16-byte unit c of a key row, four elements a step).
template <class C>
struct QueryTile {
  static constexpr int kPieces = C::QR * C::D / 8;
  static constexpr int kPer = (kPieces + kAttendWarps * 32 - 1) / (kAttendWarps * 32);
  uint4 x[kPer];

  __device__ __forceinline__ void load(const AttendParams& p, const AttendTile& it, int G) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int v = threadIdx.x + u * kAttendWarps * 32, qi = v / (C::D / 8), c8 = v % (C::D / 8);
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      const int f = it.f0 + qi;
      if ((kPieces % (kAttendWarps * 32) == 0 || v < kPieces) && f < it.nf) {
        const int r = it.row0 + f / G, hq = it.kvh * G + f % G;
        x[u] = __ldcg(reinterpret_cast<const uint4*>(p.q + (int64_t)r * p.q_stride + hq * C::D + c8 * 8));
      }
    }
  }
  // to shared memory: fragments [MT][NK][32 lanes], the rows' score factors and positions
  __device__ __forceinline__ void stage(const AttendParams& p, const AttendTile& it, int G, uint8_t* frag,
                                        float* factor, int* tpos) const {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int v = threadIdx.x + u * kAttendWarps * 32, qi = v / (C::D / 8), c8 = v % (C::D / 8);
      float f = p.scale_log2;
      uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      if (!C::kBf16) {
        uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                              __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
        m = max(m & 0xffffu, m >> 16);
#pragma unroll
        for (int o = C::D / 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        // the row's largest exponent E: q / 2^(E - 127) is below 2 (E = 0, and
        // rows of zeros, count as E = 1; an infinity or NaN makes the row NaN)
        const int E = min(max((int)(m >> 7), 1), 253);
        const float down = __uint_as_float((uint32_t)(254 - E) << 23);
        f = m >= 0x7f80u ? __uint_as_float(0x7fffffffu)
                         : __fmul_rn(p.scale_log2, __uint_as_float((uint32_t)E << 23));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = pack_f16x2(__fmul_rn(__uint_as_float(w[i] << 16), down),
                            __fmul_rn(__uint_as_float(w[i] & 0xffff0000u), down));
      }
      if (kPieces % (kAttendWarps * 32) != 0 && v >= kPieces) continue;
      const int mt = qi >> 4, g = qi & 7, hi = (qi >> 3) & 1;
      // 16-byte unit of the key row that holds these elements, its lane and steps
      const int c = C::kBf16 ? c8 : c8 >> 1;
      int lane_q, k0;
      if (C::RB == 64) {
        lane_q = c;
        k0 = 0;
      } else {
        lane_q = (c & 7) >> 1;
        k0 = (c >> 3) * 2 + (c & 1);
      }
      k0 = C::kBf16 ? k0 * 2 : k0 * 4 + (c8 & 1) * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // four elements: a step's (k, k + 1) and (k + 8, k + 9) of the lane
        uint32_t* dst = reinterpret_cast<uint32_t*>(frag + (((mt * C::NK + k0 + i) * 32) + g * 4 + lane_q) * 16);
        dst[hi] = w[2 * i];
        dst[2 + hi] = w[2 * i + 1];
      }
      if (c8 == 0) {
        factor[qi] = f;
        tpos[qi] = it.first + (it.f0 + qi) / G;
      }
    }
  }
};

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
// what a chunk does to them.
template <class C>
struct AttendRows {
  static constexpr int MT = C::MT, CP = C::CP, NT = C::NT, NO = C::NO, W = kAttendWarps;
  static constexpr bool kBf16 = C::kBf16;
  const AttendParams& p;
  uint8_t* smem;
  int warp, lane, g, q4, my_page, my_nt;
  float o[MT][NO][4], m_run[MT][2], l_run[MT][2];

  __device__ __forceinline__ AttendRows(const AttendParams& p_, uint8_t* smem_) : p(p_), smem(smem_) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    g = lane >> 2;
    q4 = lane & 3;
    my_page = NT == 2 ? warp : warp >> 1;
    my_nt = NT == 2 ? 0 : warp & 1;
  }
  __device__ __forceinline__ float* s_max() const { return reinterpret_cast<float*>(smem + C::kOffMax); }
  __device__ __forceinline__ float* s_sum() const { return reinterpret_cast<float*>(smem + C::kOffSum); }
  __device__ __forceinline__ float* s_fac(int qb) const { return reinterpret_cast<float*>(smem + C::kOffRow) + qb * C::QR; }
  __device__ __forceinline__ int* s_t(int qb) const { return reinterpret_cast<int*>(smem + C::kOffRow) + (2 + qb) * C::QR; }
  __device__ __forceinline__ float* s_m() const { return reinterpret_cast<float*>(smem + C::kOffRow) + 4 * C::QR; }
  __device__ __forceinline__ uint4* s_p() const { return reinterpret_cast<uint4*>(smem + C::kOffP); }
  __device__ __forceinline__ bool sees(int t, int pos) const {
    return pos <= t && (p.window <= 0 || pos > t - p.window || pos < p.sinks);
  }

  __device__ __forceinline__ void open() {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        m_run[mt][r] = -INFINITY;
        l_run[mt][r] = 0.0f;
#pragma unroll
        for (int x = 0; x < NO; ++x) o[mt][x][2 * r] = o[mt][x][2 * r + 1] = 0.0f;
      }
  }

  // Scores of this warp's positions of the chunk, in log2 units with the
  // value's exponent added, -inf where a row does not see them.
  // kEdge: some row does not see some position, or a page is not there.
  template <bool kEdge>
  __device__ __forceinline__ void scores(uint32_t kbase, const uint8_t* sc, int base, uint32_t loaded, int qb,
                                         float (&s)[MT][NT][4], float (&iv)[NT][2]) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.0f;
    const bool have = !kEdge || ((loaded >> my_page) & 1);
    if (have) {
      const uint32_t kp = kbase + my_page * C::kPageBytes;
      const uint4* qf = reinterpret_cast<const uint4*>(smem + C::kOffQ + qb * C::kQBytes) + lane;
      constexpr int kUnits = C::RB / 64;               // 16-byte units of a key row per lane
      constexpr int kSteps = C::NK / kUnits;           // k16 steps per unit
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        uint32_t kx[NT][4];
        const int c = C::RB == 64 ? q4 : (u >> 1) * 8 + 2 * q4 + (u & 1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t a = kp + page_off<C::RB>(pos_of_col<kBf16>((my_nt + nt) * 8 + g), c);
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(kx[nt][0]), "=r"(kx[nt][1]), "=r"(kx[nt][2]), "=r"(kx[nt][3])
                       : "r"(a));
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t b0[NT], b1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (kBf16) {
              b0[nt] = kx[nt][(2 * k) & 3];
              b1[nt] = kx[nt][(2 * k + 1) & 3];
            } else {
              b0[nt] = f16x2_of_lo(kx[nt][k & 3]);
              b1[nt] = f16x2_of_hi(kx[nt][k & 3]);
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint4 av = qf[(mt * C::NK + u * kSteps + k) * 32];
            const uint32_t a[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16<kBf16>(s[mt][nt], a, b0[nt], b1[nt]);
          }
        }
      }
    }
    float ks[NT][2], ev[NT][2];
    if (!kBf16) {  // columns 2 q4 + e of tile nt are position 4 q4 + 2 nt + e: four bytes of the page's exponents
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(sc + my_page * kPage + 4 * q4);
      const uint32_t vw = *reinterpret_cast<const uint32_t*>(sc + (CP + my_page) * kPage + 4 * q4);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int sh = 8 * (2 * (my_nt + nt) + e);
          const uint32_t bk = (kw >> sh) & 255u, bv = (vw >> sh) & 255u;
          ks[nt][e] = __uint_as_float(bk << 23);  // (255: infinity, times a score of zero codes: NaN)
          ev[nt][e] = bv == kExpNaN ? __uint_as_float(0x7fffffffu) : (float)((int)bv - 127);
          iv[nt][e] = exp_byte_inverse((int)bv);
        }
    }
    const float* fac = s_fac(qb);
    const int* tp = s_t(qb);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int qi = mt * 16 + g + 8 * r;
        const float f = fac[qi];
        const int t = kEdge ? tp[qi] : 0;
        float mx = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = s[mt][nt][2 * r + e];
            x = kBf16 ? __fmul_rn(x, f) : __fmaf_rn(x, __fmul_rn(f, ks[nt][e]), ev[nt][e]);
            if (kEdge)
              x = have && sees(t, base + my_page * kPage + pos_of_col<kBf16>((my_nt + nt) * 8 + 2 * q4 + e)) ? x
                                                                                                            : -INFINITY;
            mx = fmaxf(mx, x);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (q4 == 0) s_max()[qi * W + warp] = mx;
      }
  }

  // The scores' weights against the rows' running maxima, to shared memory as
  // A fragments; accumulators and sums are scaled to the new maxima.
  template <bool kEdge>
  __device__ __forceinline__ void weights(const float (&s)[MT][NT][4], const float (&iv)[NT][2], bool last) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t hi[2][NT], lo[2][NT];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int qi = mt * 16 + g + 8 * r;
        const float4* mr = reinterpret_cast<const float4*>(s_max() + qi * W);
        const float4 a = mr[0], b = mr[1];
        float m = fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
        m = fmaxf(m, m_run[mt][r]);
        // a row that has seen nothing yet: every weight is 2^-inf = 0
        const float ref = m == -INFINITY ? 0.0f : m;
        const float alpha = m == m_run[mt][r] ? 1.0f : ex2(__fsub_rn(m_run[mt][r], ref));
        m_run[mt][r] = m;
        float sum = 0.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pv[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = s[mt][nt][2 * r + e];
            pv[e] = ex2(__fsub_rn(x, ref));
            if (kBf16)
              sum = __fadd_rn(sum, pv[e]);
            else if (kEdge)  // (the exponent of a masked place may be anything)
              sum = x == -INFINITY ? sum : __fmaf_rn(pv[e], iv[nt][e], sum);
            else
              sum = __fmaf_rn(pv[e], iv[nt][e], sum);
          }
          if (kBf16) {
            hi[r][nt] = pack_bf16x2(pv[0], pv[1]);
            lo[r][nt] = pack_bf16x2(__fsub_rn(pv[0], bf16r(pv[0])), __fsub_rn(pv[1], bf16r(pv[1])));
          } else {
            hi[r][nt] = pack_f16x2(pv[0], pv[1]);
          }
        }
        l_run[mt][r] = __fmaf_rn(l_run[mt][r], alpha, sum);
#pragma unroll
        for (int x = 0; x < NO; ++x) {
          o[mt][x][2 * r] = __fmul_rn(o[mt][x][2 * r], alpha);
          o[mt][x][2 * r + 1] = __fmul_rn(o[mt][x][2 * r + 1], alpha);
        }
        if (last) {
          float l = l_run[mt][r];
          l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 1));
          l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 2));
          if (q4 == 0) {
            s_sum()[qi * W + warp] = l;
            if (warp == 0) s_m()[qi] = m;
          }
        }
      }
      // A fragment of the page's 16 positions: rows (g, g + 8) x columns of (tile 0, tile 1)
      uint4* dst = s_p() + (mt * CP + my_page) * 32 + lane;
      if (NT == 2) {
        *dst = make_uint4(hi[0][0], hi[1][0], hi[0][NT - 1], hi[1][NT - 1]);
        if (kBf16) dst[MT * CP * 32] = make_uint4(lo[0][0], lo[1][0], lo[0][NT - 1], lo[1][NT - 1]);
      } else {
        reinterpret_cast<uint2*>(dst)[my_nt] = make_uint2(hi[0][0], hi[1][0]);
        if (kBf16) reinterpret_cast<uint2*>(dst + MT * CP * 32)[my_nt] = make_uint2(lo[0][0], lo[1][0]);
      }
    }
  }

  // O += P V for page j and column tile x, whose values the lane holds as (b0, b1).
  __device__ __forceinline__ void times(int j, int x, uint32_t b0, uint32_t b1) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint4 av = s_p()[(mt * CP + j) * 32 + lane];
      const uint32_t a[4] = {av.x, av.y, av.z, av.w};
      mma_16<kBf16>(o[mt][x], a, b0, b1);
      if (kBf16) {
        const uint4 lv = s_p()[((MT + mt) * CP + j) * 32 + lane];
        const uint32_t al[4] = {lv.x, lv.y, lv.z, lv.w};
        mma_16<kBf16>(o[mt][x], al, b0, b1);
      }
    }
  }

  // An infinity or NaN of a bf16 page in a place that some row does not see
  // must not meet that row's weight of zero: it is taken out here and added to
  // the rows that see it.  (The lane's words: positions 2 q4, 2 q4 + 1 and 8
  // more of page j, column g of tile x.)
  __device__ __forceinline__ void set_apart(int base, int j, int x, int qb, uint32_t& b0, uint32_t& b1) {
    auto bad2 = [](uint32_t w) {
      return ((w & 0x7f80u) == 0x7f80u ? 1u : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? 2u : 0u);
    };
    const uint32_t bad = bad2(b0) | (bad2(b1) << 2);
    uint32_t who = __ballot_sync(0xffffffffu, bad != 0);
    while (who) {
      const int src = __ffs(who) - 1;
      who &= who - 1;
      const uint32_t w0 = __shfl_sync(0xffffffffu, b0, src), w1 = __shfl_sync(0xffffffffu, b1, src);
      const uint32_t bb = __shfl_sync(0xffffffffu, bad, src);
      const int col = src >> 2, pos0 = base + j * kPage + 2 * (src & 3);
      for (int k = 0; k < 4; ++k) {
        if (!((bb >> k) & 1u) || q4 != col >> 1) continue;
        const uint32_t w = k < 2 ? w0 : w1;
        const float v = __uint_as_float((k & 1) ? w & 0xffff0000u : w << 16);
        const int pos = pos0 + (k >> 1) * 8 + (k & 1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (sees(s_t(qb)[mt * 16 + g + 8 * r], pos)) {
              if (col & 1) o[mt][x][2 * r + 1] = __fadd_rn(o[mt][x][2 * r + 1], v);
              else o[mt][x][2 * r] = __fadd_rn(o[mt][x][2 * r], v);
            }
      }
    }
    if (bad & 1u) b0 &= 0xffff0000u;
    if (bad & 2u) b0 &= 0x0000ffffu;
    if (bad & 4u) b1 &= 0xffff0000u;
    if (bad & 8u) b1 &= 0x0000ffffu;
  }

  // O += P V on this warp's columns.
  template <bool kEdge>
  __device__ __forceinline__ void values(uint32_t vbase, int base, uint32_t loaded, int qb) {
    if constexpr (!kBf16) {
#pragma unroll
      for (int j = 0; j < CP; j += 2) {
        if (kEdge && !((loaded >> j) & 3u)) continue;
#pragma unroll
        for (int u = 0; u < (NO + 1) / 2; ++u) {
          uint32_t r[4];
          ldsm_b8_x2_trans(vbase + (j + (lane >> 4)) * C::kPageBytes + page_off<C::RB>(lane & 15, warp * C::DW / 16 + u), r);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // page j + h
            if (kEdge && !((loaded >> (j + h)) & 1u)) continue;
#pragma unroll
            for (int y = 0; y < (NO == 1 ? 1 : 2); ++y) {  // columns 8 y .. of the 16-column unit
              const uint32_t w = NO == 1 ? ((warp & 1) ? r[2 * h + 1] : r[2 * h]) : r[2 * h + y];
              uint32_t b0 = f16x2_of_lo(w), b1 = f16x2_of_hi(w);
              if (kEdge) {
                // what lies in places that a row does not see may be any byte:
                // a NaN code must not meet its weight of zero
                const uint32_t top = 0x5f005f00u;  // 448
                asm("min.f16x2 %0, %0, %1;" : "+r"(b0) : "r"(top));
                asm("min.f16x2 %0, %0, %1;" : "+r"(b1) : "r"(top));
              }
              times(j + h, NO == 1 ? 0 : 2 * u + y, b0, b1);
            }
          }
        }
      }
    } else {
      auto one = [&](int j, int x, uint32_t b0, uint32_t b1) {
        if (kEdge) {
          if (!((loaded >> j) & 1u)) return;
          set_apart(base, j, x, qb, b0, b1);
        }
        times(j, x, b0, b1);
      };
      if constexpr (NO == 1) {  // one 8-column unit, two pages a load
#pragma unroll
        for (int j = 0; j < CP; j += 2) {
          if (kEdge && !((loaded >> j) & 3u)) continue;
          uint32_t r0, r1, r2, r3;
          ldsm_x4_trans(vbase + (j + (lane >> 4)) * C::kPageBytes + page_off<C::RB>(lane & 15, warp), r0, r1, r2, r3);
          one(j, 0, r0, r1);
          one(j + 1, 0, r2, r3);
        }
      } else {
#pragma unroll
        for (int j = 0; j < CP; ++j) {
          if (kEdge && !((loaded >> j) & 1u)) continue;
#pragma unroll
          for (int x = 0; x < NO; x += 2) {
            uint32_t r0, r1, r2, r3;
            ldsm_x4_trans(vbase + j * C::kPageBytes + page_off<C::RB>(lane & 15, warp * NO + x + (lane >> 4)), r0, r1,
                          r2, r3);
            one(j, x, r0, r1);
            one(j, x + 1, r2, r3);
          }
        }
      }
    }
  }

  // The item's partial: accumulators from every warp, (max, sum) from the first threads.
  __device__ __forceinline__ void partial(const AttendTile& it, int split, int G) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int f = it.f0 + mt * 16 + g + 8 * r;
        if (f >= it.nf) continue;
        const size_t slot = ((size_t)(it.row0 + f / G) * p.n_q_heads + it.kvh * G + f % G) * p.max_splits + split;
        float* dst = p.part_o + slot * C::D + warp * C::DW + 2 * q4;
#pragma unroll
        for (int x = 0; x < NO; ++x)
          *reinterpret_cast<float2*>(dst + 8 * x) = make_float2(o[mt][x][2 * r], o[mt][x][2 * r + 1]);
      }
    const int tid = threadIdx.x, f = it.f0 + tid;
    if (tid < C::QR && f < it.nf) {
      const float* sr = s_sum() + tid * W;
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) l = __fadd_rn(l, sr[w]);
      const size_t slot = ((size_t)(it.row0 + f / G) * p.n_q_heads + it.kvh * G + f % G) * p.max_splits + split;
      p.part_ml[slot] = make_float2(s_m()[tid], l);
    }
  }
};

template <class C>
__device__ void attend_consume(const AttendParams& p, const AttendWork<C>& wk, uint8_t* smem, uint64_t* full,
                               uint64_t* empty) {
  AttendRows<C> rows(p, smem);
  QueryTile<C> qt;
  const AttendDesc* desc = reinterpret_cast<const AttendDesc*>(smem + C::kOffDesc);
  int qb = 0;
  {  // the first item's queries
    AttendWalk<C> w;
    w.start(wk, blockIdx.x);
    if (!w.valid) return;
    qt.load(p, w.it.tile, wk.G);
    qt.stage(p, w.it.tile, wk.G, smem + C::kOffQ, rows.s_fac(0), rows.s_t(0));
  }
  rows.open();
  named_sync(2, kAttendWarps * 32);
  for (int n = 0;; ++n) {
    const int st = n % C::kStages;
    // A warp whose wait ran out says so at the chunk's first barrier, where all
    // of them then leave.
    const bool ok = mbar_wait(&full[st], (n / C::kStages) & 1);
    const AttendDesc& d = desc[st];
    const int flags = ok ? d.flags : kDescEnd;
    if (flags & kDescEnd) {
      if (sync_or(2, kAttendWarps * 32, !ok) && p.status && threadIdx.x == 0) atomicOr(p.status, ST_TIMEOUT);
      return;
    }
    const int base = d.base;
    const uint32_t loaded = (uint32_t)d.loaded;
    const bool last = flags & kDescLast;
    if (flags & kDescNext) qt.load(p, d.next, wk.G);
    const uint32_t kbase = smem_u32(smem + st * C::kStageBytes), vbase = kbase + C::CP * C::kPageBytes;
    const uint8_t* sc = smem + C::kOffScale + st * C::kScaleBytes;
    auto chunk = [&](auto edge) {
      constexpr bool kEdge = decltype(edge)::value;
      float s[C::MT][C::NT][4], iv[C::NT][2];
      rows.template scores<kEdge>(kbase, sc, base, loaded, qb, s, iv);
      if (sync_or(2, kAttendWarps * 32, false)) return false;
      rows.template weights<kEdge>(s, iv, last);
      if (flags & kDescNext)
        qt.stage(p, d.next, wk.G, smem + C::kOffQ + (qb ^ 1) * C::kQBytes, rows.s_fac(qb ^ 1), rows.s_t(qb ^ 1));
      named_sync(2, kAttendWarps * 32);
      rows.template values<kEdge>(vbase, base, loaded, qb);
      return true;
    };
    if (!((flags & kDescEdge) ? chunk(std::true_type{}) : chunk(std::false_type{}))) {
      if (p.status && threadIdx.x == 0) atomicOr(p.status, ST_TIMEOUT);
      return;
    }
    if (last) {
      rows.partial(d.now, d.split, wk.G);
      rows.open();
      qb ^= 1;
    }
    fence_proxy_async_smem();  // reads of the stage precede its next TMA write
    __syncwarp();
    if (rows.lane == 0) mbar_arrive(&empty[st]);
  }
}

template <int D, int FMT, int MT>
__global__ void __launch_bounds__(kAttendThreads, AttendCfg<D, FMT, MT>::kPerSm)
    k_attend(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const AttendParams p) {
  using C = AttendCfg<D, FMT, MT>;
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
    attend_consume<C>(p, wk, smem, full, empty);
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

template <int D, int FMT, int MT>
cudaError_t attend_launch_t(const CUtensorMap& kmap, const CUtensorMap& vmap, const AttendParams& p, int num_sms,
                            cudaStream_t s, bool pdl) {
  using C = AttendCfg<D, FMT, MT>;
  const int smem = C::smem_bytes(p.rows.n_seq);
  // CTAs per SM at this much shared memory: asked once for each size
  static std::atomic<int64_t> known{0};
  int64_t k = known.load(std::memory_order_relaxed);
  cudaError_t e = cudaSuccess;
  if ((int)(k >> 8) != smem) {
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_attend<D, FMT, MT>, kAttendThreads, smem);
    if (e != cudaSuccess) return e;
    k = ((int64_t)smem << 8) | n;
    known.store(k, std::memory_order_relaxed);
  }
  const int per_sm = (int)(k & 255);
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  // a bound on the call's work items (the lengths are known on the device only)
  const int G = p.n_q_heads / p.n_kv_heads;
  const int64_t tiles = (int64_t)p.rows.n_rows * G / C::QR + p.rows.n_seq;
  const int64_t items = tiles * p.n_kv_heads * p.max_splits;
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
  e = cudaLaunchKernelEx(&cfg, k_attend<D, FMT, MT>, kmap, vmap, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)((int64_t)p.rows.n_rows * p.n_q_heads));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;  // the merge may be resident before the partials are complete: it waits for them
  return cudaLaunchKernelEx(&cfg, k_attend_merge<D>, p);
}

// Query tiles of 16, 32 or 64 rows: the smallest that hold a sequence's rows
// at once, so that its pages are read and widened once.  A row's result is
// the same in each (the rows of an mma do not meet).
template <int D, int FMT>
cudaError_t attend_launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const AttendParams& p, int num_sms,
                          cudaStream_t s, bool pdl) {
  const int64_t f = (int64_t)p.rows.max_rows * (p.n_q_heads / p.n_kv_heads);
  if (f <= 16) return attend_launch_t<D, FMT, 1>(kmap, vmap, p, num_sms, s, pdl);
  if (f <= 32 || D == 256) return attend_launch_t<D, FMT, 2>(kmap, vmap, p, num_sms, s, pdl);
  return attend_launch_t<D, FMT, D == 256 ? 2 : 4>(kmap, vmap, p, num_sms, s, pdl);
}

template <int D, int FMT, int MT>
cudaError_t attend_prepare_t() {
  using C = AttendCfg<D, FMT, MT>;
  return cudaFuncSetAttribute(k_attend<D, FMT, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              C::smem_bytes(kAttendMaxSeq));
}
template <int D, int FMT>
cudaError_t attend_prepare() {
  cudaError_t e;
  if ((e = attend_prepare_t<D, FMT, 1>()) != cudaSuccess || (e = attend_prepare_t<D, FMT, 2>()) != cudaSuccess) return e;
  return attend_prepare_t<D, FMT, D == 256 ? 2 : 4>();
}

}  // namespace
}  // namespace sv
