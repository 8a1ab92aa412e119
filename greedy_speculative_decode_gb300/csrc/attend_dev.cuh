// attend_dev.cuh -- attention of a ragged batch's rows over a paged cache.
//
// Row i of sequence s stands at position t = first[s] + i and sees the
// positions p <= t, with a window W only those with p > t - W or p < sinks:
//   s_p = scale * q . k_p,  o = sum_p softmax(s)_p v_p,  lse = ln sum_p exp(s_p).
// The cache is read once per tile of 8 N query rows (token rows x the query
// heads of a kv head, packed one behind the other whatever the group size), so
// few rows are bound by its bytes.  A CTA of four warps takes a split (a range
// of positions) for a kv head and a tile; each warp works by itself on its
// share of the positions, with its own ring of asynchronous copies and its own
// softmax statistics and accumulators, no barrier.  Two pages (one where a
// position's row has 256 bytes or more) at a time:
//   Scores, transposed: S^T = K Q^T.  A page's 16 positions are the 16 rows
//     of an mma, eight query rows its columns, so single-token decode with a
//     group of up to eight heads wastes none of it.  K goes from 8 to 16 bits
//     in registers.
//   Online softmax; the weights are transposed in registers (movmatrix).  The
//     reference that weights are taken against moves only when a row's maximum
//     has risen by more than 2^8 over it (weights reach 2^8, which f16 and fp32
//     hold as exactly as those below one), so accumulators are seldom rescaled.
//     A warp sums at most 64 positions of a split, four warps meet: bf16 values
//     of up to 2^112 stay within fp32 whatever the weights.  (Weights taken
//     times 2^-16 would keep all of them in range, but the tensor cores flush
//     sums below 2^-126: values below 2^-108 would be lost instead.)
//   O^T += V^T P^T, all columns.  A transposing load of bytes makes V's operand
//     (four consecutive positions of a column in a word).
// At the split's end the warps' results meet in shared memory and go out as its
// partial; a second kernel merges the splits.
//
// What bounds it (32 query over 8 kv heads of 128, 8 bits; the call with its
// merge): single-token decode of 32 sequences up to 8192 long 84 us, the
// cache's 432 MB read at 5.6 TB/s; more query rows are bound by the
// instructions around the products and the latency between them (0.45
// instructions a cycle and scheduler): 4 rows at 32768 29 us, 16 sequences of 4
// rows in windows of 4096 45 us, a block of 128 rows at 4096 74 us.
//
// An 8-bit cache's exponents cost an addition each.  The key's scales its
// score; the value's, ev, is added to the score in log2 units, t' = log2(e) s +
// ev, and the weights are p' = 2^(t' - ref): they already carry the value's
// scale, the largest is between 2^-8 and 2^8, and f16 (11 bits, the tensor cores' type that holds
// every e4m3 code) rounds them relative to the largest contribution.  The
// denominator takes p' 2^-ev, unrounded, in fp32.  Queries go to f16 divided
// by a power of two near their row's largest value: exact for elements within
// 2^-17 of it, and below that off by at most 2^-25 of it.  A bf16 cache keeps
// bf16 queries, and the weights are taken as the sum of two bf16 values
// (about 2^-16), since one would shift outputs by up to half a bf16 step.
//
// Splits are ranges of absolute positions (attend_split_start), and a row's
// arithmetic does not depend on the rows, sequences or tiles beside it: a
// page a row does not see leaves its maximum, sum and accumulators as they
// are, bit for bit.  So each row's result is the same in every batch.
#pragma once
#include "paged_dev.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

namespace sv {
namespace {

constexpr int kAttendWarps = 4;  // of a CTA
constexpr int kAttendThreads = kAttendWarps * 32;
constexpr float kAttendSlack = 8.0f;  // log2 of what a row's maximum may exceed its reference by
constexpr float kAttendNone = -3.0e38f;  // reference of a row that has seen nothing (finite: a weight is 2^(-inf) = 0)
constexpr float kAttendFar = -126.0f;  // 2^x is a normal fp32 number from here on

// A tile of query rows.
struct AttendTile {
  int row0, f0, nf, kvh;  // the sequence's first row, the tile's first query row, the sequence's query rows
  int first;              // position of the sequence's first row
};

// CTAs per SM: what the rings (64 KB at rows of 128 bytes, two stages of two
// pages of K and V for each warp) and N D / 4 accumulators a lane leave room for.
__host__ __device__ constexpr int attend_per_sm(int d, bool bf16, int n) {
  const int rb = d * (bf16 ? 2 : 1);
  return rb == 512 ? 1 : n * d >= 512 ? (rb == 256 ? 1 : 2) : rb == 256 ? 2 : n * d <= 64 ? 4 : 3;
}

template <int D_, int FMT_, int N_>
struct AttendCfg {
  static constexpr int D = D_, FMT = FMT_, N = N_;  // N: query tiles of 8 rows
  static constexpr bool kBf16 = FMT == SV_KV_BF16;
  static constexpr int RB = D * (kBf16 ? 2 : 1);  // bytes of a position's row
  static constexpr int kPageBytes = kPage * RB;
  static constexpr int PW = RB <= 128 ? 2 : 1;    // pages a warp takes at a time
  static constexpr int kWarpPos = PW * kPage;     // their positions
  static constexpr int kChunk = kAttendWarps * kWarpPos;
  static constexpr int kStageBytes = 2 * PW * kPageBytes;  // pages of K, pages of V
  static constexpr int kStages = RB == 256 ? 3 : 2;  // of a warp's ring: one at hand, the others on their way
  static constexpr int kPerSm = attend_per_sm(D, kBf16, N);  // CTAs per SM that registers are cut for
  static constexpr int NK = D / 16;               // k16 steps of a score
  static constexpr int U = D / 16;                // 16-column units of the output
  static constexpr int QR = 8 * N;                // query rows of a tile
  static constexpr bool kQRegs = N * NK <= 8;     // query fragments stay in registers
  // the warps' meeting: each leaves its accumulators in the stage it has done
  // with, all columns or a part of them at a time
  static constexpr int kRounds = QR * D * 4 > kStageBytes ? QR * D * 4 / kStageBytes : 1;
  static constexpr int kCols = D / kRounds;
  static_assert(kCols % 32 == 0, "columns of a round");
  // shared memory
  static constexpr int kScaleBytes = kBf16 ? 0 : 2 * PW * kPage;   // exponents of a stage (one a position)
  static constexpr int kRing = kAttendWarps * kStages;             // stages of all warps
  static constexpr int kOffScale = kRing * kStageBytes;
  static constexpr int kOffQ = kOffScale + kRing * kScaleBytes;    // query fragments [N][NK][32 lanes][2 words]
  static constexpr int kQBytes = kQRegs ? 0 : N * NK * 256;
  static constexpr int kOffMl = kOffQ + kQBytes;                   // [QR][4 warps] (reference, sum)
  static constexpr int kOffRow = kOffMl + QR * 32;                 // [QR] score factors, positions, places among the partials
  static constexpr int kOffPlace = kOffRow + 3 * QR * 4;           // [4 warps] the CTA's place in its run
  static constexpr int kOffSeq = kOffPlace + kAttendWarps * 80;    // [n_seq + 1] chunks before, first, row start
  static constexpr int smem_bytes(int n_seq) { return 128 + kOffSeq + 4 * (3 * n_seq + 2); }
  static_assert(128 + kOffSeq + 4 * (3 * kAttendMaxSeq + 2) <= 227 * 1024, "shared memory of a CTA");
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

// l 2^d for d <= 0, also where 2^d by itself is below fp32's range (a
// denominator of values near 2^-100 is large, one of values near 2^100 small).
__device__ __forceinline__ float times_ex2(float l, float d) {
  const float h = __fmul_rn(d, 0.5f);
  return d < kAttendFar ? __fmul_rn(__fmul_rn(l, ex2(h)), ex2(h)) : __fmul_rn(l, ex2(d));
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

// An 8 x 8 matrix of 16-bit values, transposed across the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t r) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(r));
  return d;
}

// The splits a range of rows t0 .. t1 of one sequence sees some position of:
// 0 .. n_sink - 1 and lo .. hi.
struct SplitRange {
  int n_sink, lo, n;  // n: splits in all
  __device__ __forceinline__ int at(int j) const { return j < n_sink ? j : lo + j - n_sink; }
};
// (limit: positions the block table reaches; those beyond are unseen)
__device__ __forceinline__ SplitRange splits_seen(int t0, int t1, int window, int sinks, int limit) {
  SplitRange r = {0, 0, 0};
  t1 = min(t1, limit - 1);
  if (t1 < 0) return r;
  const int hi = attend_split_of(t1);
  const int64_t w0 = (int64_t)t0 - window + 1;
  if (window > 0 && w0 > 0) {
    r.lo = w0 > t1 ? hi + 1 : attend_split_of((int)w0);
    if (sinks > 0) r.n_sink = min(r.lo, attend_split_of(min(sinks - 1, t1)) + 1);
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

// Where a CTA is in its run: a list (sequence, and x = kv head * tiles + tile),
// the place i in it, and the number u of that chunk in the call.
template <class C>
struct AttendPlace {
  AttendTile tile;
  ChunkList list;
  int seq, tiles, x, i, u, end;
  int t0, t1;           // positions of the tile's first and last token row
  int vis_lo, vis_end;  // positions that some row of the tile reaches, sinks apart

  __device__ __forceinline__ bool start(const AttendWork<C>& wk) {
    u = (int)((int64_t)wk.total * blockIdx.x / gridDim.x);
    end = (int)((int64_t)wk.total * (blockIdx.x + 1) / gridDim.x);
    if (u >= end) return false;
    int lo = 0, hi = wk.p.rows.n_seq;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (wk.before[mid] <= u) lo = mid; else hi = mid;
    }
    seq = lo;
    open_seq(wk);
    x = (u - wk.before[seq]) / list.n;
    i = (u - wk.before[seq]) % list.n;
    // to the first item that begins here
    while (i > 0 && i < list.n && split_at(i) == split_at(i - 1)) {
      ++u;
      ++i;
    }
    if (i == list.n) return next_list(wk);
    open_tile(wk);
    return u < end;
  }
  __device__ __forceinline__ int split_at(int k) const { return attend_split_of(list.at(k) * C::kChunk); }
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
    vis_lo = wk.p.window > 0 ? (int)max((int64_t)t0 - wk.p.window + 1, (int64_t)0) : 0;
    vis_end = min(t1 + 1, wk.p.rows.limit());
  }
  // The list's last place of this CTA's run + 1: the items that begin before `end`.
  __device__ __forceinline__ int run_end() const {
    if (list.n - i <= end - u) return list.n;
    int e = i + (end - u);
    while (e < list.n && split_at(e) == split_at(e - 1)) ++e;
    return e;
  }
  // Behind the places i .. e - 1; false: the CTA's work is done.
  __device__ __forceinline__ bool past(const AttendWork<C>& wk, int e) {
    u += e - i;
    i = e;
    return i == list.n && next_list(wk);
  }
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
  // Whether positions a .. a + n - 1 hold one that some row of the tile sees.
  __device__ __forceinline__ bool sees(int a, int n, int sinks) const {
    return a < vis_end && (a + n > vis_lo || a < sinks);
  }
};

// Chunks of each sequence, as running totals in shared memory (all threads).
template <class C>
__device__ int attend_plan(const AttendParams& p, int G, int* before, int* first, int* start) {
  const int tid = threadIdx.x, S = p.rows.n_seq;
  // (rows outside this launch's are left out: a sequence cut by row_lo begins with the position of that row)
  for (int s = tid; s <= S; s += kAttendThreads) {
    const int at = p.rows.row_start ? p.rows.row_start[s] : s * p.rows.rows_each;
    start[s] = min(max(at, p.row_lo), p.row_hi);
    if (s < S)  // (2^30 and up to 2^28 rows; more is a row start below zero)
      first[s] = first_of(p.rows, s) + (int)min(max((int64_t)p.row_lo - at, (int64_t)0), (int64_t)1 << 28);
  }
  __syncthreads();
  bool back = false;  // row starts that decrease: the counts below would not hold
  for (int s = tid; s < S; s += kAttendThreads) {
    const int n = max(0, start[s + 1] - start[s]);
    back |= start[s + 1] < start[s];
    const int tiles = (n * G + C::QR - 1) / C::QR;
    const ChunkList l = chunks_seen<C>(first[s], first[s] + n - 1, p.window, p.sinks, p.rows.limit());
    before[s] = n > 0 ? tiles * p.n_kv_heads * l.n : 0;
    if (n > 0 && first[s] + n > p.rows.limit() && p.status) atomicOr(p.status, ST_BAD_PAGE);
  }
  if (__syncthreads_or(back)) {
    if (tid == 0 && p.status) atomicOr(p.status, ST_BAD_PAGE);
    return 0;
  }
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

// ------------------------------------------------------------------ a warp's loads
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Page `page` of a kv head as a stage's h-th: 2 RB / 64 copies of 16 bytes
// a lane, swizzled as page_off says, and an 8-bit page's exponents (one a
// position).
template <class C>
__device__ __forceinline__ void fetch_page(const AttendParams& p, int page, int kvh, int lane, int h, uint32_t stage,
                                           uint32_t scale) {
  constexpr int kUnitsRow = C::RB / 16, kPer = C::kPageBytes / 512;  // units of a row; copies of a lane
  const size_t ph = (size_t)page * p.n_kv_heads + kvh;
  const uint8_t* k = p.k + ph * C::kPageBytes + lane * 16;
  const uint8_t* v = p.v + ph * C::kPageBytes + lane * 16;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    const uint32_t dst = stage + h * C::kPageBytes + page_off<C::RB>(e / kUnitsRow, e % kUnitsRow);
    copy16(dst, k + 512 * i);
    copy16(dst + C::PW * C::kPageBytes, v + 512 * i);
  }
  if (!C::kBf16 && p.block == 1 && lane < 2)
    copy16(scale + (C::PW * lane + h) * kPage, (lane ? p.v_exp : p.k_exp) + ph * kPage);
}

// ------------------------------------------------------------------ the arithmetic
// The statistics and accumulators of a warp in the course of a split.  A lane
// (g, q4) holds positions g and g + 8 of a page (in pos_of_row's order)
// against query rows 2 q4, 2 q4 + 1 of each query tile, then columns g and
// g + 8 of each unit against them.
template <class C>
struct AttendRows {
  static constexpr int N = C::N, U = C::U, PW = C::PW;
  static constexpr bool kBf16 = C::kBf16;
  const AttendParams& p;
  uint2* s_q;  // query fragments in shared memory, where they do not stay in registers
  uint8_t* smem;
  int warp, lane, g, q4;
  float o[U][N][4], m_run[N][2], l_run[N][2];
  uint32_t qr[C::kQRegs ? N * C::NK : 1][2];

  __device__ __forceinline__ AttendRows(const AttendParams& p_, uint8_t* smem_) : p(p_), smem(smem_) {
    warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    lane = threadIdx.x & 31;
    g = lane >> 2;
    q4 = lane & 3;
    s_q = reinterpret_cast<uint2*>(smem + C::kOffQ) + lane;
  }
  __device__ __forceinline__ float* s_fac() const { return reinterpret_cast<float*>(smem + C::kOffRow); }
  __device__ __forceinline__ int* s_t() const { return reinterpret_cast<int*>(smem + C::kOffRow) + C::QR; }
  __device__ __forceinline__ int* s_slot() const { return reinterpret_cast<int*>(smem + C::kOffRow) + 2 * C::QR; }
  __device__ __forceinline__ bool sees(int t, int pos) const {
    return pos <= t && (p.window <= 0 || pos > t - p.window || pos < p.sinks);
  }

  // A tile's queries as B fragments.  Lane (g, q4) takes row g of each query
  // tile, the elements it meets in K: its 16-byte units of a key row, four
  // elements a k16 step.  (Every warp writes the same to shared memory, and
  // reads back its own.  The warps meet between two tiles' queries, see
  // attend_cta, so none finds another tile's.)
  __device__ __forceinline__ void queries(const AttendTile& it, int G) {
    constexpr int kUnits = C::RB / 64, kV = kBf16 ? 1 : 2, kSteps = C::NK / kUnits;  // kV: 16-byte loads a unit
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int f = it.f0 + n * 8 + g;
      const bf16* row = p.q + (int64_t)(it.row0 + f / G) * p.q_stride + (it.kvh * G + f % G) * C::D;
      uint4 x[kUnits][kV];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int c = C::RB == 64 ? q4 : (u >> 1) * 8 + 2 * q4 + (u & 1);
#pragma unroll
        for (int v = 0; v < kV; ++v)
          x[u][v] = f < it.nf ? __ldcg(reinterpret_cast<const uint4*>(row) + c * kV + v) : make_uint4(0u, 0u, 0u, 0u);
      }
      float down = 1.0f, up = p.scale_log2;
      if (!kBf16) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
#pragma unroll
          for (int v = 0; v < kV; ++v)
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[u][v].x & 0x7fff7fffu, x[u][v].y & 0x7fff7fffu),
                                     __vmaxu2(x[u][v].z & 0x7fff7fffu, x[u][v].w & 0x7fff7fffu)));
        m = max(m & 0xffffu, m >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // the row's largest exponent E: q / 2^(E - 127) is below 2 (E = 0, and
        // rows of zeros, count as E = 1; an infinity or NaN makes the row NaN)
        const int E = min(max((int)(m >> 7), 1), 253);
        down = __uint_as_float((uint32_t)(254 - E) << 23);
        up = m >= 0x7f80u ? __uint_as_float(0x7fffffffu) : __fmul_rn(p.scale_log2, __uint_as_float((uint32_t)E << 23));
      }
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const uint4 w = x[u][kBf16 ? 0 : k >> 1];
          uint32_t b0 = (k & 1) ? w.z : w.x, b1 = (k & 1) ? w.w : w.y;
          if (!kBf16) {
            b0 = pack_f16x2(__fmul_rn(__uint_as_float(b0 << 16), down), __fmul_rn(__uint_as_float(b0 & 0xffff0000u), down));
            b1 = pack_f16x2(__fmul_rn(__uint_as_float(b1 << 16), down), __fmul_rn(__uint_as_float(b1 & 0xffff0000u), down));
          }
          const int at = n * C::NK + u * kSteps + k;
          if constexpr (C::kQRegs) {
            qr[at][0] = b0;
            qr[at][1] = b1;
          } else {
            s_q[at * 32] = make_uint2(b0, b1);
          }
        }
      // the rows' score factors, positions and places among the partials (-1: no row)
      if (q4 == 0) {
        s_fac()[n * 8 + g] = up;
        s_t()[n * 8 + g] = it.first + f / G;
        s_slot()[n * 8 + g] = f < it.nf ? (it.row0 - p.row_lo + f / G) * p.n_q_heads + it.kvh * G + f % G : -1;
      }
    }
    __syncwarp();
  }

  __device__ __forceinline__ void open() {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      m_run[n][0] = m_run[n][1] = kAttendNone;
      l_run[n][0] = l_run[n][1] = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) o[u][n][0] = o[u][n][1] = o[u][n][2] = o[u][n][3] = 0.0f;
    }
  }

  // An infinity or NaN of a bf16 page in a place that some row does not see
  // must not meet that row's weight of zero: it is taken out here and added to
  // the rows that see it, whose accumulators it makes infinite or NaN.  On a
  // page that all rows see the products do that; which of the two comes out
  // is decided at the end (far_value).  (a: columns g, g + 8 of unit u, positions 2 q4, 2 q4
  // + 1 and 8 more of the page; the accumulators of these columns are held by
  // the same quad of lanes.)
  __device__ __forceinline__ void set_apart(int base, bool have, int u, uint32_t (&a)[4]) {
    auto bad = [](uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; };
    if (!__any_sync(0xffffffffu, bad(a[0]) || bad(a[1]) || bad(a[2]) || bad(a[3]))) return;
    for (int src = 0; src < 4; ++src)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = __shfl_sync(0xffffffffu, a[k], (lane & ~3) | src);
        for (int e = 0; e < 2; ++e) {
          const uint32_t b = e ? w & 0xffff0000u : w << 16;
          if ((b & 0x7f800000u) != 0x7f800000u) continue;
          const int pos = base + (k >> 1) * 8 + 2 * src + e;
#pragma unroll
          for (int n = 0; n < N; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (have && sees(s_t()[n * 8 + 2 * q4 + c], pos)) {
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

  // The warp's pages of a chunk: scores in log2 units with the value's exponent added, -inf
  // where a row does not see the position; the references and sums; O^T.
  // kEdge: some row does not see some position, or a page is not there (have).
  template <bool kEdge>
  __device__ __forceinline__ void pages(uint32_t kp, const uint8_t* sc, int base, uint32_t have, const uint32_t (&ke)[PW],
                                        const uint32_t (&ve)[PW]) {
    const uint32_t vp = kp + PW * C::kPageBytes;
    const int pos = pos_of_row<kBf16>(g), pos8 = pos_of_row<kBf16>(g + 8);
    // The lane's positions, two a page: key scale, value exponent ev and 2^-ev.  A byte
    // of 255 makes the score 0 * inf and ev inf * 0: NaN.
    float ks[PW][2], ev[PW][2], iv[PW][2];
    if (!kBf16) {
#pragma unroll
      for (int j = 0; j < PW; ++j) {
        uint32_t kw, vw;
        if (p.block == 1) {  // positions pos and pos + 2: two bytes of a word of the page's exponents
          const uint8_t* w = sc + j * kPage + (pos & ~3);
          kw = *reinterpret_cast<const uint32_t*>(w) >> (8 * (pos & 3));
          vw = *reinterpret_cast<const uint32_t*>(w + PW * kPage) >> (8 * (pos & 3));
        } else {
          kw = ke[j] * 0x00010001u;
          vw = ve[j] * 0x00010001u;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (bytes below the writer's smallest, as a zeroed cache has, count as that one:
          // 2^-ev of a block of zeros stays in range)
          const uint32_t bk = (kw >> (16 * h)) & 255u, bv = max((vw >> (16 * h)) & 255u, (uint32_t)kExpMinByte);
          ks[j][h] = __uint_as_float(bk << 23);
          iv[j][h] = __uint_as_float((254u - bv) << 23);
          // 2^23 + bv as a float, less 2^23 + 127
          ev[j][h] = __fmaf_rn(__uint_as_float(bv << 23), 0.0f, __fsub_rn(__uint_as_float(0x4b000000u | bv), 8388735.0f));
        }
      }
    }
    float s[PW][N][4];
#pragma unroll
    for (int j = 0; j < PW; ++j)
#pragma unroll
      for (int n = 0; n < N; ++n) s[j][n][0] = s[j][n][1] = s[j][n][2] = s[j][n][3] = 0.0f;
    constexpr int kUnits = C::RB / 64;      // 16-byte units of a key row per lane
    constexpr int kSteps = C::NK / kUnits;  // k16 steps per unit
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      uint32_t x[PW][2][4];
      const int c = C::RB == 64 ? q4 : (u >> 1) * 8 + 2 * q4 + (u & 1);
#pragma unroll
      for (int j = 0; j < PW; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[j][h][0]), "=r"(x[j][h][1]), "=r"(x[j][h][2]), "=r"(x[j][h][3])
                       : "r"(kp + j * C::kPageBytes + page_off<C::RB>(h ? pos8 : pos, c)));
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t a[PW][4];
#pragma unroll
        for (int j = 0; j < PW; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            a[j][h] = kBf16 ? x[j][h][(2 * k) & 3] : f16x2_of_lo(x[j][h][k & 3]);
            a[j][2 + h] = kBf16 ? x[j][h][(2 * k + 1) & 3] : f16x2_of_hi(x[j][h][k & 3]);
          }
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int f = n * C::NK + u * kSteps + k;
          uint32_t b0, b1;
          if constexpr (C::kQRegs) {
            b0 = qr[f][0];
            b1 = qr[f][1];
          } else {
            const uint2 b = s_q[f * 32];
            b0 = b.x;
            b1 = b.y;
          }
#pragma unroll
          for (int j = 0; j < PW; ++j) mma_16<kBf16>(s[j][n], a[j], b0, b1);
        }
      }
    }
    float top[N][2], low = 0.0f;
    bool rise = false;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float fc = s_fac()[n * 8 + 2 * q4 + c];
        const int t = kEdge ? s_t()[n * 8 + 2 * q4 + c] : 0;
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < PW; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& x = s[j][n][2 * h + c];
            x = kBf16 ? __fmul_rn(x, fc) : __fmaf_rn(__fmul_rn(x, fc), ks[j][h], ev[j][h]);
            if (kEdge)
              x = ((have >> j) & 1u) && sees(t, base + j * kPage + (h ? pos8 : pos)) ? x : -INFINITY;
            m = fmaxf(m, x);
          }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        top[n][c] = m;
        rise |= m > __fadd_rn(m_run[n][c], kAttendSlack);
      }
    if (__any_sync(0xffffffffu, rise)) {
      float alpha[N][2];
      bool scaled = false;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const bool up = top[n][c] > __fadd_rn(m_run[n][c], kAttendSlack);
          const float d = up ? __fsub_rn(m_run[n][c], top[n][c]) : 0.0f;
          alpha[n][c] = ex2(d);
          l_run[n][c] = times_ex2(l_run[n][c], d);
          scaled |= up && m_run[n][c] != kAttendNone;  // (behind a row's first pages there is nothing to scale)
          m_run[n][c] = up ? top[n][c] : m_run[n][c];
        }
      if (__any_sync(0xffffffffu, scaled)) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[u][n][e] = __fmul_rn(o[u][n][e], alpha[n][e & 1]);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < PW; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& x = s[j][n][2 * h + c];
            x = __fsub_rn(x, m_run[n][c]);
            if (!kBf16) low = fminf(low, kEdge && x == -INFINITY ? 0.0f : x);
          }
    // The weights and, in the denominators, p' 2^-ev.  Where p' itself is below
    // fp32's range the latter need not be (a block of zeros has ev = -100): it
    // is then 2^(log2(e) s - ref) directly.
    uint32_t hi[PW][N][2], lo[kBf16 ? PW : 1][N][2];
    auto weights = [&](auto far) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < PW; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& x = s[j][n][2 * h + c];
              const float e = ex2(x);
              float y;
              if (kBf16)
                y = __fadd_rn(sum, e);
              else if (far.value && x < kAttendFar)
                y = __fadd_rn(sum, ex2(__fsub_rn(x, ev[j][h])));
              else
                y = __fmaf_rn(e, iv[j][h], sum);
              // (the exponent of a masked place may be anything)
              sum = kEdge && !kBf16 && x == -INFINITY ? sum : y;
              x = e;
            }
          l_run[n][c] = __fadd_rn(l_run[n][c], sum);
        }
#pragma unroll
        for (int j = 0; j < PW; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float x = s[j][n][2 * h], y = s[j][n][2 * h + 1];
            if (kBf16) {
              hi[j][n][h] = transposed(pack_bf16x2(x, y));
              lo[kBf16 ? j : 0][n][h] = transposed(pack_bf16x2(__fsub_rn(x, bf16r(x)), __fsub_rn(y, bf16r(y))));
            } else {
              hi[j][n][h] = transposed(pack_f16x2(x, y));
            }
          }
      }
    };
    if (!kBf16 && __any_sync(0xffffffffu, low < kAttendFar)) weights(std::true_type());
    else weights(std::false_type());
#pragma unroll
    for (int u = 0; u < U; u += 2) {
#pragma unroll
      for (int j = 0; j < PW; ++j) {
        const uint32_t vj = vp + j * C::kPageBytes;
        uint32_t r[4];
        if constexpr (!kBf16) ldsm_b8_x2_trans(vj + page_off<C::RB>(lane & 15, u + (lane >> 4)), r);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t a[4];
          if constexpr (!kBf16) {
            a[0] = f16x2_of_lo(r[2 * y]);
            a[1] = f16x2_of_lo(r[2 * y + 1]);
            a[2] = f16x2_of_hi(r[2 * y]);
            a[3] = f16x2_of_hi(r[2 * y + 1]);
            if (kEdge) {
              // what lies in places that a row does not see may be any byte: a
              // NaN code must not meet its weight of zero
              const uint32_t top = 0x5f005f00u;  // 448
#pragma unroll
              for (int k = 0; k < 4; ++k) asm("min.f16x2 %0, %0, %1;" : "+r"(a[k]) : "r"(top));
            }
          } else {
            ldsm_x4_trans(vj + page_off<C::RB>(lane & 15, (u + y) * 2 + (lane >> 4)), a[0], a[2], a[1], a[3]);
            if (kEdge) set_apart(base + j * kPage, (have >> j) & 1u, u + y, a);
          }
#pragma unroll
          for (int n = 0; n < N; ++n) {
            mma_16<kBf16>(o[u + y][n], a, hi[j][n][0], hi[j][n][1]);
            if (kBf16) mma_16<kBf16>(o[u + y][n], a, lo[kBf16 ? j : 0][n][0], lo[kBf16 ? j : 0][n][1]);
          }
        }
      }
    }
  }

  // The split's partial: the four warps' results merged in warp order.  `left`:
  // the stage each warp has done with, kRing / 4 stages apart.  (Columns are
  // stored at c ^ 8 (row / 2 mod 4): the lanes of a store meet 32 banks.)
  __device__ __forceinline__ void partial(int split, uint8_t* left) {
    constexpr int W = kAttendWarps, T = kAttendThreads, kStride = C::kStages * C::kStageBytes;
    float2* s_ml = reinterpret_cast<float2*>(smem + C::kOffMl);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = l_run[n][c];
        l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 4));
        l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 8));
        l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 16));
        if (g == 0) s_ml[(n * 8 + 2 * q4 + c) * W + warp] = make_float2(m_run[n][c], l);
      }
    constexpr int kUR = U / C::kRounds, kV = C::kCols / 4;  // units and float4 columns of a round
    __syncwarp();                                           // every lane has read its pages
#pragma unroll
    for (int rd = 0; rd < C::kRounds; ++rd) {
      float* mine = reinterpret_cast<float*>(left + warp * kStride);
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int u = 0; u < kUR; ++u) {
            float* dst = mine + (n * 8 + 2 * q4 + c) * C::kCols;
            dst[(16 * u + g) ^ (8 * q4)] = o[rd * kUR + u][n][c];
            dst[(16 * u + 8 + g) ^ (8 * q4)] = o[rd * kUR + u][n][2 + c];
          }
      named_sync(2, T);
      // T / QR threads a query row, each every (T / QR)-th float4 of it
      constexpr int kPer = T / C::QR;
      const int qi = threadIdx.x / kPer, slot = s_slot()[qi];
      if (slot >= 0) {
        float2 ml[W];
        float M = kAttendNone, l = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          ml[w] = s_ml[qi * W + w];
          M = fmaxf(M, ml[w].x);
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float d = __fsub_rn(ml[w].x, M);
          ml[w].x = ex2(d);
          l = __fadd_rn(l, times_ex2(ml[w].y, d));
        }
        const size_t at = (size_t)slot * p.max_splits + split;
        if (rd == 0 && threadIdx.x % kPer == 0) p.part_ml[at] = make_float2(M, l);
        float* dst = p.part_o + at * C::D + rd * C::kCols;
#pragma unroll
        for (int v = threadIdx.x % kPer; v < kV; v += kPer) {
          float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(left + w * kStride) +
                                                              qi * C::kCols + ((4 * v) ^ (8 * ((qi >> 1) & 3))));
            a.x = __fmaf_rn(x.x, ml[w].x, a.x);
            a.y = __fmaf_rn(x.y, ml[w].x, a.y);
            a.z = __fmaf_rn(x.z, ml[w].x, a.z);
            a.w = __fmaf_rn(x.w, ml[w].x, a.w);
          }
          *reinterpret_cast<float4*>(dst + 4 * v) = a;
        }
      }
      named_sync(2, T);  // the stages, and s_ml, are free again
    }
  }
};

// A CTA's run, list by list.
template <class C>
__device__ void attend_cta(const AttendParams& p, const AttendWork<C>& wk, uint8_t* smem) {
  constexpr int S = C::kStages, PW = C::PW;
  AttendPlace<C> at;
  bool waited = !p.early;
  if (!at.start(wk)) {
    if (!waited) pdl_wait();  // so that the grid completes in order
    return;
  }
  AttendRows<C> rows(p, smem);
  const int warp = rows.warp, lane = rows.lane;
  const uint32_t ring = smem_u32(smem) + warp * S * C::kStageBytes;
  const uint8_t* scales = smem + C::kOffScale + warp * S * C::kScaleBytes;
  const uint32_t scales_at = smem_u32(scales);
  // (What only the next list needs of the place waits in shared memory, so that
  // the loop over a list has the registers.)
  static_assert(sizeof(AttendPlace<C>) <= 80, "a warp's place");
  volatile int* kept = reinterpret_cast<int*>(smem + C::kOffPlace + warp * 80);
  constexpr int kWords = sizeof(AttendPlace<C>) / 4;
  for (;;) {
    const int run = at.run_end();
    const int* table = p.rows.table + (size_t)at.seq * p.rows.table_stride;
    // This warp's pages of place j of the list that the tile sees something of
    // (a mask), and their numbers.  (Loaded a place ahead of their use, and
    // looked at only then: nothing here waits for the load.)
    auto pages_of = [&](int j, int (&pg)[PW]) {
      const int a = at.list.at(j) * C::kChunk + warp * C::kWarpPos;
      uint32_t seen = 0;
#pragma unroll
      for (int h = 0; h < PW; ++h) {
        if (j >= run || !at.sees(a + h * kPage, kPage, p.sinks)) continue;
        seen |= 1u << h;
        pg[h] = __ldg(table + a / kPage + h);
      }
      return seen;
    };
    auto request = [&](int st, uint32_t seen, const int (&pg)[PW], uint32_t& have, uint32_t (&ke)[PW], uint32_t (&ve)[PW]) {
      have = 0;
#pragma unroll
      for (int h = 0; h < PW; ++h) {
        ke[h] = ve[h] = 0;
        if (!((seen >> h) & 1u)) continue;
        if ((uint32_t)pg[h] >= (uint32_t)p.n_pages) {
          if (p.status && lane == 0) atomicOr(p.status, ST_BAD_PAGE);
          continue;
        }
        have |= 1u << h;
        fetch_page<C>(p, pg[h], at.tile.kvh, lane, h, ring + st * C::kStageBytes, scales_at + st * C::kScaleBytes);
        if (!C::kBf16 && p.block != 1) {
          const size_t ph = (size_t)pg[h] * p.n_kv_heads + at.tile.kvh;
          ke[h] = __ldg(p.k_exp + ph);
          ve[h] = __ldg(p.v_exp + ph);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // of places i, i + 1, ..: pages that are there, and a page's one exponent
    uint32_t have[S], ke[S][PW], ve[S][PW];
    int ahead[PW] = {};
    uint32_t seen;
#pragma unroll
    for (int k = 0; k < S - 1; ++k) {
      seen = pages_of(at.i + k, ahead);
      if (!waited && (at.i + k >= run || (at.list.at(at.i + k) + 1) * C::kChunk > at.tile.first)) {
        pdl_wait();  // the call's own rows are among these positions
        waited = true;
      }
      request(k, seen, ahead, have[k], ke[k], ve[k]);
    }
    seen = pages_of(at.i + S - 1, ahead);
    if (!waited) pdl_wait();
    waited = true;
    rows.queries(at.tile, wk.G);
    rows.open();
    {
      int w[kWords];
      memcpy(w, &at, sizeof w);
#pragma unroll
      for (int k = 0; k < kWords; ++k) kept[k] = w[k];  // (every lane the same)
    }
    bool any = false;  // the item has a chunk that the tile sees
    bool met = false;  // the warps have met since they wrote the queries
    int st = 0;
    for (int i = at.i; i < run; ++i) {
      // the pages S - 1 places on, into the stage that place i - 1 had (every lane has done with it)
      __syncwarp();
      request(st == 0 ? S - 1 : st - 1, seen, ahead, have[S - 1], ke[S - 1], ve[S - 1]);
      seen = pages_of(i + S, ahead);
      const int chunk = at.list.at(i) * C::kChunk, base = chunk + warp * C::kWarpPos;
      if (at.sees(chunk, C::kChunk, p.sinks)) any = true;
      if (have[0]) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        __syncwarp();
        const uint32_t kp = ring + st * C::kStageBytes;
        const uint8_t* sc = scales + st * C::kScaleBytes;
        // whether every row of the tile sees every position of the pages
        const int e = base + C::kWarpPos - 1;
        const bool all = have[0] == (1u << PW) - 1u && e <= at.t0 &&
                         (p.window <= 0 || base > at.t1 - p.window || e < p.sinks);
        if (all) rows.template pages<false>(kp, sc, base, have[0], ke[0], ve[0]);
        else rows.template pages<true>(kp, sc, base, have[0], ke[0], ve[0]);
      }
#pragma unroll
      for (int k = 0; k < S - 1; ++k) {
        have[k] = have[k + 1];
#pragma unroll
        for (int h = 0; h < PW; ++h) {
          ke[k][h] = ke[k + 1][h];
          ve[k][h] = ve[k + 1][h];
        }
      }
      uint8_t* left = smem + st * C::kStageBytes;
      st = st + 1 == S ? 0 : st + 1;
      const int split = attend_split_of(chunk);
      if (i + 1 == run || attend_split_of(at.list.at(i + 1) * C::kChunk) != split) {
        if (any) {
          rows.partial(split, left);
          rows.open();
          met = true;
        }
        any = false;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    {
      int w[kWords];
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[k] = kept[k];
      memcpy(&at, w, sizeof w);
    }
    if (!at.past(wk, run)) return;
    // Every lane is done with this tile's stages.  A run that held nothing the
    // tile sees (the later chunks of an early tile, those before a late tile's
    // window, rows of padding) had no meeting: without one a warp still at its
    // queries would write them over the next tile's.
    __syncwarp();
    if (!met) named_sync(2, kAttendThreads);
  }
}

template <int D, int FMT, int N>
__global__ void __launch_bounds__(kAttendThreads, AttendCfg<D, FMT, N>::kPerSm) k_attend(const AttendParams p) {
  using C = AttendCfg<D, FMT, N>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  // (an offset, not a rounded address: the compiler keeps knowing that this is shared memory)
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 127u);
  int* before = reinterpret_cast<int*>(smem + C::kOffSeq);
  pdl_trigger();
  if (!p.early) pdl_wait();
  const int S = p.rows.n_seq, G = p.n_q_heads / p.n_kv_heads;
  int *first = before + S + 1, *start = first + S;  // (S + 1 starts)
  AttendWork<C> wk{p, before, first, start, 0, G};
  wk.total = attend_plan<C>(p, G, before, first, start);
  attend_cta<C>(p, wk, smem);
}

// Column c of a row's output over a bf16 cache where the sum of its splits came
// out as an infinity or a NaN.
//   The row sees an infinity: hi x + lo x is a NaN where a weight's second term
// is zero or negative, and so is an infinity rescaled by a factor too small for
// fp32.  Weights are positive, so the output is the sum of the row's infinite
// values (a NaN, if there is one or if they have both signs), whatever tile the
// row was part of.  Splits with a finite partial hold none.
//   It sees none: finite partials have a sum beyond fp32.  It is taken again of
// their 2^-24-fold (2^8 for a weight, 2^16 for the splits), and the mean is
// finite.
// M: the largest reference, l: the sum of the weights.
template <int D>
__device__ __noinline__ float far_value(const AttendParams& p, const SplitRange& sr, size_t base, int seq, int t, int kvh,
                                        int c, float M, float l) {
  const int* table = p.rows.table + (size_t)seq * p.rows.table_stride;
  const bf16* v = reinterpret_cast<const bf16*>(p.v);
  float infinite = 0.0f, sum = 0.0f;
  for (int j = 0; j < sr.n; ++j) {
    const int s = sr.at(j), end = min(min(attend_split_start(s + 1), t + 1), p.rows.limit());
    const float o = __ldcg(p.part_o + (base + s) * D + c);
    sum = __fmaf_rn(o, __fmul_rn(ex2(__fsub_rn(__ldcg(&p.part_ml[base + s].x), M)), 0x1p-24f), sum);
    if (fabsf(o) < INFINITY) continue;
    for (int pos = attend_split_start(s); pos < end; pos += 4) {
      const int page = __ldg(table + pos / kPage);
      if ((uint32_t)page >= (uint32_t)p.n_pages) continue;
      const bf16* column = v + (((size_t)page * p.n_kv_heads + kvh) * kPage + pos % kPage) * D + c;
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __bfloat162float(column[i * D]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool seen = pos + i < end && (p.window <= 0 || pos + i > t - p.window || pos + i < p.sinks);
        if (seen && !(fabsf(x[i]) < INFINITY)) infinite = __fadd_rn(infinite, x[i]);
      }
      if (infinite != infinite) return infinite;
    }
  }
  return infinite != 0.0f ? infinite : __fdiv_rn(sum, __fmul_rn(l, 0x1p-24f));
}

// The splits of one (row, query head) merged: out = sum_s o_s 2^(m_s - M) /
// sum_s l_s 2^(m_s - M), in a fixed order for the splits that the row sees,
// whatever else is in the call: the j-th of them belongs to strand j mod 8, each
// strand is added up in order and then the strands; the denominators of 32
// splits are added as a tree, and the groups of 32 in order.
//   kWide: a block for each, a warp a strand (few rows, many splits: the
// partials are requested side by side).  Else a warp does all of it.
constexpr int kStrands = 8;
template <int D, bool kWide>
__global__ void __launch_bounds__(256) k_attend_merge(const __grid_constant__ AttendParams p) {
  constexpr int V = D / 32, W = kStrands, B = 8;  // V: elements a lane, columns V * lane ..
  extern __shared__ float s_dyn[];                // factors [max_splits], denominators [max_splits / 32] of a unit
  __shared__ float s_red[W], s_o[kWide ? W : 1][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = kWide ? blockIdx.x : blockIdx.x * W + warp;  // (row - row_lo) * n_q_heads + head
  const int groups = (p.max_splits + 31) / 32;
  float* s_f = s_dyn + (kWide ? 0 : warp * groups * 33);
  float* s_l = s_f + groups * 32;
  const int r = p.row_lo + unit / p.n_q_heads, hq = unit % p.n_q_heads;
  pdl_trigger();
  int seq, i, t = 0;
  const bool row = r < p.row_hi && find_row(p.rows, r, seq, i);
  if (row) t = first_of(p.rows, seq) + i;
  const SplitRange sr = splits_seen(t, t, p.window, p.sinks, p.rows.limit());
  pdl_wait();
  if (!row) return;  // (a whole block, or a warp that meets no other)
  auto meet = [] { if (kWide) __syncthreads(); else __syncwarp(); };
  const int first = kWide ? threadIdx.x : lane, step = kWide ? 256 : 32;
  const size_t base = (size_t)unit * p.max_splits;
  float M = -INFINITY;
  for (int j = first; j < sr.n; j += step) M = fmaxf(M, __ldcg(&p.part_ml[base + sr.at(j)].x));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (kWide) {
    if (lane == 0) s_red[warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, s_red[w]);
  }
  const float ref = M == -INFINITY ? 0.0f : M;
  for (int j0 = first - lane; j0 < sr.n; j0 += step) {
    const int j = j0 + lane;
    float l = 0.0f, f = 0.0f;
    if (j < sr.n) {
      const float2 ml = __ldcg(&p.part_ml[base + sr.at(j)]);
      const float d = __fsub_rn(ml.x, ref);
      f = ex2(d);
      l = times_ex2(ml.y, d);
    }
    s_f[j] = f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, o));
    if (lane == 0) s_l[j0 / 32] = l;
  }
  meet();
  auto load = [&](int j, float (&x)[V]) {
    const float* src = p.part_o + (base + sr.at(j)) * D + lane * V;
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
  };
  float l = 0.0f;
  for (int k = 0; k < (sr.n + 31) / 32; ++k) l = __fadd_rn(l, s_l[k]);
  const bool none = l == 0.0f;  // a row that sees nothing: zeros
  bf16* out = p.out + (int64_t)r * p.out_stride + hq * D;
  float zero = 0.0f;  // a NaN when a sum is not finite
  if constexpr (kWide) {  // this warp's strand, eight of its splits at a time
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
    for (int j0 = warp; j0 < sr.n; j0 += W * B) {
      float x[B][V];
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (j0 + W * b < sr.n) load(j0 + W * b, x[b]);
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (j0 + W * b < sr.n) {
          const float f = s_f[j0 + W * b];
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = __fmaf_rn(x[b][e], f, acc[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = acc[e];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += 256) {
      float a = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) a = __fadd_rn(a, s_o[w][c]);
      zero = __fmaf_rn(a, 0.0f, zero);
      out[c] = __float2bfloat16_rn(none ? 0.0f : __fdiv_rn(a, l));
    }
  } else {  // all strands, one split of each at a time
    float acc[W][V];
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[w][e] = 0.0f;
    for (int j0 = 0; j0 < sr.n; j0 += W) {
      float x[W][V];
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (j0 + w < sr.n) load(j0 + w, x[w]);
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (j0 + w < sr.n) {
          const float f = s_f[j0 + w];
#pragma unroll
          for (int e = 0; e < V; ++e) acc[w][e] = __fmaf_rn(x[w][e], f, acc[w][e]);
        }
    }
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      float a = 0.0f, b = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        a = __fadd_rn(a, acc[w][e]);
        b = __fadd_rn(b, acc[w][e + 1]);
      }
      zero = __fmaf_rn(a, 0.0f, __fmaf_rn(b, 0.0f, zero));
      *reinterpret_cast<uint32_t*>(out + lane * V + e) = none ? 0u : pack_bf16x2(__fdiv_rn(a, l), __fdiv_rn(b, l));
    }
  }
  if (zero != 0.0f && l == l && p.k_exp == nullptr) {
    const int kvh = hq / (p.n_q_heads / p.n_kv_heads);
    asm volatile("" ::: "memory");  // (the thread's own stores above, of pairs)
#pragma unroll 1
    for (int c = kWide ? threadIdx.x : lane * V; c < (kWide ? D : (lane + 1) * V); c += kWide ? 256 : 1) {
      if (fabsf(__bfloat162float(out[c])) < INFINITY) continue;
      out[c] = __float2bfloat16_rn(far_value<D>(p, sr, base, seq, t, kvh, c, M, l));
    }
  }
  if (p.lse && lane == 0 && (!kWide || warp == 0))
    p.lse[(size_t)r * p.n_q_heads + hq] = none ? -INFINITY : __fmul_rn(__fadd_rn(M, log2f(l)), 0.6931471805599453f);
  asm volatile("fence.proxy.async.global;" ::: "memory");  // a context reads it next by bulk copies
}

template <int D, int FMT, int N>
cudaError_t attend_launch_t(const AttendParams& p, int num_sms,
                            cudaStream_t s, bool pdl) {
  using C = AttendCfg<D, FMT, N>;
  const int smem = C::smem_bytes(p.rows.n_seq);
  // CTAs per SM at this much shared memory: asked once for each device and size
  static std::atomic<int64_t> of_device[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::atomic<int64_t>& known = of_device[dev];
  int64_t k = known.load(std::memory_order_relaxed);
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
  const int64_t n_rows = p.row_hi - p.row_lo, tiles = n_rows * G / C::QR + p.rows.n_seq;
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
  e = cudaLaunchKernelEx(&cfg, k_attend<D, FMT, N>, p);
  if (e != cudaSuccess) return e;
  const int64_t units = n_rows * p.n_q_heads;
  const size_t words = (size_t)((p.max_splits + 31) / 32) * 33;
  cfg.blockDim = dim3(256);
  cfg.numAttrs = 1;  // the merge may be resident before the partials are complete: it waits for them
  // A warp for each result where there are enough of them to fill the device, or
  // few splits to be had in parallel.  (128 rows of 32 heads over 4k: the call
  // 73.6 us with a warp each, 84.7 with a block each; 8 x 16 rows 39.3 and 44.5,
  // 16 x 4 in windows of 4096 44.7 and 49.0, 32 rows over 8k 83.6 and 83.2.)
  if ((units >= 4 * num_sms || p.max_splits <= 8) && words * 4 * kStrands <= kMergeMaxSmem) {
    cfg.gridDim = dim3((unsigned)((units + kStrands - 1) / kStrands));
    cfg.dynamicSmemBytes = words * 4 * kStrands;
    return cudaLaunchKernelEx(&cfg, k_attend_merge<D, false>, p);
  }
  cfg.gridDim = dim3((unsigned)units);
  cfg.dynamicSmemBytes = words * 4;
  return cudaLaunchKernelEx(&cfg, k_attend_merge<D, true>, p);
}

// Query tiles of 8 rows where they hold a sequence's rows, else of 16.  (Tiles
// of 32 read and widened a page half as often, but at 128 accumulators a lane
// eight warps an SM were too few: 8 x 16 rows at 4k took 49 us, with tiles of
// 16 and twelve warps 39; a prefill block of 128 rows 78 and 74.)  A row's
// result is the same in either (the columns of an mma do not meet).
template <int D, int FMT>
cudaError_t attend_launch(const AttendParams& p, int num_sms, cudaStream_t s, bool pdl) {
  const int64_t f = (int64_t)p.rows.max_rows * (p.n_q_heads / p.n_kv_heads);
  return f <= 8 ? attend_launch_t<D, FMT, 1>(p, num_sms, s, pdl) : attend_launch_t<D, FMT, 2>(p, num_sms, s, pdl);
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
  if ((e = attend_prepare_t<D, FMT, 1>()) != cudaSuccess) return e;
  // the factors of as many splits as a table reaches positions
  if ((e = cudaFuncSetAttribute(k_attend_merge<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kMergeMaxSmem)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(k_attend_merge<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kMergeMaxSmem)) != cudaSuccess)
    return e;
  return attend_prepare_t<D, FMT, 2>();
}

}  // namespace
}  // namespace sv
