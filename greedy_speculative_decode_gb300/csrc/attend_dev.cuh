// attend_dev.cuh -- attention of a ragged batch's rows over a paged cache.
//
// Row i of sequence s stands at position t = first[s] + i and sees the
// positions p <= t, with a window W only those with p > t - W or p < sinks:
//   s_p = scale * q . k_p,  o = sum_p softmax(s)_p v_p,  lse = ln sum_p exp(s_p).
// The cache is read once per tile of 8 N query rows (token rows x the query
// heads of a kv head, packed one behind the other whatever the group size), so
// few rows are bound by its bytes.  A CTA of four warps walks a split's chunks
// of four pages, warp w its page w, each warp by itself: its own ring of
// asynchronous copies and its own softmax statistics and accumulators, no barrier.
//   Scores, transposed: S^T = K Q^T.  The page's 16 positions are the 16 rows
//     of an mma, eight query rows its columns, so single-token decode with a
//     group of up to eight heads wastes none of it.  K goes from 8 to 16 bits
//     in registers.
//   Online softmax over pages; the weights are transposed in registers
//     (movmatrix).
//   O^T += V^T P^T, all columns.  A transposing load of bytes makes V's operand
//     (four consecutive positions of a column in a word).
// At the split's end the four warps' results meet in shared memory and go out
// as the split's partial; a second kernel merges the splits.
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
// Splits are ranges of absolute positions (attend_split_start), and a row's
// arithmetic does not depend on the rows, sequences or tiles beside it: a
// page a row does not see leaves its maximum, sum and accumulators as they
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
constexpr int kAttendThreads = kAttendWarps * 32;

// A tile of query rows.
struct AttendTile {
  int row0, f0, nf, kvh;  // the sequence's first row, the tile's first query row, the sequence's query rows
  int first;              // position of the sequence's first row
};
// (by what the rings and 32 N D / 128 accumulators a lane leave room for)
__host__ __device__ constexpr int kAttendPerSm(int d, bool bf16, int n) {
  const int rb = d * (bf16 ? 2 : 1);
  if (rb == 512) return 1;
  if (n * d >= 512) return 2;
  if (rb == 256) return 2;
  return n * d >= 256 ? 3 : n * d >= 128 ? 4 : 5;
}

template <int D_, int FMT_, int N_>
struct AttendCfg {
  static constexpr int D = D_, FMT = FMT_, N = N_;  // N: query tiles of 8 rows
  static constexpr bool kBf16 = FMT == SV_KV_BF16;
  static constexpr int RB = D * (kBf16 ? 2 : 1);  // bytes of a position's row
  static constexpr int kPageBytes = kPage * RB;
  static constexpr int kChunk = kAttendWarps * kPage;
  static constexpr int kStageBytes = 2 * kPageBytes;
  // pages of K and V in a warp's ring: one at hand, the others on their way.
  // The warps of an SM together keep about 80 KB on the way.
  static constexpr int kStages = N == 4 || RB == 512 ? 2 : RB == 256 ? 3 : 2;
  static constexpr int kPerSm = kAttendPerSm(D, kBf16, N);  // CTAs per SM that registers are cut for
  static constexpr int NK = D / 16;               // k16 steps of a score
  static constexpr int U = D / 16;                // 16-column units of the output
  static constexpr int QR = 8 * N;                // query rows of a tile
  static constexpr bool kQRegs = N * NK <= 16;    // query fragments stay in registers
  // the meeting of the warps, a part of the columns at a time (8 KB of accumulators)
  static constexpr int kColsMax = 64 / N;
  static constexpr int kCols = kColsMax < D ? kColsMax : D;
  static constexpr int kRounds = D / kCols;
  static constexpr int kColStride = kCols + 4;    // floats of a query row (4 mod 16: no bank conflicts)
  static_assert(kCols % 16 == 0 && kColStride % 16 == 4, "columns of a round");
  // shared memory
  static constexpr int kScaleBytes = kBf16 ? 0 : 2 * kPage;        // exponents of a stage (one a position)
  static constexpr int kRing = kAttendWarps * kStages;             // stages of all warps
  static constexpr int kOffScale = kRing * kStageBytes;
  static constexpr int kOffQ = kOffScale + kRing * kScaleBytes;    // query fragments [N][NK][32 lanes][2 words]
  static constexpr int kQBytes = N * NK * 256;
  static constexpr int kOffO = kOffQ + kQBytes;                    // [4 warps][QR][kColStride] accumulators
  static constexpr int kOffMl = kOffO + kAttendWarps * QR * kColStride * 4;  // [QR][4 warps] (max, sum)
  static constexpr int kOffRow = kOffMl + QR * 32;                 // [QR] score factors, positions, slots
  static constexpr int kOffSeq = kOffRow + 3 * QR * 4;             // [n_seq + 1] chunks before, first, row start
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
    vis_lo = wk.p.window > 0 ? max(t0 - wk.p.window + 1, 0) : 0;
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

// ------------------------------------------------------------------ a warp's loads
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Page `page` of a kv head into a stage: 2 RB / 64 copies of 16 bytes a lane,
// swizzled as page_off says, and an 8-bit page's exponents (one a position).
template <class C>
__device__ __forceinline__ void fetch_page(const AttendParams& p, int page, int kvh, int lane, uint32_t stage,
                                           uint32_t scale) {
  constexpr int kUnitsRow = C::RB / 16, kPer = C::kPageBytes / 512;  // units of a row; copies of a lane
  const size_t ph = (size_t)page * p.n_kv_heads + kvh;
  const uint8_t* k = p.k + ph * C::kPageBytes + lane * 16;
  const uint8_t* v = p.v + ph * C::kPageBytes + lane * 16;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    const uint32_t dst = stage + page_off<C::RB>(e / kUnitsRow, e % kUnitsRow);
    copy16(dst, k + 512 * i);
    copy16(dst + C::kPageBytes, v + 512 * i);
  }
  if (!C::kBf16 && p.block == 1 && lane < 2) copy16(scale + lane * kPage, (lane ? p.v_exp : p.k_exp) + ph * kPage);
}

// ------------------------------------------------------------------ the arithmetic
// The statistics and accumulators of a warp in the course of a split.  A lane
// (g, q4) holds positions g and g + 8 of a page (in pos_of_row's order)
// against query rows 2 q4, 2 q4 + 1 of each query tile, then columns g and
// g + 8 of each unit against them.
template <class C>
struct AttendRows {
  static constexpr int N = C::N, U = C::U, W = kAttendWarps;
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
  __device__ __forceinline__ float* s_o() const { return reinterpret_cast<float*>(smem + C::kOffO); }
  __device__ __forceinline__ float2* s_ml() const { return reinterpret_cast<float2*>(smem + C::kOffMl); }
  __device__ __forceinline__ float* s_fac() const { return reinterpret_cast<float*>(smem + C::kOffRow); }
  __device__ __forceinline__ int* s_t() const { return reinterpret_cast<int*>(smem + C::kOffRow) + C::QR; }
  __device__ __forceinline__ int* s_slot() const { return reinterpret_cast<int*>(smem + C::kOffRow) + 2 * C::QR; }
  __device__ __forceinline__ const uint2* s_q() const { return reinterpret_cast<const uint2*>(smem + C::kOffQ) + lane; }
  __device__ __forceinline__ bool sees(int t, int pos) const {
    return pos <= t && (p.window <= 0 || pos > t - p.window || pos < p.sinks);
  }

  // A tile's queries as B fragments, the rows' score factors, positions and
  // output slots (all warps).  A piece is 8 elements of one query row; they go
  // to the lanes and k16 steps that meet the same elements of K (a lane's
  // 16-byte unit of a key row, four elements a step).
  __device__ __forceinline__ void queries(const AttendTile& it, int G) {
    constexpr int kPieces = C::QR * C::D / 8, T = kAttendThreads;
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

  __device__ __forceinline__ void open() {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      m_run[n][0] = m_run[n][1] = -INFINITY;
      l_run[n][0] = l_run[n][1] = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) o[u][n][0] = o[u][n][1] = o[u][n][2] = o[u][n][3] = 0.0f;
    }
  }

  // An infinity or NaN of a bf16 page in a place that some row does not see
  // must not meet that row's weight of zero: it is taken out here and added to
  // the rows that see it.  (a: columns g, g + 8 of unit u, positions 2 q4, 2 q4
  // + 1 and 8 more of the page; the accumulators of these columns are held by
  // the same quad of lanes.)
  __device__ __forceinline__ void set_apart(int base, int u, uint32_t (&a)[4]) {
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

  // One page: scores in log2 units with the value's exponent added, -inf where
  // a row does not see the position; the running maxima and sums; O^T.
  // kEdge: some row does not see some position.
  template <bool kEdge>
  __device__ __forceinline__ void page(uint32_t kp, uint32_t vp, const uint8_t* sc, int base, uint32_t exps) {
    float s[N][4];
#pragma unroll
    for (int n = 0; n < N; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
    const int pos = pos_of_row<kBf16>(g), pos8 = pos_of_row<kBf16>(g + 8);
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
    float ks[2], ev[2], iv[2];
    if (!kBf16) {  // positions pos and pos + 2: two bytes of a word of the page's exponents
      uint32_t kw, vw;
      if (p.block == 1) {
        kw = *reinterpret_cast<const uint32_t*>(sc + (pos & ~3)) >> (8 * (pos & 3));
        vw = *reinterpret_cast<const uint32_t*>(sc + kPage + (pos & ~3)) >> (8 * (pos & 3));
      } else {
        kw = (exps & 255u) * 0x00010001u;
        vw = (exps >> 8) * 0x00010001u;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t bk = (kw >> (16 * h)) & 255u, bv = (vw >> (16 * h)) & 255u;
        ks[h] = __uint_as_float(bk << 23);  // (255: infinity, times a score of zero codes: NaN)
        ev[h] = bv == kExpNaN ? __uint_as_float(0x7fffffffu) : (float)((int)bv - 127);
        iv[h] = exp_byte_inverse((int)bv);
      }
    }
    uint32_t hi[N][2], lo[kBf16 ? N : 1][2];
    bool moved = false;
    float alpha[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float2 f = reinterpret_cast<const float2*>(s_fac())[n * 4 + q4];
      const int2 t = kEdge ? reinterpret_cast<const int2*>(s_t())[n * 4 + q4] : make_int2(0, 0);
      float pv[4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float& x = s[n][2 * h + c];
          const float fc = c ? f.y : f.x;
          x = kBf16 ? __fmul_rn(x, fc) : __fmaf_rn(x, __fmul_rn(fc, ks[h]), ev[h]);
          if (kEdge) x = sees(c ? t.y : t.x, base + (h ? pos8 : pos)) ? x : -INFINITY;
        }
        float m = fmaxf(s[n][c], s[n][2 + c]);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        m = fmaxf(m, m_run[n][c]);
        // a row that has seen nothing yet: every weight is 2^-inf = 0
        const float ref = m == -INFINITY ? 0.0f : m;
        const bool same = m == m_run[n][c];
        alpha[n][c] = same ? 1.0f : ex2(__fsub_rn(m_run[n][c], ref));
        moved |= !same;
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
        l_run[n][c] = __fmaf_rn(l_run[n][c], alpha[n][c], sum);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (kBf16) {
          hi[n][h] = transposed(pack_bf16x2(pv[2 * h], pv[2 * h + 1]));
          lo[kBf16 ? n : 0][h] = transposed(pack_bf16x2(__fsub_rn(pv[2 * h], bf16r(pv[2 * h])),
                                                        __fsub_rn(pv[2 * h + 1], bf16r(pv[2 * h + 1]))));
        } else {
          hi[n][h] = transposed(pack_f16x2(pv[2 * h], pv[2 * h + 1]));
        }
      }
    }
    // (a maximum seldom moves after a split's first pages; times one is skipped)
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[u][n][e] = __fmul_rn(o[u][n][e], alpha[n][e & 1]);
    }
#pragma unroll
    for (int u = 0; u < U; u += 2) {
      uint32_t r[4];
      if constexpr (!kBf16) ldsm_b8_x2_trans(vp + page_off<C::RB>(lane & 15, u + (lane >> 4)), r);
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
          ldsm_x4_trans(vp + page_off<C::RB>(lane & 15, (u + y) * 2 + (lane >> 4)), a[0], a[2], a[1], a[3]);
          if (kEdge) set_apart(base, u + y, a);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
          mma_16<kBf16>(o[u + y][n], a, hi[n][0], hi[n][1]);
          if (kBf16) mma_16<kBf16>(o[u + y][n], a, lo[kBf16 ? n : 0][0], lo[kBf16 ? n : 0][1]);
        }
      }
    }
  }

  // The split's partial: (max, sum) and accumulators of the four warps merged
  // in warp order, a part of the columns at a time.
  __device__ __forceinline__ void partial(int split) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = l_run[n][c];
        l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 4));
        l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 8));
        l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, 16));
        if (g == 0) s_ml()[(n * 8 + 2 * q4 + c) * W + warp] = make_float2(m_run[n][c], l);
      }
    constexpr int kUR = U / C::kRounds;            // units a round
    constexpr int kV = C::kCols / 4;               // float4 columns of a query row
    const int tid = threadIdx.x;
#pragma unroll
    for (int rd = 0; rd < C::kRounds; ++rd) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float* dst = s_o() + (warp * C::QR + n * 8 + 2 * q4 + c) * C::kColStride + g;
#pragma unroll
          for (int u = 0; u < kUR; ++u) {
            dst[16 * u] = o[rd * kUR + u][n][c];
            dst[16 * u + 8] = o[rd * kUR + u][n][2 + c];
          }
        }
      named_sync(2, kAttendThreads);
      for (int e = tid; e < C::QR * kV; e += kAttendThreads) {
        const int qi = e / kV, v = e % kV, slot = s_slot()[qi];
        if (slot < 0) continue;
        const float2* ml = s_ml() + qi * W;
        float M = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, ml[w].x);
        const float ref = M == -INFINITY ? 0.0f : M;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float f = ex2(__fsub_rn(ml[w].x, ref));
          const float4 x = *reinterpret_cast<const float4*>(s_o() + (w * C::QR + qi) * C::kColStride + 4 * v);
          l = __fmaf_rn(ml[w].y, f, l);
          a.x = __fmaf_rn(x.x, f, a.x);
          a.y = __fmaf_rn(x.y, f, a.y);
          a.z = __fmaf_rn(x.z, f, a.z);
          a.w = __fmaf_rn(x.w, f, a.w);
        }
        const size_t at = (size_t)slot * p.max_splits + split;
        if (rd == 0 && v == 0) p.part_ml[at] = make_float2(M, l);
        *reinterpret_cast<float4*>(p.part_o + at * C::D + rd * C::kCols + 4 * v) = a;
      }
      named_sync(2, kAttendThreads);
    }
  }
};

// A CTA's run, list by list.
template <class C>
__device__ void attend_cta(const AttendParams& p, const AttendWork<C>& wk, uint8_t* smem) {
  constexpr int S = C::kStages;
  AttendPlace<C> at;
  if (!at.start(wk)) return;
  AttendRows<C> rows(p, smem);
  const int warp = rows.warp, lane = rows.lane;
  const uint32_t ring = smem_u32(smem) + warp * S * C::kStageBytes;
  const uint8_t* scales = smem + C::kOffScale + warp * S * C::kScaleBytes;
  const uint32_t scales_at = smem_u32(scales);
  for (;;) {
    const int run = at.run_end();
    const int* table = p.rows.table + (size_t)at.seq * p.rows.table_stride;
    // This warp's page of place j of the list: its number, -1 where the tile
    // sees nothing of it (or there is none)
    auto page_of = [&](int j) {
      if (j >= run) return -1;
      const int a = at.list.at(j) * C::kChunk + warp * kPage;
      if (!at.sees(a, kPage, p.sinks)) return -1;
      const int pg = __ldg(table + a / kPage);
      if ((uint32_t)pg < (uint32_t)p.n_pages) return pg;
      if (p.status && lane == 0) atomicOr(p.status, ST_BAD_PAGE);
      return -1;
    };
    uint32_t have = 0, exps[S];  // bit k, exps[k]: of place i + k
    int issued = 0;
    auto request = [&](int j, int pg, uint32_t& ex) {
      if (pg >= 0) {
        const int st = issued % S;
        fetch_page<C>(p, pg, at.tile.kvh, lane, ring + st * C::kStageBytes, scales_at + st * C::kScaleBytes);
        if (!C::kBf16 && p.block != 1) {
          const size_t ph = (size_t)pg * p.n_kv_heads + at.tile.kvh;
          ex = (uint32_t)__ldg(p.k_exp + ph) | (uint32_t)__ldg(p.v_exp + ph) << 8;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      ++issued;
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) {
      const int pg = page_of(at.i + k);
      have |= (pg >= 0 ? 1u : 0u) << k;
      request(at.i + k, pg, exps[k]);
    }
    int ahead = page_of(at.i + S - 1);
    rows.queries(at.tile, wk.G);
    named_sync(2, kAttendThreads);
    rows.keep_queries();
    rows.open();
    bool any = false;  // the item has a chunk that the tile sees
    int st = 0;
    for (int i = at.i; i < run; ++i) {
      // the page S - 1 places on, into the stage that place i - 1 had (every lane has done with it)
      __syncwarp();
      have |= (ahead >= 0 ? 1u : 0u) << (S - 1);
      request(i + S - 1, ahead, exps[S - 1]);
      ahead = page_of(i + S);
      const int chunk = at.list.at(i) * C::kChunk, base = chunk + warp * kPage;
      any |= at.sees(chunk, C::kChunk, p.sinks);
      if (have & 1u) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        __syncwarp();
        const uint32_t kp = ring + st * C::kStageBytes;
        const uint8_t* sc = scales + st * C::kScaleBytes;
        // whether every row of the tile sees every position of the page
        const bool all = base + kPage - 1 <= at.t0 &&
                         (p.window <= 0 || base > at.t1 - p.window || base + kPage - 1 < p.sinks);
        if (all) rows.template page<false>(kp, kp + C::kPageBytes, sc, base, exps[0]);
        else rows.template page<true>(kp, kp + C::kPageBytes, sc, base, exps[0]);
      }
      have >>= 1;
#pragma unroll
      for (int k = 0; k < S - 1; ++k) exps[k] = exps[k + 1];
      st = st + 1 == S ? 0 : st + 1;
      const int split = attend_split_of(chunk);
      if (i + 1 == run || attend_split_of(at.list.at(i + 1) * C::kChunk) != split) {
        if (any) {
          rows.partial(split);
          rows.open();
        }
        any = false;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!at.past(wk, run)) return;
    named_sync(2, kAttendThreads);  // every warp is done with this tile's queries
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
  pdl_wait();
  const int S = p.rows.n_seq, G = p.n_q_heads / p.n_kv_heads;
  int *first = before + S + 1, *start = first + S;  // (S + 1 starts)
  AttendWork<C> wk{p, before, first, start, 0, G};
  wk.total = attend_plan<C>(p, G, before, first, start);
  attend_cta<C>(p, wk, smem);
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
  const SplitRange sr = splits_seen(t, t, p.window, p.sinks, p.rows.limit());
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
cudaError_t attend_launch_t(const AttendParams& p, int num_sms,
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
  e = cudaLaunchKernelEx(&cfg, k_attend<D, FMT, N>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)((int64_t)p.rows.n_rows * p.n_q_heads));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;  // the merge may be resident before the partials are complete: it waits for them
  return cudaLaunchKernelEx(&cfg, k_attend_merge<D>, p);
}

// Query tiles of 8, 16 or 32 rows (16 at most for heads of 256): the smallest
// that hold a sequence's rows at once, so that its pages are read and widened
// as seldom as accumulators in registers allow.  A row's result is the same in
// each (the columns of an mma do not meet).
template <int D, int FMT>
cudaError_t attend_launch(const AttendParams& p, int num_sms,
                          cudaStream_t s, bool pdl) {
  const int64_t f = (int64_t)p.rows.max_rows * (p.n_q_heads / p.n_kv_heads);
  if (f <= 8) return attend_launch_t<D, FMT, 1>(p, num_sms, s, pdl);
  if (f <= 16 || D == 256) return attend_launch_t<D, FMT, 2>(p, num_sms, s, pdl);
  return attend_launch_t<D, FMT, D == 256 ? 2 : 4>(p, num_sms, s, pdl);
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
  if ((e = attend_prepare_t<D, FMT, 1>()) != cudaSuccess || (e = attend_prepare_t<D, FMT, 2>()) != cudaSuccess) return e;
  return attend_prepare_t<D, FMT, D == 256 ? 2 : 4>();
}

}  // namespace
}  // namespace sv
