// shared_dev.cuh -- attention of many query rows to a prefix whose pages they share.
//
// Sequences of a group have the same pages for their first positions.  The
// query rows of all of them (rows x the query heads of a kv head) are attended to
// these positions at once, so that the prefix is read once for every 128 or 256
// query rows instead of once a sequence:
//   S = Q K^T (128 query rows x 128 positions), P = 2^(S - ref), O += P V
// on the tensor cores (tcgen05), S and O in tensor memory.  What each sequence has
// behind the prefix goes through k_attend; a merge adds both.
//
// A CTA has two streams of steps, each with its scores, accumulators and softmax
// warpgroups, so that one's products run beside the other's exponentials: two
// tiles of 128 query rows that share the chunks of K and V they load, or, of a
// single tile, the even and the odd chunks.  (Rows of 256 elements leave tensor
// memory for one stream only; its scores alternate between two places.)
//   Warps 0-7, 8-15: softmax of a stream.  Each of its two warpgroups takes half of a
//     chunk's positions, a query row a thread; the halves exchange their largest score
//     in shared memory.  Scores are read from tensor memory, the weights go back there
//     over them as the A operand of P V.  The reference of a row moves only when its
//     maximum rises by more than 2^8 over it, so the accumulators are seldom read back
//     and rescaled.  (A warpgroup a stream, a whole row a thread: 132 us for 128 x 1 behind
//     16384 where two took 120, 92 and 81 for 64 x 4 behind 4096.)
//   Warp 16: its elected thread issues the multiplies.  Warps 17, 18: loads of K and V.
//   Warps 20-23 (8-bit caches): codes to f16, once for all query rows of the CTA.
// (One stream, D = 256: softmax warps 0-7, then 8, 9 and 10, 12-15.)
//
// Types, as in attend_dev.cuh: a bf16 cache's weights are the sum of two bf16
// values (2^-16); over an 8-bit cache weights are f16 and carry the value's
// exponent, t' = log2(e) s + ev, queries go to f16 divided by a power of two near
// their row's largest value; sums, references and accumulators are fp32.  Where the
// exponents of a chunk's keys lie within 2^15 of one another and its values' within
// 2^7 they are folded into the f16 operands instead (exact: a code has 4 bits), and
// its scores and sums need no factor a position; other chunks ("uneven") do.
//
// Work is divided as chunks of all (group, kv head, tiles) lists one behind the
// other.  Where every list is enough for a CTA each has a number of them for itself,
// else all lists are cut into equal runs.  Each CTA leaves a partial (reference, sum,
// accumulators) for each list its run touches, and the merge adds them in order.
// (A new list costs a CTA some 5 us: queries, and a partial.  Equal runs throughout:
// 78 us for 128 x 1 behind 16384, now 72; 71 and 59 for 64 x 4 behind 4096.)
//
// Measured (32 / 8 heads of 128 unless noted; the whole call, then this kernel): bf16,
// 64 x 1 behind 32768: 78 and 45 us, 134 MB of prefix, of which the products alone are
// 24 us of a tensor pipe (three of 64 cycles for each 16 columns: S, P's two terms);
// e4m3, 32 x 1 behind 8192: 38 and 17; 64 x 4 behind 4096, 28 / 4 heads: 58; bf16, d 256,
// 13 x 2, 8 / 1 heads: 35; d 64, 64 x 1 behind 8192, 4 / 2 heads: 25, bf16 33.  Where every
// chunk is uneven: e4m3, 32 x 1 behind 8192: 50; d 64: 32.
//   Neither memory nor the pipe is full (52 % for bf16, 37 % for e4m3): a stream's step
// is a chain, S, softmax, P V, and two of them overlap; the softmax's warps issue an
// instruction every other cycle.
#pragma once
#include "paged_dev.cuh"
#include "shared.h"
#include "tc_dev.cuh"

#include <cfloat>
#include <cuda_fp16.h>

namespace sv {

bool make_bf16_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint32_t box_rows);

namespace {

constexpr float kShSlack = 8.0f;     // log2 of what a row's maximum may rise by before its reference follows
// log2 of a row's largest weight when its reference is set.  f16 weights lie as high
// in their range as the slack lets them: their steps below 2^-14 are then 2^-32 of
// the largest, which leaves 2^-25 where a chunk's values are scaled by up to 2^-7.
__host__ __device__ constexpr float sh_bias(bool bf16) { return bf16 ? 0.0f : 7.0f; }
constexpr int kShKeySpread = 15, kShValueSpread = 7;  // of the exponents of an even chunk
constexpr float kShNone = -3.0e38f;  // reference of a row that has seen nothing
constexpr float kShBig = 1048576.0f;  // 2^20: half a step of a reference is 1 / 32 of log2
constexpr float kShFar = -126.0f;    // 2^x is a normal fp32 number from here on

template <int D_, int FMT_>
struct ShCfg {
  static constexpr int D = D_, FMT = FMT_;
  static constexpr bool kBf16 = FMT == SV_KV_BF16;
  static constexpr int NS = shared_streams(D), CP = shared_chunk(D), kPages = CP / kPage, kHalves = D / 64;
  static constexpr int kQBytes = kSharedTile * D * 2;  // a tile of queries
  static constexpr int kOpBytes = CP * D * 2;          // K or V of a chunk, as an operand
  static constexpr int kOps = kBf16 ? (D == 64 ? 8 : 5) : (D == 64 ? 4 : 3);
  static constexpr int kRawBytes = kBf16 ? 0 : CP * D;  // its codes
  static constexpr int kRaws = kBf16 ? 0 : D == 64 ? 4 : 3;
  static constexpr int kRings = 4;  // chunks whose scales and page masks are kept
  static constexpr int kSoftWarps = 8 * NS;  // two warpgroups a stream
  static constexpr int kMmaWarp = kSoftWarps, kLoadWarp = kSoftWarps + 1, kWidenWarp = kSoftWarps + 4;
  static constexpr int kThreads = (kWidenWarp + (kBf16 ? 0 : 4)) * 32;
  // tensor memory: scores (and weights over them) of two steps, accumulators of each stream
  static constexpr uint32_t kScoreCol = CP, kOutCol = 512 - NS * D;
  static_assert(2 * kScoreCol <= kOutCol, "columns of tensor memory");
  // shared memory
  static constexpr int kOffQ = 0, kOffOp = NS * kQBytes, kOffRaw = kOffOp + kOps * kOpBytes;
  static constexpr int kOffExp = kOffRaw + kRaws * kRawBytes;        // [kRaws][2][CP] exponent bytes
  static constexpr int kOffScale = kOffExp + kRaws * 2 * (kBf16 ? 0 : CP);  // [kRings][3][CP] 2^ek, ev, 2^-ev
  static constexpr int kOffLow = kOffScale + (kBf16 ? 0 : kRings * 3 * CP * 4);
  static constexpr int kOffBar = kOffLow;
  static constexpr int kBars = 2 * kOps + 2 * kRaws + kRings + 2 /*s_full*/ + 2 /*p_full*/ + 2 /*pv*/ + 2 /*q*/ + 1 /*drain*/;
  static constexpr int kOffMeta = kOffBar + kBars * 8;  // [8] what a chunk holds (sh_meta)
  static constexpr int kOffRawMeta = kOffMeta + 32;     // [8] the same for an item of codes
  // [2 score places][2 halves][128 rows] largest scores and sums; before a segment's first
  // step [places][128] token rows of the query rows (-1: none)
  static constexpr int kOffRow = kOffRawMeta + 32;
  static constexpr int kOffTmem = kOffRow + 4 * kSharedTile * 4;
  static constexpr int kOffFailed = kOffTmem + 4;     // whether a wait of the CTA has given up
  static constexpr int kOffLast = kOffTmem + 16;      // [8] the last copy into each place of the ring that is loaded, + 1
  static constexpr int kSmem = kOffLast + 32;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

// idesc of the two products: f16 or bf16 operands, fp32 accumulators; B of P V lies along N.
template <class C>
__device__ __forceinline__ constexpr uint32_t sh_idesc(int N, bool b_mn) {
  return (1u << 4) | (C::kBf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(kSharedTile >> 4) << 24);
}

// Two fp32 values in one instruction's operands.
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void split(uint64_t x, uint32_t& lo, uint32_t& hi) { asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A value that all lanes of a warp have, in a uniform register (a reduction's result
// is one): descriptors worked out from such values cost the multiplying warp a few
// instructions, not a move for each operand of each multiply.
__device__ __forceinline__ uint32_t sh_uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }

__device__ __forceinline__ float sh_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// l 2^d for d <= 0, also where 2^d by itself is below fp32's range.
__device__ __forceinline__ float sh_times_ex2(float l, float d) {
  const float h = __fmul_rn(d, 0.5f);
  return d < kShFar ? __fmul_rn(__fmul_rn(l, sh_ex2(h)), sh_ex2(h)) : __fmul_rn(l, sh_ex2(d));
}
__device__ __forceinline__ uint32_t sh_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ------------------------------------------------------------------ the division of the work
// A run of chunks i0 .. i1 - 1 of one list.
struct ShSegment {
  SharedGroup g;
  int kvh, pair, w;  // w: tiles of the list
  int i0, i1;
};

__device__ __forceinline__ SharedGroup sh_group(const SharedGroup* plan, int g) {
  SharedGroup r;
  const int4* src = reinterpret_cast<const int4*>(plan + g);
  const int4 a = __ldcg(src), b = __ldcg(src + 1);
  r.unit0 = a.x; r.eff = a.y; r.s0 = a.z; r.row0 = a.w; r.R = b.x; r.chunks = b.y; r.tiles = b.z; r.aligned = b.w;
  return r;
}

// Of G CTAs and U units: the CTA that has unit u where runs are equal (that of CTA c
// begins with unit U c / G), and the first CTA of a list that begins with unit u where
// they end with lists.
__device__ __forceinline__ int sh_owner(int u, int U, int G) {
  return (int)((((unsigned long long)u + 1) * G - 1) / (unsigned)U);
}
__device__ __forceinline__ int sh_first(int u, int U, int G) {
  return (int)((2ull * u * G + U) / (2ull * U));
}

template <int NS>
struct ShRun {
  const SharedGroup* plan;
  int n_kv;
  int u, hi;  // the next unit, the end of the CTA's
  int gi;     // group that u is in
  SharedGroup g;
  __device__ __forceinline__ ShRun(const SharedParams& p, int cta) : plan(p.plan), n_kv(p.a.n_kv_heads) {
    const int2 a = __ldcg(reinterpret_cast<const int2*>(p.begin + cta));
    hi = __ldcg(&p.begin[cta + 1].unit);
    g = sh_group(&p.begin[cta].g, 0);
    u = a.x;
    gi = a.y;
  }
  __device__ __forceinline__ bool next(ShSegment& s) {
    while (u < hi) {
      const int per = g.chunks * g.tiles, at = u - g.unit0;
      if (at >= per * n_kv) {
        g = sh_group(plan, ++gi);
        continue;
      }
      s.g = g;
      s.kvh = at / per;
      const int in = at - s.kvh * per;
      s.pair = in / (g.chunks * NS);
      s.w = min(NS, g.tiles - s.pair * NS);
      const int unit = g.unit0 + s.kvh * per + s.pair * NS * g.chunks;
      const bool two = s.w == 2;
      s.i0 = two ? (u - unit + 1) >> 1 : u - unit;
      s.i1 = min(g.chunks, two ? (hi - unit + 1) >> 1 : hi - unit);
      const bool rest = s.i1 == g.chunks;
      u = rest ? unit + g.chunks * s.w : hi;
      if (s.i1 > s.i0) return true;
    }
    return false;
  }
};

// Row of the planes where a segment's tiles begin.
__device__ __forceinline__ long long sh_slot(const SharedParams& p, const SharedGroup& g, int kvh, int pair, int ns, int cta) {
  return (long long)g.row0 * p.a.n_q_heads + (long long)kvh * g.R + (long long)pair * ns * kSharedTile + (long long)cta * kSharedTile;
}

// The steps of a segment.  Two tiles (both): step j is chunk j / 2 for stream j mod
// 2.  One tile: step j is chunk j, for stream j mod NS.  Operands are loaded in
// the order in which the steps first need them: S(0), S(1), then P V(j), S(j + 2).
struct ShOrder {
  int n;      // chunks
  bool both;
  __device__ __forceinline__ int steps() const { return both ? 2 * n : n; }
  __device__ __forceinline__ int chunk(int j) const { return both ? j >> 1 : j; }
  // place of K (V) of chunk c among the 2 n operands
  __device__ __forceinline__ int k_at(int c) const { return both ? 2 * c : c == 0 ? 0 : 2 * c - 1; }
  __device__ __forceinline__ int v_at(int c) const { return both ? 2 * c + 1 : c == n - 1 ? 2 * n - 1 : 2 * c + 2; }
  // the i-th operand: its chunk, and whether it is V
  __device__ __forceinline__ int item(int i, bool& v) const {
    if (both) {
      v = i & 1;
      return i >> 1;
    }
    if (i == 0) { v = false; return 0; }
    if (i >= 2 * n - 2) { v = i == 2 * n - 1 || n > 1; return i == 2 * n - 1 ? n - 1 : n - 2; }
    v = !(i & 1);
    return v ? (i - 2) >> 1 : (i + 1) >> 1;
  }
};

template <class C>
struct ShSmem {
  uint8_t* base;
  uint64_t* bar;
  uint32_t limit_ns;  // of a wait
  __device__ __forceinline__ ShSmem(uint8_t* b, uint32_t ns) : base(b), bar(reinterpret_cast<uint64_t*>(b + C::kOffBar)), limit_ns(ns) {}
  __device__ __forceinline__ uint8_t* q(int x) const { return base + C::kOffQ + x * C::kQBytes; }
  __device__ __forceinline__ uint8_t* op(int s) const { return base + C::kOffOp + s * C::kOpBytes; }
  __device__ __forceinline__ uint8_t* raw(int s) const { return base + C::kOffRaw + s * C::kRawBytes; }
  __device__ __forceinline__ uint8_t* exps(int s) const { return base + C::kOffExp + s * 2 * C::CP; }
  __device__ __forceinline__ float* scale(int s) const { return reinterpret_cast<float*>(base + C::kOffScale) + s * 3 * C::CP; }
  __device__ __forceinline__ volatile uint32_t* meta() const { return reinterpret_cast<uint32_t*>(base + C::kOffMeta); }
  __device__ __forceinline__ volatile uint32_t* raw_meta() const { return reinterpret_cast<uint32_t*>(base + C::kOffRawMeta); }
  __device__ __forceinline__ float* meet(int y) const { return reinterpret_cast<float*>(base + C::kOffRow) + y * 2 * kSharedTile; }
  __device__ __forceinline__ int* rows(int x) const { return reinterpret_cast<int*>(meet(x)); }  // (the stream's own place)
  __device__ __forceinline__ uint32_t* tmem() const { return reinterpret_cast<uint32_t*>(base + C::kOffTmem); }
  // barriers
  __device__ __forceinline__ uint64_t* op_full(int s) const { return bar + s; }
  __device__ __forceinline__ uint64_t* op_empty(int s) const { return bar + C::kOps + s; }
  __device__ __forceinline__ uint64_t* raw_full(int s) const { return bar + 2 * C::kOps + s; }
  __device__ __forceinline__ uint64_t* raw_empty(int s) const { return bar + 2 * C::kOps + C::kRaws + s; }
  __device__ __forceinline__ uint64_t* sc_empty(int s) const { return bar + 2 * C::kOps + 2 * C::kRaws + s; }
  __device__ __forceinline__ uint64_t* rest(int i) const { return bar + 2 * C::kOps + 2 * C::kRaws + C::kRings + i; }
  __device__ __forceinline__ uint64_t* s_full(int x) const { return rest(x); }       // scores of a step are there
  __device__ __forceinline__ uint64_t* p_full(int x) const { return rest(2 + x); }   // its weights are
  __device__ __forceinline__ uint64_t* pv_done(int x) const { return rest(4 + x); }  // its product P V is
  __device__ __forceinline__ uint64_t* q_full(int x) const { return rest(6 + x); }   // a stream's queries are
  __device__ __forceinline__ uint64_t* drain() const { return rest(8); }
  // (By their addresses in shared memory: through generic pointers, whose halves were kept in
  // registers, 128 x 1 behind 16384 took 66.6 us, so 66.1.)
  __device__ __forceinline__ void put_word(int off, uint32_t x) const {
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(smem_u32(base) + off), "r"(x) : "memory");
  }
  __device__ __forceinline__ uint32_t word(int off) const {
    uint32_t r;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(r) : "r"(smem_u32(base) + off) : "memory");
    return r;
  }
  __device__ __forceinline__ bool failed() const { return word(C::kOffFailed) != 0u; }
  __device__ __forceinline__ void fail() const { put_word(C::kOffFailed, 1u); }
  __device__ __forceinline__ uint32_t last(int st) const { return word(C::kOffLast + 4 * st); }

  // A whole warp's wait.  Its lanes go on together: one that fell behind, and that
  // nothing else waits for, could otherwise look for a phase when the next but one
  // has already come, which has the same parity.
  //   False: it gave up, or another warp of the CTA has; from then on a wait of the CTA
  // lasts two looks (4 us each).  Loads, widening and multiplies then end.  The softmax's
  // warps go on, over scores that mean nothing, to the end of the run: they meet at
  // named barriers, which have no limit, so one of them that left would hold up those
  // that did not fail.  What they write lies in the CTA's own partials.
  __device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity) const {
    bool ok = mbar_try_wait(b, parity);
    if (!ok) {
      const unsigned long long t0 = globaltimer_ns();
      for (uint32_t i = 1;; ++i) {
        ok = mbar_try_wait(b, parity);
        if (ok || failed()) break;
        if (((i & 255u) == 0u || limit_ns < 1000000u) && globaltimer_ns() - t0 > limit_ns) {
          fail();
          break;
        }
      }
    }
    return __all_sync(0xffffffffu, ok);
  }
};

// What a chunk holds: the pages that are there (bits 0-7); whether it is even (bit
// 8): over an 8-bit cache the exponents of its keys lie within 15 of one another,
// and those of its values within 7, so that f16 holds the codes exactly times
// 2^(exponent - largest); whether it is plain: even, and all pages there; then the largest
// exponents (bytes, bits 16 and 24).
constexpr uint32_t kShEven = 256u, kShPlain = 512u;
__device__ __forceinline__ float sh_meta_key(uint32_t m) { return __uint_as_float(((m >> 16) & 255u) << 23); }
__device__ __forceinline__ float sh_meta_value(uint32_t m) { return (float)((int)(m >> 24) - 127); }

// ------------------------------------------------------------------ loads
// The operands of a CTA's run in the order of their loads.
template <class C>
struct ShItems {
  ShRun<C::NS> run;
  ShSegment s;
  ShOrder ord;
  int i;
  uint32_t at;                // the item's number
  uint32_t chunk_no, chunk0;  // chunks before the segment; number of the item's chunk
  int c;                      // the item's chunk within its segment
  bool is_v, more;
  __device__ __forceinline__ ShItems(const SharedParams& p)
      : run(p, blockIdx.x), ord{0, false}, i(-1), at(0xffffffffu), chunk_no(0), more(true) {}
  // To the next item (the first one at first); more: there is one.
  __device__ __forceinline__ void step() {
    ++at;
    if (++i == 2 * ord.n) {
      chunk_no += ord.n;
      i = 0;
      more = run.next(s);
      if (!more) return;
      ord = {s.i1 - s.i0, s.w == 2};
    }
    c = ord.item(i, is_v);
    chunk0 = chunk_no + c;
  }
};

// A warp for K and one for V.  Lane l < kPages looks up page l of a chunk; its part
// of the operand: boxes of a bf16 page straight into the operand's layout (a page
// that is not there reads as zeros: a row beyond the tensor), or an 8-bit page's
// codes.  Page numbers are looked up two operands ahead.
template <class C, bool kValues>
__device__ void sh_load(const SharedParams& p, const CUtensorMap* map, const ShSmem<C>& sm) {
  const int lane = threadIdx.x & 31;
  const uint32_t lead = tc_elect();
  ShItems<C> it(p);
  struct Item {
    int page, kvh;
    bool there, wanted;  // there: an item at all; wanted: with a page for this lane
    uint32_t at, chunk;
  };
  Item now = {-1, 0, false, false, 0, 0}, next = now;
  constexpr uint32_t kRing = C::kBf16 ? C::kOps : C::kRaws;
  const uint64_t pol = policy_evict_last();
  for (int k = 0;; ++k) {
    // the operand two on: its page numbers
    Item far = {-1, 0, false, false, 0, 0};
    do {
      if (it.more) it.step();
    } while (it.more && it.is_v != kValues);
    if (it.more) {
      const int pos = (it.s.i0 + it.c) * C::CP + lane * kPage;
      far.there = true;
      far.wanted = lane < C::kPages && pos < it.s.g.eff;
      if (far.wanted) far.page = __ldcg(p.a.rows.table + (size_t)it.s.g.s0 * p.a.rows.table_stride + pos / kPage);
      far.kvh = it.s.kvh;
      far.at = it.at;
      far.chunk = it.chunk0;
    }
    if (!now.there) {  // (the first two rounds, or the end)
      if (k >= 2) break;
      now = next;
      next = far;
      continue;
    }
    const uint32_t at = now.at;
    const int st = at % kRing;
    if (at >= kRing && !sm.wait(C::kBf16 ? sm.op_empty(st) : sm.raw_empty(st), ((at / kRing) & 1u) ^ 1u)) return;
    if (lead) sm.put_word(C::kOffLast + 4 * st, at + 1);
    const bool have = (uint32_t)now.page < (uint32_t)p.a.n_pages;
    uint4 ke = make_uint4(0u, 0u, 0u, 0u), ve = ke;
    if (!C::kBf16 && have) {
      const size_t ph = (size_t)now.page * p.a.n_kv_heads + now.kvh;
      if (p.a.block == 1) {
        ke = __ldcg(reinterpret_cast<const uint4*>(p.a.k_exp) + ph);
        ve = __ldcg(reinterpret_cast<const uint4*>(p.a.v_exp) + ph);
      } else {
        const uint32_t a = __ldcg(p.a.k_exp + ph) * 0x01010101u, b = __ldcg(p.a.v_exp + ph) * 0x01010101u;
        ke = make_uint4(a, a, a, a);
        ve = make_uint4(b, b, b, b);
      }
    }
    if (!kValues && !have && now.wanted && p.a.status) atomicOr(p.a.status, ST_BAD_PAGE);
    const uint32_t there = __ballot_sync(0xffffffffu, have);
    uint32_t meta = there | kShEven;
    const uint32_t plain = there == (1u << C::kPages) - 1u ? kShPlain : 0u;
    // (row of the pool's positions; none beyond the last)
    const int row = have ? (now.page * p.a.n_kv_heads + now.kvh) * kPage : p.a.n_pages * p.a.n_kv_heads * kPage;
    if constexpr (C::kBf16) {
      if (lead) {
        if (!kValues) sm.meta()[now.chunk & 7] = meta | plain;
        mbar_arrive_expect_tx(sm.op_full(st), C::kOpBytes);
      }
      __syncwarp();
#pragma unroll 1
      for (int pg = 0; pg < C::kPages; ++pg) {
        const int r = __shfl_sync(0xffffffffu, row, pg);
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h)
          if (lead) tma_load_2d(sm.op(st) + h * C::CP * 128 + pg * kPage * 128, map, h * 64, r, sm.op_full(st), pol);
      }
    } else {
      if (lead) mbar_arrive_expect_tx(sm.raw_full(st), (uint32_t)__popc(there) * kPage * C::D);
      __syncwarp();
      const uint8_t* pool = kValues ? p.a.v : p.a.k;
#pragma unroll 1
      for (int pg = 0; pg < C::kPages; ++pg) {
        const int r = __shfl_sync(0xffffffffu, row, pg);
        if (lead && (there >> pg & 1u))
          bulk_load(sm.raw(st) + pg * kPage * C::D, pool + (size_t)r * C::D, kPage * C::D, sm.raw_full(st));
      }
      // the exponents, while the codes are on their way
      // (bytes below the writer's smallest, as a zeroed cache has, count as that one for values)
      const uint32_t least = kExpMinByte * 0x01010101u;
      ve = make_uint4(__vmaxu4(ve.x, least), __vmaxu4(ve.y, least), __vmaxu4(ve.z, least), __vmaxu4(ve.w, least));
      auto top = [](const uint4& e) {
        const uint32_t m = __vmaxu4(__vmaxu4(e.x, e.y), __vmaxu4(e.z, e.w)), h = __vmaxu4(m, m >> 16);
        return max(h & 255u, (h >> 8) & 255u);
      };
      auto low = [](const uint4& e) {
        const uint32_t m = __vminu4(__vminu4(e.x, e.y), __vminu4(e.z, e.w)), h = __vminu4(m, (m >> 16) | (m << 16));
        return min(h & 255u, (h >> 8) & 255u);
      };
      const uint32_t kt = __reduce_max_sync(0xffffffffu, have ? top(ke) : 0u), kl = __reduce_min_sync(0xffffffffu, have ? low(ke) : 255u);
      const uint32_t vt = __reduce_max_sync(0xffffffffu, have ? top(ve) : 0u), vl = __reduce_min_sync(0xffffffffu, have ? low(ve) : 255u);
      if (kt == kExpNaN || vt == kExpNaN || kt > kl + kShKeySpread || vt > vl + kShValueSpread) meta &= ~kShEven;
      meta |= (kt << 16) | (vt << 24) | (meta & kShEven ? plain : 0u);
      if (lane < C::kPages) {
        if (!kValues) reinterpret_cast<uint4*>(sm.exps(st))[lane] = ke;
        reinterpret_cast<uint4*>(sm.exps(st) + C::CP)[lane] = ve;
      }
      if (lead) sm.raw_meta()[st] = meta;
      __syncwarp();
      if (lead) mbar_arrive(sm.raw_full(st));
    }
    now = next;
    next = far;
  }
}

// After a failure: the last copy into each place has landed, or the wait for it runs out.
template <class C>
__device__ void sh_load_drain(const ShSmem<C>& sm) {
  constexpr uint32_t kRing = C::kBf16 ? C::kOps : C::kRaws;
  for (uint32_t st = 0; st < kRing; ++st) {
    const uint32_t n = sm.last(st);
    if (n > 0) mbar_wait(C::kBf16 ? sm.op_full(st) : sm.raw_full(st), ((n - 1) / kRing) & 1u);
  }
}

// ------------------------------------------------------------------ 8-bit codes to f16 operands
// Four warps.  (Eight: 75 us for 128 x 1 behind 16384, with four 72.)  An even chunk's codes are scaled to its largest exponents; of
// another the codes go as they are, and the scores take the exponents (sm.scale).
template <class C>
__device__ void sh_widen(const SharedParams& p, const ShSmem<C>& sm) {
  constexpr int kWidth = 128;
  const int tid = threadIdx.x - C::kWidenWarp * 32;
  ShItems<C> it(p);
  for (;;) {
    it.step();
    if (!it.more) break;
    const uint32_t c = it.chunk0, at = it.at;
    const int st = at % C::kRaws, os = at % C::kOps;
    if (!sm.wait(sm.raw_full(st), (at / C::kRaws) & 1u)) return;
    if (at >= C::kOps && !sm.wait(sm.op_empty(os), ((at / C::kOps) & 1u) ^ 1u)) return;
    const uint32_t meta = sm.raw_meta()[st];
    const bool even = meta & kShEven;
    const uint8_t* exps = sm.exps(st) + (it.is_v ? C::CP : 0);
    const int most = it.is_v ? meta >> 24 : (meta >> 16) & 255;
    if (!it.is_v) {
      const int ring = c % C::kRings;
      if (c >= C::kRings && !sm.wait(sm.sc_empty(ring), ((c / C::kRings) & 1u) ^ 1u)) return;
      if (!even && tid < C::CP) {
        const uint32_t bk = sm.exps(st)[tid], bv = sm.exps(st)[C::CP + tid];
        float* f = sm.scale(ring);
        f[tid] = exp_byte_value(bk);
        f[C::CP + tid] = bv == kExpNaN ? exp_byte_value(bv) : (float)((int)bv - 127);
        f[2 * C::CP + tid] = __uint_as_float((254u - min(bv, 254u)) << 23);
      }
      if (tid == 0) sm.meta()[c & 7] = meta;
    }
    // A thread has a position (half of one of 256 codes), which has one exponent, in
    // units of 16 codes.  Lanes begin with different units: the eight of a quarter warp
    // then read eight different 16-byte columns and (128 codes a position) write eight.
    constexpr int kThreadsRow = kWidth / C::CP, kRowUnits = C::D / 16, kMine = kRowUnits / kThreadsRow;
    const int pos = tid / kThreadsRow, u0 = tid % kThreadsRow * kMine;
    const uint8_t* raw = sm.raw(st) + pos * C::D;
    const uint32_t dst = smem_u32(sm.op(os)) + pos * 128;
    const bool have = (meta >> (pos / kPage)) & 1u;
    uint32_t by = 0x3c003c00u;  // 1, or 2^(the position's exponent - the largest): at least 2^-15
    if (have && even) {
      const int e = exps[pos] - most;
      by = (e > -15 ? (uint32_t)(15 + e) << 10 : 0x0200u) * 0x00010001u;
    }
    auto scaled = [&](uint32_t h) {
      uint32_t r;
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(by));
      return r;
    };
    uint4 w[kMine];
    int unit[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      unit[k] = u0 + ((k + (C::D == 64 ? pos >> 1 : pos)) & (kMine - 1));
      w[k] = *reinterpret_cast<const uint4*>(raw + unit[k] * 16);
      if (!have) w[k] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const uint32_t half = dst + (unit[k] >> 2) * C::CP * 128, col = 2 * (unit[k] & 3);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool second = (kThreadsRow == 1 ? e : e ^ (tid & 1)) != 0;
        const uint32_t a = second ? w[k].z : w[k].x, b = second ? w[k].w : w[k].y;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(half + (((col + second) ^ (pos & 7)) << 4)), "r"(scaled(f16x2_of_lo(a))),
                     "r"(scaled(f16x2_of_hi(a))), "r"(scaled(f16x2_of_lo(b))), "r"(scaled(f16x2_of_hi(b)))
                     : "memory");
      }
    }
    fence_proxy_async_smem();  // the multiplies read the operand through the async proxy, and copies overwrite the codes
    mbar_arrive(sm.op_full(os));
    mbar_arrive(sm.raw_empty(st));
  }
}

// ------------------------------------------------------------------ multiplies
// A place in the ring of operands, and the parity of its phase.
template <int N>
struct ShPlace {
  uint32_t slot, phase;
  __device__ __forceinline__ void go(uint32_t n) {  // (n <= N)
    slot += n;
    if (slot >= N) {
      slot -= N;
      phase ^= 1u;
    }
  }
};

// One warp, of which one lane issues.  The tensor cores take a multiply of 128 x 128 x
// 16 every 64 cycles and hold some eight of them ahead: what the warp does between two
// batches is kept to a few instructions.
template <class C>
__device__ void sh_multiply(const SharedParams& p, const ShSmem<C>& sm, uint32_t tmem) {
  constexpr int CP = C::CP, D = C::D;
  constexpr uint32_t kScores = sh_idesc<C>(CP, false), kValues = sh_idesc<C>(D, true);
  const uint32_t lead = tc_elect();
  tmem = sh_uniform(tmem);
  ShRun<C::NS> run(p, blockIdx.x);
  ShSegment s;
  // parities: of the streams' queries, of the two score places (a bit each).  A segment of a
  // single step has none for the second stream, which does not arrive for it either: it
  // may be several such segments ahead, or one behind.
  uint32_t seg = 0, steps = 0;
  bool ok = true;
  ShPlace<C::kOps> k = {0, 0};
  const uint64_t q_desc = tc_sdesc(sh_uniform(smem_u32(sm.q(0))));
  const uint32_t op_base = sh_uniform(smem_u32(sm.op(0)));
  const uint64_t k_desc = tc_sdesc(op_base), v_desc = tc_sdesc_mn(op_base, CP * 128);
  while (ok && run.next(s)) {
    const int chunks = (int)sh_uniform(s.i1 - s.i0);
    const bool both = sh_uniform(s.w) == 2u;
    const int n = both ? 2 * chunks : chunks;
    ShPlace<C::kOps> v = k;
    v.go(both || n == 1 ? 1 : 2);
    for (int j = -2; j < n; ++j) {
      const uint32_t x = j & 1, stream = C::NS == 2 ? x : 0;
      const bool last = !both || x;  // of the steps with these operands
      if (j >= 0) {
        ok = sm.wait(sm.p_full(x), steps >> x & 1u) && sm.wait(sm.op_full(v.slot), v.phase);
        if (!ok) break;
        steps ^= 1u << x;
        tc_fence_after();
        const uint64_t b = v_desc + v.slot * (C::kOpBytes >> 4);
        const uint32_t o = tmem + C::kOutCol + stream * D, w = tmem + x * C::kScoreCol;
#pragma unroll
        for (int t = 0; t < (C::kBf16 ? 2 : 1); ++t)
#pragma unroll
          for (int i = 0; i < CP / 16; ++i)
            tc_mma_ts_if(lead, o, w + (i / 2) * 32 + t * 16 + (i % 2) * 8, b + (i * 16 * 128 >> 4), kValues, j >= C::NS || t > 0 || i > 0);
        tc_commit_if(lead, sm.pv_done(x));
        if (last) {
          tc_commit_if(lead, sm.op_empty(v.slot));
          v.go(!both && j == n - 2 ? 1 : 2);
        }
      }
      if (j + 2 < n) {
        ok = (j + 2 >= C::NS || sm.wait(sm.q_full(stream), seg >> stream & 1u)) && sm.wait(sm.op_full(k.slot), k.phase);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = q_desc + stream * (C::kQBytes >> 4), b = k_desc + k.slot * (C::kOpBytes >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          tc_mma_if(lead, tmem + x * C::kScoreCol, a + (((i / 4) * kSharedTile * 128 + (i % 4) * 32) >> 4),
                    b + (((i / 4) * CP * 128 + (i % 4) * 32) >> 4), kScores, i > 0);
        tc_commit_if(lead, sm.s_full(x));
        if (last) {
          tc_commit_if(lead, sm.op_empty(k.slot));
          k.go(!both && j == -2 ? 1 : 2);
        }
      }
    }
    // the next segment's first operand is behind the last of V: v went by two from there
    k.slot = v.slot == 0 ? C::kOps - 1 : v.slot - 1;
    k.phase = v.slot == 0 ? v.phase ^ 1u : v.phase;
    seg ^= C::NS == 2 && n > 1 ? 3u : 1u;
  }
  // every multiply has completed before tensor memory is freed
  tc_commit_if(lead, sm.drain());
  if (!mbar_wait(sm.drain(), 0)) sm.fail();
  __syncwarp();
}

// ------------------------------------------------------------------ softmax
// A stream: two warpgroups, thread r of each has query row r of the tile, the first
// the lower half of a chunk's positions, the second the upper one.
template <class C>
struct ShSoft {
  static constexpr int CP = C::CP, D = C::D, W = CP / 2;  // W: a thread's positions of a chunk
  const SharedParams& p;
  const ShSmem<C>& sm;
  const int x, h, r;        // stream, half, row of the tile
  const uint32_t lane_off;  // the warp's lanes of tensor memory
  const uint32_t tmem;
  float ref, l, fac;
  uint32_t most;               // largest value exponent (byte) of the segment's chunks so far
  uint32_t steps0 = 0, steps1 = 0;  // steps of each score place so far

  __device__ __forceinline__ ShSoft(const SharedParams& p_, const ShSmem<C>& sm_, uint32_t tm)
      : p(p_), sm(sm_), x(threadIdx.x >> 8), h((threadIdx.x >> 7) & 1), r(threadIdx.x & 127), lane_off((uint32_t)(threadIdx.x & 96) << 16), tmem(tm) {}

  __device__ __forceinline__ uint32_t steps(int y) const { return y ? steps1 : steps0; }
  __device__ __forceinline__ void open() {
    ref = kShNone;
    l = 0.0f;
    most = 0;
  }

  // The tile's queries, as an operand of 64-column halves with 128-byte swizzled
  // rows: copied there as they are, then scaled in place, a row a thread.  Their
  // factor is positive (the sign goes to the queries), so that the largest product is
  // the largest score.
  __device__ __forceinline__ void queries(const ShSegment& s, int tile, int G) {
    constexpr int U = D / 8;  // 16-byte units of a row
    const uint32_t dst = smem_u32(sm.q(x));
    const int f0 = tile * kSharedTile;
    if (h == 0) sm.rows(x)[r] = f0 + r < s.g.R ? (f0 + r) / G : -1;
    meet();
    const bf16* q = p.a.q + (int64_t)s.g.row0 * p.a.q_stride + s.kvh * G * D;
#pragma unroll 4
    for (int i = 0; i < U / 2; ++i) {
      const int idx = (2 * i + h) * 128 + r, row = idx / U, u = idx % U;
      const int token = sm.rows(x)[row], head = f0 + row - token * G;
      const uint32_t to = dst + (u >> 3) * kSharedTile * 128 + row * 128 + (((u & 7) ^ (row & 7)) << 4);
      if (token >= 0)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(q + token * p.a.q_stride + head * D + u * 8) : "memory");
      else
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0u) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    meet();
    const uint32_t flip = p.a.scale_log2 < 0.0f ? 0x80008000u : 0u;
    fac = fmaxf(fabsf(p.a.scale_log2), 0x1p-126f);  // (and not zero: a score of -infinity stays one)
    auto unit = [&](int u) { return dst + (u >> 3) * kSharedTile * 128 + r * 128 + (((u & 7) ^ (r & 7)) << 4); };
    auto load = [&](int u) {
      uint4 w;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(unit(u)));
      return w;
    };
    float down = 1.0f;
    if (!C::kBf16) {
      uint32_t m = 0;
#pragma unroll 4
      for (int u = 0; u < U; ++u) {
        const uint4 w = load(u);
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
      }
      m = max(m & 0xffffu, m >> 16);
      // the row's largest exponent E: q / 2^(E - 127) is below 2 (an infinity or NaN makes the row NaN)
      const int E = min(max((int)(m >> 7), 1), 253);
      down = __uint_as_float((uint32_t)(254 - E) << 23);
      fac = m >= 0x7f80u ? __uint_as_float(0x7fffffffu) : __fmul_rn(fac, __uint_as_float((uint32_t)E << 23));
      meet();  // (both halves have looked)
    }
    if (!C::kBf16 || flip) {
#pragma unroll 2
      for (int u = h * U / 2; u < (h + 1) * U / 2; ++u) {
        uint4 w = load(u);
        auto two = [&](uint32_t v) {
          if (!C::kBf16) v = sh_f16x2(__fmul_rn(__uint_as_float(v << 16), down), __fmul_rn(__uint_as_float(v & 0xffff0000u), down));
          return v ^ flip;
        };
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(unit(u)), "r"(two(w.x)), "r"(two(w.y)), "r"(two(w.z)), "r"(two(w.w))
                     : "memory");
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(sm.q_full(x));
    open();
  }

  __device__ __forceinline__ uint32_t scores_at(int y) const { return tmem + lane_off + y * C::kScoreCol + h * W; }
  __device__ __forceinline__ void meet() const { named_sync(1 + x, 256); }
  // The larger of both halves' numbers of the row (on score place y).  The next ones
  // are written when this step's weights, which both give, have been used.
  __device__ __forceinline__ float larger(float v, int y) const {
    float* s = sm.meet(y);
    s[h * kSharedTile + r] = v;
    meet();
    return fmaxf(v, s[(h ^ 1) * kSharedTile + r]);
  }

  // The reference follows a row's largest score `top` of step j where it has risen by more than the slack.
  __device__ __forceinline__ void follow(float top, int j, int y) {
    constexpr float kBias = sh_bias(C::kBf16);
    const bool up = __fsub_rn(top, ref) > kShSlack + kBias;  // (the difference is exact, a sum need not be)
    if (!__any_sync(0xffffffffu, up)) return;
    top = __fsub_rn(top, kBias);
    const float d = up ? __fsub_rn(ref, top) : 0.0f, a = sh_ex2(d);
    const bool scaled = up && ref != kShNone;
    l = sh_times_ex2(l, d);
    ref = up ? top : ref;
    if (!__any_sync(0xffffffffu, scaled)) return;  // (behind a row's first chunk there is nothing to scale)
    // the product before this step (with two streams it ran before these scores did)
    if (C::NS == 1 && j > 0) sm.wait(sm.pv_done(y ^ 1), (steps(y ^ 1) - 1u) & 1u);
    tc_fence_after();
    const uint32_t o = tmem + lane_off + C::kOutCol + (C::NS == 2 ? x : 0) * D;
#pragma unroll 1
    for (int c = h * D / 2; c < (h + 1) * D / 2; c += 32) {
      uint32_t v[32];
      tc_ld32(o + c, v);
      tc_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__fmul_rn(__uint_as_float(v[e]), a));
      tc_st32(o + c, v);
    }
    tc_wait_st();
  }

  // 32 columns' weights over their scores, where the product reads them: two 16-bit
  // values a column, 16 columns; of a bf16 cache the second terms in the other 16.
  __device__ __forceinline__ void put(uint32_t place, const uint32_t (&w)[32]) {
    uint32_t hi[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)  // (a bf16 weight's first term: its upper half)
      hi[e] = C::kBf16 ? __byte_perm(w[2 * e], w[2 * e + 1], 0x7632)
                       : sh_f16x2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
    tc_st16(place, hi);
    if (C::kBf16) {  // the second: the rest, rounded
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        uint32_t a, b;  // (a weight is not negative: its upper half with the sign set is what is taken off)
        split(add2(pair_of(w[2 * e], w[2 * e + 1]), pair_of((w[2 * e] & 0xffff0000u) | 0x80000000u, (w[2 * e + 1] & 0xffff0000u) | 0x80000000u)), a, b);
        hi[e] = pack_bf16x2(__uint_as_float(a), __uint_as_float(b));
      }
      tc_st16(place + 16, hi);
    }
  }

  // From a product to a score.  Not infinite, so that a product of zero is a score of
  // zero; a NaN where the query row has one, or an infinity.
  __device__ __forceinline__ float factor(float key) const {
    if (C::kBf16) return fac;
    float f;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(__fmul_rn(fac, key)), "f"(FLT_MAX));
    return f;
  }

  // A plain chunk: t' = s f + ev for all of it.  Weights 2^(t' - ref); the
  // denominator takes them times 2^-ev, or where values of the segment have
  // exponents so much larger that a weight may be below fp32's range although its
  // share of the denominator counts, 2^(s f - ref).
  //   Scores are read twice, 32 columns at a time, in loops that are not unrolled
  // further: the warps' code then fits the instruction caches and their registers the
  // file.  (Nearly all of an SM's L1 is shared memory here: what a register spills
  // comes back from L2.)
  __device__ __forceinline__ void plain(int j, int y, uint32_t meta) {
    const uint32_t place = scores_at(y);
    uint32_t v[32];
    float m[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < W; c += 32) {
      tc_ld32(place + c, v);
      tc_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; i += 2) m[i / 2 & 1] = max3(m[i / 2 & 1], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
    }
    const float f = factor(sh_meta_key(meta)), ev = C::kBf16 ? 0.0f : sh_meta_value(meta);
    follow(__fmaf_rn(larger(fmaxf(m[0], m[1]), y), f, ev), j, y);
    bool far = false;
    if (!C::kBf16) {
      const uint32_t e = meta >> 24;
      most = max(most, e);
      far = e + 60u < most;
    }
    // Large scores: a reference is rounded, so the product less it, which is rounded once,
    // would not be what `follow` compared; take the rounded score less the reference.
    const bool big = __any_sync(0xffffffffu, fabsf(ref) > kShBig && ref != kShNone);
    const float fac1 = big ? 1.0f : f, off = big ? 0.0f : __fsub_rn(ev, ref), off_key = big ? -ev : -ref;
    const uint64_t f2 = pair_of(__float_as_uint(fac1), __float_as_uint(fac1)), off2 = pair_of(__float_as_uint(off), __float_as_uint(off));
    uint64_t sum2 = 0;
    float direct = 0.0f;
#pragma unroll 1
    for (int c = 0; c < W; c += 32) {
      tc_ld32(place + c, v);
      tc_wait_ld();
      if (big) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__fsub_rn(__fmaf_rn(__uint_as_float(v[i]), f, ev), ref));
      }
      if (!C::kBf16 && far) {
#pragma unroll
        for (int i = 0; i < 32; ++i) direct = __fadd_rn(direct, sh_ex2(__fmaf_rn(__uint_as_float(v[i]), fac1, off_key)));
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        uint32_t a, b;
        split(fma2(pair_of(v[i], v[i + 1]), f2, off2), a, b);
        v[i] = __float_as_uint(sh_ex2(__uint_as_float(a)));
        v[i + 1] = __float_as_uint(sh_ex2(__uint_as_float(b)));
        sum2 = add2(sum2, pair_of(v[i], v[i + 1]));
      }
      put(place + c, v);
    }
    uint32_t even_sum, odd_sum;
    split(sum2, even_sum, odd_sum);
    const float all = __fadd_rn(__uint_as_float(even_sum), __uint_as_float(odd_sum));
    if (C::kBf16) l = __fadd_rn(l, all);
    else l = far ? __fadd_rn(l, direct) : __fmaf_rn(all, __uint_as_float((254u - (meta >> 24)) << 23), l);
  }

  // Any chunk: pages may be missing, exponents differ by position (sc: 2^ek, ev, 2^-ev of each).
  __device__ __forceinline__ void uneven(int j, int y, uint32_t meta, const float* sc) {
    const uint32_t place = scores_at(y);
    const bool even = C::kBf16 || meta & kShEven;
    const float kf = factor(sh_meta_key(meta)), vs = C::kBf16 ? 0.0f : sh_meta_value(meta);
    const float iv = __uint_as_float((254u - (meta >> 24)) << 23);
    const uint32_t there = meta >> (h * (W / kPage));
    sc += h * W;
    uint32_t w[32];
    auto scores = [&](int c) {  // in log2 units, with the value's exponent
      tc_ld32(place + c, w);
      tc_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        // (rounded once, as a plain chunk's)
        const float t = C::kBf16 ? __fmul_rn(__uint_as_float(w[i]), fac)
                        : even   ? __fmaf_rn(__uint_as_float(w[i]), kf, vs)
                                 : __fmaf_rn(__uint_as_float(w[i]), factor(sc[c + i]), sc[CP + c + i]);
        w[i] = (there >> ((c + i) / kPage)) & 1u ? __float_as_uint(t) : 0xff800000u;
      }
    };
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < W; c += 32) {
      scores(c);
#pragma unroll
      for (int i = 0; i < 32; i += 2) top = max3(top, __uint_as_float(w[i]), __uint_as_float(w[i + 1]));
    }
    follow(larger(top, y), j, y);
    if (!C::kBf16) most = max(most, meta >> 24);
    float sum = 0.0f;
#pragma unroll 1
    for (int c = 0; c < W; c += 32) {
      scores(c);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float z = __fsub_rn(__uint_as_float(w[i]), ref), e = sh_ex2(z);
        if (C::kBf16)
          sum = __fadd_rn(sum, e);
        else if (z < kShFar)  // 2^z is below fp32's range, the position's share of the denominator need not be
          sum = __fadd_rn(sum, z == -INFINITY ? 0.0f : sh_ex2(__fsub_rn(z, even ? vs : sc[CP + c + i])));
        else
          sum = __fmaf_rn(e, even ? iv : sc[2 * CP + c + i], sum);
        w[i] = __float_as_uint(e);
      }
      put(place + c, w);
    }
    l = __fadd_rn(l, sum);
  }

  // Step j of the segment, on score place y: scores to weights.  no: the chunk's number in the call.
  // idle: the warp's rows are behind the tile's last.
  __device__ __forceinline__ void step(int j, int y, uint32_t no, bool both, bool idle) {
    sm.wait(sm.s_full(y), steps(y) & 1u);
    tc_fence_after();
    const uint32_t meta = sm.meta()[no & 7];
    if (idle) meet();  // (the weights of its rows may be anything: no product of another row's meets them)
    else if (meta & kShPlain) plain(j, y, meta);
    else uneven(j, y, meta, sm.scale(no % C::kRings));
    tc_wait_st();
    tc_fence_before();
    mbar_arrive(sm.p_full(y));
    __syncwarp();
    if (!C::kBf16 && (threadIdx.x & 31) == 0) {
      mbar_arrive(sm.sc_empty(no % C::kRings));
      if (C::NS == 2 && !both) mbar_arrive(sm.sc_empty(no % C::kRings));  // (a chunk that one stream alone has)
    }
    steps0 += y ^ 1;
    steps1 += y;
  }

  // The segment's partial.  n: steps of this stream; y: the last one's score place.
  __device__ __forceinline__ void partial(const ShSegment& s, int tile, int n, int y, int cta) {
    const int f = tile * kSharedTile + r;
    const long long at = (long long)x * p.plane + sh_slot(p, s.g, s.kvh, s.pair, C::NS, cta) + r;
    if (n > 0) {
      sm.wait(sm.pv_done(y), (steps(y) - 1u) & 1u);
      tc_fence_after();
      const uint32_t o = tmem + lane_off + C::kOutCol + (C::NS == 2 ? x : 0) * D;
      // through the warp's part of the stream's queries, which have done their work: 16
      // columns of its 32 rows at a time, so that a store writes 64 bytes of eight rows
      const int lane = threadIdx.x & 31;
      const uint32_t stage = smem_u32(sm.q(x)) + ((threadIdx.x >> 5) & 7) * (C::kQBytes / 8);
      const int rows = s.g.R - (f - lane);  // of the warp's that are there
      float* out = p.o + (at - lane) * D;
#pragma unroll 1
      for (int c = h * D / 2; c < (h + 1) * D / 2; c += 32) {
        uint32_t v[32];
        tc_ld32(o + c, v);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)), "r"(v[16 * k + 4 * e]),
                         "r"(v[16 * k + 4 * e + 1]), "r"(v[16 * k + 4 * e + 2]), "r"(v[16 * k + 4 * e + 3])
                         : "memory");
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = e * 8 + lane / 4, u = lane & 3;
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(stage + row * 64 + ((u ^ ((row >> 1) & 3)) << 4)));
            if (row < rows) *reinterpret_cast<uint4*>(out + row * D + c + 16 * k + 4 * u) = w;
          }
          __syncwarp();
        }
      }
      tc_fence_before();
    }
    float* sum = sm.meet(y);
    if (h == 1) sum[r] = l;
    meet();
    if (h == 0 && f < s.g.R) p.ml[at] = make_float2(ref, __fadd_rn(l, sum[r]));
    meet();  // (the place is free again)
  }

  __device__ void run() {
    const int G = p.a.n_q_heads / p.a.n_kv_heads;
    ShRun<C::NS> run(p, blockIdx.x);
    ShSegment s;
    uint32_t chunk_no = 0;
    while (run.next(s)) {
      const ShOrder ord{s.i1 - s.i0, s.w == 2};
      const int n = ord.steps(), tile = s.pair * C::NS + (ord.both ? x : 0);
      if (x < n) queries(s, tile, G);
      else open();
      const bool idle = tile * kSharedTile + (r & 96) >= s.g.R;
      int mine = 0, y = C::NS == 2 ? x : 0;
      for (int j = C::NS == 2 ? x : 0; j < n; j += C::NS) {
        y = j & 1;
        step(j, y, chunk_no + ord.chunk(j), ord.both, idle);
        ++mine;
      }
      partial(s, tile, mine, y, blockIdx.x);
      chunk_no += ord.n;
    }
  }
};

template <int D, int FMT>
__global__ void __launch_bounds__(ShCfg<D, FMT>::kThreads, 1)
    k_shared_prefix(const __grid_constant__ SharedParams p, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap) {
  using C = ShCfg<D, FMT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const ShSmem<C> sm(smem, p.wait_ns);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  if (C::kBf16 && threadIdx.x == C::kLoadWarp * 32) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kOps; ++i) {
      mbar_init(sm.op_full(i), C::kBf16 ? 1 : 128);
      mbar_init(sm.op_empty(i), 1);
    }
    for (int i = 0; i < C::kRaws; ++i) {
      mbar_init(sm.raw_full(i), 2);  // (the codes are asked for, the exponents are there)
      mbar_init(sm.raw_empty(i), 128);
    }
    for (int i = 0; i < C::kRings; ++i) mbar_init(sm.sc_empty(i), C::kSoftWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(sm.s_full(i), 1);
      mbar_init(sm.p_full(i), 256);
      mbar_init(sm.pv_done(i), 1);
      mbar_init(sm.q_full(i), 256);
    }
    mbar_init(sm.drain(), 1);
    fence_barrier_init();
    sm.put_word(C::kOffFailed, 0u);
    for (int i = 0; i < 8; ++i) sm.put_word(C::kOffLast + 4 * i, 0u);
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(sm.tmem())) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem();
  pdl_wait();  // the plan
  pdl_trigger();
  if (warp < C::kSoftWarps) {
    ShSoft<C>(p, sm, tmem).run();
  } else if (warp == C::kMmaWarp) {
    sh_multiply<C>(p, sm, tmem);
  } else if (warp == C::kLoadWarp) {
    sh_load<C, false>(p, &kmap, sm);
  } else if (warp == C::kLoadWarp + 1) {
    sh_load<C, true>(p, &vmap, sm);
  } else if (warp >= C::kWidenWarp) {
    if constexpr (!C::kBf16) sh_widen<C>(p, sm);
  }
  tc_fence_before();
  __syncthreads();
  if (sm.failed()) {  // (without a failure every copy has been waited for by what reads it)
    if (threadIdx.x == 0 && p.a.status) atomicOr(p.a.status, ST_TIMEOUT);
    if (warp == C::kLoadWarp) sh_load_drain<C>(sm);
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ------------------------------------------------------------------ merge
// Column c of a row over a bf16 cache where a partial, or the partials' sum, is not
// finite: the sum of the infinite values that the row sees (with a NaN, or both
// signs, a NaN), or where there are none the mean of the partials times 2^-24
// (see far_value in attend_dev.cuh).
template <int D>
__device__ __noinline__ float sh_far_value(const SharedParams& p, const int* table, int t, int kvh, int c, bool partials_fine,
                                           float scaled_mean) {
  if (partials_fine) return scaled_mean;
  const bf16* v = reinterpret_cast<const bf16*>(p.a.v);
  float infinite = 0.0f;
  const int end = min(t + 1, p.a.rows.limit());
  for (int pos = 0; pos < end; pos += 4) {
    const int page = __ldg(table + pos / kPage);
    if ((uint32_t)page >= (uint32_t)p.a.n_pages) continue;
    const bf16* column = v + (((size_t)page * p.a.n_kv_heads + kvh) * kPage + pos % kPage) * D + c;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __bfloat162float(column[i * D]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (pos + i < end && !(fabsf(x[i]) < INFINITY)) infinite = __fadd_rn(infinite, x[i]);
    if (infinite != infinite) return infinite;
  }
  return infinite != 0.0f ? infinite : scaled_mean;
}

// The partials of one (row, query head): segments of the prefix, then splits of the
// row's own positions.  W warps (of a block of eight) take every W-th of them each and
// add up in order.
template <int D, bool kBf16, int W>
__global__ void __launch_bounds__(256) k_shared_merge(const __grid_constant__ SharedParams p) {
  constexpr int V = D / 32, NS = shared_streams(D), B = V == 8 ? 4 : 8, kUnits = 8 / W;
  __shared__ float s_o[8][D], s_m[8], s_l[8];
  __shared__ int s_bad[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = warp % W, w0 = warp - mine;
  const int unit = blockIdx.x * kUnits + warp / W;
  const int H = p.a.n_q_heads, r = p.a.row_lo + unit / H, hq = unit % H, G = H / p.a.n_kv_heads, kvh = hq / G;
  int seq = 0, i = 0, t = -1, from = 0, gi = -1;
  const bool row = r < p.a.row_hi && find_row(p.a.rows, r, seq, i);
  pdl_trigger();
  // (the plan was complete before the prefix's kernel began its work, and that before
  // this one could start: only the partials are waited for)
  int c0 = 0, c1 = 0, planes = 1, plane = 0;  // the prefix: CTAs c0 .. c1 - 1, one or two partials each
  long long slot = 0;
  if (row) {
    from = __ldcg(p.from + seq);
    gi = __ldcg(p.group + seq);
    const SharedGroup end = sh_group(p.plan, p.n_groups);
    t = first_of(p.a.rows, seq) + i;
    if (t >= 0 && from > 0 && gi >= 0) {
      const SharedGroup g = sh_group(p.plan, gi);
      const int f = (r - g.row0) * G + hq % G, pair = f / (NS * kSharedTile), w = min(NS, g.tiles - pair * NS);
      const int first = g.unit0 + kvh * g.chunks * g.tiles + pair * NS * g.chunks;
      if (end.aligned) {
        c0 = sh_first(first, end.unit0, end.eff);
        c1 = sh_first(first + g.chunks * w, end.unit0, end.eff);
      } else {
        c0 = sh_owner(first, end.unit0, end.eff);
        c1 = sh_owner(first + (g.chunks - 1) * w, end.unit0, end.eff) + 1;
      }
      planes = w == 2 ? 1 : NS;
      plane = w == 2 ? f / kSharedTile & 1 : 0;
      slot = sh_slot(p, g, kvh, pair, NS, 0) + f % kSharedTile;
    }
  }
  const int n1 = (c1 - c0) * planes;
  // its own positions: the splits from `from` on
  const int last = min(t, p.a.rows.limit() - 1);
  const int s0 = last >= from ? attend_split_of(from) : 0, n2 = last >= from ? attend_split_of(last) - s0 + 1 : 0, n = n1 + n2;
  const size_t own = (size_t)unit * p.a.max_splits + s0;
  auto place = [&](int j) {  // of partial j < n1
    return (long long)(planes == 2 ? j & 1 : plane) * p.plane + slot + (long long)(c0 + (planes == 2 ? j >> 1 : j)) * kSharedTile;
  };
  auto sums_of = [&](int j) { return j < n1 ? p.ml + place(j) : p.a.part_ml + own + (j - n1); };
  auto out_of = [&](int j) { return j < n1 ? p.o + place(j) * D : p.a.part_o + (own + (j - n1)) * D; };
  pdl_wait();
  float M = kShNone, l = 0.0f, acc[V];
  bool bad = false;  // a partial that is not finite
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.0f;
  // this warp's partials, 32 references and sums at a time, then B accumulators (whose
  // loads need not wait for the sums: what has seen nothing is left out afterwards)
  for (int first = mine; first < n; first += 32 * W) {
    const int cnt = min(32, (n - first + W - 1) / W);
    float2 ml = make_float2(kShNone, 0.0f);
    if (lane < cnt) ml = __ldcg(sums_of(first + W * lane));
    float f = 0.0f;
    uint32_t some = 0;
    for (int b0 = 0; b0 < cnt; b0 += B) {
      float x[B][V];
#pragma unroll
      for (int b = 0; b < B; ++b) {
#pragma unroll
        for (int e = 0; e < V; ++e) x[b][e] = 0.0f;
        if (b0 + b >= cnt) continue;
        const float* src = out_of(first + W * (b0 + b)) + lane * V;
        if constexpr (V == 2) {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
          x[b][0] = v.x; x[b][1] = v.y;
        } else {
#pragma unroll
          for (int e = 0; e < V; e += 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src + e));
            x[b][e] = v.x; x[b][e + 1] = v.y; x[b][e + 2] = v.z; x[b][e + 3] = v.w;
          }
        }
      }
      if (b0 == 0) {
        // (a partial that has seen nothing has no accumulators; one of NaN scores has a NaN sum)
        const bool saw = !(ml.y == 0.0f);
        some = __ballot_sync(0xffffffffu, saw);
        float top = saw ? ml.x : kShNone;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, M);
        const float d0 = __fsub_rn(M, top), f0 = sh_ex2(d0), d = __fsub_rn(ml.x, top);
        f = saw ? sh_ex2(d) : 0.0f;
        float part = saw ? sh_times_ex2(ml.y, d) : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part = __fadd_rn(part, __shfl_xor_sync(0xffffffffu, part, o));
        l = __fadd_rn(sh_times_ex2(l, d0), part);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = d0 < 0.0f ? __fmul_rn(acc[e], f0) : acc[e];
        M = top;
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const float fb = __shfl_sync(0xffffffffu, f, b0 + b);
        if (b0 + b < 32 && (some >> (b0 + b)) & 1u) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            if (kBf16) bad |= !(fabsf(x[b][e]) < INFINITY);
            acc[e] = __fmaf_rn(x[b][e], fb, acc[e]);
          }
        }
      }
    }
  }
  if (W > 1) {
    const int any = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = l;
      s_bad[warp] = any;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = acc[e];
    __syncthreads();
  }
  if (!row) return;
  // the unit's warps take D / W columns each: lane's column c, c + 32, ...
  float f[W];
  if (W > 1) {
    M = kShNone;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, s_m[w0 + w]);
    l = 0.0f;
    bad = false;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float d = __fsub_rn(s_m[w0 + w], M);
      f[w] = sh_ex2(d);
      l = __fadd_rn(l, sh_times_ex2(s_l[w0 + w], d));
      bad |= s_bad[w0 + w] != 0;
    }
  } else {
    bad = __any_sync(0xffffffffu, bad);
  }
  const bool none = l == 0.0f;
  constexpr int kCols = D / W >= 32 ? D / W / 32 : 1;
  bf16* out = p.a.out + (int64_t)r * p.a.out_stride + hq * D;
#pragma unroll
  for (int k = 0; k < (W > 1 ? kCols : V / 2); ++k) {
    float y[2];
    int c[2];
#pragma unroll
    for (int e = 0; e < (W > 1 ? 1 : 2); ++e) {
      float a = 0.0f;
      if (W > 1) {
        c[e] = (mine * kCols + k) * 32 + lane;
        if (c[e] >= D) break;
#pragma unroll
        for (int w = 0; w < W; ++w)
          if (!(s_l[w0 + w] == 0.0f)) a = __fmaf_rn(s_o[w0 + w][c[e]], f[w], a);
      } else {
        c[e] = lane * V + 2 * k + e;
        a = acc[2 * k + e];
      }
      y[e] = none ? 0.0f : __fdiv_rn(a, l);
      if (kBf16 && l == l && !none && !(fabsf(a) < INFINITY)) {
        // the sum again, of the partials times 2^-24
        float small = 0.0f;
        for (int j = 0; j < n; ++j) {
          const float2 ml = __ldcg(sums_of(j));
          if (!(ml.y == 0.0f)) small = __fmaf_rn(__ldcg(out_of(j) + c[e]), __fmul_rn(sh_ex2(__fsub_rn(ml.x, M)), 0x1p-24f), small);
        }
        y[e] = sh_far_value<D>(p, p.a.rows.table + (size_t)seq * p.a.rows.table_stride, t, kvh, c[e], !bad,
                               __fdiv_rn(small, __fmul_rn(l, 0x1p-24f)));
      }
      if (W > 1) out[c[e]] = __float2bfloat16_rn(y[e]);
    }
    if (W == 1) *reinterpret_cast<uint32_t*>(out + c[0]) = pack_bf16x2(y[0], y[1]);
  }
  if (p.a.lse && lane == 0 && mine == 0)
    p.a.lse[(size_t)r * H + hq] = none ? -INFINITY : __fmul_rn(__fadd_rn(M, log2f(l)), 0.6931471805599453f);
}

template <int D, int FMT>
cudaError_t shared_prepare() {
  using C = ShCfg<D, FMT>;
  return cudaFuncSetAttribute(k_shared_prefix<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
}

template <int D, int FMT>
cudaError_t shared_launch(const SharedParams& p, cudaStream_t s) {
  using C = ShCfg<D, FMT>;
  CUtensorMap km = {}, vm = {};
  if (C::kBf16) {
    const uint64_t rows = (uint64_t)p.a.n_pages * p.a.n_kv_heads * kPage;
    if (!make_bf16_map(&km, p.a.k, rows, D, kPage) || !make_bf16_map(&vm, p.a.v, rows, D, kPage)) return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_shared_prefix<D, FMT>, p, km, vm);
}

template <int D, int W>
cudaError_t shared_merge_t(const SharedParams& p, int64_t units, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((units * W + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.a.k_exp ? cudaLaunchKernelEx(&cfg, k_shared_merge<D, false, W>, p) : cudaLaunchKernelEx(&cfg, k_shared_merge<D, true, W>, p);
}

// Warps for a result: as many as the device holds at once, at most eight.
template <int D>
cudaError_t shared_merge_launch(const SharedParams& p, int num_sms, cudaStream_t s) {
  const int64_t units = (int64_t)(p.a.row_hi - p.a.row_lo) * p.a.n_q_heads, most = 16 * (int64_t)num_sms;
  if (units * 8 <= most) return shared_merge_t<D, 8>(p, units, s);
  if (units * 4 <= most) return shared_merge_t<D, 4>(p, units, s);
  if (units * 2 <= most) return shared_merge_t<D, 2>(p, units, s);
  return shared_merge_t<D, 1>(p, units, s);
}

}  // namespace
}  // namespace sv
