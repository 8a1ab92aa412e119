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
// warpgroup, so that one's products run beside the other's exponentials: two
// tiles of 128 query rows that share the chunks of K and V they load, or, of a
// single tile, the even and the odd chunks.  (Rows of 256 elements leave tensor
// memory for one stream only; its scores alternate between two places.)
//   Warps 0-3, 4-7: softmax of a stream, a query row a thread.  Scores are read from
//     tensor memory, the weights go back there over them as the A operand of P V.
//     The reference of a row moves only when its maximum rises by more than 2^8
//     over it, so the accumulators are seldom read back and rescaled.
//   Warp 8: one thread issues the multiplies.  Warp 9: loads.
//   Warps 12-15 (8-bit caches): codes to f16, once for all query rows of the CTA.
//
// Types, as in attend_dev.cuh: a bf16 cache's weights are the sum of two bf16
// values (2^-16); over an 8-bit cache weights are f16 and carry the value's
// exponent, t' = log2(e) s + ev, queries go to f16 divided by a power of two near
// their row's largest value; sums, references and accumulators are fp32.
//
// Work is divided as chunks of all (group, kv head, tiles) lists one behind the
// other, in equal runs for the CTAs; each CTA leaves a partial (reference, sum,
// accumulators) for each list its run touches, and the merge adds them in order.
#pragma once
#include "paged_dev.cuh"
#include "shared.h"
#include "tc_dev.cuh"

#include <cuda_fp16.h>

namespace sv {

bool make_bf16_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint32_t box_rows);

namespace {

constexpr float kShSlack = 8.0f;     // log2 of what a row's maximum may exceed its reference by
constexpr float kShNone = -3.0e38f;  // reference of a row that has seen nothing
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
  static constexpr int kThreads = kBf16 ? 384 : 512;
  // registers: of the launch, of a softmax thread, of the others (their sum must not be above the launch's)
  static constexpr int kRegs = kBf16 ? 168 : 128, kRegsSoft = kBf16 ? 232 : 200, kRegsOther = kBf16 ? 40 : 56;
  static_assert(2 * kRegsSoft + (kThreads / 128 - 2) * kRegsOther <= kThreads / 128 * kRegs, "registers of the warpgroups");
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
  static constexpr int kOffMask = kOffBar + kBars * 8;  // [8] pages of a chunk that are there
  static constexpr int kOffRawMask = kOffMask + 32;     // [8] the same for an item of codes
  static constexpr int kOffTmem = kOffRawMask + 32;
  static constexpr int kSmem = 1024 + kOffTmem + 16;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

// idesc of the two products: f16 or bf16 operands, fp32 accumulators; B of P V lies along N.
template <class C>
__device__ __forceinline__ constexpr uint32_t sh_idesc(int N, bool b_mn) {
  return (1u << 4) | (C::kBf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(kSharedTile >> 4) << 24);
}

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
  long long unit;  // of the list's first chunk
};

__device__ __forceinline__ SharedGroup sh_group(const SharedGroup* plan, int g) {
  SharedGroup r;
  const int4* src = reinterpret_cast<const int4*>(plan + g);
  const int4 a = __ldcg(src), b = __ldcg(src + 1);
  r.unit0 = (long long)(uint32_t)a.x | ((long long)a.y << 32);
  r.eff = a.z; r.s0 = a.w; r.row0 = b.x; r.R = b.y; r.chunks = b.z; r.tiles = b.w;
  return r;
}

// CTA that has unit u of U, of G CTAs.
__device__ __forceinline__ int sh_owner(long long u, long long U, int G) { return (int)(((u + 1) * G - 1) / U); }

template <int NS>
struct ShRun {
  const SharedGroup* plan;
  int n_groups, n_kv;
  long long u, hi;  // the next unit, the end of the CTA's
  int gi;           // group that u is in
  __device__ __forceinline__ ShRun(const SharedParams& p, int cta) : plan(p.plan), n_groups(p.n_groups), n_kv(p.a.n_kv_heads) {
    const SharedGroup end = sh_group(plan, n_groups);
    u = hi = 0;
    gi = -1;
    if (cta >= end.eff || end.unit0 == 0) return;
    u = end.unit0 * cta / end.eff;
    hi = end.unit0 * (cta + 1) / end.eff;
    int lo = 0, top = n_groups;
    while (top - lo > 1) {
      const int mid = (lo + top) >> 1;
      if (__ldcg(&plan[mid].unit0) <= u) lo = mid; else top = mid;
    }
    gi = lo;
  }
  __device__ __forceinline__ bool next(ShSegment& s) {
    while (u < hi) {
      s.g = sh_group(plan, gi);
      const long long per = (long long)s.g.chunks * s.g.tiles, at = u - s.g.unit0;
      if (at >= per * n_kv) {
        ++gi;
        continue;
      }
      s.kvh = (int)(at / per);
      const long long in = at - s.kvh * per;
      s.pair = (int)(in / ((long long)s.g.chunks * NS));
      s.w = min(NS, s.g.tiles - s.pair * NS);
      s.unit = s.g.unit0 + s.kvh * per + (long long)s.pair * NS * s.g.chunks;
      s.i0 = (int)((u - s.unit + s.w - 1) / s.w);
      s.i1 = (int)min((long long)s.g.chunks, (hi - s.unit + s.w - 1) / s.w);
      const bool rest = s.i1 == s.g.chunks;
      u = rest ? s.unit + (long long)s.g.chunks * s.w : hi;
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
  __device__ __forceinline__ ShSmem(uint8_t* b) : base(b), bar(reinterpret_cast<uint64_t*>(b + C::kOffBar)) {}
  __device__ __forceinline__ uint8_t* q(int x) const { return base + C::kOffQ + x * C::kQBytes; }
  __device__ __forceinline__ uint8_t* op(int s) const { return base + C::kOffOp + s * C::kOpBytes; }
  __device__ __forceinline__ uint8_t* raw(int s) const { return base + C::kOffRaw + s * C::kRawBytes; }
  __device__ __forceinline__ uint8_t* exps(int s) const { return base + C::kOffExp + s * 2 * C::CP; }
  __device__ __forceinline__ float* scale(int s) const { return reinterpret_cast<float*>(base + C::kOffScale) + s * 3 * C::CP; }
  __device__ __forceinline__ volatile int* mask() const { return reinterpret_cast<int*>(base + C::kOffMask); }
  __device__ __forceinline__ volatile int* raw_mask() const { return reinterpret_cast<int*>(base + C::kOffRawMask); }
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
};

// ------------------------------------------------------------------ loads
// One warp.  Lane l < kPages looks up page l of a chunk and asks for its part of
// the operand: boxes of a bf16 page straight into the operand's layout (a page that is not there reads as
// zeros: a row beyond the tensor), or an 8-bit page's codes and exponents.
template <class C>
__device__ bool sh_load(const SharedParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap, const ShSmem<C>& sm) {
  const int lane = threadIdx.x & 31;
  ShRun<C::NS> run(p, blockIdx.x);
  ShSegment s;
  uint32_t at = 0, chunk_no = 0;  // operands, and chunks, so far
  bool ok = true;
  while (ok && run.next(s)) {
    const int* table = p.a.rows.table + (size_t)s.g.s0 * p.a.rows.table_stride;
    const ShOrder ord{s.i1 - s.i0, s.w == 2};
    for (int i = 0; i < 2 * ord.n && ok; ++i, ++at) {
      bool is_v;
      const int c = ord.item(i, is_v);
      const int pos = (s.i0 + c) * C::CP + lane * kPage;
      int page = -1;
      if (lane < C::kPages && pos < s.g.eff) {
        page = __ldg(table + pos / kPage);
        if ((uint32_t)page >= (uint32_t)p.a.n_pages) {
          if (p.a.status && !is_v) atomicOr(p.a.status, ST_BAD_PAGE);
          page = -1;
        }
      }
      const int there = (int)__ballot_sync(0xffffffffu, page >= 0);
      if constexpr (C::kBf16) {
        const int st = at % C::kOps;
        if (at >= C::kOps && !mbar_wait(sm.op_empty(st), ((at / C::kOps) & 1u) ^ 1u)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          if (!is_v) sm.mask()[(chunk_no + c) & 7] = there;
          mbar_arrive_expect_tx(sm.op_full(st), C::kOpBytes);
        }
        __syncwarp();
        if (lane < C::kPages) {
          const int64_t row = page >= 0 ? ((int64_t)page * p.a.n_kv_heads + s.kvh) * kPage : (int64_t)p.a.n_pages * p.a.n_kv_heads * kPage;
          const uint64_t pol = policy_evict_last();
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_2d(sm.op(st) + h * C::CP * 128 + lane * kPage * 128, is_v ? vmap : kmap, h * 64, (int)row, sm.op_full(st), pol);
        }
      } else {
        const int st = at % C::kRaws;
        uint4 ke = make_uint4(0u, 0u, 0u, 0u), ve = ke;
        const size_t ph = page >= 0 ? (size_t)page * p.a.n_kv_heads + s.kvh : 0;
        if (page >= 0 && !is_v) {  // (the scores need both)
          if (p.a.block == 1) {
            ke = __ldg(reinterpret_cast<const uint4*>(p.a.k_exp) + ph);
            ve = __ldg(reinterpret_cast<const uint4*>(p.a.v_exp) + ph);
          } else {
            const uint32_t a = __ldg(p.a.k_exp + ph) * 0x01010101u, b = __ldg(p.a.v_exp + ph) * 0x01010101u;
            ke = make_uint4(a, a, a, a);
            ve = make_uint4(b, b, b, b);
          }
        }
        if (at >= C::kRaws && !mbar_wait(sm.raw_empty(st), ((at / C::kRaws) & 1u) ^ 1u)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (!is_v && lane < C::kPages) {
          reinterpret_cast<uint4*>(sm.exps(st))[lane] = ke;
          reinterpret_cast<uint4*>(sm.exps(st) + C::CP)[lane] = ve;
        }
        if (lane == 0) sm.raw_mask()[st] = there;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(sm.raw_full(st), (uint32_t)__popc(there) * kPage * C::D);
        __syncwarp();
        if (page >= 0)
          bulk_load(sm.raw(st) + lane * kPage * C::D, (is_v ? p.a.v : p.a.k) + ph * kPage * C::D, kPage * C::D, sm.raw_full(st));
      }
    }
    chunk_no += ord.n;
  }
  // copies in flight have landed before the CTA goes on
  __syncwarp();
  constexpr uint32_t kRing = C::kBf16 ? C::kOps : C::kRaws;
  if (lane == 0)
    for (uint32_t k = at > kRing ? at - kRing : 0; k < at; ++k) {
      if (!mbar_wait(C::kBf16 ? sm.op_full(k % kRing) : sm.raw_full(k % kRing), (k / kRing) & 1u)) break;
    }
  return ok;
}

// ------------------------------------------------------------------ 8-bit codes to f16 operands
template <class C>
__device__ bool sh_widen(const SharedParams& p, const ShSmem<C>& sm) {
  const int tid = threadIdx.x & 127;
  ShRun<C::NS> run(p, blockIdx.x);
  ShSegment s;
  uint32_t at = 0, chunk_no = 0;
  while (run.next(s)) {
    const ShOrder ord{s.i1 - s.i0, s.w == 2};
    for (int i = 0; i < 2 * ord.n; ++i, ++at) {
      bool is_v;
      const uint32_t c = chunk_no + ord.item(i, is_v);
      const int st = at % C::kRaws, os = at % C::kOps;
      if (!mbar_wait(sm.raw_full(st), (at / C::kRaws) & 1u)) return false;
      if (at >= C::kOps && !mbar_wait(sm.op_empty(os), ((at / C::kOps) & 1u) ^ 1u)) return false;
      const int there = sm.raw_mask()[st];
      if (!is_v) {
        const int ring = c % C::kRings;
        if (c >= C::kRings && !mbar_wait(sm.sc_empty(ring), ((c / C::kRings) & 1u) ^ 1u)) return false;
        if (tid < C::CP) {
          // (bytes below the writer's smallest, as a zeroed cache has, count as that one; 255: NaN)
          const uint32_t bk = sm.exps(st)[tid], bv = max((uint32_t)sm.exps(st)[C::CP + tid], (uint32_t)kExpMinByte);
          float* f = sm.scale(ring);
          f[tid] = exp_byte_value(bk);
          f[C::CP + tid] = bv == kExpNaN ? exp_byte_value(bv) : (float)((int)bv - 127);
          f[2 * C::CP + tid] = __uint_as_float((254u - min(bv, 254u)) << 23);
        }
        if (tid == 0) sm.mask()[c & 7] = there;
      }
      const uint8_t* raw = sm.raw(st);
      const uint32_t dst = smem_u32(sm.op(os));
      constexpr int kUnits = C::CP * C::D / 16, kRow = C::D / 16;  // 16 codes each; of a position
#pragma unroll
      for (int k = 0; k < kUnits / 128; ++k) {
        const int u = tid + k * 128, pos = u / kRow, c16 = u % kRow;
        uint4 w = *reinterpret_cast<const uint4*>(raw + u * 16);
        if (!((there >> (pos / kPage)) & 1)) w = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
        const uint32_t half = dst + (c16 >> 2) * C::CP * 128 + pos * 128;
        // a quarter warp's lanes write eight different 16-byte places of a 128-byte row
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int second = C::D == 64 ? e : e ^ ((c16 >> 2) & 1), unit = 2 * (c16 & 3) + second;
          const uint32_t a = second ? x[2] : x[0], b = second ? x[3] : x[1];
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(half + ((unit ^ (pos & 7)) << 4)), "r"(f16x2_of_lo(a)),
                       "r"(f16x2_of_hi(a)), "r"(f16x2_of_lo(b)), "r"(f16x2_of_hi(b))
                       : "memory");
        }
      }
      fence_proxy_async_smem();  // the multiplies read the operand through the async proxy, and copies overwrite the codes
      mbar_arrive(sm.op_full(os));
      mbar_arrive(sm.raw_empty(st));
    }
    chunk_no += ord.n;
  }
  return true;
}

// ------------------------------------------------------------------ multiplies
template <class C>
__device__ bool sh_multiply(const SharedParams& p, const ShSmem<C>& sm, uint32_t tmem) {
  constexpr int CP = C::CP, D = C::D;
  constexpr uint32_t kScores = sh_idesc<C>(CP, false), kValues = sh_idesc<C>(D, true);
  ShRun<C::NS> run(p, blockIdx.x);
  ShSegment s;
  uint32_t at0 = 0, step0 = 0, seg = 0;
  bool ok = true;
  uint32_t used[2] = {0, 0};  // uses of each score place so far
  while (ok && run.next(s)) {
    const ShOrder ord{s.i1 - s.i0, s.w == 2};
    const int n = ord.steps();
    auto scores = [&](int j) {
      const int x = j & 1, stream = C::NS == 2 ? x : 0, c = ord.chunk(j);
      const uint32_t at = at0 + ord.k_at(c);
      if (j < C::NS && !mbar_wait(sm.q_full(stream), seg & 1u)) return false;
      if (!mbar_wait(sm.op_full(at % C::kOps), (at / C::kOps) & 1u)) return false;
      tc_fence_after();
      const uint32_t a = smem_u32(sm.q(stream)), b = smem_u32(sm.op(at % C::kOps));
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        tc_mma(tmem + x * C::kScoreCol, tc_sdesc(a + (k / 4) * kSharedTile * 128 + (k % 4) * 32),
               tc_sdesc(b + (k / 4) * CP * 128 + (k % 4) * 32), kScores, k > 0);
      tc_commit(sm.s_full(x));
      if (!ord.both || x == 1) tc_commit(sm.op_empty(at % C::kOps));
      return true;
    };
    ok = scores(0) && (n < 2 || scores(1));
    for (int j = 0; j < n && ok; ++j) {
      const int x = j & 1, stream = C::NS == 2 ? x : 0, c = ord.chunk(j);
      const uint32_t at = at0 + ord.v_at(c);
      ok = mbar_wait(sm.p_full(x), used[x] & 1u) && mbar_wait(sm.op_full(at % C::kOps), (at / C::kOps) & 1u);
      if (!ok) break;
      ++used[x];
      tc_fence_after();
      const uint32_t b = smem_u32(sm.op(at % C::kOps)), o = tmem + C::kOutCol + stream * D, w = tmem + x * C::kScoreCol;
#pragma unroll
      for (int t = 0; t < (C::kBf16 ? 2 : 1); ++t)
#pragma unroll
        for (int k = 0; k < CP / 16; ++k)
          tc_mma_ts(o, w + t * (CP / 2) + k * 8, tc_sdesc_mn(b + k * 16 * 128, CP * 128), kValues, j >= C::NS || t > 0 || k > 0);
      tc_commit(sm.pv_done(x));
      if (!ord.both || x == 1) tc_commit(sm.op_empty(at % C::kOps));
      if (j + 2 < n) ok = scores(j + 2);
    }
    at0 += 2 * ord.n;
    step0 += n;
    ++seg;
  }
  // every multiply has completed before tensor memory is freed
  tc_commit(sm.drain());
  if (!mbar_wait(sm.drain(), 0)) ok = false;
  return ok;
}

// ------------------------------------------------------------------ softmax
// A warpgroup's stream: thread r has query row r of the tile.
template <class C>
struct ShSoft {
  static constexpr int CP = C::CP, D = C::D;
  const SharedParams& p;
  const ShSmem<C>& sm;
  const int x, r;           // stream, row of the tile
  const uint32_t lane_off;  // the warp's lanes of tensor memory
  const uint32_t tmem;
  float ref, l, fac;
  uint32_t steps[2] = {0, 0};  // steps of each score place so far

  __device__ __forceinline__ ShSoft(const SharedParams& p_, const ShSmem<C>& sm_, uint32_t tm)
      : p(p_), sm(sm_), x(threadIdx.x >> 7), r(threadIdx.x & 127), lane_off((uint32_t)(threadIdx.x & 96) << 16), tmem(tm) {}

  // The row's queries, as an operand of 64-column halves with 128-byte swizzled rows.
  __device__ __forceinline__ void queries(const ShSegment& s, int tile, int G) {
    const int f = tile * kSharedTile + r;
    const bool there = f < s.g.R;
    const bf16* row = there ? p.a.q + (int64_t)(s.g.row0 + f / G) * p.a.q_stride + (s.kvh * G + f % G) * D : p.a.q;
    const uint32_t dst = smem_u32(sm.q(x)) + r * 128;
    const uint32_t zero = 0u;
    float down = 1.0f;
    fac = p.a.scale_log2;
    uint32_t flip = 0u;
    if (C::kBf16) {  // (a positive factor, so that the largest score is the largest product)
      if (fac < 0.0f) flip = 0x80008000u;
      fac = fmaxf(fabsf(fac), 0x1p-126f);  // (and not zero: a score of -infinity stays one)
    } else {
      uint32_t m = 0;
#pragma unroll 4
      for (int u = 0; u < D / 8; ++u) {
        const uint4 w = there ? __ldg(reinterpret_cast<const uint4*>(row) + u) : make_uint4(zero, zero, zero, zero);
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
      }
      m = max(m & 0xffffu, m >> 16);
      // the row's largest exponent E: q / 2^(E - 127) is below 2 (an infinity or NaN makes the row NaN)
      const int E = min(max((int)(m >> 7), 1), 253);
      down = __uint_as_float((uint32_t)(254 - E) << 23);
      fac = m >= 0x7f80u ? __uint_as_float(0x7fffffffu) : __fmul_rn(fac, __uint_as_float((uint32_t)E << 23));
    }
#pragma unroll 4
    for (int u = 0; u < D / 8; ++u) {
      uint4 w = there ? __ldg(reinterpret_cast<const uint4*>(row) + u) : make_uint4(zero, zero, zero, zero);
      if (C::kBf16) {
        w.x ^= flip; w.y ^= flip; w.z ^= flip; w.w ^= flip;
      } else {
        auto two = [&](uint32_t v) {
          return sh_f16x2(__fmul_rn(__uint_as_float(v << 16), down), __fmul_rn(__uint_as_float(v & 0xffff0000u), down));
        };
        w = make_uint4(two(w.x), two(w.y), two(w.z), two(w.w));
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (u >> 3) * kSharedTile * 128 + (((u & 7) ^ (r & 7)) << 4)),
                   "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                   : "memory");
    }
    fence_proxy_async_smem();
    mbar_arrive(sm.q_full(x));
    ref = kShNone;
    l = 0.0f;
  }

  // Step j of the segment, on score place y: scores to weights.  no: the chunk's number in the call.
  __device__ __forceinline__ bool step(int j, int y, uint32_t no, bool both) {
    if (!mbar_wait(sm.s_full(y), steps[y] & 1u)) return false;
    tc_fence_after();
    const uint32_t place = tmem + lane_off + y * C::kScoreCol;
    uint32_t w[CP / 32][32];
#pragma unroll
    for (int c = 0; c < CP / 32; ++c) tc_ld32(place + 32 * c, w[c]);
    tc_wait_ld();
    auto at = [&](int c) -> uint32_t& { return w[c / 32][c % 32]; };
    const int there = sm.mask()[no & 7];
    const float* sc = sm.scale(no % C::kRings);
    // scores in log2 units (a bf16 cache: before the factor), with the value's exponent
    float top = -INFINITY;
    if constexpr (!C::kBf16) {
#pragma unroll
      for (int c = 0; c < CP; c += 4) {
        const float4 ks = *reinterpret_cast<const float4*>(sc + c), ev = *reinterpret_cast<const float4*>(sc + CP + c);
        at(c) = __float_as_uint(__fmaf_rn(__fmul_rn(__uint_as_float(at(c)), fac), ks.x, ev.x));
        at(c + 1) = __float_as_uint(__fmaf_rn(__fmul_rn(__uint_as_float(at(c + 1)), fac), ks.y, ev.y));
        at(c + 2) = __float_as_uint(__fmaf_rn(__fmul_rn(__uint_as_float(at(c + 2)), fac), ks.z, ev.z));
        at(c + 3) = __float_as_uint(__fmaf_rn(__fmul_rn(__uint_as_float(at(c + 3)), fac), ks.w, ev.w));
      }
    }
    if (there != (1 << C::kPages) - 1) {  // pages that are not there
#pragma unroll
      for (int c = 0; c < CP; ++c)
        if (!((there >> (c / kPage)) & 1)) at(c) = 0xff800000u;
    }
#pragma unroll
    for (int c = 0; c < CP; ++c) top = fmaxf(top, __uint_as_float(at(c)));
    if (C::kBf16) top = __fmul_rn(top, fac);
    if (__any_sync(0xffffffffu, top > __fadd_rn(ref, kShSlack))) {
      const bool up = top > __fadd_rn(ref, kShSlack);
      const float d = up ? __fsub_rn(ref, top) : 0.0f, a = sh_ex2(d);
      const bool scaled = up && ref != kShNone;
      l = sh_times_ex2(l, d);
      ref = up ? top : ref;
      if (__any_sync(0xffffffffu, scaled)) {
        // (the product before this step: with two streams it ran before these scores did)
        if (C::NS == 1 && j > 0 && !mbar_wait(sm.pv_done(y ^ 1), (steps[y ^ 1] - 1u) & 1u)) return false;
        tc_fence_after();
        const uint32_t o = tmem + lane_off + C::kOutCol + (C::NS == 2 ? x : 0) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          tc_ld32(o + c, v);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__fmul_rn(__uint_as_float(v[e]), a));
          tc_st32(o + c, v);
        }
        tc_wait_st();
      }
    }
    // weights and their sum
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (C::kBf16) {
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        const float e = sh_ex2(__fmaf_rn(__uint_as_float(at(c)), fac, -ref));
        sum[c & 3] = __fadd_rn(sum[c & 3], e);
        at(c) = __float_as_uint(e);
      }
#pragma unroll
      for (int c = 0; c < CP; c += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t a = at(c + 2 * e), b = at(c + 2 * e + 1);
          // the first term: the value's upper half; the second: the rest, rounded
          hi[e] = __byte_perm(a, b, 0x7632);
          lo[e] = pack_bf16x2(__fsub_rn(__uint_as_float(a), __uint_as_float(a & 0xffff0000u)),
                              __fsub_rn(__uint_as_float(b), __uint_as_float(b & 0xffff0000u)));
        }
        tc_st16(place + c / 2, hi);
        tc_st16(place + CP / 2 + c / 2, lo);
      }
    } else {
      float low = 0.0f;
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        const float z = __fsub_rn(__uint_as_float(at(c)), ref);
        at(c) = __float_as_uint(z);
        low = fminf(low, z);
      }
      const bool far = __any_sync(0xffffffffu, low < kShFar);
#pragma unroll
      for (int c = 0; c < CP; c += 4) {
        const float4 iv = *reinterpret_cast<const float4*>(sc + 2 * CP + c);
        const float f[4] = {iv.x, iv.y, iv.z, iv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float z = __uint_as_float(at(c + e)), v = sh_ex2(z);
          at(c + e) = __float_as_uint(v);
          if (far && z < kShFar) {  // p' is below fp32's range, p need not be
            const float ev = sc[CP + c + e];
            if (z != -INFINITY) sum[e] = __fadd_rn(sum[e], sh_ex2(__fsub_rn(z, ev)));
          } else {
            sum[e] = __fmaf_rn(v, f[e], sum[e]);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < CP; c += 64) {
        uint32_t h[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) h[e] = sh_f16x2(__uint_as_float(at(c + 2 * e)), __uint_as_float(at(c + 2 * e + 1)));
        tc_st32(place + c / 2, h);
      }
    }
    l = __fadd_rn(l, __fadd_rn(__fadd_rn(sum[0], sum[1]), __fadd_rn(sum[2], sum[3])));
    tc_wait_st();
    tc_fence_before();
    mbar_arrive(sm.p_full(y));
    __syncwarp();
    if (!C::kBf16 && (threadIdx.x & 31) == 0) {
      mbar_arrive(sm.sc_empty(no % C::kRings));
      if (C::NS == 2 && !both) mbar_arrive(sm.sc_empty(no % C::kRings));  // (a chunk that one stream alone has)
    }
    ++steps[y];
    return true;
  }

  // The segment's partial.  n: steps of this stream; y: the last one's score place.
  __device__ __forceinline__ bool partial(const ShSegment& s, int tile, int n, int y, int cta) {
    const int f = tile * kSharedTile + r;
    const long long at = (long long)x * p.plane + sh_slot(p, s.g, s.kvh, s.pair, C::NS, cta) + r;
    if (n > 0) {
      if (!mbar_wait(sm.pv_done(y), (steps[y] - 1u) & 1u)) return false;
      tc_fence_after();
      const uint32_t o = tmem + lane_off + C::kOutCol + (C::NS == 2 ? x : 0) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        tc_ld32(o + c, v);
        tc_wait_ld();
        if (f < s.g.R) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + at * D + c);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
      tc_fence_before();
    }
    if (f < s.g.R) p.ml[at] = make_float2(ref, l);
    return true;
  }

  __device__ bool run() {
    const int G = p.a.n_q_heads / p.a.n_kv_heads;
    ShRun<C::NS> run(p, blockIdx.x);
    ShSegment s;
    uint32_t chunk_no = 0;
    while (run.next(s)) {
      const ShOrder ord{s.i1 - s.i0, s.w == 2};
      const int n = ord.steps(), tile = s.pair * C::NS + (ord.both ? x : 0);
      if (C::NS == 1 || x < n) queries(s, tile, G);
      else { ref = kShNone; l = 0.0f; mbar_arrive(sm.q_full(x)); }
      int mine = 0, y = 0;
      for (int j = C::NS == 2 ? x : 0; j < n; j += C::NS) {
        y = j & 1;
        if (!step(j, y, chunk_no + ord.chunk(j), ord.both)) return false;
        ++mine;
      }
      if (!partial(s, tile, mine, y, blockIdx.x)) return false;
      chunk_no += ord.n;
    }
    return true;
  }
};

template <int D, int FMT>
__global__ void __launch_bounds__(ShCfg<D, FMT>::kThreads, 1)
    k_shared_prefix(const __grid_constant__ SharedParams p, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap) {
  using C = ShCfg<D, FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const ShSmem<C> sm(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kOps; ++i) {
      mbar_init(sm.op_full(i), C::kBf16 ? 1 : 128);
      mbar_init(sm.op_empty(i), 1);
    }
    for (int i = 0; i < C::kRaws; ++i) {
      mbar_init(sm.raw_full(i), 1);
      mbar_init(sm.raw_empty(i), 128);
    }
    for (int i = 0; i < C::kRings; ++i) mbar_init(sm.sc_empty(i), C::NS == 2 ? 8 : 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(sm.s_full(i), 1);
      mbar_init(sm.p_full(i), 128);
      mbar_init(sm.pv_done(i), 1);
      mbar_init(sm.q_full(i), 128);
    }
    mbar_init(sm.drain(), 1);
    fence_barrier_init();
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
  bool ok = true;
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoft));
    if (C::NS == 2 || warp < 4) ok = ShSoft<C>(p, sm, tmem).run();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == 8) {
      if (lane == 0) ok = sh_multiply<C>(p, sm, tmem);
    } else if (warp == 9) {
      ok = sh_load<C>(p, &kmap, &vmap, sm);
    } else if (warp >= 12) {
      if constexpr (!C::kBf16) ok = sh_widen<C>(p, sm);
    }
  }
  if (!ok && p.a.status) atomicOr(p.a.status, ST_TIMEOUT);
  tc_fence_before();
  __syncthreads();
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
// row's own positions, added up in that order.  A warp for each result.
template <int D, bool kBf16>
__global__ void __launch_bounds__(256) k_shared_merge(const __grid_constant__ SharedParams p) {
  constexpr int V = D / 32, NS = shared_streams(D), CP = shared_chunk(D), B = 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x * 8 + warp;
  const int H = p.a.n_q_heads, r = p.a.row_lo + unit / H, hq = unit % H, G = H / p.a.n_kv_heads;
  int seq, i;
  const bool row = r < p.a.row_hi && find_row(p.a.rows, r, seq, i);
  pdl_trigger();
  pdl_wait();
  if (!row) return;
  const int t = first_of(p.a.rows, seq) + i, from = __ldcg(p.from + seq), gi = __ldcg(p.group + seq), kvh = hq / G;
  // the prefix: CTAs c0 .. c1 - 1, one or two partials each
  int c0 = 0, c1 = 0, planes = 1, plane = 0;
  long long slot = 0;
  if (t >= 0 && from > 0 && gi >= 0) {
    const SharedGroup g = sh_group(p.plan, gi), end = sh_group(p.plan, p.n_groups);
    const int f = (r - g.row0) * G + hq % G, pair = f / (NS * kSharedTile), w = min(NS, g.tiles - pair * NS);
    const long long first = g.unit0 + (long long)kvh * g.chunks * g.tiles + (long long)pair * NS * g.chunks;
    c0 = sh_owner(first, end.unit0, end.eff);
    c1 = sh_owner(first + (long long)(g.chunks - 1) * w, end.unit0, end.eff) + 1;
    planes = w == 2 ? 1 : NS;
    plane = w == 2 ? f / kSharedTile & 1 : 0;
    slot = sh_slot(p, g, kvh, pair, NS, 0) + f % kSharedTile;
  }
  const int n1 = (c1 - c0) * planes;
  // its own positions: the splits from `from` on
  const int last = min(t, p.a.rows.limit() - 1);
  const int s0 = last >= from ? attend_split_of(from) : 0, n2 = last >= from ? attend_split_of(last) - s0 + 1 : 0, n = n1 + n2;
  const size_t own = (size_t)unit * p.a.max_splits + s0;
  auto place = [&](int j) {  // of partial j < n1
    return (long long)(planes == 2 ? j & 1 : plane) * p.plane + slot + (long long)(c0 + (planes == 2 ? j >> 1 : j)) * kSharedTile;
  };
  auto ml_of = [&](int j) { return j < n1 ? __ldcg(p.ml + place(j)) : __ldcg(p.a.part_ml + own + (j - n1)); };
  float M = kShNone;
  for (int j = lane; j < n; j += 32) M = fmaxf(M, ml_of(j).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float l = 0.0f, acc[V], bad = 0.0f, small[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = small[e] = 0.0f;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const float2 ml = j0 + lane < n ? ml_of(j0 + lane) : make_float2(kShNone, 0.0f);
    // (a partial that has seen nothing has no accumulators; one of NaN scores has a NaN sum)
    const bool saw = !(ml.y == 0.0f);
    const float d = __fsub_rn(ml.x, M), f = saw ? sh_ex2(d) : 0.0f;
    float part = saw ? sh_times_ex2(ml.y, d) : 0.0f;
    const uint32_t some = __ballot_sync(0xffffffffu, saw);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part = __fadd_rn(part, __shfl_xor_sync(0xffffffffu, part, o));
    l = __fadd_rn(l, part);
    for (int k0 = 0; k0 < min(32, n - j0); k0 += B) {
      float x[B][V];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int j = j0 + k0 + b;
        const bool have = (some >> (k0 + b)) & 1u;  // (bits behind the last partial are clear)
        const float* src = !have ? nullptr : j < n1 ? p.o + place(j) * D : p.a.part_o + (own + (j - n1)) * D;
#pragma unroll
        for (int e = 0; e < V; ++e) x[b][e] = 0.0f;
        if (have) {
          if constexpr (V == 2) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(src + lane * V));
            x[b][0] = v.x; x[b][1] = v.y;
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 4) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(src + lane * V + e));
              x[b][e] = v.x; x[b][e + 1] = v.y; x[b][e + 2] = v.z; x[b][e + 3] = v.w;
            }
          }
        }
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const float fb = __shfl_sync(0xffffffffu, f, k0 + b);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          acc[e] = __fmaf_rn(x[b][e], fb, acc[e]);
          if (kBf16) {
            small[e] = __fmaf_rn(x[b][e], __fmul_rn(fb, 0x1p-24f), small[e]);
            bad = __fmaf_rn(x[b][e], 0.0f, bad);
          }
        }
      }
    }
  }
  const bool none = l == 0.0f;
  bf16* out = p.a.out + (int64_t)r * p.a.out_stride + hq * D + lane * V;
  float y[V];
#pragma unroll
  for (int e = 0; e < V; ++e) y[e] = none ? 0.0f : __fdiv_rn(acc[e], l);
  if (kBf16 && l == l && !none) {
    const int* table = p.a.rows.table + (size_t)seq * p.a.rows.table_stride;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (!(fabsf(acc[e]) < INFINITY))
        y[e] = sh_far_value<D>(p, table, t, kvh, lane * V + e, bad == 0.0f, __fdiv_rn(small[e], __fmul_rn(l, 0x1p-24f)));
  }
#pragma unroll
  for (int e = 0; e < V; e += 2) *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(y[e], y[e + 1]);
  if (p.a.lse && lane == 0)
    p.a.lse[(size_t)r * H + hq] = none ? -INFINITY : __fmul_rn(__fadd_rn(M, log2f(l)), 0.6931471805599453f);
}

template <int D, int FMT>
cudaError_t shared_prepare() {
  using C = ShCfg<D, FMT>;
  cudaError_t e = cudaFuncSetAttribute(k_shared_prefix<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // The warpgroups' registers come out of what the launch got: with fewer the kernel would wait for ever.
  cudaFuncAttributes at;
  if ((e = cudaFuncGetAttributes(&at, k_shared_prefix<D, FMT>)) != cudaSuccess) return e;
  return at.numRegs >= C::kRegs ? cudaSuccess : cudaErrorInvalidConfiguration;
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

template <int D>
cudaError_t shared_merge_launch(const SharedParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int64_t units = (int64_t)(p.a.row_hi - p.a.row_lo) * p.a.n_q_heads;
  cfg.gridDim = dim3((unsigned)((units + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.a.k_exp ? cudaLaunchKernelEx(&cfg, k_shared_merge<D, false>, p) : cudaLaunchKernelEx(&cfg, k_shared_merge<D, true>, p);
}

}  // namespace
}  // namespace sv
