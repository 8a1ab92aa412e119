// k_logprobs.cu -- log probabilities of given tokens, entropies and the most
// probable tokens of rows of logits.
//
// With y = scale log2(e) x for a row's logits x, one pass keeps, against a
// reference m that follows the largest y seen,
//   l = sum 2^(y - m),  t = sum 2^(y - m) (y - m),
// so that log2 sum 2^y = m + log2 l, log2 p = y - m - log2 l and the entropy is
// ln2 (log2 l - t / l): nothing of the row is read twice for them.  All in fp32;
// a warp shares its reference (it moves seldom, and alike for all lanes), and
// lanes, warps and CTAs are added up in a fixed order.
//
// The k most probable tokens come from the same pass: it leaves the largest
// logit of each of at most 512 chunks (128 of a short row) (consecutive ids) in shared
// memory.  The k-th largest of those is a bound that every one of the k reaches;
// at most k chunks have to be read again (from L2), those above the bound and,
// of those equal to it, the first: k tokens of theirs are at least as probable
// as any of a later one, with lower ids.
//
// What bounds it: for many rows memory, and instructions nearly as much (of bf16: widen,
// maximum, scale and subtract, exponential, two sums; 2048 x 151936, 622 MB, in 109 us,
// 0.84 of the copy rate; 1000 x 151936 with 5 alternatives, 304 MB, 78 us, of which a
// third is the second look, when an SM has few loads on their way); for a few rows the
// chain of load, meeting and second look (1 x 151936 fp32 with 20 alternatives 10.3 us in
// a graph, 5.8 without any; 24 x 262144 bf16 with 5 12.0).  A row of fewer chunks than
// alternatives has all its logits put in order, one by one: 2000 x 1024 bf16 9.8 us with
// one alternative, 78 with 5.  A row is a cluster of 1 to 8 CTAs, so that few rows fill
// the device too; they meet over distributed shared memory.
// (Two CTAs a row where there are rows for every SM: 500 x 151936 fp32 with 20 91 us, when
// one took 75.  Sums of pairs in one instruction, fma.f32x2: 148 us for the first case,
// when the form without took 129.)
#include "sv_internal.h"
#include "sv_ptx.cuh"

#include <algorithm>
#include <cfloat>
#include <cooperative_groups.h>

#include "logprobs.h"

namespace sv {
namespace {

namespace cg = cooperative_groups;

// Threads of a CTA: 128 for short rows, of which an SM then holds more.
constexpr int kLpWide = 512, kLpNarrow = 128;
constexpr int kLpMost = kLogprobsMaxTop;
constexpr float kLpFar = 536870912.0f;  // 2^29: half a step of a reference below it is at most 16
// Reference of what has seen nothing: logits below it (masks of -1e30 or the type's lowest
// value) weigh nothing, where a reference of their own would be off by more than 2^127.
constexpr float kLpNone = -kLpFar;
constexpr float kLpSlack = 4.0f;    // log2 of what a weight may be before the reference follows
static_assert(kLpMost == 32, "a lane holds one of a warp's best");

__device__ __forceinline__ float lp_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The larger of both, a NaN if there is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// fp32 values in the order of unsigned words; -0 and 0 are the same.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
constexpr uint32_t kOrderNegInf = 0x007fffffu;  // of -infinity

template <class T>
struct LpVec;
template <>
struct LpVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void open(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return __ldcg(p); }
  static __device__ __forceinline__ uint4 finite(const uint4& w) { return w; }
  static __device__ __forceinline__ float largest(const uint4& w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
  // word i of the 16 bytes from element v, where only lo .. hi - 1 are there
  static __device__ __forceinline__ uint32_t part(const float* p, int v, int i, int lo, int hi) {
    return v + i >= lo && v + i < hi ? __float_as_uint(__ldcg(p + v + i)) : 0xff800000u;
  }
};
template <>
struct LpVec<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void open(const uint4& w, float (&x)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float one(const bf16* p) { return __uint_as_float((uint32_t)__ldcg(reinterpret_cast<const unsigned short*>(p)) << 16); }
  // The same with finite values, of -1e30, for infinities (an impossible token's 0 * inf is zero
  // then); a NaN stays one.
  static __device__ __forceinline__ uint4 finite(const uint4& w) {
    uint4 r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r.x) : "r"(w.x), "r"(0xf14af14au));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r.y) : "r"(w.y), "r"(0xf14af14au));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r.z) : "r"(w.z), "r"(0xf14af14au));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r.w) : "r"(w.w), "r"(0xf14af14au));
    return r;
  }
  static __device__ __forceinline__ float largest(const uint4& w) {
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t part(const bf16* p, int v, int i, int lo, int hi) {
    uint32_t w = 0;
    for (int e = 0; e < 2; ++e) {
      const int at = v + 2 * i + e;
      w |= (at >= lo && at < hi ? (uint32_t)__ldcg(reinterpret_cast<const unsigned short*>(p + at)) : 0xff80u) << (16 * e);
    }
    return w;
  }
};

// A row in blocks of 32 N elements from the 16-byte boundary at or before its
// first one: element v of that count is token v - lead.
template <class T, int TH>
struct LpRow {
  static constexpr int N = LpVec<T>::N, kBlock = 32 * N;
  const T* base;
  int lead, vocab, blocks, shift, chunks;  // 2^shift: blocks of a chunk; a thread looks at one chunk
  __device__ __forceinline__ LpRow(const T* row, int vocab_) : vocab(vocab_) {
    lead = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    base = row - lead;
    blocks = (int)(((int64_t)lead + vocab + kBlock - 1) / kBlock);
    shift = 0;
    while (blocks > TH << shift) ++shift;
    chunks = (blocks + (1 << shift) - 1) >> shift;
  }
  // This lane's 16 bytes of block b, which lies within the row.  (Element numbers are at
  // most vocab + 8 and a block: below 2^31.)
  __device__ __forceinline__ uint4 load(int b, int lane) const {
    return __ldcg(reinterpret_cast<const uint4*>(base + b * kBlock + lane * N));
  }
  // Of one that may not: -infinity outside the row, of which no byte is read.
  __device__ __forceinline__ uint4 edge(int b, int lane) const {
    const int v = b * kBlock + lane * N;
    if (v >= lead && v + N <= lead + vocab) return load(b, lane);
    auto part = [&](int i) { return LpVec<T>::part(base, v, i, lead, lead + vocab); };
    return make_uint4(part(0), part(1), part(2), part(3));
  }
};

// A warp's best tokens, sorted: lane i has the i-th (id -1: none).
struct LpBest {
  uint32_t key;
  int id;
  __device__ __forceinline__ static bool better(uint32_t k, int i, uint32_t k2, int i2) {
    return k > k2 || (k == k2 && (uint32_t)i < (uint32_t)i2);
  }
  __device__ __forceinline__ void add(uint32_t k, int i, int lane) {
    const int at = __popc(__ballot_sync(0xffffffffu, better(key, id, k, i)));
    const uint32_t uk = __shfl_up_sync(0xffffffffu, key, 1);
    const int ui = __shfl_up_sync(0xffffffffu, id, 1);
    if (lane == at) { key = k; id = i; }
    if (lane > at) { key = uk; id = ui; }
  }
};

template <int TH>
struct LpShared {
  static constexpr int kWarps = TH / 32;
  float m[kWarps], l[kWarps], t[kWarps];
  float cta[3];                  // the CTA's (m, l, t)
  uint32_t chunk[TH];            // largest logit of each of this CTA's chunks
  int chosen[kLpMost], n_chosen;
  uint32_t key[TH];              // candidates
  int id[TH];
  int warp_n[kWarps];
  uint2 best[kLpMost];           // the CTA's best: order and id (-1: none)
};

// The best `most` of the threads' candidates (have: this thread has one), in order, into s.best.
template <int TH>
__device__ __forceinline__ void lp_rank(LpShared<TH>& s, bool have, uint32_t key, int id, int most) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t mask = __ballot_sync(0xffffffffu, have);
  if (lane == 0) s.warp_n[warp] = __popc(mask);
  if (tid < kLpMost) s.best[tid] = make_uint2(0u, 0xffffffffu);
  __syncthreads();
  int before = 0, n = 0;
#pragma unroll
  for (int w = 0; w < TH / 32; ++w) {
    before += w < warp ? s.warp_n[w] : 0;
    n += s.warp_n[w];
  }
  if (have) {
    const int at = before + __popc(mask & ((1u << lane) - 1u));
    s.key[at] = key;
    s.id[at] = id;
  }
  __syncthreads();
  if (tid < n) {
    key = s.key[tid];
    id = s.id[tid];
    int rank = 0;
    for (int i = 0; i < n; ++i) rank += LpBest::better(s.key[i], s.id[i], key, id);
    if (rank < most) s.best[rank] = make_uint2(key, (uint32_t)id);
  }
  __syncthreads();
}

// (x - X) c, where x - X may be beyond fp32's range though the product is not (x of 3e38
// and -3e38 with c = 1/4).
__device__ __forceinline__ float lp_below(float x, float X, float c) {
  const float d = __fsub_rn(x, X);
  if (d > -INFINITY) return __fmul_rn(d, c);
  const float h = __fmul_rn(__fsub_rn(__fmul_rn(0.5f, x), __fmul_rn(0.5f, X)), c);
  return __fadd_rn(h, h);
}

// A row whose largest y = x c is beyond kLpFar: a reference rounded to fp32 would lie too
// far from it for 2^(y - m), and c x may be beyond fp32's range (rows masked with -1e30 or
// the type's lowest value throughout); or a row of a call that sums plainly (lp_plain).
// Its largest logit X (-infinity: none is finite) and the sums of z = (x - X) c.  Each CTA
// reads the whole row, plainly: such rows are rare.
template <class T, int TH>
__device__ __noinline__ void lp_far_row(LpShared<TH>& s, const T* logits, int vocab, float c, float& X, float& L, float& E) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  X = -INFINITY;
#pragma unroll 1
  for (int i = tid; i < vocab; i += TH) X = fmaxf(X, LpVec<T>::one(logits + i));
  X = warp_max(X);
  __syncthreads();  // (the warps' numbers have been read)
  if (lane == 0) s.m[warp] = X;
  __syncthreads();
  for (int i = 0; i < TH / 32; ++i) X = fmaxf(X, s.m[i]);
  L = E = 0.0f;
#pragma unroll 1
  for (int i = tid; X > -INFINITY && i < vocab; i += TH) {
    const float z = lp_below(LpVec<T>::one(logits + i), X, c), q = lp_ex2(z);
    L = __fadd_rn(L, q);
    E = __fmaf_rn(q, fmaxf(z, -1000.0f), E);  // (an impossible token's 0 * inf is zero)
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    L = __fadd_rn(L, __shfl_xor_sync(0xffffffffu, L, o));
    E = __fadd_rn(E, __shfl_xor_sync(0xffffffffu, E, o));
  }
  if (lane == 0) {
    s.l[warp] = L;
    s.t[warp] = E;
  }
  __syncthreads();
  L = E = 0.0f;
  for (int i = 0; i < TH / 32; ++i) {
    L = __fadd_rn(L, s.l[i]);
    E = __fadd_rn(E, s.t[i]);
  }
}

template <class T, int TH, bool kTop, bool kEntropy>
__global__ void __launch_bounds__(TH) k_logprobs(const LogprobsParams p) {
  using V = LpVec<T>;
  // (bf16 blocks by twos, with one check of the reference: 2048 x 151936 109 us, one by one
  // 127; of fp32 500 x 151936 with 20 alternatives would take 80, one by one 73)
  constexpr int N = V::N, kAhead = 4, kAtOnce = N == 8 ? 2 : 1;
  constexpr int kLpThreads = TH, kLpWarps = TH / 32;
  using Row = LpRow<T, TH>;
  __shared__ LpShared<TH> s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / CS;
  pdl_trigger();
  pdl_wait();  // (what the kernels ahead wrote is read past L1, which this one may have shared with them)
  const T* logits = static_cast<const T*>(p.logits) + (int64_t)r * p.stride;
  const Row row(logits, p.vocab);
  const float c = p.scale_log2;
  const int c0 = (int)((int64_t)rank * row.chunks / CS), c1 = (int)((int64_t)(rank + 1) * row.chunks / CS);
  const int b0 = c0 << row.shift, b1 = min(c1 << row.shift, row.blocks);
  if (kTop) {
    s.chunk[tid] = 0;
    __syncthreads();
  }
  float m = kLpNone, l = 0.0f, t = 0.0f;
  // A lane's 16 bytes of block b, and of another one (of rows without alternatives).
  auto add = [&](const uint4& w, int b, const auto&... other) {
    constexpr int NV = 1 + sizeof...(other);
    float x[NV][N];
    V::open(kEntropy ? V::finite(w) : w, x[0]);  // (of bf16 values all finite, four instructions for eight)
    const float one = V::largest(w);
    float top = one, next = 0.0f;
    if constexpr (NV == 2) {
      V::open(kEntropy ? V::finite(other...) : (other, ...), x[1]);
      next = V::largest(other...);
      top = fmaxf(top, next);
    }
    // (the reference follows when it falls behind by 2^4)
    const bool far = __fmaf_rn(top, c, -m) > kLpSlack;
    float chunk = 0.0f;  // (used at the end: nothing here waits for it)
    if (kTop) {
      chunk = warp_max(one);
      if (NV == 2) next = warp_max(next);
    }
    if (__any_sync(0xffffffffu, far)) {
      const float y = __fmul_rn(kTop ? NV == 2 ? fmaxf(chunk, next) : chunk : warp_max(top), c);
      if (__fsub_rn(y, m) > kLpSlack) {
        const float d = __fsub_rn(m, y), f = lp_ex2(d);
        t = f > 0.0f ? __fmul_rn(f, __fmaf_rn(d, l, t)) : 0.0f;
        l = __fmul_rn(f, l);
        m = y;
      }
    }
    const float before = t;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float z = __fmaf_rn(x[v][e], c, -m), q = lp_ex2(z);
        l = __fadd_rn(l, q);
        if (kEntropy) t = __fmaf_rn(q, z, t);
        x[v][e] = z;
      }
    if (kEntropy && N == 4 && t != t) {  // an impossible token's 0 * inf is zero (a NaN among the logits has made l one)
      t = before;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float z = fmaxf(x[v][e], -1000.0f);
          t = __fmaf_rn(lp_ex2(z), z, t);
        }
    }
    if (kTop && lane == 0) {
      atomicMax(&s.chunk[b >> row.shift], order_of(chunk));
      if (NV == 2) atomicMax(&s.chunk[(b + kLpWarps) >> row.shift], order_of(next));
    }
  };
  // Blocks that lie within the row, each warp's next three on their way while one is
  // worked on; the row's ends by themselves.
  const int whole0 = max(b0, row.lead > 0 ? 1 : 0), whole1 = min(b1, (row.lead + row.vocab) / Row::kBlock);
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const int b = i ? row.blocks - 1 : 0;
    if (warp == i && b >= b0 && b < b1 && (b < whole0 || b >= whole1) && !(i && b == 0)) add(row.edge(b, lane), b);
  }
  uint4 w[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (whole0 + warp + i * kLpWarps < whole1) w[i] = row.load(whole0 + warp + i * kLpWarps, lane);
  }
#pragma unroll 1
  for (int b = whole0 + warp; b < whole1; b += kAhead * kLpWarps) {
#pragma unroll
    for (int i = 0; i < kAhead; i += kAtOnce) {
      const int bi = b + i * kLpWarps;
      if (bi >= whole1) break;
      const uint4 now = w[i];
      if constexpr (kAtOnce == 2) {
        const uint4 then = w[i + 1];
        if (bi + kLpWarps >= whole1) {  // a last one alone
          add(now, bi);
          break;
        }
        if (bi + kAhead * kLpWarps < whole1) w[i] = row.load(bi + kAhead * kLpWarps, lane);
        if (bi + (kAhead + 1) * kLpWarps < whole1) w[i + 1] = row.load(bi + (kAhead + 1) * kLpWarps, lane);
        add(now, bi, then);
      } else {
        if (bi + kAhead * kLpWarps < whole1) w[i] = row.load(bi + kAhead * kLpWarps, lane);
        add(now, bi);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    l = __fadd_rn(l, __shfl_xor_sync(0xffffffffu, l, o));
    t = __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, o));
  }
  if (lane == 0) {
    s.m[warp] = m;
    s.l[warp] = l;
    s.t[warp] = t;
  }
  __syncthreads();
  // (m, l, t) of n parts, in order
  auto meet = [&](int n, auto part, float& M, float& L, float& E) {
    M = kLpNone;
    for (int i = 0; i < n; ++i) M = fmaxf(M, part(i, 0));
    L = E = 0.0f;
    for (int i = 0; i < n; ++i) {
      const float li = part(i, 1), d = __fsub_rn(part(i, 0), M), f = lp_ex2(d);
      L = __fmaf_rn(f, li, L);
      if (!(f == 0.0f)) E = __fmaf_rn(f, __fmaf_rn(d, li, part(i, 2)), E);
    }
  };
  float M, L, E;
  meet(kLpWarps, [&](int i, int k) { return k == 0 ? s.m[i] : k == 1 ? s.l[i] : s.t[i]; }, M, L, E);
  if (CS > 1) {
    if (tid == 0) {
      s.cta[0] = M;
      s.cta[1] = L;
      s.cta[2] = E;
    }
    cluster.sync();
    float all[3] = {kLpNone, 0.0f, 0.0f};  // lane i: CTA i's
    if (lane < CS) {
      const float* other = cluster.map_shared_rank(s.cta, lane);
#pragma unroll
      for (int k = 0; k < 3; ++k) all[k] = other[k];
    }
    meet(CS, [&](int i, int k) { return __shfl_sync(0xffffffffu, all[k], i); }, M, L, E);
  }
  float X = 0.0f;
  const bool is_far = !(fabsf(M) < (N == 8 ? p.far : kLpFar));  // (the same for all CTAs of the row)
  if (is_far) {
    lp_far_row<T, TH>(s, logits, p.vocab, c, X, L, E);
    M = X;
  }
  // A row with a NaN or an infinity, or of nothing but -infinity, has no distribution.
  const float NaN = __uint_as_float(0x7fffffffu), ln2 = 0.6931471805599453f;
  const bool good = L > 0.0f && L < INFINITY && fabsf(M) < INFINITY;
  const float l2 = good ? log2f(L) : NaN;
  auto log_prob = [&](float x) {
    const float z = is_far ? lp_below(x, X, c) : __fmaf_rn(x, c, -M), v = __fmul_rn(__fsub_rn(z, l2), ln2);
    // (a finite logit's is finite: where z is beyond fp32's range l2 is nothing beside it, nor is a
    // row's M that is not far)
    return v == -INFINITY && x > -INFINITY ? fmaxf(lp_below(x, is_far ? X : 0.0f, __fmul_rn(c, ln2)), -FLT_MAX) : v;
  };
  if (rank == 0) {
    for (int i = tid; i < p.n_tokens; i += kLpThreads) {
      const int tok = __ldcg(p.tokens + (int64_t)r * p.n_tokens + i);
      float v = 0.0f;  // a token of -1: an unused place
      if (tok >= 0 && tok < p.vocab) v = log_prob(V::one(logits + tok));
      else if (tok != -1) {
        v = NaN;
        if (p.status) atomicOr(p.status, ST_BAD_TOKEN);
      }
      p.out[(int64_t)r * p.n_tokens + i] = v;
    }
    if (tid == 0) {
      if (p.lse) {
        const float far_lse = fminf(fmaxf(__fmaf_rn(X, __fmul_rn(c, ln2), __fmul_rn(l2, ln2)), -FLT_MAX), FLT_MAX);
        p.lse[r] = is_far && good ? far_lse : __fmul_rn(__fadd_rn(M, l2), ln2);
      }
      if (p.entropy) p.entropy[r] = max_nan(__fmul_rn(__fsub_rn(l2, __fdiv_rn(E, L)), ln2), 0.0f);
    }
  }
  if (!kTop) {
    if (CS > 1) cluster.sync();  // the others read this CTA's numbers
    return;
  }
  // ---- the most probable tokens
  const int k = p.top;
  uint32_t key = 0;
  if (tid < row.chunks) {
    const int at = (int)((((int64_t)tid + 1) * CS - 1) / row.chunks);  // the CTA that has chunk tid
    key = CS > 1 ? cluster.map_shared_rank(s.chunk, at)[tid] : s.chunk[tid];
  }
  if (!good) key = 0;  // (no tokens to name)
  // The largest bound that k chunks reach, bit by bit (of bf16 values the upper 16 say all).
  constexpr int kLow = sizeof(T) == 2 ? 16 : 0;
  key >>= kLow;
  const uint32_t none = kOrderNegInf >> kLow;
  uint32_t bound = 0;
  bool exact = false;
#pragma unroll 1
  for (uint32_t bit = 0x80000000u >> kLow; bit && !exact; bit >>= 1) {
    const int n = __syncthreads_count(key >= (bound | bit));
    if (n >= k) {
      bound |= bit;
      exact = n == k;
    }
  }
  // Chunks above the bound, and the first of those equal to it (all that reach it, where they are k).
  bool take = key > none && key >= bound;
  if (!exact && bound > 0) {
    const int above = __syncthreads_count(key > bound);
    const uint32_t eq = __ballot_sync(0xffffffffu, key == bound);
    if (lane == 0) s.warp_n[warp] = __popc(eq);
    __syncthreads();
    int before = __popc(eq & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) before += s.warp_n[w];
    if (key == bound && before >= k - above) take = false;
  }
  bound <<= kLow;
  if (tid == 0) s.n_chosen = 0;
  __syncthreads();
  if (take && tid >= c0 && tid < c1) s.chosen[atomicAdd(&s.n_chosen, 1)] = tid;
  __syncthreads();
  LpBest best = {0u, -1};
  const int items = s.n_chosen << row.shift;
#pragma unroll 1
  for (int i = warp; i < items; i += kLpWarps) {
    const int b = (s.chosen[i >> row.shift] << row.shift) + (i & ((1 << row.shift) - 1));
    if (b >= row.blocks) continue;
    float x[N];
    V::open(row.edge(b, lane), x);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const uint32_t ke = order_of(x[e]);
      const int id = (int)((int64_t)b * Row::kBlock + lane * N + e - row.lead);
      uint32_t left = __ballot_sync(0xffffffffu, ke > kOrderNegInf && ke >= bound);
      while (left) {
        const int from = __ffs(left) - 1;
        left &= left - 1;
        best.add(__shfl_sync(0xffffffffu, ke, from), __shfl_sync(0xffffffffu, id, from), lane);
      }
    }
  }
  lp_rank(s, best.id >= 0, best.key, best.id, k);
  if (CS > 1) {
    cluster.sync();
    if (rank == 0) {  // thread (CTA i, place j) takes that one's j-th
      const int i = tid / kLpMost, j = tid % kLpMost;
      uint2 other = make_uint2(0u, 0xffffffffu);
      if (i < CS) other = cluster.map_shared_rank(s.best, i)[j];
      __syncthreads();  // this CTA's own are in registers now
      lp_rank(s, (int)other.y >= 0, other.x, (int)other.y, k);
    }
  }
  if (rank == 0 && tid < k) {
    const uint2 o = s.best[tid];
    const bool there = (int)o.y >= 0;
    const float x = __uint_as_float((o.x >> 31) ? o.x ^ 0x80000000u : ~o.x);
    if (p.top_values) p.top_values[(int64_t)r * k + tid] = !good ? NaN : there ? log_prob(x) : -INFINITY;
    if (p.top_ids) p.top_ids[(int64_t)r * k + tid] = (int)o.y;
  }
  if (CS > 1) cluster.sync();
}

constexpr int kLpAlone = 120 << 10;

template <class T, int TH, bool kTop, bool kEntropy>
cudaError_t prepare_t() {
  return cudaFuncSetAttribute(k_logprobs<T, TH, kTop, kEntropy>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpAlone);
}

template <class T, int TH>
cudaError_t prepare_e() {
  cudaError_t e;
  if ((e = prepare_t<T, TH, false, false>()) != cudaSuccess || (e = prepare_t<T, TH, false, true>()) != cudaSuccess ||
      (e = prepare_t<T, TH, true, false>()) != cudaSuccess)
    return e;
  return prepare_t<T, TH, true, true>();
}

template <class T, int TH, bool kTop, bool kEntropy>
cudaError_t launch_t(const LogprobsParams& p, int n_rows, int cs, int num_sms, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)n_rows * cs);
  cfg.blockDim = dim3(TH);
  cfg.stream = s;
  // Few CTAs: an SM for each, by asking for more than half of its shared memory (a
  // cluster's CTAs would share SMs: 24 x 262144 bf16 with 5 alternatives 15.0 us, now 13.6,
  // 100 x 151936 bf16 16.0, now 12.5).
  if ((int64_t)n_rows * cs <= num_sms) cfg.dynamicSmemBytes = kLpAlone;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_logprobs<T, TH, kTop, kEntropy>, p);
}

template <class T, int TH>
cudaError_t launch_e(const LogprobsParams& p, int n_rows, int cs, int num_sms, cudaStream_t s) {
  if (p.entropy) return p.top ? launch_t<T, TH, true, true>(p, n_rows, cs, num_sms, s) : launch_t<T, TH, false, true>(p, n_rows, cs, num_sms, s);
  return p.top ? launch_t<T, TH, true, false>(p, n_rows, cs, num_sms, s) : launch_t<T, TH, false, false>(p, n_rows, cs, num_sms, s);
}

template <class T>
cudaError_t launch_d(const LogprobsParams& p, int n_rows, int num_sms, cudaStream_t s) {
  constexpr int kBlock = 32 * LpVec<T>::N;
  // Rows of up to 16 blocks for each of a narrow CTA's warps.
  if (p.vocab <= kLpNarrow / 32 * 16 * kBlock) return launch_e<T, kLpNarrow>(p, n_rows, 1, num_sms, s);
  // CTAs of a row: up to one an SM in all, while each warp has a block of its own.
  // (1, 2, 4, 8 and 16 of them: 1 row of 151936 fp32 with 20 alternatives 20.3, 15.4, 11.9,
  // 10.5 and 11.8 us, where the rule takes 8; 24 rows of 262144 bf16 with 5 19.4, 15.3,
  // 12.2, 14.7 and 30.2, where it takes 4.)
  int cs = 1;
  while (cs < 8 && (int64_t)n_rows * cs * 2 <= num_sms && p.vocab / kBlock >= 2 * cs * (kLpWide / 32)) cs *= 2;
  return launch_e<T, kLpWide>(p, n_rows, cs, num_sms, s);
}

}  // namespace

cudaError_t prepare_logprobs() {
  cudaError_t e;
  if ((e = prepare_e<float, kLpWide>()) != cudaSuccess || (e = prepare_e<float, kLpNarrow>()) != cudaSuccess ||
      (e = prepare_e<bf16, kLpWide>()) != cudaSuccess)
    return e;
  return prepare_e<bf16, kLpNarrow>();
}

// Whether rows of bf16 logits are summed plainly for their entropy: where -1e30 times the scale
// is beyond fp32's range, or not so far down that a weight of it is zero beside any
// reference (below -2^32).
static bool lp_plain(float c) { return c > 0x1p28f || c < 0x1p-67f; }

cudaError_t launch_logprobs(const LogprobsParams& params, int n_rows, bool is_bf16, int num_sms, cudaStream_t s) {
  LogprobsParams p = params;
  p.far = is_bf16 && p.entropy && lp_plain(p.scale_log2) ? 0.0f : kLpFar;
  return is_bf16 ? launch_d<bf16>(p, n_rows, num_sms, s) : launch_d<float>(p, n_rows, num_sms, s);
}

}  // namespace sv
