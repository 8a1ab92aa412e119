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
// logit of each of at most 512 chunks of the row (consecutive ids) in shared
// memory.  The k-th largest of those is a bound that every one of the k reaches;
// at most k chunks have to be read again (from L2), those above the bound and,
// of those equal to it, the first: k tokens of theirs are at least as probable
// as any of a later one, with lower ids.
//
// What bounds it: memory for many rows, the chain of load, meeting and second
// look for a few.  A row is a cluster of 1 to 16 CTAs, so that few rows fill the
// device too; they meet over distributed shared memory.
#include "sv_internal.h"
#include "sv_ptx.cuh"

#include <algorithm>
#include <cooperative_groups.h>

#include "logprobs.h"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;
constexpr int kLpChunks = kLpThreads;  // of a row: a thread looks at one each
constexpr int kLpMost = kLogprobsMaxTop;
constexpr float kLpNone = -3.0e38f;  // reference of what has seen nothing
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
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
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
  static __device__ __forceinline__ float one(const bf16* p) { return __bfloat162float(*p); }
};

// A row in blocks of 32 N elements from the 16-byte boundary at or before its
// first one: element v of that count is token v - lead.
template <class T>
struct LpRow {
  static constexpr int N = LpVec<T>::N, kBlock = 32 * N;
  const T* base;
  int lead, vocab, blocks, per, chunks;  // per: blocks of a chunk
  __device__ __forceinline__ LpRow(const T* row, int vocab_) : vocab(vocab_) {
    lead = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    base = row - lead;
    blocks = (int)(((int64_t)lead + vocab + kBlock - 1) / kBlock);
    per = (blocks + kLpChunks - 1) / kLpChunks;
    chunks = (blocks + per - 1) / per;
  }
  // This lane's part of block b is whole, to be loaded as 16 bytes; else element by element.
  __device__ __forceinline__ bool whole(int b, int lane) const {
    const int64_t v = (int64_t)b * kBlock + lane * N;
    return v >= lead && v + N <= (int64_t)lead + vocab;
  }
  __device__ __forceinline__ uint4 load(int b, int lane) const {
    return __ldg(reinterpret_cast<const uint4*>(base + (int64_t)b * kBlock + lane * N));
  }
  __device__ __forceinline__ void edge(int b, int lane, float (&x)[N]) const {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int64_t v = (int64_t)b * kBlock + lane * N + e;
      x[e] = v >= lead && v < (int64_t)lead + vocab ? LpVec<T>::one(base + v) : -INFINITY;
    }
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

struct LpShared {
  float m[kLpWarps], l[kLpWarps], t[kLpWarps];
  float cta[3];                  // the CTA's (m, l, t)
  uint32_t chunk[kLpChunks];     // largest logit of each of this CTA's chunks
  int chosen[kLpMost], n_chosen;
  uint32_t key[kLpThreads];      // candidates
  int id[kLpThreads];
  int warp_n[kLpWarps];
  uint32_t best_key[kLpMost];    // the CTA's best
  int best_id[kLpMost], n_best;
};

// The best `most` of the threads' candidates (have: this thread has one), in order, into s.best_*.
__device__ __forceinline__ void lp_rank(LpShared& s, bool have, uint32_t key, int id, int most) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t mask = __ballot_sync(0xffffffffu, have);
  if (lane == 0) s.warp_n[warp] = __popc(mask);
  __syncthreads();
  int before = 0, n = 0;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) {
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
    if (rank < most) {
      s.best_key[rank] = key;
      s.best_id[rank] = id;
    }
  }
  if (tid == 0) s.n_best = min(n, most);
  __syncthreads();
}

template <class T, bool kTop>
__global__ void __launch_bounds__(kLpThreads) k_logprobs(const LogprobsParams p) {
  using V = LpVec<T>;
  constexpr int N = V::N, kBatch = 4;
  __shared__ LpShared s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / CS;
  const T* logits = static_cast<const T*>(p.logits) + (int64_t)r * p.stride;
  const LpRow<T> row(logits, p.vocab);
  const float c = p.scale_log2;
  const int c0 = (int)((int64_t)rank * row.chunks / CS), c1 = (int)((int64_t)(rank + 1) * row.chunks / CS);
  const int b0 = c0 * row.per, b1 = min(c1 * row.per, row.blocks);
  if (kTop) {
    s.chunk[tid] = 0;
    __syncthreads();
  }
  float m = kLpNone, l = 0.0f, t = 0.0f;
  for (int b = b0 + warp; b < b1; b += kBatch * kLpWarps) {
    uint4 w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (b + i * kLpWarps < b1 && row.whole(b + i * kLpWarps, lane)) w[i] = row.load(b + i * kLpWarps, lane);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int bi = b + i * kLpWarps;
      if (bi >= b1) break;
      float x[N];
      if (row.whole(bi, lane)) V::open(w[i], x);
      else row.edge(bi, lane, x);
      float top = x[0];
#pragma unroll
      for (int e = 1; e < N; ++e) top = fmaxf(top, x[e]);
      top = warp_max(top);
      if (kTop && lane == 0) atomicMax(&s.chunk[bi / row.per], order_of(top));
      const float y = __fmul_rn(top, c);
      if (y > m) {
        const float d = __fsub_rn(m, y), f = lp_ex2(d);
        t = f > 0.0f ? __fmul_rn(f, __fmaf_rn(d, l, t)) : 0.0f;
        l = __fmul_rn(f, l);
        m = y;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        // (2^z (z) of an impossible token is zero, not 0 * inf; a NaN stays one)
        const float z = max_nan(__fmaf_rn(x[e], c, -m), -1000.0f), q = lp_ex2(z);
        l = __fadd_rn(l, q);
        t = __fmaf_rn(q, z, t);
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
  // A row with a NaN or an infinity, or of nothing but -infinity, has no distribution.
  const float NaN = __uint_as_float(0x7fffffffu), ln2 = 0.6931471805599453f;
  const bool good = L > 0.0f && L < INFINITY && fabsf(M) < INFINITY;
  const float l2 = good ? log2f(L) : NaN;
  auto log_prob = [&](float x) { return __fmul_rn(__fsub_rn(__fmaf_rn(x, c, -M), l2), ln2); };
  if (rank == 0) {
    for (int i = tid; i < p.n_tokens; i += kLpThreads) {
      const int tok = __ldg(p.tokens + (int64_t)r * p.n_tokens + i);
      float v = 0.0f;  // a token of -1: an unused place
      if (tok >= 0 && tok < p.vocab) v = log_prob(V::one(logits + tok));
      else if (tok != -1) {
        v = NaN;
        if (p.status) atomicOr(p.status, ST_BAD_TOKEN);
      }
      p.out[(int64_t)r * p.n_tokens + i] = v;
    }
    if (tid == 0) {
      if (p.lse) p.lse[r] = __fmul_rn(__fadd_rn(M, l2), ln2);
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
  // The largest bound that k chunks reach, bit by bit.
  uint32_t bound = 0;
  bool exact = false;
  for (uint32_t bit = 0x80000000u; bit && !exact; bit >>= 1) {
    const int n = __syncthreads_count(key >= (bound | bit));
    if (n >= k) {
      bound |= bit;
      exact = n == k;
    }
  }
  // Chunks above the bound, and the first of those equal to it (all that reach it, where they are k).
  bool take = key > kOrderNegInf && key >= bound;
  if (!exact && bound > 0) {
    const int above = __syncthreads_count(key > bound);
    const uint32_t eq = __ballot_sync(0xffffffffu, key == bound);
    if (lane == 0) s.warp_n[warp] = __popc(eq);
    __syncthreads();
    int before = __popc(eq & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) before += s.warp_n[w];
    if (key == bound && before >= k - above) take = false;
  }
  if (tid == 0) s.n_chosen = 0;
  __syncthreads();
  if (take && tid >= c0 && tid < c1) s.chosen[atomicAdd(&s.n_chosen, 1)] = tid;
  __syncthreads();
  LpBest best = {0u, -1};
  const int items = s.n_chosen * row.per;
  for (int i = warp; i < items; i += kLpWarps) {
    const int b = s.chosen[i / row.per] * row.per + i % row.per;
    if (b >= row.blocks) continue;
    float x[N];
    if (row.whole(b, lane)) V::open(row.load(b, lane), x);
    else row.edge(b, lane, x);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const uint32_t ke = order_of(x[e]);
      const int id = (int)((int64_t)b * LpRow<T>::kBlock + lane * N + e - row.lead);
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
      bool have = false;
      if (i < CS) {
        have = j < *cluster.map_shared_rank(&s.n_best, i);
        if (have) {
          key = cluster.map_shared_rank(s.best_key, i)[j];
          best.id = cluster.map_shared_rank(s.best_id, i)[j];
        }
      }
      __syncthreads();  // this CTA's own are in registers now
      lp_rank(s, have, key, best.id, k);
    }
  }
  if (rank == 0 && tid < k) {
    const bool there = tid < s.n_best;
    const uint32_t o = there ? s.best_key[tid] : 0;
    const float x = __uint_as_float((o >> 31) ? o ^ 0x80000000u : ~o);
    if (p.top_values) p.top_values[(int64_t)r * k + tid] = !good ? NaN : there ? log_prob(x) : -INFINITY;
    if (p.top_ids) p.top_ids[(int64_t)r * k + tid] = there ? s.best_id[tid] : -1;
  }
  if (CS > 1) cluster.sync();
}

template <class T, bool kTop>
cudaError_t launch_t(const LogprobsParams& p, int n_rows, int cs, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)n_rows * cs);
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_logprobs<T, kTop>, p);
}

template <class T>
cudaError_t prepare_t() {
  cudaError_t e = cudaFuncSetAttribute(k_logprobs<T, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(k_logprobs<T, false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

}  // namespace

cudaError_t prepare_logprobs() {
  cudaError_t e = prepare_t<float>();
  return e != cudaSuccess ? e : prepare_t<bf16>();
}

cudaError_t launch_logprobs(const LogprobsParams& p, int n_rows, bool is_bf16, int num_sms, cudaStream_t s) {
  // CTAs of a row: as many as keep two on an SM busy, while each warp has a block of its own.
  const int blocks = p.vocab / (32 * (is_bf16 ? LpVec<bf16>::N : LpVec<float>::N));
  int cs = 1;
  while (cs < 16 && (int64_t)n_rows * cs * 2 <= 2 * num_sms && blocks >= 2 * cs * kLpWarps) cs *= 2;
  if (is_bf16) return p.top ? launch_t<bf16, true>(p, n_rows, cs, s) : launch_t<bf16, false>(p, n_rows, cs, s);
  return p.top ? launch_t<float, true>(p, n_rows, cs, s) : launch_t<float, false>(p, n_rows, cs, s);
}

}  // namespace sv
