// k_shared.cu -- the plan of attention to shared prefixes, and the launches of its
// kernels (shared_dev.cuh).
#include "shared_dev.cuh"

#include <algorithm>

namespace sv {
namespace {

// What the groups share: eff, the positions that lie in shared pages and that all
// rows of the group see (whole pages of them), and the work this makes.  One
// thread a sequence, then one a group.
__global__ void __launch_bounds__(1024) k_shared_plan(const __grid_constant__ SharedParams p, int chunk, int streams) {
  __shared__ int s_eff[1024], s_lead[1024], s_start[1025];  // s_lead: a group's first sequence with rows that see something
  __shared__ int s_sum[32], s_sum2[32], s_unit[1025], s_list[1025];  // units and lists before each group
  __shared__ int2 s_first[256];  // of each list, where CTAs' runs end with lists: its first unit, and CTA
  const int tid = threadIdx.x, S = p.a.rows.n_seq, N = p.n_groups, G = p.a.n_q_heads / p.a.n_kv_heads;
  pdl_trigger();
  pdl_wait();
  auto given_start = [&](int s) { return p.a.rows.row_start ? __ldcg(p.a.rows.row_start + s) : s * p.a.rows.rows_each; };
  auto start_of = [&](int s) { return min(max(given_start(s), 0), p.a.rows.n_rows); };  // (as k_attend reads them)
  int first = 0, n = 0;
  if (tid < S) {
    const int at = given_start(tid);
    first = first_of(p.a.rows, tid) + (at < 0 ? (int)min(-(int64_t)at, (int64_t)1 << 28) : 0);
    n = start_of(tid + 1) - start_of(tid);
  }
  if (tid < 32) s_sum[tid] = s_sum2[tid] = 0;
  for (int g = tid; g <= N; g += blockDim.x)
    s_start[g] = p.group_start ? min(max(__ldcg(p.group_start + g), 0), S) : (int)((long long)S * g / N);
  if (tid < N) {
    const int most = min(max(__ldcg(p.length + tid), 0), p.a.rows.limit());
    s_eff[tid] = most;
    s_lead[tid] = S;
  }
  __syncthreads();
  // Groups or rows that run backwards: nothing is shared.  (Of rows that do, the merge's
  // search could find one below its group's first, whose partials are elsewhere.)
  const bool back = __syncthreads_or((tid < N && s_start[tid + 1] < s_start[tid]) || n < 0);
  if (back && tid == 0 && p.a.status) atomicOr(p.a.status, ST_BAD_PAGE);
  int gi = -1;
  if (tid < S) {
    if (!back && tid >= s_start[0] && tid < s_start[N]) {
      int lo = 0, hi = N;  // the last group that begins at or before the sequence
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= tid) lo = mid; else hi = mid;
      }
      gi = lo;
      if (n > 0 && first + n > 0) {  // (rows of padding alone see nothing)
        atomicMin(&s_eff[gi], max(first, 0) + 1);
        atomicMin(&s_lead[gi], tid);
      }
    }
    p.group[tid] = gi;
  }
  __syncthreads();
  SharedGroup g = {};
  int units = 0;
  if (tid < N) {
    g.s0 = s_lead[tid];
    if (!back && g.s0 < S) {
      g.row0 = start_of(s_start[tid]);
      const int rows = start_of(s_start[tid + 1]) - g.row0;
      if (rows > 0) {
        g.eff = s_eff[tid] / kPage * kPage;
        g.R = rows * G;
        g.chunks = (g.eff + chunk - 1) / chunk;
        g.tiles = (g.R + kSharedTile - 1) / kSharedTile;
      }
    }
    s_eff[tid] = g.eff;
    units = p.a.n_kv_heads * g.chunks * g.tiles;
  }
  // A CTA has whole chunks: two units, where a list has two tiles.
  const int least = __syncthreads_or(units > 0 && g.tiles > 1) ? streams : 1;
  // units and lists before each group
  const int lane = tid & 31, warp = tid >> 5;
  const int lists = units > 0 ? p.a.n_kv_heads * ((g.tiles + streams - 1) / streams) : 0;
  int x = units, y = lists;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += a;
      y += b;
    }
  }
  if (lane == 31) {
    s_sum[warp] = x;
    s_sum2[warp] = y;
  }
  __syncthreads();
  int before = 0, all = 0, before2 = 0, all2 = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    before += w < warp ? s_sum[w] : 0;
    before2 += w < warp ? s_sum2[w] : 0;
    all += s_sum[w];
    all2 += s_sum2[w];
  }
  const int ctas = min(p.grid, max(all / least, 1));
  // Lists of at least a CTA's share each: then a CTA works on one alone.
  const int small = g.chunks * (g.tiles % streams ? g.tiles % streams : streams);
  const int aligned = __syncthreads_and(units == 0 || (long long)small * ctas >= all) && all2 <= ctas;
  if (tid < N) {
    g.unit0 = before + x - units;
    s_unit[tid] = g.unit0;
    s_list[tid] = before2 + y - lists;
    p.plan[tid] = g;
  }
  if (tid == 0) {
    SharedGroup end = {};
    end.unit0 = all;
    end.eff = ctas;
    end.aligned = aligned;
    p.plan[N] = end;
  }
  __syncthreads();
  auto last_at = [](const int* v, int n, int u) {  // the last of n that is at most u
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (v[mid] <= u) lo = mid; else hi = mid;
    }
    return lo;
  };
  if (aligned && tid < all2) {
    const int gi = last_at(s_list, N, tid);
    const SharedGroup q = p.plan[gi];  // (written by this block before the barrier)
    const int pairs = (q.tiles + streams - 1) / streams, i = tid - s_list[gi];
    const int u = q.unit0 + i / pairs * q.chunks * q.tiles + i % pairs * streams * q.chunks;
    s_first[tid] = make_int2(u, sh_first(u, all, ctas));
  }
  __syncthreads();
  if (tid <= p.grid) {  // where each CTA's run begins
    int u = all;
    if (tid < ctas && all > 0) {
      u = (int)((unsigned long long)all * tid / ctas);
      if (aligned) {
        int lo = 0, hi = all2;  // its list
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_first[mid].y <= tid) lo = mid; else hi = mid;
        }
        const int2 a = s_first[lo], b = lo + 1 < all2 ? s_first[lo + 1] : make_int2(all, ctas);
        const SharedGroup q = p.plan[last_at(s_unit, N, a.x)];
        const int w = (b.x - a.x) / q.chunks;  // its tiles
        u = a.x + (int)((long long)q.chunks * (tid - a.y) / (b.y - a.y)) * w;
      }
    }
    const int lo = last_at(s_unit, N, u);
    p.begin[tid].unit = u;
    p.begin[tid].group = lo;
    p.begin[tid].g = p.plan[lo];
  }
  if (tid < S) p.from[tid] = gi >= 0 ? s_eff[gi] : 0;
}

}  // namespace

bool shared_units_fit(const RowBatch& b, int n_groups, int n_q_heads, int n_kv_heads, int head_dim) {
  const int64_t chunks = b.limit() / shared_chunk(head_dim) + 1;
  const int64_t tiles = (int64_t)b.n_rows * (n_q_heads / n_kv_heads) / kSharedTile + n_groups;
  return chunks * tiles <= INT32_MAX / 2 / n_kv_heads;
}

cudaError_t prepare_shared_kernels() {
  cudaError_t e;
  if ((e = shared_prepare<64, SV_KV_BF16>()) != cudaSuccess || (e = shared_prepare<64, SV_KV_E4M3>()) != cudaSuccess ||
      (e = shared_prepare<128, SV_KV_BF16>()) != cudaSuccess || (e = shared_prepare<128, SV_KV_E4M3>()) != cudaSuccess ||
      (e = shared_prepare<256, SV_KV_BF16>()) != cudaSuccess)
    return e;
  return shared_prepare<256, SV_KV_E4M3>();
}

cudaError_t launch_shared_prefix(const SharedParams& p, int fmt, int head_dim, cudaStream_t s) {
  const int most = std::max(p.a.rows.n_seq, p.grid + 1);  // (a thread each)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(std::min(1024, (most + 31) / 32 * 32));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_shared_plan, p, shared_chunk(head_dim), shared_streams(head_dim));
  if (e != cudaSuccess) return e;
  const bool b = fmt == SV_KV_BF16;
  switch (head_dim) {
    case 64: return b ? shared_launch<64, SV_KV_BF16>(p, s) : shared_launch<64, SV_KV_E4M3>(p, s);
    case 128: return b ? shared_launch<128, SV_KV_BF16>(p, s) : shared_launch<128, SV_KV_E4M3>(p, s);
    case 256: return b ? shared_launch<256, SV_KV_BF16>(p, s) : shared_launch<256, SV_KV_E4M3>(p, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_shared_merge(const SharedParams& p, int head_dim, int num_sms, cudaStream_t s) {
  switch (head_dim) {
    case 64: return shared_merge_launch<64>(p, num_sms, s);
    case 128: return shared_merge_launch<128>(p, num_sms, s);
    case 256: return shared_merge_launch<256>(p, num_sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace sv
