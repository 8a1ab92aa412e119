// sv_pages.cu -- C entry points of the operators on a cache's pages and of the
// log probabilities: argument checks and the launches.
#include <cmath>
#include <mutex>

#include "logprobs.h"
#include "pages.h"

namespace sv {
namespace {

// Per-device set-up of the kernels here, and the device's SM count.
std::mutex g_mu;
int g_sms[kMaxDevices];

int device_setup(int* num_sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SV_E_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_sms[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return SV_E_CUDA;
    if (prepare_pages() != cudaSuccess || prepare_logprobs() != cudaSuccess) return SV_E_CUDA;
    g_sms[dev] = n;
  }
  *num_sms = g_sms[dev];
  return SV_OK;
}

int launched(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_E_CUDA; }

bool bad4(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
bool odd4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }  // (null is fine)
bool bad16(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

bool read_pages(const sv_kv_pages* a, PageTable& t) {
  if (!a || a->n_seq < 1 || a->n_seq > kPagesMaxSeq || a->table_stride < 1 || a->table_stride > (1 << 23) / kPage ||
      a->n_pages < 1 || a->n_pages >= (1 << 27))
    return false;
  if (bad4(a->block_table) || bad4(a->length) || bad4(a->held) || bad4(a->refs)) return false;
  t = {a->n_seq, a->table_stride, a->n_pages, a->block_table, a->length, a->held, a->refs};
  return true;
}

// Where a plan's results go: `out`, or in place.
bool read_out(const sv_kv_pages* pages, const sv_kv_pages* out, const PageTable& in, PageTable& t, bool& in_place) {
  in_place = out == nullptr || out == pages;
  t = in;
  if (in_place) return true;
  if (!read_pages(out, t) || t.n_seq != in.n_seq || t.width != in.width || t.n_pages != in.n_pages) return false;
  const int same = (t.table == in.table) + (t.length == in.length) + (t.held == in.held) + (t.refs == in.refs);
  in_place = same == 4;
  return same == 0 || same == 4;
}

// A pool as the copy takes it; geometry in `c`.
bool read_pool(const sv_kv_pool& a, KvPool& c) {
  if (a.format != SV_KV_BF16 && a.format != SV_KV_E4M3) return false;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return false;
  if (a.n_pages < 1 || a.n_kv_heads < 1 || a.n_kv_heads > 65535 || bad16(a.k) || bad16(a.v)) return false;
  if ((int64_t)a.n_pages * a.n_kv_heads * kPage >= INT32_MAX) return false;
  c = {};
  c.fmt = a.format;
  c.n_pages = a.n_pages;
  c.n_kv_heads = a.n_kv_heads;
  c.head_dim = a.head_dim;
  c.block = 1;
  c.k = static_cast<uint8_t*>(a.k);
  c.v = static_cast<uint8_t*>(a.v);
  if (a.format == SV_KV_E4M3) {
    if (a.scale_block != 1 && a.scale_block != kPage) return false;
    if (bad16(a.k_exp) || bad16(a.v_exp)) return false;
    c.block = a.scale_block;
    c.k_exp = a.k_exp;
    c.v_exp = a.v_exp;
  }
  return true;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

int sv_kv_fork_workspace(const sv_kv_pages* pages, int64_t* bytes) {
  PageTable t;
  if (!bytes || !read_pages(pages, t)) return SV_E_INVAL;
  *bytes = 4 * ((int64_t)t.n_pages + (int64_t)t.n_seq * t.width);
  return SV_OK;
}

int sv_kv_fork(const sv_kv_pages* pages, const int32_t* source, const int32_t* keep, const int32_t* room,
               const sv_kv_pages* out, int32_t* moves_dev, void* workspace_dev, int64_t workspace_bytes,
               int32_t* status_dev, void* cuda_stream) {
  ForkParams p = {};
  if (!read_pages(pages, p.in) || !read_out(pages, out, p.in, p.out, p.in_place)) return SV_E_INVAL;
  if (odd4(source) || odd4(keep) || odd4(room) || odd4(status_dev) || !moves_dev ||
      (reinterpret_cast<uintptr_t>(moves_dev) & 7u) || bad16(workspace_dev))
    return SV_E_INVAL;
  int64_t need = 0;
  if (sv_kv_fork_workspace(pages, &need) != SV_OK) return SV_E_INVAL;
  if (workspace_bytes < need) return SV_E_NOMEM;
  int num_sms = 0;
  const int rc = device_setup(&num_sms);
  if (rc != SV_OK) return rc;
  p.source = source;
  p.keep = keep;
  p.room = room;
  p.moves = reinterpret_cast<int2*>(moves_dev);
  p.count = static_cast<int*>(workspace_dev);
  p.staged = p.count + p.in.n_pages;
  p.status = status_dev;
  return launched(launch_fork(p, static_cast<cudaStream_t>(cuda_stream)));
}

int sv_kv_compact(const sv_kv_pages* pages, const sv_kv_pages* out, int32_t* moves_dev, int32_t n_moves,
                  int32_t* where_dev, int32_t* status_dev, void* cuda_stream) {
  CompactParams p = {};
  if (!read_pages(pages, p.in) || !read_out(pages, out, p.in, p.out, p.in_place)) return SV_E_INVAL;
  if (!moves_dev || (reinterpret_cast<uintptr_t>(moves_dev) & 7u) || n_moves < 1 || bad4(where_dev) || odd4(status_dev))
    return SV_E_INVAL;
  int num_sms = 0;
  const int rc = device_setup(&num_sms);
  if (rc != SV_OK) return rc;
  p.moves = reinterpret_cast<int2*>(moves_dev);
  p.n_moves = n_moves;
  p.where = where_dev;
  p.status = status_dev;
  return launched(launch_compact(p, static_cast<cudaStream_t>(cuda_stream)));
}

int sv_kv_copy(const sv_kv_pool* from, const sv_kv_pool* into, int n_pools, const int32_t* moves_dev, int32_t n_moves,
               int32_t* status_dev, void* cuda_stream) {
  if (!from || n_pools < 1 || n_moves < 1 || !moves_dev || (reinterpret_cast<uintptr_t>(moves_dev) & 7u) || odd4(status_dev))
    return SV_E_INVAL;
  if (!into) into = from;
  KvPool f0, t0;
  for (int i = 0; i < n_pools; ++i) {
    KvPool f, t;
    if (!read_pool(from[i], f) || !read_pool(into[i], t)) return SV_E_INVAL;
    if (i == 0) {
      f0 = f;
      t0 = t;
    }
    if (f.fmt != f0.fmt || f.n_kv_heads != f0.n_kv_heads || f.head_dim != f0.head_dim || f.block != f0.block ||
        f.n_pages != f0.n_pages || t.fmt != f0.fmt || t.n_kv_heads != f0.n_kv_heads || t.head_dim != f0.head_dim ||
        t.block != f0.block || t.n_pages != t0.n_pages)
      return SV_E_INVAL;
  }
  int num_sms = 0;
  const int rc = device_setup(&num_sms);
  if (rc != SV_OK) return rc;
  CopyParams p;  // (pools beyond n_pools are not read)
  p.moves = reinterpret_cast<const int2*>(moves_dev);
  p.n_moves = n_moves;
  p.n_from = f0.n_pages;
  p.n_to = t0.n_pages;
  p.page_bytes = f0.n_kv_heads * kPage * f0.row_bytes();
  p.exp_bytes = f0.fmt == SV_KV_E4M3 ? f0.n_kv_heads * kPage / f0.block : 0;
  p.status = status_dev;
  for (int i = 0; i < n_pools; i += kCopyPools) {
    p.n_pools = n_pools - i < kCopyPools ? n_pools - i : kCopyPools;
    for (int j = 0; j < p.n_pools; ++j) {
      KvPool f, t;
      if (!read_pool(from[i + j], f) || !read_pool(into[i + j], t)) return SV_E_INVAL;
      p.pool[j] = {f.k, f.v, f.k_exp, f.v_exp, t.k, t.v, t.k_exp, t.v_exp};
    }
    const int r = launched(launch_copy(p, num_sms, static_cast<cudaStream_t>(cuda_stream)));
    if (r != SV_OK) return r;
  }
  return SV_OK;
}

int sv_logprobs(const void* logits_dev, int dtype, int64_t stride, int n_rows, int vocab, float scale,
                const int32_t* tokens_dev, int n_tokens, float* out_dev, float* lse_dev, float* entropy_dev, int top,
                float* top_values_dev, int32_t* top_ids_dev, int32_t* status_dev, void* cuda_stream) {
  if (dtype != SV_LOGITS_F32 && dtype != SV_LOGITS_BF16) return SV_E_INVAL;
  const uintptr_t at = reinterpret_cast<uintptr_t>(logits_dev);
  if (!logits_dev || at % (dtype == SV_LOGITS_F32 ? 4 : 2) || n_rows < 1 || vocab < 1 || vocab > (1 << 30) ||
      (n_rows > 1 && stride < vocab) || stride < 0)
    return SV_E_INVAL;
  if (n_rows > (1 << 26) || n_tokens < 0 || top < 0 || top > kLogprobsMaxTop) return SV_E_INVAL;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale_log2 > 0.0f) || !std::isfinite(scale_log2)) return SV_E_INVAL;
  if (n_tokens > 0 && (bad4(tokens_dev) || bad4(out_dev))) return SV_E_INVAL;
  if (top > 0 && !top_values_dev && !top_ids_dev) return SV_E_INVAL;
  if (odd4(lse_dev) || odd4(entropy_dev) || odd4(top_values_dev) || odd4(top_ids_dev) || odd4(status_dev)) return SV_E_INVAL;
  int num_sms = 0;
  const int rc = device_setup(&num_sms);
  if (rc != SV_OK) return rc;
  LogprobsParams p = {};
  p.logits = logits_dev;
  p.stride = stride;
  p.vocab = vocab;
  p.n_tokens = n_tokens;
  p.top = top;
  p.scale_log2 = scale_log2;
  p.tokens = tokens_dev;
  p.out = out_dev;
  p.lse = lse_dev;
  p.entropy = entropy_dev;
  p.top_values = top_values_dev;
  p.top_ids = top_ids_dev;
  p.status = status_dev;
  return launched(launch_logprobs(p, n_rows, dtype == SV_LOGITS_BF16, num_sms, static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
