// sv_paged.cu -- C entry points of the paged-cache operators: argument
// checks and the launches.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "paged.h"

namespace sv {

cudaError_t prepare_attend_64();
cudaError_t prepare_attend_128();
cudaError_t prepare_attend_256();
cudaError_t launch_attend_64(const AttendParams&, int, int, cudaStream_t, bool);
cudaError_t launch_attend_128(const AttendParams&, int, int, cudaStream_t, bool);
cudaError_t launch_attend_256(const AttendParams&, int, int, cudaStream_t, bool);

cudaError_t prepare_attend_kernels() {
  cudaError_t e;
  if ((e = prepare_attend_64()) != cudaSuccess || (e = prepare_attend_128()) != cudaSuccess) return e;
  return prepare_attend_256();
}

cudaError_t launch_attend(const AttendParams& p, int fmt, int head_dim, int num_sms, cudaStream_t s, bool pdl) {
  switch (head_dim) {
    case 64: return launch_attend_64(p, fmt, num_sms, s, pdl);
    case 128: return launch_attend_128(p, fmt, num_sms, s, pdl);
    case 256: return launch_attend_256(p, fmt, num_sms, s, pdl);
  }
  return cudaErrorInvalidValue;
}

namespace {

// Per-device set-up of the attention kernels, and the device's SM count.
struct DeviceSetup {
  int num_sms = 0;
};
std::mutex g_mu;
DeviceSetup g_dev[kMaxDevices];

int device_setup(int* num_sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SV_E_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_dev[dev].num_sms == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return SV_E_CUDA;
    if (prepare_attend_kernels() != cudaSuccess) return SV_E_CUDA;
    g_dev[dev].num_sms = n;
  }
  *num_sms = g_dev[dev].num_sms;
  return SV_OK;
}

bool bad16(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// The pool and the rows as the kernels take them; false: not valid.
bool read_pool(const sv_kv_pool* a, KvPool& c) {
  if (!a || (a->format != SV_KV_BF16 && a->format != SV_KV_E4M3)) return false;
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256) return false;
  if (a->n_pages < 1 || a->n_kv_heads < 1 || bad16(a->k) || bad16(a->v)) return false;
  // the interface's limit: positions of all heads count in 32 bits
  if ((int64_t)a->n_pages * a->n_kv_heads * kPage >= INT32_MAX) return false;
  c = {};
  c.fmt = a->format;
  c.n_pages = a->n_pages;
  c.n_kv_heads = a->n_kv_heads;
  c.head_dim = a->head_dim;
  c.block = 1;
  c.k = static_cast<uint8_t*>(a->k);
  c.v = static_cast<uint8_t*>(a->v);
  if (a->format == SV_KV_E4M3) {
    if (a->scale_block != 1 && a->scale_block != kPage) return false;
    if (bad16(a->k_exp) || bad16(a->v_exp)) return false;
    c.block = a->scale_block;
    c.k_exp = a->k_exp;
    c.v_exp = a->v_exp;
  }
  return true;
}

bool read_rows(const sv_row_batch* a, RowBatch& b) {
  if (!a || a->n_seq < 1 || a->n_rows < 1 || a->table_stride < 1 || !a->block_table || !a->first) return false;
  // positions stay below 2^23 (the attention's merge keeps a word for each
  // split) and rows below 2^28: their sums fit 32 bits
  if (a->table_stride > (1 << 23) / kPage || a->n_rows > (1 << 28)) return false;
  b = {};
  b.n_seq = a->n_seq;
  b.n_rows = a->n_rows;
  b.table_stride = a->table_stride;
  b.table = a->block_table;
  b.first = a->first;
  b.row_start = a->row_start;
  if (a->row_start) {
    b.max_rows = a->max_rows > 0 && a->max_rows < a->n_rows ? a->max_rows : a->n_rows;
  } else {
    if (a->n_rows % a->n_seq) return false;
    b.max_rows = b.rows_each = a->n_rows / a->n_seq;
  }
  return true;
}

bool bad_stride(int64_t stride, int width) { return stride < width || stride % 8 != 0; }

int64_t round256(int64_t b) { return (b + 255) & ~int64_t(255); }

int max_splits(const RowBatch& b) { return attend_split_of(b.limit() - 1) + 1; }

// An attention call's rows are taken in blocks (a row's result depends neither
// on the rows beside it nor on the block), so that their partials fill no more
// than 512 MB, or than 64 rows need and at most 4 GB.  A prompt of 8192 rows of
// 32 heads of 128: 4.5 ms over an 8-bit cache and 6.8 over a bf16 one; all rows
// at once, with 4.9 GB of partials, take 6.1 and 11.1 ms.  (Blocks of 128 MB
// 4.5 and 6.6, of 64 MB 4.8 and 6.9.)  Blocks of few rows leave SMs without
// work: 32 rows at 1000, their table cut for 2^20 positions, take 20 us at once
// (2.2 GB), 51 in blocks of 7 (512 MB).
constexpr int64_t kPartials = int64_t(512) << 20, kPartialsWide = int64_t(4) << 30;
constexpr int64_t kWideRows = 64;

int64_t partial_bytes(int64_t rows, int n_q_heads, int splits, int head_dim) {
  const int64_t slots = rows * n_q_heads * splits;
  return round256(slots * (int64_t)sizeof(float2)) + slots * head_dim * (int64_t)sizeof(float);
}

// Rows of a block: of nearly equal blocks, a multiple of 16 rows each.
int block_rows(const RowBatch& b, int n_q_heads, int head_dim) {
  const int64_t row = partial_bytes(1, n_q_heads, max_splits(b), head_dim);
  const int64_t most = std::max<int64_t>({1, kPartials / row, std::min(kWideRows, kPartialsWide / row)});
  if (most >= b.n_rows) return b.n_rows;
  const int64_t blocks = (b.n_rows + most - 1) / most, each = (b.n_rows + blocks - 1) / blocks;
  return (int)std::min(most, (each + 15) / 16 * 16);
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

int sv_kv_write(const sv_kv_pool* pool, const sv_row_batch* rows, const void* k_dev, int64_t k_stride,
                const void* v_dev, int64_t v_stride, int32_t* status_dev, void* cuda_stream) {
  KvPool c;
  RowBatch b;
  if (!read_pool(pool, c) || !read_rows(rows, b)) return SV_E_INVAL;
  const int width = c.n_kv_heads * c.head_dim;
  if (bad16(k_dev) || bad16(v_dev) || bad_stride(k_stride, width) || bad_stride(v_stride, width)) return SV_E_INVAL;
  if ((int64_t)b.n_rows * width / 8 > UINT32_MAX) return SV_E_INVAL;
  if (c.n_kv_heads > 65535) return SV_E_INVAL;
  KvSource src = {static_cast<const bf16*>(k_dev), static_cast<const bf16*>(v_dev), k_stride, v_stride, 0};
  return launch_kv_write(c, b, src, status_dev, static_cast<cudaStream_t>(cuda_stream), false) == cudaSuccess
             ? SV_OK
             : SV_E_CUDA;
}

int sv_kv_fetch(const sv_kv_pool* pool, const sv_row_batch* rows, void* k_dev, int64_t k_stride, void* v_dev,
                int64_t v_stride, int32_t* status_dev, void* cuda_stream) {
  KvPool c;
  RowBatch b;
  if (!read_pool(pool, c) || !read_rows(rows, b)) return SV_E_INVAL;
  const int width = c.n_kv_heads * c.head_dim;
  if (bad16(k_dev) || bad16(v_dev) || bad_stride(k_stride, width) || bad_stride(v_stride, width)) return SV_E_INVAL;
  if ((int64_t)b.n_rows * width / 8 > UINT32_MAX) return SV_E_INVAL;
  return launch_kv_fetch(c, b, static_cast<bf16*>(k_dev), k_stride, static_cast<bf16*>(v_dev), v_stride, status_dev,
                         static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
             ? SV_OK
             : SV_E_CUDA;
}

int sv_attend_workspace(const sv_kv_pool* pool, const sv_row_batch* rows, int n_q_heads, int64_t* bytes) {
  RowBatch b;
  if (!pool || !bytes || n_q_heads < 1 || !read_rows(rows, b)) return SV_E_INVAL;
  if (pool->head_dim != 64 && pool->head_dim != 128 && pool->head_dim != 256) return SV_E_INVAL;
  if ((int64_t)b.n_rows * n_q_heads > INT32_MAX) return SV_E_INVAL;
  *bytes = partial_bytes(block_rows(b, n_q_heads, pool->head_dim), n_q_heads, max_splits(b), pool->head_dim);
  return SV_OK;
}

int sv_attend(const sv_kv_pool* pool, const sv_row_batch* rows, int n_q_heads, const void* q_dev, int64_t q_stride,
              void* out_dev, int64_t out_stride, float* lse_dev, int window, int sinks, float scale,
              void* workspace_dev, int64_t workspace_bytes, int32_t* status_dev, void* cuda_stream) {
  KvPool c;
  RowBatch b;
  if (!read_pool(pool, c) || !read_rows(rows, b)) return SV_E_INVAL;
  if (n_q_heads < 1 || n_q_heads % c.n_kv_heads || window < 0 || sinks < 0 || !std::isfinite(scale)) return SV_E_INVAL;
  if (b.n_seq > kAttendMaxSeq) return SV_E_INVAL;
  const int width = n_q_heads * c.head_dim;
  if (bad16(q_dev) || bad16(out_dev) || bad_stride(q_stride, width) || bad_stride(out_stride, width)) return SV_E_INVAL;
  int64_t need = 0;
  if (sv_attend_workspace(pool, rows, n_q_heads, &need) != SV_OK) return SV_E_INVAL;
  if ((reinterpret_cast<uintptr_t>(workspace_dev) & 255u) || !workspace_dev) return SV_E_INVAL;
  if (workspace_bytes < need) return SV_E_NOMEM;
  // 32-bit counts on the device, of a block of rows: chunks of 16 positions for
  // every kv head and tile of at least 8 query rows
  const int each = block_rows(b, n_q_heads, c.head_dim);
  const int64_t f = (int64_t)each * n_q_heads;
  if ((f / 8 + (int64_t)b.n_seq * c.n_kv_heads) * (b.limit() / 16 + 1) > INT32_MAX) return SV_E_INVAL;
  int num_sms = 0;
  const int rc = device_setup(&num_sms);
  if (rc != SV_OK) return rc;
  AttendParams p = {};
  p.rows = b;
  p.q = static_cast<const bf16*>(q_dev);
  p.out = static_cast<bf16*>(out_dev);
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.lse = lse_dev;
  p.k = c.k;
  p.v = c.v;
  p.k_exp = c.k_exp;
  p.v_exp = c.v_exp;
  p.n_q_heads = n_q_heads;
  p.n_kv_heads = c.n_kv_heads;
  p.n_pages = c.n_pages;
  p.block = c.block;
  p.window = window;
  p.sinks = sinks;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.max_splits = max_splits(b);
  p.part_ml = static_cast<float2*>(workspace_dev);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace_dev) +
                                      round256(f * p.max_splits * (int64_t)sizeof(float2)));
  p.status = status_dev;
  for (int lo = 0; lo < b.n_rows; lo += each) {
    p.row_lo = lo;
    p.row_hi = std::min(lo + each, b.n_rows);
    if (launch_attend(p, c.fmt, c.head_dim, num_sms, static_cast<cudaStream_t>(cuda_stream), false) != cudaSuccess)
      return SV_E_CUDA;
  }
  return SV_OK;
}

}  // extern "C"
