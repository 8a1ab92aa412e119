// paged.h -- the paged-cache operators: writing rows into a cache, fetching
// them back, and attention of rows over it (launch interface).
#pragma once
#include "sv_internal.h"

namespace sv {

// A pool of pages: codes [n_pages, n_kv_heads, 16, head_dim] (bf16 or e4m3)
// and, for e4m3, exponent bytes [n_pages, n_kv_heads, 16 / block].
struct KvPool {
  int fmt, n_pages, n_kv_heads, head_dim, block;
  uint8_t *k, *v, *k_exp, *v_exp;
  int row_bytes() const { return head_dim * (fmt == SV_KV_BF16 ? 2 : 1); }
};

// The rows of a call: sequence s brings rows row_start[s] .. row_start[s + 1]
// - 1 (or, with no row_start, rows_each rows), at positions first[s] onward.
// Rows at negative positions are padding.
struct RowBatch {
  int n_seq, n_rows, rows_each, max_rows, table_stride;
  const int* table;      // [n_seq, table_stride]
  const int* first;      // [n_seq]
  const int* row_start;  // [n_seq + 1] or null
  const int* cap;        // positions from *cap on have no pages (a context's table may be stale there), or null
  __host__ __device__ int limit() const { return table_stride * kPage; }  // positions the table reaches
};

// Where new rows' K and V come from: dense rows (stride elements apart, heads
// side by side), or the pages of a bf16 staging pool of src_pages pages in
// which position p of the (single) sequence lies in page (p / 16) % src_pages.
struct KvSource {
  const bf16 *k, *v;
  int64_t k_stride, v_stride;
  int src_pages;
};

cudaError_t launch_kv_write(const KvPool& c, const RowBatch& b, const KvSource& src, int* status, cudaStream_t s,
                            bool pdl);
cudaError_t launch_kv_fetch(const KvPool& c, const RowBatch& b, bf16* k, int64_t k_stride, bf16* v,
                            int64_t v_stride, int* status, cudaStream_t s);

constexpr int kMaxDevices = 64;  // that the attention keeps settings of

// Most sequences of an attention call: each CTA keeps three words per
// sequence in shared memory.
constexpr int kAttendMaxSeq = 1024;

// Splits of the attention's work: ranges of absolute positions, 128 each below
// position 1024 (a short context has many CTAs at work), 256 beyond.
constexpr int kAttendSplitA = 128, kAttendRegionA = 1024, kAttendSplitB = 256;
__host__ __device__ inline int attend_split_of(int pos) {
  return pos < kAttendRegionA ? pos / kAttendSplitA
                              : kAttendRegionA / kAttendSplitA + (pos - kAttendRegionA) / kAttendSplitB;
}
__host__ __device__ inline int attend_split_start(int split) {
  const int n = kAttendRegionA / kAttendSplitA;
  return split < n ? split * kAttendSplitA : kAttendRegionA + (split - n) * kAttendSplitB;
}
// The merge keeps a factor for each split in shared memory: 160 KB hold those
// of the 2^23 positions that a table may reach.
constexpr int kMergeMaxSmem = 160 * 1024;

struct AttendParams {
  RowBatch rows;
  const bf16* q;  // [n_rows, n_q_heads, head_dim], rows q_stride elements apart
  bf16* out;
  int64_t q_stride, out_stride;
  float* lse;  // [n_rows, n_q_heads] natural-log sum of exponentials, or null
  const uint8_t *k, *v, *k_exp, *v_exp;
  int row_lo, row_hi;  // the batch's rows that this launch takes (partials count from row_lo)
  int n_q_heads, n_kv_heads, n_pages, block, window, sinks;
  float scale_log2;  // softmax scale * log2(e)
  int max_splits;
  float2* part_ml;  // [row_hi - row_lo, n_q_heads, max_splits] (running max in log2 units, sum)
  float* part_o;    // [row_hi - row_lo, n_q_heads, max_splits, head_dim]
  int* status;      // or null
  // Whether first, the tables and what the cache holds below first were there
  // before the kernel ahead of this one began (a context's steps): they are then
  // read, and the first pages requested, before the wait for that kernel.
  bool early;
  // First position of each sequence that this launch takes ([n_seq], multiples of
  // the page), or null: those before are another kernel's, which merges too.
  const int* from;
  bool free;  // nothing of the kernel ahead of this one is read or overwritten: it is waited for at the end
};

cudaError_t prepare_attend_kernels();
cudaError_t launch_attend(const AttendParams& p, int fmt, int head_dim, int num_sms, cudaStream_t s, bool pdl);

}  // namespace sv
