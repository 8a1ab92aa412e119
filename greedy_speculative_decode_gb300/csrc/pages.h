// pages.h -- pages of a cache handed out, shared, packed and copied (launch interface).
#pragma once
#include "paged.h"

namespace sv {

constexpr int kPagesMaxSeq = 1024;  // rows of a table: one for each thread of a CTA
constexpr int kCopyPools = 32;      // pools of one copy launch

// sv_kv_pages as the kernels take it.
struct PageTable {
  int n_seq, width, n_pages;
  int *table, *length, *held, *refs;
};

struct ForkParams {
  PageTable in, out;
  bool in_place;  // out is in
  const int *source, *keep, *room;  // each [n_seq] or null
  int2* moves;                      // [n_seq]
  int* count;                       // workspace [n_pages]: rows that will hold a page
  int* staged;                      // workspace [n_seq, width], in place: entries that another row's become
  int* status;
};

struct CompactParams {
  PageTable in, out;
  bool in_place;
  int2* moves;  // [n_moves]
  int n_moves;
  int* where;   // [n_pages]: a page's new number, -1 for a free one
  int* status;
};

struct CopyParams {
  struct Pool {
    const uint8_t *k, *v, *k_exp, *v_exp;
    uint8_t *k_to, *v_to, *k_exp_to, *v_exp_to;
  } pool[kCopyPools];
  const int2* moves;
  int n_pools, n_moves, n_from, n_to;  // pages of the pools read and written
  int page_bytes, exp_bytes;           // of K or V of a page
  int* status;
};

cudaError_t prepare_pages();
cudaError_t launch_fork(const ForkParams& p, cudaStream_t s);
cudaError_t launch_compact(const CompactParams& p, cudaStream_t s);
cudaError_t launch_copy(const CopyParams& p, int num_sms, cudaStream_t s);

}  // namespace sv
