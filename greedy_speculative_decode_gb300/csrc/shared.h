// shared.h -- attention of a batch whose sequences share the pages of a prefix
// (launch interface).
#pragma once
#include "paged.h"

namespace sv {

// Query rows of a tile: the M of a multiply.
constexpr int kSharedTile = 128;
// Tiles that a CTA has at once, and positions of a chunk.
__host__ __device__ constexpr int shared_streams(int d) { return d <= 128 ? 2 : 1; }
__host__ __device__ constexpr int shared_chunk(int d) { return d <= 128 ? 128 : 64; }

// A group of sequences, as k_shared_plan leaves it.
struct SharedGroup {
  int unit0;     // units of work before it (a unit: a chunk for a tile); behind the last group the total
  int eff;       // positions that all its rows see and share; behind the last group the CTAs that take part
  int s0;        // its first sequence with rows that see something, whose table is read
  int row0, R;   // its first row, and its query rows for a kv head
  int chunks, tiles;
  int aligned;   // behind the last group: whether CTAs' runs end with lists (sh_first)
};

// Where a CTA's run begins: the unit, its group, and a copy of that.
struct SharedBegin {
  int unit, group, unused[2];
  SharedGroup g;
};

struct SharedParams {
  AttendParams a;  // q, out, lse, the pool, and the partials of the rows' own positions
  int n_groups;
  const int* group_start;  // [n_groups + 1] or null: groups of n_seq / n_groups sequences
  const int* length;       // [n_groups]
  // workspace
  SharedGroup* plan;  // [n_groups + 1]
  int* from;          // [n_seq] first position of a sequence that is not shared
  int* group;         // [n_seq] its group, or -1
  SharedBegin* begin; // [grid + 1]
  float2* ml;         // [streams][plane] a segment's references and sums
  float* o;           // [streams][plane][head_dim]
  int64_t plane;      // rows of a stream's
  int grid;           // CTAs of the prefix kernel
  uint32_t wait_ns;   // how long one of its waits may last
};

cudaError_t prepare_shared_kernels();
// Whether the units of a call count in 32 bits.
bool shared_units_fit(const RowBatch& b, int n_groups, int n_q_heads, int n_kv_heads, int head_dim);
// The plan and the prefix, for all rows.
cudaError_t launch_shared_prefix(const SharedParams& p, int fmt, int head_dim, cudaStream_t s);
// Rows a.row_lo .. a.row_hi - 1: the prefix's partials and the own positions' merged.
cudaError_t launch_shared_merge(const SharedParams& p, int head_dim, int num_sms, cudaStream_t s);

}  // namespace sv
