// logprobs.h -- log probabilities of given tokens (launch interface).
#pragma once
#include "sv_internal.h"

namespace sv {

constexpr int kLogprobsMaxTop = 32;  // alternatives of a row

struct LogprobsParams {
  const void* logits;  // [n_rows, vocab] fp32 or bf16, rows `stride` elements apart
  int64_t stride;
  int vocab, n_tokens, top;
  float scale_log2;  // scale * log2(e), above zero
  const int* tokens;  // [n_rows, n_tokens]
  float *out, *lse, *entropy, *top_values;  // out [n_rows, n_tokens]; the others [n_rows] and [n_rows, top], or null
  int* top_ids;
  int* status;
  float far;  // bf16 rows whose largest scale_log2 x is as far from zero are summed plainly (launch_logprobs sets it)
};

cudaError_t prepare_logprobs();
cudaError_t launch_logprobs(const LogprobsParams& p, int n_rows, bool is_bf16, int num_sms, cudaStream_t s);

}  // namespace sv
