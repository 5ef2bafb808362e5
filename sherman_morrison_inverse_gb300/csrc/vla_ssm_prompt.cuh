// How vla_ssm_scan runs a call on the tensor cores (vla_ssm_prompt.cu).
#pragma once

#include "vla_layer.cuh"

namespace vla {

struct PromptPlan {
  bool fits;              // the form takes these sizes and type, and is the faster one (alignment is seen
                          // at the launch)
  int nn;                 // states rounded up: 64 or 128
  int nseg;               // segments a sequence is cut into
  long long seg_chunks;   // chunks of 128 tokens a segment
  long long whole;        // the first of the (sequence, slice) pairs that are not cut
  size_t ws_bytes;
};

// tokens: of all sequences together
PromptPlan ssm_prompt_plan(long long n_seq, long long tokens, long long max_len, long long H, long long P, long long N,
                           bool bf16, int sm_count);

// *used = false: some operand's alignment or strides do not fit, nothing was launched.
cudaError_t launch_ssm_prompt(const SsmArgs& a, const PromptPlan& plan, cudaStream_t s, bool* used);

}  // namespace vla
