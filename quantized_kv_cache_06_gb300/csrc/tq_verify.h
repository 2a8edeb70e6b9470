// Verification of drafted tokens (tq_verify.cu): internal declarations.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tq {

struct VerifyArgs {
  const void* logits;
  int logits_dtype;
  int64_t logits_stride;
  int num_rows;
  int vocab;
  const void* draft;  // may be null
  int draft_dtype;
  int64_t draft_stride;
  const int32_t* row_start;
  int num_seqs;
  const int32_t* tokens;
  const int32_t* parents;      // null: chains
  const float* temperature;    // null: 1
  const float* u_accept;       // null without draft
  const float* u_sample;
  int32_t* path;
  int max_path;
  int32_t* path_lens;
  int32_t* next_token;
  void* workspace;
  int32_t* status;  // may be null
};
size_t verify_workspace(int num_rows, int vocab, int num_seqs);
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream);

}  // namespace tq
