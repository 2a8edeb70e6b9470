// Step planning and row commits (tq_step.cu): internal declarations.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tq {

struct PlanArgs {
  const int32_t* seq_lens;
  const int32_t* new_lens;
  const int32_t* seq_blocks;
  int num_seqs;
  int32_t* block_table;
  int max_blocks_per_seq;
  int32_t* free_blocks;  // ring of num_blocks entries
  const int32_t* free_state;  // {head, count}
  int64_t num_blocks;
  int block_size;
  int64_t max_rows;
  int64_t* slots;
  int32_t* q_seq;
  int32_t* q_len;
  int32_t* row_start;
  int32_t* seq_lens_out;
  int32_t* seq_blocks_out;
  int32_t* free_state_out;
  int32_t* status;  // may be null
};
cudaError_t launch_plan_step(const PlanArgs& a, cudaStream_t stream);

struct CommitArgs {
  uint8_t* k_pages;
  int k_slab;  // bytes of one token's K rows, all heads (0: no K pages)
  uint8_t* v_pages;
  int v_slab;
  int64_t num_blocks;
  int block_size;
  const int32_t* block_table;
  int num_seqs;
  int max_blocks_per_seq;
  const int32_t* ctx_lens;
  const int32_t* path;
  const int32_t* path_lens;
  int max_path;
  int32_t* seq_lens_out;
  int32_t* status;  // may be null
};
cudaError_t launch_commit_tree(const CommitArgs& a, cudaStream_t stream);

}  // namespace tq
