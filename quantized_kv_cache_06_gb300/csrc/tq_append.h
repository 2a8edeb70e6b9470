// Head norms with position rotation, and the append into packed pages (tq_append.cu): internal
// declarations.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tq {

struct AppendArgs {
  // rows of head_dim elements, heads of a token contiguous, tokens `stride` elements apart
  const void* q;
  int64_t q_stride;
  int num_q_heads;  // 0: no queries
  const void* k;
  int64_t k_stride;
  int num_k_heads;
  const void* v;
  int64_t v_stride;
  int num_v_heads;
  int dtype;
  int64_t num_tokens;
  int head_dim;
  void* q_out;  // dense, of the input type
  int64_t q_out_stride;
  void* k_out;  // dense keys (k_pages is then null)
  int64_t k_out_stride;
  // packed rows
  const int64_t* slots;
  int64_t num_slots;
  uint8_t* k_pages;
  int k_bits;
  uint8_t* v_pages;
  int v_bits;
  const float* signs;
  const float* k_centroids;
  const float* v_centroids;
  // norms (null: none) and position rotation (cos_sin null: none)
  const float* q_weight;
  const float* k_weight;
  float eps;
  const int32_t* positions;
  int position_offset;
  const float* cos_sin;
  int64_t num_positions;
  int rot_dim;
  int interleaved;
  int32_t* status;  // may be null
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);

constexpr int kAppendWarps = 8;
constexpr int kAppendCtas = 2;  // CTAs of an SM

constexpr int kRunGroups = 8;   // groups of a run (fp32: half as many)

// How a call is cut: blocks of tokens, each side's groups of 32 / (head_dim / 16) heads over a block
// in runs of `run` groups, a warp a run.
struct AppendSide {
  const unsigned char* in;
  int64_t in_step;            // bytes between tokens
  unsigned char* out;         // dense rows, or pages
  int64_t out_step;           // bytes between tokens, or of a packed row
  int64_t slot_step;          // bytes of a packed token
  int heads, groups, first;   // first: of its runs in a block
  uint32_t inv_groups;        // ceil(2^32 / groups), groups 2 .. 2^14: u / groups = umulhi(u, inv_groups) for u < 8 groups
  int normed;
};
struct AppendPlan {
  AppendArgs a;
  int block_tokens, blocks;
  int run;                    // groups of a run
  AppendSide side[3];         // q, k, v
  int items[3];               // runs of a block
  int block_items;
  int warps;                  // that take part
  int step_block, step_part, carry;  // from one run of a warp to its next
  int grid;
  int full;                   // every side's heads fill its groups
  int vec;                    // inputs and dense outputs: 16-byte accesses
  int table_vec;              // table rows: 16-byte loads
};
// By type, dense or packed (one translation unit each).
cudaError_t launch_append_f32(const AppendPlan& p, cudaStream_t stream);
cudaError_t launch_append_f16(const AppendPlan& p, cudaStream_t stream);
cudaError_t launch_append_bf16(const AppendPlan& p, cudaStream_t stream);
cudaError_t launch_append_packed_f32(const AppendPlan& p, cudaStream_t stream);
cudaError_t launch_append_packed_f16(const AppendPlan& p, cudaStream_t stream);
cudaError_t launch_append_packed_bf16(const AppendPlan& p, cudaStream_t stream);

}  // namespace tq
