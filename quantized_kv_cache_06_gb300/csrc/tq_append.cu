// Host side of tq_norm_rope and tq_append_kv: how a call is cut into warps' work (kernel:
// tq_append.cuh).
#include <algorithm>

#include "tq_append.h"
#include "tq_internal.h"

namespace tq {
namespace {

bool vec_ok(const void* p, int64_t stride, int size) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  if (a.status) {
    const cudaError_t err = cudaMemsetAsync(a.status, 0, sizeof(int32_t), stream);
    if (err != cudaSuccess) return err;
  }
  AppendPlan p{};
  p.a = a;
  const int rpw = 32 / (a.head_dim / 16), size = a.dtype == kF32 ? 4 : 2, sms = device_sms();
  p.heads[0] = a.num_q_heads;
  p.heads[1] = a.num_k_heads;
  p.heads[2] = a.num_v_heads;
  int64_t total = 0;
  for (int i = 0; i < 3; ++i) {
    p.groups[i] = (p.heads[i] + rpw - 1) / rpw;
    total += p.groups[i];
  }
  if (a.num_tokens == 0 || total == 0) return cudaSuccess;
  p.vec = vec_ok(a.q, a.q_stride, size) && vec_ok(a.k, a.k_stride, size) && vec_ok(a.v, a.v_stride, size) &&
          vec_ok(a.q_out, a.q_out_stride, size) && vec_ok(a.k_out, a.k_out_stride, size);
  p.table_vec = reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0 && a.rot_dim % 8 == 0;
  p.signs_vec = reinterpret_cast<uintptr_t>(a.signs) % 16 == 0;
  // Stretches of eight groups share a token's coefficients and hide the copies' latency; shorter ones
  // where they leave warps idle.
  const int64_t warps = (int64_t)sms * kAppendCtas * kAppendWarps;
  const int want = (int)std::max<int64_t>(1, std::min<int64_t>(8, a.num_tokens * total / (2 * warps)));
  const int most = size == 2 ? 4 : 2;  // run_groups
  p.run = std::min(want, most);
  p.chain = want / p.run;
  // Blocks of four tokens where a side's groups of one token are fewer than a stretch.
  p.block_tokens = want > 1 ? 4 : 1;
  const int64_t blocks = (a.num_tokens + p.block_tokens - 1) / p.block_tokens;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  p.blocks = (int)blocks;
  for (int i = 0; i < 3; ++i) {
    p.items[i] = (p.groups[i] * p.block_tokens + p.run * p.chain - 1) / (p.run * p.chain);
    p.block_items += p.items[i];
  }
  const int64_t ctas = (blocks * p.block_items + kAppendWarps - 1) / kAppendWarps;
  p.grid = (int)std::min<int64_t>(ctas, (int64_t)sms * kAppendCtas);
  p.step_block = p.grid * kAppendWarps / p.block_items;
  p.step_part = p.grid * kAppendWarps % p.block_items;
  const bool packed = a.k_pages || a.v_pages;
  switch (a.dtype) {
    case kF32: return packed ? launch_append_packed_f32(p, stream) : launch_append_f32(p, stream);
    case kF16: return packed ? launch_append_packed_f16(p, stream) : launch_append_f16(p, stream);
    case kBF16: return packed ? launch_append_packed_bf16(p, stream) : launch_append_bf16(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
