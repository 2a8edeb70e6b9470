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
  const int heads[3] = {a.num_q_heads, a.num_k_heads, a.num_v_heads};
  const void* in[3] = {a.q, a.k, a.v};
  const int64_t stride[3] = {a.q_stride, a.k_stride, a.v_stride};
  int64_t total = 0;
  p.full = 1;
  for (int i = 0; i < 3; ++i) {
    AppendSide& s = p.side[i];
    s.in = static_cast<const unsigned char*>(in[i]);
    s.in_step = stride[i] * size;
    s.heads = heads[i];
    s.groups = (heads[i] + rpw - 1) / rpw;
    s.inv_groups = s.groups > 1 ? (uint32_t)((0x100000000ull + s.groups - 1) / s.groups) : 0;
    s.normed = (i == 0 ? a.q_weight : i == 1 ? a.k_weight : nullptr) != nullptr;
    p.full &= heads[i] % rpw == 0;
    total += s.groups;
  }
  auto packed_row = [&](int bits) { return (int64_t)a.head_dim * bits / 8 + 4; };
  p.side[0].out = static_cast<unsigned char*>(a.q_out);
  p.side[0].out_step = a.q_out_stride * size;
  p.side[1].out = a.k_pages ? a.k_pages : static_cast<unsigned char*>(a.k_out);
  p.side[1].out_step = a.k_pages ? packed_row(a.k_bits) : a.k_out_stride * size;
  p.side[2].out = a.v_pages;
  p.side[2].out_step = packed_row(a.v_bits);
  for (int i = 1; i < 3; ++i) p.side[i].slot_step = p.side[i].out_step * heads[i];
  if (a.num_tokens == 0 || total == 0) return cudaSuccess;
  p.vec = vec_ok(a.q, a.q_stride, size) && vec_ok(a.k, a.k_stride, size) && vec_ok(a.v, a.v_stride, size) &&
          vec_ok(a.q_out, a.q_out_stride, size) && vec_ok(a.k_out, a.k_out_stride, size);
  p.table_vec = reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0 && a.rot_dim % 8 == 0;
  // Runs of eight groups share a token's coefficients and hide the copies' latency; shorter ones where
  // they leave warps idle.
  const int64_t warps = (int64_t)sms * kAppendCtas * kAppendWarps;
  const int most = size == 2 ? kRunGroups : kRunGroups / 2;
  p.run = 1;
  while (2 * p.run <= most && a.num_tokens * total / (2 * warps) >= 2 * p.run) p.run *= 2;
  // Blocks of four tokens where a side's groups of one token are fewer than a run.
  p.block_tokens = p.run > 1 ? 4 : 1;
  const int64_t blocks = (a.num_tokens + p.block_tokens - 1) / p.block_tokens;
  p.blocks = (int)blocks;
  for (int i = 0; i < 3; ++i) {
    p.items[i] = (p.side[i].groups * p.block_tokens + p.run - 1) / p.run;
    p.side[i].first = p.block_items;
    p.block_items += p.items[i];
  }
  const int64_t ctas = (blocks * p.block_items + kAppendWarps - 1) / kAppendWarps;
  p.grid = (int)std::min<int64_t>(ctas, (int64_t)sms * kAppendCtas);
  // Whole blocks a turn, and every warp one part further at each: runs of packed rows take several
  // times those of dense ones, and each warp gets its share of all.  (More parts than warps: as they come.)
  p.warps = p.grid * kAppendWarps;
  if (p.warps >= p.block_items) {
    p.warps -= p.warps % p.block_items;
    p.step_block = p.warps / p.block_items;
    p.step_part = 1;
    p.carry = 0;
  } else {
    p.step_block = 0;
    p.step_part = p.warps;
    p.carry = 1;
  }
  const bool packed = a.k_pages || a.v_pages;
  switch (a.dtype) {
    case kF32: return packed ? launch_append_packed_f32(p, stream) : launch_append_f32(p, stream);
    case kF16: return packed ? launch_append_packed_f16(p, stream) : launch_append_f16(p, stream);
    case kBF16: return packed ? launch_append_packed_bf16(p, stream) : launch_append_bf16(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
