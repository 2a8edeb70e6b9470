// Attention of query rows with a visible set of their own over packed pages (tq_attn.cu,
// tq_attn_tc.cu): drafted-token trees, and prefill / decode with capped or biased scores.
// Internal declarations.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tq {

struct AttnArgs {
  const void* q;
  int q_dtype;
  int num_rows;
  int num_q_heads;
  int num_kv_heads;
  int head_dim;
  const uint8_t* k_pages;
  int k_bits;
  const uint8_t* v_pages;
  int v_bits;
  int64_t num_blocks;
  int block_size;
  const int32_t* block_table;
  int num_seqs;
  int max_blocks_per_seq;
  const int32_t* q_seq;
  // biased prefill / decode (null q_len: tree)
  const int32_t* q_len;
  const int32_t* prefix_lens;  // may be null
  const int32_t* doc_starts;   // may be null
  int window;                  // 0: none
  const float* alibi;          // slopes per q head, may be null
  // tree
  const int32_t* ctx_lens;
  const uint32_t* mask;  // [num_rows][mask_words]
  int mask_words;
  float softcap;  // 0: none
  float scale;    // <= 0: 1 / sqrt(head_dim)
  const float* signs;
  const float* k_centroids;
  const float* v_centroids;
  void* out;
  int out_dtype;
  void* workspace;
  int32_t* status;  // may be null
  float k_alpha;    // fp16 scales of the centroids (tensor-core kernel)
  float v_alpha;
};

constexpr int kAttnTile = 128;  // tokens per tile of the schedule

// Whether the tensor-core kernel takes a cap as cap - 2 cap / (1 + e^(2 s / cap)), with 2 / cap in
// the queries' factor: two instructions a score, off by 1.6e-7 of the cap (4e-5 at 256, a sixth
// of the rounding of an fp16 weight; 0.09 at 1e6).  A cap below 2^-10 could take the queries' factor
// out of range.  The others get the scores as they are and a form that holds anywhere.
inline __host__ __device__ bool cap_folded(float c) { return c >= 0.0009765625f && c <= 256.f; }

// A run of query rows of one sequence that a CTA takes together, and the tiles they see:
// nA tiles from tA0 (the prefix interval), then nB tiles from tB0.  The parts are cut from a line
// of places, one a tile and `lead` before the first tile of each window, for its start and end.
struct AttnWindow {
  int row0, nrows, seq;
  int tA0, nA, tB0, nB;
  int tile_base;     // place of the first tile
  int tiles_before;  // tiles of all windows before
  // reductions over the rows, in tokens (schedule kernel)
  int p_lo, p_hi, w_lo, w_hi;
};

// Workspace: header, windows, window of each row, partial results of the CTAs.
struct AttnHeader {
  int num_windows;
  int total;  // places
  int lead;   // places before a window's first tile
  int pad;
};

struct AttnPlan {
  bool tc;          // tensor-core kernel (else the SIMT kernel)
  int cols;         // (row, q head of the group) columns per CTA
  int parts;        // partitions of the tile list; grid = parts * kv heads
  size_t off_windows, off_row_window, off_acc, off_ml, off_rot, off_top;
  size_t workspace_bytes;
};

AttnPlan plan_attn(const AttnArgs& a, int num_sms);
// Enqueues status reset, schedule, attention and combine.
cudaError_t launch_attn(const AttnArgs& a, const AttnPlan& p, cudaStream_t stream);

// Device view of the workspace.
struct AttnWork {
  AttnHeader* head;
  AttnWindow* win;
  int* row_window;
  float* acc;  // [grid][2][cols][D]: piece 0 continues a window, piece 1 starts one that goes on
  float* ml;   // [grid][2][cols][2]
  // tensor-core kernel: rotated queries R q * q_mul and their largest coordinates, [rows][q heads];
  // the rows of windows that one CTA finishes come back in their place, in rotated space
  float* q_rot;
  float* q_top;
  float q_mul;
  int cols, parts, rows_per_window;
  int lead;  // where windows are many: places a window's start and end are worth
};
constexpr int kAttnMaxLead = 8;

bool attn_tc_supported(const AttnArgs& a);
int attn_tc_cols(const AttnArgs& a);
int attn_tc_lead(int cols);
cudaError_t launch_attn_tc(const AttnArgs& a, const AttnWork& w, cudaStream_t stream);

#ifdef __CUDACC__
// The tokens a query row sees: [p0, p1), [w0, w1) and base + j for the set bits j of its mask
// (bits: the highest set bit + 1; without a mask base is the row's position).
struct RowSees {
  int p0, p1, w0, w1, base, bits;
};
struct RowView : RowSees {
  int seq;  // -1: none
  bool bad;
};

__device__ __forceinline__ RowView row_view(const AttnArgs& a, int i) {
  RowView v{};
  v.seq = -1;
  const int seq = a.q_seq[i];
  if (seq < 0 || seq >= a.num_seqs) {
    v.bad = seq != -1;  // -1 is a padding row
    return v;
  }
  v.seq = seq;
  const int cap = (int)min((int64_t)a.max_blocks_per_seq * a.block_size, (int64_t)0x7fffff00);
  if (a.q_len) {
    int len = a.q_len[i];
    v.bad = len < 0 || len > cap;
    len = min(max(len, 0), cap);
    v.base = len - 1;
    const int doc = a.doc_starts ? max(a.doc_starts[i], 0) : 0;
    v.w1 = len;
    v.w0 = max(a.window > 0 ? max(0, len - a.window) : 0, doc);
    if (a.prefix_lens) {
      const int pre = a.prefix_lens[seq];
      v.bad |= pre < 0 || pre > cap;
      v.p0 = doc;
      v.p1 = min(max(pre, 0), cap);
    }
  } else {
    const int ctx = a.ctx_lens[seq];
    v.bad = ctx < 0 || ctx > cap;
    v.w1 = min(max(ctx, 0), cap);
    v.base = v.w1;
    const uint32_t* m = a.mask + (int64_t)i * a.mask_words;
    for (int k = a.mask_words - 1; k >= 0; --k) {
      const uint32_t w = m[k];
      if (w) {
        v.bits = 32 * k + 32 - __clz((int)w);
        break;
      }
    }
    if (v.base + v.bits > cap) {
      v.bad = true;
      v.bits = cap - v.base;
    }
  }
  if (v.p1 <= v.p0) v.p0 = v.p1 = 0;
  if (v.w1 <= v.w0) v.w0 = v.w1 = 0;
  return v;
}

// Whether a row sees token t.
__device__ __forceinline__ bool row_sees(const RowSees& v, const uint32_t* mask, int t) {
  bool s = (t >= v.w0 && t < v.w1) || (t >= v.p0 && t < v.p1);
  const int j = t - v.base;
  if (v.bits > 0 && j >= 0 && j < v.bits) s |= (mask[j >> 5] >> (j & 31)) & 1u;
  return s;
}

// Parts that hold places: with fewer places than parts, one each (the combine walks every part
// between a window's first tile and its last, so none of them may be empty).
__device__ __forceinline__ int live_parts(const AttnWork& w, int total) { return min(w.parts, total); }
// E consecutive floats another kernel of the call wrote (aligned to 4 E bytes; plain loads: the
// memory is written again within the call).
template <int E>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[E]) {
  if constexpr (E == 2) {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x;
    v[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  }
}
// The first place of partition p of `parts` over `total` places.
__device__ __forceinline__ int part_begin(int total, int p, int parts) { return (int)((int64_t)total * p / parts); }
// The partition that holds place g.
__device__ __forceinline__ int part_of(int total, int g, int parts) {
  return (int)(((int64_t)(g + 1) * parts - 1) / total);
}
// The window that holds place g (num_windows > 0, 0 <= g <= total): the last one whose tiles start at
// or before it, or the first.
__device__ __forceinline__ int window_of(const AttnWork& w, int g) {
  int lo = 0, hi = w.head->num_windows;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (w.win[mid].tile_base <= g) lo = mid;
    else hi = mid;
  }
  return lo;
}
#endif

}  // namespace tq
