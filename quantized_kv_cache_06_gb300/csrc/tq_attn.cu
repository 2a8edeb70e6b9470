// Attention of query rows with a visible set of their own over packed TurboQuant pages
// (sm_103a): schedule, SIMT kernel, combine.
//
// TurboQuant docs: "vLLM Usage" (Runtime Dispatch: the cache plus mixed prefill/decode reads
// the packed cache) and "Architecture" (Diagnostic vs Serving Paths: keys consumed
// compressed, values accumulated from packed indices).  The pages know only the causal set;
// here row i of sequence s sees the union of an interval [p0, p1) (a bidirectional prefix),
// an interval [w0, w1) (the causal window, cut at its document) and single drafted tokens
// behind the context (the set bits of its mask):
//   x_t = f(scale nu_k <R q, c[idx_k]>) - slope |len - 1 - t|,  f(s) = cap tanh(s / cap)
//   out = R^T ( sum_t p_t nu_v c[idx_v] / sum_t p_t ),          p_t = exp(x_t - max)
//
// Work split.  The schedule cuts the rows into windows (runs of one sequence, up to the
// columns a CTA holds) and lists the 128-token tiles any row of a window sees; the list of
// all windows' tiles is cut into equal parts, and CTA (part, kv head) takes one of them.  So
// every CTA has as much to do whatever the lengths, tiles that no row sees (outside
// a window or a document) are never read, and the CTAs of one part read the interleaved rows
// of all heads at the same time, which keeps them in L2.  Where a CTA takes several windows, their
// starts and ends count too (a prompt's first windows have a tile or two each, single tokens among
// them many).  A window that lies in one part is finished there; the pieces of the others are merged
// by the combine, in tile order, so the result does not depend on timing.
//
// Three launches, the later two as programmatic dependents: the schedule (one CTA; for the
// tensor-core kernel the other CTAs rotate the queries, one warp a row, which costs the attention
// CTAs 130 instructions a column less), the attention, the combine (rotates back).
//
// The SIMT kernel below is the fp32 form: fp32 outputs, and head dims 16 and 32.  A warp owns four
// columns; lane = token for the scores, lane = coordinate for the values.  It is bound by the
// issue of its FMAs and shared-memory reads (64 tokens, 8 drafted, 16 / 2 heads: 41 us on the device,
// 40 of them here: the latency of a CTA's window of four rows, three steps of 32 tokens).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "tq_attn.h"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr float kAttnLog2e = 1.4426950408889634f;
constexpr int kSchedThreads = 1024;

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// Inclusive block scan (max or sum) of one int per thread; `tmp` holds 33 ints.
template <bool SUM>
__device__ __forceinline__ int block_scan(int v, int* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFullMask, v, o);
    if (lane >= o) v = SUM ? v + u : max(v, u);
  }
  __syncthreads();
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = tmp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFullMask, w, o);
      if (lane >= o) w = SUM ? w + u : max(w, u);
    }
    tmp[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v = SUM ? v + tmp[warp - 1] : max(v, tmp[warp - 1]);
  return v;
}

// CTA 0: windows, their visible tiles and the tile prefix.  The others (tensor-core kernel; D its
// head dim, else 0): the queries rotated, one warp per (row, q head).
template <int D>
__global__ void __launch_bounds__(kSchedThreads) attn_schedule_kernel(AttnArgs a, AttnWork w) {
  if constexpr (D > 0) {
    if (blockIdx.x > 0) {
      constexpr int E = D / 32;
      const int lane = threadIdx.x & 31;
      const int64_t id = (int64_t)(blockIdx.x - 1) * (kSchedThreads / 32) + (threadIdx.x >> 5);
      pdl_launch();
      if (id >= (int64_t)a.num_rows * a.num_q_heads) return;
      float v[E];
      const int64_t at = id * D + lane * E;
      if (reinterpret_cast<uintptr_t>(a.q) % 16 != 0) {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = load_as_f32(a.q, at + i, a.q_dtype);
      } else if (a.q_dtype == kF32) {
        load_chunk<float, E>(static_cast<const float*>(a.q) + at, v);
      } else if (a.q_dtype == kF16) {
        load_chunk<__half, E>(static_cast<const __half*>(a.q) + at, v);
      } else {
        load_chunk<__nv_bfloat16, E>(static_cast<const __nv_bfloat16*>(a.q) + at, v);
      }
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] *= w.q_mul * __ldg(a.signs + lane * E + i);
      fwht_warp<E>(v);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        w.q_rot[at + i] = v[i];
        top = fmaxf(top, fabsf(v[i]));
      }
      top = warp_max(top);
      if (lane == 0) w.q_top[id] = top;
      return;
    }
  }
  __shared__ int tmp[33];
  __shared__ int carry_start, carry_win, carry_places, carry_tiles;
  const int tid = threadIdx.x, T = a.num_rows;
  const int last = kSchedThreads - 1;
  if (tid == 0) {
    carry_start = -1;
    carry_win = 0;
    carry_places = 0;
    carry_tiles = 0;
    if (a.status) *a.status = kOk;
  }
  pdl_launch();
  __syncthreads();
  // rows -> windows
  for (int base = 0; base < T; base += kSchedThreads) {
    const int i = base + tid;
    const bool run = i < T && (i == 0 || a.q_seq[i] != a.q_seq[i - 1]);
    const int start = max(block_scan<false>(run ? i : -1, tmp), carry_start);
    const bool first = i < T && (i - start) % w.rows_per_window == 0;
    const int idx = block_scan<true>(first ? 1 : 0, tmp) + carry_win - 1;
    if (i < T) w.row_window[i] = idx;
    if (first) {
      AttnWindow win{};
      win.row0 = i;
      win.p_lo = win.w_lo = 0x7fffffff;
      w.win[idx] = win;
    }
    __syncthreads();
    if (tid == last) {
      carry_start = start;
      carry_win = idx + 1;
    }
    __syncthreads();
  }
  const int nwin = carry_win;
  // Windows count in the parts where there are many (with one or two a part, every part has its own
  // start and end anyway): 4 chunks of 1000 rows 590 -> 420 us; 255 single tokens and a prompt of
  // 1700 rows 969 -> 759, the prompt alone 245 -> 162.
  const int lead = nwin > 2 * w.parts ? w.lead : 0;
  // rows -> the token ranges of their windows (ranges meet in L2: the windows of a row chunk
  // may be shared by threads of several warps)
  for (int i = tid; i < T; i += kSchedThreads) {
    const RowView v = row_view(a, i);
    if (v.bad && a.status) atomicMax(a.status, (int32_t)kInvalidArg);
    AttnWindow* win = w.win + w.row_window[i];
    atomicMax(&win->nrows, i - win->row0 + 1);
    if (i == win->row0) win->seq = v.seq;
    if (v.p1 > v.p0) {
      atomicMin(&win->p_lo, v.p0);
      atomicMax(&win->p_hi, v.p1);
    }
    const int hi = v.bits > 0 ? max(v.w1, v.base + v.bits) : v.w1;
    if (hi > 0) {
      atomicMin(&win->w_lo, v.w1 > v.w0 ? v.w0 : v.base);
      atomicMax(&win->w_hi, hi);
    }
  }
  __threadfence();
  __syncthreads();
  // windows -> tiles
  for (int base = 0; base < nwin; base += kSchedThreads) {
    const int k = base + tid;
    int n = 0;
    if (k < nwin) {
      AttnWindow* win = w.win + k;
      const int p_lo = __ldcg(&win->p_lo), p_hi = __ldcg(&win->p_hi);
      const int w_lo = __ldcg(&win->w_lo), w_hi = __ldcg(&win->w_hi);
      int a0 = 0, a1 = 0, b0 = 0, b1 = 0;
      if (p_hi > 0) a0 = p_lo / kAttnTile, a1 = (p_hi + kAttnTile - 1) / kAttnTile;
      if (w_hi > 0) b0 = w_lo / kAttnTile, b1 = (w_hi + kAttnTile - 1) / kAttnTile;
      if (a1 > a0 && b1 > b0 && a1 >= b0 && b1 >= a0) {  // they touch: one range
        b0 = min(a0, b0);
        b1 = max(a1, b1);
        a0 = a1 = 0;
      }
      win->tA0 = a0;
      win->nA = a1 - a0;
      win->tB0 = b0;
      win->nB = b1 - b0;
      n = win->nA + win->nB;
    }
    const int incl = block_scan<true>(n > 0 ? n + lead : 0, tmp) + carry_places;
    const int tiles = lead > 0 ? block_scan<true>(n, tmp) + carry_tiles : incl;
    if (k < nwin) {
      w.win[k].tile_base = incl - n;
      w.win[k].tiles_before = tiles - n;
    }
    __syncthreads();
    if (tid == last) {
      carry_places = incl;
      carry_tiles = tiles;
    }
    __syncthreads();
  }
  if (tid == 0) {
    w.head->num_windows = nwin;
    w.head->total = carry_places;
    w.head->lead = lead;
  }
}

// ---------------------------------------------------------------- SIMT attention

constexpr int kSimtWarps = 8;
constexpr int kSimtPer = 4;  // columns per warp
constexpr int kSimtCols = kSimtWarps * kSimtPer;
constexpr int kSimtTok = 32;  // tokens per step

template <int D>
constexpr int simt_smem_bytes() {
  return (kSimtCols * D + kSimtTok * (D + 1) + kSimtTok * D + 2 * kSimtTok + 64) * 4 + kSimtCols * (int)sizeof(RowView);
}

// Walsh-Hadamard transform of N vectors of D values in shared memory by one warp.
template <int D, int N = 1>
__device__ __forceinline__ void fwht_shared(float* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 1; h < D; h <<= 1) {
    __syncwarp();
#pragma unroll
    for (int p = lane; p < N * D / 2; p += 32) {  // (pairs of one vector follow those of the one before)
      const int i = (p / h) * 2 * h + p % h;
      const float x = v[i], y = v[i + h];
      v[i] = x + y;
      v[i + h] = x - y;
    }
  }
  __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kSimtWarps * 32) attn_simt_kernel(AttnArgs a, AttnWork w) {
  constexpr int E = (D + 31) / 32;
  extern __shared__ __align__(16) float smem[];
  float* q_s = smem;                       // [cols][D], rotated, scale folded in
  float* k_s = q_s + kSimtCols * D;        // [32][D + 1]
  float* v_s = k_s + kSimtTok * (D + 1);   // [32][D]
  float* kn_s = v_s + kSimtTok * D;        // key norms (NaN never read: ok_s)
  float* vn_s = kn_s + kSimtTok;
  float* cb_s = vn_s + kSimtTok;           // K and V centroids, 32 each
  RowView* view = reinterpret_cast<RowView*>(cb_s + 64);
  __shared__ int ok_s[kSimtTok];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.num_kv_heads, G = a.num_q_heads / H;
  const int h = blockIdx.x % H, part = blockIdx.x / H;
  const int bs = a.block_size;
  const int rbk = D * a.k_bits / 8 + 4, rbv = D * a.v_bits / 8 + 4;
  if (tid < 32) cb_s[tid] = tid < (1 << a.k_bits) ? a.k_centroids[tid] : 0.f;
  else if (tid < 64) cb_s[tid] = tid - 32 < (1 << a.v_bits) ? a.v_centroids[tid - 32] : 0.f;
  const float scale = a.scale > 0.f ? a.scale : 1.0f / sqrtf((float)D);
  const float qmul = scale / sqrtf((float)D);
  pdl_launch();
  pdl_wait();
  const int total = w.head->total;
  const int parts = live_parts(w, total);
  if (part >= parts) return;
  const int g0 = part_begin(total, part, parts), g1 = part_begin(total, part + 1, parts);

  for (int g = g0, wi = window_of(w, g0); g < g1; ++wi) {
    const AttnWindow win = w.win[wi];
    const int n = win.nA + win.nB;
    const int t_first = g - win.tile_base, t_last = min(n, t_first + (g1 - g));
    g += max(0, t_last - t_first);
    if (t_first >= t_last) continue;
    const int cols = win.nrows * G;
    __syncthreads();
    // rotated queries, the four columns' loads and stages together
    constexpr int R = (D + 31) / 32;
    float qv[kSimtPer][R];
#pragma unroll
    for (int m = 0; m < kSimtPer; ++m) {
      const int col = min(warp * kSimtPer + m, cols - 1);
      const int64_t at = ((int64_t)(win.row0 + col / G) * a.num_q_heads + h * G + col % G) * D;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (D >= 32 || lane < D) qv[m][i] = load_as_f32(a.q, at + lane + 32 * i, a.q_dtype) * a.signs[lane + 32 * i] * qmul;
    }
    if (lane < kSimtPer && warp * kSimtPer + lane < cols)
      view[warp * kSimtPer + lane] = row_view(a, win.row0 + (warp * kSimtPer + lane) / G);
#pragma unroll
    for (int m = 0; m < kSimtPer; ++m)
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (D >= 32 || lane < D) q_s[(warp * kSimtPer + m) * D + lane + 32 * i] = qv[m][i];
    fwht_shared<D, kSimtPer>(q_s + warp * kSimtPer * D);
    __syncwarp();
    float o[kSimtPer][E], mx[kSimtPer], sum[kSimtPer];
#pragma unroll
    for (int m = 0; m < kSimtPer; ++m) {
      mx[m] = -INFINITY;
      sum[m] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[m][e] = 0.f;
    }
    const int32_t* table = a.block_table + (int64_t)win.seq * a.max_blocks_per_seq;
    const int cap = (int)min((int64_t)a.max_blocks_per_seq * bs, (int64_t)0x7fffff00);
    const int n_sub = (t_last - t_first) * (kAttnTile / kSimtTok);
    for (int sub = 0; sub < n_sub; ++sub) {
      const int tile = t_first + sub / (kAttnTile / kSimtTok);
      const int t0 = (tile < win.nA ? win.tA0 + tile : win.tB0 + tile - win.nA) * kAttnTile +
                     sub % (kAttnTile / kSimtTok) * kSimtTok;
      const int hi = max(win.p_hi, win.w_hi);
      if (t0 >= hi) continue;
      __syncthreads();
      // dequantise 32 tokens; a task is a run of coordinates of one row (32 of them in whole words;
      // D = 16: the row, whose bytes may start anywhere)
      constexpr int kRun = D < 32 ? D : 32, kRuns = D / kRun;
      for (int i = tid; i < 2 * kSimtTok * kRuns; i += kSimtWarps * 32) {
        const int comp = i / (kSimtTok * kRuns), t = i / kRuns % kSimtTok, run = i % kRuns;
        const int tok = t0 + t;
        const bool there = tok < hi && tok < cap;
        const int block = there ? table[tok / bs] : -1;
        const bool ok = block >= 0 && block < a.num_blocks;
        const int bits = comp ? a.v_bits : a.k_bits, rb = comp ? rbv : rbk;
        const uint8_t* row = (comp ? a.v_pages : a.k_pages) + (((int64_t)max(block, 0) * bs + tok % bs) * H + h) * rb;
        uint32_t words[6] = {0, 0, 0, 0, 0, 0}, norm = 0;
        if (ok) {
          if constexpr (D >= 32) {
#pragma unroll
            for (int k = 0; k < 5; ++k)
              if (k < bits) words[k] = __ldg(reinterpret_cast<const uint32_t*>(row) + run * bits + k);
            norm = __ldg(reinterpret_cast<const uint32_t*>(row) + (rb - 4) / 4);
          } else {
#pragma unroll
            for (int k = 0; k < 10; ++k)
              if (k < 2 * bits) words[k >> 2] |= (uint32_t)row[k] << (8 * (k & 3));
#pragma unroll
            for (int k = 0; k < 4; ++k) norm |= (uint32_t)row[rb - 4 + k] << (8 * k);
          }
        }
        if (run == 0) {
          (comp ? vn_s : kn_s)[t] = __uint_as_float(norm);
          if (comp == 0) ok_s[t] = ok;
        }
        float* to = comp ? v_s + t * D + run * kRun : k_s + t * (D + 1) + run * kRun;
        auto expand = [&](auto tag) {
          constexpr int B = decltype(tag)::value;
#pragma unroll
          for (int j = 0; j < kRun; ++j) {
            const int w0 = j * B / 32, sh = j * B % 32;
            const uint32_t f = sh + B <= 32 ? words[w0] >> sh : __funnelshift_r(words[w0], words[w0 + 1], sh);
            to[j] = cb_s[comp * 32 + (f & ((1u << B) - 1u))];
          }
        };
        if (bits == 4) expand(std::integral_constant<int, 4>{});
        else if (bits == 3) expand(std::integral_constant<int, 3>{});
        else if (bits == 2) expand(std::integral_constant<int, 2>{});
        else expand(std::integral_constant<int, 5>{});
      }
      __syncthreads();
      const int tok = t0 + lane;
      const bool ok = ok_s[lane] != 0;
      // the warp's four columns together: a key or value element read once serves all of them
      const int first_col = warp * kSimtPer;
      if (first_col >= cols) continue;  // (no barrier follows before the next step's)
      float dot[kSimtPer];
#pragma unroll
      for (int m = 0; m < kSimtPer; ++m) dot[m] = 0.f;
      const float* key = k_s + lane * (D + 1);
#pragma unroll 4
      for (int j = 0; j < D; j += 4) {
        const float x0 = key[j], x1 = key[j + 1], x2 = key[j + 2], x3 = key[j + 3];
#pragma unroll
        for (int m = 0; m < kSimtPer; ++m) {
          const float4 qq = *reinterpret_cast<const float4*>(q_s + (first_col + m) * D + j);
          dot[m] = fmaf(qq.x, x0, dot[m]);
          dot[m] = fmaf(qq.y, x1, dot[m]);
          dot[m] = fmaf(qq.z, x2, dot[m]);
          dot[m] = fmaf(qq.w, x3, dot[m]);
        }
      }
      float pv[kSimtPer];
      bool lost = false;  // a row sees this token, but its block lies outside the pages
#pragma unroll
      for (int m = 0; m < kSimtPer; ++m) {
        const int col = first_col + m;
        pv[m] = 0.f;
        if (col >= cols) continue;
        const int row = win.row0 + col / G;
        const bool asks = row_sees(view[col], a.mask ? a.mask + (int64_t)row * a.mask_words : nullptr, tok);
        const bool see = asks && ok;
        lost |= asks && !ok;
        float x = -INFINITY;
        if (see) {
          x = dot[m] * kn_s[lane];
          if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
          if (a.alibi) x -= a.alibi[h * G + col % G] * fabsf((float)(view[col].base - tok));
          x *= kAttnLog2e;
        }
        if (!__any_sync(kFullMask, see)) continue;
        const float top = fmaxf(mx[m], warp_max(x));
        // every visible score -inf (an infinite norm): weights of an empty row, not NaN
        const float ref = top == -INFINITY ? 0.f : top;
        const float p = exp2f(x - ref);
        const float corr = exp2f(mx[m] - ref);
        mx[m] = top;
        sum[m] = sum[m] * corr + warp_sum(p);
#pragma unroll
        for (int e = 0; e < E; ++e) o[m][e] *= corr;
        pv[m] = p != 0.f ? p * vn_s[lane] : 0.f;
      }
      if (lost && a.status) atomicMax(a.status, (int32_t)kBlockOutOfRange);
#pragma unroll 4
      for (int t = 0; t < kSimtTok; ++t) {
        float val[E];
#pragma unroll
        for (int e = 0; e < E; ++e) val[e] = v_s[t * D + (D >= 32 ? lane + 32 * e : lane & (D - 1))];
#pragma unroll
        for (int m = 0; m < kSimtPer; ++m) {
          const float pt = __shfl_sync(kFullMask, pv[m], t);
#pragma unroll
          for (int e = 0; e < E; ++e) o[m][e] = fmaf(pt, val[e], o[m][e]);
        }
      }
    }
    // results: the whole window here, or a piece of it
    const bool whole = t_first == 0 && t_last == n;
#pragma unroll
    for (int m = 0; m < kSimtPer; ++m) {
      const int col = warp * kSimtPer + m;
      if (col >= cols) continue;
      if (whole) {
        float* buf = q_s + col * D;  // the query is no longer needed
        const float inv = sum[m] != 0.f ? 1.f / (sum[m] * sqrtf((float)D)) : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (D >= 32 || lane < D) buf[lane + 32 * e] = o[m][e] * inv;
        fwht_shared<D>(buf);
        const int64_t at = ((int64_t)(win.row0 + col / G) * a.num_q_heads + h * G + col % G) * D;
        for (int j = lane; j < D; j += 32) store_from_f32(a.out, at + j, a.out_dtype, buf[j] * a.signs[j]);
      } else {
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (t_first == 0 ? 1 : 0)) * w.cols + col;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (D >= 32 || lane < D) w.acc[slot * D + lane + 32 * e] = o[m][e];
        if (lane == 0) {
          w.ml[2 * slot] = mx[m];
          w.ml[2 * slot + 1] = sum[m];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- combine

constexpr int kCombineWarps = 8;

// One warp per (row, q head): merges the pieces of a window that several parts hold, and
// zeroes the rows that see nothing.  Rows of the tensor-core kernel are rotated back here, those
// of the SIMT kernel that one CTA finished are done.
template <int D, bool TC>
__global__ void __launch_bounds__(kCombineWarps * 32) attn_combine_kernel(AttnArgs a, AttnWork w) {
  constexpr int E = (D + 31) / 32;
  __shared__ float buf_s[kCombineWarps][D];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kCombineWarps + warp;
  if (id >= (int64_t)a.num_rows * a.num_q_heads) return;
  const int row = (int)(id / a.num_q_heads), qh = (int)(id % a.num_q_heads);
  const int H = a.num_kv_heads, G = a.num_q_heads / H, h = qh / G;
  const AttnWindow* win = w.win + w.row_window[row];
  const int n = win->nA + win->nB;
  if (n == 0) {
    for (int j = lane; j < D; j += 32) store_from_f32(a.out, id * D + j, a.out_dtype, 0.f);
    return;
  }
  const int total = w.head->total, base = win->tile_base;
  const int parts = live_parts(w, total);
  const int c0 = part_of(total, base, parts), c1 = part_of(total, base + n - 1, parts);
  if (c0 == c1) {
    if constexpr (TC) {
      float v[E];
      load_floats<E>(w.q_rot + id * D + lane * E, v);
      fwht_warp<E>(v);
#pragma unroll
      for (int i = 0; i < E; ++i)
        store_from_f32(a.out, id * D + lane * E + i, a.out_dtype, v[i] * __ldg(a.signs + lane * E + i));
    }
    return;
  }
  const int col = (row - win->row0) * G + qh % G;
  auto slot_of = [&](int c) -> int64_t { return (((int64_t)c * H + h) * 2 + (c == c0 ? 1 : 0)) * w.cols + col; };
  float top = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, w.ml[2 * slot_of(c)]);
  top = warp_max(top);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const int64_t s = slot_of(c);
    const float f = exp2f(w.ml[2 * s] - ref);
    sum = fmaf(f, w.ml[2 * s + 1], sum);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (D >= 32 || lane < D) o[e] = fmaf(f, w.acc[s * D + lane + 32 * e], o[e]);
  }
  // (the tensor-core kernel's pieces hold 1 / sqrt(D) already)
  const float inv = sum != 0.f ? (TC ? 1.f / sum : 1.f / (sum * sqrtf((float)D))) : 0.f;
  float* buf = buf_s[warp];
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (D >= 32 || lane < D) buf[lane + 32 * e] = o[e] * inv;
  fwht_shared<D>(buf);
  for (int j = lane; j < D; j += 32) store_from_f32(a.out, id * D + j, a.out_dtype, buf[j] * a.signs[j]);
}

// A launch that may start before the kernel ahead of it on the stream has finished (its
// griddepcontrol.wait waits for that).
template <typename K>
cudaError_t launch_after(K kern, int grid, int block, size_t smem, cudaStream_t stream, const AttnArgs& a,
                         const AttnWork& w) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, a, w);
  if (err == cudaSuccess) count_launches(1);
  return err;
}

template <int D>
cudaError_t launch_simt(const AttnArgs& a, const AttnWork& w, cudaStream_t stream) {
  constexpr int smem = simt_smem_bytes<D>();
  const cudaError_t err = cudaFuncSetAttribute(attn_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  return launch_after(attn_simt_kernel<D>, w.parts * a.num_kv_heads, kSimtWarps * 32, smem, stream, a, w);
}

template <int D, bool TC = false>
cudaError_t launch_combine(const AttnArgs& a, const AttnWork& w, cudaStream_t stream) {
  const int64_t warps = (int64_t)a.num_rows * a.num_q_heads;
  const int64_t grid = (warps + kCombineWarps - 1) / kCombineWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_after(attn_combine_kernel<D, TC>, (int)grid, kCombineWarps * 32, 0, stream, a, w);
}

}  // namespace

AttnPlan plan_attn(const AttnArgs& a, int num_sms) {
  AttnPlan p{};
  p.tc = attn_tc_supported(a);
  p.cols = p.tc ? attn_tc_cols(a) : kSimtCols;
  // tensor cores: one CTA (all of TMEM) an SM; SIMT: two, which hide each other's barriers
  const int ctas = p.tc ? num_sms : 2 * num_sms;
  p.parts = std::max(1, ctas / std::max(1, a.num_kv_heads));
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)std::max(0, a.num_rows);
  p.off_windows = 256;
  p.off_row_window = up(p.off_windows + rows * sizeof(AttnWindow));
  p.off_acc = up(p.off_row_window + rows * sizeof(int));
  const size_t slots = (size_t)p.parts * a.num_kv_heads * 2 * p.cols;
  p.off_ml = up(p.off_acc + slots * a.head_dim * sizeof(float));
  p.off_rot = up(p.off_ml + slots * 2 * sizeof(float));
  const size_t qs = p.tc ? rows * a.num_q_heads : 0;
  p.off_top = up(p.off_rot + qs * a.head_dim * sizeof(float));
  p.workspace_bytes = up(p.off_top + qs * sizeof(float));
  return p;
}

cudaError_t launch_attn(const AttnArgs& a, const AttnPlan& p, cudaStream_t stream) {
  if (a.num_rows == 0) return a.status ? cudaMemsetAsync(a.status, 0, sizeof(int32_t), stream) : cudaSuccess;
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  AttnWork w;
  w.head = reinterpret_cast<AttnHeader*>(ws);
  w.win = reinterpret_cast<AttnWindow*>(ws + p.off_windows);
  w.row_window = reinterpret_cast<int*>(ws + p.off_row_window);
  w.acc = reinterpret_cast<float*>(ws + p.off_acc);
  w.ml = reinterpret_cast<float*>(ws + p.off_ml);
  w.cols = p.cols;
  w.lead = p.tc ? attn_tc_lead(p.cols) : 0;  // (the SIMT kernel's windows start at no cost beside their tiles')
  w.parts = p.parts;
  w.rows_per_window = p.cols / (a.num_q_heads / a.num_kv_heads);
  w.q_rot = reinterpret_cast<float*>(ws + p.off_rot);
  w.q_top = reinterpret_cast<float*>(ws + p.off_top);
  if (p.tc) {
    // scale, log2 e, the rotation's 1 / sqrt(D) and the keys' alpha in one factor; scores with an
    // ordinary cap are taken as 2 log2(e) s / cap, whose power of two gives the tanh
    const float scale = a.scale > 0.f ? a.scale : 1.0f / sqrtf((float)a.head_dim);
    w.q_mul = (cap_folded(a.softcap) ? 2.f * scale / a.softcap : scale) * kAttnLog2e / (sqrtf((float)a.head_dim) * a.k_alpha);
    const int64_t ctas = ((int64_t)a.num_rows * a.num_q_heads + kSchedThreads / 32 - 1) / (kSchedThreads / 32) + 1;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (a.head_dim == 64) attn_schedule_kernel<64><<<(int)ctas, kSchedThreads, 0, stream>>>(a, w);
    else if (a.head_dim == 128) attn_schedule_kernel<128><<<(int)ctas, kSchedThreads, 0, stream>>>(a, w);
    else attn_schedule_kernel<256><<<(int)ctas, kSchedThreads, 0, stream>>>(a, w);
  } else {
    attn_schedule_kernel<0><<<1, kSchedThreads, 0, stream>>>(a, w);
  }
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  count_launches(1);
  if (p.tc) {
    err = launch_attn_tc(a, w, stream);
    if (err != cudaSuccess) return err;
    if (a.head_dim == 64) return launch_combine<64, true>(a, w, stream);
    if (a.head_dim == 128) return launch_combine<128, true>(a, w, stream);
    return launch_combine<256, true>(a, w, stream);
  }
  switch (a.head_dim) {
    case 16: err = launch_simt<16>(a, w, stream); break;
    case 32: err = launch_simt<32>(a, w, stream); break;
    case 64: err = launch_simt<64>(a, w, stream); break;
    case 128: err = launch_simt<128>(a, w, stream); break;
    case 256: err = launch_simt<256>(a, w, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (err != cudaSuccess) return err;
  switch (a.head_dim) {
    case 16: return launch_combine<16>(a, w, stream);
    case 32: return launch_combine<32>(a, w, stream);
    case 64: return launch_combine<64>(a, w, stream);
    case 128: return launch_combine<128>(a, w, stream);
    default: return launch_combine<256>(a, w, stream);
  }
}

}  // namespace tq
