// Verification of drafted tokens against the target's distribution, from given random numbers,
// sm_103a.
//
// TurboQuant docs: "vLLM Usage" and "Architecture" leave the engine's sampling to the host
// framework; this call stands between the attention of a drafted tree and the commit of the
// accepted rows.
//
// With p = softmax(logits / temperature) of a node's row and u its random number, a token drawn
// from weights w_0, w_1, ... is the first i whose running sum passes u times the whole sum.
//   * No draft probabilities (drafted tokens are fixed): a token is drawn from p at every row; the
//     walk goes on to the child that carries it.
//   * Draft probabilities q (children drawn from q): child x is kept when u q(x) < r(x) with
//     r = max(a p - b q, 0), at first (a, b) = (1, 0).  A refusal subtracts q once more:
//     Z = sum max(a p - (b + 1) q, 0), (a, b) <- (a, b + 1) / Z, as max(max(x, 0) - q, 0) =
//     max(x - q, 0) for q >= 0.  All refused: a token from r.
//
// Weights are 2^((x - m) c), c = log2(e) / temperature in two parts, m the row's largest logit.
// Sums that decide which token is drawn are 64-bit integers (fixed point), so they do not depend
// on any order, and their error is that of the weights (about 1e-7 each, independent).
//
// Two launches.  1. Every warp takes consecutive pieces of 1024 logits, the next one's under way, and
// leaves each piece's largest logit and its sum of weights (or its first largest, where the temperature
// is 0).  2. One CTA takes a sequence (a cluster with draft probabilities, of which one CTA decides and
// all share the passes over a row): rows' sums from the pieces, then only the pieces that hold a drawn
// token are read again, and with draft probabilities the rows of refused tokens once per refusal.
//
// Bound (GB300): of the first launch the logits' bytes (256 trees, 1153 rows of 131072 bf16, 303 MB
// read once: 55 us, 82 % of the copy bandwidth; 253 warp instructions a piece, 64 % of the issue slots,
// the exponentials' pipe as busy); of the second latency (10 us behind it; with draft probabilities 20 us,
// of which the refused rows' 50 MB of logits and probabilities take 8).  Whole calls: 64 us, and 37 us for
// 64 chains of 5 rows.  Measured and not kept: pieces dealt out one by one, a row's temperature looked up
// for each (256 trees 131 us); every CTA of a cluster walking for itself (the same time, and barriers that
// would hang on buffers that change under the call).
//
// Rows may start at any multiple of their element's size: pieces are laid out from the aligned
// address at or before the row's start, so all but a row's first and last 16 bytes are loaded 16
// bytes at a time.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_verify.h"

namespace cg = cooperative_groups;

namespace tq {
namespace {

constexpr int kPiece = 1024;      // logits of a piece
constexpr int kStatWarps = 8;
constexpr int kPickWarps = 16;    // most warps of a sequence's CTA
constexpr int kDraftWarps = 8;
constexpr int kDraftCtas = 8;     // CTAs of a sequence's cluster (with draft probabilities)

using u64 = unsigned long long;

struct RowInfo {
  float max, inv;  // largest logit; 1 / sum of weights
  int32_t pick;    // token drawn (no draft probabilities, or temperature 0); -1: no distribution
  int32_t pad;
};

struct VerifyWork {
  float2* stats;   // [rows][pieces]: largest logit, sum of weights (its bits: first largest)
  RowInfo* rows;   // [rows]
  float2* pq;      // [rows]: p and q of the row's token under its parent
  u64* rest;       // [seqs][pieces]: sums of max(a p - b q, 0)
  int pieces;
};

// pieces of a row that starts `shift` elements behind an aligned address
inline int pieces_of(int vocab, int shift) { return (int)(((int64_t)vocab + shift + kPiece - 1) / kPiece); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Largest of a warp's numbers, none of them NaN.
__device__ __forceinline__ float largest_of_warp(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Scale of a row: c = log2(e) / temperature in two parts, and the difference below which a
// weight is zero (NaN differences, of NaN logits or where all are -inf, go there too).
struct Scale {
  float hi, lo, least;
};
__device__ __forceinline__ Scale scale_of(float temp) {
  constexpr double kLog2e = 1.4426950408889634074;
  constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
  Scale s;
  s.hi = kHi / temp;
  s.lo = (fmaf(-s.hi, temp, kHi) + kLo) / temp;
  s.least = -150.0f / s.hi;
  return s;
}
__device__ __forceinline__ float weight(float x, float m, const Scale& s) {
  const float t = fmaxf(x - m, s.least);
  return ex2(fmaf(t, s.hi, t * s.lo));
}

// Whether a sequence takes its largest logits: temperature 0, or one outside [2^-100, 2^100].
__device__ __forceinline__ bool is_greedy(float temp) { return !(temp >= 0x1p-100f && temp <= 0x1p100f); }

// The sequence of a row: the last s with row_start[s] <= row.
__device__ __forceinline__ int seq_of(const int32_t* row_start, int seqs, int row) {
  int lo = 0, hi = seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(row_start + mid) <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Two elements of a 32-bit word.
template <typename T>
__device__ __forceinline__ float2 two(uint32_t w);
template <>
__device__ __forceinline__ float2 two<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 two<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// A lane's 32 logits of a piece: register v * VEC + e holds element first(v) + e of the row.
template <typename T>
struct Piece {
  static constexpr int VEC = 16 / (int)sizeof(T), NV = 32 / VEC;
  const T* row;
  int vocab;
  int shift;  // elements between the aligned address and the row's start
  __device__ __forceinline__ void open(const VerifyArgs& a, int64_t r) {
    row = static_cast<const T*>(a.logits) + r * a.logits_stride;
    vocab = a.vocab;
    shift = (int)((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % VEC);
  }
  __device__ __forceinline__ int first(int piece, int v, int lane) const {
    return piece * kPiece + v * 32 * VEC + lane * VEC - shift;
  }
  __device__ __forceinline__ void load(int piece, int lane, uint4 (&raw)[NV]) const {
    const int begin = piece * kPiece - shift;
    if (begin >= 0 && begin + kPiece <= vocab) {
      const uint4* at = reinterpret_cast<const uint4*>(row + begin) + lane;
#pragma unroll
      for (int v = 0; v < NV; ++v) raw[v] = at[32 * v];
      return;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = first(piece, v, lane);
      if (i >= 0 && i + VEC <= vocab) {
        raw[v] = *reinterpret_cast<const uint4*>(row + i);
      } else {
        T* e = reinterpret_cast<T*>(&raw[v]);
#pragma unroll
        for (int k = 0; k < VEC; ++k) e[k] = i + k >= 0 && i + k < vocab ? row[i + k] : from_f32<T>(-CUDART_INF_F);
      }
    }
  }
  // elements e and e + 1 (e even) of vector v
  static __device__ __forceinline__ float2 pair(const uint4 (&raw)[NV], int v, int e) {
    const uint32_t w[4] = {raw[v].x, raw[v].y, raw[v].z, raw[v].w};
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]));
    else return two<T>(w[e / 2]);
  }
  static __device__ __forceinline__ float at(const uint4 (&raw)[NV], int v, int e) {
    const float2 p = pair(raw, v, e & ~1);
    return (e & 1) ? p.y : p.x;
  }
  // the lane's largest element (NaN left out; -inf where there is none)
  static __device__ __forceinline__ float largest(const uint4 (&raw)[NV]) {
    if constexpr (sizeof(T) == 4) {
      float m = -CUDART_INF_F;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        m = fmaxf(m, fmaxf(fmaxf(at(raw, v, 0), at(raw, v, 1)), fmaxf(at(raw, v, 2), at(raw, v, 3))));
      return m;
    } else {
      using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      T2 m[4];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const uint32_t w[4] = {raw[v].x, raw[v].y, raw[v].z, raw[v].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const T2 x = *reinterpret_cast<const T2*>(&w[k]);
          m[k] = v == 0 ? x : __hmax2(m[k], x);
        }
      }
      const T2 all = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
      const float2 f = two<T>(*reinterpret_cast<const uint32_t*>(&all));
      return fmaxf(fmaxf(f.x, f.y), -CUDART_INF_F);
    }
  }
};

__device__ __forceinline__ float2 weights(float2 x, float m, const Scale& s) {
  float2 t = __fadd2_rn(x, make_float2(-m, -m));
  t.x = fmaxf(t.x, s.least);
  t.y = fmaxf(t.y, s.least);
  const float2 y = __ffma2_rn(t, make_float2(s.hi, s.hi), __fmul2_rn(t, make_float2(s.lo, s.lo)));
  return make_float2(ex2(y.x), ex2(y.y));
}

// ---------------------------------------------------------------- pieces

// A warp takes `per` consecutive pieces, the next one's logits under way while it works on one:
// a row's temperature is looked up once.
template <typename T>
__global__ void __launch_bounds__(kStatWarps * 32, sizeof(T) == 4 ? 2 : 3)
verify_stats_kernel(VerifyArgs a, VerifyWork w, int64_t per) {
  using P = Piece<T>;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = a.num_seqs > 0 ? min(a.num_rows, max(0, a.row_start[a.num_seqs])) : 0;
  const int64_t items = (int64_t)rows * w.pieces;
  int64_t item = ((int64_t)blockIdx.x * kStatWarps + warp) * per;
  const int64_t end = min(items, item + per);
  if (item >= end) return;
  int r = (int)(item / w.pieces), piece = (int)(item - (int64_t)r * w.pieces);
  P p;
  p.open(a, r);
  uint4 next[P::NV];
  p.load(piece, lane, next);
  bool fresh = true, greedy = false;
  Scale s;
#pragma unroll 1
  for (; item < end; ++item) {
    uint4 raw[P::NV];
#pragma unroll
    for (int v = 0; v < P::NV; ++v) raw[v] = next[v];
    const int here = r, first = p.first(piece, 0, lane);
    if (++piece == w.pieces) {
      piece = 0;
      ++r;
      if (item + 1 < end) p.open(a, r);
    }
    if (item + 1 < end) p.load(piece, lane, next);
    if (fresh) {
      const float temp = a.temperature ? __ldg(a.temperature + seq_of(a.row_start, a.num_seqs, here)) : 1.f;
      greedy = is_greedy(temp);
      s = scale_of(greedy ? 1.f : temp);
    }
    fresh = r != here;
    const float m = largest_of_warp(P::largest(raw));
    float2 st = make_float2(m, 0.f);
    if (greedy) {
      unsigned best = 0x7fffffffu;
#pragma unroll
      for (int v = P::NV - 1; v >= 0; --v)
#pragma unroll
        for (int e = P::VEC - 1; e >= 0; --e)
          if (P::at(raw, v, e) == m) best = (unsigned)(first + v * 32 * P::VEC + e);
      st.y = __uint_as_float(__reduce_min_sync(kFullMask, best));
    } else {
      float2 sum[4];
#pragma unroll
      for (int v = 0; v < P::NV; ++v)
#pragma unroll
        for (int e = 0; e < P::VEC; e += 2) {
          const int k = (v * P::VEC + e) / 2;
          const float2 x = weights(P::pair(raw, v, e), m, s);
          sum[k & 3] = k < 4 ? x : __fadd2_rn(sum[k & 3], x);
        }
      const float2 all = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
      st.y = warp_sum(all.x + all.y);
    }
    if (lane == 0) w.stats[item] = st;
  }
}

// ---------------------------------------------------------------- drawing a token

__device__ __forceinline__ u64 shfl_u64(u64 v, int lane) { return __shfl_sync(kFullMask, v, lane); }
__device__ __forceinline__ u64 warp_scan_u64(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 u = __shfl_up_sync(kFullMask, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
  return v;
}
// u in [0, 1) of a whole sum (numbers outside, and NaN, go to the nearest end).
__device__ __forceinline__ u64 part_of(float u, u64 total) {
  if (!(u > 0.f) || total == 0) return 0;
  if (u >= 1.f) return total - 1;
  return min((u64)((double)u * (double)total), total - 1);
}

// The first element e of a piece whose running sum of value(v, e) passes `target`, by a warp;
// where rounding leaves none, the last with a value.  -1: the piece has none.
template <typename T, typename F>
__device__ __forceinline__ int find_in_piece(const Piece<T>& p, int piece, int lane, u64 target, F value) {
  constexpr int VEC = Piece<T>::VEC, NV = Piece<T>::NV;
  u64 run = 0;
  int last = -1;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    u64 part = 0;
    int tail = -1;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const u64 x = value(v, e);
      part += x;
      if (x) tail = e;
    }
    const u64 incl = warp_scan_u64(part, lane);
    const unsigned hit = __ballot_sync(kFullMask, run + incl > target);
    if (hit) {
      const int src = __ffs(hit) - 1;
      u64 at = run + incl - part;
      int found = -1;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        at += value(v, e);
        if (found < 0 && at > target) found = e;
      }
      return p.first(piece, v, src) + __shfl_sync(kFullMask, found, src);
    }
    const unsigned some = __ballot_sync(kFullMask, tail >= 0);
    if (some) {
      const int src = 31 - __clz(some);
      last = p.first(piece, v, src) + __shfl_sync(kFullMask, tail, src);
    }
    run += shfl_u64(incl, 31);
  }
  return last;
}

// The piece in which the running sum of sums(k), k < pieces, passes u times the whole, by a
// warp; `target` becomes the rest inside it.
template <typename F>
__device__ __forceinline__ int find_piece(int pieces, int lane, float u, u64& target, F sums) {
  const int per = (pieces + 31) / 32;
  u64 part = 0;
  for (int k = lane * per; k < min(pieces, (lane + 1) * per); ++k) part += sums(k);
  const u64 incl = warp_scan_u64(part, lane);
  const u64 goal = part_of(u, shfl_u64(incl, 31));
  const unsigned hit = __ballot_sync(kFullMask, incl > goal);
  const int src = hit ? __ffs(hit) - 1 : 31;
  u64 rest = goal - (incl - part);
  int found = 0;
  if (lane == src) {
    for (int k = lane * per; k < min(pieces, (lane + 1) * per); ++k) {
      const u64 x = sums(k);
      found = k;
      if (x > rest) break;
      rest -= x;
    }
  }
  target = shfl_u64(rest, src);
  return __shfl_sync(kFullMask, found, src);
}

__device__ __forceinline__ u64 fixed(float v, float unit) { return (u64)__float2ll_rn(v * unit); }

// A row's pieces, in the warp's shared memory where they fit: they are gone through several times.
constexpr int kHeld = 256;
__device__ __forceinline__ const float2* hold_stats(const VerifyWork& w, int64_t r, float2* room, int lane) {
  const float2* st = w.stats + r * w.pieces;
  if (w.pieces > kHeld) return st;
  __syncwarp();
  for (int k = lane; k < w.pieces; k += 32) room[k] = __ldcg(st + k);
  __syncwarp();
  return room;
}
// Largest logit of a row, from its pieces.
__device__ __forceinline__ float row_top(const float2* st, int pieces, int lane) {
  float m = -CUDART_INF_F;
  for (int k = lane; k < pieces; k += 32) m = fmaxf(m, st[k].x);
  return largest_of_warp(m);
}
__device__ __forceinline__ bool has_distribution(float top) { return fabsf(top) < CUDART_INF_F; }

// First largest logit of a row with largest logit `top`.
__device__ __forceinline__ int row_best(const float2* st, int pieces, int lane, float top) {
  unsigned best = 0x7fffffffu;
  for (int k = lane; k < pieces; k += 32)
    if (st[k].x == top) best = min(best, __float_as_uint(st[k].y));
  return (int)__reduce_min_sync(kFullMask, best);
}

// Fixed-point unit of a row's weights: at most `vocab` of them, at most 1 each.
__device__ __forceinline__ float row_unit(int vocab) { return pow2i(62 - (32 - __clz(vocab))); }

// A token from p, by a warp.
template <typename T>
__device__ __forceinline__ int draw_token(const VerifyArgs& a, const VerifyWork& w, const float2* st, int64_t r, float top,
                                          const Scale& s, float u, int lane) {
  const float unit = row_unit(a.vocab);
  u64 target;
  const int piece = find_piece(w.pieces, lane, u, target,
                               [&](int k) { return fixed(st[k].y * weight(st[k].x, top, s), unit); });
  Piece<T> p;
  p.open(a, r);
  uint4 raw[Piece<T>::NV];
  p.load(piece, lane, raw);
  int i = find_in_piece<T>(p, piece, lane, target,
                               [&](int v, int e) { return fixed(weight(Piece<T>::at(raw, v, e), top, s), unit); });
  if (i < 0) {  // weights too small for the unit one by one, not together: the piece's largest
    float m = -CUDART_INF_F;
    unsigned best = 0x7fffffffu;
#pragma unroll
    for (int v = 0; v < Piece<T>::NV; ++v)
#pragma unroll
      for (int e = 0; e < Piece<T>::VEC; ++e) {
        const float x = Piece<T>::at(raw, v, e);
        if (x > m) m = x, best = (unsigned)(p.first(piece, v, lane) + e);
      }
    const float all = warp_max(m);
    if (m != all) best = 0x7fffffffu;
    i = (int)__reduce_min_sync(kFullMask, best);
  }
  return i;
}

// Rows [r0, r0 + n) of a sequence; none where row_start is not ascending inside [0, num_rows].
__device__ __forceinline__ int rows_of(const VerifyArgs& a, int s, int& r0) {
  r0 = a.row_start[s];
  const int r1 = a.row_start[s + 1];
  const bool ok = r0 >= 0 && r1 >= r0 && r1 <= a.num_rows;
  if (!ok && a.status && threadIdx.x == 0) atomicMax(a.status, (int32_t)kInvalidArg);
  return ok ? r1 - r0 : 0;
}
// A sequence's tokens and parents, in shared memory up to kNodes of them.
constexpr int kNodes = 256;
struct Nodes {
  const int32_t* tokens;
  const int32_t* parents;  // null: a chain
  int n;
  // by a CTA of `threads` threads (a barrier follows before they are read)
  __device__ __forceinline__ void open(const VerifyArgs& a, int r0, int rows, int32_t (*room)[kNodes], int threads) {
    n = rows;
    tokens = a.tokens + r0;
    parents = a.parents ? a.parents + r0 : nullptr;
    if (n > kNodes) return;
    for (int i = threadIdx.x; i < n; i += threads) {
      room[0][i] = tokens[i];
      if (parents) room[1][i] = parents[i];
    }
    tokens = room[0];
    if (parents) parents = room[1];
  }
  __device__ __forceinline__ int parent(int i) const { return parents ? parents[i] : i - 1; }
  // First child i >= from of node c that `match` accepts (-1: none), by a warp.
  template <typename F>
  __device__ __forceinline__ int next_child(int c, int from, int lane, F match) const {
    if (!parents) return from == c + 1 && from < n && match(from) ? from : -1;  // a chain: one child a node
    for (int b = from; b < n; b += 32) {
      const int i = b + lane;
      const unsigned mask = __ballot_sync(kFullMask, i < n && parents[i] == c && match(i));
      if (mask) return b + __ffs(mask) - 1;
    }
    return -1;
  }
};

// Temperatures out of range and parents that are no earlier nodes are reported.
__device__ __forceinline__ void check_sequence(const VerifyArgs& a, int s, int r0, int n, int first, int step) {
  if (!a.status) return;
  bool bad = false;
  if (first == 0 && n > 0 && a.temperature) {
    const float t = a.temperature[s];
    bad = t != 0.f && is_greedy(t);
  }
  if (a.parents)
    for (int i = 1 + first; i < n; i += step) {
      const int up = a.parents[r0 + i];
      bad |= up < 0 || up >= i;
    }
  if (bad) atomicMax(a.status, (int32_t)kInvalidArg);
}

// ---------------------------------------------------------------- no draft probabilities

template <typename T>
__global__ void __launch_bounds__(kPickWarps * 32) verify_pick_kernel(VerifyArgs a, VerifyWork w) {
  extern __shared__ float2 held[];  // kHeld of every warp
  __shared__ int32_t node_room[2][kNodes], pick_room[kNodes];
  const int s = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  int r0;
  const int n = rows_of(a, s, r0);
  check_sequence(a, s, r0, n, threadIdx.x, blockDim.x);
  Nodes nodes;
  nodes.open(a, r0, n, node_room, blockDim.x);
  const float temp = a.temperature ? a.temperature[s] : 1.f;
  const bool greedy = is_greedy(temp);
  const Scale sc = scale_of(greedy ? 1.f : temp);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  bool none = false;
  for (int i = warp; i < n; i += warps) {
    const int64_t r = r0 + i;
    const float2* st = hold_stats(w, r, held + warp * kHeld, lane);
    const float top = row_top(st, w.pieces, lane);
    int pick = -1;
    if (!has_distribution(top)) none = true;
    else if (greedy) pick = row_best(st, w.pieces, lane, top);
    else pick = draw_token<T>(a, w, st, r, top, sc, a.u_sample[r], lane);
    if (lane == 0) (n <= kNodes ? pick_room[i] : w.rows[r].pick) = pick;
  }
  if (none && a.status && lane == 0) atomicMax(a.status, (int32_t)kInvalidArg);
  __syncthreads();
  if (warp != 0) return;
  int32_t* path = a.path + (int64_t)s * a.max_path;
  int len = 0, next = -1;
  if (n > 0) {
    int c = 0;
    while (true) {
      if (lane == 0) path[len] = c;
      ++len;
      next = n <= kNodes ? pick_room[c] : w.rows[r0 + c].pick;
      if (next < 0 || len == a.max_path) break;
      const int child = nodes.next_child(c, c + 1, lane, [&](int i) { return nodes.tokens[i] == next; });
      if (child < 0) break;
      c = child;
    }
  }
  for (int j = len + lane; j < a.max_path; j += 32) path[j] = -1;
  if (lane == 0) {
    a.path_lens[s] = len;
    a.next_token[s] = next;
  }
}

// ---------------------------------------------------------------- draft probabilities

// A lane's 32 draft probabilities beside a Piece<T>.
template <typename T, typename Q>
__device__ __forceinline__ void load_draft(const VerifyArgs& a, const Piece<T>& p, int64_t r, int piece, int lane,
                                           float (&q)[32]) {
  constexpr int VEC = Piece<T>::VEC, NV = Piece<T>::NV;
  const Q* row = static_cast<const Q*>(a.draft) + r * a.draft_stride;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = p.first(piece, v, lane);
    constexpr int bytes = VEC * (int)sizeof(Q);
    constexpr int step = bytes < 16 ? bytes : 16, per = step / (int)sizeof(Q);
    if (i >= 0 && i + VEC <= a.vocab && reinterpret_cast<uintptr_t>(row + i) % step == 0) {
#pragma unroll
      for (int k = 0; k < bytes / step; ++k) {
        alignas(16) Q e[per];
        if constexpr (step == 16) *reinterpret_cast<uint4*>(e) = reinterpret_cast<const uint4*>(row + i)[k];
        else *reinterpret_cast<uint2*>(e) = reinterpret_cast<const uint2*>(row + i)[k];
#pragma unroll
        for (int u = 0; u < per; ++u) q[v * VEC + k * per + u] = fmaxf(to_f32<Q>(e[u]), 0.f);
      }
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        q[v * VEC + k] = i + k >= 0 && i + k < a.vocab ? fmaxf(to_f32<Q>(row[i + k]), 0.f) : 0.f;
    }
  }
}

constexpr float kRestUnit = 0x1p60f;  // sums of max(a p - b q, 0) are at most 1

// The first CTA of a sequence's cluster works out the rows and walks; the others take their share of
// the passes over a row, told by the first alone which row and with what coefficients, so that all
// meet at the same barriers whatever the buffers hold.
template <typename T, typename Q>
__global__ void __launch_bounds__(kDraftWarps * 32, 2) verify_draft_kernel(VerifyArgs a, VerifyWork w) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int s = blockIdx.x / ranks, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (a CTA's shared memory may be written by another once it runs)
  auto started = cluster.barrier_arrive();
  constexpr int threads = kDraftWarps * 32;
  const int warps = ranks * kDraftWarps, gwarp = rank * kDraftWarps + warp;
  struct Pass {
    int row;             // -1: no more
    float a, b, top;     // max(a weight - b q, 0)
  };
  __shared__ float2 held[kDraftWarps][kHeld];
  __shared__ int32_t node_room[2][kNodes];
  __shared__ float4 row_room[kNodes];
  __shared__ float2 pq_room[kNodes];
  __shared__ u64 rest_room[kHeld];
  __shared__ Pass todo;
  const float temp = a.temperature ? a.temperature[s] : 1.f;
  const bool greedy = is_greedy(temp);
  const Scale sc = scale_of(greedy ? 1.f : temp);
  int r0 = 0, n = 0;
  Nodes nodes;
  float4* rows = row_room;
  float2* pqs = pq_room;
  if (rank == 0) {
    n = rows_of(a, s, r0);
    check_sequence(a, s, r0, n, threadIdx.x, threads);
    nodes.open(a, r0, n, node_room, threads);
    if (n > kNodes) {
      rows = reinterpret_cast<float4*>(w.rows + r0);
      pqs = w.pq + r0;
    }
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (rank == 0) {
    // rows' largest logits, sums (their inverses) and, greedy, first largest logits
    bool none = false;
    for (int i = warp; i < n; i += kDraftWarps) {
      const float2* st = hold_stats(w, r0 + i, held[warp], lane);
      const float top = row_top(st, w.pieces, lane);
      float inv = 0.f;
      int pick = -1;
      if (!has_distribution(top)) {
        none = true;
      } else if (greedy) {
        pick = row_best(st, w.pieces, lane, top);
      } else {
        const float unit = row_unit(a.vocab);
        u64 sum = 0;
        for (int k = lane; k < w.pieces; k += 32) sum += fixed(st[k].y * weight(st[k].x, top, sc), unit);
        inv = unit / (float)warp_sum_u64(sum);
        pick = 0;
      }
      if (lane == 0) rows[i] = make_float4(top, inv, __int_as_float(pick), 0.f);
    }
    if (none && a.status && lane == 0) atomicMax(a.status, (int32_t)kInvalidArg);
    __syncthreads();
    // p and q of every drafted token
    for (int i = 1 + (int)threadIdx.x; i < n; i += threads) {
      const int up = nodes.parent(i), tok = nodes.tokens[i];
      float2 pq = make_float2(-1.f, 0.f);  // never kept
      if (up >= 0 && up < i && tok >= 0 && tok < a.vocab) {
        const int64_t r = r0 + up;
        const float4 info = rows[up];
        const int pick = __float_as_int(info.z);
        if (greedy) {
          pq.x = pick == tok ? 1.f : -1.f;
        } else if (pick >= 0) {
          const float x = to_f32<T>(static_cast<const T*>(a.logits)[r * a.logits_stride + tok]);
          pq.y = fmaxf(to_f32<Q>(static_cast<const Q*>(a.draft)[r * a.draft_stride + tok]), 0.f);
          pq.x = weight(x, info.x, sc) * info.y;
        }
      }
      pqs[i] = pq;
    }
    __syncthreads();
  }
  // the walk, by the first CTA's first warp
  const bool walks = rank == 0 && warp == 0;
  cluster.barrier_wait(std::move(started));
  int c = 0, from = 1;
  float ca = 1.f, cb = 0.f;      // r = max(ca p - cb q, 0) at node c
  float da = 1.f, db = 0.f;      // the coefficients whose sums the last pass took (db 0: none at c)
  bool again = false;
  int32_t* path = a.path + (int64_t)s * a.max_path;
  const float4 no_row = make_float4(0.f, 0.f, __int_as_float(-1), 0.f);
  float4 info = walks && n > 0 ? rows[0] : no_row;
  if (walks && lane == 0 && n > 0) path[0] = 0;
  int len = n > 0 ? 1 : 0;
  while (true) {
    if (walks) {
      int need = -1;
      while (!again && __float_as_int(info.z) >= 0 && len < a.max_path) {
        const int child = nodes.next_child(c, from, lane, [](int) { return true; });
        if (child < 0) break;
        const float2 pq = pqs[child];
        const float r = fmaf(ca, pq.x, -cb * pq.y);
        if (greedy ? pq.x > 0.f : (r > 0.f && a.u_accept[r0 + child] * pq.y < r)) {
          c = child;
          from = c + 1;
          ca = da = 1.f;
          cb = db = 0.f;
          info = rows[c];
          if (lane == 0) path[len] = c;
          ++len;
        } else {
          from = child + 1;
          const int tok = nodes.tokens[child];
          if (greedy || tok < 0 || tok >= a.vocab) continue;  // not drawn from q
          da = ca, db = cb + 1.f;
          need = c;
          break;
        }
      }
      if (again) need = c;
      const Pass next{need < 0 ? -1 : r0 + need, da * info.y, db, info.x};
      if (lane < ranks) *cluster.map_shared_rank(&todo, lane) = next;
    }
    cluster.sync();
    const Pass now = todo;
    if (now.row < 0) break;
    Piece<T> p;
    p.open(a, now.row);
    u64* rest = w.rest + (int64_t)s * w.pieces;
    for (int k = gwarp; k < w.pieces; k += warps) {
      uint4 raw[Piece<T>::NV];
      float q[32];
      p.load(k, lane, raw);
      load_draft<T, Q>(a, p, now.row, k, lane, q);
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < Piece<T>::NV; ++v)
#pragma unroll
        for (int e = 0; e < Piece<T>::VEC; e += 2) {
          const float2 x = weights(Piece<T>::pair(raw, v, e), now.top, sc);
          sum += fmaxf(fmaf(now.a, x.x, -now.b * q[v * Piece<T>::VEC + e]), 0.f);
          sum += fmaxf(fmaf(now.a, x.y, -now.b * q[v * Piece<T>::VEC + e + 1]), 0.f);
        }
      const u64 all = warp_sum_u64(fixed(sum, kRestUnit));
      if (lane == 0) __stcg(rest + k, all);
    }
    cluster.sync();
    if (walks) {
      u64 sum = 0;
      for (int k = lane; k < w.pieces; k += 32) {
        const u64 x = __ldcg(rest + k);
        if (w.pieces <= kHeld) rest_room[k] = x;
        sum += x;
      }
      __syncwarp();
      sum = warp_sum_u64(sum);
      if (again) {
        again = false;
      } else if (sum > 0) {
        const float z = (float)sum / kRestUnit;
        ca = da / z;
        cb = db / z;
      } else {  // nothing is left: the distribution before the subtraction stays
        da = ca, db = cb;
        again = db > 0.f;
      }
    }
  }
  if (!walks) return;
  int next = -1;
  if (__float_as_int(info.z) >= 0) {
    const int64_t r = r0 + c;
    const float u = a.u_sample[r];
    if (greedy) {
      next = __float_as_int(info.z);
    } else {
      int i = -1;
      if (db > 0.f) {
        const u64* rest = w.pieces <= kHeld ? rest_room : w.rest + (int64_t)s * w.pieces;
        u64 target;
        const int piece = find_piece(w.pieces, lane, u, target, [&](int k) { return rest[k]; });
        Piece<T> p;
        p.open(a, r);
        uint4 raw[Piece<T>::NV];
        float q[32];
        p.load(piece, lane, raw);
        load_draft<T, Q>(a, p, r, piece, lane, q);
        const float pa = da * info.y;
        i = find_in_piece<T>(p, piece, lane, target, [&](int v, int e) {
          return fixed(fmaxf(fmaf(pa, weight(Piece<T>::at(raw, v, e), info.x, sc), -db * q[v * Piece<T>::VEC + e]), 0.f),
                       kRestUnit);
        });
      }
      // from p where nothing was refused (or no weight is above the unit)
      if (i < 0) i = draw_token<T>(a, w, hold_stats(w, r, held[0], lane), r, info.x, sc, u, lane);
      next = i;
    }
  }
  for (int j = len + lane; j < a.max_path; j += 32) path[j] = -1;
  if (lane == 0) {
    a.path_lens[s] = len;
    a.next_token[s] = next;
  }
}

// Laid out for rows at any address.
VerifyWork layout(void* workspace, int rows, int vocab, int seqs, size_t* bytes) {
  VerifyWork w{};
  w.pieces = pieces_of(vocab, 7);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t first = at;
    at = (at + n + 255) / 256 * 256;
    return workspace ? static_cast<unsigned char*>(workspace) + first : nullptr;
  };
  w.stats = reinterpret_cast<float2*>(take((size_t)rows * w.pieces * sizeof(float2)));
  w.rows = reinterpret_cast<RowInfo*>(take((size_t)rows * sizeof(RowInfo)));
  w.pq = reinterpret_cast<float2*>(take((size_t)rows * sizeof(float2)));
  w.rest = reinterpret_cast<u64*>(take((size_t)seqs * w.pieces * sizeof(u64)));
  *bytes = at;
  return w;
}

// The second kernel is a programmatic dependent of the first: its set-up overlaps it.
template <typename K>
cudaError_t launch_after(K kern, int grid, int threads, int cluster, int smem, cudaStream_t stream, const VerifyArgs& a,
                         const VerifyWork& w) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, a, w);
  if (err == cudaSuccess) count_launches(1);
  return err;
}

template <typename T>
cudaError_t launch_verify_typed(const VerifyArgs& a, VerifyWork w, cudaStream_t stream) {
  const int sms = device_sms();
  // rows that all start at 16-byte boundaries have no piece more
  const bool even = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && (a.num_rows < 2 || a.logits_stride * sizeof(T) % 16 == 0);
  w.pieces = pieces_of(a.vocab, even ? 0 : 16 / (int)sizeof(T) - 1);
  const int64_t items = (int64_t)a.num_rows * w.pieces, resident = (int64_t)sms * (sizeof(T) == 4 ? 2 : 3) * kStatWarps;
  const int64_t per = std::max<int64_t>(1, (items + resident - 1) / resident);
  const int64_t ctas = ((items + per - 1) / per + kStatWarps - 1) / kStatWarps;
  verify_stats_kernel<T><<<(int)std::max<int64_t>(1, ctas), kStatWarps * 32, 0, stream>>>(a, w, per);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  count_launches(1);
  if (!a.draft) {
    // twice the warps of an average sequence's rows: ragged ones take one turn too
    const int warps = std::max(1, std::min(kPickWarps, 2 * ((a.num_rows + a.num_seqs - 1) / a.num_seqs)));
    return launch_after(verify_pick_kernel<T>, a.num_seqs, warps * 32, 1, warps * kHeld * (int)sizeof(float2), stream, a, w);
  }
  // as many CTAs a sequence as run at once, and as its rows' pieces keep busy
  int ctas_seq = kDraftCtas;
  while (ctas_seq > 1 && ((int64_t)a.num_seqs * ctas_seq > 2 * sms || ctas_seq * kDraftWarps >= 2 * w.pieces)) ctas_seq /= 2;
  const int64_t dgrid = (int64_t)a.num_seqs * ctas_seq;
  if (dgrid > 0x7fffffff) return cudaErrorInvalidValue;
  const int threads = kDraftWarps * 32;
  switch (a.draft_dtype) {
    case kF32: return launch_after(verify_draft_kernel<T, float>, (int)dgrid, threads, ctas_seq, 0, stream, a, w);
    case kF16: return launch_after(verify_draft_kernel<T, __half>, (int)dgrid, threads, ctas_seq, 0, stream, a, w);
    case kBF16: return launch_after(verify_draft_kernel<T, __nv_bfloat16>, (int)dgrid, threads, ctas_seq, 0, stream, a, w);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

size_t verify_workspace(int num_rows, int vocab, int num_seqs) {
  size_t bytes = 0;
  layout(nullptr, num_rows, vocab, num_seqs, &bytes);
  return bytes;
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream) {
  if (a.status) {
    const cudaError_t err = cudaMemsetAsync(a.status, 0, sizeof(int32_t), stream);
    if (err != cudaSuccess) return err;
  }
  if (a.num_seqs == 0) return cudaSuccess;
  size_t bytes = 0;
  const VerifyWork w = layout(a.workspace, a.num_rows, a.vocab, a.num_seqs, &bytes);
  switch (a.logits_dtype) {
    case kF32: return launch_verify_typed<float>(a, w, stream);
    case kF16: return launch_verify_typed<__half>(a, w, stream);
    case kBF16: return launch_verify_typed<__nv_bfloat16>(a, w, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
