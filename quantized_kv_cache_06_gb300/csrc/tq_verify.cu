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
//   * Draft probabilities q (children drawn from q): child x is kept when u q(x) < r(x), r = p at first;
//     refused, r becomes max(r - q, 0) over its sum.  All refused: a token from r.
//
// Two levels of precision.  fp32 weights 2^((x - m) c), c = log2(e) / temperature in two parts, m the
// piece's largest logit, give every border of a row's running sum to about 10^-6 of the whole, and a
// derived bound of that.  A vocabulary of 131072 has tokens no wider than that, so a number that lies
// within the bound of its token's borders (about a tenth of the draws at that size), and every refusal, is
// decided by a pass over the row with weights of two floats, to 2^-40 of the whole.  Sums are integers at
// both levels: results do not depend on any order.
//
// Launches.  1. Every warp takes consecutive pieces of 1024 logits, the next one's under way, and
// leaves each piece's largest logit and its sum of weights (or its first largest, where the temperature
// is 0).  2. A cluster takes a sequence: one CTA decides and all share the passes over a row.  Many
// sequences without draft probabilities have a CTA each instead, and 3. clusters for those that need a pass.
//
// Bound (GB300): of the first launch the logits' bytes (256 trees, 1153 rows of 131072 bf16, 303 MB
// read once: 55 us, 82 % of the copy bandwidth; 253 warp instructions a piece, 64 % of the issue slots,
// the exponentials' pipe as busy); of the others latency, and in a pass the fp32 pipe (40 operations an
// element: 64 refused rows of 131072 take 15 us for their sums and 26 us for what refusals leave).  Whole
// calls: 89 us, and 88 us for 64 chains of 5 rows with draft probabilities.  Measured and not kept:
// pieces dealt out one by one, a row's temperature looked up for each (256 trees 131 us); every CTA of a
// cluster walking for itself (the same time, and barriers that would hang on buffers that change under the
// call); passes by 12 or 16 warps a CTA (the same time: they wait for the fp32 pipe); 64-bit conversions
// of every element in a pass (64 chains 116 us).
//
// Rows may start at any multiple of their element's size: pieces are laid out from the aligned
// address at or before the row's start, so all but a row's first and last 16 bytes are loaded 16
// bytes at a time.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
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
constexpr int kWalkWarps = 8;    // of a CTA of a cluster
constexpr int kWalkCtas = 8;     // most CTAs of a cluster

using u64 = unsigned long long;

struct RowInfo {
  float max, sum;  // largest logit; sum of weights
  int32_t pick;    // token drawn (no draft probabilities, or temperature 0), or one of the two below
  int32_t seq;     // whose temperature the row's pieces are of (0 once a walk holds the row)
};
constexpr int kNoPick = -1;      // no distribution
constexpr int kUnsure = -2;      // fp32 weights do not tell

struct VerifyWork {
  float2* stats;   // [rows][pieces]: largest logit, sum of weights (its bits: first largest)
  RowInfo* rows;   // [rows]
  float2* pq;      // [rows]: weight and q of the row's token under its parent
  u64* rest;       // [clusters][pieces][vectors of a piece]: sums of max(W - G q, 0)
  int32_t* list;   // [1 + seqs]: how many sequences the second launch left to the third, and which
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
  // vector v of a piece
  __device__ __forceinline__ uint4 load_one(int piece, int v, int lane) const {
    const int i = first(piece, v, lane);
    if (i >= 0 && i + VEC <= vocab) return *reinterpret_cast<const uint4*>(row + i);
    uint4 raw;
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int k = 0; k < VEC; ++k) e[k] = i + k >= 0 && i + k < vocab ? row[i + k] : from_f32<T>(-CUDART_INF_F);
    return raw;
  }
  // elements e and e + 1 (e even) of vector v
  static __device__ __forceinline__ float2 pair(const uint4 (&raw)[NV], int v, int e) { return pair_of(raw[v], e); }
  static __device__ __forceinline__ float2 pair_of(const uint4& raw, int e) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[e]), __uint_as_float(w[e + 1]));
    else return two<T>(w[e / 2]);
  }
  static __device__ __forceinline__ float at(const uint4 (&raw)[NV], int v, int e) { return one(raw[v], e); }
  static __device__ __forceinline__ float one(const uint4& raw, int e) {
    const float2 p = pair_of(raw, e & ~1);
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
  if (blockIdx.x == 0 && threadIdx.x == 0) w.list[0] = 0;
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
    const bool begins = piece == 0;
    if (++piece == w.pieces) {
      piece = 0;
      ++r;
      if (item + 1 < end) p.open(a, r);
    }
    if (item + 1 < end) p.load(piece, lane, next);
    if (fresh) {
      const int seq = seq_of(a.row_start, a.num_seqs, here);
      if (begins && lane == 0) w.rows[here].seq = seq;
      const float temp = a.temperature ? __ldg(a.temperature + seq) : 1.f;
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

// The first element of a piece whose running sum of value(x) passes `target`, by a warp, and the running
// sums before and behind it; where rounding leaves none, the last with a value (-1: there is none), and
// `target` for both.  (Rolled: a warp comes here once, and waits longer for instructions than for their
// results.)
template <typename T, typename F>
__device__ __forceinline__ int find_in_piece(const Piece<T>& p, int piece, int lane, u64 target, u64& before, u64& behind,
                                             F value) {
  constexpr int VEC = Piece<T>::VEC, NV = Piece<T>::NV;
  uint4 raw[NV];
  p.load(piece, lane, raw);
  u64 run = 0;
  int last = -1;
#pragma unroll 1
  for (int v = 0; v < NV; ++v) {
    const uint4 now = raw[0];
#pragma unroll
    for (int k = 0; k + 1 < NV; ++k) raw[k] = raw[k + 1];
    u64 values[VEC], part = 0;
    int tail = -1;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      values[e] = value(Piece<T>::one(now, e));
      part += values[e];
      if (values[e]) tail = e;
    }
    const u64 incl = warp_scan_u64(part, lane);
    const unsigned hit = __ballot_sync(kFullMask, run + incl > target);
    if (hit) {
      const int src = __ffs(hit) - 1;
      u64 at = run + incl - part, lo = 0, hi = 0;
      int found = -1;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const u64 next = at + values[e];
        if (found < 0 && next > target) found = e, lo = at, hi = next;
        at = next;
      }
      before = shfl_u64(lo, src);
      behind = shfl_u64(hi, src);
      return p.first(piece, v, src) + __shfl_sync(kFullMask, found, src);
    }
    const unsigned some = __ballot_sync(kFullMask, tail >= 0);
    if (some) {
      const int src = 31 - __clz(some);
      last = p.first(piece, v, src) + __shfl_sync(kFullMask, tail, src);
    }
    run += shfl_u64(incl, 31);
  }
  before = behind = target;
  return last;
}

// The piece in which the running sum of sums(k), k < pieces, passes u times the whole (`goal` of
// `total`), by a warp; `target` becomes the rest inside it.
template <typename F>
__device__ __forceinline__ int find_piece(int pieces, int lane, float u, u64& total, u64& goal, u64& target, F sums) {
  const int per = (pieces + 31) / 32;
  u64 part = 0;
  for (int k = lane * per; k < min(pieces, (lane + 1) * per); ++k) part += sums(k);
  const u64 incl = warp_scan_u64(part, lane);
  total = shfl_u64(incl, 31);
  goal = part_of(u, total);
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
// (a row that two sequences of a descending row_start claim is one's alone)
__device__ __forceinline__ bool has_distribution(const VerifyWork& w, int64_t r, int s, float top) {
  return fabsf(top) < CUDART_INF_F && __ldcg(&w.rows[r].seq) == s;
}

// First largest logit of a row with largest logit `top`.
__device__ __forceinline__ int row_best(const float2* st, int pieces, int lane, float top) {
  unsigned best = 0x7fffffffu;
  for (int k = lane; k < pieces; k += 32)
    if (st[k].x == top) best = min(best, __float_as_uint(st[k].y));
  return (int)__reduce_min_sync(kFullMask, best);
}

// Fixed-point unit of a row's weights: at most `vocab` of them, at most 1 each.
__device__ __forceinline__ float row_unit(int vocab) { return pow2i(62 - (32 - __clz(vocab))); }

// How far fp32 weights 2^y may be off, relative to themselves:
//   kPowError |y|  the exponent's roundings: one of x - m, one of the product, 2^-24 |y| each, times ln 2;
//   kSumError      ex2's error, below 2^-22 (2^-22.7 over every fp32 in [-126, 0]), of a weight within its
//                  piece and of the piece's within the row, and 12 roundings of 2^-24 in sums (three of a
//                  lane's accumulators, three joins, five exchanges) and the product of the two.
// The mean of |y| over a row's tokens, weighted, is its entropy less log2 of the weights' sum, which is
// at least 1: below log2 of the vocabulary.
constexpr float kPowError = 0.7f * 0x1p-23f, kSumError = 0x1p-21f + 13 * 0x1p-24f;

// A token from p, by a warp: kUnsure where the borders of the token found are nearer to the number than
// they may be off.  With errors d_i of the weights, a running sum P of the whole S is off u S by
// (1 - u) times the errors behind it less u times those in front: at most 2 u (1 - u) S where all are
// bounded alike, max(u, 1 - u) S where their mean is.
template <typename T>
__device__ __noinline__ int draw_token(const VerifyArgs& a, const VerifyWork& w, const float2* st, int64_t r, float top,
                                          const Scale& s, float u, int lane) {
  const float unit = row_unit(a.vocab);
  u64 total, goal, target, before, behind;
  const int piece = find_piece(w.pieces, lane, u, total, goal, target,
                               [&](int k) { return fixed(st[k].y * weight(st[k].x, top, s), unit); });
  Piece<T> p;
  p.open(a, r);
  const int i = find_in_piece<T>(p, piece, lane, target, before, behind,
                                 [&](float x) { return fixed(weight(x, top, s), unit); });
  const float whole = (float)total, share = (float)goal / whole;
  const float near = whole * (kSumError * 2.f * share * (1.f - share) +
                              kPowError * (float)(32 - __clz(a.vocab)) * fmaxf(share, 1.f - share)) * 1.001f +
                     (float)(w.pieces + kPiece);  // roundings to the unit
  return (float)(target - before) > near && (float)(behind - target) > near ? i : kUnsure;
}

// Rows [r0, r0 + n) of a sequence; none where row_start is not ascending inside [0, num_rows], or
// passes its last entry: the first launch takes no rows behind that.
__device__ __forceinline__ int rows_of(const VerifyArgs& a, int s, int& r0) {
  r0 = a.row_start[s];
  const int r1 = a.row_start[s + 1];
  const bool ok = r0 >= 0 && r1 >= r0 && r1 <= min(a.num_rows, a.row_start[a.num_seqs]);
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
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  bool none = false;
  for (int i = warp; i < n; i += warps) {
    const int64_t r = r0 + i;
    const float2* st = hold_stats(w, r, held + warp * kHeld, lane);
    const float top = row_top(st, w.pieces, lane);
    int pick = -1;
    if (!has_distribution(w, r, s, top)) none = true;
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
  if (next == kUnsure) {  // left to verify_walk_kernel
    if (n <= kNodes)
      for (int i = lane; i < n; i += 32) w.rows[r0 + i].pick = pick_room[i];
    if (lane == 0) {
      const int at = atomicAdd(w.list, 1);
      if (at >= 0 && at < a.num_seqs) w.list[1 + at] = s;  // (always, but in a workspace that another call uses)
    }
    return;
  }
  for (int j = len + lane; j < a.max_path; j += 32) path[j] = -1;
  if (lane == 0) {
    a.path_lens[s] = len;
    a.next_token[s] = next;
  }
}

// ---------------------------------------------------------------- weights beyond fp32
//
// W = 2^54 2^y, y = (x - m) c, as two floats: x - m is exact as a sum of two, its product with the two
// parts of c too but for parts below 2^-46 |y|, and with y = k / 1024 + g
//   2^y = 2^(k div 1024) T (1 + z + z^2 / 2 + z^3 / 6), z = g ln 2, |z| < 2^-11.5,
// T = 2^((k mod 1024) / 1024) from a table of two floats, the head of T z by an exact product.  W is off by
// less than 2^-45 (1 + |y|) of itself (20 million logits and temperatures against 64-bit significands).  A
// lane adds a vector's weights with exact sums of the heads and rounds once to a whole number; a vector's
// sum of those fits 64 bits, a row's takes 128.
// (37 fp32 operations an element, 8 others and a lookup: this GPU's fp64 would take many times that.)

struct HiLo {
  float h, l;
};
constexpr int kCells = 1024;
struct alignas(16) Pow2Table {
  HiLo e[kCells];
};
constexpr Pow2Table make_pow2() {
  Pow2Table t{};
  for (int j = 0; j < kCells; ++j) {
    const double z = 0.69314718055994530942 * j / kCells;
    double sum = 0;
    for (int n = 20; n >= 1; --n) sum = z / n * (1.0 + sum);  // e^z - 1
    const float h = (float)(1.0 + sum);
    t.e[j].h = h;
    t.e[j].l = (float)(1.0 - (double)h + sum);
  }
  return t;
}
__device__ const Pow2Table kPow2 = make_pow2();

constexpr int kUnitBits = 54;

struct Exact {
  float top, hi, lo;  // m; c
  float least;        // weights of logits below are 0
};
__device__ __forceinline__ Exact exact_of(float top, const Scale& s) {
  return {top, s.hi, s.lo, fmaxf(top - 100.0f / s.hi, -FLT_MAX)};
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 less(float2 a, float2 b) { return __ffma2_rn(b, both(-1.f), a); }

// W of two logits (NaN and -inf: 0), `table` kPow2's entries.
__device__ __forceinline__ void exact_weights(float2 at, const Exact& s, const HiLo* table, float2& h, float2& l) {
  const float2 x = make_float2(fmaxf(at.x, s.least), fmaxf(at.y, s.least)), nm = both(-s.top);
  const float2 t = __fadd2_rn(x, nm), b = less(t, x);
  const float2 tl = __fadd2_rn(less(x, less(t, b)), less(nm, b));
  const float2 y = __fmul2_rn(t, both(s.hi));
  float2 yl = __ffma2_rn(t, both(s.hi), make_float2(-y.x, -y.y));
  yl = __ffma2_rn(t, both(s.lo), yl);
  yl = __ffma2_rn(tl, both(s.hi), yl);
  constexpr float kRound = 12288.0f;  // 1.5 * 2^13: neighbours are 1 / 1024 apart
  const float2 k = __fadd2_rn(y, both(kRound));
  const float2 g = less(y, __fadd2_rn(k, both(-kRound)));
  const uint32_t kx = __float_as_uint(k.x), ky = __float_as_uint(k.y);
  const HiLo tx = table[kx % kCells], ty = table[ky % kCells];
  // k div 1024 + kUnitBits as an exponent
  constexpr uint32_t kBias = ((uint32_t)(127 + kUnitBits) * kCells - 0x46400000u) << 13;
  const uint32_t ux = (kx * 8192u + kBias) & 0xff800000u, uy = (ky * 8192u + kBias) & 0xff800000u;
  const float2 unit = make_float2(__uint_as_float(at.x >= s.least ? ux : 0u), __uint_as_float(at.y >= s.least ? uy : 0u));
  constexpr double kLn2 = 0.69314718055994530942;
  constexpr float kLnHi = (float)kLn2, kLnLo = (float)(kLn2 - (double)kLnHi);
  const float2 z = __fmul2_rn(g, both(kLnHi));
  float2 zl = __ffma2_rn(g, both(kLnHi), make_float2(-z.x, -z.y));
  zl = __ffma2_rn(g, both(kLnLo), zl);
  zl = __ffma2_rn(yl, both(kLnHi), zl);
  const float2 e = __fadd2_rn(z, zl);
  zl = __ffma2_rn(__fmul2_rn(e, e), __ffma2_rn(e, both(1.0f / 6), both(0.5f)), zl);  // e^(z + zl) - 1 - z
  const float2 th = make_float2(tx.h, ty.h), tt = make_float2(tx.l, ty.l);
  const float2 p = __fmul2_rn(th, z);
  float2 rest = __fadd2_rn(__ffma2_rn(th, z, make_float2(-p.x, -p.y)), tt);
  rest = __ffma2_rn(tt, z, rest);
  rest = __ffma2_rn(th, zl, rest);
  h = __fadd2_rn(th, p);
  l = __fadd2_rn(less(p, less(h, th)), rest);
  h = __fmul2_rn(h, unit);
  l = __fmul2_rn(l, unit);
}
// max(W - G q, 0), G in two parts.
__device__ __forceinline__ void exact_rest(float2& h, float2& l, float2 q, float gh, float gl) {
  const float2 p = __fmul2_rn(q, both(gh));
  const float2 pl = __ffma2_rn(q, both(gl), __ffma2_rn(q, both(gh), make_float2(-p.x, -p.y)));
  const float2 d = less(h, p);
  const float2 e = less(less(h, d), p);  // exact wherever the rest may be above zero
  l = __fadd2_rn(e, less(l, pl));
  h = d;
  if (!(h.x + l.x > 0.f)) h.x = l.x = 0.f;  // (an infinite q too)
  if (!(h.y + l.y > 0.f)) h.y = l.y = 0.f;
}
// Nearest whole number, by its bits (below 2^63; a conversion to 64 bits takes 64 cycles of a warp).
__device__ __forceinline__ int64_t nearest(float x) {
  const int32_t bits = __float_as_int(x), up = ((bits >> 23) & 255) - 150;
  const uint32_t digits = ((uint32_t)bits & 0x7fffffu) | 0x800000u;
  const uint64_t v = up >= 0 ? (uint64_t)digits << up : up > -25 ? (uint64_t)((digits + (1u << (-up - 1))) >> -up) : 0;
  return bits < 0 ? -(int64_t)v : (int64_t)v;
}
__device__ __forceinline__ u64 whole(float h, float l) { return (u64)max((int64_t)0, nearest(h) + nearest(l)); }
// (h, l) += (x, xl), by an exact sum of the heads
__device__ __forceinline__ void add_exact(float2& h, float2& l, float2 x, float2 xl) {
  const float2 s = __fadd2_rn(h, x), b = less(s, h);
  l = __fadd2_rn(__fadd2_rn(l, xl), __fadd2_rn(less(h, less(s, b)), less(x, b)));
  h = s;
}

using u128 = unsigned __int128;
__device__ __forceinline__ u128 make_u128(u64 hi, u64 lo) { return (u128)hi << 64 | lo; }
__device__ __forceinline__ double to_double(u128 v) { return (double)(u64)(v >> 64) * 0x1p64 + (double)(u64)v; }
__device__ __forceinline__ u128 warp_scan_u128(u128 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u128 u = make_u128(__shfl_up_sync(kFullMask, (u64)(v >> 64), o), __shfl_up_sync(kFullMask, (u64)v, o));
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ u128 shfl_u128(u128 v, int lane) {
  return make_u128(shfl_u64((u64)(v >> 64), lane), shfl_u64((u64)v, lane));
}
// The whole part of u times a sum (numbers outside [0, 1), and NaN, go to the nearest end).
__device__ __forceinline__ u128 part_of_u128(float u, u128 total) {
  if (!(u > 0.f) || total == 0) return 0;
  if (u >= 1.f) return total - 1;
  const uint32_t bits = __float_as_uint(u), ex = bits >> 23;
  const uint32_t digits = ex ? (bits & 0x7fffffu) | 0x800000u : bits;  // u = digits 2^-down
  const uint32_t down = 150u - max(ex, 1u);
  return down < 128u ? (u128)digits * total >> down : 0;
}

// Draft probabilities beside a vector of logits, the first at element i of the row.
template <typename Q, int VEC>
__device__ __forceinline__ void load_draft(const Q* row, int vocab, int i, float (&q)[VEC]) {
  constexpr int bytes = VEC * (int)sizeof(Q);
  constexpr int step = bytes < 16 ? bytes : 16, per = step / (int)sizeof(Q);
  if (i >= 0 && i + VEC <= vocab && reinterpret_cast<uintptr_t>(row + i) % step == 0) {
#pragma unroll
    for (int k = 0; k < bytes / step; ++k) {
      alignas(16) Q e[per];
      if constexpr (step == 16) *reinterpret_cast<uint4*>(e) = reinterpret_cast<const uint4*>(row + i)[k];
      else *reinterpret_cast<uint2*>(e) = reinterpret_cast<const uint2*>(row + i)[k];
#pragma unroll
      for (int u = 0; u < per; ++u) q[k * per + u] = fmaxf(to_f32<Q>(e[u]), 0.f);
    }
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) q[k] = i + k >= 0 && i + k < vocab ? fmaxf(to_f32<Q>(row[i + k]), 0.f) : 0.f;
  }
}

// A pass over a row by a cluster: sums of max(W - G q, 0), a vector of a piece each.
struct Pass {
  int row;        // -1: no more
  float top;
  float gh, gl;   // G; 0: sums of W
};

// The numbers of one vector, by a warp.  REST: G is not 0.  (No branch among its pairs: they run side by side.)
template <typename T, typename Q, bool REST>
struct Vector {
  static constexpr int VEC = Piece<T>::VEC, NV = Piece<T>::NV;
  uint4 raw;
  float q[VEC];
  __device__ __forceinline__ void load(const VerifyArgs& a, const Piece<T>& p, const Pass& now, int k, int lane) {
    raw = p.load_one(k / NV, k % NV, lane);
    if constexpr (REST)
      load_draft<Q, VEC>(static_cast<const Q*>(a.draft) + now.row * a.draft_stride, a.vocab, p.first(k / NV, k % NV, lane), q);
  }
  // elements e and e + 1
  __device__ __forceinline__ void pair(const Pass& now, const Exact& ex, const HiLo* table, int e, float2& h, float2& l) const {
    exact_weights(Piece<T>::pair_of(raw, e), ex, table, h, l);
    if constexpr (REST) exact_rest(h, l, make_float2(q[e], q[e + 1]), now.gh, now.gl);
  }
  // the lane's sum
  __device__ __forceinline__ u64 sum(const Pass& now, const Exact& ex, const HiLo* table) const {
    float2 h, l;
    pair(now, ex, table, 0, h, l);
#pragma unroll
    for (int e = 2; e < VEC; e += 2) {
      float2 x, xl;
      pair(now, ex, table, e, x, xl);
      add_exact(h, l, x, xl);
    }
    const float s = h.x + h.y, b = s - h.x;
    return whole(s, (l.x + l.y) + ((h.x - (s - b)) + (h.y - b)));
  }
};

// A pass by the warps of a cluster: warp i takes vectors i * share .. and leaves their sums in `rest`;
// its own is returned.  (A function of its own: the walk's state would take the registers of its loop.)
template <typename T, typename Q, bool REST>
__device__ __noinline__ u128 pass_over(const VerifyArgs& a, const Pass now, const Exact ex, u64* rest, int vectors, int share,
                                       int gwarp, const HiLo* table, int lane) {
  using V = Vector<T, Q, REST>;
  const int end = min(vectors, (gwarp + 1) * share);
  Piece<T> p;
  p.open(a, now.row);
  V v;
  u128 all = 0;
  int k = gwarp * share;
  if (k < end) v.load(a, p, now, k, lane);
#pragma unroll 1
  for (; k < end; ++k) {
    const V here = v;
    if (k + 1 < end) v.load(a, p, now, k + 1, lane);
    const u64 sum = warp_sum_u64(here.sum(now, ex, table));
    if (lane == 0) __stcg(rest + k, sum);
    all += sum;
  }
  return all;
}

constexpr int kMaxWarps = kWalkCtas * kWalkWarps;  // of a cluster
struct WarpSum {
  u64 hi, lo;
};
__device__ __forceinline__ u128 sum_of(const WarpSum& x) { return make_u128(x.hi, x.lo); }

// The first of n numbers whose running sum passes `left`, by a warp (there is one); `left` becomes the rest
// in it.
template <typename F>
__device__ __forceinline__ int find_sum(int n, int lane, u128& left, F number) {
  const int per = (n + 31) / 32;
  u128 part = 0;
  for (int k = lane * per; k < min(n, (lane + 1) * per); ++k) part += number(k);
  const u128 incl = warp_scan_u128(part, lane);
  const unsigned hit = __ballot_sync(kFullMask, incl > left);
  const int src = hit ? __ffs(hit) - 1 : 31;
  u128 rest = left - (incl - part);
  int found = 0;
  if (lane == src) {
    for (int k = lane * per; k < min(n, (lane + 1) * per); ++k) {
      const u128 x = number(k);
      found = k;
      if (x > rest) break;
      rest -= x;
    }
  }
  left = shfl_u128(rest, src);
  return __shfl_sync(kFullMask, found, src);
}

// The first token whose running sum passes u times the whole `total`, by a warp, from the sums of a pass.
template <typename T, typename Q, bool REST>
__device__ __noinline__ int draw_exact(const VerifyArgs& a, const Pass& now, const Scale& s, const WarpSum* warp_sums, int warps,
                                       const u64* rest, int vectors, int share, u128 total, float u, const HiLo* table,
                                       int lane) {
  using V = Vector<T, Q, REST>;
  if (total == 0) return kNoPick;
  u128 left = part_of_u128(u, total);
  const int first = share * find_sum(warps, lane, left, [&](int i) { return sum_of(warp_sums[i]); });
  const int k = first + find_sum(min(share, vectors - first), lane, left, [&](int i) { return (u128)__ldcg(rest + first + i); });
  const u64 target = (u64)left;
  Piece<T> p;
  p.open(a, now.row);
  V v;
  v.load(a, p, now, k, lane);
  const Exact ex = exact_of(now.top, s);
  u64 values[V::VEC], sum = 0;
  int tail = -1;
#pragma unroll
  for (int e = 0; e < V::VEC; e += 2) {
    float2 h, l;
    v.pair(now, ex, table, e, h, l);
    values[e] = (u64)max(0ll, __float2ll_rn(h.x) + __float2ll_rn(l.x));
    values[e + 1] = (u64)max(0ll, __float2ll_rn(h.y) + __float2ll_rn(l.y));
    sum += values[e] + values[e + 1];
    if (values[e]) tail = e;
    if (values[e + 1]) tail = e + 1;
  }
  const u64 upto = warp_scan_u64(sum, lane);
  const unsigned hit = __ballot_sync(kFullMask, upto > target), some = __ballot_sync(kFullMask, tail >= 0);
  if ((hit | some) == 0) return kNoPick;  // (logits that changed under the call)
  // where the sum's rounding leaves no token: the last with a weight
  const int who = hit ? __ffs(hit) - 1 : 31 - __clz(some);
  u64 at = upto - sum;
  int which = -1;
#pragma unroll
  for (int e = 0; e < V::VEC; ++e) {
    at += values[e];
    if (which < 0 && at > target) which = e;
  }
  if (which < 0) which = tail;
  return p.first(k / V::NV, k % V::NV, who) + __shfl_sync(kFullMask, which, who);
}

// ---------------------------------------------------------------- the walk by clusters

constexpr int kMaxClusters = 1024;     // of a launch (each has its sums in the workspace)
// fp32 tells that a drafted token is kept where u q S is below W by more than this share: S is off by
// less than 2^-17 (see kSumError, kPowError: 30 2^-23), W by 2^-22 + 0.7 2^-23 |y|, |y| < 150.
constexpr float kKeptNear = 0x1p-15f;

// A cluster takes sequences in turn: all of them, or (`listed`) those that verify_pick_kernel left.
//
// With draft probabilities, in whole numbers: W the weights of node c, N their sum and G = 0 at first.
// Child x is kept when u q(x) N < W_x - G q(x); refused, G becomes G + N and N the sum of max(W - G q,
// 0) (both stay where that is 0): r = max(W - G q, 0) / N, as max(max(x, 0) - q, 0) = max(x - q, 0) for
// q >= 0.  fp32 sums of the first launch decide where they can: on children kept, and on the token that
// follows a node of which no child was refused.
//
// The first CTA of a cluster works out the rows and walks; the others take their share of the passes over
// a row, told by the first alone which sequence, which row and with what G, so that all meet at the same
// barriers whatever the buffers hold.
template <typename T, typename Q, bool DRAFT>
__global__ void __launch_bounds__(kWalkWarps * 32, 2) verify_walk_kernel(const __grid_constant__ VerifyArgs a, const __grid_constant__ VerifyWork w, int listed) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (a CTA's shared memory may be written by another once it runs)
  auto started = cluster.barrier_arrive();
  constexpr int threads = kWalkWarps * 32;
  const int warps = ranks * kWalkWarps, gwarp = rank * kWalkWarps + warp, vectors = w.pieces * Piece<T>::NV;
  const int share = (vectors + warps - 1) / warps;  // vectors of a warp
  __shared__ __align__(16) HiLo table[kCells];
  __shared__ float2 held[kWalkWarps][kHeld];
  __shared__ int32_t node_room[2][kNodes], pick_room[kNodes];
  __shared__ float4 row_room[kNodes];
  __shared__ float2 pq_room[kNodes];
  __shared__ Pass todo;
  __shared__ int turn;
  __shared__ WarpSum warp_sums[kMaxWarps];
  for (int i = threadIdx.x; i < kCells / 2; i += threads)
    reinterpret_cast<float4*>(table)[i] = __ldg(reinterpret_cast<const float4*>(&kPow2) + i);
  const bool walks = rank == 0 && warp == 0;
  u64* rest = w.rest + (int64_t)(blockIdx.x / ranks) * vectors;
  const float near = kKeptNear + (float)w.pieces / row_unit(a.vocab);  // (roundings to the unit)
  cluster.barrier_wait(std::move(started));
  if (listed) asm volatile("griddepcontrol.wait;\n" ::: "memory");

  for (int at = blockIdx.x / ranks; at < a.num_seqs; at += gridDim.x / ranks) {
    int s = at;
    if (listed) {
      if (walks) {
        s = at < __ldcg(w.list) ? __ldcg(w.list + 1 + at) : -1;
        if (s >= a.num_seqs) s = -1;
        if (lane < ranks) *cluster.map_shared_rank(&turn, lane) = s;
      }
      cluster.sync();
      s = turn;
      if (s < 0) break;
    }
    const float temp = a.temperature ? a.temperature[s] : 1.f;
    const bool greedy = is_greedy(temp);
    const Scale sc = scale_of(greedy ? 1.f : temp);
    int r0 = 0, n = 0;
    Nodes nodes;
    float4* rows = row_room;
    float2* pqs = pq_room;
    if (rank == 0 || (!DRAFT && !listed)) n = rows_of(a, s, r0);
    if (rank == 0) {
      if (!listed) check_sequence(a, s, r0, n, threadIdx.x, threads);
      nodes.open(a, r0, n, node_room, threads);
      if (n > kNodes) {
        rows = reinterpret_cast<float4*>(w.rows + r0);
        pqs = w.pq + r0;
      }
    }
    if (!listed) asm volatile("griddepcontrol.wait;\n" ::: "memory");
    bool none = false;
    if constexpr (!DRAFT) {
      if (listed) {
        if (rank == 0 && n <= kNodes)
          for (int i = threadIdx.x; i < n; i += threads) pick_room[i] = __ldcg(&w.rows[r0 + i].pick);
      } else {
        for (int i = gwarp; i < n; i += warps) {
          const int64_t r = r0 + i;
          const float2* st = hold_stats(w, r, held[warp], lane);
          const float top = row_top(st, w.pieces, lane);
          int pick = kNoPick;
          if (!has_distribution(w, r, s, top)) none = true;
          else if (greedy) pick = row_best(st, w.pieces, lane, top);
          else pick = draw_token<T>(a, w, st, r, top, sc, a.u_sample[r], lane);
          if (lane == 0) {
            if (n <= kNodes) *cluster.map_shared_rank(&pick_room[i], 0) = pick;
            else __stcg(&w.rows[r].pick, pick);
          }
        }
      }
      cluster.sync();
    } else if (rank == 0) {
      // rows' largest logits, sums and, greedy, first largest logits
      for (int i = warp; i < n; i += kWalkWarps) {
        const float2* st = hold_stats(w, r0 + i, held[warp], lane);
        const float top = row_top(st, w.pieces, lane);
        float all = 0.f;
        int pick = kNoPick;
        if (!has_distribution(w, r0 + i, s, top)) {
          none = true;
        } else if (greedy) {
          pick = row_best(st, w.pieces, lane, top);
        } else {
          const float unit = row_unit(a.vocab);
          u64 sum = 0;
          for (int k = lane; k < w.pieces; k += 32) sum += fixed(st[k].y * weight(st[k].x, top, sc), unit);
          all = (float)warp_sum_u64(sum) / unit;
          pick = 0;
        }
        if (lane == 0) rows[i] = make_float4(top, all, __int_as_float(pick), 0.f);
      }
      __syncthreads();
      // weight and q of every drafted token
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
            pq.x = weight(x, info.x, sc);
          }
        }
        pqs[i] = pq;
      }
      __syncthreads();
    }
    if (none && a.status && lane == 0) atomicMax(a.status, (int32_t)kInvalidArg);

    // The walk, by the first CTA's first warp.
    int32_t* path = a.path + (int64_t)s * a.max_path;
    int c = 0, from = 1, len = 0, next = kNoPick;
    bool exact = false, holds = false;  // N is; the sums of the last pass are those of G at node c
    double G = 0.0, N = 0.0;
    u128 total = 0;  // of the last pass
    float4 info = make_float4(0.f, 0.f, __int_as_float(kNoPick), 0.f);
    if (walks && n > 0) {
      if (lane == 0) path[0] = 0;
      len = 1;
      if constexpr (DRAFT) info = rows[0];
    }
    auto pass_of = [&](double g) {
      const float gh = (float)g;
      return Pass{r0 + c, info.x, gh, (float)(g - (double)gh)};
    };
    auto drawn = [&] {
      const Pass now = pass_of(G);
      const float u = a.u_sample[r0 + c];
      if constexpr (DRAFT) {
        if (G > 0.0) return draw_exact<T, Q, true>(a, now, sc, warp_sums, warps, rest, vectors, share, total, u, table, lane);
      }
      return draw_exact<T, Q, false>(a, now, sc, warp_sums, warps, rest, vectors, share, total, u, table, lane);
    };
    // Goes on as far as it can: the G of the pass that it needs, -1 at the end.
    auto walk = [&]() -> double {
      if (n == 0) return -1.0;
      if constexpr (!DRAFT) {
        while (true) {
          next = n <= kNodes ? pick_room[c] : __ldcg(&w.rows[r0 + c].pick);
          if (next == kUnsure) {
            if (!holds) {
              info.x = row_top(hold_stats(w, r0 + c, held[0], lane), w.pieces, lane);
              return 0.0;
            }
            next = drawn();
          }
          if (next < 0 || len == a.max_path) return -1.0;
          const int child = nodes.next_child(c, c + 1, lane, [&](int i) { return nodes.tokens[i] == next; });
          if (child < 0) return -1.0;
          c = child;
          holds = false;
          if (lane == 0) path[len] = c;
          ++len;
        }
      } else {
        while (__float_as_int(info.z) >= 0 && len < a.max_path) {
          const int child = nodes.next_child(c, from, lane, [](int) { return true; });
          if (child < 0) break;
          const float2 pq = pqs[child];
          bool kept;
          if (greedy) {
            kept = pq.x > 0.f;
          } else {
            const int tok = nodes.tokens[child];
            if (tok < 0 || tok >= a.vocab) {  // not drawn from q
              from = child + 1;
              continue;
            }
            const float u = a.u_accept[r0 + child];
            if (!exact) {
              kept = pq.x * (1.f - near) - u * pq.y * info.y > 0x1p-110f;
              if (!kept) return 0.0;
            } else {
              const float x = to_f32<T>(static_cast<const T*>(a.logits)[(int64_t)(r0 + c) * a.logits_stride + tok]);
              float2 h, l;
              exact_weights(both(x), exact_of(info.x, sc), table, h, l);
              const double r = (double)h.x + (double)l.x - (G > 0.0 ? G * pq.y : 0.0);
              kept = r > 0.0 && (double)u * pq.y * N < r;
            }
          }
          if (kept) {
            c = child;
            from = c + 1;
            exact = holds = false;
            G = N = 0.0;
            info = rows[c];
            if (lane == 0) path[len] = c;
            ++len;
          } else {
            from = child + 1;
            if (!greedy) return G + N;
          }
        }
        if (__float_as_int(info.z) < 0 || greedy) {
          next = __float_as_int(info.z);
        } else if (!exact) {
          const int64_t r = r0 + c;
          next = draw_token<T>(a, w, hold_stats(w, r, held[0], lane), r, info.x, sc, a.u_sample[r], lane);
          if (next == kUnsure) return 0.0;
        } else {
          if (!holds) return G;
          next = drawn();
        }
        return -1.0;
      }
    };
    while (true) {
      double g = -1.0;
      if (walks) {
        g = walk();
        Pass ask = pass_of(g);
        if (g < 0.0) ask.row = -1;
        if (lane < ranks) *cluster.map_shared_rank(&todo, lane) = ask;
      }
      cluster.sync();
      const Pass now = todo;
      if (now.row < 0) break;
      u128 mine;
      if (DRAFT && now.gh > 0.f) mine = pass_over<T, Q, DRAFT>(a, now, exact_of(now.top, sc), rest, vectors, share, gwarp, table, lane);
      else mine = pass_over<T, Q, false>(a, now, exact_of(now.top, sc), rest, vectors, share, gwarp, table, lane);
      if (lane == 0) *cluster.map_shared_rank(&warp_sums[gwarp], 0) = WarpSum{(u64)(mine >> 64), (u64)mine};
      cluster.sync();
      if (walks) {
        u128 part = 0;
        for (int i = lane; i < warps; i += 32) part += sum_of(warp_sums[i]);
        total = shfl_u128(warp_scan_u128(part, lane), 31);
        const double sum = to_double(total);
        holds = true;
        if (!exact) {
          exact = true;
          N = sum;
        } else if (g > G) {
          if (sum > 0.0) G = g, N = sum;
          else holds = false;  // nothing is left: the distribution before the subtraction stays
        }
      }
    }
    if (walks) {
      for (int j = len + lane; j < a.max_path; j += 32) path[j] = -1;
      if (lane == 0) {
        a.path_lens[s] = len;
        a.next_token[s] = next;
      }
    }
    if (at + (int)(gridDim.x / ranks) < a.num_seqs) cluster.sync();
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
  w.rest = reinterpret_cast<u64*>(take((size_t)std::min(seqs, kMaxClusters) * w.pieces * 8 * sizeof(u64)));
  w.list = reinterpret_cast<int32_t*>(take(((size_t)seqs + 1) * sizeof(int32_t)));
  *bytes = at;
  return w;
}

// A kernel is a programmatic dependent of the one before: its set-up overlaps it.
template <typename K, typename... Args>
cudaError_t launch_after(K kern, int grid, int threads, int cluster, int smem, cudaStream_t stream, Args... args) {
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
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, args...);
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
  // as many CTAs a sequence as run at once, and as its rows' vectors keep busy
  const int vectors = w.pieces * Piece<T>::NV, threads = kWalkWarps * 32;
  int ctas_seq = kWalkCtas;
  while (ctas_seq > 1 && ctas_seq * kWalkWarps >= 2 * vectors) ctas_seq /= 2;
  int clusters = std::min(a.num_seqs, kMaxClusters);
  if (!a.draft && (int64_t)a.num_seqs * ctas_seq > 2 * sms) {
    // many sequences: a CTA each, with twice the warps of an average one's rows (ragged ones take one turn
    // too), and clusters for those that it leaves
    const int warps = std::max(1, std::min(kPickWarps, 2 * ((a.num_rows + a.num_seqs - 1) / a.num_seqs)));
    err = launch_after(verify_pick_kernel<T>, a.num_seqs, warps * 32, 1, warps * kHeld * (int)sizeof(float2), stream, a, w);
    if (err != cudaSuccess) return err;
    clusters = std::min(clusters, std::max(1, 2 * sms / ctas_seq));
    return launch_after(verify_walk_kernel<T, float, false>, clusters * ctas_seq, threads, ctas_seq, 0, stream, a, w, 1);
  }
  while (ctas_seq > 1 && (int64_t)a.num_seqs * ctas_seq > 2 * sms) ctas_seq /= 2;
  const int grid = clusters * ctas_seq;
  if (!a.draft) return launch_after(verify_walk_kernel<T, float, false>, grid, threads, ctas_seq, 0, stream, a, w, 0);
  switch (a.draft_dtype) {
    case kF32: return launch_after(verify_walk_kernel<T, float, true>, grid, threads, ctas_seq, 0, stream, a, w, 0);
    case kF16: return launch_after(verify_walk_kernel<T, __half, true>, grid, threads, ctas_seq, 0, stream, a, w, 0);
    case kBF16: return launch_after(verify_walk_kernel<T, __nv_bfloat16, true>, grid, threads, ctas_seq, 0, stream, a, w, 0);
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
