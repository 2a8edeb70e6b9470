// Norms of each query and key head with the position rotation, one pass, and the same on the
// way into the packed pages, sm_103a.
//
// TurboQuant docs: "vLLM Usage" (TQ Byte Layout, Slot Mapping: a token's row goes to its flat
// slot; TQ Packed Page Contract: write_tq4_kv encodes K and V rows).
//
// Per head row x of D channels, in fp32:
//   norm      x <- w x / sqrt(mean x^2 + eps)
//   rotation  (a, b) <- (a cos - b sin, b cos + a sin), pairs (i, i + r/2) or (2i, 2i + 1)
//   encoding  (K and V) nu = ||x||, y = H (s x) / (sqrt(D) nu), index = #{k : boundary_k < y},
//             packed LSB first, nu appended
// D / 16 lanes share a row.  Lane l holds channels 8 l .. 8 l + 7 and D / 2 + 8 l .. + 7: the
// pairs of either style lie in one lane, 16-byte loads cover 16-bit types, the transform has four
// stages inside a lane and log2(D / 16) by shuffles, and eight indices are `bits` whole bytes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "tq_append.h"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kAppendWarps = 8;
constexpr int kAppendCtas = 2;  // CTAs of an SM

struct AppendPlan {
  AppendArgs a;
  int per_item;         // groups of 32 / (D / 16) heads that a warp takes together
  int items[3];         // items of a token's q, k, v
  int items_per_token;
  int64_t step_t;       // tokens and items between two items of a warp
  int step_part;
  int vec;              // inputs and dense outputs: 16-byte accesses
  int table_vec;        // table rows: 16-byte loads
};

// Sum over the LPR lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = LPR / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int m = LPR / 2; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, m));
  return v;
}
__device__ __forceinline__ float sum_squares(const float2 (&x)[8]) {
  float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s0 = __ffma2_rn(x[i], x[i], s0);
    s1 = __ffma2_rn(x[i + 4], x[i + 4], s1);
  }
  return (s0.x + s0.y) + (s1.x + s1.y);
}

// A lane's two chunks of eight elements, as they lie in memory.
template <typename T>
struct Raw {
  static constexpr int N = 16 * (int)sizeof(T) / 16;
  uint4 w[N];
  // chunks at p and p + half, at any alignment
  __device__ __forceinline__ void load(const T* p, int half) {
    T* e = reinterpret_cast<T*>(w);
#pragma unroll
    for (int j = 0; j < 16; ++j) e[j] = p[j < 8 ? j : half + j - 8];
  }
  template <bool VEC>
  __device__ __forceinline__ void store(T* p, int half) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(p + (i < N / 2 ? 0 : half))[i % (N / 2)] = w[i];
    } else {
      const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
      for (int j = 0; j < 16; ++j) p[j < 8 ? j : half + j - 8] = e[j];
    }
  }
  __device__ __forceinline__ void get(float2 (&x)[8]) const {
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = make_float2(to_f32<T>(e[2 * i]), to_f32<T>(e[2 * i + 1]));
  }
  __device__ __forceinline__ void set(const float2 (&x)[8]) {
    T* e = reinterpret_cast<T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[2 * i] = from_f32<T>(x[i].x);
      e[2 * i + 1] = from_f32<T>(x[i].y);
    }
  }
};

// Eight floats at p (16-byte aligned with `vec`).
__device__ __forceinline__ void load8(const float* __restrict__ p, bool vec, float2 (&v)[4]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
      v[2 * i] = make_float2(f.x, f.y);
      v[2 * i + 1] = make_float2(f.z, f.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__ldg(p + 2 * i), __ldg(p + 2 * i + 1));
  }
}

// Largest power of two exponent of a row whose sum of squares leaves [2^-100, 2^100]: the row
// is scaled by 2^-ex (exact).  0 where the row is zero or not finite.
template <int LPR>
__device__ __forceinline__ int row_exponent(const float2 (&x)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
  m = row_max<LPR>(m);
  int ex = 0;
  if (m > 0.f && m <= 3.402823466e38f) frexpf(m, &ex);
  return ex;
}

// 1 / sqrt(mean x^2 + eps).  A row beyond the range of its squares is scaled by a power of two
// first, x with it.
template <int LPR>
__device__ __forceinline__ float norm_factor(float2 (&x)[8], float eps) {
  constexpr int D = 16 * LPR;
  float ss = row_sum<LPR>(sum_squares(x));
  // squares that underflow count only where eps is as small
  const bool odd = !(ss <= 0x1p100f) || (ss < 0x1p-100f && eps < 0x1p-80f);
  if (__any_sync(kFullMask, odd)) {
    int ex = row_exponent<LPR>(x);
    if (odd) {
      // eps in the scaled row's units stays below 2^100 (underflowing, it has no weight)
      if (ex < 0 && eps > 0.f) ex = max(ex, (ilogbf(eps) - 100) / 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = make_float2(scale_pow2(x[i].x, -ex), scale_pow2(x[i].y, -ex));
      eps = ldexpf(eps, -2 * ex);
    }
    const float again = row_sum<LPR>(sum_squares(x));
    if (odd) ss = again;
  }
  return rsqrtf(fmaf(ss, 1.0f / D, eps));
}

// What a token's rows are multiplied by: y[i] = x[i] p[i] + other(x)[i] s[i], weights, signs and
// rotation in one.  `mode` says where the other channel of a pair lies.
enum Mode { kPlain, kHalves, kPairs, kStaged };  // (no pair; slot i ^ 4; the same float2; by shared memory)
struct Coef {
  float2 p[8], s[8];
};

// Coefficients of a token: weights `w` (null: 1), signs `sg` (null: 1), the position's table row `cs`
// (null: no rotation).  Channel e's other one is e +- rot / 2, or e ^ 1.
template <int LPR>
__device__ __forceinline__ void token_coef(Coef& f, int mode, const float* __restrict__ w, const float* __restrict__ sg,
                                           const float* __restrict__ cs, int rot, bool tvec, int l) {
  constexpr int D = 16 * LPR;
  const int half = rot / 2;
  const float2 one = make_float2(1.f, 1.f);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int e0 = c * (D / 2) + 8 * l;  // the chunk's first channel
    float2 wv[4], cv[4], sv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wv[i] = cv[i] = one, sv[i] = make_float2(0.f, 0.f);
    if (w) load8(w + e0, true, wv);
    if (mode == kPairs) {
      const int p0 = e0 / 2;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p0 + i < half) {
          const float a = __ldg(cs + p0 + i), b = __ldg(cs + half + p0 + i);
          cv[i] = make_float2(a, a);
          sv[i] = __fmul2_rn(make_float2(wv[i].y, wv[i].x), make_float2(-b, b));
        }
    } else if (mode == kHalves || (mode == kStaged && rot % 16 == 0)) {
      if (e0 < rot) {  // the whole chunk is of one half
        const bool first = e0 < half;
        const int p0 = first ? e0 : e0 - half;
        float2 ow[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ow[i] = one;
        if (w) load8(w + (first ? e0 + half : p0), true, ow);
        load8(cs + p0, tvec, cv);
        load8(cs + half + p0, tvec, sv);
        const float2 sign = first ? make_float2(-1.f, -1.f) : one;
#pragma unroll
        for (int i = 0; i < 4; ++i) sv[i] = __fmul2_rn(__fmul2_rn(sv[i], sign), ow[i]);
      }
    } else if (mode == kStaged) {
      float* cf = reinterpret_cast<float*>(cv);
      float* sf = reinterpret_cast<float*>(sv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        if (e >= rot) continue;
        const bool first = e < half;
        const int p = first ? e : e - half;
        const float ow = w ? __ldg(w + (first ? e + half : p)) : 1.f;
        cf[i] = __ldg(cs + p);
        sf[i] = (first ? -ow : ow) * __ldg(cs + half + p);
      }
    }
    float2 g[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = one;
    if (sg) load8(sg + e0, false, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.p[4 * c + i] = __fmul2_rn(__fmul2_rn(wv[i], cv[i]), g[i]);
      f.s[4 * c + i] = __fmul2_rn(sv[i], g[i]);
    }
  }
}

template <int LPR>
__device__ __forceinline__ void apply_coef(float2 (&x)[8], const Coef& f, int mode, int rot, int l, float* mine) {
  constexpr int D = 16 * LPR;
  if (mode == kPlain) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], f.p[i]);
  } else if (mode == kHalves) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = x[i], b = x[4 + i];
      x[i] = __ffma2_rn(a, f.p[i], __fmul2_rn(b, f.s[i]));
      x[4 + i] = __ffma2_rn(b, f.p[4 + i], __fmul2_rn(a, f.s[4 + i]));
    }
  } else if (mode == kPairs) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __ffma2_rn(x[i], f.p[i], __fmul2_rn(make_float2(x[i].y, x[i].x), f.s[i]));
  } else {
    const int half = rot / 2;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      *reinterpret_cast<float4*>(mine + (i >> 2) * (D / 2) + 8 * l + 2 * (i & 3)) =
          make_float4(x[i].x, x[i].y, x[i + 1].x, x[i + 1].y);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int e0 = c * (D / 2) + 8 * l;
      float2 other[4];
      if (rot % 16 == 0) {
        const float4* at = reinterpret_cast<const float4*>(mine + (e0 < half ? e0 + half : e0 < rot ? e0 - half : e0));
        const float4 u = at[0], v = at[1];
        other[0] = make_float2(u.x, u.y), other[1] = make_float2(u.z, u.w);
        other[2] = make_float2(v.x, v.y), other[3] = make_float2(v.z, v.w);
      } else {
        float* o = reinterpret_cast<float*>(other);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = e0 + i;
          o[i] = mine[e < half ? e + half : e < rot ? e - half : e];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[4 * c + i] = e0 + 2 * i < rot ? __ffma2_rn(x[4 * c + i], f.p[4 * c + i], __fmul2_rn(other[i], f.s[4 * c + i]))
                                        : __fmul2_rn(x[4 * c + i], f.p[4 * c + i]);
    }
  }
}

// Unnormalised Walsh-Hadamard transform of a row (natural order; the stages commute).
template <int LPR>
__device__ __forceinline__ void fwht_row(float2 (&x)[8], int l) {
  const float2 minus1 = make_float2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = make_float2(x[i].x + x[i].y, x[i].x - x[i].y);
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)  // h = 1, 2: inside a chunk; 4: between the two chunks
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & h) == 0) {
        const float2 a = x[i], b = x[i + h];
        x[i] = __fadd2_rn(a, b);
        x[i + h] = __ffma2_rn(b, minus1, a);
      }
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) {
    const float sg = (l & m) ? -1.f : 1.f;
    const float2 s2 = make_float2(sg, sg);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 p = make_float2(__shfl_xor_sync(kFullMask, x[i].x, m), __shfl_xor_sync(kFullMask, x[i].y, m));
      x[i] = __ffma2_rn(x[i], s2, p);
    }
  }
}

// Quantiser of a codebook.  128 equal cells cover the decision points' span; a cell holds the
// number of points in cells before it, so the index is that and one comparison for each point that
// the cell itself may hold (`steps`, the most of any cell: 1 for a Lloyd-Max codebook).  Cells come
// from one monotone function of u for points and coordinates alike, so its rounding does not
// matter.  32 words of counts and at most 32 points: neither lookup has bank conflicts.
struct Quant {
  float point[32];      // decision points, then +inf
  uint8_t below[128];   // 4 * (points in cells before this one)
  float mul, add;       // span to [0, 1]
  int steps;
};
// 127 times the clamped coordinate, as the bits of a subnormal: the cell's number
__device__ __forceinline__ uint32_t cell_of(float u, float mul, float add) {
  float t;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(t) : "f"(u), "f"(mul), "f"(add));  // NaN: 0
  return __float_as_uint(t * 0x1.fcp-143f);  // 127 * 2^-149
}
// Set up by a warp from n = 2^bits ascending centroids (points: rounded midpoints).
__device__ __forceinline__ void build_quant(Quant& q, const float* __restrict__ c, int n, int lane) {
  const float pt = lane < n - 1 ? 0.5f * (__ldg(c + lane) + __ldg(c + lane + 1)) : __int_as_float(0x7f800000);
  const float lo = __shfl_sync(kFullMask, pt, 0), hi = __shfl_sync(kFullMask, pt, n - 2);
  const float mul = hi > lo ? 1.0f / (hi - lo) : 0.f, add = -lo * mul;
  const int cell = lane < n - 1 ? (int)cell_of(pt, mul, add) : 128;
  q.point[lane] = pt;
  int most = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int below = 0, here = 0;
    for (int k = 0; k < n - 1; ++k) {
      const int ck = __shfl_sync(kFullMask, cell, k);
      below += ck < lane + 32 * j;
      here += ck == lane + 32 * j;
    }
    q.below[lane + 32 * j] = (uint8_t)(4 * below);
    most = max(most, here);
  }
  most = __reduce_max_sync(kFullMask, most);
  if (lane == 0) q.mul = mul, q.add = add, q.steps = most;
}

// Encodes rows of signed coordinates x, whose own norm is `factor` times theirs (all lanes of the
// warp take part; `dst` null: nothing stored).
template <int LPR, int B>
__device__ __forceinline__ void encode_row(float2 (&x)[8], float factor, const Quant& q, int l, uint8_t* dst) {
  constexpr int D = 16 * LPR, IB = D * B / 8;
  float ss = row_sum<LPR>(sum_squares(x));
  int ex = 0;
  bool bad = false;
  const bool odd = !(ss <= 0x1p100f) || ss < 0x1p-100f;
  if (__any_sync(kFullMask, odd)) {
    const int e = row_exponent<LPR>(x);
    if (odd) {
      ex = e;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = make_float2(scale_pow2(x[i].x, -ex), scale_pow2(x[i].y, -ex));
    }
    const float again = row_sum<LPR>(sum_squares(x));
    if (odd) ss = again;
    bad = !(ss <= 3.402823466e38f);  // a NaN or infinite coordinate: a zero row's indices
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (bad) x[i] = make_float2(0.f, 0.f);
  }
  const float rs = (ss > 0.f && !bad) ? rsqrtf(ss) : 0.f;
  const float nu = bad ? ss : scale_pow2(ss * rs * factor, ex);
  fwht_row<LPR>(x, l);
  constexpr float kInvSqrtD = LPR == 1 ? 0.25f : LPR == 2 ? 0.17677669529663689f : LPR == 4 ? 0.125f
                              : LPR == 8 ? 0.088388347648318447f : 0.0625f;
  const float inv = rs * kInvSqrtD;
  const float2 inv2 = make_float2(inv, inv);
  const float mul = q.mul, add = q.add;
  const int steps = q.steps;
  const unsigned char* below = q.below;
  const unsigned char* point = reinterpret_cast<const unsigned char*>(q.point);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], inv2);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    using Word = typename std::conditional<(B > 4), uint64_t, uint32_t>::type;
    Word word = 0;  // 4 times the indices
    if (steps == 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = (j & 1) ? x[4 * c + j / 2].y : x[4 * c + j / 2].x;
        const uint32_t four = below[cell_of(u, mul, add)];
        const bool up = u > *reinterpret_cast<const float*>(point + four);
        if (j == 0) word = (four >> 2) + (up ? 1 : 0);
        else word += ((Word)four << (B * j - 2)) + (up ? (Word)1 << (B * j) : 0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = (j & 1) ? x[4 * c + j / 2].y : x[4 * c + j / 2].x;
        uint32_t four = below[cell_of(u, mul, add)];
        for (int k = 0; k < steps; ++k)
          if (u > *reinterpret_cast<const float*>(point + four)) four += 4;
        word |= (Word)(four >> 2) << (B * j);
      }
    }
    // a chunk's B bytes: whole words where the lanes of a row's quad share them
    uint8_t* at = dst + c * (IB / 2) + B * l;
    if constexpr (B == 4) {
      if (dst) *reinterpret_cast<uint32_t*>(at) = word;
    } else if constexpr (B == 2 && LPR >= 2) {
      const uint32_t next = __shfl_down_sync(kFullMask, word, 1);
      if (dst && (l & 1) == 0) *reinterpret_cast<uint32_t*>(at) = word | next << 16;
    } else if constexpr (B == 3 && LPR >= 4) {
      const uint32_t next = __shfl_down_sync(kFullMask, word, 1);
      const int k = l & 3;  // word k of three: 24 bits of lane k less 8 k, then lane k + 1's
      if (dst && k < 3) *reinterpret_cast<uint32_t*>(at + k) = word >> (8 * k) | next << (24 - 8 * k);
    } else if constexpr (B == 5 && LPR >= 4) {
      const uint64_t before = __shfl_up_sync(kFullMask, word, 1);
      const int k = l & 3;  // word k of five: the last 8 k bits of lane k - 1, then lane k's
      if (dst) {
        *reinterpret_cast<uint32_t*>(at - k) = (uint32_t)(word << (8 * k) | (k ? before >> (40 - 8 * k) : 0));
        if (k == 3) *reinterpret_cast<uint32_t*>(at + 1) = (uint32_t)(word >> 8);
      }
    } else if (dst) {
#pragma unroll
      for (int k = 0; k < B; ++k) at[k] = (uint8_t)(word >> (8 * k));
    }
  }
  if (dst && l == 0) {
    if constexpr (D == 16) {  // rows of 8 to 14 bytes: 2-byte aligned
      const uint32_t w = __float_as_uint(nu);
      *reinterpret_cast<uint16_t*>(dst + IB) = (uint16_t)w;
      *reinterpret_cast<uint16_t*>(dst + IB + 2) = (uint16_t)(w >> 16);
    } else {
      *reinterpret_cast<float*>(dst + IB) = nu;
    }
  }
}

__device__ __forceinline__ uint32_t smem_address(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// Groups of rows in flight of a warp, 1 KB (16-bit types) or 2 KB each.
template <typename T>
__host__ __device__ constexpr int stages() {
  return sizeof(T) == 2 ? 4 : 3;
}
// Dynamic shared memory: the copies in flight, and room to exchange pairs.
template <typename T>
__host__ __device__ constexpr int ring_bytes() {
  return kAppendWarps * stages<T>() * 32 * 16 * (int)sizeof(T);
}
constexpr int kStageBytes = kAppendWarps * 512 * 4;

// One side of a token, or some of its groups of heads.
template <typename T, int LPR>
struct Item {
  int64_t t;
  int part, side, heads, g, end;
  const T* src;  // this lane's elements of group 0's first row
  __device__ __forceinline__ void open(const AppendPlan& p, int l) {
    constexpr int RPW = 32 / LPR;
    const AppendArgs& a = p.a;
    side = part < p.items[0] ? 0 : part < p.items[0] + p.items[1] ? 1 : 2;
    g = (part - (side > 0 ? p.items[0] : 0) - (side > 1 ? p.items[1] : 0)) * p.per_item;
    heads = side == 0 ? a.num_q_heads : side == 1 ? a.num_k_heads : a.num_v_heads;
    end = min((heads + RPW - 1) / RPW, g + p.per_item);
    src = static_cast<const T*>(side == 0 ? a.q : side == 1 ? a.k : a.v) +
          t * (side == 0 ? a.q_stride : side == 1 ? a.k_stride : a.v_stride) + 8 * l;
  }
  __device__ __forceinline__ void next(const AppendPlan& p) {
    t += p.step_t;
    part += p.step_part;
    if (part >= p.items_per_token) part -= p.items_per_token, ++t;
  }
  // rows behind the last head are read as the first: they are not stored
  __device__ __forceinline__ const T* rows(int group, int row) const {
    const int head = group * (32 / LPR) + row;
    return src + (head < heads ? head : 0) * (16 * LPR);
  }
};

// PACK: some rows are packed (a dense call needs neither quantisers nor their code).  VEC: rows
// are 16-byte aligned; their copies run ahead of the arithmetic, across items, each lane's own
// elements through its own shared memory, so that nothing has to be waited for but the copies.
template <typename T, int LPR, bool PACK, bool VEC>
__global__ void __launch_bounds__(kAppendWarps * 32, kAppendCtas) append_kernel(AppendPlan p) {
  constexpr int D = 16 * LPR, RPW = 32 / LPR, S = stages<T>(), N = Raw<T>::N;
  __shared__ Quant quant[PACK ? 2 : 1];
  extern __shared__ __align__(16) unsigned char dynamic[];
  const AppendArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % LPR, row = lane / LPR;
  unsigned char* ring = dynamic + warp * (S * N * 512) + lane * 16;
  float* stage = reinterpret_cast<float*>(dynamic + (VEC ? ring_bytes<T>() : 0)) + warp * 512 + row * D;
  Item<T, LPR> it, ahead;
  {
    const uint32_t item = blockIdx.x * kAppendWarps + warp;
    it.t = item / (uint32_t)p.items_per_token;
    it.part = (int)(item - (uint32_t)it.t * (uint32_t)p.items_per_token);
    ahead.t = it.t;
    ahead.part = it.part;
  }
  int slot_in = 0, slot_out = 0;
  if (VEC && ahead.t < a.num_tokens) ahead.open(p, l);
  auto produce = [&] {
    if (ahead.t < a.num_tokens) {
      const T* from = ahead.rows(ahead.g, row);
      const uint32_t to = smem_address(ring) + slot_in * (N * 512);
#pragma unroll
      for (int i = 0; i < N; ++i) copy16(to + i * 512, reinterpret_cast<const uint4*>(from + (i < N / 2 ? 0 : D / 2)) + i % (N / 2));
      slot_in = slot_in + 1 == S ? 0 : slot_in + 1;
      if (++ahead.g == ahead.end) {
        ahead.next(p);
        if (ahead.t < a.num_tokens) ahead.open(p, l);
      }
    }
    copies_commit();
  };
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < S - 1; ++i) produce();
  }
  if constexpr (PACK) {
    if (warp == 0 && a.k_pages) build_quant(quant[0], a.k_centroids, 1 << a.k_bits, lane);
    if (warp == 1 && a.v_pages) build_quant(quant[1], a.v_centroids, 1 << a.v_bits, lane);
    __syncthreads();
  }
  for (; it.t < a.num_tokens; it.next(p)) {
    it.open(p, l);
    const int64_t t = it.t;
    bool skip = false;
    const float* cs = nullptr;
    if (a.positions) {
      const int64_t pos = (int64_t)a.positions[t] + a.position_offset;
      if (pos < 0) {
        skip = true;  // a padding row
      } else if (a.cos_sin) {
        if (pos >= a.num_positions) {
          if (a.status && lane == 0) atomicMax(a.status, (int32_t)kInvalidArg);
          skip = true;
        } else if (it.side < 2) {
          cs = a.cos_sin + pos * a.rot_dim;
        }
      }
    }
    const bool dense = !PACK || it.side == 0;
    int64_t slot = 0;
    if (!dense) {
      slot = a.slots[t];
      if (slot >= a.num_slots && !skip && a.status && lane == 0) atomicMax(a.status, (int32_t)kSlotOutOfRange);
      skip |= slot < 0 || slot >= a.num_slots;
    }
    const float* w = it.side == 0 ? a.q_weight : it.side == 1 ? a.k_weight : nullptr;
    const int mode = !cs ? kPlain : a.interleaved ? kPairs : a.rot_dim == D ? kHalves : kStaged;
    Coef f;
    if (!skip) token_coef<LPR>(f, mode, w, dense ? nullptr : a.signs, cs, a.rot_dim, p.table_vec, l);
    for (int g = it.g; g < it.end; ++g) {
      Raw<T> raw;
      if constexpr (VEC) {
        copies_wait<S - 2>();
        const unsigned char* from = ring + slot_out * (N * 512);
#pragma unroll
        for (int i = 0; i < N; ++i) raw.w[i] = *reinterpret_cast<const uint4*>(from + i * 512);
        slot_out = slot_out + 1 == S ? 0 : slot_out + 1;
      } else {
        raw.load(it.rows(g, row), D / 2);
      }
      float2 x[8];
      raw.get(x);
      if constexpr (VEC) produce();
      if (skip) continue;
      float factor = 1.f;
      if (w) factor = norm_factor<LPR>(x, a.eps);
      apply_coef<LPR>(x, f, mode, a.rot_dim, l, stage);
      const int head = g * RPW + row;
      const bool live = head < it.heads;
      if (dense) {
        const float2 f2 = make_float2(factor, factor);
        if (w) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], f2);
        }
        Raw<T> out;
        out.set(x);
        T* dst = static_cast<T*>(it.side == 0 ? a.q_out : a.k_out) +
                 t * (it.side == 0 ? a.q_out_stride : a.k_out_stride) + 8 * l + head * D;
        if (live) out.template store<VEC>(dst, D / 2);
      } else if constexpr (PACK) {
        const int bits = it.side == 1 ? a.k_bits : a.v_bits;
        uint8_t* dst = live ? (it.side == 1 ? a.k_pages : a.v_pages) + (slot * it.heads + head) * (int64_t)(D * bits / 8 + 4)
                            : nullptr;
        const Quant& q = quant[it.side - 1];
        switch (bits) {
          case 2: encode_row<LPR, 2>(x, factor, q, l, dst); break;
          case 3: encode_row<LPR, 3>(x, factor, q, l, dst); break;
          case 4: encode_row<LPR, 4>(x, factor, q, l, dst); break;
          default: encode_row<LPR, 5>(x, factor, q, l, dst); break;
        }
      }
    }
  }
  if constexpr (VEC) copies_wait<0>();
}

template <typename T, int LPR, bool PACK, bool VEC>
cudaError_t launch_append_kernel(const AppendPlan& p, int grid, cudaStream_t stream) {
  auto kern = append_kernel<T, LPR, PACK, VEC>;
  const bool staged = p.a.cos_sin && !p.a.interleaved && p.a.rot_dim < p.a.head_dim;
  const int smem = (VEC ? ring_bytes<T>() : 0) + (staged ? kStageBytes : 0);
  if (smem > 46 * 1024) {
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
  }
  kern<<<grid, kAppendWarps * 32, smem, stream>>>(p);
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) count_launches(1);
  return err;
}
template <typename T, int LPR>
cudaError_t launch_append_as(const AppendPlan& p, int grid, cudaStream_t stream) {
  const bool pack = p.a.k_pages || p.a.v_pages;
  if (p.vec) return pack ? launch_append_kernel<T, LPR, true, true>(p, grid, stream)
                         : launch_append_kernel<T, LPR, false, true>(p, grid, stream);
  return pack ? launch_append_kernel<T, LPR, true, false>(p, grid, stream)
              : launch_append_kernel<T, LPR, false, false>(p, grid, stream);
}
template <typename T>
cudaError_t launch_append_typed(const AppendPlan& p, int grid, cudaStream_t stream) {
  switch (p.a.head_dim) {
    case 16: return launch_append_as<T, 1>(p, grid, stream);
    case 32: return launch_append_as<T, 2>(p, grid, stream);
    case 64: return launch_append_as<T, 4>(p, grid, stream);
    case 128: return launch_append_as<T, 8>(p, grid, stream);
    case 256: return launch_append_as<T, 16>(p, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

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
  const int groups[3] = {(a.num_q_heads + rpw - 1) / rpw, (a.num_k_heads + rpw - 1) / rpw, (a.num_v_heads + rpw - 1) / rpw};
  const int64_t total = (int64_t)groups[0] + groups[1] + groups[2];
  if (a.num_tokens == 0 || total == 0) return cudaSuccess;
  p.vec = vec_ok(a.q, a.q_stride, size) && vec_ok(a.k, a.k_stride, size) && vec_ok(a.v, a.v_stride, size) &&
          vec_ok(a.q_out, a.q_out_stride, size) && vec_ok(a.k_out, a.k_out_stride, size);
  p.table_vec = reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0 && a.rot_dim % 8 == 0;
  // a token's coefficients serve up to eight groups of heads; fewer where that leaves warps idle
  const int64_t warps = (int64_t)sms * kAppendCtas * kAppendWarps;
  p.per_item = (int)std::max<int64_t>(1, std::min<int64_t>(8, a.num_tokens * total / (2 * warps)));
  for (int i = 0; i < 3; ++i) p.items[i] = (groups[i] + p.per_item - 1) / p.per_item;
  p.items_per_token = p.items[0] + p.items[1] + p.items[2];
  const int64_t ctas = (a.num_tokens * p.items_per_token + kAppendWarps - 1) / kAppendWarps;
  const int grid = (int)std::min<int64_t>(ctas, (int64_t)sms * kAppendCtas);
  p.step_t = (int64_t)grid * kAppendWarps / p.items_per_token;
  p.step_part = (int)((int64_t)grid * kAppendWarps % p.items_per_token);
  switch (a.dtype) {
    case kF32: return launch_append_typed<float>(p, grid, stream);
    case kF16: return launch_append_typed<__half>(p, grid, stream);
    case kBF16: return launch_append_typed<__nv_bfloat16>(p, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
