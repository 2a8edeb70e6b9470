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
// Weights, the transform's signs and the rotation are one product and one sum a channel, y = x p +
// x' s, with p and s worked out once for a token's heads.  A key's norm factor is not applied to its
// coordinates: u is scale free, the stored norm takes it.
//
// A warp takes runs of up to eight groups of 32 / (D / 16) heads and copies the next run's rows by
// cp.async while it works on one.  Packed sides cost it three to four times what dense ones do, so
// each warp's runs go through all sides in turn.
//
// Bound (GB300, 32768 tokens, 32 / 8 heads, D 128, bf16, norms; copy bandwidth 6684 GB/s):
//   tq_norm_rope, 688 MB     114 us, 90 % of that bandwidth
//   tq_append_kv K4 / V4, 724 MB   146 us, 74 %: issue.  An encoded group takes 490 to 560 warp
//     instructions (transform 116, quantiser 108, norm and store 70, the rest rows, places and loops),
//     a dense one 175; 62 % of the issue slots are used, by 16 warps an SM (registers: the coefficients
//     of a token take 32).
// Measured and not kept: 24 warps of 80 registers (spills: 212 us) or 20 of 96 (193 us); values in tiles
// of 16 rows with the transform on mma.sync (fewer instructions, but 64 accumulators beside the runs'
// state: 203 us, values alone 41 -> 45 us); an index by halving the decision points in shared memory (12
// instructions instead of 6.5); partial rotations through shared memory where they pair up between lanes
// (80 -> 67 us for 8200 tokens); runs that a warp's position alone gave to sides (165 -> 160 us).
#pragma once

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
  // chunks at p and p + half; any alignment without `vec`
  __device__ __forceinline__ void load(const T* p, int half, bool vec) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint4*>(p + (i < N / 2 ? 0 : half))[i % (N / 2)];
    } else {
      T* e = reinterpret_cast<T*>(w);
#pragma unroll
      for (int j = 0; j < 16; ++j) e[j] = p[j < 8 ? j : half + j - 8];
    }
  }
  __device__ __forceinline__ void store(T* p, int half, bool vec) const {
    if (vec) {
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

// ---- rows whose sum of squares leaves [2^-100, 2^100] (out of line: they are rare, but in the kernel
// for any call, where the lanes behind a side's last head hold zero rows) ------------------------
//
// Such a row is scaled by 2^-ex, ex the exponent of its largest magnitude (0 where that is 0 or not
// finite), which is exact.  `odd`: this lane's row is one.

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
// Whether ss (>= 0 or NaN) lies outside [the float of bits `least`, 2^100].
__device__ __forceinline__ bool outside(float ss, uint32_t least) { return __float_as_uint(ss) - least > 0x71800000u - least; }
// Scales x; returns the sum of squares (unchanged where the row is not odd); `eps`, the norm's, goes
// with the row and bounds ex from below: in the row's units it stays below 2^100.
template <int LPR>
__device__ __noinline__ float scale_rows(float2 (&x)[8], float ss, bool odd, float* eps, int* ex_out) {
  int ex = row_exponent<LPR>(x);
  if (!odd) ex = 0;
  if (eps && ex < 0 && *eps > 0.f) ex = max(ex, (ilogbf(*eps) - 100) / 2);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = make_float2(scale_pow2(x[i].x, -ex), scale_pow2(x[i].y, -ex));
  const float again = row_sum<LPR>(sum_squares(x));
  if (eps) *eps = ldexpf(*eps, -2 * ex);
  *ex_out = ex;
  return odd ? again : ss;
}

// 1 / sqrt(mean x^2 + eps).
template <int LPR>
__device__ __forceinline__ float norm_factor(float2 (&x)[8], float eps) {
  constexpr int D = 16 * LPR;
  float ss = row_sum<LPR>(sum_squares(x));
  // squares that underflow count only where eps is as small
  const uint32_t least = eps < 0x1p-80f ? 0x0d800000u : 0u;  // the bits of 2^-100
  const bool odd = outside(ss, least);
  if (__any_sync(kFullMask, odd)) {
    float2 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    int ex;
    float e = eps;
    ss = scale_rows<LPR>(y, ss, odd, &e, &ex);
    eps = e;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i];
  }
  return rsqrtf(fmaf(ss, 1.0f / D, eps));
}

__device__ __forceinline__ uint32_t smem_address(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t shared_u8(uint32_t at) {
  uint32_t v;
  asm("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ void add_if_greater(uint32_t& v, float u, float pt, uint32_t one) {
  asm("{\n .reg .pred p;\n setp.gt.f32 p, %1, %2;\n @p add.u32 %0, %0, %3;\n}\n" : "+r"(v) : "f"(u), "f"(pt), "r"(one));
}

// ---- weights, signs and rotation: y[e] = x[e] p[e] + x[e'] s[e], e' the other channel of e's pair ----

// Where it lies.  kAny: as the call has it.
enum Mode { kPlain, kHalves, kPairs, kStaged, kAny };  // no pair; slot i ^ 4; same float2; by shared memory

// A side's part of p and s that every token shares: p[e] = weight(e) sign(e), s[e] = -+ weight(e')
// sign(e), 0 behind the rotated channels.  (Encoded sides carry the transform's signs.)  In the order
// that lanes read them, four channels each: lane after lane, for the first and the second half of a
// lane's eight channels.
struct Shared {
  float p[256], s[256];
};
__device__ __forceinline__ int shared_place(int e, int D) {
  const int half = e >= D / 2, in = e - half * (D / 2);
  return ((2 * half + ((in >> 2) & 1)) * (D / 16) + (in >> 3)) * 4 + (in & 3);
}
__device__ __forceinline__ void build_shared(Shared& f, int mode, int D, const float* __restrict__ w,
                                             const float* __restrict__ sg, int rot, int first, int step) {
  const int half = rot / 2;
  for (int e = first; e < D; e += step) {
    const float g = sg ? __ldg(sg + e) : 1.f;
    const int at = shared_place(e, D);
    f.p[at] = (w ? __ldg(w + e) : 1.f) * g;
    float s = 0.f;
    if (mode != kPlain && e < rot) {
      const bool head = mode == kPairs ? (e & 1) == 0 : e < half;
      const int other = mode == kPairs ? e ^ 1 : head ? e + half : e - half;
      s = (w ? __ldg(w + other) : 1.f) * (head ? -g : g);
    }
    f.s[at] = s;
  }
}

struct Coef {
  float2 p[8], s[8];
};
// a lane's eight channels of half c
template <int LPR>
__device__ __forceinline__ void shared8(const float* p, int c, int l, float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 f = reinterpret_cast<const float4*>(p)[(2 * c + i) * LPR + l];
    v[2 * i] = make_float2(f.x, f.y);
    v[2 * i + 1] = make_float2(f.z, f.w);
  }
}
template <int LPR>
__device__ __forceinline__ void plain_coef(float2 (&p)[8], const Shared& f, int l) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float2 v[4];
    shared8<LPR>(f.p, c, l, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[4 * c + i] = v[i];
  }
}

// A token's coefficients, `cs` its table row (rot / 2 cosines, then the sines).
template <int LPR>
__device__ __forceinline__ void token_coef(Coef& f, const Shared& sh, int mode, const float* __restrict__ cs, int rot,
                                           bool tvec, int l) {
  constexpr int D = 16 * LPR;
  const int half = rot / 2;
  float2 cv[4], nv[4];
  if (mode == kHalves) {  // both chunks turn by the same angles
    load8(cs + 8 * l, tvec, cv);
    load8(cs + half + 8 * l, tvec, nv);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int e0 = c * (D / 2) + 8 * l;  // the chunk's first channel
    float2 pv[4], sv[4];
    shared8<LPR>(sh.p, c, l, pv);
    shared8<LPR>(sh.s, c, l, sv);
    if (mode == kPairs) {
      const int p0 = e0 / 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) cv[i] = make_float2(1.f, 1.f), nv[i] = make_float2(0.f, 0.f);
      if (tvec && p0 + 4 <= half) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(cs + p0));
        const float4 b = __ldg(reinterpret_cast<const float4*>(cs + half + p0));
        const float cf[4] = {a.x, a.y, a.z, a.w}, sf[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) cv[i] = make_float2(cf[i], cf[i]), nv[i] = make_float2(sf[i], sf[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (p0 + i < half) {
            const float a = __ldg(cs + p0 + i), b = __ldg(cs + half + p0 + i);
            cv[i] = make_float2(a, a), nv[i] = make_float2(b, b);
          }
      }
    } else if (mode == kStaged) {
#pragma unroll
      for (int i = 0; i < 4; ++i) cv[i] = make_float2(1.f, 1.f), nv[i] = make_float2(0.f, 0.f);
      if (rot % 16 == 0) {  // the whole chunk is of one half
        if (e0 < rot) {
          load8(cs + (e0 < half ? e0 : e0 - half), tvec, cv);
          load8(cs + (e0 < half ? e0 + half : e0), tvec, nv);
        }
      } else {
        float* cf = reinterpret_cast<float*>(cv);
        float* sf = reinterpret_cast<float*>(nv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = e0 + i, t = e < half ? e : e - half;
          if (e < rot) cf[i] = __ldg(cs + t), sf[i] = __ldg(cs + half + t);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.p[4 * c + i] = __fmul2_rn(pv[i], cv[i]);
      f.s[4 * c + i] = __fmul2_rn(sv[i], nv[i]);
    }
  }
}

template <int LPR>
__device__ __forceinline__ void apply_coef(float2 (&x)[8], const Coef& f, int mode, int rot, int l, float* mine) {
  constexpr int D = 16 * LPR;
  if (mode == kHalves) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = x[i], b = x[4 + i];
      x[i] = __ffma2_rn(a, f.p[i], __fmul2_rn(b, f.s[i]));
      x[4 + i] = __ffma2_rn(b, f.p[4 + i], __fmul2_rn(a, f.s[4 + i]));
    }
  } else if (mode == kPairs) {
    if (rot == D) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __ffma2_rn(x[i], f.p[i], __fmul2_rn(make_float2(x[i].y, x[i].x), f.s[i]));
    } else {  // (the neighbour of a channel that stays may be infinite)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = (i >> 2) * (D / 2) + 8 * l + 2 * (i & 3) < rot;
        const float2 other = in ? make_float2(x[i].y, x[i].x) : make_float2(0.f, 0.f);
        x[i] = __ffma2_rn(x[i], f.p[i], __fmul2_rn(other, f.s[i]));
      }
    }
  } else if (rot <= D / 2 && rot % 16 == 0 && (rot & (rot - 1)) == 0) {
    // a power of two of at least 16 in the first half: chunks of eight pair up between lanes (staged in
    // shared memory they cost twice the time: 8200 tokens of rot 64, D 128)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 other = make_float2(__shfl_xor_sync(kFullMask, x[i].x, rot / 16), __shfl_xor_sync(kFullMask, x[i].y, rot / 16));
      if (8 * l >= rot) other = make_float2(0.f, 0.f);
      x[i] = __ffma2_rn(x[i], f.p[i], __fmul2_rn(other, f.s[i]));
      x[4 + i] = __fmul2_rn(x[4 + i], f.p[4 + i]);
    }
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
        if (e0 >= rot) other[0] = other[1] = other[2] = other[3] = make_float2(0.f, 0.f);
      } else {
        float* o = reinterpret_cast<float*>(other);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = e0 + i;
          o[i] = e < half ? mine[e + half] : e < rot ? mine[e - half] : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[4 * c + i] = __ffma2_rn(x[4 * c + i], f.p[4 * c + i], __fmul2_rn(other[i], f.s[4 * c + i]));
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

// Quantisers of the two packed sides.  128 equal cells cover the span of a codebook's decision
// points; a cell holds the number of points in cells before it, so the index is that and one
// comparison for each point that the cell itself may hold (`steps`, the most of any cell: 1 for a
// Lloyd-Max codebook).  Cells come from one monotone function of u for points and coordinates
// alike, so its rounding does not matter.  32 words of counts and at most 32 points a side: neither
// lookup has bank conflicts.
struct Quants {
  float point[2][32];      // a side's decision points, then +inf
  uint8_t below[2][128];   // offset in `point` of the first point that is in no earlier cell
  float mul[2], add[2];    // span to [0, 1]
  int steps[2];
};
// base + 127 t for the clamped t = u mul + add, as the bits of a subnormal (base: one too)
__device__ __forceinline__ uint32_t cell_of(float u, float mul, float add, float base) {
  float t;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(t) : "f"(u), "f"(mul), "f"(add));  // NaN: 0
  return __float_as_uint(fmaf(t, 0x1.fcp-143f, base));  // 127 * 2^-149
}
__device__ __forceinline__ uint2 cells_of(float2 u, float mul, float add, float base) {
  float2 t;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(t.x) : "f"(u.x), "f"(mul), "f"(add));
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(t.y) : "f"(u.y), "f"(mul), "f"(add));
  const float2 c = __ffma2_rn(t, make_float2(0x1.fcp-143f, 0x1.fcp-143f), make_float2(base, base));
  return make_uint2(__float_as_uint(c.x), __float_as_uint(c.y));
}
// Set up by a warp from n = 2^bits ascending centroids (points: rounded midpoints).
__device__ __forceinline__ void build_quant(Quants& q, int side, const float* __restrict__ c, int n, int lane) {
  const float pt = lane < n - 1 ? 0.5f * (__ldg(c + lane) + __ldg(c + lane + 1)) : __int_as_float(0x7f800000);
  const float lo = __shfl_sync(kFullMask, pt, 0), hi = __shfl_sync(kFullMask, pt, n - 2);
  const float mul = hi > lo ? 1.0f / (hi - lo) : 0.f, add = -lo * mul;
  const int cell = lane < n - 1 ? (int)cell_of(pt, mul, add, 0.f) : 128;
  q.point[side][lane] = pt;
  int most = 0;
#pragma unroll 1
  for (int j = 0; j < 4; ++j) {
    int below = 0, here = 0;
    for (int k = 0; k < n - 1; ++k) {
      const int ck = __shfl_sync(kFullMask, cell, k);
      below += ck < lane + 32 * j;
      here += ck == lane + 32 * j;
    }
    q.below[side][lane + 32 * j] = (uint8_t)(4 * (below + 32 * side));
    most = max(most, here);
  }
  most = __reduce_max_sync(kFullMask, most);
  if (lane == 0) q.mul[side] = mul, q.add[side] = add, q.steps[side] = most;
}
// A side's quantiser in registers.
struct Quant {
  float mul, add, base;
  int steps, side;
  __device__ __forceinline__ void open(const Quants& q, int s) {
    mul = q.mul[s];
    add = q.add[s];
    base = __int_as_float((int)smem_address(q.below[s]));
    steps = q.steps[s];
    side = s;
  }
};

// Codebooks of which a cell holds several points (out of line; no Lloyd-Max codebook is one).
template <int B>
__device__ __noinline__ uint32_t fours_slow(float2 u, float2 v, Quant q, const float* points) {
  const float x[4] = {u.x, u.y, v.x, v.y};
  uint32_t sum = 0;
  for (int j = 0; j < 4; ++j) {
    uint32_t offset = shared_u8(cell_of(x[j], q.mul, q.add, q.base));
    for (int k = 0; k < q.steps; ++k)
      if (x[j] > points[offset / 4]) offset += 4;
    sum += offset << (B * j);
  }
  return sum;
}

// Encodes rows of signed coordinates x, whose own norm is `factor` times theirs (all lanes of the
// warp take part; `dst` null: nothing stored).
template <int LPR, int B>
__device__ __forceinline__ void encode_row(float2 (&x)[8], float factor, const Quant& q, const float* points, int l,
                                           uint8_t* dst) {
  constexpr int D = 16 * LPR, IB = D * B / 8;
  float ss = row_sum<LPR>(sum_squares(x)), back = 1.f;
  const bool odd = outside(ss, 0x0d800000u);
  if (__any_sync(kFullMask, odd)) {
    float2 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    int ex;
    ss = scale_rows<LPR>(y, ss, odd, nullptr, &ex);
    const bool bad = !(ss <= 3.402823466e38f);  // a NaN or infinite coordinate: a zero row's indices
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bad ? make_float2(0.f, 0.f) : y[i];
    // the norm is sqrt(ss) factor 2^ex below; zero rows and rows that are not finite keep theirs
    back = pow2i(ex / 2);
    factor *= pow2i(ex - ex / 2);
    if (bad) back = factor = 1.f;
    if (ss == 0.f) ss = 0x1p-126f, factor = 0.f;
  }
  float rs;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(ss));  // ss in the normal range, or not finite
  // (the norm that is stored is correctly rounded, as the writer's; the coordinates' own factor needs
  // fewer bits: its error, below 2^-22, is as that of the transform's sums)
  const bool finite = ss <= 3.402823466e38f;
  const float nu = finite ? sqrtf(ss) * factor * back : ss;
  if (!finite) rs = 0.f;
  fwht_row<LPR>(x, l);
  constexpr float kInvSqrtD = LPR == 1 ? 0.25f : LPR == 2 ? 0.17677669529663689f : LPR == 4 ? 0.125f
                              : LPR == 8 ? 0.088388347648318447f : 0.0625f;
  const float inv = rs * kInvSqrtD;
  const float2 inv2 = make_float2(inv, inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], inv2);
  // offsets of a side's points start at 128 side: four of them, B bits apart
  const uint32_t start = 0u - (uint32_t)q.side * 128u * (1u + (1u << B) + (1u << (2 * B)) + (1u << (3 * B)));
  uint32_t fours[4];  // 4 times four indices, B bits apart
  if (q.steps == 1) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      fours[h] = start;
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float2 u = x[2 * h + j / 2];
        const uint2 cell = cells_of(u, q.mul, q.add, q.base);
        uint32_t o0 = shared_u8(cell.x), o1 = shared_u8(cell.y);
        const char* at = reinterpret_cast<const char*>(points);
        add_if_greater(o0, u.x, *reinterpret_cast<const float*>(at + o0), 4u);
        add_if_greater(o1, u.y, *reinterpret_cast<const float*>(at + o1), 4u);
        fours[h] += o0 * (1u << (B * j));
        fours[h] += o1 * (1u << (B * j + B));
      }
    }
  } else {
#pragma unroll
    for (int h = 0; h < 4; ++h)
      fours[h] = start + fours_slow<B>(x[2 * h], x[2 * h + 1], q, points);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t half[2] = {fours[2 * c], fours[2 * c + 1]};
    using Word = typename std::conditional<(B > 4), uint64_t, uint32_t>::type;
    const Word word = (Word)(half[0] >> 2) | (Word)(half[1] >> 2) << (4 * B);
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

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// Groups of rows (1 KB each, fp32 2 KB) of a run, and as many copies in flight a warp.
template <typename T>
__host__ __device__ constexpr int run_groups() {
  return sizeof(T) == 2 ? kRunGroups : kRunGroups / 2;
}
// Dynamic shared memory: the rows in flight, and room to exchange pairs.
constexpr int kRingBytes = kAppendWarps * kRunGroups * 1024;
constexpr int kStageBytes = kAppendWarps * 512 * 4;

// A run: consecutive groups of heads of one side (0: q, 1: k, 2: v) over a block of tokens, token by
// token; a warp's unit of work.
struct Run {
  int block, part;  // which
  int side;
  int t, g, n;      // token and group of its first group; groups
  __device__ __forceinline__ void open(const AppendPlan& p) {
    side = part < p.items[0] ? 0 : part < p.items[0] + p.items[1] ? 1 : 2;
    const int groups = p.side[side].groups;
    const int u = (part - p.side[side].first) * p.run;
    const int k = groups == 1 ? u : (int)__umulhi((uint32_t)u, p.side[side].inv_groups);
    t = block * p.block_tokens + k;
    g = u - k * groups;
    n = max(0, min(p.run, min(p.block_tokens - k, (int)p.a.num_tokens - t) * groups - g));
  }
  // to the next run that has groups; n = 0 behind the last
  __device__ __forceinline__ void next(const AppendPlan& p) {
    do {
      block += p.step_block;
      part += p.step_part;
      if (part >= p.block_items) part -= p.block_items, block += p.carry;
      n = 0;
      if (block >= p.blocks) return;
      open(p);
    } while (n == 0);
  }
};

// PACK: some rows are packed (a dense call needs neither quantisers nor their code).  RING: rows are
// 16-byte aligned; while a warp works on a run the next one's rows are copied, each into the place of
// the group just read, each lane's own elements through its own shared memory: nothing has to be waited
// for but the copies.
template <typename T, int LPR, int MODE, bool PACK, bool RING>
__global__ void __launch_bounds__(kAppendWarps * 32, kAppendCtas) append_kernel(const __grid_constant__ AppendPlan p) {
  constexpr int D = 16 * LPR, RPW = 32 / LPR, U = run_groups<T>(), N = Raw<T>::N;
  constexpr int kGroup = RPW * D * (int)sizeof(T);  // bytes of a group's rows
  __shared__ Quants quants;
  __shared__ __align__(16) Shared shared[3];
  extern __shared__ __align__(16) unsigned char dynamic[];
  const AppendArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % LPR, row = lane / LPR;
  float* stage = reinterpret_cast<float*>(dynamic + (RING ? kRingBytes : 0)) + warp * 512 + row * D;
  const int mine = (row * D + 8 * l) * (int)sizeof(T);  // this lane's elements in a group's rows
  unsigned char* const ring = dynamic + warp * (kRunGroups * 1024) + lane * 16;
  Run it;
  {
    const uint32_t item = blockIdx.x * kAppendWarps + warp;
    it.block = item / (uint32_t)p.block_items;
    it.part = (int)(item - (uint32_t)it.block * (uint32_t)p.block_items);
    it.n = 0;
    if ((int)item >= p.warps) it.block = p.blocks;  // (a warp too many)
    if (it.block < p.blocks) it.open(p);
    if (it.n == 0) it.next(p);
  }
  // The positions and slots of a run's tokens, the j-th token's in lane j.
  int32_t pos_in = 0;
  int64_t slot_in = 0;
  auto look_up = [&](const Run& w) {
    if (lane < U && w.n > 0 && w.t + lane < (int)a.num_tokens) {
      if (a.positions) pos_in = __ldg(a.positions + w.t + lane);
      if (PACK && w.side > 0) slot_in = __ldg(a.slots + w.t + lane);
    }
  };
  // The rows that are copied next: group c_g of c_groups of a token, c_left to go of the run.
  const unsigned char* c_from = nullptr;
  int64_t c_wrap = 0;
  int c_g = 0, c_groups = 0, c_heads = 0, c_left = 0;
  auto aim = [&](const Run& w) {
    c_left = w.n;
    if (w.n == 0) return;
    const AppendSide& sd = p.side[w.side];
    c_groups = sd.groups;
    c_heads = sd.heads;
    c_g = w.g;
    c_from = sd.in + (int64_t)w.t * sd.in_step + w.g * kGroup + mine;
    c_wrap = sd.in_step - (int64_t)sd.groups * kGroup;
  };
  auto copy_next = [&](uint32_t to) {
    if constexpr (RING) {
      if (c_left > 0) {
        if (p.full || c_g * RPW + row < c_heads) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            copy16(to + i * 512, c_from + (i < N / 2 ? 0 : D / 2 * (int)sizeof(T)) + i % (N / 2) * 16);
        }
        --c_left;
        c_from += kGroup;
        if (++c_g == c_groups) c_g = 0, c_from += c_wrap;
      }
      copies_commit();
    }
  };
  const uint32_t ring_at = smem_address(ring);
  if constexpr (RING) {
    // lanes of rows behind a side's last head keep what they held: ones, to begin with
    if (!p.full) {
#pragma unroll
      for (int i = 0; i < U * N; ++i)
        *reinterpret_cast<uint4*>(ring + i * 512) = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    }
  }
  look_up(it);
  aim(it);
#pragma unroll 1
  for (int j = 0; j < U; ++j) copy_next(ring_at + j * (N * 512));
  const int mode = MODE == kAny ? (!a.cos_sin ? kPlain : a.interleaved ? kPairs : a.rot_dim == D ? kHalves : kStaged) : MODE;
  if constexpr (PACK) {
    if (warp == 0 && a.k_pages) build_quant(quants, 0, a.k_centroids, 1 << a.k_bits, lane);
    if (warp == 1 && a.v_pages) build_quant(quants, 1, a.v_centroids, 1 << a.v_bits, lane);
  }
  static_assert(kAppendWarps == 8, "two warps for the quantisers, two a side for the shared parts");
  if (warp >= 2) {
    const int side = (warp - 2) >> 1;
    build_shared(shared[side], side == 2 ? kPlain : mode, D, side == 0 ? a.q_weight : side == 1 ? a.k_weight : nullptr,
                 PACK && side > 0 ? a.signs : nullptr, a.rot_dim, (warp & 1) * 32 + lane, 64);
  }
  __syncthreads();

  Coef f;
  int coef_side = -1;  // the side that is not rotated whose coefficients f holds
  // One run: `use(x, factor, to, live, normed)` takes each group's rows.  turns_tag: 1 the side is
  // rotated, 0 it is not, -1 as the run has it.
  auto take = [&](const Run& w, int32_t pos_all, int64_t slot_all, auto dense_tag, auto turns_tag, int step, auto use) {
    constexpr bool dense = decltype(dense_tag)::value;
    constexpr int kTurns = decltype(turns_tag)::value;
    const int side = w.side;
    const AppendSide& sd = p.side[side];
    const bool normed = sd.normed;
    const bool turned = kTurns >= 0 ? kTurns != 0 : side < 2 && mode != kPlain;
    if (!turned && coef_side != side) plain_coef<LPR>(f.p, shared[side], l);
    coef_side = turned ? -1 : side;
    // every lane's token: its position and slot
    const int64_t pos = a.positions ? (int64_t)pos_all + a.position_offset : 0;
    const bool far = a.cos_sin && pos >= a.num_positions;
    const bool astray = !dense && slot_all >= a.num_slots && pos >= 0;
    const uint32_t good = __ballot_sync(kFullMask, pos >= 0 && !far && (dense || (uint64_t)slot_all < (uint64_t)a.num_slots));
    if (__any_sync(kFullMask, far || astray)) {
      if (a.status && lane < U && w.t + lane < (int)a.num_tokens) {
        if (far) atomicMax(a.status, (int32_t)kInvalidArg);
        if (astray) atomicMax(a.status, (int32_t)kSlotOutOfRange);
      }
    }
    // this lane's place in the first group's rows of its lane's token (k-th of the run)
    int64_t place;
    if constexpr (dense) place = (int64_t)(w.t + lane) * sd.out_step;
    else place = slot_all * sd.slot_step;
    int k = 0, left = w.n, m = min(left, sd.groups - w.g);  // token of the run, groups left, of the token
    int head = w.g * RPW + row;
    uint32_t at = ring_at;
#pragma unroll 1
    while (true) {  // a token's groups
      if ((good >> k) & 1u) {
        unsigned char* to = sd.out + __shfl_sync(kFullMask, place, k);
        if constexpr (dense) to += (head - row) * (D * (int)sizeof(T)) + mine;
        else to += head * (int)sd.out_step;
        if (turned)
          token_coef<LPR>(f, shared[side], mode, a.cos_sin + (uint64_t)__shfl_sync(kFullMask, (uint32_t)pos, k) * (uint32_t)a.rot_dim,
                          a.rot_dim, p.table_vec, l);
#pragma unroll 1
        for (int j = 0; j < m; ++j) {
          const bool live = p.full || head < sd.heads;
          Raw<T> raw;
          if constexpr (RING) {
            copies_wait<U - 1>();
#pragma unroll
            for (int i = 0; i < N; ++i)
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(raw.w[i].x), "=r"(raw.w[i].y), "=r"(raw.w[i].z), "=r"(raw.w[i].w)
                           : "r"(at + i * 512)
                           : "memory");
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) raw.w[i] = make_uint4(0, 0, 0, 0);
            if (live)
              raw.load(reinterpret_cast<const T*>(sd.in + (int64_t)(w.t + k) * sd.in_step + (head - row) * (D * (int)sizeof(T)) + mine),
                       D / 2, p.vec);
          }
          float2 x[8];
          raw.get(x);
          copy_next(at);
          at += N * 512;
          float factor = 1.f;
          if (normed) factor = norm_factor<LPR>(x, a.eps);
          if (turned) {
            apply_coef<LPR>(x, f, mode, a.rot_dim, l, stage);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], f.p[i]);
          }
          use(x, factor, to, live, normed);
          to += step;
          head += RPW;
        }
      } else {
        if constexpr (RING) {
#pragma unroll 1
          for (int j = 0; j < m; ++j) {
            copies_wait<U - 1>();  // (what is on its way here has to be there before the next is sent)
            copy_next(at);
            at += N * 512;
          }
        }
      }
      left -= m;
      if (left == 0) break;
      m = min(left, sd.groups);
      head = row;
      ++k;
    }
    if constexpr (RING) {  // places that this run did not use
#pragma unroll 1
      for (int j = w.n; j < U; ++j) {
        copy_next(at);
        at += N * 512;
      }
    }
  };
  while (it.n > 0) {
    const int32_t pos_all = pos_in;
    const int64_t slot_all = slot_in;
    Run ahead = it;
    ahead.next(p);
    look_up(ahead);
    aim(ahead);
    using Any = std::integral_constant<int, -1>;
    using Turns = std::integral_constant<int, MODE == kAny ? -1 : MODE != kPlain>;
    if (!PACK || it.side == 0) {
      take(it, pos_all, slot_all, std::true_type{}, Turns{}, kGroup,
           [&](float2 (&x)[8], float factor, unsigned char* to, bool live, bool normed) {
             if (normed) {
               const float2 f2 = make_float2(factor, factor);
#pragma unroll
               for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], f2);
             }
             Raw<T> out;
             out.set(x);
             if (live) out.store(reinterpret_cast<T*>(to), D / 2, RING || p.vec);
           });
    } else if constexpr (PACK) {
      Quant q;
      q.open(quants, it.side - 1);
      const int bits = it.side == 1 ? a.k_bits : a.v_bits, step = RPW * (D * bits / 8 + 4);
      const float* points = &quants.point[0][0];
      if constexpr (MODE == kAny) {  // (one body for all widths: this form is not for speed)
        take(it, pos_all, slot_all, std::false_type{}, Any{}, step,
             [&](float2 (&x)[8], float factor, unsigned char* to, bool live, bool) {
               uint8_t* dst = live ? to : nullptr;
               switch (bits) {
                 case 2: encode_row<LPR, 2>(x, factor, q, points, l, dst); break;
                 case 3: encode_row<LPR, 3>(x, factor, q, points, l, dst); break;
                 case 4: encode_row<LPR, 4>(x, factor, q, points, l, dst); break;
                 default: encode_row<LPR, 5>(x, factor, q, points, l, dst); break;
               }
             });
      } else {
        auto packed = [&](auto tag) {
          constexpr int B = decltype(tag)::value;
          take(it, pos_all, slot_all, std::false_type{}, Any{}, step,
               [&](float2 (&x)[8], float factor, unsigned char* to, bool live, bool) {
                 encode_row<LPR, B>(x, factor, q, points, l, live ? to : nullptr);
               });
        };
        switch (bits) {
          case 2: packed(std::integral_constant<int, 2>{}); break;
          case 3: packed(std::integral_constant<int, 3>{}); break;
          case 4: packed(std::integral_constant<int, 4>{}); break;
          default: packed(std::integral_constant<int, 5>{}); break;
        }
      }
    }
    it = ahead;
  }
  if constexpr (RING) copies_wait<0>();
}

template <typename T, int LPR, int MODE, bool PACK, bool RING>
cudaError_t launch_append_kernel(const AppendPlan& p, cudaStream_t stream) {
  auto kern = append_kernel<T, LPR, MODE, PACK, RING>;
  const bool staged = p.a.cos_sin && !p.a.interleaved && p.a.rot_dim < p.a.head_dim;
  const int smem = (RING ? kRingBytes : 0) + (staged ? kStageBytes : 0);
  if (RING) {
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes + kStageBytes);
    if (err != cudaSuccess) return err;
  }
  kern<<<p.grid, kAppendWarps * 32, smem, stream>>>(p);
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) count_launches(1);
  return err;
}

// Head dims of 64 and more with aligned rows take a kernel of their mode (values alone, 32768 tokens of
// 8 heads: 41 us, 70 in the one for any call); the rest one for any call.
template <typename T, int LPR, bool PACK>
cudaError_t launch_append_mode(const AppendPlan& p, cudaStream_t stream) {
  if constexpr (LPR >= 4) {
    if (p.vec) {
      if (!p.a.cos_sin) return launch_append_kernel<T, LPR, kPlain, PACK, true>(p, stream);
      if (p.a.interleaved) return launch_append_kernel<T, LPR, kPairs, PACK, true>(p, stream);
      if (p.a.rot_dim == p.a.head_dim) return launch_append_kernel<T, LPR, kHalves, PACK, true>(p, stream);
      return launch_append_kernel<T, LPR, kStaged, PACK, true>(p, stream);
    }
  }
  return launch_append_kernel<T, LPR, kAny, PACK, false>(p, stream);
}
template <typename T, bool PACK>
cudaError_t launch_append_typed(const AppendPlan& p, cudaStream_t stream) {
  switch (p.a.head_dim) {
    case 16: return launch_append_mode<T, 1, PACK>(p, stream);
    case 32: return launch_append_mode<T, 2, PACK>(p, stream);
    case 64: return launch_append_mode<T, 4, PACK>(p, stream);
    case 128: return launch_append_mode<T, 8, PACK>(p, stream);
    case 256: return launch_append_mode<T, 16, PACK>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace tq
