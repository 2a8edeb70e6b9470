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

#include "tq_append.h"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kAppendWarps = 8;

struct AppendPlan {
  AppendArgs a;
  int q_groups, k_groups, v_groups;  // groups of 32 / (D / 16) heads of a token
  int per_item;                      // groups a warp takes together
  int items_per_token;
  int vec;        // inputs and dense outputs: 16-byte accesses
  int table_vec;  // table rows: 16-byte loads
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

// Eight consecutive elements at p.
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, float2 (&v)[4]) {
  if (vec) {
    constexpr int W = 16 / (int)sizeof(T);  // elements of 16 bytes
#pragma unroll
    for (int i = 0; i < 8 / W; ++i) {
      const uint4 w = reinterpret_cast<const uint4*>(p)[i];
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int j = 0; j < W; j += 2) v[(i * W + j) / 2] = make_float2(to_f32<T>(e[j]), to_f32<T>(e[j + 1]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j += 2) v[j / 2] = make_float2(to_f32<T>(p[j]), to_f32<T>(p[j + 1]));
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, const float2 (&v)[4]) {
  if (vec) {
    constexpr int W = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / W; ++i) {
      uint4 w;
      T* e = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int j = 0; j < W; j += 2) {
        e[j] = from_f32<T>(v[(i * W + j) / 2].x);
        e[j + 1] = from_f32<T>(v[(i * W + j) / 2].y);
      }
      reinterpret_cast<uint4*>(p)[i] = w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      p[j] = from_f32<T>(v[j / 2].x);
      p[j + 1] = from_f32<T>(v[j / 2].y);
    }
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

// x <- w x / sqrt(mean x^2 + eps).  A row beyond the range of its squares is scaled first.
template <int LPR>
__device__ __forceinline__ void norm_row(float2 (&x)[8], const float* __restrict__ w, float eps, int l) {
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
  const float inv = rsqrtf(fmaf(ss, 1.0f / D, eps));
  const float2 i2 = make_float2(inv, inv);
  const float4* w4 = reinterpret_cast<const float4*>(w);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 g = __ldg(w4 + (c * (D / 2) + 8 * l) / 4 + h);
      x[4 * c + 2 * h] = __fmul2_rn(__fmul2_rn(x[4 * c + 2 * h], i2), make_float2(g.x, g.y));
      x[4 * c + 2 * h + 1] = __fmul2_rn(__fmul2_rn(x[4 * c + 2 * h + 1], i2), make_float2(g.z, g.w));
    }
  }
}

// Position rotation of a row; `cs` is the position's table row (rot_dim / 2 cosines, then
// sines).  `stage` is the warp's room for its rows (half style with rot_dim < D).
template <int LPR>
__device__ __forceinline__ void rotate_row(float2 (&x)[8], const float* __restrict__ cs, int rot, bool pairs, bool tvec,
                                           int l, int row, float* stage) {
  constexpr int D = 16 * LPR;
  const int half = rot / 2;
  if (pairs) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int p0 = (c * (D / 2) + 8 * l) / 2;  // first of the chunk's four pairs
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p0 + j >= half) continue;
        const float cv = __ldg(cs + p0 + j), sv = __ldg(cs + half + p0 + j);
        const float2 v = x[4 * c + j];
        x[4 * c + j] = make_float2(fmaf(v.x, cv, -v.y * sv), fmaf(v.y, cv, v.x * sv));
      }
    }
  } else if (rot == D) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 cv, sv;
      if (tvec) {
        cv = __ldg(reinterpret_cast<const float2*>(cs + 8 * l) + j);
        sv = __ldg(reinterpret_cast<const float2*>(cs + half + 8 * l) + j);
      } else {
        cv = make_float2(__ldg(cs + 8 * l + 2 * j), __ldg(cs + 8 * l + 2 * j + 1));
        sv = make_float2(__ldg(cs + half + 8 * l + 2 * j), __ldg(cs + half + 8 * l + 2 * j + 1));
      }
      const float2 a = x[j], b = x[4 + j];
      const float2 ns = make_float2(-sv.x, -sv.y);
      x[j] = __ffma2_rn(a, cv, __fmul2_rn(b, ns));
      x[4 + j] = __ffma2_rn(b, cv, __fmul2_rn(a, sv));
    }
  } else {
    float* mine = stage + row * D;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float2*>(mine + (i >> 2) * (D / 2) + 8 * l + 2 * (i & 3)) = x[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float* v = reinterpret_cast<float*>(&x[i]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int e = (i >> 2) * (D / 2) + 8 * l + 2 * (i & 3) + u;
        if (e >= rot) continue;
        const bool first = e < half;
        const int p = first ? e : e - half;
        const float cv = __ldg(cs + p), sv = __ldg(cs + half + p);
        const float other = mine[first ? e + half : e - half];
        v[u] = first ? fmaf(v[u], cv, -other * sv) : fmaf(v[u], cv, other * sv);
      }
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

// Encodes a row (all lanes of the warp take part; `dst` null: nothing stored).
template <int LPR, int B>
__device__ __forceinline__ void encode_row(float2 (&x)[8], const float* __restrict__ bnd, const float2 (&sg)[8], int l,
                                           uint8_t* dst) {
  constexpr int D = 16 * LPR, IB = D * B / 8;
  float ss = row_sum<LPR>(sum_squares(x));
  int ex = 0;
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
  }
  const bool bad = !(ss <= 3.402823466e38f);  // a NaN or infinite coordinate: a zero row's indices
  const float rs = (ss > 0.f && !bad) ? rsqrtf(ss) : 0.f;
  const float nu = bad ? ss : scale_pow2(ss * rs, ex);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], sg[i]);
  fwht_row<LPR>(x, l);
  constexpr float kInvSqrtD = LPR == 1 ? 0.25f : LPR == 2 ? 0.17677669529663689f : LPR == 4 ? 0.125f
                              : LPR == 8 ? 0.088388347648318447f : 0.0625f;
  const float inv = rs * kInvSqrtD;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint64_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 p = x[4 * c + j / 2];
      const float u = bad ? 0.f : ((j & 1) ? p.y : p.x) * inv;
      int idx = 0;  // #{k : boundary_k < u}, by halves
#pragma unroll
      for (int s = 1 << (B - 1); s > 0; s >>= 1)
        if (u > bnd[idx + s - 1]) idx += s;
      word |= (uint64_t)idx << (B * j);
    }
    if (dst) {
      uint8_t* at = dst + c * (IB / 2) + B * l;
      if constexpr (B == 4) {
        *reinterpret_cast<uint32_t*>(at) = (uint32_t)word;
      } else if constexpr (B == 2) {
        *reinterpret_cast<uint16_t*>(at) = (uint16_t)word;
      } else {
#pragma unroll
        for (int k = 0; k < B; ++k) at[k] = (uint8_t)(word >> (8 * k));
      }
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

template <typename T, int LPR>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(AppendPlan p) {
  constexpr int D = 16 * LPR, RPW = 32 / LPR;
  __shared__ float bnd[2][32];
  __shared__ __align__(16) float stage_all[kAppendWarps][RPW * D];
  const AppendArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % LPR, row = lane / LPR;
  if (threadIdx.x < 62) {
    const int side = threadIdx.x >= 31, i = threadIdx.x - 31 * side;
    const uint8_t* pages = side ? a.v_pages : a.k_pages;
    const float* c = side ? a.v_centroids : a.k_centroids;
    const int n = pages ? (1 << (side ? a.v_bits : a.k_bits)) - 1 : 0;
    if (i < n) bnd[side][i] = 0.5f * (c[i] + c[i + 1]);
  }
  __syncthreads();
  float2 sg[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sg[i] = make_float2(1.f, 1.f);
    const int e = (i >> 2) * (D / 2) + 8 * l + 2 * (i & 3);
    if (a.signs) sg[i] = make_float2(__ldg(a.signs + e), __ldg(a.signs + e + 1));
  }
  const int groups = p.q_groups + p.k_groups + p.v_groups;
  const int64_t items = a.num_tokens * p.items_per_token;
  for (int64_t item = (int64_t)blockIdx.x * kAppendWarps + warp; item < items; item += (int64_t)gridDim.x * kAppendWarps) {
    const int64_t t = item / p.items_per_token;
    const int part = (int)(item - t * p.items_per_token);
    const float* cs = nullptr;
    if (a.positions) {
      const int64_t pos = (int64_t)a.positions[t] + a.position_offset;
      if (pos < 0) continue;  // a padding row
      if (a.cos_sin) {
        if (pos >= a.num_positions) {
          if (a.status && lane == 0) atomicMax(a.status, (int32_t)kInvalidArg);
          continue;
        }
        cs = a.cos_sin + pos * a.rot_dim;
      }
    }
    int64_t slot = -1;
    if (a.slots) {
      slot = a.slots[t];
      if (slot >= a.num_slots) {
        if (a.status && lane == 0) atomicMax(a.status, (int32_t)kSlotOutOfRange);
        slot = -1;
      }
    }
    const int end = min(groups, (part + 1) * p.per_item);
    for (int g = part * p.per_item; g < end; ++g) {
      const int side = g < p.q_groups ? 0 : g < p.q_groups + p.k_groups ? 1 : 2;
      const int heads = side == 0 ? a.num_q_heads : side == 1 ? a.num_k_heads : a.num_v_heads;
      const int head = (g - (side == 0 ? 0 : side == 1 ? p.q_groups : p.q_groups + p.k_groups)) * RPW + row;
      const bool dense = side == 0 || (side == 1 && a.k_out);
      if (!dense && slot < 0) continue;
      const bool live = head < heads;
      const T* src = static_cast<const T*>(side == 0 ? a.q : side == 1 ? a.k : a.v) +
                     t * (side == 0 ? a.q_stride : side == 1 ? a.k_stride : a.v_stride) + (int64_t)(live ? head : 0) * D;
      float2 x[8];
      {
        float2 lo[4], hi[4];
        load8<T>(src + 8 * l, p.vec, lo);
        load8<T>(src + D / 2 + 8 * l, p.vec, hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = lo[i], x[4 + i] = hi[i];
      }
      if (side < 2) {
        const float* w = side == 0 ? a.q_weight : a.k_weight;
        if (w) norm_row<LPR>(x, w, a.eps, l);
        if (cs) rotate_row<LPR>(x, cs, a.rot_dim, a.interleaved, p.table_vec, l, row, stage_all[warp]);
      }
      if (dense) {
        if (live) {
          T* dst = static_cast<T*>(side == 0 ? a.q_out : a.k_out) + t * (side == 0 ? a.q_out_stride : a.k_out_stride) +
                   (int64_t)head * D;
          const float2 lo[4] = {x[0], x[1], x[2], x[3]}, hi[4] = {x[4], x[5], x[6], x[7]};
          store8<T>(dst + 8 * l, p.vec, lo);
          store8<T>(dst + D / 2 + 8 * l, p.vec, hi);
        }
      } else {
        const int bits = side == 1 ? a.k_bits : a.v_bits;
        uint8_t* dst = live ? (side == 1 ? a.k_pages : a.v_pages) + (slot * heads + head) * (int64_t)(D * bits / 8 + 4) : nullptr;
        const float* b = bnd[side - 1];
        switch (bits) {
          case 2: encode_row<LPR, 2>(x, b, sg, l, dst); break;
          case 3: encode_row<LPR, 3>(x, b, sg, l, dst); break;
          case 4: encode_row<LPR, 4>(x, b, sg, l, dst); break;
          default: encode_row<LPR, 5>(x, b, sg, l, dst); break;
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_append_typed(const AppendPlan& p, int grid, cudaStream_t stream) {
  const int threads = kAppendWarps * 32;
  switch (p.a.head_dim) {
    case 16: append_kernel<T, 1><<<grid, threads, 0, stream>>>(p); break;
    case 32: append_kernel<T, 2><<<grid, threads, 0, stream>>>(p); break;
    case 64: append_kernel<T, 4><<<grid, threads, 0, stream>>>(p); break;
    case 128: append_kernel<T, 8><<<grid, threads, 0, stream>>>(p); break;
    case 256: append_kernel<T, 16><<<grid, threads, 0, stream>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) count_launches(1);
  return err;
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
  const int rpw = 32 / (a.head_dim / 16), size = a.dtype == kF32 ? 4 : 2;
  auto groups = [&](int heads) { return (heads + rpw - 1) / rpw; };
  p.q_groups = groups(a.num_q_heads);
  p.k_groups = groups(a.num_k_heads);
  p.v_groups = groups(a.num_v_heads);
  const int total = p.q_groups + p.k_groups + p.v_groups;
  if (a.num_tokens == 0 || total == 0) return cudaSuccess;
  p.vec = vec_ok(a.q, a.q_stride, size) && vec_ok(a.k, a.k_stride, size) && vec_ok(a.v, a.v_stride, size) &&
          vec_ok(a.q_out, a.q_out_stride, size) && vec_ok(a.k_out, a.k_out_stride, size);
  p.table_vec = vec_ok(a.cos_sin, a.rot_dim / 2, 4);
  p.per_item = 1;
  p.items_per_token = total;
  const int64_t ctas = (a.num_tokens * p.items_per_token + kAppendWarps - 1) / kAppendWarps;
  const int grid = (int)std::min<int64_t>(ctas, (int64_t)device_sms() * 16);
  switch (a.dtype) {
    case kF32: return launch_append_typed<float>(p, grid, stream);
    case kF16: return launch_append_typed<__half>(p, grid, stream);
    case kBF16: return launch_append_typed<__nv_bfloat16>(p, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
