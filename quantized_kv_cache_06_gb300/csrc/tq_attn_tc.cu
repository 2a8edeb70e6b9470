// Tensor-core attention of query rows with a visible set of their own over packed TurboQuant
// pages (sm_103a, tcgen05): drafted trees, biased prefill, single tokens.
//
// TurboQuant docs: "vLLM Usage" (Runtime Dispatch: the cache plus mixed prefill/decode reads
// the packed cache) and "Architecture" (Diagnostic vs Serving Paths: keys consumed
// compressed, values accumulated from packed indices).
//
// For a tile of 128 tokens of one kv head and the window's columns (query row, q head of the
// group), both products are taken transposed, tokens (or dims) on the 128 lanes and the
// columns on N, so that a window of any number of columns fills the tensor cores' M:
//   S^T [tokens x cols] = Khat [tokens x D]  Q^T           A = Khat in TMEM, B = Q (K-major)
//   O^T [dims x cols]  += Vhat^T [dims x tokens] P^T       A = Vhat, B = P^T, both stored as
//                                                          they are produced (MN-major)
// Khat = fp16(alpha_k c[idx]) never touches shared memory: the thread that owns a token
// expands its packed row in registers and stores it to its own lane of TMEM.  Vhat goes to
// shared memory in 16-byte chunks, swizzled.  The norms are per token, so per lane: nu_k
// multiplies the score, nu_v the weight.
//
// Precision.  fp16 outputs (SPLIT): Q and P' = hi + lo in fp16, the lo parts as further k-steps
// into the same accumulators, so what is left is the rounding of the centroids (alpha puts them
// near fp16 grid points).  One part for P' would hold twice the columns (tree 4 x 131072 0.73 ms),
// at an error of one and a half times the output's own rounding.  bf16 outputs: one fp16 part
// each, eight times finer than the output's own rounding.  The window's queries are scaled by one
// power of two, by one each where their sizes differ much.  The weights that fp16 holds are products
// p nu_v, so a column is taken relative to the largest product it has seen, not the largest p: no
// query and no norm leaves the fp16 range, and no row is the worse for its neighbours' or for a
// giant norm that has no weight in it.  Sums, maxima and both products are fp32.
//
// Softmax in base 2; the reference of a column moves only when a product passes its place by 2^6, so
// most tiles rescale nothing; when one does, the softmax warps scale O^T in TMEM themselves
// (the product before has completed by then).
//
// Roles of the warps: 0-3 keys, 4-7 values, 8-15 softmax (lane quadrant = warp % 4, in two
// sets), 16 and 17 MMA issue (scores, values).  A window of more than half the MMA columns has
// both sets on one tile, each with its groups of 16 columns; a smaller one makes two streams of
// one set that take alternate tiles, each with its own references, sums and O^T, merged when the
// window ends: the chain of waits, TMEM reads and votes of one tile then hides behind the
// other's.
//
// Packed rows: a dequantising lane copies the rows of its own token with 16-byte cp.async (the
// aligned span around the head's bytes; by words where a slab is not whole 16 bytes, H not a
// multiple of 4), up to six tiles deep, so no thread waits for another's copy.  TMA boxes of 16
// rows x 80 bytes took ten cycles a row, 2700 a tile.
//
// What bounds it: not memory (64 x 8192 tokens: single tokens 0.24 ms, 1.2 TB/s; tree of 32 nodes
// 0.66 ms, 0.42 PFLOP/s), nor the tensor pipe (a sixth busy).  One more tile of 128 columns takes
// 2.6 us, of single tokens 1.7, most of it the softmax warps' in the weights; dequantisation and the
// products hide behind that.  All roles together issue 11700 instructions a tile, half of the slots.
// One more window of as many tiles takes 29 us and 4.6 (its queries, a first tile's references, masked
// tiles, sums and outputs).  Twice the softmax warps, or a product and a vote for each half of the
// columns, change nothing of a tile; code size does: five programs share the instruction cache, and
// unrolling the two dequantisation loops cost a quarter (tree 0.84 -> 1.03 ms).  Hence the rolled loops, the paths apart for changed scores and moved references,
// and rows read word by word from shared memory (a tenth against holding them in registers).
//
// All waits are bounded: one that runs out records the timeout, every role leaves its loop, the
// copies and MMAs in flight are waited for and TMEM is freed.
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

constexpr float kLog2eA = 1.4426950408889634f;
constexpr int kTok = kAttnTile;  // tokens per tile = MMA lanes
constexpr int kKeyWarps = 4, kValWarps = 4, kSoftSets = 2, kSoftWarps = 4 * kSoftSets;
constexpr int kMmaWarp = kKeyWarps + kValWarps + kSoftWarps;
constexpr int kTcThreads = 32 * (kMmaWarp + 4);  // whole warpgroups (two warps idle)
constexpr int kSoftThreads = 32 * kSoftWarps;
// Registers a thread: 96 at launch (640 threads); the softmax warps, which hold sums of up to 64
// columns, take what the others leave (a spill there goes to L2: little L1 is left beside the
// shared memory).  128 (dequant + dequant + issue) + 256 soft <= 640 * 96.
constexpr int kRegsIssue = 64;
constexpr int kMaxRing = 6;
constexpr int kNorms = 6;  // tiles whose norms are kept: keys and values run at most five tiles ahead of the softmax
// A column's reference r: its weights are 2^(x - r), its products 2^(x - r) nu_v 2^-8.  When it is
// set, the largest product goes to 2^kProductExp; it moves when one passes that by 2^kSlack, so 2^14
// at most is written, well inside fp16.  A scaled norm counts as kNormLow or more, so that tokens of no
// value cannot make weights that overflow the sums.  (The 2^-8 keeps the weights of norms of up to
// 2^127 above the smallest float.)
constexpr float kSlack = 6.0f, kProductExp = 8.0f;
constexpr float kMaxProduct = 16384.0f;  // 2^(kProductExp + kSlack)
constexpr float kNormScale = 0.00390625f, kNormUnscale = 256.0f;
constexpr float kNormLow = 3.552713678800501e-15f;  // 2^-48: a norm of 2^-40
// Where a token's factor is above this, scores could pass 2^24 (|S| is 2^15 at most) and the rounding
// of x kn a weight's exponent: such tiles are changed in place first, which rounds them once.
constexpr float kLargeFactor = 512.0f;
constexpr int kBarSoft = 1;               // named barrier of all softmax warps; 2, 3: of a stream
constexpr int kNoToken = -0x7fffffff - 1;  // the entry of a token that is not there: no block
constexpr float kNoMax = -3e38f;          // reference of a column that has seen nothing: below any score
constexpr int kNoQuery = -1000;           // exponent of a query that is zero, not finite, or sees nothing
// Binades by which a window's queries may differ under one power of two: the smallest keeps its
// largest coordinate above 2 in fp16, an absolute error of 2^-25 (lo part) against it.
constexpr int kQuerySpread = 8;

template <int D, bool SPLIT, int N>
struct Tc {
  static constexpr int kN = N;                           // MMA columns, window columns at most
  static constexpr int kGroups = (kN + 31) / 32;      // groups of 16 columns per softmax thread
  static constexpr int kHalves = D == 256 ? 2 : 1;       // 128-dim halves of O^T
  static constexpr int kKCols = D / 2;                   // TMEM columns of a key tile
  static constexpr int kVSlots = D == 256 ? 2 : D == 128 ? 3 : 4;  // slots of 64 tokens' values
  // TMEM columns
  static constexpr int kS = 0;
  static constexpr int kO = 2 * kN;
  static constexpr int kK = kO + kHalves * kN;
  static_assert(kK + 2 * kKCols <= 512, "TMEM columns");
  // shared memory (offsets from a 1024-byte aligned base)
  static constexpr int kQPart = kN * D * 2;  // a part of the queries
  static constexpr int kQBytes = (SPLIT ? 2 : 1) * kQPart;
  static constexpr int kVBytes = kTok / 2 * D * 2;
  static constexpr int kPCols = (SPLIT ? 2 : 1) * kN;    // columns of P: the lo parts behind all hi parts
  static constexpr int kPBytes = kTok * (kPCols < 64 ? 64 : kPCols) * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffV = kOffQ + kQBytes;
  static constexpr int kOffP = kOffV + kVSlots * kVBytes;
  static constexpr int kOffRows = kOffP + kPBytes;                 // int4 (p0, p1, w0, w1)[kN], int2 (base, bits)[kN]
  // floats [kN]: -reference, correction, slope; part [4][kN]
  static constexpr int kOffCol = kOffRows + (kN * (int)sizeof(RowSees) + 15) / 16 * 16;
  static constexpr int kOffQExp = kOffCol + 7 * kN * 4;            // int16 [kN]: exponents of the queries
  static constexpr int kOffMeta = kOffQExp + kN * 2;               // uint32 valid[kNorms][4], a bit per token
  static constexpr int kOffNorm = kOffMeta + kNorms * 16;  // float2 (nu_k, nu_v) [kNorms][128]
  static constexpr int kOffTab = (kOffNorm + kNorms * kTok * 8 + 127) / 128 * 128;  // key and value tables, ring
  static constexpr int kRegsDequant = D == 256 ? 96 : 64;
  static constexpr int kRegsSoft = (640 * 96 - 128 * (2 * kRegsDequant + kRegsIssue)) / 256 / 8 * 8;
};

// Bytes of a packed row's span in the ring: the 16-byte aligned span that holds a row wherever
// it starts (a multiple of 4), rounded to an odd number of 16-byte units: the words of 32 rows
// then meet four to a bank, no more.
__host__ __device__ constexpr int span_bytes(int d, int bits) {
  int s = (d * bits / 8 + 4 + 12 + 15) / 16 * 16;
  return (s / 16) % 2 ? s : s + 16;
}

// Lookup tables in shared memory: 4-byte entries, a copy for each lane (entry e of lane l at
// e * 128 + 4 l), so no lookup meets another lane's bank: pairs of centroids by the 2 b bits of
// two neighbouring indices, 5 bits single centroids.  4-bit values take none: 32 KB more would
// leave too little for the ring, and sharing the keys' table was slower than byte permutes (64 x
// 8192 tokens, K4/V4: tree 818 against 780 us, single tokens 322 against 306 us): the lookups load
// the shared-memory pipe, the permutes the integer pipe.
__host__ __device__ constexpr int key_table_bytes(int bits) { return (bits == 5 ? 32 : 1 << (2 * bits)) * 128; }
__host__ __device__ constexpr int value_table_bytes(int bits) { return bits == 4 ? 0 : key_table_bytes(bits); }

struct TcAttnArgs {
  AttnArgs a;
  AttnWork w;
  int ring;        // stages of packed rows, 1 .. kMaxRing
  int wide;        // slabs are whole 16 bytes: rows come in 16-byte copies (else by words)
  int bs_log;      // log2 of the block size, -1 if it is not a power of two
  uint32_t tries;  // of a bounded wait
};

// ---------------------------------------------------------------- primitives

__device__ __forceinline__ uint32_t smem_a(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {  // never suspends
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {  // by a whole warp, one elected lane
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
// D (+)= A B, kind::f16, A in TMEM or in shared memory, B in shared memory; called by a whole warp,
// issued by one elected lane (the operands stay in uniform registers that way).
// Descriptors come as their low words (address and leading offset); the high word is the same
// for all: eight rows (K-major) or k-lines (MN-major) of 128 bytes, the next eight 1024 bytes on,
// 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) {
  return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 bd;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 bd, {%2, %5};\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 ad, bd;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 ad, {%1, %5};\n mov.b64 bd, {%2, %5};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "n"(kDescHigh)
      : "memory");
}
// f16 x f16 -> f32, M 128; `mn`: both operands MN-major.
__device__ __forceinline__ uint32_t mma_idesc(int n, bool mn) {
  return (1u << 4) | (mn ? (1u << 15) | (1u << 16) : 0u) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void st_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t ld_s32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ex2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpa(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync %0, %1;\n" ::"n"(kBarSoft), "n"(kSoftThreads) : "memory"); }
__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool named_any(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
// Exponent of a power of two near x > 0 (finite): floor(log2 x), -126 for zero and subnormals.
__device__ __forceinline__ int exp_of(float x) { return max((int)((__float_as_uint(x) >> 23) & 0xffu) - 127, -126); }

// cap2 tanh(x / cap2) for caps of any size: near zero, where 1 - 2 / (1 + e^2h) would leave the
// roundings of numbers of the cap's size, by tanh's Taylor series to h^9 (the next term is 2.5e-7
// of the result at h = 0.35); beyond, those roundings are 1e-6 of the score at most.
__device__ __forceinline__ float far_cap(float x, float cap2, float inv_cap2) {
  const float h = x * inv_cap2, g = h * h;
  const float near = x * fmaf(g, fmaf(g, fmaf(g, fmaf(g, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
  const float far = fmaf(-2.f * cap2, rcpa(1.f + ex2a(2.f * kLog2eA * h)), cap2);
  return fabsf(h) < 0.35f ? near : far;
}

// ---------------------------------------------------------------- dequantisation

// 32 consecutive coordinates from the first BITS words of w, two per lookup (5 bits: one).
template <int BITS>
__device__ __forceinline__ void expand32_table(const uint32_t* w, uint32_t tab_lane, uint32_t (&out)[16]) {
  if constexpr (BITS == 5) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint32_t v[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int bit = 5 * (2 * i + k), j = bit >> 5, sh = bit & 31;
        const uint32_t f = (sh <= 27 ? w[j] >> sh : __funnelshift_r(w[j], w[j + 1], sh)) & 31u;
        v[k] = ld_s32(tab_lane + f * 128u);
      }
      out[i] = __byte_perm(v[0], v[1], 0x5410);
    }
  } else {
    constexpr int W = 2 * BITS;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int bit = W * i, j = bit >> 5, sh = bit & 31;
      uint32_t f;
      if constexpr (BITS == 4) f = __byte_perm(w[j], 0, 0x4440 + (sh >> 3));
      else f = (sh <= 32 - W ? w[j] >> sh : __funnelshift_r(w[j], w[j + 1], sh)) & ((1u << W) - 1u);
      out[i] = ld_s32(tab_lane + f * 128u);
    }
  }
}

// 4-bit values: centroids fp16(alpha c) as byte tables in registers, the low and the high bytes of
// eight entries per register pair.  A PRMT whose selector is four indices of three bits returns
// the bytes of four coordinates.  The codebook is odd (c[15 - i] = -c[i]), so eight magnitudes and
// a sign do; ODD false takes all 16 entries and a select by the fourth bit.
template <bool ODD>
struct ByteTable {
  uint32_t lo[ODD ? 2 : 4], hi[ODD ? 2 : 4];
  __device__ __forceinline__ void load(const float* c, float alpha) {
#pragma unroll
    for (int r = 0; r < (ODD ? 2 : 4); ++r) {
      lo[r] = hi[r] = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t u = __half_as_ushort(__float2half_rn(__ldg(c + (ODD ? 8 : 0) + 4 * r + k) * alpha));
        lo[r] |= (u & 255u) << (8 * k);
        hi[r] |= (u >> 8) << (8 * k);
      }
    }
  }
};

// Eight consecutive coordinates (a word) as four fp16 pairs.
template <bool ODD>
__device__ __forceinline__ void expand8(uint32_t w, const ByteTable<ODD>& t, uint32_t (&out)[4]) {
  uint32_t sel = w;
  if constexpr (ODD) sel ^= ((~w & 0x88888888u) >> 3) * 7u;  // index 7 - k is -c[8 + k]
  sel &= 0x77777777u;
  const uint32_t z = w << 4;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t s = k ? sel >> 16 : sel;
    uint32_t m;  // bytes 0xff where bit 3 of the index is set (the sign-replicating selector form)
    if (k == 0) asm("prmt.b32 %0, %1, %2, 0xd9c8;\n" : "=r"(m) : "r"(z), "r"(w));
    else asm("prmt.b32 %0, %1, %2, 0xfbea;\n" : "=r"(m) : "r"(z), "r"(w));
    uint32_t lo = __byte_perm(t.lo[0], t.lo[1], s), hi = __byte_perm(t.hi[0], t.hi[1], s);
    if constexpr (ODD) {
      hi |= ~m & 0x80808080u;
    } else {
      lo = (lo & ~m) | (__byte_perm(t.lo[2], t.lo[3], s) & m);
      hi = (hi & ~m) | (__byte_perm(t.hi[2], t.hi[3], s) & m);
    }
    out[2 * k] = __byte_perm(lo, hi, 0x5140);
    out[2 * k + 1] = __byte_perm(lo, hi, 0x7362);
  }
}

// ---------------------------------------------------------------- the kernel

template <int D, bool SPLIT, int N>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ TcAttnArgs p) {
  using C = Tc<D, SPLIT, N>;
  const AttnArgs& a = p.a;
  const AttnWork& w = p.w;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[kNorms + 27];
  __shared__ uint32_t tmem_slot;
  __shared__ int dead, fail[2][2], fail_all;
  __shared__ int full_lo_s, full_hi_s, pre_lo_s, pre_hi_s, q_low, q_high;
  unsigned char* smem = smem_raw + ((1024u - (smem_a(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_a(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.num_kv_heads, G = a.num_q_heads / H, g_log = 31 - __clz(G);  // G: a power of two
  const int h = blockIdx.x % H, part = blockIdx.x / H;
  const int rbk = D * a.k_bits / 8 + 4, rbv = D * a.v_bits / 8 + 4;
  const int spk = span_bytes(D, a.k_bits), spv = span_bytes(D, a.v_bits);
  const int skip_k = p.wide ? (h * rbk) % 16 : 0, skip_v = p.wide ? (h * rbv) % 16 : 0;
  const int stage_bytes = kTok * (spk + spv);
  const uint32_t ktab = base + C::kOffTab, vtab = ktab + key_table_bytes(a.k_bits);
  const uint32_t ring = vtab + value_table_bytes(a.v_bits);

  auto bar = [&](int i) -> uint32_t { return smem_a(bars) + 8u * i; };
  const int B0 = kNorms;
  auto n_full = [&](int b) { return bar(b); };  // values' norms of a tile
  auto k_full = [&](int b) { return bar(B0 + b); };
  auto k_empty = [&](int b) { return bar(B0 + 2 + b); };
  auto v_full = [&](int b) { return bar(B0 + 4 + b); };  // one per value slot
  auto v_empty = [&](int b) { return bar(B0 + 8 + b); };
  auto s_full = [&](int b) { return bar(B0 + 12 + b); };  // two per stream
  auto s_empty = [&](int b) { return bar(B0 + 16 + b); };
  auto p_full = [&](int s) { return bar(B0 + 20 + s); };  // one per stream
  auto p_empty = [&](int s) { return bar(B0 + 22 + s); };
  const uint32_t q_full = bar(B0 + 24), drained = bar(B0 + 25);
  volatile int* dead_v = &dead;

  // A bounded wait of one thread; a role that has seen another give up leaves too.
  auto wait1 = [&](uint32_t b, uint32_t parity) -> bool {
    for (uint32_t i = 0; i < p.tries; ++i) {
      if (__builtin_expect(bar_try(b, parity), 1)) return true;
      if (*dead_v) break;
    }
    *dead_v = 1;  // reported at the end
    return false;
  };
  // The same by a whole warp, with one answer.
  auto wait = [&](uint32_t b, uint32_t parity) -> bool { return __all_sync(kFullMask, wait1(b, parity)); };

  if (tid == 0) {
    dead = 0;
    fail[0][0] = fail[0][1] = fail[1][0] = fail[1][1] = fail_all = 0;
    for (int b = 0; b < kNorms; ++b) bar_init(n_full(b), kValWarps);
    for (int b = 0; b < 2; ++b) {
      bar_init(k_full(b), kKeyWarps);
      bar_init(k_empty(b), 1);
      bar_init(p_full(b), kSoftWarps);
      bar_init(p_empty(b), 1);
    }
    for (int b = 0; b < 4; ++b) {
      bar_init(v_full(b), kValWarps / 2);
      bar_init(v_empty(b), 1);
      bar_init(s_full(b), 1);
      bar_init(s_empty(b), kSoftWarps);
    }
    bar_init(q_full, kSoftWarps);
    bar_init(drained, 1);
    bar_init(drained + 8, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_a(&tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  {
    auto entry = [&](const float* c, float alpha, int e) -> uint32_t {
      return (uint32_t)__half_as_ushort(__float2half_rn(__ldg(c + e) * alpha));
    };
    const int kw = key_table_bytes(a.k_bits) / 4, vw = value_table_bytes(a.v_bits) / 4;
    uint32_t* t = reinterpret_cast<uint32_t*>(smem + C::kOffTab);
    const int mask = (1 << a.k_bits) - 1;
    for (int e = warp; e < kw / 32; e += kTcThreads / 32)
      t[e * 32 + lane] = a.k_bits == 5 ? entry(a.k_centroids, a.k_alpha, e)
                                       : entry(a.k_centroids, a.k_alpha, e & mask) |
                                             entry(a.k_centroids, a.k_alpha, e >> a.k_bits) << 16;
    const int vmask = (1 << a.v_bits) - 1;
    for (int e = warp; e < vw / 32; e += kTcThreads / 32)
      t[kw + e * 32 + lane] = a.v_bits == 5 ? entry(a.v_centroids, a.v_alpha, e)
                                            : entry(a.v_centroids, a.v_alpha, e & vmask) |
                                                  entry(a.v_centroids, a.v_alpha, e >> a.v_bits) << 16;
  }
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_slot;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  const int4 head = *reinterpret_cast<const int4*>(w.head);
  const int num_windows = head.x, total = head.y, lead = head.z;
  const int parts = live_parts(w, total);
  const int g0 = part < parts ? part_begin(total, part, parts) : 0;
  const int g1 = part < parts ? part_begin(total, part + 1, parts) : 0;
  // Calls f(window, first tile, end tile) for every window with tiles in this part.
  auto for_windows = [&](auto f) {
    if (g0 >= g1) return;
    for (int g = g0, wi = window_of(w, g0); g < g1 && wi < num_windows; ++wi) {
      const AttnWindow win = w.win[wi];
      const int first = max(0, g - win.tile_base), last = min(win.nA + win.nB, g1 - win.tile_base);
      if (last <= first) continue;
      g = win.tile_base + last;
      if (!f(win, first, last)) return;
    }
  };
  // Queries come rotated (q_rot, with the softmax scale), outputs leave in rotated space.
  auto tile_token = [&](const AttnWindow& win, int tile) -> int {
    return (tile < win.nA ? win.tA0 + tile : win.tB0 + tile - win.nA) * kTok;
  };
  auto pad_cols = [&](const AttnWindow& win) -> int { return (win.nrows * G + 15) / 16 * 16; };
  // Two streams of tiles when the window's MMA columns fit half of the TMEM regions.
  auto streams_of = [&](int padded) -> int { return padded <= C::kN / 2 ? 2 : 1; };

  // The part's tiles, from the window of its first place on.
  auto part_tiles = [&](int wi) -> int {
    if (lead == 0 || g0 >= g1) return g1 - g0;
    auto before = [&](int g, const AttnWindow& win) -> int {
      return win.tiles_before + max(0, min(win.nA + win.nB, g - win.tile_base));
    };
    return before(g1, w.win[window_of(w, g1)]) - before(g0, w.win[wi]);
  };

  // Packed rows: a lane copies the rows of its token itself, `ring` tiles deep, so no other thread
  // waits for them.  A cursor walks the part's tiles ahead of their use.
  struct Cursor {
    int g, wi, end, n_a, t_a, t_b, hi;  // place, window, place behind its tiles; its intervals, last token + 1
    const int32_t* table;
  };
  const int cap = (int)min((int64_t)a.max_blocks_per_seq * a.block_size, (int64_t)0x7fffff00);
  auto enter = [&](Cursor& c) {  // the window of the first tile at c.g (c.g < g1) or behind it, from c.wi on
    for (;; ++c.wi) {
      if (c.wi >= num_windows) {
        c.g = g1;
        return;
      }
      const AttnWindow win = w.win[c.wi];
      c.end = win.tile_base + win.nA + win.nB;
      if (c.g >= c.end) continue;
      c.g = max(c.g, win.tile_base);
      c.n_a = win.tile_base + win.nA;
      c.t_a = win.tA0 - win.tile_base;
      c.t_b = win.tB0 - c.n_a;
      c.hi = min(max(win.p_hi, win.w_hi), cap);
      c.table = a.block_table + (int64_t)win.seq * a.max_blocks_per_seq;
      return;
    }
  };
  // the table entry of token `lane_tok` of tile c.g (kNoToken: none there); then on to the next tile
  auto next_entry = [&](Cursor& c, int lane_tok, int& off) -> int {
    off = 0;
    if (c.g >= g1) return kNoToken;
    if (c.g >= c.end) {
      enter(c);
      if (c.g >= g1) return kNoToken;
    }
    const int tok = (c.g + (c.g < c.n_a ? c.t_a : c.t_b)) * kTok + lane_tok;
    ++c.g;
    if (tok >= c.hi) return kNoToken;
    const int col = p.bs_log >= 0 ? tok >> p.bs_log : tok / a.block_size;
    off = tok - col * a.block_size;
    return __ldg(c.table + col);
  };
  // Starts the copies of the row at (block, off) to `dst`; whether there is one.
  auto copy_row = [&](const uint8_t* from, int slab, int skip, int rb, uint32_t dst, int block, int off) -> bool {
    const bool ok = block >= 0 && block < a.num_blocks;
    if (ok) {
      const uint8_t* src = from + ((int64_t)block * a.block_size + off) * slab;
      if (p.wide) {
        for (int c = 0; c < skip + rb; c += 16)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst + c), "l"(src + c) : "memory");
      } else {
        for (int c = 0; c < rb; c += 4)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst + c), "l"(src + c) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    return ok;
  };
  // All but the newest ring - 1 groups of this thread have landed.
  auto landed = [&]() {
    switch (p.ring) {
      case 1: asm volatile("cp.async.wait_group 0;\n" ::: "memory"); break;
      case 2: asm volatile("cp.async.wait_group 1;\n" ::: "memory"); break;
      case 3: asm volatile("cp.async.wait_group 2;\n" ::: "memory"); break;
      case 4: asm volatile("cp.async.wait_group 3;\n" ::: "memory"); break;
      case 5: asm volatile("cp.async.wait_group 4;\n" ::: "memory"); break;
      default: asm volatile("cp.async.wait_group 5;\n" ::: "memory"); break;
    }
  };
  // Every MMA of an issuing warp has finished before TMEM is freed.
  auto drain = [&]() {
    const uint32_t b = drained + (warp == kMmaWarp ? 0 : 8);
    tc_commit(b);
    for (uint32_t i = 0; i < kDefaultWaitTries && !bar_try(b, 0); ++i) {
    }
    __syncwarp();
  };
  if (warp < kKeyWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kRegsDequant));
    // ------------------------------------------------ keys: packed row -> this lane of TMEM
    auto keys = [&](auto bits_tag) {
      constexpr int BITS = decltype(bits_tag)::value;
      constexpr int SPAN = span_bytes(D, BITS);
      const uint32_t tab = ktab + lane * 4;
      const int t_lane = warp * 32 + lane;
      const uint32_t row = ring + (uint32_t)(t_lane * SPAN);
      const uint32_t dst = tmem + ((uint32_t)(32 * warp) << 16) + C::kK;
      float2* norms = reinterpret_cast<float2*>(smem + C::kOffNorm);
      uint32_t* valid = reinterpret_cast<uint32_t*>(smem + C::kOffMeta);
      const uint8_t* from = a.k_pages + h * rbk - skip_k;
      Cursor cur{g0, g0 < g1 ? window_of(w, g0) : 0, g0, 0, 0, 0, 0, nullptr};  // (entered by the first entry)
      uint32_t there = 0;  // bit s: stage s holds a row
      const int n_tiles = part_tiles(cur.wi);
      int next_off, next = next_entry(cur, t_lane, next_off);  // entries are loaded a tile before their copies
      int st = 0;
      // (rounds before tile 0 only fill the ring)
#pragma unroll 1
      for (int it = -p.ring; it < n_tiles; ++it) {
        if (it >= 0) {
          landed();
          const uint32_t here = row + st * stage_bytes + skip_k;
          const bool ok = (there >> st) & 1u;
          // norms and validity go on to the softmax warps (what they say is ordered by k_full,
          // n_full, the product and its completion)
          const int slot = it % kNorms;
          norms[slot * kTok + t_lane].x = __uint_as_float(ld_s32(here + D * BITS / 8));
          const uint32_t m = __ballot_sync(kFullMask, ok);
          if (lane == 0) valid[4 * slot + warp] = m;
          const int b = it & 1;
          if (!wait(k_empty(b), ((it >> 1) & 1) ^ 1)) break;
          tc_after();
#pragma unroll 1
          for (int g = 0; g < D / 32; ++g) {
            uint32_t o[16];
            uint32_t wd[BITS + 1];
#pragma unroll
            for (int i = 0; i < BITS; ++i) wd[i] = ld_s32(here + 4 * (BITS * g + i));
            wd[BITS] = 0;
            expand32_table<BITS>(wd, tab, o);
            tm_st16(dst + b * C::kKCols + 16 * g, o);
          }
          tm_wait_st();
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(k_full(b));
        }
        // the stage's row has been read: the row `ring` tiles on
        const int block = next, off = next_off;
        next = next_entry(cur, t_lane, next_off);
        const bool copied = copy_row(from, H * rbk, skip_k, rbk, row + st * stage_bytes, block, off);
        there = copied ? there | (1u << st) : there & ~(1u << st);
        if (++st == p.ring) st = 0;
      }
    };
    if (a.k_bits == 4) keys(std::integral_constant<int, 4>{});
    else if (a.k_bits == 3) keys(std::integral_constant<int, 3>{});
    else if (a.k_bits == 2) keys(std::integral_constant<int, 2>{});
    else keys(std::integral_constant<int, 5>{});
    asm volatile("cp.async.wait_all;\n" ::: "memory");  // no copy outlives its use
  } else if (warp < kKeyWarps + kValWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kRegsDequant));
    // ------------------------------------------------ values: packed row -> swizzled k-line
    auto values = [&](auto bits_tag, auto odd_tag) {
      constexpr int BITS = decltype(bits_tag)::value;
      constexpr int SPAN = span_bytes(D, BITS);
      ByteTable<decltype(odd_tag)::value> table;
      if constexpr (BITS == 4) table.load(a.v_centroids, a.v_alpha);
      const uint32_t tab = vtab + lane * 4;
      const int half = (warp - kKeyWarps) >> 1, t = ((warp - kKeyWarps) & 1) * 32 + lane;  // token t of 64
      const int t_lane = 64 * half + t;
      const uint32_t row = ring + (uint32_t)(kTok * spk + t_lane * SPAN);
      const uint32_t line = base + C::kOffV + (uint32_t)((t >> 3) * 1024 + (t & 7) * 128);
      float2* norms = reinterpret_cast<float2*>(smem + C::kOffNorm);
      const uint8_t* from = a.v_pages + h * rbv - skip_v;
      Cursor cur{g0, g0 < g1 ? window_of(w, g0) : 0, g0, 0, 0, 0, 0, nullptr};  // (entered by the first entry)
      const int n_tiles = part_tiles(cur.wi);
      int next_off, next = next_entry(cur, t_lane, next_off);
      int st = 0;
      int slot = half % C::kVSlots, vph = 1;  // slot 2 it + half, round by round
#pragma unroll 1
      for (int it = -p.ring; it < n_tiles; ++it) {
        if (it >= 0) {
          landed();
          const uint32_t here = row + st * stage_bytes + skip_v;
          norms[(it % kNorms) * kTok + t_lane].y = __uint_as_float(ld_s32(here + D * BITS / 8));
          __syncwarp();
          if (lane == 0) bar_arrive(n_full(it % kNorms));
          if (!wait(v_empty(slot), vph)) break;
          const uint32_t to = line + slot * C::kVBytes;
#pragma unroll 1
          for (int g = 0; g < D / 32; ++g) {
            uint32_t o[16], wd[BITS + 1];
#pragma unroll
            for (int i = 0; i < BITS; ++i) wd[i] = ld_s32(here + 4 * (BITS * g + i));
            wd[BITS] = 0;
            if constexpr (BITS == 4) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t x[4];
                expand8(wd[e], table, x);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[4 * e + i] = x[i];
              }
            } else {
              expand32_table<BITS>(wd, tab, o);
            }
            const uint32_t at = to + (g >> 1) * (64 * 128) + (((uint32_t)(t & 7) ^ (uint32_t)(4 * (g & 1))) << 4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              st_v4(at ^ (uint32_t)(e << 4), o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          fence_async();
          __syncwarp();
          if (lane == 0) bar_arrive(v_full(slot));
          slot += 2;
          if (slot >= C::kVSlots) slot -= C::kVSlots, vph ^= 1;
        }
        const int block = next, off = next_off;
        next = next_entry(cur, t_lane, next_off);
        copy_row(from, H * rbv, skip_v, rbv, row + st * stage_bytes, block, off);
        if (++st == p.ring) st = 0;
      }
    };
    using No = std::integral_constant<bool, false>;
    if (a.v_bits == 4) {
      bool odd = true;  // the codebook's halves mirror each other
      for (int e = 0; e < 8; ++e) odd = odd && __ldg(a.v_centroids + e) == -__ldg(a.v_centroids + 15 - e);
      if (odd) values(std::integral_constant<int, 4>{}, std::integral_constant<bool, true>{});
      else values(std::integral_constant<int, 4>{}, No{});
    } else if (a.v_bits == 3) values(std::integral_constant<int, 3>{}, No{});
    else if (a.v_bits == 2) values(std::integral_constant<int, 2>{}, No{});
    else values(std::integral_constant<int, 5>{}, No{});
    asm volatile("cp.async.wait_all;\n" ::: "memory");
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kRegsSoft));
    // ------------------------------------------------ softmax, queries and outputs
    const int sw = warp - kKeyWarps - kValWarps;  // softmax warp
    const int quad = warp & 3, set = sw >> 2;
    const int stid = tid - 32 * (kKeyWarps + kValWarps);
    const int t_lane = 32 * quad + lane;  // token of the tile (dim of the output)
    int4* row_spans = reinterpret_cast<int4*>(smem + C::kOffRows);             // p0, p1, w0, w1
    int2* row_bits = reinterpret_cast<int2*>(smem + C::kOffRows + C::kN * 16);  // base, bits
    float* negm_s = reinterpret_cast<float*>(smem + C::kOffCol);  // -reference; -inf where there is no column
    float* corr_s = negm_s + C::kN;
    float* slope_s = corr_s + C::kN;
    float* part_s = slope_s + C::kN;  // [4][kN]
    short* q_exp_s = reinterpret_cast<short*>(smem + C::kOffQExp);
    const uint32_t* valid = reinterpret_cast<const uint32_t*>(smem + C::kOffMeta);
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    const float2* norms = reinterpret_cast<const float2*>(smem + C::kOffNorm);
    const uint32_t p_line = base + C::kOffP + (uint32_t)((t_lane >> 3) * 1024 + (t_lane & 7) * 128);
    const bool capped = cap_folded(a.softcap), far = a.softcap > 0.f && !capped, biased = a.alibi != nullptr;
    const float cap2 = a.softcap * kLog2eA, inv_cap2 = fminf(1.f / cap2, 3e38f);
    const float inv_av = kNormUnscale / (a.v_alpha * sqrtf((float)D));
    // 16 values of every lane to lane i's v[0], over all lanes, of value i % 16: halves of the values
    // exchanged four times, 16 shuffles in all.
    auto over_lanes = [&](float (&v)[16], auto op) {
#pragma unroll
      for (int m = 8; m >= 1; m >>= 1)
#pragma unroll
        for (int i = 0; i < m; ++i) {
          const float keep = lane & m ? v[i + m] : v[i], give = lane & m ? v[i] : v[i + m];
          v[i] = op(keep, __shfl_xor_sync(kFullMask, give, m));
        }
      v[0] = op(v[0], __shfl_xor_sync(kFullMask, v[0], 16));
    };
    int it = 0;
    uint32_t sph = 0, pph = 0;

    for_windows([&](const AttnWindow& win, int first, int last) -> bool {
      const int cols = win.nrows * G, padded = pad_cols(win);
      const int streams = streams_of(padded), pitch = C::kN / streams;
      const int sets = kSoftSets / streams, stream = set / sets;
      const int c_first = 16 * (set % sets), c_step = 16 * sets;  // this thread's groups of columns
      const int col0 = stream * pitch;                             // the stream's part of the column arrays
      const int bar_id = kBarSoft + 1 + stream, bar_n = 128 * sets;
      const uint32_t weight = (uint32_t)streams;  // arrivals of this warp where all softmax warps count
      // ---- queries of the window, rotated already: scaled by powers of two, hi (and lo)
      if (stid == 0) {
        full_lo_s = pre_lo_s = 0;
        full_hi_s = pre_hi_s = 0x7fffffff;
        q_low = 1000;
        q_high = kNoQuery;
      }
      const int64_t q_first = (int64_t)win.row0 * a.num_q_heads + h * G;  // (row, q head) of column 0
      auto q_index = [&](int c) -> int64_t { return q_first + (int64_t)(c >> g_log) * a.num_q_heads + (c & (G - 1)); };
      const float top = stid < cols ? w.q_top[q_index(stid)] : 0.f;  // (on its way with the row's lengths)
      soft_sync();
      if (stid < win.nrows) {
        const RowView v = row_view(a, win.row0 + stid);
        row_spans[stid] = make_int4(v.p0, v.p1, v.w0, v.w1);
        row_bits[stid] = make_int2(v.base, v.bits);
        atomicMax(&full_lo_s, v.w0);
        atomicMin(&full_hi_s, v.w1);
        atomicMax(&pre_lo_s, v.p0);
        atomicMin(&pre_hi_s, v.p1);
      }
      soft_sync();
      if (stid < C::kN) {
        const int c = stid & (pitch - 1);
        negm_s[stid] = c < cols ? -kNoMax : -INFINITY;  // no column there: never a new reference
        slope_s[stid] = biased && stid < cols ? a.alibi[h * G + (stid & (G - 1))] * kLog2eA : 0.f;
        // the largest coordinate to below 2^10; not of rows that see nothing, which may hold any bits
        int e = kNoQuery;
        if (stid < cols) {
          const int4 v = row_spans[stid >> g_log];
          if ((v.y > v.x || v.w > v.z || row_bits[stid >> g_log].y > 0) && top > 0.f && top < INFINITY)
            e = max(exp_of(top) - 9, -126);
        }
        q_exp_s[stid] = (short)e;
        const int high = __reduce_max_sync(kFullMask, e), low = __reduce_min_sync(kFullMask, e == kNoQuery ? 1000 : e);
        if (lane == 0) {
          atomicMax(&q_high, high);
          atomicMin(&q_low, low);
        }
      }
      soft_sync();
      // One power of two for all of them, which a token's factor takes back; where their sizes differ
      // by more than 2^kQuerySpread, so that the small ones would lose bits, one for each column, taken
      // back where scores are changed.
      const bool mixed = q_high - q_low > kQuerySpread;
      const int qe = q_high == kNoQuery ? 0 : q_high;
      auto q_exp_of = [&](int c) -> int {
        const int e = mixed ? q_exp_s[c] : kNoQuery;
        return e == kNoQuery ? qe : e;
      };
      const float q_up = mixed ? 1.f : pow2i(qe);
      const bool cold = mixed || far, always = capped || biased || cold;
      const int full_lo = full_lo_s, full_hi = full_hi_s, pre_lo = pre_lo_s, pre_hi = pre_hi_s;
      constexpr int kAhead = 4;  // columns loaded together
      for (int col4 = sw; col4 < cols; col4 += kAhead * kSoftWarps) {
        float v[kAhead][D / 32];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          load_floats<D / 32>(w.q_rot + q_index(min(col4 + e * kSoftWarps, cols - 1)) * D + lane * (D / 32), v[e]);
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          const int col = col4 + e * kSoftWarps;
          if (col >= cols) continue;
          const float q_down = pow2i(-q_exp_of(col));
#pragma unroll
          for (int i = 0; i < D / 32; i += 2) {
            const int d = lane * (D / 32) + i;
            const float x0 = v[e][i] * q_down, x1 = v[e][i + 1] * q_down;
            const uint32_t hi = pack2(x0, x1);
            const uint32_t at = (uint32_t)((d >> 6) * (C::kN * 128) + (((d & 63) * 2) & 15));
            const uint32_t ch = (uint32_t)((d & 63) >> 3);
            unsigned char* to = smem + C::kOffQ + at + col * 128 + ((ch ^ (col & 7)) << 4);
            *reinterpret_cast<uint32_t*>(to) = hi;
            if constexpr (SPLIT) {
              const __half2 hh = *reinterpret_cast<const __half2*>(&hi);
              *reinterpret_cast<uint32_t*>(to + C::kQPart) = pack2(x0 - __low2float(hh), x1 - __high2float(hh));
            }
          }
        }
      }
      fence_async();
      soft_sync();
      if (lane == 0) bar_arrive(q_full);

      // ---- tiles
      const int hi_tok = max(win.p_hi, win.w_hi), tiles = last - first;
      float2 l[C::kGroups * 8];
#pragma unroll
      for (int i = 0; i < C::kGroups * 8; ++i) l[i] = make_float2(0.f, 0.f);
      bool broken = false;
      for (int k = 0; k < tiles; ++k) {
        const int sb = k & (2 * streams - 1), slot = it++ % kNorms;
        const uint32_t this_s = (sph >> sb) & 1, this_p = (pph >> (k & (streams - 1))) & 1;
        sph ^= 1u << sb;
        pph ^= 1u << (k & (streams - 1));
        if ((k & (streams - 1)) != stream || broken) continue;
        const int t0 = tile_token(win, first + k), tok = t0 + t_lane;
        const uint32_t s_at = lanes + C::kS + sb * pitch;
        bool ok = wait(s_full(sb), this_s);
        tc_after();
        const float2 kv = norms[slot * kTok + t_lane];
        const uint4 vv = *reinterpret_cast<const uint4*>(valid + 4 * slot);
        const bool p_free = bar_test(p_empty(stream), this_p ^ 1);  // asked now, needed at the first store
        float kn = kv.x * q_up;
        const float vn = kv.y;
        const bool real = (((quad == 0 ? vv.x : quad == 1 ? vv.y : quad == 2 ? vv.z : vv.w) >> lane) & 1u) && tok < hi_tok;
        const bool all = (vv.x & vv.y & vv.z & vv.w) == 0xffffffffu && ((t0 >= full_lo && t0 + kTok <= full_hi) ||
                                                                         (t0 >= pre_lo && t0 + kTok <= pre_hi));
        // Scores of columns c0 .. c0 + 15.
        auto fetch = [&](int c0, float2 (&x)[8]) {
          uint32_t u[16];
          tm_ld16(s_at + c0, u);
          tm_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
        };
        bool seen = true;  // a column of this thread sees its token
        if (__builtin_expect(always || !all || __any_sync(kFullMask, fabsf(kn) > kLargeFactor), 0)) {
          if (__builtin_expect(cold, 0)) {
            // a query's own power of two, caps out of the ordinary; what follows finds the scores
            // like the others (a pass of its own, so that no code of it is among what runs often)
#pragma unroll 1
            for (int c0 = c_first; c0 < cols; c0 += c_step) {
              uint32_t u[16];
              tm_ld16(s_at + c0, u);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float x = __uint_as_float(u[i]) * kn * (mixed ? pow2i(q_exp_of(c0 + i)) : 1.f);
                u[i] = __float_as_uint(far ? far_cap(x, cap2, inv_cap2) : x);
              }
              tm_st16(s_at + c0, u);
            }
            tm_wait_st();
            kn = 1.f;
          }
          // Scores in place: nu_k, cap, distance, -inf where the token is not seen; what follows
          // takes them with a factor of one.  (A loop apart, so that plain tiles keep their code
          // together in the instruction cache.)
          seen = false;
          bool lost = false;  // a row sees this token, but its block lies outside the pages
#pragma unroll 1
          for (int c0 = c_first; c0 < cols; c0 += c_step) {
            float2 x[8];
            fetch(c0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(x[i], make_float2(kn, kn));
            if (capped) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                x[i].x = fmaf(-2.f * cap2, rcpa(1.f + ex2a(x[i].x)), cap2);
                x[i].y = fmaf(-2.f * cap2, rcpa(1.f + ex2a(x[i].y)), cap2);
              }
            }
            if (biased) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                x[i].x -= slope_s[c0 + 2 * i] * fabsf((float)(row_bits[(c0 + 2 * i) >> g_log].x - tok));
                x[i].y -= slope_s[c0 + 2 * i + 1] * fabsf((float)(row_bits[(c0 + 2 * i + 1) >> g_log].x - tok));
              }
            }
            uint32_t see = 0xffffu;  // bit i: column c0 + i
            if (!all) {
              see = 0;
              // (four rows together, so that their loads are)
              const int r_end = min((c0 + 16) >> g_log, win.nrows);
#pragma unroll 1
              for (int r0 = c0 >> g_log; r0 < r_end; r0 += 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int r = min(r0 + e, r_end - 1);
                  const int4 v = row_spans[r];
                  bool s = (tok >= v.z && tok < v.w) || (tok >= v.x && tok < v.y);
                  if (a.mask) {
                    const int2 b = row_bits[r];
                    const int j = tok - b.x;
                    const bool node = j >= 0 && j < b.y;
                    const uint32_t word =
                        __ldg(a.mask + (int64_t)(win.row0 + r) * a.mask_words + (node ? j >> 5 : 0));
                    s |= node && ((word >> (j & 31)) & 1u);
                  }
                  lost |= s && !real;
                  if (s && real) see |= ((1u << G) - 1u) << ((r << g_log) - c0);
                }
              }
            }
            seen |= see != 0;
            uint32_t u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              u[i] = (see >> i) & 1u ? __float_as_uint(i & 1 ? x[i >> 1].y : x[i >> 1].x) : 0xff800000u;
            tm_st16(s_at + c0, u);
          }
          tm_wait_st();
          kn = 1.f;
          if (lost && a.status) atomicMax(a.status, (int32_t)kBlockOutOfRange);
        }
        const float2 kn2 = make_float2(kn, kn);
        const bool vfin = fabsf(vn) < INFINITY;
        const float vs = vfin ? vn * kNormScale : 0.f, vs_top = fmaxf(fabsf(vs), kNormLow);
        const uint32_t sx = (uint32_t)(t_lane & 7);
        auto p_addr = [&](int c) -> uint32_t { return p_line + (c >> 6) * (kTok * 128) + ((((c & 63) >> 3) ^ sx) << 4); };
        volatile int* fl = &fail[stream][(k / streams) & 1];

        // The columns' references by the tile's largest products; where `sums`, the tile's weights
        // taken back out of the sums (a weight that moves a reference leaves a rounding of itself,
        // scaled away with it; an infinite one leaves nothing of the sum either), which go to the
        // new references with O^T.  Little code, as it runs seldom and then comes from far: with a
        // reduction per column and both passes unrolled it took 20 us a window.
        auto move_references = [&](bool sums) {
          // (rounded up throughout: a product may come out smaller for it, never too large)
          const float lv = __log2f(vs_top);
#pragma unroll 1
          for (int c0 = c_first; c0 < cols; c0 += c_step) {
            float2 x[8];
            float v[16];
            fetch(c0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[2 * i] = __fmaf_ru(x[i].x, kn, lv), v[2 * i + 1] = __fmaf_ru(x[i].y, kn, lv);
            over_lanes(v, [](float m, float n) { return fmaxf(m, n); });
            if (lane < 16) part_s[quad * C::kN + col0 + c0 + lane] = v[0];
          }
          named_sync(bar_id, bar_n);
          const int c = stid - 128 * sets * stream;  // a column for each thread of the stream
          if (c < cols) {
            float top = part_s[col0 + c];
#pragma unroll
            for (int i = 1; i < 4; ++i) top = fmaxf(top, part_s[i * C::kN + col0 + c]);
            const float old = -negm_s[col0 + c];
            top = __fadd_ru(top, -kProductExp);
            const bool up = top - old > kSlack;
            corr_s[col0 + c] = up ? ex2a(old - top) : 1.f;
            if (up) negm_s[col0 + c] = -top;
          }
          named_sync(bar_id, bar_n);
          if (!sums) return;
#pragma unroll
          for (int g = 0; g < C::kGroups; ++g) {
            const int c0 = c_first + c_step * g;
            if (c0 >= cols) continue;
            float2 x[8];
            fetch(c0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 m2 = *reinterpret_cast<const float2*>(negm_s + col0 + c0 + 2 * i);
              const float2 f2 = *reinterpret_cast<const float2*>(corr_s + col0 + c0 + 2 * i);
              const float2 y = __ffma2_rn(x[i], kn2, m2);
              float2& li = l[8 * g + i];
              // (a factor that underflows leaves nothing either)
              li.x = li.x == INFINITY || f2.x == 0.f ? 0.f : fmaf(li.x, f2.x, -ex2a(y.x));
              li.y = li.y == INFINITY || f2.y == 0.f ? 0.f : fmaf(li.y, f2.y, -ex2a(y.y));
            }
          }
          tc_after();
#pragma unroll 1
          for (int c0 = c_first; c0 < cols; c0 += c_step) {
#pragma unroll 1
            for (int hf = 0; hf < C::kHalves; ++hf) {
              const uint32_t at = lanes + C::kO + hf * C::kN + col0 + c0;
              uint32_t u[16];
              tm_ld16(at, u);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * corr_s[col0 + c0 + i]);
              tm_st16(at, u);
            }
          }
          tm_wait_st();
        };

        // Weights with the references as they are; when a column's has to move, the tile is taken
        // once more with the new ones.  A first tile has none yet.
        bool moved = k < streams, waited = false;
        for (;;) {
          if (__builtin_expect(moved, 0)) move_references(k >= streams);
          const float2 vs2 = make_float2(vs, vs);
          float over = 0.f;  // largest weight
#pragma unroll
          for (int g = 0; g < C::kGroups; ++g) {
            const int c0 = c_first + c_step * g;
            if (c0 >= cols) continue;
            float2 x[8];
            fetch(c0, x);
            uint32_t o[8], r[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 m4 = *reinterpret_cast<const float4*>(negm_s + col0 + c0 + 4 * i);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float2 y = __ffma2_rn(x[2 * i + e], kn2, e ? make_float2(m4.z, m4.w) : make_float2(m4.x, m4.y));
                y.x = ex2a(y.x);
                y.y = ex2a(y.y);
                over = fmaxf(over, fmaxf(y.x, y.y));
                l[8 * g + 2 * i + e] = __fadd2_rn(l[8 * g + 2 * i + e], y);
                y = __fmul2_rn(y, vs2);
                o[2 * i + e] = pack2(y.x, y.y);
                if constexpr (SPLIT) {
                  const __half2 hh = *reinterpret_cast<const __half2*>(&o[2 * i + e]);
                  r[2 * i + e] = pack2(y.x - __low2float(hh), y.y - __high2float(hh));
                }
              }
            }
            if (g == 0 && !waited) {  // the stream's product before is done: P and O are free
              if (!__all_sync(kFullMask, p_free)) ok = wait(p_empty(stream), this_p ^ 1) && ok;
              if (!ok) *fl = 1;
            }
            st_v4(p_addr(col0 + c0), o[0], o[1], o[2], o[3]);
            st_v4(p_addr(col0 + c0 + 8), o[4], o[5], o[6], o[7]);
            if constexpr (SPLIT) {
              st_v4(p_addr(C::kN + col0 + c0), r[0], r[1], r[2], r[3]);
              st_v4(p_addr(C::kN + col0 + c0 + 8), r[4], r[5], r[6], r[7]);
            }
          }
          const bool first_pass = !waited;
          waited = true;
          if (!first_pass) break;
          const bool move = !moved && over * vs_top > kMaxProduct;
          if (__builtin_expect(!named_any(bar_id, bar_n, move || !ok), 1)) break;
          if (*fl) {  // the same for all warps of the stream
            broken = true;
            break;
          }
          moved = true;
        }
        if (broken) continue;
        if (__builtin_expect(__any_sync(kFullMask, real && seen && !vfin), 0)) {
          // a value norm that is infinite or NaN: where its token has weight, the output takes it
          // (its weights above were zero)
#pragma unroll 1
          for (int c0 = c_first; c0 < cols; c0 += c_step) {
            float2 x[8];
            fetch(c0, x);
            if (!vfin && real && seen) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float y = (i & 1 ? x[i >> 1].y : x[i >> 1].x) * kn + negm_s[col0 + c0 + i];
                const uint32_t at = p_addr(col0 + c0 + (i & 8)) + 2 * (i & 7);
                const uint16_t v = !(ex2a(y) == 0.f) ? __half_as_ushort(__float2half_rn(vn)) : (uint16_t)0;
                asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(at), "h"(v) : "memory");
              }
            }
          }
        }
        fence_async();
        tc_before();
        __syncwarp();
        if (lane == 0) {
          bar_arrive_n(s_empty(sb), weight);
          bar_arrive_n(p_full(stream), weight);
        }
      }

      // ---- outputs of the window
      const int live = min(streams, tiles);  // streams that took a tile
      if (stream < live && !broken && !wait(p_empty(stream), ((pph >> stream) & 1) ^ 1)) broken = true;
      if (broken) *(volatile int*)&fail_all = 1;
      // sums over the 128 lanes
#pragma unroll
      for (int g = 0; g < C::kGroups; ++g) {
        const int c0 = c_first + c_step * g;
        if (c0 >= cols) continue;
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[2 * i] = l[8 * g + i].x, v[2 * i + 1] = l[8 * g + i].y;
        over_lanes(v, [](float m, float n) { return m + n; });
        if (lane < 16) part_s[quad * C::kN + col0 + c0 + lane] = v[0];
      }
      soft_sync();
      if (*(volatile int*)&fail_all) return false;
      tc_after();
      const int64_t slot0 = ((int64_t)blockIdx.x * 2 + (first == 0 ? 1 : 0)) * w.cols;
      const bool whole = first == 0 && last == win.nA + win.nB;
      if (stid < cols) {  // streams -> window: factors of their O^T
        const float ma = -negm_s[stid], mb = live > 1 ? -negm_s[pitch + stid] : kNoMax;
        const float top = fmaxf(ma, mb);
        const float fa = ex2a(ma - top), fb = live > 1 ? ex2a(mb - top) : 0.f;
        auto sum4 = [&](int c) -> float {
          return (part_s[c] + part_s[C::kN + c]) + (part_s[2 * C::kN + c] + part_s[3 * C::kN + c]);
        };
        const float sum = fa * sum4(stid) + (live > 1 ? fb * sum4(pitch + stid) : 0.f);
        const float f = !whole ? inv_av : sum != 0.f ? inv_av / sum : 0.f;
        corr_s[stid] = fa * f;
        if (live > 1) corr_s[pitch + stid] = fb * f;
        if (!whole) {
          w.ml[2 * (slot0 + stid)] = top;
          w.ml[2 * (slot0 + stid) + 1] = sum;
        }
      }
      soft_sync();
      // this lane's dim of columns c0 .. c0 + 15 (half hf of the dims)
      auto load_o = [&](int hf, int c0, float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
#pragma unroll 1
        for (int s = 0; s < live; ++s) {
          uint32_t u[16];
          tm_ld16(lanes + C::kO + hf * C::kN + s * pitch + c0, u);
          tm_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = fmaf(__uint_as_float(u[i]), corr_s[s * pitch + c0 + i], x[i]);
        }
      };
      // a whole window's rows take the place of its queries, a piece goes to its slot; the
      // combine rotates them back
#pragma unroll 1
      for (int c0 = 16 * set; c0 < cols; c0 += 16 * kSoftSets)
#pragma unroll 1
        for (int hf = 0; hf < C::kHalves; ++hf) {
          float x[16];
          load_o(hf, c0, x);
          if (D == 64 && quad >= 2) continue;  // lanes 64.. repeat the 64 dims
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c0 + i < cols)
              (whole ? w.q_rot + q_index(c0 + i) * D : w.acc + (slot0 + c0 + i) * D)[hf * 128 + t_lane] = x[i];
        }
      tc_before();
      soft_sync();  // the arrays and O are free for the next window
      return true;
    });
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsIssue));
    if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issue: scores
    // (the shuffles tell the compiler that the warp agrees; offsets are added to the low words of
    // the descriptors in units of 16 bytes: no carry leaves the address)
    const uint32_t q_at = desc_low(base + C::kOffQ, 16);
    int it = 0, unit = 0;
    uint32_t sph = 0;  // phases of the score buffers
    for_windows([&](const AttnWindow& win, int first, int last) -> bool {
      const int padded = __shfl_sync(kFullMask, pad_cols(win), 0);
      const int tiles = __shfl_sync(kFullMask, last - first, 0);
      const int streams = streams_of(padded), pitch = C::kN / streams;
      const uint32_t ids = mma_idesc(padded, false);
      if (!wait(q_full, unit & 1)) return false;
      ++unit;
      for (int k = 0; k < tiles; ++k, ++it) {
        const int b = it & 1, sb = k & (2 * streams - 1);
        if (!wait(k_full(b), (it >> 1) & 1) || !wait(n_full(it % kNorms), (it / kNorms) & 1) || !wait(s_empty(sb), ((sph >> sb) & 1) ^ 1)) return false;
        sph ^= 1u << sb;
        tc_after();
#pragma unroll 1
        for (int lo = 0; lo < (SPLIT ? 2 : 1); ++lo)
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ts(tmem + C::kS + sb * pitch, tmem + C::kK + b * C::kKCols + ks * 8,
                   q_at + ((lo * C::kQPart + (ks >> 2) * (C::kN * 128) + (ks & 3) * 32) >> 4), ids, lo > 0 || ks > 0);
        tc_commit(s_full(sb));
        tc_commit(k_empty(b));
      }
      return true;
    });
    drain();
    } else if (warp == kMmaWarp + 1) {
    // ------------------------------------------------ MMA issue: values
    const uint32_t v_at = desc_low(base + C::kOffV, D == 64 ? 0 : 64 * 128), p_at = desc_low(base + C::kOffP, kTok * 128);
    int vslot = 0, vph = 0;
    uint32_t pph = 0;  // phases of the streams' weights
    for_windows([&](const AttnWindow& win, int first, int last) -> bool {
      const int padded = __shfl_sync(kFullMask, pad_cols(win), 0);
      const int tiles = __shfl_sync(kFullMask, last - first, 0);
      const int streams = streams_of(padded), pitch = C::kN / streams;
      const uint32_t idp = mma_idesc(padded, true);
      for (int k = 0; k < tiles; ++k) {  // O^T of its stream += V^T P^T
        const int s = k & (streams - 1);
        auto p_of = [&](int c) -> uint32_t { return p_at + (uint32_t)(((c >> 6) * (kTok * 128) + (c & 63) * 2) >> 4); };
        const uint32_t p_s = p_of(s * pitch), p_lo = p_of(C::kN + s * pitch);
        const uint32_t o_s = tmem + C::kO + s * pitch;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (!wait(v_full(vslot), vph)) return false;
          if (half == 0 && !wait(p_full(s), (pph >> s) & 1)) return false;
          tc_after();
#pragma unroll
          for (int hf = 0; hf < C::kHalves; ++hf)
#pragma unroll
            for (int ks = 0; ks < kTok / 32; ++ks)
              mma_ss(o_s + hf * C::kN, v_at + ((vslot * C::kVBytes + hf * 2 * 64 * 128 + ks * 2048) >> 4),
                     p_s + ((half * (kTok / 2 * 128) + ks * 2048) >> 4), idp, k >= streams || half > 0 || ks > 0);
          if constexpr (SPLIT)
#pragma unroll
            for (int hf = 0; hf < C::kHalves; ++hf)
#pragma unroll
              for (int ks = 0; ks < kTok / 32; ++ks)
                mma_ss(o_s + hf * C::kN, v_at + ((vslot * C::kVBytes + hf * 2 * 64 * 128 + ks * 2048) >> 4),
                       p_lo + ((half * (kTok / 2 * 128) + ks * 2048) >> 4), idp, true);
          tc_commit(v_empty(vslot));
          if (++vslot == C::kVSlots) vslot = 0, vph ^= 1;
        }
        pph ^= 1u << s;
        tc_commit(p_empty(s));
      }
      return true;
    });
    drain();
    }
  }

  tc_before();
  __syncthreads();
  tc_after();
  if (tid == 0 && dead && a.status) atomicMax(a.status, (int32_t)kTimeout);
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
}

// ---------------------------------------------------------------- launch

template <int D, bool SPLIT, int N>
cudaError_t launch_tc(const AttnArgs& a, const AttnWork& w, cudaStream_t stream) {
  using C = Tc<D, SPLIT, N>;
  TcAttnArgs t{};
  t.a = a;
  t.w = w;
  t.tries = wait_tries();
  t.bs_log = -1;
  for (int k = 0; k < 31; ++k)
    if (a.block_size == (1 << k)) t.bs_log = k;
  const int rk = a.num_kv_heads * (D * a.k_bits / 8 + 4), rv = a.num_kv_heads * (D * a.v_bits / 8 + 4);
  const int spk = span_bytes(D, a.k_bits), spv = span_bytes(D, a.v_bits);
  t.wide = rk % 16 == 0 && rv % 16 == 0;
  constexpr int limit = 227 * 1024 - 448;  // the static arrays take their part
  const int stage = kTok * (spk + spv);
  const int fixed = 1024 + C::kOffTab + key_table_bytes(a.k_bits) + value_table_bytes(a.v_bits);
  t.ring = std::min(kMaxRing, (limit - fixed) / stage);
  // (one stage is left for 4-bit keys and 5-bit values of 256 channels, two or more otherwise)
  if (t.ring < 1) return cudaErrorInvalidValue;
  const int smem = fixed + t.ring * stage;
  auto kern = attn_tc_kernel<D, SPLIT, N>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(w.parts * a.num_kv_heads);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, kern, t);
  if (err == cudaSuccess) count_launches(1);
  return err;
}

}  // namespace

bool attn_tc_supported(const AttnArgs& a) {
  return (a.head_dim == 64 || a.head_dim == 128 || a.head_dim == 256) && (a.out_dtype == kF16 || a.out_dtype == kBF16);
}

// Columns of a window: as many as shared memory and TMEM allow, or 32 where the sequences' rows
// fill no more on average (single tokens, short trees): less code and a deeper ring (64 single
// tokens of 2000: 133 against 151 us; eight rows each: 155 against 182).  That average counts the
// table's idle rows too, and a long run of rows in narrow windows reads and expands every tile
// again for each of them (4 x 1000 rows in a table of 512: 3078 against 1227 us).  So it decides
// only where a wrong guess costs little, up to 2048 columns in all, and where the rows are no more
// than the sequences, as single tokens are; else windows are wide (256 sequences of eight rows then
// take 638 against 532 us).
constexpr int kFewCols = 32, kFewTotal = 2048;
constexpr int most_cols(int d, bool split) { return d < 256 ? (split ? 64 : 128) : split ? 32 : 64; }

// A window's start and end in tiles: 29 us beside 2.6 a tile at 128 columns (less where it holds
// fewer), 4.6 beside 1.7 where it is narrow.
int attn_tc_lead(int cols) { return cols == kFewCols ? 3 : kAttnMaxLead; }

int attn_tc_cols(const AttnArgs& a) {
  const int64_t cols = (int64_t)a.num_rows * (a.num_q_heads / a.num_kv_heads);
  const bool few = cols <= (int64_t)kFewCols * a.num_seqs && (cols <= kFewTotal || a.num_rows <= a.num_seqs);
  return few ? kFewCols : most_cols(a.head_dim, a.out_dtype == kF16);
}

cudaError_t launch_attn_tc(const AttnArgs& a, const AttnWork& w, cudaStream_t stream) {
  const bool few = w.cols == kFewCols;
  auto of = [&](auto dim, auto split) -> cudaError_t {
    constexpr int D = decltype(dim)::value;
    constexpr bool SPLIT = decltype(split)::value;
    if (few) return launch_tc<D, SPLIT, kFewCols>(a, w, stream);
    return launch_tc<D, SPLIT, most_cols(D, SPLIT)>(a, w, stream);
  };
  auto of_dim = [&](auto dim) -> cudaError_t {
    return a.out_dtype == kF16 ? of(dim, std::integral_constant<bool, true>{}) : of(dim, std::integral_constant<bool, false>{});
  };
  if (a.head_dim == 64) return of_dim(std::integral_constant<int, 64>{});
  if (a.head_dim == 128) return of_dim(std::integral_constant<int, 128>{});
  return of_dim(std::integral_constant<int, 256>{});
}

}  // namespace tq
