// Step planning (block tables, slot maps and row lists from request lengths) and the commit
// of accepted rows, sm_103a.
//
// TurboQuant docs: "vLLM Usage" (Slot Mapping: token t of a sequence sits at
// block_table[t / block_size] * block_size + t % block_size) and "Architecture" (Cache
// Storage Objects: PackedPageCache, addressed by flat slot).
//
// Plan.  With L_s cached tokens, n_s new ones and B_s blocks, sequence s needs
//   need_s = max(0, ceil((L_s + n_s) / bs) - B_s)
// new blocks; three exclusive prefix sums over the sequences -- of n_s, need_s and the
// returned blocks -- place every row, every new block and every returned block, so all
// outputs are written independently of one another.  ONE launch: a cluster of CTAs, each of
// which scans all the sequences (a few KB out of L2), then writes its share of the rows.  A
// cluster barrier between reading and writing lets every output be its own input (lengths,
// block counts, ring state).  A row finds its sequence by binary search of the prefix in
// shared memory.  Bound: latency for a decode step (a launch, one pass over the inputs, a scan,
// one barrier: 64 requests 6 us on the device), for a long prompt the latency of table reads on
// eight SMs (131072 rows of 1024 requests 23 us, 2.1 MB).
//
// Commit.  Accepted node j of a sequence moves from token ctx + path[j] to ctx + j, path
// strictly ascending, so path[j] >= j: a later source is never an earlier destination, and
// one thread per 16-byte column that takes the rows in order needs no buffer and no barrier; it
// keeps eight rows in flight.  One CTA takes a sequence's columns: its context length may be
// overwritten by the same call.  Bound: latency (1024 requests, 4096 rows moved, 9 MB: 7 us).
#include <cooperative_groups.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_step.h"

namespace cg = cooperative_groups;

namespace tq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
// Codes of tq_status that only the planner reports.
constexpr int32_t kOutOfBlocks = 7;

// One chunk of up to 1024 sequences in shared memory: exclusive prefixes over all sequences
// before each (rows, new blocks, returned blocks), and the lengths they came from.
struct PlanChunk {
  int64_t rows[kPlanThreads + 1];
  int64_t fresh[kPlanThreads + 1];
  int64_t back[kPlanThreads + 1];
  int32_t len[kPlanThreads];
  int32_t blocks[kPlanThreads];
  int64_t warp_sum[3][kPlanWarps];
};

__device__ __forceinline__ int64_t warp_scan(int64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(kFullMask, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The entry e of the prefix array p[0 .. n] with p[e] <= x < p[e + 1] (p[0] <= x < p[n]).
__device__ __forceinline__ int find_entry(const int64_t* p, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same from a known entry lo at or before it: doubling steps, then halves.  Rows of a warp
// are neighbours, so the entry is the known one or close behind it.
__device__ __forceinline__ int find_from(const int64_t* p, int n, int lo, int64_t x) {
  int step = 1;
  while (lo + step < n && p[lo + step] <= x) lo += step, step *= 2;
  for (; step >= 1; step >>= 1)
    if (lo + step < n && p[lo + step] <= x) lo += step;
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_step_kernel(PlanArgs a) {
  __shared__ PlanChunk c;
  __shared__ int bad_any;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = a.num_seqs, bs = a.block_size;
  const int64_t W = a.max_blocks_per_seq, NB = a.num_blocks;
  const int chunks = (S + kPlanThreads - 1) / kPlanThreads;
  const int64_t head = a.free_state[0], count = a.free_state[1];
  if (tid == 0) bad_any = 0;

  // Loads chunk k and scans it on top of (rows0, fresh0, back0); advances the three.
  auto scan_chunk = [&](int k, int64_t& rows0, int64_t& fresh0, int64_t& back0) {
    const int s = k * kPlanThreads + tid;
    int64_t v[3] = {0, 0, 0};
    __syncthreads();  // the chunk before is done with the arrays
    if (s < S) {
      const int64_t len = a.seq_lens[s], blk = a.seq_blocks[s], add = a.new_lens[s];
      bool bad = len < 0 || blk < 0 || blk > W || len > blk * bs;
      if (add < 0) {
        v[2] = blk;
      } else {
        const int64_t want = (len + add + bs - 1) / bs;
        bad |= want > W || len + add > 0x7fffffffLL;
        v[0] = add;
        v[1] = want > blk ? want - blk : 0;
      }
      if (bad) {
        bad_any = 1;
        v[0] = v[1] = v[2] = 0;
      }
      c.len[tid] = (int32_t)len;
      c.blocks[tid] = (int32_t)blk;
    }
    int64_t incl[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      incl[q] = warp_scan(v[q]);
      if (lane == 31) c.warp_sum[q][warp] = incl[q];
    }
    __syncthreads();
    if (warp < 3) {
      const int64_t w = c.warp_sum[warp][lane];
      const int64_t wi = warp_scan(w);
      c.warp_sum[warp][lane] = wi - w;
    }
    __syncthreads();
    const int64_t base[3] = {rows0, fresh0, back0};
    int64_t* out[3] = {c.rows, c.fresh, c.back};
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int64_t e = base[q] + c.warp_sum[q][warp] + incl[q];
      out[q][tid + 1] = e;
      if (tid == 0) out[q][0] = base[q];
    }
    __syncthreads();
    rows0 = c.rows[kPlanThreads];
    fresh0 = c.fresh[kPlanThreads];
    back0 = c.back[kPlanThreads];
  };

  // ---- totals and the all-or-nothing checks --------------------------------------------
  __syncthreads();
  int64_t rows = 0, fresh = 0, back = 0;
  for (int k = 0; k < chunks; ++k) scan_chunk(k, rows, fresh, back);
  int32_t code = kOk;
  if (bad_any || rows > a.max_rows || head < 0 || count < 0 || count > NB || (NB > 0 ? head >= NB : head != 0))
    code = kInvalidArg;
  else if (fresh > count) code = kOutOfBlocks;
  else if (count + back > NB) code = kInvalidArg;  // returned entries would meet those being taken
  if (rank == 0 && tid == 0 && a.status) *a.status = code;
  if (code != kOk) rows = fresh = back = 0;

  // ---- outputs, chunk by chunk -----------------------------------------------------------
  int64_t r0 = 0, f0 = 0, b0 = 0;
  for (int k = 0; k < chunks; ++k) {
    const int64_t rfirst = r0, bfirst = b0;
    if (chunks > 1) scan_chunk(k, r0, f0, b0);
    else r0 = rows, b0 = back;
    cluster.sync();  // every CTA has read this chunk's inputs and the ring state
    const int n = min(kPlanThreads, S - k * kPlanThreads);
    const int s = k * kPlanThreads + tid;
    if (tid < n && warp % ranks == rank) {
      const bool gone = c.back[tid + 1] > c.back[tid];
      const int64_t add = c.rows[tid + 1] - c.rows[tid], more = c.fresh[tid + 1] - c.fresh[tid];
      const bool drop = code == kOk && (gone || a.new_lens[s] < 0);
      a.row_start[s] = code == kOk ? (int32_t)c.rows[tid] : 0;
      a.seq_lens_out[s] = drop ? 0 : (int32_t)(c.len[tid] + (code == kOk ? add : 0));
      a.seq_blocks_out[s] = drop ? 0 : (int32_t)(c.blocks[tid] + (code == kOk ? more : 0));
    }
    if (code != kOk) continue;
    // rows: slot, sequence, length; the first token of a new block also enters it in the table
    // (a warp takes consecutive rows; in a long step four rounds of 32 are in flight, searched from
    // the entry of the row before: 28 -> 23 us for 131072 rows of 1024 sequences)
    const int64_t warps = (int64_t)ranks * kPlanWarps;
    const int64_t share = (r0 - rfirst + warps * 32 - 1) / (warps * 32) * 32;
    const int64_t wr = rfirst + ((int64_t)rank * kPlanWarps + warp) * share, wr_end = min(r0, wr + share);
    int near = 0;
    auto take = [&](auto tag, int64_t rb) {
      constexpr int U = decltype(tag)::value;
      int e[U];
      int64_t t[U], col[U];
      int32_t block[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = rb + 32 * u + lane;
        e[u] = U == 1 ? find_entry(c.rows, n, min(r, wr_end - 1)) : find_from(c.rows, n, near, min(r, wr_end - 1));
        t[u] = c.len[e[u]] + (min(r, wr_end - 1) - c.rows[e[u]]);
        // lengths stay below 2^31: a table row holds at most that many tokens
        col[u] = (uint32_t)t[u] / (uint32_t)bs;
        if (col[u] < c.blocks[e[u]]) {
          block[u] = a.block_table[(int64_t)(k * kPlanThreads + e[u]) * W + col[u]];
        } else {
          int64_t pos = head + c.fresh[e[u]] + (col[u] - c.blocks[e[u]]);
          if (pos >= NB) pos -= NB;
          block[u] = a.free_blocks[pos];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = rb + 32 * u + lane;
        if (r >= wr_end) continue;
        const int seq = k * kPlanThreads + e[u];
        if (col[u] >= c.blocks[e[u]] && t[u] == col[u] * bs) a.block_table[(int64_t)seq * W + col[u]] = block[u];
        const bool ok = block[u] >= 0 && block[u] < NB;
        if (!ok && a.status) atomicMax(a.status, (int32_t)kBlockOutOfRange);
        a.slots[r] = ok ? (int64_t)block[u] * bs + (t[u] - col[u] * bs) : -1;
        a.q_seq[r] = seq;
        a.q_len[r] = (int32_t)(t[u] + 1);
      }
      near = __shfl_sync(kFullMask, e[U - 1], 31);
    };
    if (share <= 32) {
      if (wr < wr_end) take(std::integral_constant<int, 1>{}, wr);
    } else {
      if (wr < wr_end) near = find_entry(c.rows, n, wr);
      for (int64_t rb = wr; rb < wr_end; rb += 128) take(std::integral_constant<int, 4>{}, rb);
    }
    // returned blocks, to the tail of the ring
    for (int64_t p = bfirst + (int64_t)rank * kPlanThreads + tid; p < b0; p += (int64_t)ranks * kPlanThreads) {
      const int e = find_entry(c.back, n, p);
      int64_t pos = head + count + p;
      pos -= pos / NB * NB;
      a.free_blocks[pos] = a.block_table[(int64_t)(k * kPlanThreads + e) * W + (p - c.back[e])];
    }
  }
  if (chunks == 0) cluster.sync();
  // rows behind the last one
  for (int64_t r = rows + (int64_t)rank * kPlanThreads + tid; r < a.max_rows; r += (int64_t)ranks * kPlanThreads) {
    a.slots[r] = -1;
    a.q_seq[r] = -1;
    a.q_len[r] = 0;
  }
  if (rank == 0 && tid == 0) {
    a.row_start[S] = (int32_t)rows;
    int64_t h = head + fresh;
    if (code == kOk && h >= NB && NB > 0) h -= NB;
    a.free_state_out[0] = (int32_t)h;
    a.free_state_out[1] = (int32_t)(count - fresh + back);
  }
}

// ---------------------------------------------------------------- commit

constexpr int kCommitMaxThreads = 1024;
constexpr int kCommitChunk = 64;  // path entries staged at a time
constexpr int kCommitBatch = 8;   // rows in flight per thread

template <typename V>
__global__ void __launch_bounds__(kCommitMaxThreads) commit_tree_kernel(CommitArgs a) {
  __shared__ int64_t src[kCommitChunk], dst[kCommitChunk];  // flat slots; -1: nothing to move
  const int s = blockIdx.x, tid = threadIdx.x, bs = a.block_size, threads = blockDim.x;
  const int64_t cap = min((int64_t)a.max_blocks_per_seq * bs, (int64_t)0x7fffffff);  // lengths are int32
  const int kcols = a.k_slab / (int)sizeof(V), vcols = a.v_slab / (int)sizeof(V);
  const int64_t ctx = a.ctx_lens[s];
  int n = a.path_lens[s];
  const int32_t* path = a.path + (int64_t)s * a.max_path;
  int bad = ctx < 0 || ctx > cap || n < 0 || n > a.max_path;
  if (bad) n = 0;
  for (int j = tid; j < n; j += threads) {
    const int p = path[j];
    bad |= p < 0 || ctx + p >= cap || (j > 0 && path[j - 1] >= p);
  }
  bad = __syncthreads_or(bad);
  if (bad) n = 0;
  if (tid == 0) {
    a.seq_lens_out[s] = (int32_t)(ctx + n);
    if (bad && a.status) atomicMax(a.status, (int32_t)kInvalidArg);
  }
  const int32_t* table = a.block_table + (int64_t)s * a.max_blocks_per_seq;
  for (int j0 = 0; j0 < n; j0 += kCommitChunk) {
    const int m = min(kCommitChunk, n - j0);
    __syncthreads();
    if (tid < m) {
      const int64_t from = ctx + path[j0 + tid], to = ctx + j0 + tid;
      const int64_t fb = table[from / bs], tb = table[to / bs];
      const bool ok = fb >= 0 && fb < a.num_blocks && tb >= 0 && tb < a.num_blocks;
      if (!ok && a.status) atomicMax(a.status, (int32_t)kBlockOutOfRange);
      src[tid] = ok && from != to ? fb * bs + from % bs : -1;
      dst[tid] = tb * bs + to % bs;
    }
    __syncthreads();
    for (int col = tid; col < kcols + vcols; col += threads) {
      const bool key = col < kcols;
      V* base = reinterpret_cast<V*>(key ? a.k_pages : a.v_pages) + (key ? col : col - kcols);
      const int64_t stride = key ? kcols : vcols;
      for (int j = 0; j < m; j += kCommitBatch) {
        V v[kCommitBatch];
#pragma unroll
        for (int u = 0; u < kCommitBatch; ++u)
          if (j + u < m && src[j + u] >= 0) v[u] = base[src[j + u] * stride];
#pragma unroll
        for (int u = 0; u < kCommitBatch; ++u)
          if (j + u < m && src[j + u] >= 0) base[dst[j + u] * stride] = v[u];
      }
    }
  }
}

template <typename V>
cudaError_t launch_commit_as(const CommitArgs& a, cudaStream_t stream) {
  // a thread per column, at least as many as path entries are staged at a time
  const int cols = (a.k_slab + a.v_slab) / (int)sizeof(V);
  const int threads = std::min(kCommitMaxThreads, std::max(128, (cols + 31) / 32 * 32));
  static_assert(kCommitChunk <= 128, "entries are staged one a thread");
  commit_tree_kernel<V><<<a.num_seqs, threads, 0, stream>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) count_launches(1);
  return err;
}

}  // namespace

cudaError_t launch_plan_step(const PlanArgs& a, cudaStream_t stream) {
  // one CTA up to 4096 rows (4 a thread), then one more per 4096 rows up to a portable
  // cluster of 8: a larger cluster costs a longer barrier
  int ranks = 1;
  while (ranks < 8 && a.max_rows > (int64_t)ranks * 4096) ranks *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, plan_step_kernel, a);
  if (err == cudaSuccess) count_launches(1);
  return err;
}

cudaError_t launch_commit_tree(const CommitArgs& a, cudaStream_t stream) {
  if (a.status) {
    const cudaError_t err = cudaMemsetAsync(a.status, 0, sizeof(int32_t), stream);
    if (err != cudaSuccess) return err;
  }
  if (a.num_seqs == 0) return cudaSuccess;
  const int both = a.k_slab | a.v_slab;  // the widest column every token's slab is a multiple of
  if (both % 16 == 0) return launch_commit_as<uint4>(a, stream);
  if (both % 4 == 0) return launch_commit_as<uint32_t>(a, stream);
  if (both % 2 == 0) return launch_commit_as<uint16_t>(a, stream);
  return launch_commit_as<uint8_t>(a, stream);
}

}  // namespace tq
