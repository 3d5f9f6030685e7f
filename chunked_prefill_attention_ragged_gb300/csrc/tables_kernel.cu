// Block tables and slot maps from request lengths, on the GPU.
//
// For request r with s tokens in the cache and m new ones, the table has to name
// ceil((s + m) / block_size) blocks.  Blocks it holds beyond that go back on the free stack,
// missing ones are taken from its top, in request order; new token i of the request then
// lives at position p = s + i, flat slot table[r][p / block_size] * block_size + p % block_size
// (the slot rule of vLLM "vllm/models/deepseek_v4/sparse_mla.py",
// _build_c128a_topk_metadata_kernel, decode branch; slot -1 marks a token without a place).
//
// Everything is decided by exclusive prefix sums over the requests of (new tokens, blocks to
// give back, blocks to take), so the result does not depend on the order in which threads run.
// The sums are made by every CTA for itself (at most 8192 requests, a few per thread); then
// give back | take | slot map are three phases over flat lists of blocks or tokens, whose
// request is found by binary search in shared memory.  The phases are separated by barriers of
// one cluster, so that one launch does it all: what bounds the call is its latency (about
// 20 bytes per request and 8 per token).
#include <climits>

#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024;
constexpr int kClusterCtas = 8;

struct Sums {
  int64_t tok;
  int rel, need;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.tok + b.tok, a.rel + b.rel, a.need + b.need};
}
__device__ __forceinline__ Sums shfl_up(const Sums& a, int d) {
  return {__shfl_up_sync(0xffffffffu, a.tok, d), __shfl_up_sync(0xffffffffu, a.rel, d),
          __shfl_up_sync(0xffffffffu, a.need, d)};
}

__device__ __forceinline__ void flag(int32_t* status, int code) {
  if (status) atomicOr(status, code);
}

// The last r with start[r] <= x (start non-decreasing, start[0] = 0).
__device__ __forceinline__ int owner(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// One cluster (kCluster) or one CTA.
template <bool kCluster>
__global__ void __launch_bounds__(kThreads) tables_kernel(const TablesParams p) {
  extern __shared__ int smem[];
  const int b = p.batch, stride = b + 1;
  int* s_tok = smem;                  // exclusive sums, [b + 1]
  int* s_rel = s_tok + stride;
  int* s_need = s_rel + stride;
  int* s_held = s_need + stride;      // blocks held before, and after
  int* s_after = s_held + stride;
  __shared__ Sums warp_sum[kThreads / 32];
  __shared__ int s_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = kCluster ? (int)cluster_ctarank() : 0;
  const int nthr = kCluster ? kThreads * kClusterCtas : kThreads;
  const int gtid = rank * kThreads + tid;
  auto sync_all = [] {
    if constexpr (kCluster) cluster_sync(); else __syncthreads();
  };
  const int base_raw = p.free_count[0];
  const int base = min(max(base_raw, 0), p.free_capacity);
  if (gtid == 0 && base != base_raw) flag(p.status, MLA_DEVSTAT_BAD_INDEX);

  // Exclusive sums: a thread's consecutive requests, then its warp, then the CTA.
  const int per = (b + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, b), r1 = min(r0 + per, b);
  Sums mine{0, 0, 0};
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    int s = p.seq_lens[r], m = p.new_lens[r], h = p.num_held[r];
    bad |= s < 0 || m < 0 || h < 0 || h > p.max_blocks;
    s = max(s, 0);
    m = max(m, 0);
    h = min(max(h, 0), p.max_blocks);
    const int64_t target = ((int64_t)s + m + p.block_size - 1) / p.block_size;
    const bool fits = target <= p.max_blocks;
    bad |= !fits;
    const int want = fits ? (int)target : h;   // a request too long for its row changes nothing
    s_tok[r] = m;
    s_held[r] = h;
    s_after[r] = want;
    mine = mine + Sums{m, max(h - want, 0), max(want - h, 0)};
  }
  if (bad) flag(p.status, MLA_DEVSTAT_BAD_INDEX);
  Sums incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = shfl_up(incl, d);
    if (lane >= d) incl = incl + o;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) s_taken = 0;
  __syncthreads();
  Sums before{0, 0, 0}, total{0, 0, 0};
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before = before + warp_sum[w];
    total = total + warp_sum[w];
  }
  Sums run{before.tok + incl.tok - mine.tok, before.rel + incl.rel - mine.rel, before.need + incl.need - mine.need};
  const int released = total.rel;
  const int64_t top = (int64_t)base + released;   // stack height once everything is given back
  int taken = 0;
  bool short_of = false;
  for (int r = r0; r < r1; ++r) {
    const int m = s_tok[r], h = s_held[r], want = s_after[r];
    const int rel = max(h - want, 0), need = max(want - h, 0);
    s_tok[r] = (int)min(run.tok, (int64_t)INT_MAX);
    s_rel[r] = run.rel;
    s_need[r] = run.need;
    run = run + Sums{m, rel, need};
    // First come, first served: a request is served when all up to it can be.
    if (need > 0) {
      if (run.need <= top) taken = run.need;
      else { s_after[r] = h; short_of = true; }
    }
  }
  if (tid == 0) {
    s_tok[b] = (int)min(total.tok, (int64_t)INT_MAX);
    s_rel[b] = total.rel;
    s_need[b] = total.need;
    if (total.tok > INT_MAX || (p.slot_mapping && total.tok > p.num_tokens)) flag(p.status, MLA_DEVSTAT_BAD_INDEX);
  }
  if (short_of) flag(p.status, MLA_DEVSTAT_NO_BLOCKS);
  if (taken) atomicMax(&s_taken, taken);
  sync_all();   // every CTA has read the old state; the sums are in place
  taken = s_taken;

  // Give back: block k of the list goes where the k-th take from the top will look, so that
  // what a step reserved and gave back leaves the stack as it was.
  for (int k = gtid; k < released; k += nthr) {
    const int r = owner(s_rel, b, k);
    int32_t* entry = p.block_table + (int64_t)r * p.max_blocks + s_after[r] + (k - s_rel[r]);
    const int64_t at = top - 1 - k;
    const int blk = *entry;
    *entry = -1;
    if (at < p.free_capacity) p.free_blocks[at] = blk;
    else flag(p.status, MLA_DEVSTAT_BAD_INDEX);
  }
  for (int r = gtid; r <= b; r += nthr) {
    if (p.qo_indptr) p.qo_indptr[r] = s_tok[r];
    if (r < b) {
      p.num_held[r] = s_after[r];
      if (p.kv_lens) {
        const int64_t len = (int64_t)max(p.seq_lens[r], 0) + max(p.new_lens[r], 0);
        p.kv_lens[r] = (int)min(len, (int64_t)INT_MAX);
      }
    }
  }
  if (gtid == 0) p.free_count[0] = (int)min(top - taken, (int64_t)p.free_capacity);
  sync_all();

  for (int k = gtid; k < taken; k += nthr) {
    const int r = owner(s_need, b, k);
    const int64_t at = top - 1 - k;
    int blk = at < p.free_capacity ? p.free_blocks[at] : -1;
    if (blk < 0) {
      flag(p.status, MLA_DEVSTAT_BAD_INDEX);
      blk = -1;
    }
    p.block_table[(int64_t)r * p.max_blocks + s_held[r] + (k - s_need[r])] = blk;
  }
  if (!p.slot_mapping) return;
  sync_all();

  const int live = s_tok[b];
  for (int64_t t = gtid; t < p.num_tokens; t += nthr) {
    int64_t slot = -1;
    if (t < live) {
      const int r = owner(s_tok, b, (int)t);
      const int64_t pos = (int64_t)max(p.seq_lens[r], 0) + (t - s_tok[r]);
      const int64_t bi = pos / p.block_size;
      const int blk = bi < p.max_blocks ? p.block_table[(int64_t)r * p.max_blocks + bi] : -1;
      if (blk >= 0) slot = (int64_t)blk * p.block_size + (pos - bi * p.block_size);
    }
    p.slot_mapping[t] = slot;
  }
}

}  // namespace

cudaError_t launch_tables(const TablesParams& p, cudaStream_t stream) {
  const int smem = 5 * (p.batch + 1) * (int)sizeof(int);
  static PerDeviceOnce configured;
  cudaError_t e = configured.run([] {
    const int most = 5 * (kMaxTableBatch + 1) * (int)sizeof(int);
    cudaError_t r = cudaFuncSetAttribute(tables_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(tables_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (e != cudaSuccess) return e;
  if (p.num_tokens <= 4096) {
    tables_kernel<false><<<1, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kClusterCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kClusterCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tables_kernel<true>, p);
}

}  // namespace mla
