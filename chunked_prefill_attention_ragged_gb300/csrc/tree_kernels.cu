// The two small steps around tree attention: visibility of drafted nodes before it, and the
// accepted nodes' cache rows after it.
//
// tree_mask: a drafted node sees itself and its ancestors.  With parent(i) < i,
//   M(i) = {i} u M(parent(i)),  depth(i) = 1 + depth(parent(i)),  M(-1) = {}, depth(-1) = -1,
// written as bits, and its token position, context length + depth.  One CTA per tree, 256 nodes at a
// time, by doubling: with J the 2^k-th ancestor and M the nearest 2^k of them (itself the first),
//   M'(i) = M(i) u M(J(i)),  J'(i) = J(J(i)),
// log2(depth) steps in shared memory, as far as the ancestors are of the same 256; what is above the
// lowest of those is the finished row of its parent.  The depth is the number of bits less one.  Bound
// by latency (two loads, the steps, a store: 5 us, and 6 for 256 trees of up to 100 nodes, where one
// thread per node walking up its chain took 11); the work grows with nodes * mask_words only.
//
// tree_commit: row (s + path[i]) of the request moves to row (s + i), for i = 0 .. count - 1
// with path strictly increasing, so path[j] >= j.  A thread owns 16 bytes of the row in one
// layer and goes up i in groups of eight, all eight loads before the eight stores: a store to
// row i cannot hit a later source, because path[j] >= j > i.  No scratch, no barrier between
// the moves.  Bound by latency for one layer (path -> table -> row -> row), by HBM for many.
#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kMaskThreads = 128;
constexpr int kNodeWords = 4;
constexpr int kNodes = 64 * kNodeWords;   // nodes at a time

__device__ __forceinline__ void flag(int32_t* status) {
  if (status) atomicOr(status, MLA_DEVSTAT_BAD_INDEX);
}

__global__ void __launch_bounds__(kMaskThreads)
tree_mask_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ qo_indptr,
                 const int32_t* __restrict__ kv_lens, int64_t total_rows, int words, int64_t* mask, int32_t* positions, int32_t* status) {
  const int r = blockIdx.x;
  const int64_t q0 = qo_indptr[r], q1 = qo_indptr[r + 1];
  if (q0 < 0 || q1 < q0 || q1 > total_rows) {
    if (threadIdx.x == 0) flag(status);
    return;
  }
  const int n = (int)(q1 - q0);
  const int base = kv_lens ? kv_lens[r] - n : 0;
  const int32_t* par = parents + q0;
  __shared__ uint64_t m[2][kNodes][kNodeWords];
  __shared__ int16_t j[2][kNodes];      // ancestor inside the group, -1: none
  __shared__ int32_t above[kNodes];     // parent before the group, -1: none
  for (int i0 = 0; i0 < n; i0 += kNodes) {
    const int here = min(kNodes, n - i0), used = (here + 63) >> 6, w0 = i0 >> 6;
    bool bad = false;
    for (int i = threadIdx.x; i < here; i += kMaskThreads) {
      int up = __ldg(par + i0 + i);
      if (up < -1 || up >= i0 + i) {
        bad = true;
        up = -1;
      }
      bad |= i0 + i >= 64 * (int64_t)words;
      j[0][i] = (int16_t)(up >= i0 ? up - i0 : -1);
      above[i] = up >= i0 ? -1 : up;
      for (int w = 0; w < used; ++w) m[0][i][w] = (i >> 6) == w ? 1ull << (i & 63) : 0ull;
    }
    if (bad) flag(status);
    int at = 0;
    bool more = true;
    while (__syncthreads_or(more)) {   // halves what is left of the longest chain: at most 9 times
      more = false;
      for (int i = threadIdx.x; i < here; i += kMaskThreads) {
        const int up = j[at][i], far = up >= 0 ? j[at][up] : -1;
        for (int w = 0; w < used; ++w) m[at ^ 1][i][w] = m[at][i][w] | (up >= 0 ? m[at][up][w] : 0ull);
        j[at ^ 1][i] = (int16_t)far;
        more |= far >= 0;
      }
      at ^= 1;
    }
    // The chain leaves the group behind its lowest node here.
    for (int i = threadIdx.x; i < here; i += kMaskThreads) {
      int len = 0, top = -1;
      for (int w = 0; w < used; ++w) {
        const uint64_t bits = m[at][i][w];
        len += __popcll(bits);
        if (top < 0 && bits) top = 64 * w + __ffsll((long long)bits) - 1;
      }
      const int up = above[top];
      j[at ^ 1][i] = (int16_t)top;
      if (positions) positions[q0 + i0 + i] = (up >= 0 ? positions[q0 + up] : base - 1) + len;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < here * words; k += kMaskThreads) {   // (words <= 1024: fits)
      const int i = k / words, w = k - i * words;
      uint64_t bits = 0;
      if (w >= w0) {
        if (w - w0 < used) bits = m[at][i][w - w0];
      } else {
        const int up = above[j[at ^ 1][i]];
        if (up >= 0) bits = (uint64_t)mask[(q0 + up) * words + w];   // (written by this CTA, groups ago)
      }
      mask[(q0 + i0) * words + k] = (int64_t)bits;
    }
    __syncthreads();
  }
}

constexpr int kCommitThreads = 256;
constexpr int kCommitRows = 128;   // accepted rows resolved at a time
constexpr int kGroup = 8;

__global__ void __launch_bounds__(kCommitThreads)
tree_commit_kernel(const CommitParams p) {
  __shared__ int64_t src[kCommitRows], dst[kCommitRows];   // flat slots; -1: leave this row
  __shared__ int stop;
  const int r = blockIdx.y, tid = threadIdx.x;
  const int32_t* path = p.paths + (int64_t)r * p.max_accept;
  // The first rows' path entries come with the count, not after it.
  const bool mine = tid < kCommitRows && tid < p.max_accept;
  const int first_node = mine ? path[tid] : 0, first_before = mine && tid > 0 ? path[tid - 1] : -1;
  int count = p.counts[r];
  if (count < 0 || count > p.max_accept) {
    if (tid == 0 && blockIdx.x == 0) flag(p.status);
    count = min(max(count, 0), p.max_accept);
  }
  const int64_t base = p.seq_lens[r];
  const int chunks = p.row_chunks;
  const int64_t item = (int64_t)blockIdx.x * kCommitThreads + tid;
  const bool live = item < (int64_t)p.num_layers * chunks;
  uint4* column = nullptr;
  if (live) column = p.cache + (item / chunks) * p.layer_chunks + item % chunks;
  for (int i0 = 0; i0 < count; i0 += kCommitRows) {
    const int here = min(kCommitRows, count - i0);
    if (tid == 0) stop = here;
    __syncthreads();
    if (tid < here) {
      const int i = i0 + tid, node = i0 ? path[i] : first_node, before = i0 ? path[i - 1] : first_before;
      if (node < 0 || base < 0 || before >= node) atomicMin(&stop, tid);
      auto slot = [&](int64_t pos) -> int64_t {
        const int64_t bi = pos / p.block_size;
        if (pos < 0 || bi >= p.max_blocks) return -1;
        const int64_t blk = p.block_table[(int64_t)r * p.max_blocks + bi];
        return blk >= 0 && blk < p.num_blocks ? blk * p.block_size + (pos - bi * p.block_size) : -1;
      };
      int64_t a = -1, b = -1;
      if (node != i) {
        a = slot(base + node);
        b = slot(base + i);
        if (a < 0 || b < 0) {
          a = -1;
          if (blockIdx.x == 0) flag(p.status);
        }
      }
      src[tid] = a;
      dst[tid] = b;
    }
    __syncthreads();
    const int n = stop;
    if (live) {
      for (int k0 = 0; k0 < n; k0 += kGroup) {
        uint4 v[kGroup];
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
          if (k0 + k < n && src[k0 + k] >= 0) v[k] = column[src[k0 + k] * chunks];
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
          if (k0 + k < n && src[k0 + k] >= 0) column[dst[k0 + k] * chunks] = v[k];
      }
    }
    if (n < here) {   // not increasing from here on: nothing more is moved
      if (tid == 0 && blockIdx.x == 0) flag(p.status);
      return;
    }
    __syncthreads();   // src, dst and stop are reused
  }
}

}  // namespace

cudaError_t launch_tree_mask(const int32_t* parents, const int32_t* qo_indptr, const int32_t* kv_lens, int batch,
                             int64_t total_rows, int words, int64_t* mask, int32_t* positions, int32_t* status,
                             cudaStream_t stream) {
  tree_mask_kernel<<<batch, kMaskThreads, 0, stream>>>(parents, qo_indptr, kv_lens, total_rows, words, mask, positions,
                                                      status);
  return cudaGetLastError();
}

cudaError_t launch_tree_commit(const CommitParams& p, int batch, cudaStream_t stream) {
  const int64_t items = (int64_t)p.num_layers * p.row_chunks;
  const int64_t grid = (items + kCommitThreads - 1) / kCommitThreads;
  tree_commit_kernel<<<dim3((unsigned)grid, (unsigned)batch), kCommitThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
