// Block tables and slot maps from request lengths, on the GPU.
//
// For request r with s tokens in the cache and m new ones, the table has to name
// ceil((s + m) / block_size) blocks.  Blocks it holds beyond that go back on the free stack,
// missing ones are taken from its top, in request order; new token i of the request then
// lives at position p = s + i, flat slot table[r][p / block_size] * block_size + p % block_size (-1:
// a token without a place).
//
// Everything is decided by exclusive prefix sums over the requests of (new tokens, blocks given
// back, blocks to take), so that the result does not depend on the order in which threads run.  With
// R blocks given back and the stack's height c before, the k-th block taken is the one at stack index
// c + R - 1 - k, where block k of those given back goes: so for k < R it is that block itself, which
// moves from one table row to the other without the stack between, and every block is one thread's.
//
// Entries of a row behind those in use may hold anything.  A request that is not served would reach them:
// as far as it would have needed them they are made -1, so that neither its slots here nor the calls that
// read the table next (a commit writes by it) touch a block that it does not hold.
//
// Two forms.  Up to 8192 tokens to map, one CTA does it all: sums, blocks, slots, with its own
// barriers between (what bounds it is latency: about 20 bytes per request and 8 per token).  More,
// and one kernel moves the blocks and a second one writes the lengths and the slots, each CTA of
// both making the sums for itself (at most 8192 requests, a few per thread): the map of 530 thousand
// tokens took 77 us from eight CTAs and 9 us from a grid.  A call that takes blocks for 256 requests and
// one that gives them back, together, by the first and the second form: 12.3 and 18.5 us for 1024
// tokens, 24.6 both for 8192, 34.8 and 22.6 for 16384.
#include <climits>

#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int64_t kOneCtaTokens = 8192;
constexpr int kSlotThreads = 512, kSlotsPerThread = 4;

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

// The sums in shared memory (exclusive, [batch + 1] each), and what a request holds before and after.
struct Shared {
  int *tok, *rel, *need, *held, *after;
  int taken;      // blocks taken: the needs of the requests that are served, a prefix of those that need any
  int released;
  int base;       // height of the stack before
  int64_t top;    // height with everything given back
  bool refused;   // some request is not served
};

// Blocks that a request of l cached and m new tokens needs.
__device__ __forceinline__ int64_t blocks_of(const TablesParams& p, int l, int m) {
  return ((int64_t)max(l, 0) + max(m, 0) + p.block_size - 1) / p.block_size;
}

__device__ void make_sums(const TablesParams& p, int* smem, bool report, Shared* out) {
  __shared__ Sums warp_sum[kMaxThreads / 32];
  __shared__ int s_taken;
  const int b = p.batch, stride = b + 1, threads = blockDim.x;
  Shared s;
  s.tok = smem;
  s.rel = s.tok + stride;
  s.need = s.rel + stride;
  s.held = s.need + stride;
  s.after = s.held + stride;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int count = p.free_count[0];
  const int per = (b + threads - 1) / threads;
  const int r0 = min(tid * per, b), r1 = min(r0 + per, b);
  Sums mine{0, 0, 0};
  bool bad = false, refused = false;
  for (int r = r0; r < r1; ++r) {
    int l = p.seq_lens[r], m = p.new_lens[r], h = p.num_held[r];
    bad |= l < 0 || m < 0 || h < 0 || h > p.max_blocks;
    l = max(l, 0);
    m = max(m, 0);
    h = min(max(h, 0), p.max_blocks);
    bad |= (int64_t)l + m > INT_MAX;   // (kv_lens says INT_MAX)
    const int64_t target = blocks_of(p, l, m);
    const bool fits = target <= p.max_blocks;
    bad |= !fits;
    refused |= !fits;
    const int want = fits ? (int)target : h;   // a request too long for its row changes nothing
    s.tok[r] = m;
    s.held[r] = h;
    s.after[r] = want;
    mine = mine + Sums{m, max(h - want, 0), max(want - h, 0)};
  }
  if (report && bad) flag(p.status, MLA_DEVSTAT_BAD_INDEX);
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
  for (int w = 0; w < threads / 32; ++w) {
    if (w < warp) before = before + warp_sum[w];
    total = total + warp_sum[w];
  }
  Sums run{before.tok + incl.tok - mine.tok, before.rel + incl.rel - mine.rel, before.need + incl.need - mine.need};
  s.released = total.rel;
  s.base = min(max(count, 0), p.free_capacity);
  s.top = (int64_t)s.base + s.released;
  int taken = 0;
  bool short_of = false;
  for (int r = r0; r < r1; ++r) {
    const int m = s.tok[r], h = s.held[r], want = s.after[r];
    const int rel = max(h - want, 0), need = max(want - h, 0);
    s.tok[r] = (int)min(run.tok, (int64_t)INT_MAX);
    s.rel[r] = run.rel;
    s.need[r] = run.need;
    run = run + Sums{m, rel, need};
    // First come, first served: a request is served when all up to it can be.
    if (need > 0) {
      if (run.need <= s.top) taken = run.need;
      else { s.after[r] = h; short_of = true; }
    }
  }
  if (tid == 0) {
    s.tok[b] = (int)min(total.tok, (int64_t)INT_MAX);
    s.rel[b] = total.rel;
    s.need[b] = total.need;
    if (report && (count != s.base || total.tok > INT_MAX || (p.slot_mapping && total.tok > p.num_tokens)))
      flag(p.status, MLA_DEVSTAT_BAD_INDEX);
  }
  if (report && short_of) flag(p.status, MLA_DEVSTAT_NO_BLOCKS);
  if (taken) atomicMax(&s_taken, taken);
  s.refused = __syncthreads_or(refused || short_of) != 0;
  s.taken = s_taken;
  *out = s;
}

// The entries that a request which is not served would have needed beyond those it holds; a warp a row.
__device__ __forceinline__ void clear_refused(const TablesParams& p, const Shared& s, int first, int step) {
  for (int r = first >> 5; r < p.batch; r += step >> 5) {
    const int held = s.after[r], end = (int)min(blocks_of(p, p.seq_lens[r], p.new_lens[r]), (int64_t)p.max_blocks);
    for (int j = held + (threadIdx.x & 31); j < end; j += 32) p.block_table[(int64_t)r * p.max_blocks + j] = -1;
  }
}

// Block k of those given back or taken, for k = first, first + step, ...: out of its row, into the
// row that takes it or onto the stack; or off the stack into the row.
__device__ __forceinline__ void move_blocks(const TablesParams& p, const Shared& s, int first, int step) {
  constexpr int kAtOnce = 4;   // loads under way together
  const int n = max(s.released, s.taken);
  for (int64_t k0 = first; k0 < n; k0 += kAtOnce * step) {
    int32_t* entry[kAtOnce];
    int blk[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int64_t k = k0 + i * step;
      const int64_t at = s.top - 1 - k;
      entry[i] = nullptr;
      blk[i] = -1;
      if (k < s.released) {
        const int r = owner(s.rel, p.batch, (int)k);
        entry[i] = p.block_table + (int64_t)r * p.max_blocks + s.after[r] + (k - s.rel[r]);
        blk[i] = *entry[i];
      } else if (k < n && at < p.free_capacity) {
        blk[i] = p.free_blocks[at];
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int64_t k = k0 + i * step;
      const int64_t at = s.top - 1 - k;
      if (k >= n) break;
      if (entry[i]) *entry[i] = -1;
      if (k < s.taken) {
        if (blk[i] < 0) {
          flag(p.status, MLA_DEVSTAT_BAD_INDEX);
          blk[i] = -1;
        }
        const int r = owner(s.need, p.batch, (int)k);
        p.block_table[(int64_t)r * p.max_blocks + s.held[r] + (k - s.need[r])] = blk[i];
      } else if (at < p.free_capacity) {
        if (blk[i] < 0) flag(p.status, MLA_DEVSTAT_BAD_INDEX);   // (where it came from: now, not when it is taken)
        p.free_blocks[at] = blk[i];
      } else {
        flag(p.status, MLA_DEVSTAT_BAD_INDEX);   // the stack is full
      }
    }
  }
}

__device__ __forceinline__ void write_lengths(const TablesParams& p, const Shared& s, int first, int step) {
  for (int r = first; r <= p.batch; r += step) {
    if (p.qo_indptr) p.qo_indptr[r] = s.tok[r];
    if (r < p.batch) {
      p.num_held[r] = s.after[r];
      if (p.kv_lens) {
        const int64_t len = (int64_t)max(p.seq_lens[r], 0) + max(p.new_lens[r], 0);
        p.kv_lens[r] = (int)min(len, (int64_t)INT_MAX);
      }
    }
  }
  if (first == 0) p.free_count[0] = (int)min(s.top - s.taken, (int64_t)p.free_capacity);
}

// Slots of tokens t .. t + n - 1.
__device__ __forceinline__ void write_slots(const TablesParams& p, const int* tok, int64_t t, int n) {
  const int live = tok[p.batch];
  int r = t < live ? owner(tok, p.batch, (int)t) : p.batch;
  int64_t seen = -1, base = -1;   // block index last looked up, its first slot
  for (int i = 0; i < n; ++i, ++t) {
    if (t >= p.num_tokens) return;
    int64_t slot = -1;
    if (t < live) {
      while (t >= tok[r + 1]) {   // (ends: t < tok[batch])
        ++r;
        seen = -1;
      }
      const int64_t pos = (int64_t)max(p.seq_lens[r], 0) + (t - tok[r]);
      const int64_t bi = pos / p.block_size;
      if (bi != seen) {
        seen = bi;
        const int blk = bi < p.max_blocks ? p.block_table[(int64_t)r * p.max_blocks + bi] : -1;
        base = blk >= 0 ? (int64_t)blk * p.block_size : -1;
      }
      if (base >= 0) slot = base + (pos - bi * p.block_size);
    }
    p.slot_mapping[t] = slot;
  }
}

__global__ void __launch_bounds__(kMaxThreads) tables_kernel(const TablesParams p) {
  extern __shared__ int smem[];
  Shared s;
  make_sums(p, smem, true, &s);
  move_blocks(p, s, threadIdx.x, blockDim.x);
  if (s.refused) clear_refused(p, s, threadIdx.x, blockDim.x);
  write_lengths(p, s, threadIdx.x, blockDim.x);
  if (!p.slot_mapping) return;
  __syncthreads();
  for (int64_t t = threadIdx.x; t < p.num_tokens; t += blockDim.x) write_slots(p, s.tok, t, 1);
}

// The old lengths stay until the second kernel: every CTA reads them.
__global__ void __launch_bounds__(kMaxThreads) tables_blocks_kernel(const TablesParams p) {
  extern __shared__ int smem[];
  grid_launch_dependents();
  Shared s;
  make_sums(p, smem, blockIdx.x == 0, &s);
  move_blocks(p, s, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x);
  if (s.refused) clear_refused(p, s, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x);
}

// CTA 0 alone reads and writes what a request holds; the others only sum the new tokens.  The sums are
// made while the first kernel moves the blocks (it changes nothing that they are made of), then its end is
// waited for.
__global__ void __launch_bounds__(kSlotThreads) tables_slots_kernel(const TablesParams p) {
  extern __shared__ int smem[];
  if (blockIdx.x == 0) {
    Shared s;
    make_sums(p, smem, false, &s);
    grid_dependency_wait();
    write_lengths(p, s, threadIdx.x, kSlotThreads);
  } else {
    __shared__ int64_t warp_sum[kSlotThreads / 32];
    const int b = p.batch, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (b + kSlotThreads - 1) / kSlotThreads;
    const int r0 = min(tid * per, b), r1 = min(r0 + per, b);
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r) {
      const int m = max(p.new_lens[r], 0);
      smem[r] = m;
      mine += m;
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t run = incl - mine, total = 0;
    for (int w = 0; w < kSlotThreads / 32; ++w) {
      if (w < warp) run += warp_sum[w];
      total += warp_sum[w];
    }
    for (int r = r0; r < r1; ++r) {
      const int m = smem[r];
      smem[r] = (int)min(run, (int64_t)INT_MAX);
      run += m;
    }
    if (tid == 0) smem[b] = (int)min(total, (int64_t)INT_MAX);
    __syncthreads();
    grid_dependency_wait();
  }
  // (Neighbouring threads have neighbouring tokens, a thread every kSlotThreads-th.)
  const int64_t t0 = (int64_t)blockIdx.x * kSlotThreads * kSlotsPerThread + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kSlotsPerThread; ++i) write_slots(p, smem, t0 + i * kSlotThreads, 1);
}

int sums_bytes(int batch) { return 5 * (batch + 1) * (int)sizeof(int); }

}  // namespace

cudaError_t launch_tables(const TablesParams& p, cudaStream_t stream) {
  const int smem = sums_bytes(p.batch);
  static PerDeviceOnce configured;
  cudaError_t e = configured.run([] {
    const int most = sums_bytes(kMaxTableBatch);
    const void* kernels[3] = {(const void*)tables_kernel, (const void*)tables_blocks_kernel,
                              (const void*)tables_slots_kernel};
    for (const void* k : kernels) {
      const cudaError_t r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (r != cudaSuccess) return r;
    }
    return cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  if (p.num_tokens <= kOneCtaTokens) {
    // A small CTA starts a microsecond sooner; with room for many blocks many may have to move (8320
    // given back: 62 us with 128 threads).
    const int64_t room = (int64_t)p.batch * p.max_blocks;
    const int threads = room <= 1024 && p.num_tokens <= 512 && p.batch <= 128 ? 128 : kMaxThreads;
    tables_kernel<<<1, threads, smem, stream>>>(p);
    return cudaGetLastError();
  }
  tables_blocks_kernel<<<8, kMaxThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t per_cta = (int64_t)kSlotThreads * kSlotsPerThread;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.num_tokens + per_cta - 1) / per_cta));
  cfg.blockDim = dim3(kSlotThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tables_slots_kernel, p);
}

}  // namespace mla
