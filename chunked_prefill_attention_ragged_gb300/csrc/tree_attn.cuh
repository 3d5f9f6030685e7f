// What the kernels of tree attention share: the requests as they see them, the split of the
// work among workers, the way from key positions to cache rows, visibility, and waits.
#pragma once
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace mla {

// (node, head) pairs per unit and keys per tile, unless a kernel says otherwise (the ROWS and KEYS below).
constexpr int TREE_ROWS = 128;
constexpr int TREE_KEYS = 128;

struct TreeLaunch {
  TreeParams t;
  int workers;         // clusters of two CTAs, or CTAs
  int32_t oob_row;     // a row coordinate past the cache: the copy fills it with zeros
  int block_shift;     // log2 of the block size, or -1
  int o_align32;
  int has_cap;
  float scale_log2, cap_log2, cap_inv;
  uint64_t wait_limit_ns;
  int force_timeout;
};

// What both kernels' launches have in common.
inline TreeLaunch tree_launch(const TreeParams& t, int workers) {
  TreeLaunch p = {};
  p.t = t;
  p.workers = workers;
  const int bs = t.block_size;
  p.oob_row = (int32_t)(t.max_blocks > 0 ? (uint64_t)t.num_blocks * (uint64_t)bs : 1);
  p.block_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (bs == 1 << i) p.block_shift = i;
  p.o_align32 = (reinterpret_cast<uintptr_t>(t.o) & 31u) == 0;
  const float LOG2E = 1.4426950408889634f;
  p.has_cap = t.soft_cap > 0.f;
  p.scale_log2 = t.sm_scale * LOG2E;
  p.cap_log2 = p.has_cap ? t.soft_cap * LOG2E : 0.f;
  p.cap_inv = p.has_cap ? std::fmin(t.sm_scale / t.soft_cap, 1e38f) : 0.f;
  const uint64_t forced = forced_timeout_ns();
  p.force_timeout = forced != 0;
  p.wait_limit_ns = forced ? forced : kWaitLimitNs;
  return p;
}

// Workspace: one record per worker, two slots per worker.
// The unit that the boundary before a worker cuts, if it is the unit's first such boundary: parts
// k = 0 .. parts - 1 belong to workers w - 1 + k, each that worker's first part (slot 0) except that
// part 0 may be a later one (slot0).
struct JoinRec {
  int64_t pair0;       // first pair of the unit
  int npairs;
  int parts;           // 0: nothing to join here
  int slot0, pad[3];
};
constexpr int MAX_WORKERS = 256;
constexpr size_t WS_SLOTS = MAX_WORKERS * sizeof(JoinRec);
// A slot: O (fp32) as 64 groups of eight columns, each [128 rows][8], so that a warp, whose threads
// have a row each, writes and reads 1 KB at a time; then the rows' (m in log2 units, l).
__device__ __forceinline__ size_t slot_at(int row, int col) { return ((size_t)(col >> 3) * TREE_ROWS + row) * 32; }
constexpr size_t SLOT_ML = (size_t)TREE_ROWS * 512 * 4;
constexpr size_t SLOT_BYTES = SLOT_ML + TREE_ROWS * 2 * 4;

// One lane's look at a barrier, whose result can be used later; for wait_warp's `seen`.
__device__ __forceinline__ uint32_t look_warp(uint32_t bar, uint32_t parity) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, 0, 0;\n\t"
      "@e mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r)
      : "r"(bar), "r"(parity)
      : "memory");
  return r;
}

// A bounded wait of a converged warp, polled by one lane: 32 lanes polling, in five warps that
// wait most of the time, slow the softmax's exponentials down (they share the queue to the
// special function units and shared memory).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          uint64_t limit_ns, uint32_t seen = 0) {
  if (__any_sync(0xffffffffu, seen != 0)) {
    __syncwarp();
    return true;
  }
  auto poll = [&]() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, 0, 0;\n\t"
        "@e mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r)
        : "r"(bar), "r"(parity)
        : "memory");
    return __any_sync(0xffffffffu, r != 0) != 0;
  };
  bool ok = poll();
  if (!ok) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
      ok = poll();
      if (ok) break;
      if ((it & 63) == 0) {
        const bool late = global_timer_ns() - t0 > limit_ns;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
          if (late) {
            *abort_flag = 1;
            if (status) atomicOr(status, MLA_DEVSTAT_TIMEOUT);
          }
          break;
        }
      }
    }
  }
  __syncwarp();   // what the polling lane acquired, all lanes see
  return ok;
}

// A barrier of `THREADS` threads, and whether any of them says yes.  Warps that wait for the same thing leave the
// looking to one of them and meet it here: sixteen warps that look all the time take a third of the issue slots.
template <int THREADS>
__device__ __forceinline__ bool meet(int id, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)yes), "r"(id), "n"(THREADS)
      : "memory");
  return r != 0;
}

// One request as the kernel sees it.
struct Req {
  int q0, nodes;       // rows; 0 nodes when the request is empty or refused
  int64_t ctx;         // positions every node sees (negative: the first nodes are not cached)
  int kv;              // positions that may be read
  int units, tiles;
};

struct ReqWords {
  int q0, q1, len;
};
__device__ __forceinline__ ReqWords load_words(const TreeParams& p, int r) {
  return {__ldg(p.qo_indptr + r), __ldg(p.qo_indptr + r + 1), __ldg(p.kv_lens + r)};
}
template <int ROWS = TREE_ROWS, int KEYS = TREE_KEYS>
__device__ __forceinline__ Req make_req(const TreeParams& p, const ReqWords& w, bool report) {
  Req q;
  const int64_t reach = (int64_t)p.max_blocks * p.block_size;
  const bool rows_ok = w.q0 >= 0 && w.q1 >= w.q0 && w.q1 <= p.total_rows;
  const bool len_ok = w.len >= 0 && w.len <= reach;
  if (report && p.status && (!rows_ok || !len_ok)) atomicOr(p.status, MLA_DEVSTAT_BAD_INDEX);
  q.q0 = w.q0;
  q.nodes = rows_ok ? w.q1 - w.q0 : 0;
  q.ctx = (int64_t)w.len - q.nodes;
  q.kv = len_ok ? w.len : (w.len < 0 ? 0 : (int)reach);
  q.units = (int)(((int64_t)q.nodes * p.num_heads + ROWS - 1) / ROWS);
  q.tiles = q.units ? max(1, (int)(((int64_t)q.kv + KEYS - 1) / KEYS)) : 0;
  return q;
}
template <int ROWS = TREE_ROWS, int KEYS = TREE_KEYS>
__device__ __forceinline__ Req load_req(const TreeParams& p, int r, bool report) {
  return make_req<ROWS, KEYS>(p, load_words(p, r), report);
}

// Where a worker's piece starts.
struct StartRec {
  int req, unit, tile;
  Req q;
};

// A part of a worker's piece: tiles [lo, hi) of one unit.
struct Part {
  Req q;
  int r;
  int64_t pair0;       // first pair of the unit, counted over the batch
  int npairs;
  int lo, hi;
  bool whole;          // the unit's every tile
  int slot;            // 0: the worker's first part, 1: a later one (its last, if not whole)
};

template <int ROWS, int KEYS>
struct PartsOf {
  const TreeParams& p;
  int64_t left;
  int r, unit, tile, index;
  Req q;
  __device__ PartsOf(const TreeParams& tp, const StartRec& s, int64_t count)
      : p(tp), left(count), r(s.req), unit(s.unit), tile(s.tile), index(0), q(s.q) {}
  __device__ bool next(Part* out) {
    if (left <= 0) return false;
    while (unit >= q.units) {   // to the next request that has rows
      if (++r >= p.batch) return false;   // (lengths changed under the kernel: out of bounds is not read)
      unit = 0;
      q = load_req<ROWS, KEYS>(p, r, false);
    }
    const int n = (int)min((int64_t)(q.tiles - tile), left);
    out->q = q;
    out->r = r;
    const int64_t first = (int64_t)unit * ROWS;
    out->pair0 = (int64_t)q.q0 * p.num_heads + first;
    out->npairs = (int)min((int64_t)ROWS, (int64_t)q.nodes * p.num_heads - first);
    out->lo = tile;
    out->hi = tile + n;
    out->whole = n == q.tiles;
    out->slot = index == 0 ? 0 : 1;
    ++index;
    left -= n;
    tile = 0;
    ++unit;
    return true;
  }
};
using Parts = PartsOf<TREE_ROWS, TREE_KEYS>;

// From key positions to cache rows: first the block as the table has it (its load is under way while
// the caller does other things), then the row to copy.  A key past the readable ones, or in a block
// that the table does not name, is the row past the cache (read as zeros), the latter flagged; of a box
// in which the readable keys end, what lies behind them comes along.
constexpr int32_t PAST_END = -0x7fffffff - 1;
__device__ __forceinline__ int block_of(const TreeLaunch& p, int key) {
  return p.block_shift >= 0 ? key >> p.block_shift : key / p.t.block_size;
}
__device__ __forceinline__ int32_t table_block(const TreeLaunch& p, const Part& u, int64_t key) {
  if (key >= u.q.kv) return PAST_END;
  const int32_t blk = __ldg(p.t.block_table + (int64_t)u.r * p.t.max_blocks + block_of(p, (int)key));
  return blk == PAST_END ? -1 : blk;   // (so named in the table, it is a bad id like any other)
}
__device__ __forceinline__ int32_t block_row(const TreeLaunch& p, int32_t blk, int64_t key) {
  if (blk < 0 || (int64_t)blk >= p.t.num_blocks) {
    if (blk != PAST_END && p.t.status) atomicOr(p.t.status, MLA_DEVSTAT_BAD_INDEX);
    return p.oob_row;
  }
  return (int32_t)((int64_t)blk * p.t.block_size + ((int)key - block_of(p, (int)key) * p.t.block_size));
}
// 64 keys from key0 on by boxes of `step` keys, lane k with box k.
__device__ __forceinline__ int32_t box_block(const TreeLaunch& p, const Part& u, int64_t key0, int step, int lane) {
  return lane * step < 64 ? table_block(p, u, key0 + lane * step) : PAST_END;
}
// And row by row, a lane keys lane and 32 + lane.
struct KeyBlocks {
  int32_t b[2];
};
struct KeyRows {
  int32_t r[2];
};
__device__ __forceinline__ KeyBlocks find_blocks(const TreeLaunch& p, const Part& u, int64_t key0, int lane) {
  return {{table_block(p, u, key0 + lane), table_block(p, u, key0 + 32 + lane)}};
}
__device__ __forceinline__ KeyRows find_rows(const TreeLaunch& p, const KeyBlocks& k, int64_t key0, int lane) {
  return {{block_row(p, k.b[0], key0 + lane), block_row(p, k.b[1], key0 + 32 + lane)}};
}

// Visibility of 64 keys from position pos0 on for node i (row t of the batch), bit k for key k.
__device__ __forceinline__ uint64_t visible(const TreeParams& p, const Part& u, int i, int64_t pos0) {
  auto window = [&](int64_t j0) -> uint64_t {   // nodes j0 .. j0 + 63, j0 >= 0
    if (!p.mask) {
      const int64_t n = (int64_t)i - j0 + 1;
      return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
    }
    const int64_t* row = p.mask + ((int64_t)u.q.q0 + i) * p.mask_words;
    const int64_t w = j0 >> 6;
    const int sh = (int)(j0 & 63);
    uint64_t bits = w < p.mask_words ? (uint64_t)__ldg(row + w) >> sh : 0ull;
    if (sh && w + 1 < p.mask_words) bits |= (uint64_t)__ldg(row + w + 1) << (64 - sh);
    return bits;
  };
  const int64_t s = pos0 - u.q.ctx;   // node index of the first key
  uint64_t v;
  if (s <= -64) v = ~0ull;
  else if (s >= 0) v = window(s);
  else v = ((1ull << -s) - 1) | (window(0) << -s);
  const int64_t room = u.q.kv - pos0;
  if (room < 64) v &= room <= 0 ? 0ull : (1ull << room) - 1;
  return v;
}

// Quotients whose terms nearly always have 32 bits: the long division is a call of its own.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {   // 0 <= a, 0 < b
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Where worker w's piece starts and how long it is, and what is to be joined at its start; every
// thread of the CTA calls, with the words of request threadIdx.x, loaded before.
template <int NTHREADS, int ROWS = TREE_ROWS, int KEYS = TREE_KEYS>
__device__ __forceinline__ void find_piece(const TreeParams& p, const ReqWords& own, int worker, int workers,
                                           bool report, StartRec* start, int64_t* count, JoinRec* join) {
  __shared__ int64_t warp_sum[NTHREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.batch + NTHREADS - 1) / NTHREADS;
  const int r0 = min(tid * per, p.batch), r1 = min(r0 + per, p.batch);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) {
    const Req q = per == 1 ? make_req<ROWS, KEYS>(p, own, report) : load_req<ROWS, KEYS>(p, r, report);
    mine += (int64_t)q.units * q.tiles;
  }
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
  for (int w = 0; w < NTHREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const int n = (int)min((int64_t)workers, total);   // a tile is worth a worker
  // The first `more` workers have a tile more than the others.
  const int64_t each = n > 0 ? quotient(total, n) : 0, more = total - each * n;
  auto at = [&](int w) { return each * w + min((int64_t)w, more); };
  const int64_t lo = worker < n ? at(worker) : total, hi = worker < n ? at(worker + 1) : total;
  if (tid == 0) *count = hi - lo;
  if (tid == 0 && lo >= hi) *join = JoinRec{0, 0, 0, 0, {}};
  if (lo < hi && lo >= before && lo < before + mine) {
    int64_t sum = before;
    for (int r = r0; r < r1; ++r) {
      const Req q = per == 1 ? make_req<ROWS, KEYS>(p, own, false) : load_req<ROWS, KEYS>(p, r, false);
      const int64_t k = (int64_t)q.units * q.tiles;
      if (lo < sum + k) {
        const int unit = (int)quotient(lo - sum, q.tiles), tile = (int)(lo - sum - (int64_t)unit * q.tiles);
        *start = StartRec{r, unit, tile, q};
        JoinRec j{0, 0, 0, 0, {}};
        const int64_t first = lo - tile, prev = worker > 0 ? at(worker - 1) : 0;   // the unit's first tile
        if (tile > 0 && prev <= first) {
          // The last worker with a part is the one that has the unit's last tile.
          const int64_t end = first + q.tiles - 1, big = more * (each + 1);
          const int last = (int)(end < big ? quotient(end, each + 1) : more + quotient(end - big, each));
          j.pair0 = (int64_t)q.q0 * p.num_heads + (int64_t)unit * ROWS;
          j.npairs = (int)min((int64_t)ROWS, (int64_t)q.nodes * p.num_heads - (int64_t)unit * ROWS);
          j.parts = last - worker + 2;
          j.slot0 = prev < first ? 1 : 0;
        }
        *join = j;
        break;
      }
      sum += k;
    }
  }
  __syncthreads();
}

// For block sizes that are multiples of 64: lane i's row of the 64 keys from key0 + i * stride on,
// i < n, to be copied as one box.  Where only the first of them are readable the others come along
// (they lie in the same block) and have to be kept from counting; where none is, the box lies past
// the cache and is filled with zeros.  One look-up for 32 tiles: what a producer warp does between
// two copies has to be short (its code is not in the instruction cache when it comes back to it,
// and costs about 400 clocks for every 60 instructions).
__device__ __forceinline__ int32_t piece_rows(const TreeLaunch& p, const Part& u, int64_t key0, int stride, int n,
                                              int lane) {
  const int64_t key = key0 + (int64_t)lane * stride;
  return lane < n && key < u.q.kv ? block_row(p, table_block(p, u, key), key) : p.oob_row;
}

// tree_join_kernel.cu: joins the parts of units that several workers left.
cudaError_t launch_tree_join(const TreeLaunch& p, cudaStream_t stream);
// The same for units of few pairs: a slot is O (fp32) row by row, then the rows' (m in log2 units, l).
constexpr int TREE_FEW = 16;   // pairs of such a unit
constexpr size_t FEW_SLOT_ML = (size_t)TREE_FEW * 512 * 4, FEW_SLOT_BYTES = FEW_SLOT_ML + TREE_FEW * 8;
cudaError_t launch_tree_join_few(const TreeLaunch& p, cudaStream_t stream);

constexpr uint64_t TREE_DRAIN_LIMIT_NS = 200000000ull;   // own copies and products after an abort
constexpr float TREE_RESCALE_THRESHOLD = 8.0f;           // log2 units

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace mla
