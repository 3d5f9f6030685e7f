// Tree attention over the paged latent cache, absorbed-weight form, with every length on the
// device: O_lat = softmax(sm_scale * q_abs . c^T) c[:, :512] and the per-row LSE, where row
// (node i, head h) of a request with n nodes and kv cached positions sees the positions below
// kv - n and those of the nodes that its mask bits name.
//
// Mathematics.  A unit is 128 consecutive (node, head) pairs of one request.  Over tiles of 128
// keys, with scores s in log2 units and a reference m per pair that follows the running maximum,
//   P = 2^(s - m),  l += sum P,  O += P V;  when a maximum passes m + 8: O, l *= 2^(m - m').
// A unit's tiles may be shared out to several workers; each leaves (O, m, l) in fp32 and the
// second kernel joins them: with M = max m, O = sum 2^(m - M) O / sum 2^(m - M) l.
//
// Work split.  The tiles of all units, request by request, form one line that is cut into equal
// pieces, one per worker (a cluster of two CTAs on two SMs).  The lengths are on the device, so
// every worker finds its piece itself: a prefix sum over the requests.  A piece has at most two
// parts that do not cover their unit (its first and its last), so the workspace has two slots
// per worker.
//
// A cluster runs a unit with tcgen05 cta_group::2 products of M = 128, 64 pairs in each CTA: a
// 64 x 512 fp32 accumulator then takes 256 TMEM columns (both lane halves are in use: lanes
// 0-63 hold the first half of a product's columns for the 64 rows, lanes 64-127 the second),
// which leaves room for two S buffers.  A single CTA with 128 rows has no room for S beside O and
// would compute S once per half of the values.  Per CTA in shared memory: its Q rows (64 x 576),
// its 64 of the tile's 128 keys as the half of S's B operand, the tile's 128 keys x 256 of the value
// columns as the half of P V's B operand (two products of 128 columns of each CTA), and P (64 x 128).
//   warp 0     Q and K producer: Q once per unit; K in three groups of three 64-column panels
//   warp 1     even CTA: issues every product
//   warp 2     V producer: the CTA's columns, by halves of the keys
//   warp 3     TMEM allocation; brings the next tile's rows into L2, or, where rows are copied
//              one by one, loads K's last group
//   warps 4-7  softmax: two threads per pair (the two halves of the keys and of O's columns)
// Order of products: S(t + 1) before P V(t), so that the tensor cores work on the next tile while
// the softmax does this one.  Key rows come by whole boxes of 64 where the block size is a multiple
// of that, by boxes of 32, 16 or 8 where it is one of these (in the piece where the keys end, what lies
// behind them is made zero), else row by row by the producers' own lanes.  The kernel is compiled for
// each: with strides of the operands read from registers the products' issue took 3% longer.
// What bounds it: for one node a request HBM (64 requests over 4096 positions, 16 heads: 66 us with the
// join, a copy's rate while tiles run; 8 us pass before the first scores are there); for many the products
// and what feeds them (32 x 16 nodes over 8192, 128 heads: 772-815 us in replayed graphs, 0.77-0.81 of the
// measured tensor rate, and 900-930 in calls back to back, when the power cap lowers the clock: 0.74-0.76 of
// the rate that then holds.  A tile is 2176 clocks of products, 392 KB through shared memory and 272 KB from
// L2, and takes 2700-2950).  Calls of few tiles cost 14 us: 2.3 to the first copy, a tile, the state and the
// join.
//
// Roundings: scores, maxima, sums, O and the parts are fp32.  P is rounded to bf16, as products with bf16 values
// have to have it: each weight is off by up to 2^-8 of itself, O by up to 2^-8 sum P |V| / l, in practice
// less than its own rounding to bf16 adds (both: 0.0017 to 0.0020 of O's norm, O's alone 0.0017).  The sum l, and with it the LSE, is
// of the unrounded weights.
// Every wait is bounded: on time-out the CTA records MLA_DEVSTAT_TIMEOUT, drains its copies and
// products, frees TMEM and returns.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "tmem_wide.cuh"
#include "tree_attn.cuh"
#include "tree_issue.cuh"

namespace mla {
namespace {

constexpr int ROWS = TREE_ROWS, KEYS = TREE_KEYS;   // 64 rows in each CTA
constexpr int QP = 64 * 128;            // a [64 rows, 64 columns] panel: 8 KB
constexpr int NP = 9;                   // 64-column panels of 576
constexpr int KGROUPS = 3;              // K panels arrive in groups of three,
constexpr int K_ROWS8 = 3 * 8 * 128;    // by small boxes eight rows at a time: [panel][8 rows] of each
constexpr int V_HALF = 4 * QP;          // 64 keys x the CTA's 256 value columns
constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + NP * QP;
constexpr int OFF_V = OFF_K + NP * QP;
constexpr int OFF_P = OFF_V + 2 * V_HALF;
constexpr int OFF_XCHG = OFF_P + 2 * QP;            // [2 tiles][2 halves][64 rows] maxima
constexpr int OFF_BAR = OFF_XCHG + 2 * 2 * 64 * 4;
enum Bar {
  QF = 0,              // Q landed
  QE,                  // the unit's last S done: Q may be replaced
  KF,                  // [group] K panels landed
  KE = KF + KGROUPS,   // [group] their products done
  VF = KE + KGROUPS,   // [key half] V landed
  VE = VF + 2,         // [key half] its products done
  SF = VE + 2,         // [buffer] S done
  PR = SF + 2,         // P written (and the S buffer read) by every softmax warp of both CTAs
  OD,                  // P V done
  LB,                  // [key half] V to be mended landed (in this CTA)
  ZB = LB + 2,         // [key half] the odd CTA has mended its own
  XB = ZB + 2,         // [row half] maxima exchanged between the two warps of 32 rows
  FIN = XB + 2,        // every product drained
  NEVER,               // nothing arrives here: the time-out test mode waits on it
  NBAR
};
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int SMEM = OFF_MISC + 64 + 1024;   // + slack for 1024-byte alignment
static_assert(SMEM <= 227 * 1024, "shared memory budget");
constexpr int NTHREADS = 256;
constexpr uint32_t TMEM_COLS = 512;
__device__ __forceinline__ constexpr uint32_t TM_O(int chunk) { return (uint32_t)chunk * 128u; }
__device__ __forceinline__ constexpr uint32_t TM_S(int b) { return 256u + (uint32_t)b * 64u; }
constexpr uint32_t IDESC_QK = idesc_bf16_f32(ROWS, KEYS, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16_f32(ROWS, 256, false, true);

struct Ctx {
  uint32_t sbase;
  volatile int* abort_flag;
  int* status;
  uint64_t wait_limit_ns;
  uint32_t rank;
  __device__ uint32_t bar(int i) const { return sbase + OFF_BAR + 8 * i; }
  __device__ bool wait(int b, uint32_t parity) const {
    return mbar_wait_bounded(bar(b), parity, abort_flag, status, MLA_DEVSTAT_TIMEOUT, wait_limit_ns);
  }
  __device__ uint32_t look(int b, uint32_t parity) const { return look_warp(bar(b), parity); }
  __device__ bool wait_warp(int b, uint32_t parity, uint32_t seen = 0) const {
    return mla::wait_warp(bar(b), parity, abort_flag, status, wait_limit_ns, seen);
  }
  __device__ void drain(int b, uint32_t parity) const {
    int dummy = 0;
    mbar_wait_bounded(bar(b), parity, &dummy, status, MLA_DEVSTAT_TIMEOUT, TREE_DRAIN_LIMIT_NS, true);
  }
};

// Where the block size is no multiple of 8: 64 keys' rows, PANELS panels from panel0 on, to consecutive
// 8 KB panels at dst (in the swizzle that a box would have), 16 bytes a thread: eight lanes a row.  Rows
// that are not there are zeros.
template <int PANELS>
__device__ __forceinline__ void copy_rows(const TreeLaunch& p, const KeyRows& k, uint32_t dst, int panel0, int lane) {
  const int ch = lane & 7;
  const __nv_bfloat16* cache = (p.t.cache ? p.t.cache : p.t.q) + panel0 * 64 + ch * 8;
#pragma unroll 2
  for (int j = 0; j < 16; ++j) {
    const int key = 4 * j + (lane >> 3);
    const int32_t row = __shfl_sync(0xffffffffu, j < 8 ? k.r[0] : k.r[1], key & 31);
    const bool there = row != p.oob_row;
    const __nv_bfloat16* src = cache + (there ? (int64_t)row * 576 : 0);
    const uint32_t d = dst + key * 128 + ((ch ^ (key & 7)) << 4);
#pragma unroll
    for (int i = 0; i < PANELS; ++i) cp_async16(d + i * QP, src + i * 64, there ? 16 : 0);
  }
}

// ------------------------------------------------------------------ producers
// The copies of both CTAs complete on the even CTA's barriers, where the products wait for them;
// its producers announce the bytes of both.  The buffers hold one tile: what a product has read
// is loaded again at once, so the way from "read" to the copy is kept short (rows looked up a
// tile ahead, one lane).
__device__ __forceinline__ void expect_both(const Ctx& c, int b, uint32_t bytes_each) {
  if (c.rank == 0) mbar_arrive_expect_tx(c.bar(b), 2 * bytes_each);
}
// After an abort the odd CTA cannot see its copies land: they have this long.
__device__ __forceinline__ void settle() {
  const uint64_t t0 = global_timer_ns();
  while (global_timer_ns() - t0 < TREE_DRAIN_LIMIT_NS) {
  }
}

template <int R>
__device__ void run_producer_qk(const Ctx& c, const TreeLaunch& p, Parts parts, const CUtensorMap* tq,
                                const CUtensorMap* tk, volatile int* begun) {
  const int lane = threadIdx.x & 31;
  const uint32_t qf = mapa_shared(c.bar(QF), 0), kf = mapa_shared(c.bar(KF), 0);
  int tiles = 0, units = 0, issued = 0;   // tiles begun, parts, K groups
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    int32_t block = 0;
    if (R != 64) block = box_block(p, u, (int64_t)u.lo * KEYS + 64 * c.rank, 8, lane);
    if (lane == 0) {
      if (units > 0) ok = c.wait(QE, (units - 1) & 1);
      if (ok) {
        expect_both(c, QF, NP * QP);
        tma_load_3d_pair(c.sbase + OFF_Q, tq, qf, 0, (int32_t)(u.pair0 + 64 * c.rank), 0);
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok) break;
    ++units;
    int32_t ahead = 0;   // rows of 32 tiles
#pragma unroll 1
    for (int t = u.lo; t < u.hi && ok; ++t, ++tiles) {
      const int i = (t - u.lo) & 31;
      const int64_t key0 = (int64_t)t * KEYS + 64 * c.rank;
      if (i == 0 && R == 64) ahead = piece_rows(p, u, key0, KEYS, u.hi - t, lane);
      const int32_t row = __shfl_sync(0xffffffffu, ahead, i);
      if (lane == 0) *begun = tiles;
      if (R == 64) {   // one lane, three copies
        if (lane == 0) {
#pragma unroll 1
          for (int g = 0; g < KGROUPS; ++g) {
            if (tiles > 0) ok = c.wait(KE + g, (tiles - 1) & 1);
            if (!ok) break;
            expect_both(c, KF + g, 3 * QP);
            tma_load_3d_pair(c.sbase + OFF_K + 3 * g * QP, tk, kf + 8 * g, 0, row, 3 * g);
            ++issued;
          }
        }
      } else {
        const int32_t box = block_row(p, block, key0 + 8 * lane);
        if (t + 1 < u.hi) block = box_block(p, u, key0 + KEYS, 8, lane);
#pragma unroll 1
        for (int g = 0; g < KGROUPS; ++g) {
          if (lane == 0) {
            if (tiles > 0) ok = c.wait(KE + g, (tiles - 1) & 1);
            if (ok) expect_both(c, KF + g, 3 * QP);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (lane < 8) tma_load_3d_pair(c.sbase + OFF_K + 3 * g * QP + lane * K_ROWS8, tk, kf + 8 * g, 0, box, 3 * g);
          ++issued;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
  }
  // Let every copy started here land before the CTA can exit.
  if (lane == 0) {
    if (c.rank == 0) {
      if (units) c.drain(QF, (units - 1) & 1);
      for (int g = 0; g < KGROUPS; ++g) {
        const int n = (issued + KGROUPS - 1 - g) / KGROUPS;
        if (n) c.drain(KF + g, (n - 1) & 1);
      }
    } else if (!ok) {
      settle();
    }
  }
}


// From which key on there are nodes that some row of the unit may not see (kv: none; a single new token sees
// itself).
__device__ __forceinline__ int64_t first_unseen(const TreeLaunch& p, const Part& u) {
  return u.q.nodes < 2 && !p.t.mask ? u.q.kv : min(max(u.q.ctx, (int64_t)0), (int64_t)u.q.kv);
}

// A weight of 0 times a NaN or an infinity is NaN, and products take every row of the tile: in rows [from, to) of
// 64 of V, those of nodes, a NaN becomes 0 (whoever sees it has a NaN score, the row being its key too) and an
// infinity the largest finite value.  Rows lie in pieces of `low` + 1, each with its four panels; a lane has 16
// bytes of a row.  The rows are looked through by their largest magnitude, a NaN above all, and only gone over
// again if that is not finite.  (Not inline, to keep the producer's loop short.  A row at a time with a branch in
// it took 9 x up to 37 nodes from 40.9 to 43.8 us, this way 41.5; calls of single tokens do not come here.)
__device__ __noinline__ void mend_nodes(uint32_t at, int from, int to, int low) {
  const int lane = threadIdx.x & 31;
  const uint32_t base = at + (lane >> 3) * (low + 1) * 128 + (lane & 7) * 16;
  auto addr = [&](int row) { return base + (4 * (row & ~low) + (row & low)) * 128; };
  auto load = [&](int row, uint32_t* v) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr(row)) : "memory");
  };
  auto most = [](uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  };
  auto odd = [](uint32_t w) { return (((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0; };   // an exponent of all ones
  uint32_t top[4] = {0u, 0u, 0u, 0u};
  for (int row = from; row < to; row += 4) {
    uint32_t v[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) load(min(row + k, to - 1), v[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int w = 0; w < 4; ++w) top[w] = most(top[w], v[k][w]);
  }
  if (!(odd(top[0]) || odd(top[1]) || odd(top[2]) || odd(top[3]))) return;
  auto half = [](uint32_t h) { return (h & 0x7fffu) > 0x7f80u ? 0u : (h & 0x7fffu) == 0x7f80u ? h - 1 : h; };
  for (int row = from; row < to; ++row) {
    uint32_t v[4];
    load(row, v);
#pragma unroll
    for (int w = 0; w < 4; ++w) v[w] = half(v[w] & 0xffffu) | half(v[w] >> 16) << 16;
    st_shared_v4(addr(row), v[0], v[1], v[2], v[3]);
  }
}

// Where the block size is no multiple of 8, K (groups first .. first + n - 1, and Q beside group 0) or V
// (n = 2 halves) row by row: the lanes' own copies, handed to the even CTA's barriers when they have
// landed.  Bound by the threads' path from L2, 30 bytes a clock and SM: 16 requests of 4 nodes, 128 heads,
// over 4096 take 168 us with blocks of 1 or 4, 203 by gather4 (four rows of a panel a copy), 69 by boxes
// of 64.
template <bool V>
__device__ void run_rows(const Ctx& c, const TreeLaunch& p, Parts parts, const CUtensorMap* tq, int first, int n) {
  const int lane = threadIdx.x & 31;
  const bool with_q = !V && first == 0;
  const int full = V ? VF : KF + first, empty = V ? VE : KE + first;
  const uint32_t dst = c.sbase + (V ? OFF_V : OFF_K + 3 * first * QP);
  int tiles = 0, units = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    int64_t key0 = (int64_t)u.lo * KEYS + (V ? 0 : 64 * c.rank);
    KeyBlocks b0 = find_blocks(p, u, key0, lane), b1{};
    if (V) b1 = find_blocks(p, u, key0 + 64, lane);
    const int64_t unseen = V ? first_unseen(p, u) : 0;
    if (with_q) {
      if (lane == 0) {
        if (units > 0) ok = c.wait(QE, (units - 1) & 1);
        if (ok) {
          expect_both(c, QF, NP * QP);
          tma_load_3d_pair(c.sbase + OFF_Q, tq, mapa_shared(c.bar(QF), 0), 0, (int32_t)(u.pair0 + 64 * c.rank), 0);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      ++units;
    }
#pragma unroll 1
    for (int t = u.lo; t < u.hi && ok; ++t, ++tiles, key0 += KEYS) {
      const KeyRows k0 = find_rows(p, b0, key0, lane);
      KeyRows k1{};
      if (V) k1 = find_rows(p, b1, key0 + 64, lane);
      if (t + 1 < u.hi) {
        b0 = find_blocks(p, u, key0 + KEYS, lane);
        if (V) b1 = find_blocks(p, u, key0 + KEYS + 64, lane);
      }
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        if (lane == 0 && tiles > 0) ok = c.wait(empty + i, (tiles - 1) & 1);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        __syncwarp();   // (what lane 0 acquired, for the others' writes)
        if (V) copy_rows<4>(p, i ? k1 : k0, dst + i * V_HALF, 4 * (int)c.rank, lane);
        else copy_rows<3>(p, k0, dst + 3 * i * QP, 3 * (first + i), lane);
        cp_async_commit();
      }
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        if (i + 1 < n) cp_async_wait<1>();
        else cp_async_wait<0>();
        const int64_t a = key0 + 64 * i;
        if (V && a + 64 > unseen && max(a, unseen) < u.q.kv) {
          __syncwarp();   // (a row's pieces are other lanes' copies)
          mend_nodes(dst + i * V_HALF, (int)max(unseen - a, (int64_t)0), (int)min(u.q.kv - a, (int64_t)64), 63);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          if (c.rank) mbar_arrive_remote(mapa_shared(c.bar(full + i), 0));
          else mbar_arrive(c.bar(full + i));
        }
      }
    }
  }
  cp_async_wait<0>();
  if (lane == 0 && with_q) {
    if (c.rank == 0) {
      if (units) c.drain(QF, (units - 1) & 1);
    } else if (!ok) {
      settle();
    }
  }
}

template <int R>
__device__ void run_producer_v(const Ctx& c, const TreeLaunch& p, Parts parts, const CUtensorMap* tv, uint8_t* smem) {
  const int lane = threadIdx.x & 31, panel0 = 4 * (int)c.rank;
  const uint32_t vf = mapa_shared(c.bar(VF), 0);
  int tiles = 0, issued = 0;
  int mends[2] = {0, 0};   // halves mended so far
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    const int64_t unseen = first_unseen(p, u);
    int32_t ahead0 = 0, ahead1 = 0;   // rows of 32 tiles' first and second halves
    int32_t b0 = 0, b1 = 0;
    if (R != 64) {
      b0 = box_block(p, u, (int64_t)u.lo * KEYS, R, lane);
      b1 = box_block(p, u, (int64_t)u.lo * KEYS + 64, R, lane);
    }
#pragma unroll 1
    for (int t = u.lo; t < u.hi && ok; ++t, ++tiles) {
      const int j = (t - u.lo) & 31;
      const int64_t key0 = (int64_t)t * KEYS;
      if (j == 0 && R == 64) {
        ahead0 = piece_rows(p, u, key0, KEYS, u.hi - t, lane);
        ahead1 = piece_rows(p, u, key0 + 64, KEYS, u.hi - t, lane);
      }
      int32_t row0 = __shfl_sync(0xffffffffu, ahead0, j), row1 = __shfl_sync(0xffffffffu, ahead1, j);
      if (R == 64 && key0 + KEYS <= unseen) {   // one lane, two copies
        if (lane == 0) {
#pragma unroll 1
          for (int i = 0; i < 2; ++i) {
            if (tiles > 0) ok = c.wait(VE + i, (tiles - 1) & 1);
            if (!ok) break;
            expect_both(c, VF + i, V_HALF);
            tma_load_3d_pair(c.sbase + OFF_V + i * V_HALF, tv, vf + 8 * i, 0, i ? row1 : row0, panel0);
            ++issued;
          }
        }
      } else {
        if (R != 64) {
          row0 = block_row(p, b0, key0 + lane * R);
          row1 = block_row(p, b1, key0 + 64 + lane * R);
          if (t + 1 < u.hi) {
            b0 = box_block(p, u, key0 + KEYS, R, lane);
            b1 = box_block(p, u, key0 + KEYS + 64, R, lane);
          }
        }
        // The half in which the keys end brings along what lies behind them, one with nodes what some may not see.
        const int64_t valid = u.q.kv - key0;
        const int cut = valid <= 0 || valid >= KEYS || valid == 64 ? 2 : valid < 64 ? 0 : 1;
        auto nodes_in = [&](int i) { return unseen < u.q.kv && key0 + 64 * i + 64 > unseen && 64 * i < valid; };
        const bool dirty0 = cut == 0 || nodes_in(0), dirty1 = cut == 1 || nodes_in(1);
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const bool dirty = i ? dirty1 : dirty0;
          if (lane == 0) {
            if (tiles > 0) ok = c.wait(VE + i, (tiles - 1) & 1);
            if (ok) {
              if (dirty) mbar_arrive_expect_tx(c.bar(LB + i), V_HALF);
              else expect_both(c, VF + i, V_HALF);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          const uint32_t dst = c.sbase + OFF_V + i * V_HALF, bar = dirty ? mapa_shared(c.bar(LB + i), c.rank) : vf + 8 * i;
          if (lane * R < 64) tma_load_3d_pair(dst + lane * R * 512, tv, bar, 0, i ? row1 : row0, panel0);
          ++issued;
        }
        // What came along behind the last key, as far as products read (16 keys at a time), is made zero
        // (its P is 0, but 0 times what is there need not be), and nodes' rows finite.  Each CTA sees to its
        // own, then the even one says that the half is there.
#pragma unroll 1
        for (int i = 0; i < 2 && ok; ++i) {
          if (!(i ? dirty1 : dirty0)) continue;
          const uint32_t phase = (i ? mends[1]++ : mends[0]++) & 1;
          if (lane == 0) ok = c.wait(LB + i, phase);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          __syncwarp();   // (what lane 0 acquired, for the others' reads)
          uint8_t* at = smem + OFF_V + i * V_HALF;
          const int low = R - 1;   // (a power of two less one)
          if (i == cut) {
            for (int k = lane; k < (-(int)valid & 15) * 32; k += 32) {
              const int row = (int)(valid & 63) + (k >> 5), panel = (k >> 3) & 3;
              *reinterpret_cast<uint4*>(at + (4 * (row & ~low) + panel * (low + 1) + (row & low)) * 128 + (k & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
          }
          if (nodes_in(i))
            mend_nodes(c.sbase + OFF_V + i * V_HALF, (int)max(unseen - key0 - 64 * i, (int64_t)0),
                       (int)min(valid - 64 * i, (int64_t)64), low);
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            if (c.rank != 0) mbar_arrive_remote(mapa_shared(c.bar(ZB + i), 0));
            else if ((ok = c.wait(ZB + i, phase))) mbar_arrive(c.bar(VF + i));
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
  }
  if (lane == 0) {
    if (c.rank == 0) {
      for (int i = 0; i < 2; ++i) {
        const int n = (issued + 1 - i) / 2;
        if (n) c.drain(VF + i, (n - 1) & 1);
      }
    }
    if (!ok) settle();
  }
}

// Warp 3 where K comes by boxes: this CTA's keys of the tile after the one being loaded, into
// L2.  The one-tile buffers leave a load less than a tile's time, which DRAM does not keep to: with
// the rows in L2 it does.  It follows the K producer's count of tiles, which only grows (on a
// barrier's phases a warp that fell two tiles behind would wait for one that never comes), and gives
// up quietly.
template <int R>
__device__ void run_prefetch(const Ctx& c, const TreeLaunch& p, Parts parts, const CUtensorMap* tk,
                             const volatile int* begun) {
  const int lane = threadIdx.x & 31;
  int tiles = 0;
  Part u;
  while (parts.next(&u)) {
    for (int t = u.lo; t < u.hi; ++t, ++tiles) {
      const int64_t key = (int64_t)(t + 1) * KEYS + 64 * c.rank + (R < 64 ? 8 * lane : 0);
      const uint64_t t0 = global_timer_ns();
      while (*begun < tiles) {   // tile t is not being loaded yet
        __nanosleep(200);
        if (*c.abort_flag || global_timer_ns() - t0 > p.wait_limit_ns) return;
      }
      __syncwarp();
      if (t + 1 < u.hi && lane < (R < 64 ? 8 : 1) && key < u.q.kv) {
        const int32_t row = block_row(p, table_block(p, u, key), key);
#pragma unroll 1
        for (int g = 0; g < KGROUPS; ++g) tma_prefetch_3d(tk, 0, row, 3 * g);
      }
    }
  }
}

// ------------------------------------------------------------------ products (even CTA, warp 1)
template <int R>
__device__ void run_mma(const Ctx& c, const TreeLaunch& p, Parts parts, uint32_t tmem) {
  const uint64_t q_desc = sdesc_sw128(c.sbase + OFF_Q, 16, 1024);
  // A group of K lies in panels of 64 rows, or eight rows at a time with their three panels.
  constexpr bool rows8 = R > 0 && R < 64;
  constexpr uint32_t K_PANEL = rows8 ? 1024 : QP;
  const uint64_t k_desc = sdesc_sw128(c.sbase + OFF_K, 16, rows8 ? K_ROWS8 : 1024);
  // Values lie in pieces of r keys, each with its four panels: 16 keys of a product are part of one
  // piece, a whole one or two.
  constexpr int r = R > 0 ? R : 64;
  const uint64_t v_desc = sdesc_sw128(c.sbase + OFF_V, r * 128, r == 8 ? 4096 : 1024);
  constexpr uint32_t v_chunk = (uint32_t)(2 * r * 128) >> 4;
  const uint64_t p_desc = sdesc_sw128(c.sbase + OFF_P, 16, 1024);
  bool ok = true;
  if (p.force_timeout) ok = c.wait_warp(NEVER, 0);
  int st = 0, units = 0;   // S tiles issued
  // A look at a barrier takes about 100 clocks to come back, so each step's barrier is looked at
  // before the products of the step before it, and only waited for if it was not complete.
  // (Each look is of the very phase that the wait it stands for would wait for.)
  uint32_t seen_k = 0, seen_p = 0, seen_v = 0;   // the next S's first group, the next P V's P and V
  int pv = 0;              // P V tiles issued: S runs one tile ahead
  auto s_products = [&](bool last) {
    const int b = st & 1;
    const uint32_t d = __shfl_sync(0xffffffffu, tmem + TM_S(b), 0);
    // Loops kept small: with all 52 products of a tile unrolled the warps' code no longer fits the
    // instruction cache together, and the kernel ran 1.3 times as long.
    uint32_t seen = seen_k;
    seen_k = 0;
#pragma unroll 1
    for (int g = 0; g < KGROUPS; ++g) {
      if (!c.wait_warp(KF + g, st & 1, seen)) return false;
      tc_fence_after();
      if (g + 1 < KGROUPS) {
        seen = c.look(KF + g + 1, st & 1);
      } else {   // the P V that follows
        seen_p = c.look(PR, pv & 1);
        seen_v = c.look(VF, pv & 1);
      }
#pragma unroll 1
      for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t qo = (uint32_t)((3 * g + i) * QP + kk * 32) >> 4, ko = (uint32_t)(3 * g * QP + i * K_PANEL + kk * 32) >> 4;
          issue_pair(d, q_desc + qo, k_desc + ko, IDESC_QK, kk > 0 ? 1u : g + i > 0 ? 1u : 0u);
        }
      }
      commit_both(c.bar(KE + g));
    }
    commit_both(c.bar(SF + b));
    if (last) commit_both(c.bar(QE));
    ++st;
    return true;
  };
  // add: 0 for a part's first tile; keys: up to which of the tile's
  auto pv_products = [&](uint32_t add, int keys, bool s_next) {
    const int t = pv;
    const uint32_t more = __shfl_sync(0xffffffffu, add, 0);
    uint32_t seen = seen_v;
    if (!c.wait_warp(PR, t & 1, seen_p)) return false;
    seen_p = seen_v = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {   // halves of the keys
      if (!c.wait_warp(VF + i, t & 1, seen)) return false;
      tc_fence_after();
      if (i == 0) seen = c.look(VF + 1, t & 1);
      else if (s_next) seen_k = c.look(KF, st & 1);
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk > 0 && 64 * i + 16 * kk >= keys) break;
          const uint64_t po = (uint64_t)((i * QP + kk * 32) >> 4);
          const uint64_t vo = (uint64_t)(i * V_HALF >> 4) + ch * v_chunk + (((kk * 16 / r) * 4 * r + kk * 16 % r) * 128 >> 4);
          issue_pair(tmem + TM_O(ch), p_desc + po, v_desc + vo, IDESC_PV, kk > 0 ? 1u : i ? 1u : more);
        }
      }
      commit_both(c.bar(VE + i));
    }
    commit_both(c.bar(OD));
    ++pv;
    return true;
  };
  Part u;
  while (ok && parts.next(&u)) {
    const int n = __shfl_sync(0xffffffffu, u.hi - u.lo, 0);
    ok = c.wait_warp(QF, units & 1);
    ++units;
    for (int t = 0; t < n && ok; ++t) {
      // S's buffer held P V(pv - 2)'s scores, read before that tile's P was ready.
      ok = s_products(t == n - 1);
      if (ok && t > 0) ok = pv_products(t > 1 ? 1u : 0u, KEYS, t < n - 1);
    }
    // (The next part's Q and keys come later than this one's last P: its S first was no faster.)
    const int keys = __shfl_sync(0xffffffffu, (int)min((int64_t)KEYS, u.q.kv - (int64_t)(u.hi - 1) * KEYS), 0);
    if (ok) ok = pv_products(n > 1 ? 1u : 0u, keys, false);
  }
  commit_both(c.bar(FIN));
  c.drain(FIN, 0);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax (warps 4-7)
__device__ void run_softmax(const Ctx& c, const TreeLaunch& p, Parts parts, uint32_t tmem, char* ws_slots, uint8_t* smem) {
  const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3;
  const int half = q4 >> 1, rg = q4 & 1;             // key / column half, group of 32 rows
  const int row = 32 * rg + lane;                    // of the CTA's 64
  const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16);
  float* xchg = reinterpret_cast<float*>(smem + OFF_XCHG);
  const uint32_t p_row = c.sbase + OFF_P + half * QP + row * 128;
  const uint32_t pr_bar = c.rank ? mapa_shared(c.bar(PR), 0) : c.bar(PR);
  const float NEG_INF = -__int_as_float(0x7f800000);
  const float sc = p.has_cap ? 1.f : p.scale_log2;
  const float2 sc2 = make_float2(sc, sc);
  bool ok = true;
  int g = 0, xs = 0;   // tiles and exchanges so far
  // Swap a value with the thread that has the row's other half.  Two buffers in turn: the
  // partner read this one's last contents before it arrived for the exchange between.
  auto exchange = [&](float mine, float* theirs) {
    float* buf = xchg + (xs & 1) * 128;
    buf[half * 64 + row] = mine;
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar(XB + rg));
    if (!c.wait_warp(XB + rg, xs & 1)) return false;
    *theirs = buf[(half ^ 1) * 64 + row];
    ++xs;
    return true;
  };
  Part u;
  while (ok && parts.next(&u)) {
    const int pr0 = 64 * (int)c.rank + row;          // pair inside the unit
    const bool live = pr0 < u.npairs;
    const int64_t pair = u.pair0 + pr0;
    // A row without a pair computes on something harmless: the last node's mask.
    const int node = min((int)((pair - (int64_t)u.q.q0 * p.t.num_heads) / p.t.num_heads), u.q.nodes - 1);
    float m_used = NEG_INF, l = 0.f;
    for (int t = u.lo; t < u.hi; ++t, ++g) {
      const int sb = g & 1;
      if (!c.wait_warp(SF + sb, (g >> 1) & 1)) { ok = false; break; }
      tc_fence_after();
      float sv[64];
      tmem_ld64_sync(lane_addr + TM_S(sb), reinterpret_cast<uint32_t*>(sv));
      if (p.has_cap) cap_scores<64>(p, sv);
      const int64_t pos0 = (int64_t)t * KEYS + 64 * half;
      if (pos0 + 64 > min(u.q.ctx, (int64_t)u.q.kv)) {   // nodes, or the end of the keys
        const uint64_t v = visible(p.t, u, node, pos0);
#pragma unroll
        for (int k = 0; k < 64; ++k)
          if (!((v >> k) & 1)) sv[k] = NEG_INF;
      }
      float mx[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mx[k] = fmax3(fmax3(sv[8 * k], sv[8 * k + 1], sv[8 * k + 2]),
                      fmax3(sv[8 * k + 3], sv[8 * k + 4], sv[8 * k + 5]), fmaxf(sv[8 * k + 6], sv[8 * k + 7]));
      float mt = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sc;
      // The row's other thread has the other 64 keys.
      float other;
      if (!exchange(mt, &other)) { ok = false; break; }
      mt = fmaxf(mt, other);
      float m_new = m_used;
      bool rescale = false;
      if (t == u.lo) {
        m_new = mt;
      } else if (mt > m_used + TREE_RESCALE_THRESHOLD) {
        m_new = mt;
        rescale = true;
      }
      const float msub = (m_new == NEG_INF) ? 0.f : m_new;
      const float2 neg_m = make_float2(-msub, -msub);
      float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t pr[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float2 a = ffma2(make_float2(sv[2 * k], sv[2 * k + 1]), sc2, neg_m);
        const float2 e = make_float2(ex2_approx(a.x), ex2_approx(a.y));
        acc[k & 3] = fadd2(acc[k & 3], e);
        pr[k] = pack_bf16x2(e.x, e.y);   // the operand type; the sum is of the unrounded values
      }
      const float2 s01 = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
      const float sum = s01.x + s01.y;
      float alpha = 1.f;
      if (rescale) alpha = ex2_approx(m_used - m_new);
      l = l * alpha + sum;
      // The tile before this one has to be done with P, and with O if it is rescaled.
      if (g > 0 && !c.wait_warp(OD, (g - 1) & 1)) { ok = false; break; }
      if (__any_sync(0xffffffffu, rescale)) {   // tcgen05.ld/st are warp-collective
        tc_fence_after();
        const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float ov[64];
          tmem_ld64_sync(lane_addr + q * 64, reinterpret_cast<uint32_t*>(ov));
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float2 r = fmul2(make_float2(ov[2 * k], ov[2 * k + 1]), a2);
            ov[2 * k] = r.x;
            ov[2 * k + 1] = r.y;
          }
          tmem_st64_sync(lane_addr + q * 64, reinterpret_cast<uint32_t*>(ov));
        }
      }
      m_used = m_new;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        st_shared_v4(p_row + ((k ^ (row & 7)) << 4), pr[4 * k], pr[4 * k + 1], pr[4 * k + 2], pr[4 * k + 3]);
      fence_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        // What this publishes to the even CTA's issuing thread is not generic data: P was handed to
        // this CTA's async proxy by the fence above, S and O are ordered by the tcgen05 fence.  So a
        // release at CTA scope does; one at cluster scope took 2-4 thousand clocks here.
        if (c.rank) mbar_arrive_remote(pr_bar);
        else mbar_arrive(pr_bar);
      }
    }
    if (!ok) break;
    // The part's end: the row's sum, then O out of TMEM once the last product is done.
    float l_other;
    if (!exchange(l, &l_other)) break;
    const float l_row = l + l_other;
    if (!c.wait_warp(OD, (g - 1) & 1)) break;
    tc_fence_after();
    const bool empty = l_row == 0.f;   // (a NaN is passed on)
    const float inv = u.whole ? (empty ? 0.f : 1.f / l_row) : 1.f;
    const float2 inv2 = make_float2(inv, inv);
    char* slot = ws_slots + (size_t)u.slot * SLOT_BYTES;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      // TMEM columns 64 q ..: the values of CTA `half`, chunk q / 2 of 128
      const int col = 256 * half + 64 * q;
      uint32_t ov[64];
      tmem_ld64_sync(lane_addr + q * 64, ov);
      if (live && u.whole) {
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float2 r = fmul2(make_float2(__uint_as_float(ov[2 * k]), __uint_as_float(ov[2 * k + 1])), inv2);
          w[k] = empty ? 0u : pack_bf16x2(r.x, r.y);
        }
        __nv_bfloat16* d = p.t.o + pair * 512 + col;
        if (p.o_align32) {
#pragma unroll
          for (int k = 0; k < 4; ++k) st_global_v8(d + 16 * k, w + 8 * k);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            reinterpret_cast<uint4*>(d)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
      } else if (live) {
        char* d = slot + slot_at(pr0, col);
#pragma unroll
        for (int k = 0; k < 8; ++k) st_global_v8(d + slot_at(0, 8 * k), ov + 8 * k);
      }
      __syncwarp();   // (the next load is one instruction of the whole warp)
    }
    if (live && half == 0) {
      if (u.whole) {
        float lg;
        asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(l_row));
        if (p.t.lse) p.t.lse[pair] = empty ? NEG_INF : (m_used + lg) * 0.6931471805599453f;
      } else {
        reinterpret_cast<float2*>(slot + SLOT_ML)[pr0] = make_float2(m_used, l_row);
      }
    }
    tc_fence_before();   // O has been read: the next part's first P-ready lets it be overwritten
  }
}

// R: rows of a box of the cache (8, 16, 32, 64), 0: row by row.
template <int R>
__global__ void __launch_bounds__(NTHREADS, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ StartRec start;
  __shared__ int64_t count;
  __shared__ JoinRec join;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(smem + OFF_MISC + 4);
  int* begun = reinterpret_cast<int*>(smem + OFF_MISC + 8);   // tiles that the K producer has begun, less one
  const uint32_t rank = cluster_ctarank();
  const int worker = blockIdx.x >> 1;
  const Ctx c{smem_addr(smem), abort_flag, p.t.status, p.wait_limit_ns, rank};
  ReqWords words{0, 0, 0};   // (on their way while the barriers are made)
  if ((int)threadIdx.x < p.t.batch) words = load_words(p.t, threadIdx.x);
  if (warp == 1) {
    // P: every softmax warp of both CTAs; maxima: the two warps of 32 rows; rows: a warp of each CTA.
    static_assert(NBAR <= 32, "a lane each");
    const bool rows = R == 0 && ((lane >= KF && lane < KF + KGROUPS) || (lane >= VF && lane < VF + 2));
    if (lane < NBAR) mbar_init(c.bar(lane), lane == PR ? 8 : lane == XB || lane == XB + 1 || rows ? 2 : 1);
    if (lane == 0) {
      *abort_flag = 0;
      *begun = -1;
    }
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    if (R > 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  if (warp == 3) {   // one warp of each CTA of the pair, together
    tmem_alloc_pair(smem_addr(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  // Both CTAs' barriers exist, TMEM is there: waited for below.  (A release waits for the lengths' loads.)
  if (warp == 3) cluster_arrive();
  else cluster_arrive_relaxed();
  find_piece<NTHREADS>(p.t, words, worker, p.workers, blockIdx.x == 0, &start, &count, &join);
  char* ws = static_cast<char*>(p.t.workspace);
  if (threadIdx.x == 0 && rank == 0) reinterpret_cast<JoinRec*>(ws)[worker] = join;
  __syncwarp();
  cluster_wait();
  tc_fence_after();
  grid_dependency_wait();   // (rows that a kernel before this one makes are there)
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const Parts parts(p.t, start, count);
  if (warp == 0) {
    if constexpr (R > 0) run_producer_qk<R>(c, p, parts, &tm_q, &tm_k, begun);
    else run_rows<false>(c, p, parts, &tm_q, 0, KGROUPS - 1);
  } else if (warp == 2) {
    if constexpr (R > 0) run_producer_v<R>(c, p, parts, &tm_v, smem);
    else run_rows<true>(c, p, parts, &tm_q, 0, 2);
  } else if (warp == 1) {
    if (rank == 0) run_mma<R>(c, p, parts, tmem);
  } else if (warp == 3) {
    if constexpr (R > 0) run_prefetch<R>(c, p, parts, &tm_k, begun);
    else run_rows<false>(c, p, parts, &tm_q, KGROUPS - 1, 1);
  } else {
    run_softmax(c, p, parts, tmem, ws + WS_SLOTS + (size_t)worker * 2 * SLOT_BYTES, smem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // Neither CTA leaves (freeing shared memory and TMEM) while the even CTA's products may still
  // read or write the other's.  The commits of those products arrive in the odd CTA's shared memory too, the last of
  // them on barriers that nothing there waits for: the last commit of all is waited for here.
  if (warp == 1 && rank == 1) {
    if (lane == 0) c.drain(FIN, 0);
    __syncwarp();
  }
  cluster_sync();
  tc_fence_after();
  if (warp == 3) {
    __syncwarp();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

cudaLaunchConfig_t pair_config(cudaLaunchAttribute* attr, int workers, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * workers, 1, 1);
  cfg.blockDim = dim3(NTHREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const TreeLaunch);
Kernel kernel_of(int box_rows) {
  switch (box_rows) {
    case 8: return tree_attn_kernel<8>;
    case 16: return tree_attn_kernel<16>;
    case 32: return tree_attn_kernel<32>;
    case 64: return tree_attn_kernel<64>;
    default: return tree_attn_kernel<0>;
  }
}

// Clusters that run at once on the current device (0 on error).
int max_workers() {
  static PerDeviceOnce configured;
  static int workers[PerDeviceOnce::kMaxDevices] = {};
  const cudaError_t e = configured.run([] {
    cudaError_t r = cudaSuccess;
    for (int rows : {0, 8, 16, 32, 64})
      if (r == cudaSuccess)
        r = cudaFuncSetAttribute(kernel_of(rows), cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    int dev = 0, n = 0;
    if (r == cudaSuccess) r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pair_config(attr, 1, nullptr);
    r = cudaOccupancyMaxActiveClusters(&n, kernel_of(64), &cfg);
    if (r == cudaSuccess) workers[dev] = n < MAX_WORKERS ? n : MAX_WORKERS;
    return r;
  });
  int dev = 0;
  if (e != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return 0;
  return workers[dev];
}

}  // namespace

int64_t tree_workspace_bytes() {
  const int n = max_workers();
  return n > 0 ? (int64_t)(WS_SLOTS + (size_t)n * 2 * SLOT_BYTES) : 0;
}

cudaError_t launch_tree_attention(const TreeParams& t, cudaStream_t stream, bool rows_on_their_way) {
  const TreeLaunch p = tree_launch(t, max_workers());
  if (p.workers <= 0) return cudaErrorInvalidConfiguration;
  const bool any = t.max_blocks > 0;   // some cache row may be read
  const int bs = t.block_size;
  const uint64_t slots = any ? (uint64_t)t.num_blocks * (uint64_t)bs : 1;
  CUtensorMap tq, tk, tv;
  {
    const uint64_t dims[3] = {64, (uint64_t)t.total_rows * (uint64_t)t.num_heads, NP}, strides[2] = {576 * 2, 64 * 2};
    const uint32_t box[3] = {64, 64, NP};   // 64 rows, panel by panel
    if (make_tensor_map_bf16(&tq, t.q, 3, dims, strides, box) != MLA_OK) return cudaErrorInvalidValue;
  }
  // Boxes for 64-key pieces: of as many rows, 64 to 8, as the block size is a multiple of (8 rows keep a
  // box on the swizzle's 1024-byte period; by gather4 blocks of 24, 48 and 96 took 235 us where they
  // take 82, 16 requests of 4 nodes, 128 heads, over 4096); several panels in
  // one box by a map of the rows as {64 columns, rows, 9 column groups}.  Smaller boxes' keys come eight
  // rows at a time with three panels (all nine at once: 8 copies instead of 24, but products wait for
  // all of them: 86 us instead of 82 for blocks of 24), their values with four.
  const int box_rows = !any ? 0 : bs % 64 == 0 ? 64 : bs % 32 == 0 ? 32 : bs % 16 == 0 ? 16 : bs % 8 == 0 ? 8 : 0;
  if (box_rows > 0) {
    const uint64_t dims[3] = {64, slots, NP}, strides[2] = {576 * 2, 64 * 2};
    const uint32_t box_k[3] = {64, box_rows == 64 ? 64u : 8u, 3};
    const uint32_t box_v[3] = {64, (uint32_t)box_rows, 4};
    if (make_tensor_map_bf16(&tk, t.cache, 3, dims, strides, box_k) != MLA_OK ||
        make_tensor_map_bf16(&tv, t.cache, 3, dims, strides, box_v) != MLA_OK)
      return cudaErrorInvalidValue;
  } else {
    tk = tv = tq;   // (not used)
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pair_config(attr, p.workers, stream);
  if (rows_on_their_way) {   // the start beside the end of the kernel that makes them
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel_of(box_rows), tq, tk, tv, p);
  return e != cudaSuccess ? e : launch_tree_join(p, stream);
}

}  // namespace mla
