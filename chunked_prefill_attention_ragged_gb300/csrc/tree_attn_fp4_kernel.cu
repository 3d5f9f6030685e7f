// Tree attention over a cache of 4-bit entries: the mathematics and the split of the work of tree_attn_kernel.cu (a
// cluster of two CTAs runs a unit of 128 pairs with cta_group::2 products of M = 128, 64 pairs in each CTA), over
// keys and values that are made bf16 on their way into shared memory.
//
// Each CTA makes its half of a tile's keys once, as its half of S's B operand.  A key's first 512 values are its
// value too: its columns 0-255 are values of the even CTA and 256-511 of the odd one, in the swizzle that they have as
// keys.  The columns that are the CTA's own values are stored twice, the others go from its keys to the other CTA by bulk
// copies from shared memory to shared memory.  (Keys and values made from the entries by four warps each, twice the
// conversions: 32 x 1 over ragged contexts at 128 heads 106 us, 32 x 16 over 8192 1545; all values copied 102 and 1468; so
// 99 and 1408.  Stores to the other CTA, with a release at cluster scope: 166 and 2707.)  Entries go straight from L2 to
// registers: there is no room for them in shared memory beside Q (72 KB), two tiles (136 KB) and P (16 KB).
//   warp 0      Q producer
//   warp 1      even CTA: issues every product; odd CTA: tells that the copies to it landed
//   warp 2      copies to the other CTA
//   warp 3      TMEM allocation; ropes; brings entries into L2
//   warps 4-11  softmax: four threads per pair (quarters of the keys and of O's columns)
//   warps 12-19 keys
// A tile has 64 keys, so that there are two: with one of 128 its making, S, P V and the copies took turns (149 and 2207 us).
// Either S of the next tile or P V of this one is issued, whichever has its operands first (S always first: 1.5% more).
// What bounds it (32 x 1 over ragged contexts at 128 heads, 98.4 us in replayed graphs, where bf16 entries take 70.6; 64 x 1
// over 8192 at 32, 64 and 128 heads 189, 192 and 195-199, most of a unit's 128 pairs padding at 32 and 64, bf16 entries
// 112, 115 and 122; 32 x 16 over 8192 1408-1425, 0.44 of the measured tensor rate): a tile takes 3000 clocks, half of its way through the roles (two are in flight), in which 270 KB
// pass through shared memory (S 108: Q's rows are read for each product, so that one of 64 keys takes as long as one of
// 128, 30 clocks).  With a stage left out in turn the first case takes: a third of S 89 us, copies of an eighth 92, no loads
// 92, stores of a quarter of the keys 95, a quarter of P V 97, no arithmetic on codes 99; without any of them 69, waits and
// barriers alone.  Sixteen warps that make keys, or every warp looking at its barrier itself: no faster.
// Calls with more than a unit a request mostly come here without room for bf16 rows (see launch_tree_attention_fp4).
// A code becomes bf16 by moving its bits to a bf16's low exponent bits and one product by 2^126 times the
// scale, exact; scales above 2, where that factor has no bf16, take two products (a tile in which a warp
// meets one).  A row with a scale byte above 252 has NaN in its rope, which only S sees, and zeros for values,
// so that it cannot reach rows that do not see it.  Rows that are not there are zeros.
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "tmem_wide.cuh"
#include "tree_attn.cuh"
#include "tree_issue.cuh"

namespace mla {
namespace {

constexpr int ROWS = 128, KEYS = 64;
constexpr int NTHREADS = 640;
constexpr int AHEAD = 4;                // tiles between the one being made and the one brought into L2
constexpr int NP = 9;                   // 64-column panels of 576
constexpr int QP = 64 * 128;            // a panel of Q, P or V: 64 rows
constexpr int KP = KEYS / 2 * 128;      // a panel of K: the CTA's half of the keys
constexpr int V_HALF = 4 * KP;          // of V: four panels of the keys of one CTA
constexpr int K_TILE = NP * KP, V_TILE = 2 * V_HALF;
constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + NP * QP;              // two tiles
constexpr int OFF_V = OFF_K + 2 * K_TILE;           // two tiles: 64 keys x the CTA's 256 value columns
constexpr int OFF_P = OFF_V + 2 * V_TILE;           // two tiles
constexpr int OFF_XCHG = OFF_P + 2 * QP;            // [4 threads][64 rows] maxima
constexpr int OFF_BAR = OFF_XCHG + 4 * 64 * 4;
enum Bar {
  QF = 0,       // Q landed
  QE,           // the unit's last S done: Q may be replaced
  KF,           // [buffer] keys made (of both CTAs), for the products
  KL = KF + 2,  // [buffer] the CTA's own, but for the ropes, for their copies
  VF = KL + 2,  // [buffer] the peer's half of the CTA's values landed
  VR = VF + 2,  // [buffer] (even CTA) the odd one's did
  VE = VR + 2,  // [buffer] P V done: keys, values, P and, for the next rescale, O are free
  SF = VE + 2,  // [buffer] S done (in both CTAs)
  PR = SF + 2,  // [buffer] P written (and the S buffer read) by every softmax warp of both CTAs
  FIN = PR + 2, // every product drained
  NEVER,        // nothing arrives here: the time-out test mode waits on it
  NBAR
};
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int SMEM = OFF_MISC + 64 + 1024;   // + slack for 1024-byte alignment
static_assert(SMEM + 512 <= 227 * 1024, "shared memory budget");
constexpr uint32_t TMEM_COLS = 512;
__device__ __forceinline__ constexpr uint32_t TM_S(int b) { return 256u + (uint32_t)b * (KEYS / 2); }
constexpr uint32_t IDESC_QK = idesc_bf16_f32(ROWS, KEYS, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16_f32(ROWS, 256, false, true);
using PartsK = PartsOf<ROWS, KEYS>;

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
  __device__ bool wait_warp(int b, uint32_t parity) const {
    return mla::wait_warp(bar(b), parity, abort_flag, status, wait_limit_ns);
  }
  // Whether a phase is complete: one lane looks, all see what it acquired.
  __device__ bool look(int b, uint32_t parity) const {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, 0, 0;\n\t"
        "@e mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r)
        : "r"(bar(b)), "r"(parity)
        : "memory");
    const bool yes = __any_sync(0xffffffffu, r != 0);
    __syncwarp();
    return yes;
  }
  __device__ void drain(int b, uint32_t parity) const {
    int dummy = 0;
    mbar_wait_bounded(bar(b), parity, &dummy, status, MLA_DEVSTAT_TIMEOUT, TREE_DRAIN_LIMIT_NS, true);
  }
};

// Zeros, or the load: without a copy of its registers, which would wait for it.
__device__ __forceinline__ uint4 load16_if(bool there, const uint8_t* p) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)there));
  return v;
}
__device__ __forceinline__ uint32_t load1_if(bool there, const uint8_t* p) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.nc.u8 %0, [%1];\n\t}\n"
      : "=&r"(v)
      : "l"(p), "r"((uint32_t)there));
  return v;
}

// A warp's part of what it writes is there: handed to the asynchronous proxy, told to the even CTA.
__device__ __forceinline__ void tell(const Ctx& c, int b, int lane) {
  fence_async_shared();
  __syncwarp();
  if (lane == 0) {
    if (c.rank) mbar_arrive_remote(mapa_shared(c.bar(b), 0));
    else mbar_arrive(c.bar(b));
  }
}

// Warps 12-19: four of the CTA's 32 keys each.  Lane (panel % 4, row, half panel) = (l / 8, l / 2 % 4, l % 2) makes
// two pieces of 32 columns, of panel % 4 and panel % 4 + 4.  A load takes 128 bytes of four rows, and eight lanes of a
// store have eight different bank groups.
struct Pieces {
  uint4 code[2];
  uint32_t scale[2];
};
__device__ void run_rows(const Ctx& c, const TreeLaunch& p, PartsK parts) {
  const int lane = threadIdx.x & 31, w8 = (threadIdx.x >> 5) & 7, r4 = (lane >> 1) & 3;
  const int group = 2 * (lane >> 3) + (lane & 1);   // of four panels' eight
  const int row8 = 4 * (w8 & 1) + r4;               // row % 8: the swizzle
  uint32_t chunk[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) chunk[i] = ((4 * (lane & 1) + i) ^ row8) << 4;
  const uint32_t values_at = c.sbase + OFF_V + c.rank * V_HALF + (lane >> 3) * KP + (4 * w8 + r4) * 128;
  const uint32_t keys_at = c.sbase + OFF_K + (lane >> 3) * KP + (4 * w8 + r4) * 128;
  const uint8_t* cache = reinterpret_cast<const uint8_t*>(p.t.cache);
  int g = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    const int64_t end = min((int64_t)u.hi * KEYS, (int64_t)u.q.kv);
    // A block as the table has it: looked at a tile later, so that nothing waits for it here.
    auto find = [&](int64_t key) {
      return key < end ? __ldg(p.t.block_table + (int64_t)u.r * p.t.max_blocks + block_of(p, (int)key)) : 0;
    };
    auto get = [&](int32_t blk, int64_t key, Pieces* to) {
      const int32_t row = key < end ? block_row(p, blk == PAST_END ? -1 : blk, key) : p.oob_row;
      const bool there = row != p.oob_row;
      const uint8_t* e = cache + (int64_t)row * FP4_ENTRY;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        to->code[j] = load16_if(there, e + 16 * group + 128 * j);
        to->scale[j] = load1_if(there, e + FP4_SCALES + group + 8 * j);
      }
    };
    int64_t key = (int64_t)u.lo * KEYS + KEYS / 2 * (int)c.rank + 4 * w8 + r4;
    Pieces now;
    get(find(key), key, &now);
    int32_t blk = find(key + KEYS);
#pragma unroll 1
    for (int t = u.lo; t < u.hi; ++t, ++g) {
      const int b = g & 1;
      const bool big = __any_sync(0xffffffffu, max(now.scale[0], now.scale[1]) > 128);
      uint32_t r[2][16];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // 2^126 times the scale, or one after the other; values of a row that is NaN are zeros
        const uint32_t s = now.scale[j], words[4] = {now.code[j].x, now.code[j].y, now.code[j].z, now.code[j].w};
        uint32_t m = big ? 0x7e80u : (s + 126) << 7;
        if (big && s > FP4_MAX_SCALE) m = 0;
        m |= m << 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          fp4_fields(words[i], r[j] + 4 * i);
#pragma unroll
          for (int k = 0; k < 4; ++k) r[j][4 * i + k] = mul_bf16x2(r[j][4 * i + k], m);
        }
        if (big) {
          const uint32_t m2 = scale_bf16x2(s > FP4_MAX_SCALE ? 0 : s);
#pragma unroll
          for (int k = 0; k < 16; ++k) r[j][k] = mul_bf16x2(r[j][k], m2);
        }
      }
      key += KEYS;
      get(blk, key, &now);
      blk = find(key + KEYS);
      __syncwarp();
      if (w8 == 0 && g > 1) ok = c.wait_warp(VE + b, ((g >> 1) - 1) & 1);
      if (meet<256>(3, !ok)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v4(keys_at + b * K_TILE + 4 * j * KP + chunk[i], r[j][4 * i], r[j][4 * i + 1], r[j][4 * i + 2], r[j][4 * i + 3]);
      const uint32_t to = values_at + b * V_TILE;   // the columns that are the CTA's values
      if (c.rank == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) st_shared_v4(to + chunk[i], r[0][4 * i], r[0][4 * i + 1], r[0][4 * i + 2], r[0][4 * i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) st_shared_v4(to + chunk[i], r[1][4 * i], r[1][4 * i + 1], r[1][4 * i + 2], r[1][4 * i + 3]);
      }
      tell(c, KF + b, lane);
      if (lane == 0) mbar_arrive(c.bar(KL + b));
    }
  }
}

// Warp 2: the columns that are values of the other CTA go there as they are, from shared memory to shared memory.
// (That keys are made says that P V of the tile before last is done, and with it that the other CTA's buffer is free.)
__device__ void run_copies(const Ctx& c, PartsK parts) {
  const int lane = threadIdx.x & 31;
  const uint32_t other = c.rank ^ 1, from = c.sbase + OFF_K + other * V_HALF;
  const uint32_t to = mapa_shared(c.sbase + OFF_V + c.rank * V_HALF, other), full = mapa_shared(c.bar(VF), other);
  int g = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
#pragma unroll 1
    for (int t = u.lo; t < u.hi; ++t, ++g) {
      const int b = g & 1;
      ok = c.wait_warp(KL + b, (g >> 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(c.bar(VF + b), V_HALF);
        asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to + b * V_TILE),
                     "r"(from + b * K_TILE), "r"(V_HALF), "r"(full + 8 * b)
                     : "memory");
      }
      __syncwarp();
    }
  }
  if (!ok) {   // the copies under way land before a CTA can exit: they have this long
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < TREE_DRAIN_LIMIT_NS) {
    }
  }
}

// The odd CTA's warp 1: what it got landed.
__device__ void run_relay(const Ctx& c, PartsK parts) {
  const uint32_t there = mapa_shared(c.bar(VR), 0);
  int g = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
#pragma unroll 1
    for (int t = u.lo; t < u.hi && ok; ++t, ++g) {
      ok = c.wait_warp(VF + (g & 1), (g >> 1) & 1);
      if (ok && (threadIdx.x & 31) == 0) mbar_arrive_remote(there + 8 * (g & 1));
      __syncwarp();
    }
  }
}

// Warp 3: the ropes of the CTA's 32 keys, K's last panel, and the entries of the tiles to come into L2.  Lane i has
// 16 bytes of rows 4 j + i / 8, loaded a tile ahead; a row with a scale byte above 252 gets NaN.
__device__ void run_ropes(const Ctx& c, const TreeLaunch& p, PartsK parts) {
  const int lane = threadIdx.x & 31, ch = lane & 7, r0 = lane >> 3;
  const uint8_t* cache = reinterpret_cast<const uint8_t*>(p.t.cache);
  int g = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    const int64_t end = min((int64_t)u.hi * KEYS, (int64_t)u.q.kv);
    int64_t key = (int64_t)u.lo * KEYS + KEYS / 2 * c.rank + lane;
    auto find = [&](int64_t k) {
      return k < end ? __ldg(p.t.block_table + (int64_t)u.r * p.t.max_blocks + block_of(p, (int)k)) : 0;
    };
    auto row_of = [&](int32_t blk, int64_t k) {
      const int32_t row = k < end ? block_row(p, blk == PAST_END ? -1 : blk, k) : p.oob_row;
      if (row != p.oob_row) {
        const uint8_t* e = cache + (int64_t)row * FP4_ENTRY;
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("prefetch.global.L2 [%0];" ::"l"(e + 128 * i) : "memory");
      }
      return row;
    };
    uint4 rope[8], s;
    auto load = [&](int32_t rows) {
      s = load16_if(rows != p.oob_row, cache + (int64_t)rows * FP4_ENTRY + FP4_SCALES);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int32_t row = __shfl_sync(0xffffffffu, rows, 4 * j + r0);
        rope[j] = load16_if(row != p.oob_row, cache + (int64_t)row * FP4_ENTRY + FP4_ROPE + ch * 16);
      }
    };
    int32_t blk[AHEAD + 1], row[AHEAD];   // row[i]: of the tile i + 1 ahead
#pragma unroll
    for (int i = 0; i <= AHEAD; ++i) blk[i] = find(key + i * KEYS);
    load(row_of(blk[0], key));
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) row[i] = row_of(blk[i + 1], key + (i + 1) * KEYS);
    int32_t last = find(key + (AHEAD + 1) * KEYS);
#pragma unroll 1
    for (int t = u.lo; t < u.hi; ++t, ++g, key += KEYS) {
      const int b = g & 1;
      const uint32_t dst = c.sbase + OFF_K + b * K_TILE + 8 * KP + r0 * 128;
      if (g > 1 && !c.wait_warp(VE + b, ((g >> 1) - 1) & 1)) {
        ok = false;
        break;
      }
      const uint32_t bad = __ballot_sync(0xffffffffu, (above252(s.x) | above252(s.y) | above252(s.z) | above252(s.w)) != 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if ((bad >> (4 * j + r0)) & 1) rope[j] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        st_shared_v4(dst + j * 512 + ((ch ^ (4 * (j & 1) + r0)) << 4), rope[j].x, rope[j].y, rope[j].z, rope[j].w);
      }
      tell(c, KF + b, lane);
      const int32_t rows = row[0];
#pragma unroll
      for (int i = 0; i + 1 < AHEAD; ++i) row[i] = row[i + 1];
      row[AHEAD - 1] = row_of(last, key + (AHEAD + 1) * KEYS);
      load(rows);
      last = find(key + (AHEAD + 2) * KEYS);
    }
  }
}

__device__ void run_queries(const Ctx& c, PartsK parts, const CUtensorMap* tq) {
  const int lane = threadIdx.x & 31;
  int units = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    if (lane == 0) {
      if (units > 0) ok = c.wait(QE, (units - 1) & 1);
      if (ok) {
        // (both CTAs' copies complete on the even one's barrier, where the products wait)
        if (c.rank == 0) mbar_arrive_expect_tx(c.bar(QF), 2 * NP * QP);
        tma_load_3d_pair(c.sbase + OFF_Q, tq, mapa_shared(c.bar(QF), 0), 0, (int32_t)(u.pair0 + 64 * c.rank), 0);
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok) ++units;
  }
  if (lane == 0) {   // the copies land before the CTA can exit
    if (c.rank == 0) {
      if (units) c.drain(QF, (units - 1) & 1);
    } else if (!ok) {   // the odd CTA cannot see its own: they have this long
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < TREE_DRAIN_LIMIT_NS) {
      }
    }
  }
}

// ------------------------------------------------------------------ products (even CTA, warp 1)
__device__ void run_mma(const Ctx& c, const TreeLaunch& p, PartsK parts, uint32_t tmem) {
  const uint64_t q_desc = sdesc_sw128(c.sbase + OFF_Q, 16, 1024);
  const uint64_t k_desc = sdesc_sw128(c.sbase + OFF_K, 16, 1024);
  const uint64_t v_desc = sdesc_sw128(c.sbase + OFF_V, KP, 1024);
  const uint64_t p_desc = sdesc_sw128(c.sbase + OFF_P, 16, 1024);
  bool ok = true;
  if (p.force_timeout) ok = c.wait_warp(NEVER, 0);
  int st = 0, pv = 0, units = 0;
  auto s_products = [&](bool last) {
    const int b = st & 1;
    const uint32_t d = __shfl_sync(0xffffffffu, tmem + TM_S(b), 0), tile = __shfl_sync(0xffffffffu, (uint32_t)(b * K_TILE) >> 4, 0);
    tc_fence_after();
#pragma unroll 1
    for (int i = 0; i < NP; ++i) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        issue_pair(d, q_desc + ((uint32_t)(i * QP + kk * 32) >> 4), k_desc + tile + ((uint32_t)(i * KP + kk * 32) >> 4), IDESC_QK,
                   kk > 0 ? 1u : i > 0 ? 1u : 0u);
    }
    commit_both(c.bar(SF + b));
    if (last) commit_both(c.bar(QE));
    ++st;
  };
  auto pv_products = [&](uint32_t add) {
    const int b = pv & 1;
    const uint32_t more = __shfl_sync(0xffffffffu, add, 0);
    const uint32_t tile = __shfl_sync(0xffffffffu, (uint32_t)(b * V_TILE) >> 4, 0), pt = __shfl_sync(0xffffffffu, (uint32_t)(b * QP) >> 4, 0);
    tc_fence_after();
#pragma unroll 1
    for (int ch = 0; ch < 2; ++ch) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        issue_pair(tmem + ch * 128, p_desc + pt + ((uint32_t)(kk * 32) >> 4), v_desc + tile + ((uint32_t)(2 * ch * KP + (kk >> 1) * V_HALF + (kk & 1) * 2048) >> 4),
                   IDESC_PV, kk > 0 ? 1u : more);
    }
    commit_both(c.bar(VE + b));
    ++pv;
  };
  Part u;
  while (ok && parts.next(&u)) {
    const int n = __shfl_sync(0xffffffffu, u.hi - u.lo, 0);
    ok = c.wait_warp(QF, units & 1);
    ++units;
    // S's buffer holds the scores of the tile before last, read before that tile's P was ready: its P V has to be behind.
    const int s_end = st + n, pv_begin = pv;
    uint64_t since = 0;
    for (uint32_t it = 0; ok && pv < s_end; ++it) {
      const int bp = pv & 1, bs = st & 1;
      if (pv < st && c.look(PR + bp, (pv >> 1) & 1) && c.look(VF + bp, (pv >> 1) & 1) && c.look(VR + bp, (pv >> 1) & 1)) {
        pv_products(pv > pv_begin ? 1u : 0u);
        it = 0;
      } else if (st < s_end && st - pv < 2 && c.look(KF + bs, (st >> 1) & 1)) {
        s_products(st == s_end - 1);
        it = 0;
      } else if ((it & 63) == 63) {
        const uint64_t now = global_timer_ns();
        if (it == 63) since = now;
        const bool late = now - since > c.wait_limit_ns;
        if (__any_sync(0xffffffffu, late || *c.abort_flag)) {
          if (late) {
            *c.abort_flag = 1;
            if (c.status) atomicOr(c.status, MLA_DEVSTAT_TIMEOUT);
          }
          ok = false;
        }
      }
    }
  }
  commit_both(c.bar(FIN));
  c.drain(FIN, 0);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax (warps 4-11)
// Four threads a row: (half, quarter) have keys 32 half + 16 quarter .. and columns 256 half + 128 quarter ...  One of
// the eight warps looks for S and the others meet it; as these meetings have no time limit, where a wait gave up the
// warps go through the rest of their tiles without waiting.
__device__ void run_softmax(const Ctx& c, const TreeLaunch& p, PartsK parts, uint32_t tmem, char* ws_slots, uint8_t* smem) {
  const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3, sub = ((threadIdx.x >> 5) - 4) >> 2;
  const int half = q4 >> 1, rg = q4 & 1;             // key / column half, group of 32 rows
  const int row = 32 * rg + lane;                    // of the CTA's 64
  const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16);
  float* xchg = reinterpret_cast<float*>(smem + OFF_XCHG);
  const uint32_t p_row = c.sbase + OFF_P + row * 128;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const float sc = p.has_cap ? 1.f : p.scale_log2;
  const float2 sc2 = make_float2(sc, sc);
  bool ok = true;
  int g = 0;
  auto wait = [&](int b, uint32_t parity) { ok = ok && c.wait_warp(b, parity); };
  // The four threads' values of a row; a meeting of the row group's warps lies between two exchanges.
  auto exchange = [&](float mine) {
    xchg[(2 * half + sub) * 64 + row] = mine;
    meet<128>(5 + rg, false);
    return make_float4(xchg[row], xchg[64 + row], xchg[128 + row], xchg[192 + row]);
  };
  Part u;
  while (parts.next(&u)) {
    const int pr0 = 64 * (int)c.rank + row;          // pair inside the unit
    const int64_t pair = u.pair0 + pr0;
    // A row without a pair computes on something harmless: the last node's mask.
    const int node = min((int)((pair - (int64_t)u.q.q0 * p.t.num_heads) / p.t.num_heads), u.q.nodes - 1);
    float m_used = NEG_INF, l = 0.f;
#pragma unroll 1
    for (int t = u.lo; t < u.hi; ++t, ++g) {
      const int b = g & 1;
      if (q4 == 0 && sub == 0) wait(SF + b, (g >> 1) & 1);
      if (meet<256>(2, !ok)) ok = false;
      tc_fence_after();
      float sv[16];
      tmem_ld16_sync(lane_addr + TM_S(b) + 16 * sub, reinterpret_cast<uint32_t*>(sv));
      if (p.has_cap) cap_scores<16>(p, sv);
      const int64_t pos0 = (int64_t)t * KEYS + 32 * half + 16 * sub;
      if (pos0 + 16 > min(u.q.ctx, (int64_t)u.q.kv)) {   // nodes, or the end of the keys
        const uint32_t v = (uint32_t)visible(p.t, u, node, pos0);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (!((v >> k) & 1)) sv[k] = NEG_INF;
      }
      float mx[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        mx[k] = fmax3(fmax3(sv[8 * k], sv[8 * k + 1], sv[8 * k + 2]),
                      fmax3(sv[8 * k + 3], sv[8 * k + 4], sv[8 * k + 5]), fmaxf(sv[8 * k + 6], sv[8 * k + 7]));
      const float mt = fmaxf(mx[0], mx[1]) * sc;
      // The row's maximum is asked for in a part's first tile and where some row's has grown by more than the threshold;
      // elsewhere the reference stays, and no probability is above 2^threshold.
      float m_new = m_used;
      bool rescale = false;
      const bool first = t == u.lo;
      if (meet<128>(5 + rg, first || mt > m_used + TREE_RESCALE_THRESHOLD)) {
        const float4 x = exchange(mt);
        const float top = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
        if (first) {
          m_new = top;
        } else if (top > m_used + TREE_RESCALE_THRESHOLD) {
          m_new = top;
          rescale = true;
        }
      }
      const float msub = (m_new == NEG_INF) ? 0.f : m_new;
      const float2 neg_m = make_float2(-msub, -msub);
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t pr[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 a = ffma2(make_float2(sv[2 * k], sv[2 * k + 1]), sc2, neg_m);
        const float2 e = make_float2(ex2_approx(a.x), ex2_approx(a.y));
        acc[k & 1] = fadd2(acc[k & 1], e);
        pr[k] = pack_bf16x2(e.x, e.y);   // the operand type; the sum is of the unrounded values
      }
      const float2 s01 = fadd2(acc[0], acc[1]);
      const float alpha = rescale ? ex2_approx(m_used - m_new) : 1.f;
      l = l * alpha + (s01.x + s01.y);
      // (P's buffer was read by the tile before last's product, issued before this tile's S)
      if (__any_sync(0xffffffffu, rescale)) {        // O behind the last one's; tcgen05.ld/st are warp-collective
        wait(VE + (b ^ 1), ((g - 1) >> 1) & 1);
        tc_fence_after();
        const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          const uint32_t at = lane_addr + 128 * sub + q * 16;
          tmem_ld16_sync(at, reinterpret_cast<uint32_t*>(sv));
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 r = fmul2(make_float2(sv[2 * k], sv[2 * k + 1]), a2);
            sv[2 * k] = r.x;
            sv[2 * k + 1] = r.y;
          }
          tmem_st16_sync(at, reinterpret_cast<uint32_t*>(sv));
        }
      }
      m_used = m_new;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        st_shared_v4(p_row + b * QP + (((4 * half + 2 * sub + k) ^ (row & 7)) << 4), pr[4 * k], pr[4 * k + 1], pr[4 * k + 2], pr[4 * k + 3]);
      tc_fence_before();
      tell(c, PR + b, lane);
    }
    // The part's end: the row's sum, then O out of TMEM once the last product is done.
    meet<128>(5 + rg, false);
    const float4 ls = exchange(l);
    const float l_row = (ls.x + ls.y) + (ls.z + ls.w);
    wait(VE + ((g - 1) & 1), ((g - 1) >> 1) & 1);
    tc_fence_after();
    const bool live = ok && pr0 < u.npairs, empty = l_row == 0.f;   // (a NaN is passed on)
    const float inv = u.whole ? (empty ? 0.f : 1.f / l_row) : 1.f;
    const float2 inv2 = make_float2(inv, inv);
    char* slot = ws_slots + (size_t)u.slot * SLOT_BYTES;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      const int col = 256 * half + 128 * sub + 32 * q;   // TMEM columns 128 sub + 32 q ..: the values of CTA `half`
      uint32_t ov[32];
      tmem_ld32_sync(lane_addr + 128 * sub + q * 32, ov);
      if (live && u.whole) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 r = fmul2(make_float2(__uint_as_float(ov[2 * k]), __uint_as_float(ov[2 * k + 1])), inv2);
          w[k] = empty ? 0u : pack_bf16x2(r.x, r.y);
        }
        __nv_bfloat16* d = p.t.o + pair * 512 + col;
        if (p.o_align32) {
#pragma unroll
          for (int k = 0; k < 2; ++k) st_global_v8(d + 16 * k, w + 8 * k);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            reinterpret_cast<uint4*>(d)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
      } else if (live) {
        char* d = slot + slot_at(pr0, col);
#pragma unroll
        for (int k = 0; k < 4; ++k) st_global_v8(d + slot_at(0, 8 * k), ov + 8 * k);
      }
      __syncwarp();   // (the next load is one instruction of the whole warp)
    }
    if (live && half == 0 && sub == 0) {
      if (u.whole) {
        if (p.t.lse) p.t.lse[pair] = empty ? NEG_INF : (m_used + log2f(l_row)) * 0.6931471805599453f;
      } else {
        reinterpret_cast<float2*>(slot + SLOT_ML)[pr0] = make_float2(m_used, l_row);
      }
    }
    tc_fence_before();   // O has been read: the next part's first P-ready lets it be overwritten
  }
}

__global__ void __launch_bounds__(NTHREADS, 1)
tree_attn_fp4_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ TreeLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ StartRec start;
  __shared__ int64_t count;
  __shared__ JoinRec join;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(smem + OFF_MISC + 4);
  const uint32_t rank = cluster_ctarank();
  const int worker = blockIdx.x >> 1;
  const Ctx c{smem_addr(smem), abort_flag, p.t.status, p.wait_limit_ns, rank};
  ReqWords words{0, 0, 0};   // (on their way while the barriers are made)
  if ((int)threadIdx.x < p.t.batch) words = load_words(p.t, threadIdx.x);
  if (warp == 1) {
    // P: every softmax warp of both CTAs; keys: eight warps of each CTA and the ropes'.
    static_assert(NBAR <= 32, "a lane each");
    const bool keys = lane == KF || lane == KF + 1, local = lane == KL || lane == KL + 1, probs = lane == PR || lane == PR + 1;
    if (lane < NBAR) mbar_init(c.bar(lane), keys ? 18 : probs ? 16 : local ? 8 : 1);
    if (lane == 0) *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tm_q);
  if (warp == 3) {   // one warp of each CTA of the pair, together
    tmem_alloc_pair(smem_addr(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  if (warp == 3) cluster_arrive();   // (see tree_attn_kernel)
  else cluster_arrive_relaxed();
  find_piece<NTHREADS, ROWS, KEYS>(p.t, words, worker, p.workers, blockIdx.x == 0, &start, &count, &join);
  char* ws = static_cast<char*>(p.t.workspace);
  if (threadIdx.x == 0 && rank == 0) reinterpret_cast<JoinRec*>(ws)[worker] = join;
  __syncwarp();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const PartsK parts(p.t, start, count);
  if (warp < 4) {
    if (warp == 0) run_queries(c, parts, &tm_q);
    else if (warp == 1 && rank == 0) run_mma(c, p, parts, tmem);
    else if (warp == 1) run_relay(c, parts);
    else if (warp == 2) run_copies(c, parts);
    else run_ropes(c, p, parts);
  } else if (warp < 12) {
    run_softmax(c, p, parts, tmem, ws + WS_SLOTS + (size_t)worker * 2 * SLOT_BYTES, smem);
  } else {
    run_rows(c, p, parts);
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

// Clusters that run at once on the current device (0 on error), no more than the workspace has room for.
int max_workers() {
  static PerDeviceOnce configured;
  static int workers[PerDeviceOnce::kMaxDevices] = {};
  const cudaError_t e = configured.run([] {
    cudaError_t r = cudaFuncSetAttribute(tree_attn_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (r != cudaSuccess) return r;
    int dev = 0, n = 0;
    r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pair_config(attr, 1, nullptr);
    r = cudaOccupancyMaxActiveClusters(&n, tree_attn_fp4_kernel, &cfg);
    if (r != cudaSuccess) return r;
    const int64_t room = (tree_workspace_bytes() - (int64_t)WS_SLOTS) / (int64_t)(2 * SLOT_BYTES);
    workers[dev] = (int)std::min<int64_t>(n, std::min<int64_t>(room, MAX_WORKERS));
    return r;
  });
  int dev = 0;
  if (e != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return 0;
  return workers[dev];
}

int64_t pairs_of_a_request(int64_t total_rows, int num_heads, int batch) {   // on average
  return (total_rows * num_heads + batch - 1) / std::max(batch, 1);
}
// Where the bf16 rows are, in a workspace that has room for them.
int64_t expanded_at() { return (tree_workspace_bytes() + 1023) & ~int64_t(1023); }
}  // namespace

// With more pairs a request than a unit has, each row is read by two units and more, and making them bf16 once, for the
// kernel over bf16 caches, is faster than making each unit's keys again.  (Replayed graphs, without and with: 32 x 3 over
// 8192 at 64 heads, 192 pairs, 194 us and 181, 32 x 2 at 128 196 and 182, 32 x 4 373 and 276, 32 x 16 1423 and 852; 1 x 2
// over 8192 at 128 heads 35.6 and 35.8, 1 x 16 65 and 41; of one unit, 32 x 1 over 8192 at 128 heads 110 and 140.)  It takes
// 1152 bytes for each slot of the cache, whatever the call reads of it: above 4 GB of them it is left.
constexpr int64_t EXPAND_BYTES = int64_t(4) << 30;
int64_t tree_workspace_fp4_bytes(int64_t total_rows, int num_heads, int batch, int64_t num_blocks, int block_size) {
  const int64_t rows = num_blocks * block_size * (576 * 2), base = tree_workspace_bytes();
  const bool pays = batch > 0 && batch <= 65535 &&
                    pairs_of_a_request(total_rows, num_heads, batch) > ROWS && rows > 0 && rows <= EXPAND_BYTES;
  return base > 0 && pays ? expanded_at() + rows : base;
}

cudaError_t launch_tree_attention_fp4(const TreeParams& t, cudaStream_t stream) {
  const int64_t with_rows = tree_workspace_fp4_bytes(t.total_rows, t.num_heads, t.batch, t.num_blocks, t.block_size);
  if (with_rows > tree_workspace_bytes() && t.workspace_bytes >= with_rows && t.max_blocks > 0) {
    TreeParams expanded = t;
    void* rows = static_cast<char*>(t.workspace) + expanded_at();
    expanded.cache = static_cast<const __nv_bfloat16*>(rows);
    const cudaError_t e = launch_tree_expand(t, rows, stream);
    return e != cudaSuccess ? e : launch_tree_attention(expanded, stream, true);
  }
  // Requests of up to 16 pairs, on average, have units of 16.  (Replayed graphs at 16 heads, units of 128 and of 16: 64 x 1
  // over 8192 189 and 110 us, over 2000 58 and 42, over 700 30 and 26; 1 x 1 over 8192 39 and 18, over 2000 22 and 15.
  // With few tiles for the SMs, where a call is its start and its end, units of 16 lose: 1 x 1 over 64 11.6 and 13.8, over
  // 700 15.1 and 15.5; 16 x 1 over 64 12.8 and 14.7, over 700 19.0 and 22.1, over 2000 25.6 and 24.6; 64 x 1 over 64 and 300
  // even.  The lengths are on the device, and a table is as wide as the longest request that a server allows, so that the
  // rule goes by pairs alone: 3 us lost at most, up to 79 won.  Units of 32 for 64 x 1 over 8192 at 32 heads: 197, of 128
  // 202 at that time; 8 x 1 over 20000 77 and 73.)
  if (pairs_of_a_request(t.total_rows, t.num_heads, t.batch) <= TREE_FEW) return launch_tree_attention_fp4_few(t, stream);
  const TreeLaunch p = tree_launch(t, max_workers());
  if (p.workers <= 0) return cudaErrorInvalidConfiguration;
  CUtensorMap tq;
  const uint64_t dims[3] = {64, (uint64_t)t.total_rows * (uint64_t)t.num_heads, NP}, strides[2] = {576 * 2, 64 * 2};
  const uint32_t box[3] = {64, 64, NP};   // 64 rows, panel by panel
  if (make_tensor_map_bf16(&tq, t.q, 3, dims, strides, box) != MLA_OK) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pair_config(attr, p.workers, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_attn_fp4_kernel, tq, p);
  return e != cudaSuccess ? e : launch_tree_join(p, stream);
}

}  // namespace mla
