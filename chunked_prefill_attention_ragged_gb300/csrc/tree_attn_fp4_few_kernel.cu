// Tree attention over a cache of 4-bit entries for few (node, head) pairs a request: a decoding step of one
// token and up to 16 heads.
//
// The 128-pair units of tree_attn_fp4_kernel are mostly padding when a request has 16 pairs.  Here one CTA has a unit of
// N = 16 pairs and the transposed
// products: with a tile of 64 keys C (64 x 576) made bf16 once in shared memory,
//   S^T = C Q^T             (M = 64 keys, N pairs, K = 576)
//   O^T += C[:, :512]^T P^T  (M = 128 columns four times, N pairs, K = 64 keys),
// the same panels read K-major and MN-major.  The softmax over keys goes across lanes: a thread has a key and
// every pair.  The reference m of the exponentials moves only when some score passes it by 2^8 (and at a
// part's first tile), so that the usual tile needs one vote and no maxima.
//
// Tiles are shared out among the SMs as in tree_attn_kernel.cu (equal pieces of the line of all tiles, parts
// joined by a second kernel).  Two tile buffers: one is made while the other is multiplied.
//   warp 0  copies entries into a ring in shared memory     1  issues S    2  issues P V    3  TMEM; Q
//   warps 4-11  softmax and output    12-19  entries to bf16
// S and P V have a warp each: from one warp, which has to take them in a fixed order, P V waited for the next
// tile's keys or S for this tile's softmax (64 x 1 over 8192 at 16 heads: 184 us).
// Where P V's accumulator lies: columns 128 i .. of the latent in TMEM columns N i .., lane = column.
// What bounds it (64 x 1 over 8192 at 16 heads, 110 us in replayed graphs, 1.9 TB/s of entries; bf16 entries, 2.9 times the
// bytes, 107-109): 3640 clocks a tile, of
// which the warps that make keys work 3000; 277 KB pass through shared memory (entries in and out, keys in, and read by both
// products), 2160 clocks of it.  With a stage left out in turn the call takes: a quarter of the stores of keys 98 us, no loads
// of codes 101, no arithmetic on them 103, a quarter of S 106, of P V 109, no exponentials 111, entries from L2 111.
// Sixteen warps that make keys: 117 us; three tiles of 48 keys in flight and twelve such warps: 115; converting before the
// wait for the buffer: 126.  Calls of few tiles cost 16 us: Q and entries, a tile, the state and the join.
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "tmem_wide.cuh"
#include "tree_attn.cuh"
#include "tree_issue.cuh"

namespace mla {
namespace {

constexpr int N = TREE_FEW, KEYS = 64;   // pairs of a unit, keys of a tile
constexpr int NTHREADS = 640;
constexpr int PANEL = KEYS * 128;        // 64 keys x 64 columns
constexpr int TILE = 9 * PANEL;
constexpr int HALF = KEYS / 2 * FP4_ENTRY;   // half a tile's entries
constexpr uint32_t TMEM_COLS = 256;

struct Off {
  static constexpr int SLOTS = 2;   // of the ring, a tile's entries each
  static constexpr int TILES = 0, Q = 2 * TILE, P = Q + 9 * N * 128, RING = P + 2 * N * 128;
  static constexpr int MAXIMA = RING + SLOTS * KEYS * FP4_ENTRY, SUMS = MAXIMA + 4 * N * 4, BAR = SUMS + 4 * N * 4;
  static constexpr int THERE = BAR + 24 * 8, MISC = THERE + SLOTS * 8, SMEM = MISC + 64 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};
enum Bar {
  QF = 0,       // Q landed
  QE,           // the part's last S done: Q may be replaced
  CF,           // [buffer][half] panels 0-3, panels 4-8 made
  TE = CF + 4,  // [buffer] P V done: the tile, P's buffer and, for the next rescale, O are free
  SF = TE + 2,  // [buffer] S done
  PR = SF + 2,  // [buffer] P written (and the S buffer read) by the softmax warps
  EF = PR + 2,  // [slot] entries landed
  EE = EF + 2,  // [slot] entries read
  FIN = EE + 2, // [S, P V] every product drained
  NEVER = FIN + 2,   // nothing arrives here: the time-out test mode waits on it
  NBAR
};
static_assert(NBAR <= 24, "barriers");

struct Ctx {
  uint32_t sbase;
  volatile int* abort_flag;
  int* status;
  uint64_t wait_limit_ns;
  __device__ uint32_t bar(int i) const { return sbase + Off::BAR + 8 * i; }
  __device__ bool wait(int b, uint32_t parity) const {
    return mbar_wait_bounded(bar(b), parity, abort_flag, status, MLA_DEVSTAT_TIMEOUT, wait_limit_ns);
  }
  __device__ bool wait_warp(int b, uint32_t parity) const {
    return mla::wait_warp(bar(b), parity, abort_flag, status, wait_limit_ns);
  }
  __device__ void drain(int b, uint32_t parity) const {
    int dummy = 0;
    mbar_wait_bounded(bar(b), parity, &dummy, status, MLA_DEVSTAT_TIMEOUT, TREE_DRAIN_LIMIT_NS);
  }
};
using PartsN = PartsOf<N, KEYS>;

// A warp's part of what it writes is there: handed to the products' proxy.
__device__ __forceinline__ void tell(const Ctx& c, int b, int lane) {
  fence_async_shared();
  __syncwarp();
  if (lane == 0) mbar_arrive(c.bar(b));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Warp 0: half a tile's entries at a time, in runs of rows that lie side by side (`run`: as many of 32 as the
// block size is a multiple of, 8 at least, or 1), a lane a row.
__device__ void run_copies(const Ctx& c, const TreeLaunch& p, PartsN parts, uint8_t* smem) {
  constexpr int SLOTS = Off::SLOTS;
  const int lane = threadIdx.x & 31, bs = p.t.block_size;
  const int run = bs % 32 == 0 ? 32 : bs % 16 == 0 ? 16 : bs % 8 == 0 ? 8 : 1;
  volatile uint32_t* there = reinterpret_cast<volatile uint32_t*>(smem + Off::THERE);   // which rows exist
  const uint8_t* cache = reinterpret_cast<const uint8_t*>(p.t.cache);
  uint32_t put = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    const int64_t end = min((int64_t)u.hi * KEYS, (int64_t)u.q.kv);
    // A block as the table has it: looked at two steps later at the least, so that nothing waits for it here.
    auto find = [&](int64_t k) {
      return k < end ? __ldg(p.t.block_table + (int64_t)u.r * p.t.max_blocks + block_of(p, (int)k)) : 0;
    };
    int64_t key = (int64_t)u.lo * KEYS + lane;
    int32_t blk0 = find(key), blk1 = find(key + 32), blk2 = find(key + 64), blk3 = find(key + 96);
#pragma unroll 1
    for (int n = 0; n < 2 * (u.hi - u.lo); ++n, key += 32, ++put) {
      const int32_t row = key < end ? block_row(p, blk0 == PAST_END ? -1 : blk0, key) : p.oob_row;
      blk0 = blk1;
      blk1 = blk2;
      blk2 = blk3;
      blk3 = find(key + 128);
      const uint32_t have = __ballot_sync(0xffffffffu, row != p.oob_row);
      const uint32_t g = put >> 1, slot = g % SLOTS, half = 2 * slot + (put & 1), dst = c.sbase + Off::RING + half * HALF;
      if ((put & 1) == 0 && g >= SLOTS && !c.wait_warp(EE + slot, (g / SLOTS - 1) & 1)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        there[half] = have;
        if (have) mbar_arrive_expect_tx(c.bar(EF + slot), __popc(have) * FP4_ENTRY);
        else mbar_arrive(c.bar(EF + slot));
      }
      __syncwarp();
      const uint32_t mine = __popc((have >> lane) & (run == 32 ? 0xffffffffu : (1u << run) - 1));   // (the first of a run)
      if ((lane & (run - 1)) == 0 && (have >> lane & 1))
        bulk_load(dst + lane * FP4_ENTRY, cache + (int64_t)row * FP4_ENTRY, mine * FP4_ENTRY, c.bar(EF + slot));
      __syncwarp();
    }
  }
  // Let every copy started here land before the CTA can exit.
  // (A wait gives up between tiles only, with both halves of those before copied.)
  if (lane == 0)
    for (uint32_t n = put >> 1, g = n > SLOTS ? n - SLOTS : 0; g < n; ++g) c.drain(EF + g % SLOTS, (g / SLOTS) & 1);
}

// Warps 12-19: eight rows of a tile each, first panels 0-3, then 4-8, so that S begins with the first half.  A lane
// has two pieces of a half, a piece being 32 values (16 bytes of codes, one scale): lane (panel % 4, row % 4, half
// panel) = (l / 8, l / 2 % 4, l % 2), rows row % 4 and 4 + row % 4; eight lanes of a store have eight different
// bank groups.  And 16 bytes of two ropes, lane (row % 4, piece) = (l / 8, l % 8).
// The loop is kept short: with a tile's loads in registers a tile ahead, its code took three times as long beside
// the other warps' (it does not stay in the instruction cache).
__device__ void run_rows(const Ctx& c, const TreeLaunch& p, PartsN parts, uint8_t* smem) {
  constexpr int SLOTS = Off::SLOTS;
  const int lane = threadIdx.x & 31, w8 = (threadIdx.x >> 5) - 12, r4 = (lane >> 1) & 3, rr = lane >> 3;
  const int group = 2 * (lane >> 3) + (lane & 1);   // of a half's eight
  uint32_t at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    at[i] = c.sbase + Off::TILES + (lane >> 3) * PANEL + (8 * w8 + r4) * 128 + (((4 * (lane & 1) + i) ^ r4) << 4);
  const uint32_t rope_at = c.sbase + Off::TILES + 8 * PANEL + (8 * w8 + rr) * 128 + (((lane & 7) ^ rr) << 4);
  const uint32_t from = c.sbase + Off::RING + (8 * w8 + r4) * FP4_ENTRY;
  const uint32_t rope_from = c.sbase + Off::RING + (8 * w8 + rr) * FP4_ENTRY + FP4_ROPE + (lane & 7) * 16;
  const volatile uint8_t* there = smem + Off::THERE + w8;   // which of the warp's rows exist
  int g = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
#pragma unroll 1
    for (int t = u.lo; t < u.hi; ++t, ++g) {
      const int b = g & 1;
      const uint32_t slot = (uint32_t)g % SLOTS, e = from + slot * 2 * HALF;
      if (w8 == 0) ok = c.wait_warp(EF + slot, ((uint32_t)g / SLOTS) & 1) && (g < 2 || c.wait_warp(TE + b, ((g >> 1) - 1) & 1));
      if (meet<256>(3, !ok)) {
        ok = false;
        break;
      }
      // All of the tile's loads at once: their latency, under the other warps' stores, is a third of a half's time.
      uint4 code[2][2], rope[2];   // [half][row]
      uint32_t scale[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          code[k][h] = ld_shared_v4(e + h * 4 * FP4_ENTRY + 128 * k + 16 * group);
          scale[k][h] = ld_shared_u8(e + h * 4 * FP4_ENTRY + FP4_SCALES + 8 * k + group);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) rope[h] = ld_shared_v4(rope_from + slot * 2 * HALF + h * 4 * FP4_ENTRY);
      const uint32_t have = there[8 * slot];
      if (have != 255u) {   // rows that are not there are zeros
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!(have >> (4 * h + r4) & 1)) {
            code[0][h] = code[1][h] = make_uint4(0, 0, 0, 0);
            scale[0][h] = scale[1][h] = 0;
          }
          if (!(have >> (4 * h + rr) & 1)) rope[h] = make_uint4(0, 0, 0, 0);
        }
      }
      const uint32_t most[2] = {max(scale[0][0], scale[1][0]), max(scale[0][1], scale[1][1])};
      const bool big = __any_sync(0xffffffffu, max(most[0], most[1]) > 128);
      if (big) {   // a row with a scale byte above 252 is NaN: in its rope, while its values are zeros
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t nans = __ballot_sync(0xffffffffu, most[h] > FP4_MAX_SCALE);
          if (nans & (0x03030303u << (2 * rr))) rope[h] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) st_shared_v4((rope_at ^ (h << 6)) + b * TILE + h * 512, rope[h].x, rope[h].y, rope[h].z, rope[h].w);
      // (Every lane's loads have arrived: the codes', before the scales' that the vote needed, and the ropes'.)
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar(EE + slot));
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        const uint32_t to = b * TILE + k * 4 * PANEL;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // One product by 2^126 times the scale, or, where a scale is above 2, two.
          const uint32_t s = scale[0][h], words[4] = {code[0][h].x, code[0][h].y, code[0][h].z, code[0][h].w};
          uint32_t m = big ? 0x7e80u : (s + 126) << 7;
          if (big && s > FP4_MAX_SCALE) m = 0;
          m |= m << 16;
          uint32_t r[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            fp4_fields(words[i], r[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) r[i][q] = mul_bf16x2(r[i][q], m);
          }
          if (big) {
            const uint32_t m2 = scale_bf16x2(s > FP4_MAX_SCALE ? 0 : s);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q) r[i][q] = mul_bf16x2(r[i][q], m2);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) st_shared_v4((at[i] ^ (h << 6)) + to + h * 512, r[i][0], r[i][1], r[i][2], r[i][3]);
          code[0][h] = code[1][h];
          scale[0][h] = scale[1][h];
        }
        tell(c, CF + 2 * b + k, lane);
      }
    }
  }
}

// Warp 3: Q of each part.
__device__ void run_queries(const Ctx& c, PartsN parts, const CUtensorMap* tq) {
  const int lane = threadIdx.x & 31;
  int units = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    if (lane == 0) {
      if (units > 0) ok = c.wait(QE, (units - 1) & 1);
      if (ok) {
        mbar_arrive_expect_tx(c.bar(QF), 9 * N * 128);
        tma_load_3d(c.sbase + Off::Q, tq, c.bar(QF), 0, (int32_t)u.pair0, 0);
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok) ++units;
  }
  if (lane == 0 && units) c.drain(QF, (units - 1) & 1);   // (the copy lands before the CTA exits)
}

// ------------------------------------------------------------------ products (warps 1 and 2)
// (see issue_pair: a converged warp, one elected lane, operands the same in all lanes)
__device__ __forceinline__ void issue(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}\n" ::"r"(d),
      "r"((uint32_t)a), "r"((uint32_t)b), "r"((uint32_t)(a >> 32)), "r"((uint32_t)(b >> 32)), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar)
      : "memory");
}

__device__ void run_scores(const Ctx& c, const TreeLaunch& p, PartsN parts, uint32_t tmem) {
  constexpr uint32_t IDESC = idesc_bf16_f32(KEYS, N, false, false);
  const uint64_t k_desc = sdesc_sw128(c.sbase + Off::TILES, 16, 1024);
  const uint64_t q_desc = sdesc_sw128(c.sbase + Off::Q, 16, 1024);
  bool ok = true;
  if (p.force_timeout) ok = c.wait_warp(NEVER, 0);
  int g = 0, units = 0;
  Part u;
  while (ok && parts.next(&u)) {
    const int n = __shfl_sync(0xffffffffu, u.hi - u.lo, 0);
    ok = c.wait_warp(QF, units & 1);
    ++units;
    for (int t = 0; t < n && ok; ++t, ++g) {
      const int b = g & 1;
      const uint32_t d = __shfl_sync(0xffffffffu, tmem + 4 * N + b * N, 0);
      const uint32_t tile = __shfl_sync(0xffffffffu, (uint32_t)(b * TILE) >> 4, 0);
      // S's buffer: the scores of the tile before last were read before its P was ready, and its tile, which this one
      // replaced, was free after that.
#pragma unroll 1
      for (int i = 0; i < 9; ++i) {
        if ((i & 3) == 0 && i < 8) {
          if (!(ok = c.wait_warp(CF + 2 * b + (i >> 2), (g >> 1) & 1))) break;
          tc_fence_after();
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          issue(d, k_desc + tile + ((uint32_t)(i * PANEL + kk * 32) >> 4), q_desc + ((uint32_t)(i * N * 128 + kk * 32) >> 4),
                IDESC, kk > 0 ? 1u : i > 0 ? 1u : 0u);
      }
      if (!ok) break;
      commit(c.bar(SF + b));
      if (t == n - 1) commit(c.bar(QE));
    }
  }
  commit(c.bar(FIN));
  c.drain(FIN, 0);
  __syncwarp();
}

__device__ void run_values(const Ctx& c, PartsN parts, uint32_t tmem) {
  constexpr uint32_t IDESC = idesc_bf16_f32(128, N, true, false);
  const uint64_t v_desc = sdesc_sw128(c.sbase + Off::TILES, PANEL, 1024);
  const uint64_t p_desc = sdesc_sw128(c.sbase + Off::P, 16, 1024);
  bool ok = true;
  int g = 0;
  Part u;
  while (ok && parts.next(&u)) {
    const int n = __shfl_sync(0xffffffffu, u.hi - u.lo, 0);
    for (int t = 0; t < n; ++t, ++g) {
      const int b = g & 1;
      const uint32_t more = __shfl_sync(0xffffffffu, t > 0 ? 1u : 0u, 0);
      const uint32_t tile = __shfl_sync(0xffffffffu, (uint32_t)(b * TILE) >> 4, 0), pb = __shfl_sync(0xffffffffu, (uint32_t)(b * N * 128) >> 4, 0);
      // (P was made of S, and S of the tile: it is there)
      if (!(ok = c.wait_warp(PR + b, (g >> 1) & 1))) break;
      tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          issue(tmem + i * N, v_desc + tile + ((uint32_t)(2 * i * PANEL + kk * 2048) >> 4), p_desc + pb + ((uint32_t)(kk * 32) >> 4),
                IDESC, kk > 0 ? 1u : more);
      }
      commit(c.bar(TE + b));
    }
  }
  commit(c.bar(FIN + 1));
  c.drain(FIN + 1, 0);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax (warps 4-11)
__device__ __forceinline__ float warp_max(float x) {   // (passes over a NaN)
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// c * tanh(x / c) in log2 units; as cap_scores (there is why).
__device__ __forceinline__ float capped(const TreeLaunch& p, float x) {
  const float y = x * p.cap_inv, z = y * y;
  float r = x * p.scale_log2 * fmaf(z, fmaf(z, fmaf(z, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  if (fabsf(y) >= 0.25f) r = fmaf(rcp_approx(ex2_approx(y * 2.8853900817779268f) + 1.f), -2.f * p.cap_log2, p.cap_log2);
  return r;
}

// Half the pairs for each four warps.  These meet at barriers, which have no time limit, so where a wait gave up
// they go through the rest of their tiles without waiting: nobody is left alone at one.
__device__ void run_softmax(const Ctx& c, const TreeLaunch& p, PartsN parts, uint32_t tmem, char* ws_slots, uint8_t* smem) {
  constexpr int W = N / 2;   // pairs of a warp
  const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3, side = (threadIdx.x >> 7) - 1, i0 = side * W;
  const int barrier = 1 + side;
  // M = 64: rows 16 q4 .. of S^T lie in lanes 0-15 of this warp's quarter of TMEM.
  const bool mine = lane < 16;
  const int row = 16 * q4 + (lane & 15);
  const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16) + i0;
  volatile float* maxima = reinterpret_cast<volatile float*>(smem + Off::MAXIMA) + i0;
  volatile float* sums = reinterpret_cast<volatile float*>(smem + Off::SUMS) + i0;
  const uint32_t p_at = c.sbase + Off::P + i0 * 128 + (row & 7) * 2;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const float sc = p.has_cap ? 1.f : p.scale_log2;
  bool ok = true;
  int g = 0;   // tiles so far
  auto wait = [&](int b, uint32_t parity) { ok = ok && c.wait_warp(b, parity); };
  Part u;
  while (parts.next(&u)) {
    float m[W], l[W];   // m: the same in every thread
#pragma unroll
    for (int i = 0; i < W; ++i) {
      m[i] = NEG_INF;
      l[i] = 0.f;
    }
    const int64_t first = u.pair0 - (int64_t)u.q.q0 * p.t.num_heads + i0;   // this warp's first pair in its request
#pragma unroll 1
    for (int t = u.lo; t < u.hi; ++t, ++g) {
      const int b = g & 1;
      if (q4 == 0) wait(SF + b, (g >> 1) & 1);
      if (meet<128>(barrier, !ok)) ok = false;
      tc_fence_after();
      float s[W];
      tmem_ld8_sync(lane_addr + 4 * N + b * N, reinterpret_cast<uint32_t*>(s));
      if (p.has_cap) {
#pragma unroll
        for (int i = 0; i < W; ++i) s[i] = capped(p, s[i]);
      }
      const int64_t pos = (int64_t)t * KEYS + row;
      if ((int64_t)t * KEYS + KEYS > min(u.q.ctx, (int64_t)u.q.kv)) {   // nodes, or the end of the keys
        const int64_t j = pos - u.q.ctx;   // node index of the key
#pragma unroll
        for (int i = 0; i < W; ++i) {
          bool seen = pos < u.q.kv;
          if (seen && j >= 0) {
            // (a row without a pair computes on something harmless: the last node's mask)
            const int node = min((int)((first + i) / p.t.num_heads), u.q.nodes - 1);
            if (!p.t.mask) seen = j <= node;
            else seen = (j >> 6) < p.t.mask_words && ((uint64_t)__ldg(p.t.mask + ((int64_t)u.q.q0 + node) * p.t.mask_words + (j >> 6)) >> (j & 63)) & 1;
          }
          if (!seen) s[i] = NEG_INF;
        }
      }
      bool over = t == u.lo;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        s[i] = mine ? s[i] * sc : NEG_INF;
        over |= s[i] > m[i] + TREE_RESCALE_THRESHOLD;
      }
      if (meet<128>(barrier, over)) {
        // Maxima move: of every pair over the tile's keys.
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float v = warp_max(s[i]);
          if (lane == 0) maxima[q4 * N + i] = v;
        }
        meet<128>(barrier, false);
        const bool begin = t == u.lo;
        if (!begin) wait(TE + (b ^ 1), ((g - 1) >> 1) & 1);   // O is rescaled behind the last product into it
        tc_fence_after();
        float alpha[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float top = fmaxf(fmaxf(maxima[i], maxima[N + i]), fmaxf(maxima[2 * N + i], maxima[3 * N + i]));
          const bool moves = begin || top > m[i] + TREE_RESCALE_THRESHOLD;
          alpha[i] = moves && !begin ? ex2_approx(m[i] - top) : 1.f;
          if (moves) m[i] = top;
          l[i] *= alpha[i];
        }
        if (!begin) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float o[W];
            tmem_ld8_sync(lane_addr + q * N, reinterpret_cast<uint32_t*>(o));
#pragma unroll
            for (int i = 0; i < W; ++i) o[i] *= alpha[i];
            tmem_st8_sync(lane_addr + q * N, reinterpret_cast<const uint32_t*>(o));
          }
        }
      }
      // (P's buffer was read by the tile before last's product: this tile's rows waited for that.)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float e = ex2_approx(s[i] - (m[i] == NEG_INF ? 0.f : m[i]));
        l[i] += e;   // (of the unrounded weights; 0 in the lanes without a key)
        if (mine) {
          const uint32_t w = pack_bf16x2(e, 0.f);
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(p_at + (b * N + i) * 128 + (((row >> 3) ^ (i & 7)) << 4)), "h"((unsigned short)w) : "memory");
        }
      }
      fence_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar(PR + b));
    }
    // The part's end: the rows' sums, then O out of TMEM once the last product is done.
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      if (lane == 0) sums[q4 * N + i] = l[i];
    }
    meet<128>(barrier, false);
    wait(TE + ((g - 1) & 1), ((g - 1) >> 1) & 1);
    tc_fence_after();
    const int live = ok ? min(max(u.npairs - i0, 0), W) : 0;   // pairs to write
    char* slot = ws_slots + (size_t)u.slot * FEW_SLOT_BYTES;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      l[i] = (sums[i] + sums[N + i]) + (sums[2 * N + i] + sums[3 * N + i]);
      if (q4 == 0 && lane == i && i < live) {
        if (u.whole) {
          const bool empty = l[i] == 0.f;   // (a NaN is passed on)
          if (p.t.lse) p.t.lse[u.pair0 + i0 + i] = empty ? NEG_INF : (m[i] + log2f(l[i])) * 0.6931471805599453f;
        } else {
          reinterpret_cast<float2*>(slot + FEW_SLOT_ML)[i0 + i] = make_float2(m[i], l[i]);
        }
      }
      if (u.whole) l[i] = l[i] == 0.f ? 0.f : 1.f / l[i];
    }
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      float o[W];
      tmem_ld8_sync(lane_addr + q * N, reinterpret_cast<uint32_t*>(o));
      const int col = 128 * q + 32 * q4 + lane;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (i >= live) break;
        if (u.whole) p.t.o[(u.pair0 + i0 + i) * 512 + col] = __float2bfloat16_rn(l[i] == 0.f ? 0.f : o[i] * l[i]);
        else reinterpret_cast<float*>(slot)[(i0 + i) * 512 + col] = o[i];
      }
      __syncwarp();   // (the next load is one instruction of the whole warp)
    }
    tc_fence_before();   // O has been read: the next part's first P-ready lets it be overwritten
    meet<128>(barrier, false);   // (and the sums, before they are written again)
  }
}

__global__ void __launch_bounds__(NTHREADS, 1)
tree_attn_fp4_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ TreeLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ StartRec start;
  __shared__ int64_t count;
  __shared__ JoinRec join;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Off::MISC);
  int* abort_flag = reinterpret_cast<int*>(smem + Off::MISC + 4);
  const int worker = blockIdx.x;
  const Ctx c{smem_addr(smem), abort_flag, p.t.status, p.wait_limit_ns};
  ReqWords words{0, 0, 0};   // (on their way while the barriers are made)
  if ((int)threadIdx.x < p.t.batch) words = load_words(p.t, threadIdx.x);
  if (warp == 1) {
    // A half tile, entries read, P: eight warps; entries: both halves.
    const bool eight = (lane >= CF && lane < CF + 4) || lane == PR || lane == PR + 1 || lane == EE || lane == EE + 1;
    if (lane < NBAR) mbar_init(c.bar(lane), eight ? 8 : lane == EF || lane == EF + 1 ? 2 : 1);
    if (lane == 0) *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tm_q);
  if (warp == 3) {
    tmem_alloc(smem_addr(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  find_piece<NTHREADS, N, KEYS>(p.t, words, worker, p.workers, worker == 0, &start, &count, &join);
  tc_fence_after();   // (find_piece ends with a barrier of the whole CTA)
  char* ws = static_cast<char*>(p.t.workspace);
  if (threadIdx.x == 0) reinterpret_cast<JoinRec*>(ws)[worker] = join;
  __syncwarp();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const PartsN parts(p.t, start, count);
  if (warp < 4) {
    if (warp == 0) run_copies(c, p, parts, smem);
    else if (warp == 1) run_scores(c, p, parts, tmem);
    else if (warp == 2) run_values(c, parts, tmem);
    else run_queries(c, parts, &tm_q);
  } else if (warp < 12) {
    run_softmax(c, p, parts, tmem, ws + WS_SLOTS + (size_t)worker * 2 * FEW_SLOT_BYTES, smem);
  } else {
    run_rows(c, p, parts, smem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 3) {
    __syncwarp();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// CTAs that run at once on the current device (0 on error), no more than the workspace has room for.
int max_workers() {
  static PerDeviceOnce configured;
  static int workers[PerDeviceOnce::kMaxDevices] = {};
  const cudaError_t e = configured.run([] {
    cudaError_t r = cudaFuncSetAttribute(tree_attn_fp4_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Off::SMEM);
    if (r != cudaSuccess) return r;
    int dev = 0;
    r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    const int64_t room = (tree_workspace_bytes() - (int64_t)WS_SLOTS) / (int64_t)(2 * FEW_SLOT_BYTES);
    workers[dev] = (int)std::min<int64_t>(device_sm_count(), std::min<int64_t>(room, MAX_WORKERS));
    return r;
  });
  int dev = 0;
  if (e != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return 0;
  return workers[dev];
}

}  // namespace

cudaError_t launch_tree_attention_fp4_few(const TreeParams& t, cudaStream_t stream) {
  const TreeLaunch p = tree_launch(t, max_workers());
  if (p.workers <= 0) return cudaErrorInvalidConfiguration;
  CUtensorMap tq;
  const uint64_t dims[3] = {64, (uint64_t)t.total_rows * (uint64_t)t.num_heads, 9}, strides[2] = {576 * 2, 64 * 2};
  const uint32_t box[3] = {64, N, 9};   // N rows, panel by panel
  if (make_tensor_map_bf16(&tq, t.q, 3, dims, strides, box) != MLA_OK) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.workers);
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = Off::SMEM;
  cfg.stream = stream;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_attn_fp4_few_kernel, tq, p);
  return e != cudaSuccess ? e : launch_tree_join_few(p, stream);
}

}  // namespace mla
