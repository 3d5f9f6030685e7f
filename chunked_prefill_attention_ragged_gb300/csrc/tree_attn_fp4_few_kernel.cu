// Tree attention over a cache of 4-bit entries for few (node, head) pairs a request: a decoding step of one
// token and up to 16 or 32 heads.
//
// The 128 x 128 products of tree_attn_fp4_kernel make every key bf16 twice, in two CTAs, and are mostly
// padding when a request has 16 pairs.  Here one CTA has a unit of N = 16 or 32 pairs and the transposed
// products: with a tile of 64 keys C (64 x 576) made bf16 once in shared memory,
//   S^T = C Q^T             (M = 64 keys, N pairs, K = 576)
//   O^T += C[:, :512]^T P^T  (M = 128 columns four times, N pairs, K = 64 keys),
// the same panels read K-major and MN-major.  The softmax over keys goes across lanes: a thread has a key and
// every pair.  The reference m of the exponentials moves only when some score passes it by 2^8 (and at a
// part's first tile), so that the usual tile needs one vote and no maxima.
//
// Tiles are shared out among the SMs as in tree_attn_kernel.cu (equal pieces of the line of all tiles, parts
// joined by a second kernel).  Two tile buffers: one is made while the other is multiplied.
//   warp 0  Q producer    1  issues the products    2  brings rows to come into L2    3  TMEM; ropes
//   warps 4-7  softmax and output    8-15  codes to bf16: eight rows each
// Where P V's accumulator lies: columns 128 i .. of the latent in TMEM columns N i .., lane = column.
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "tmem_wide.cuh"
#include "tree_attn.cuh"

namespace mla {
namespace {

constexpr int KEYS = 64;
constexpr int NTHREADS = 512;
constexpr int LAUNCH_REGS = 128;
constexpr int REGS_CTRL = 96, REGS_SOFTMAX = 208, REGS_ROWS = 104;
static_assert(REGS_CTRL + REGS_SOFTMAX + 2 * REGS_ROWS <= 4 * LAUNCH_REGS, "register split exceeds the launch allocation");
constexpr int PANEL = KEYS * 128;        // 64 keys x 64 columns
constexpr int TILE = 9 * PANEL;
constexpr int AHEAD = 4;                 // tiles between the one being made and the one brought into L2
constexpr uint32_t TMEM_COLS = 256;

template <int N>
struct Off {
  static constexpr int TILES = 0, Q = 2 * TILE, P = Q + 9 * N * 128, FLAG = P + 2 * N * 128;
  static constexpr int MAXIMA = FLAG + 2 * 4 * 4, SUMS = MAXIMA + 4 * N * 4, BAR = SUMS + 4 * N * 4;
  static constexpr int MISC = BAR + 16 * 8, SMEM = MISC + 64 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};
enum Bar {
  QF = 0,       // Q landed
  QE,           // the part's last S done: Q may be replaced
  CF,           // [buffer][half] panels 0-3, panels 4-8 made
  TE = CF + 4,  // [buffer] P V done: the tile, P's buffer and, for the next rescale, O are free
  SF = TE + 2,  // [buffer] S done
  PR = SF + 2,  // [buffer] P written (and the S buffer read) by the four softmax warps
  XB = PR + 2,  // exchange among them
  FIN,          // every product drained
  NEVER,        // nothing arrives here: the time-out test mode waits on it
  NBAR
};
static_assert(NBAR <= 16, "barriers");

template <int R>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

template <int N>
struct Ctx {
  uint32_t sbase;
  volatile int* abort_flag;
  int* status;
  uint64_t wait_limit_ns;
  __device__ uint32_t bar(int i) const { return sbase + Off<N>::BAR + 8 * i; }
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
template <int N>
using PartsN = PartsOf<N, KEYS>;

__device__ __forceinline__ uint4 load16(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Bytes of a word above 252 (in their top bits).
__device__ __forceinline__ uint32_t above252(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x03030303u) & w & 0x80808080u; }

// A warp's part of what it writes is there: handed to the products' proxy.
template <int N>
__device__ __forceinline__ void tell(const Ctx<N>& c, int b, int lane) {
  fence_async_shared();
  __syncwarp();
  if (lane == 0) mbar_arrive(c.bar(b));
}

// Four groups of 32 values of a row piece (see tree_attn_fp4_kernel.cu: one product by 2^126 times the scale,
// or two where the scales are `big`).
__device__ __forceinline__ void put_group(const uint32_t* at, uint32_t flip, uint32_t more, const uint4& w, bool big, uint32_t m,
                                          uint32_t m2) {
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  uint32_t r[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    fp4_fields(words[i], r[i]);
#pragma unroll
    for (int k = 0; k < 4; ++k) r[i][k] = mul_bf16x2(r[i][k], m);
  }
  if (big) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) r[i][k] = mul_bf16x2(r[i][k], m2);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) st_shared_v4((at[i] ^ flip) + more, r[i][0], r[i][1], r[i][2], r[i][3]);
}

// Warps 8-15.  Lane (panel % 4, row % 4, half) = (l / 8, l / 2 % 4, l % 2); piece j: row 4 (j % 2) + row % 4 of
// the warp's eight, panel 4 (j / 2) + panel % 4.  The bytes of the tile after next are loaded when a tile is done.
struct Pieces {
  uint4 code[4];
  uint32_t scale[4];
};
template <int N>
__device__ void run_rows(const Ctx<N>& c, const TreeLaunch& p, PartsN<N> parts, volatile int* begun) {
  const int lane = threadIdx.x & 31, w8 = (threadIdx.x >> 5) - 8, r4 = (lane >> 1) & 3;
  const int group = 2 * (lane >> 3) + (lane & 1);   // of the half's eight
  uint32_t at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    at[i] = c.sbase + Off<N>::TILES + (lane >> 3) * PANEL + (8 * w8 + r4) * 128 + (((4 * (lane & 1) + i) ^ r4) << 4);
  const uint8_t* cache = reinterpret_cast<const uint8_t*>(p.t.cache);
  int g = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    const int64_t end = min((int64_t)u.hi * KEYS, (int64_t)u.q.kv);
    auto find = [&](int64_t key) {
      return key < end ? __ldg(p.t.block_table + (int64_t)u.r * p.t.max_blocks + block_of(p, (int)key)) : 0;
    };
    auto get = [&](int32_t blk, int64_t key, Pieces* to) {
      const int32_t mine = key < end ? block_row(p, blk == PAST_END ? -1 : blk, key) : p.oob_row;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t row = __shfl_sync(0xffffffffu, mine, 4 * (j & 1) + r4);
        to->code[j] = make_uint4(0, 0, 0, 0);
        to->scale[j] = 0;
        if (row != p.oob_row) {
          const uint8_t* e = cache + (int64_t)row * FP4_ENTRY;
          to->code[j] = load16(e + 128 * (j >> 1) + 16 * group);
          to->scale[j] = __ldg(e + FP4_SCALES + 8 * (j >> 1) + group);
        }
      }
    };
    int64_t key = (int64_t)u.lo * KEYS + 8 * w8 + (lane & 7);   // the row that this lane looks up
    Pieces now, next;
    get(find(key), key, &now);
    get(find(key + KEYS), key + KEYS, &next);
    int32_t blk = find(key + 2 * KEYS);
#pragma unroll 1
    for (int t = u.lo; t < u.hi; ++t, ++g) {
      if (w8 == 0 && lane == 0) *begun = g;
      __syncwarp();
      const int b = g & 1;
      if (g > 1 && !c.wait_warp(TE + b, ((g >> 1) - 1) & 1)) {
        ok = false;
        break;
      }
      const uint32_t most = max(max(now.scale[0], now.scale[1]), max(now.scale[2], now.scale[3]));
      const bool big = __any_sync(0xffffffffu, most > 128);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t s = now.scale[j];
        uint32_t m = big ? 0x7e80u : (s + 126) << 7;   // 2^126 times the scale, or one after the other
        if (s > FP4_MAX_SCALE) m = 0;                  // values of a row that is NaN are zeros
        put_group(at, (j & 1) << 6, b * TILE + (j >> 1) * 4 * PANEL + (j & 1) * 512, now.code[j], big, m | m << 16,
                  scale_bf16x2(s > FP4_MAX_SCALE ? 0 : s));
        if (j & 1) tell(c, CF + 2 * b + (j >> 1), lane);
      }
      now = next;
      get(blk, key + 2 * KEYS, &next);
      key += KEYS;
      blk = find(key + 2 * KEYS);
    }
  }
}

// Warp 3: the ropes, a tile's last panel.  Lane i has 16 bytes of rows 4 j + i / 8; a row with a scale byte
// above 252 gets NaN.
template <int N>
__device__ void run_ropes(const Ctx<N>& c, const TreeLaunch& p, PartsN<N> parts) {
  const int lane = threadIdx.x & 31, ch = lane & 7;
  const uint8_t* cache = reinterpret_cast<const uint8_t*>(p.t.cache);
  int g = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    int64_t key0 = (int64_t)u.lo * KEYS;
    KeyBlocks blocks = find_blocks(p, u, key0, lane);
#pragma unroll 1
    for (int t = u.lo; t < u.hi; ++t, ++g, key0 += KEYS) {
      const int b = g & 1;
      const uint32_t dst = c.sbase + Off<N>::TILES + b * TILE + 8 * PANEL;
      const KeyRows k = find_rows(p, blocks, key0, lane);
      if (t + 1 < u.hi) blocks = find_blocks(p, u, key0 + KEYS, lane);
      uint32_t bad[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 s = make_uint4(0, 0, 0, 0);
        if (k.r[i] != p.oob_row) s = load16(cache + (int64_t)k.r[i] * FP4_ENTRY + FP4_SCALES);
        bad[i] = __ballot_sync(0xffffffffu, (above252(s.x) | above252(s.y) | above252(s.z) | above252(s.w)) != 0);
      }
      if (g > 1 && !c.wait_warp(TE + b, ((g >> 1) - 1) & 1)) {
        ok = false;
        break;
      }
#pragma unroll 4
      for (int j = 0; j < 16; ++j) {
        const int key = 4 * j + (lane >> 3);
        const int32_t row = __shfl_sync(0xffffffffu, j < 8 ? k.r[0] : k.r[1], key & 31);
        const bool there = row != p.oob_row;
        const uint8_t* src = there ? cache + (int64_t)row * FP4_ENTRY + FP4_ROPE + ch * 16 : reinterpret_cast<const uint8_t*>(p.t.q);
        cp_async16(dst + key * 128 + ((ch ^ (key & 7)) << 4), src, there ? 16 : 0);
      }
      cp_async_commit();
      cp_async_wait<0>();
      if (bad[0] | bad[1]) {
        __syncwarp();   // (a row's pieces are other lanes' copies)
        for (int j = 0; j < 16; ++j) {
          const int key = 4 * j + (lane >> 3);
          if ((bad[j >> 3] >> (key & 31)) & 1)
            st_shared_v4(dst + key * 128 + ch * 16, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        }
      }
      tell(c, CF + 2 * b + 1, lane);
    }
  }
}

template <int N>
__device__ void run_queries(const Ctx<N>& c, PartsN<N> parts, const CUtensorMap* tq) {
  const int lane = threadIdx.x & 31;
  int units = 0;
  bool ok = true;
  Part u;
  while (ok && parts.next(&u)) {
    if (lane == 0) {
      if (units > 0) ok = c.wait(QE, (units - 1) & 1);
      if (ok) {
        mbar_arrive_expect_tx(c.bar(QF), 9 * N * 128);
        tma_load_3d(c.sbase + Off<N>::Q, tq, c.bar(QF), 0, (int32_t)u.pair0, 0);
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok) ++units;
  }
  if (lane == 0 && units) c.drain(QF, (units - 1) & 1);   // (the copy lands before the CTA exits)
}

// Warp 2: keys of the tiles to come into L2, a lane an entry; it follows the rows' count and gives up quietly.
template <int N>
__device__ void run_prefetch(const Ctx<N>& c, const TreeLaunch& p, PartsN<N> parts, const volatile int* begun) {
  const int lane = threadIdx.x & 31;
  int g = 0;
  Part u;
  while (parts.next(&u)) {
    for (int t = u.lo; t < u.hi; ++t, ++g) {
      const uint64_t t0 = global_timer_ns();
      while (*begun < g) {
        __nanosleep(100);
        if (*c.abort_flag || global_timer_ns() - t0 > p.wait_limit_ns) return;
      }
      __syncwarp();
      // (a part's first tiles, beyond those that the rows' warps load themselves, all at once)
      for (int a = t == u.lo ? 2 : AHEAD; a <= AHEAD; ++a) {
        if (t + a >= u.hi) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t key = (int64_t)(t + a) * KEYS + 32 * i + lane;
          if (key < u.q.kv) {
            const int32_t row = block_row(p, table_block(p, u, key), key);
            const uint8_t* e = reinterpret_cast<const uint8_t*>(p.t.cache) + (int64_t)row * FP4_ENTRY;
            if (row != p.oob_row) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(e), "r"(FP4_ENTRY) : "memory");
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ products (warp 1)
// (see tree_core.cuh: a converged warp, one elected lane, operands the same in all lanes)
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

template <int N>
__device__ void run_mma(const Ctx<N>& c, const TreeLaunch& p, PartsN<N> parts, uint32_t tmem) {
  constexpr uint32_t IDESC_S = idesc_bf16_f32(KEYS, N, false, false), IDESC_O = idesc_bf16_f32(128, N, true, false);
  const uint64_t k_desc = sdesc_sw128(c.sbase + Off<N>::TILES, 16, 1024);
  const uint64_t v_desc = sdesc_sw128(c.sbase + Off<N>::TILES, PANEL, 1024);
  const uint64_t q_desc = sdesc_sw128(c.sbase + Off<N>::Q, 16, 1024);
  const uint64_t p_desc = sdesc_sw128(c.sbase + Off<N>::P, 16, 1024);
  bool ok = true;
  if (p.force_timeout) ok = c.wait_warp(NEVER, 0);
  int st = 0, pv = 0, units = 0;
  auto s_products = [&](bool last) {
    const int b = st & 1;
    const uint32_t d = __shfl_sync(0xffffffffu, tmem + 4 * N + b * N, 0), phase = (st >> 1) & 1;
    const uint32_t tile = __shfl_sync(0xffffffffu, (uint32_t)(b * TILE) >> 4, 0);
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      if (!c.wait_warp(CF + 2 * b + h, phase)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int i = 4 * h; i < (h ? 9 : 4); ++i) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          issue(d, k_desc + tile + ((uint32_t)(i * PANEL + kk * 32) >> 4), q_desc + ((uint32_t)(i * N * 128 + kk * 32) >> 4),
                IDESC_S, kk > 0 ? 1u : i > 0 ? 1u : 0u);
      }
    }
    commit(c.bar(SF + b));
    if (last) commit(c.bar(QE));
    ++st;
    return true;
  };
  auto pv_products = [&](uint32_t add, int keys) {
    const int b = pv & 1;
    const uint32_t more = __shfl_sync(0xffffffffu, add, 0);
    const uint32_t tile = __shfl_sync(0xffffffffu, (uint32_t)(b * TILE) >> 4, 0), pb = __shfl_sync(0xffffffffu, (uint32_t)(b * N * 128) >> 4, 0);
    if (!c.wait_warp(PR + b, (pv >> 1) & 1)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk > 0 && 16 * kk >= keys) break;
        issue(tmem + i * N, v_desc + tile + ((uint32_t)(2 * i * PANEL + kk * 2048) >> 4), p_desc + pb + ((uint32_t)(kk * 32) >> 4),
              IDESC_O, kk > 0 ? 1u : more);
      }
    }
    commit(c.bar(TE + b));
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
      if (ok && t > 0) ok = pv_products(t > 1 ? 1u : 0u, KEYS);
    }
    const int keys = __shfl_sync(0xffffffffu, (int)min((int64_t)KEYS, u.q.kv - (int64_t)(u.hi - 1) * KEYS), 0);
    if (ok) ok = pv_products(n > 1 ? 1u : 0u, keys);
  }
  commit(c.bar(FIN));
  c.drain(FIN, 0);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax (warps 4-7)
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t at, float* x);
template <>
__device__ __forceinline__ void tmem_load<32>(uint32_t at, float* x) {
  tmem_ld32_sync(at, reinterpret_cast<uint32_t*>(x));
}
template <>
__device__ __forceinline__ void tmem_load<16>(uint32_t at, float* x) {
  tmem_ld16_sync(at, reinterpret_cast<uint32_t*>(x));
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t at, const float* x) {
  if constexpr (N == 32) tmem_st32_sync(at, reinterpret_cast<const uint32_t*>(x));
  else tmem_st16_sync(at, reinterpret_cast<const uint32_t*>(x));
}
__device__ __forceinline__ float warp_max(float x) {   // (passes over a NaN)
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// c * tanh(x / c) in log2 units; as in run_softmax of tree_core.cuh (there is why).
__device__ __forceinline__ float capped(const TreeLaunch& p, float x) {
  const float y = x * p.cap_inv, z = y * y;
  float r = x * p.scale_log2 * fmaf(z, fmaf(z, fmaf(z, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  if (fabsf(y) >= 0.25f) r = fmaf(rcp_approx(ex2_approx(y * 2.8853900817779268f) + 1.f), -2.f * p.cap_log2, p.cap_log2);
  return r;
}

template <int N>
__device__ void run_softmax(const Ctx<N>& c, const TreeLaunch& p, PartsN<N> parts, uint32_t tmem, char* ws_slots, uint8_t* smem) {
  const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3;
  // M = 64: rows 16 q4 .. of S^T lie in lanes 0-15 of this warp's quarter of TMEM.
  const bool mine = lane < 16;
  const int row = 16 * q4 + (lane & 15);
  const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16);
  volatile int* flags = reinterpret_cast<volatile int*>(smem + Off<N>::FLAG);
  volatile float* maxima = reinterpret_cast<volatile float*>(smem + Off<N>::MAXIMA);
  volatile float* sums = reinterpret_cast<volatile float*>(smem + Off<N>::SUMS);
  const uint32_t p_at = c.sbase + Off<N>::P + (row & 7) * 2;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const float sc = p.has_cap ? 1.f : p.scale_log2;
  bool ok = true;
  int g = 0, xs = 0;   // tiles and exchanges so far
  auto meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar(XB));
    return c.wait_warp(XB, xs++ & 1);
  };
  Part u;
  while (ok && parts.next(&u)) {
    float m[N], l[N];   // m: the same in every thread
#pragma unroll
    for (int i = 0; i < N; ++i) {
      m[i] = NEG_INF;
      l[i] = 0.f;
    }
    const int64_t first = u.pair0 - (int64_t)u.q.q0 * p.t.num_heads;   // the unit's first pair in its request
    for (int t = u.lo; t < u.hi; ++t, ++g) {
      const int b = g & 1;
      if (!c.wait_warp(SF + b, (g >> 1) & 1)) { ok = false; break; }
      tc_fence_after();
      float s[N];
      tmem_load<N>(lane_addr + 4 * N + b * N, s);
      if (p.has_cap) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = capped(p, s[i]);
      }
      const int64_t pos = (int64_t)t * KEYS + row;
      if ((int64_t)t * KEYS + KEYS > min(u.q.ctx, (int64_t)u.q.kv)) {   // nodes, or the end of the keys
        const int64_t j = pos - u.q.ctx;   // node index of the key
#pragma unroll
        for (int i = 0; i < N; ++i) {
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
      bool over = false;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[i] = mine ? s[i] * sc : NEG_INF;
        over |= s[i] > m[i] + TREE_RESCALE_THRESHOLD;
      }
      const bool begin = t == u.lo;
      over = __any_sync(0xffffffffu, over);
      if (lane == 0) flags[(xs & 1) * 4 + q4] = over;
      const int x = xs & 1;
      if (!meet()) { ok = false; break; }
      if (begin || (flags[4 * x] | flags[4 * x + 1] | flags[4 * x + 2] | flags[4 * x + 3])) {
        // Maxima move: of every pair over the tile's keys.
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float v = warp_max(s[i]);
          if (lane == 0) maxima[q4 * N + i] = v;
        }
        if (!meet()) { ok = false; break; }
        // O is rescaled behind the last product into it.
        if (!begin && !c.wait_warp(TE + (b ^ 1), ((g - 1) >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        float alpha[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float top = fmaxf(fmaxf(maxima[i], maxima[N + i]), fmaxf(maxima[2 * N + i], maxima[3 * N + i]));
          const bool moves = begin || top > m[i] + TREE_RESCALE_THRESHOLD;
          alpha[i] = moves && !begin ? ex2_approx(m[i] - top) : 1.f;
          if (moves) m[i] = top;
          l[i] *= alpha[i];
        }
        if (!begin) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float o[N];
            tmem_load<N>(lane_addr + q * N, o);
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] *= alpha[i];
            tmem_store<N>(lane_addr + q * N, o);
          }
        }
      }
      // P's buffer was read by the tile before last's product.
      if (g > 1 && !c.wait_warp(TE + b, ((g >> 1) - 1) & 1)) { ok = false; break; }
#pragma unroll
      for (int i = 0; i < N; ++i) {
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
    if (!ok) break;
    // The part's end: the rows' sums, then O out of TMEM once the last product is done.
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      if (lane == 0) sums[q4 * N + i] = l[i];
    }
    if (!meet()) break;
    if (!c.wait_warp(TE + ((g - 1) & 1), ((g - 1) >> 1) & 1)) break;
    tc_fence_after();
    char* slot = ws_slots + (size_t)u.slot * few_slot_bytes(N);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      l[i] = (sums[i] + sums[N + i]) + (sums[2 * N + i] + sums[3 * N + i]);
      if (q4 == 0 && lane == i && i < u.npairs) {
        if (u.whole) {
          const bool empty = l[i] == 0.f;   // (a NaN is passed on)
          if (p.t.lse) p.t.lse[u.pair0 + i] = empty ? NEG_INF : (m[i] + log2f(l[i])) * 0.6931471805599453f;
        } else {
          reinterpret_cast<float2*>(slot + (size_t)N * 512 * 4)[i] = make_float2(m[i], l[i]);
        }
      }
      if (u.whole) l[i] = l[i] == 0.f ? 0.f : 1.f / l[i];
    }
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      float o[N];
      tmem_load<N>(lane_addr + q * N, o);
      const int col = 128 * q + 32 * q4 + lane;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i >= u.npairs) break;
        if (u.whole) p.t.o[(u.pair0 + i) * 512 + col] = __float2bfloat16_rn(l[i] == 0.f ? 0.f : o[i] * l[i]);
        else reinterpret_cast<float*>(slot)[i * 512 + col] = o[i];
      }
      __syncwarp();   // (the next load is one instruction of the whole warp)
    }
    tc_fence_before();   // O has been read: the next part's first P-ready lets it be overwritten
  }
}

template <int N>
__global__ void __launch_bounds__(NTHREADS, 1)
tree_attn_fp4_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ TreeLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ StartRec start;
  __shared__ int64_t count;
  __shared__ JoinRec join;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Off<N>::MISC);
  int* abort_flag = reinterpret_cast<int*>(smem + Off<N>::MISC + 4);
  int* begun = reinterpret_cast<int*>(smem + Off<N>::MISC + 8);   // tiles that the rows' first warp has begun, less one
  const int worker = blockIdx.x;
  const Ctx<N> c{smem_addr(smem), abort_flag, p.t.status, p.wait_limit_ns};
  ReqWords words{0, 0, 0};   // (on their way while the barriers are made)
  if ((int)threadIdx.x < p.t.batch) words = load_words(p.t, threadIdx.x);
  if (warp == 1) {
    // Codes: eight warps, ropes beside the second half; P and exchanges: four.
    const bool half0 = lane == CF || lane == CF + 2, half1 = lane == CF + 1 || lane == CF + 3;
    if (lane < NBAR) mbar_init(c.bar(lane), half0 ? 8 : half1 ? 9 : lane == PR || lane == PR + 1 || lane == XB ? 4 : 1);
    if (lane == 0) {
      *abort_flag = 0;
      *begun = -1;
    }
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
  const PartsN<N> parts(p.t, start, count);
  if (warp < 4) {
    setmaxnreg_dec<REGS_CTRL>();
    if (warp == 0) run_queries<N>(c, parts, &tm_q);
    else if (warp == 1) run_mma<N>(c, p, parts, tmem);
    else if (warp == 2) run_prefetch<N>(c, p, parts, begun);
    else run_ropes<N>(c, p, parts);
  } else if (warp < 8) {
    setmaxnreg_inc<REGS_SOFTMAX>();
    run_softmax<N>(c, p, parts, tmem, ws + WS_SLOTS + (size_t)worker * 2 * few_slot_bytes(N), smem);
  } else {
    setmaxnreg_dec<REGS_ROWS>();
    run_rows<N>(c, p, parts, begun);
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
template <int N>
int max_workers() {
  static PerDeviceOnce configured;
  static int workers[PerDeviceOnce::kMaxDevices] = {};
  const cudaError_t e = configured.run([] {
    cudaError_t r = cudaFuncSetAttribute(tree_attn_fp4_few_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Off<N>::SMEM);
    if (r != cudaSuccess) return r;
    // The split of the registers takes for granted that every thread starts with LAUNCH_REGS.
    cudaFuncAttributes attrs;
    r = cudaFuncGetAttributes(&attrs, tree_attn_fp4_few_kernel<N>);
    if (r != cudaSuccess) return r;
    if (attrs.numRegs != LAUNCH_REGS) return cudaErrorInvalidConfiguration;
    int dev = 0;
    r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    const int64_t room = (tree_workspace_bytes() - (int64_t)WS_SLOTS) / (int64_t)(2 * few_slot_bytes(N));
    workers[dev] = (int)std::min<int64_t>(device_sm_count(), std::min<int64_t>(room, MAX_WORKERS));
    return r;
  });
  int dev = 0;
  if (e != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) return 0;
  return workers[dev];
}

template <int N>
cudaError_t launch(const TreeParams& t, cudaStream_t stream) {
  const TreeLaunch p = tree_launch(t, max_workers<N>());
  if (p.workers <= 0) return cudaErrorInvalidConfiguration;
  CUtensorMap tq;
  const uint64_t dims[3] = {64, (uint64_t)t.total_rows * (uint64_t)t.num_heads, 9}, strides[2] = {576 * 2, 64 * 2};
  const uint32_t box[3] = {64, N, 9};   // N rows, panel by panel
  if (make_tensor_map_bf16(&tq, t.q, 3, dims, strides, box) != MLA_OK) return cudaErrorInvalidValue;
  tree_attn_fp4_few_kernel<N><<<p.workers, NTHREADS, Off<N>::SMEM, stream>>>(tq, p);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_tree_join_few(p, N, stream);
}

}  // namespace

cudaError_t launch_tree_attention_fp4_few(const TreeParams& t, int pairs, cudaStream_t stream) {
  return pairs <= 16 ? launch<16>(t, stream) : launch<32>(t, stream);
}

}  // namespace mla
