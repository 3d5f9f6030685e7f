// What the two kernels of tree attention on tensor cores share (over a bf16 cache and over one of 4-bit
// entries): shared and tensor memory, barriers, the issue of the products and the softmax.  They differ in
// how a tile's keys come into shared memory.  Each includes this once, in its own anonymous namespace.
#pragma once
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"
#include "tmem_wide.cuh"
#include "tree_attn.cuh"

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

__device__ __forceinline__ void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// ------------------------------------------------------------------ products (even CTA, warp 1)
// The whole warp runs the issue loop and one elected lane (always the same) issues, with every
// operand in a register that the compiler knows to be the same in all lanes (values from memory
// are broadcast by a shuffle first).  With a branch for lane 0 around the loop, or operands that
// may differ by lane, a product took 50-70 clocks to issue; this way an M = 128, N = 128 product
// of the pair takes 32 and an N = 256 one 64, the tensor cores' own rate.  Descriptors are
// passed as low and high words: only the low one moves.
__device__ __forceinline__ void issue(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %4};\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}\n" ::"r"(d),
      "r"((uint32_t)a), "r"((uint32_t)b), "r"((uint32_t)(a >> 32)), "r"((uint32_t)(b >> 32)), "r"(idesc),
      "r"(accumulate)
      : "memory");
}
// Arrive on `bar` of both CTAs once the elected lane's products so far have completed.
__device__ __forceinline__ void commit_both(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}\n" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// R: rows of a box (tree_attn_kernel), or FP4 (tree_attn_fp4_kernel): K's groups are then two of four panels and
// the rope's panel.
constexpr int FP4 = 4;
template <int R>
__device__ void run_mma(const Ctx& c, const TreeLaunch& p, Parts parts, uint32_t tmem) {
  const uint64_t q_desc = sdesc_sw128(c.sbase + OFF_Q, 16, 1024);
  // A group of K lies in panels of 64 rows, or eight rows at a time with their three panels.
  constexpr bool rows8 = R == 8 || R == 16 || R == 32;
  constexpr uint32_t K_PANEL = rows8 ? 1024 : QP;
  const uint64_t k_desc = sdesc_sw128(c.sbase + OFF_K, 16, rows8 ? K_ROWS8 : 1024);
  // Values lie in pieces of r keys, each with its four panels: 16 keys of a product are part of one
  // piece, a whole one or two.
  constexpr int r = rows8 ? R : 64;
  constexpr int GP = R == FP4 ? 4 : 3;   // panels of a group of K
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
      for (int i = 0; i < GP && GP * g + i < NP; ++i) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t qo = (uint32_t)((GP * g + i) * QP + kk * 32) >> 4, ko = (uint32_t)(GP * g * QP + i * K_PANEL + kk * 32) >> 4;
          issue(d, q_desc + qo, k_desc + ko, IDESC_QK, kk > 0 ? 1u : g + i > 0 ? 1u : 0u);
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
          issue(tmem + TM_O(ch), p_desc + po, v_desc + vo, IDESC_PV, kk > 0 ? 1u : i ? 1u : more);
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
      // c * tanh(y) in log2 units, y = x / c with the logit x.  For |y| < 1/4 x times the series of tanh(y) / y,
      // whose next term is 2^-21; from there on c (1 - 2 / (e^(2y) + 1)), which is good to 2^-22 of c and so to
      // 2^-20 of the result, where below it would lose the logit's low bits (all of them under a large cap).
      // Most logits are far below their cap, so the second is worked out only for the 16 keys of a warp's rows
      // in which some logit needs it.  (9 x up to 37 nodes under a cap of 30: 40.6 us, 39.4 with the second form
      // alone; both for all keys and a choice: 41.2; tanh(y) / y as a quotient of polynomials: 41.0.)
      if (p.has_cap) {
        const float2 inv2 = make_float2(p.cap_inv, p.cap_inv), scale2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 e2 = make_float2(2.8853900817779268f, 2.8853900817779268f), one = make_float2(1.f, 1.f);
        const float2 cap2 = make_float2(p.cap_log2, p.cap_log2), m2c = make_float2(-2.f * p.cap_log2, -2.f * p.cap_log2);
        const float2 s1 = make_float2(-1.f / 3.f, -1.f / 3.f), s2 = make_float2(2.f / 15.f, 2.f / 15.f);
        const float2 s3 = make_float2(-17.f / 315.f, -17.f / 315.f);
#pragma unroll
        for (int j = 0; j < 64; j += 16) {
          float2 y[8], r[8];
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 x = make_float2(sv[j + 2 * k], sv[j + 2 * k + 1]);
            y[k] = fmul2(x, inv2);
            const float2 z = fmul2(y[k], y[k]);
            r[k] = fmul2(fmul2(x, scale2), ffma2(z, ffma2(z, ffma2(z, s3, s2), s1), one));
            top = fmax3(top, z.x, z.y);   // (passes over a NaN, which r has)
          }
          if (__any_sync(0xffffffffu, top >= 0.0625f)) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float2 a = fmul2(y[k], e2);
              const float2 d = fadd2(make_float2(ex2_approx(a.x), ex2_approx(a.y)), one);
              const float2 far = ffma2(make_float2(rcp_approx(d.x), rcp_approx(d.y)), m2c, cap2);
              if (fabsf(y[k].x) >= 0.25f) r[k].x = far.x;
              if (fabsf(y[k].y) >= 0.25f) r[k].y = far.y;
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            sv[j + 2 * k] = r[k].x;
            sv[j + 2 * k + 1] = r[k].y;
          }
        }
      }
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

}  // namespace
}  // namespace mla
