// Tree attention for requests with few (node, head) pairs (at most 64): the same function as
// tree_attn_kernel.cu computes, turned round.  A unit is N = 16, 32 or 64 pairs of one request,
// run by one CTA over tiles of 64 keys:
//   S^T = K Q^T  (M = 64 keys, N pairs),  P^T = 2^(S^T - m),
//   O^T += V^T P^T  (M = 128 value columns, four times; N pairs).
//
// Why: with few pairs the call is bound by reading the cache from DRAM, and what counts is that
// every byte is read once and that enough copies are in flight.  The pairs are the products' narrow
// side, so that 16 of them cost what 16 cost, and the cache rows are their wide side, read by S
// and by P V from the same place in shared memory (the other kernel needs its V apart from K and
// pads to 128 pairs).  What shared memory is left over by Q holds two to three tiles.
//
// Shared memory is two rings: slots of two 64-column panels of 64 keys (four per tile, the values
// and the latent part of the keys) and slots of one (the rope columns).
//   warp 0     producer of both rings
//   warp 1     issues the products: P V(t) as soon as P(t) is there, S(t + 1) when its rows have
//              landed first (the results do not depend on the order)
//   warp 2     TMEM allocation
//   warp 3     loads Q, once per unit
//   warps 4-7  a key per lane of their lower halves (its N scores are one row of S^T, M = 64), a
//              value column per thread (of O)
// The maximum of a pair is over lanes and warps, which takes long to find.  So a tile only asks
// whether any score has passed m + 8 (one vote and one exchange of flags); if one has, all maxima
// are found, by shuffles and an exchange of rows, and O is scaled.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "tmem_wide.cuh"
#include "tree_attn.cuh"

namespace mla {
namespace {

constexpr int KEYS = 64;
constexpr int PANEL = 64 * 128;         // [64 keys, 64 columns]
constexpr int PAIR = 2 * PANEL;
constexpr int NTHREADS = 256;

template <int N>
struct Lay {
  static constexpr int PAIRS = N == 16 ? 11 : N == 32 ? 10 : 8;   // slots of two panels
  static constexpr int ROPES = N == 16 ? 3 : 2;
  static constexpr int PBUF = N == 64 ? 1 : 2;                    // P buffers
  static constexpr int OFF_PAIR = 0;
  static constexpr int OFF_ROPE = OFF_PAIR + PAIRS * PAIR;
  static constexpr int OFF_Q = OFF_ROPE + ROPES * PANEL;
  static constexpr int QPANEL = N * 128;
  static constexpr int OFF_P = OFF_Q + 9 * QPANEL;
  static constexpr int OFF_XCHG = OFF_P + PBUF * QPANEL;          // [4 warps][N] maxima or sums,
  static constexpr int OFF_FLAGS = OFF_XCHG + 4 * N * 4;          // [2][4 warps] flags,
  static constexpr int OFF_SCALE = OFF_FLAGS + 32;                // [N] what O is multiplied by
  static constexpr int OFF_BAR = OFF_SCALE + N * 4;
  // barriers
  static constexpr int QF = 0, QE = 1, SF = 2, PR = 4, OD = 6, XB = 8, FIN = 9, NEVER = 10;
  static constexpr int PF = 11, PE = PF + PAIRS, RF = PE + PAIRS, RE = RF + ROPES, NBAR = RE + ROPES;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 32 + 1024;               // + slack for 1024-byte alignment
  static_assert(SMEM + 256 <= 227 * 1024, "shared memory budget");
  static constexpr uint32_t TMEM = N == 16 ? 128 : N == 32 ? 256 : 512;
  static constexpr uint32_t TM_S = 4 * N;                         // two S^T buffers behind O^T's four tiles
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(64, N, false, false);
  static constexpr uint32_t IDESC_O = idesc_bf16_f32(128, N, true, false);
};

template <int N>
struct Ctx {
  uint32_t sbase;
  volatile int* abort_flag;
  int* status;
  uint64_t limit;
  __device__ uint32_t bar(int i) const { return sbase + Lay<N>::OFF_BAR + 8 * i; }
  __device__ bool wait(int b, uint32_t parity) const {
    return mbar_wait_bounded(bar(b), parity, abort_flag, status, MLA_DEVSTAT_TIMEOUT, limit);
  }
  __device__ bool wait_all(int b, uint32_t parity) const {
    return wait_warp(bar(b), parity, abort_flag, status, limit);
  }
  __device__ bool look(int b, uint32_t parity) const {
    return __any_sync(0xffffffffu, look_warp(bar(b), parity) != 0);
  }
  __device__ void drain(int b, uint32_t parity) const {
    int dummy = 0;
    mbar_wait_bounded(bar(b), parity, &dummy, status, MLA_DEVSTAT_TIMEOUT, TREE_DRAIN_LIMIT_NS);
  }
};

// A position in a ring of L slots, and the parity of its present use.
template <int L>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ void step() {
    if (++slot == L) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// ------------------------------------------------------------------ producers
__device__ __forceinline__ void copy_keys(const TreeLaunch& p, const KeyRows& k, uint32_t dst, uint32_t bar,
                                          const CUtensorMap* tc, const CUtensorMap* tb, int panel0, int n,
                                          int lane) {
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int col = (panel0 + i) * 64;
    if (k.by_block) {
      if (lane * p.piece_rows < 64) tma_load_2d(dst + i * PANEL + lane * p.piece_rows * 128, tb, bar, col, k.r[0]);
    } else if (lane < 16) {
      tma_gather4(dst + i * PANEL + lane * 4 * 128, tc, bar, col, k.r[0], k.r[1], k.r[2], k.r[3]);
    }
  }
}

template <int N>
__device__ void run_producer(const Ctx<N>& c, const TreeLaunch& p, Parts<N, KEYS> parts, const CUtensorMap* tc,
                             const CUtensorMap* tb, const CUtensorMap* t2) {
  using L = Lay<N>;
  const int lane = threadIdx.x & 31;
  Ring<L::PAIRS> pr;
  Ring<L::ROPES> rr;
  int pairs = 0, ropes = 0;   // slots filled so far
  bool ok = true;
  auto fill = [&](int full, int empty, int used_before, uint32_t phase, uint32_t bytes) {
    int go = 1;
    if (lane == 0) {
      if (used_before) go = c.wait(empty, phase ^ 1);
      if (go) mbar_arrive_expect_tx(c.bar(full), bytes);
    }
    return __shfl_sync(0xffffffffu, go, 0) != 0;
  };
  Part u;
  while (ok && parts.next(&u)) {
    int32_t ahead = 0;   // rows of 32 tiles
#pragma unroll 1
    for (int t = u.lo; t < u.hi && ok; ++t) {
      const int i = (t - u.lo) & 31;
      if (i == 0 && p.grouped) ahead = piece_rows(p, u, (int64_t)t * KEYS, KEYS, u.hi - t, lane);
      const int32_t row = __shfl_sync(0xffffffffu, ahead, i);
      if (p.grouped) {   // one lane, five copies
        if (lane == 0) {
          if (ropes >= L::ROPES) ok = c.wait(L::RE + rr.slot, rr.phase ^ 1);
          if (ok) {
            mbar_arrive_expect_tx(c.bar(L::RF + rr.slot), PANEL);
            tma_load_2d(c.sbase + L::OFF_ROPE + rr.slot * PANEL, tb, c.bar(L::RF + rr.slot), 8 * 64, row);
            ++ropes;
          }
        }
        rr.step();
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          if (lane == 0 && ok) {
            if (pairs >= L::PAIRS) ok = c.wait(L::PE + pr.slot, pr.phase ^ 1);
            if (ok) {
              mbar_arrive_expect_tx(c.bar(L::PF + pr.slot), PAIR);
              tma_load_3d(c.sbase + L::OFF_PAIR + pr.slot * PAIR, t2, c.bar(L::PF + pr.slot), 0, row, 2 * j);
              ++pairs;
            }
          }
          pr.step();
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        continue;
      }
      ropes = __shfl_sync(0xffffffffu, ropes, 0);
      pairs = __shfl_sync(0xffffffffu, pairs, 0);
      const int64_t key0 = (int64_t)t * KEYS;
      const KeyRows k = find_rows(p, u, find_blocks(p, u, key0, lane), key0, lane);
      ok = fill(L::RF + rr.slot, L::RE + rr.slot, ropes >= L::ROPES, rr.phase, PANEL);
      if (!ok) break;
      copy_keys(p, k, c.sbase + L::OFF_ROPE + rr.slot * PANEL, c.bar(L::RF + rr.slot), tc, tb, 8, 1, lane);
      ++ropes;
      rr.step();
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        ok = fill(L::PF + pr.slot, L::PE + pr.slot, pairs >= L::PAIRS, pr.phase, PAIR);
        if (!ok) break;
        copy_keys(p, k, c.sbase + L::OFF_PAIR + pr.slot * PAIR, c.bar(L::PF + pr.slot), tc, tb, 2 * j, 2, lane);
        ++pairs;
        pr.step();
      }
    }
  }
  // Let every copy started here land before the CTA can exit.
  if (lane == 0) {
    for (int i = pairs > L::PAIRS ? pairs - L::PAIRS : 0; i < pairs; ++i)
      c.drain(L::PF + i % L::PAIRS, (i / L::PAIRS) & 1);
    for (int i = ropes > L::ROPES ? ropes - L::ROPES : 0; i < ropes; ++i)
      c.drain(L::RF + i % L::ROPES, (i / L::ROPES) & 1);
  }
}

// One lane: the next unit's Q as soon as the products with this one's are done.
template <int N>
__device__ void run_q(const Ctx<N>& c, Parts<N, KEYS> parts, const CUtensorMap* tq) {
  using L = Lay<N>;
  int units = 0;
  Part u;
  while (parts.next(&u)) {
    if (units > 0 && !c.wait(L::QE, (units - 1) & 1)) break;
    mbar_arrive_expect_tx(c.bar(L::QF), 9 * L::QPANEL);
    for (int i = 0; i < 9; ++i)
      tma_load_2d(c.sbase + L::OFF_Q + i * L::QPANEL, tq, c.bar(L::QF), i * 64, (int32_t)u.pair0);
    ++units;
  }
  if (units) c.drain(L::QF, (units - 1) & 1);
}

// ------------------------------------------------------------------ products (warp 1)
// The whole warp runs the loop, one elected lane issues (see tree_attn_kernel.cu).
__device__ __forceinline__ void issue(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}\n" ::"r"(d),
      "r"((uint32_t)a), "r"((uint32_t)b), "r"((uint32_t)(a >> 32)), "r"((uint32_t)(b >> 32)), "r"(idesc),
      "r"(accumulate)
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
__device__ void run_mma(const Ctx<N>& c, const TreeLaunch& p, Parts<N, KEYS> parts, uint32_t tmem) {
  using L = Lay<N>;
  const uint64_t pair_k = sdesc_sw128(c.sbase + L::OFF_PAIR, 16, 1024);      // keys as rows
  const uint64_t pair_v = sdesc_sw128(c.sbase + L::OFF_PAIR, PANEL, 1024);   // value columns as rows
  const uint64_t rope_k = sdesc_sw128(c.sbase + L::OFF_ROPE, 16, 1024);
  const uint64_t q_desc = sdesc_sw128(c.sbase + L::OFF_Q, 16, 1024);
  const uint64_t p_desc = sdesc_sw128(c.sbase + L::OFF_P, 16, 1024);
  Ring<L::PAIRS> sp, vp;      // pair slots of the next S, of the next P V
  Ring<L::ROPES> sr;
  int s = 0, v = 0, units = 0;   // tiles of S and P V issued
  bool ok = true;
  if (p.force_timeout) ok = c.wait_all(L::NEVER, 0);
  // Whether tile s's rows have all landed: five looks at once, one vote.
  auto landed = [&]() {
    uint32_t r = look_warp(c.bar(L::RF + sr.slot), sr.phase);
    Ring<L::PAIRS> k = sp;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r &= look_warp(c.bar(L::PF + k.slot), k.phase);
      k.step();
    }
    return __any_sync(0xffffffffu, r != 0) != 0;
  };
  auto s_products = [&](bool last) {   // the rows are there
    __syncwarp();
    tc_fence_after();
    const uint32_t d = __shfl_sync(0xffffffffu, tmem + L::TM_S + (s & 1) * N, 0);
    {
      const uint64_t a = rope_k + (uint64_t)(__shfl_sync(0xffffffffu, sr.slot, 0) * PANEL >> 4);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        issue(d, a + (kk * 32 >> 4), q_desc + ((8 * L::QPANEL + kk * 32) >> 4), L::IDESC_S, kk > 0 ? 1u : 0u);
      commit(c.bar(L::RE + sr.slot));
      sr.step();
    }
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      const uint64_t a = pair_k + (uint64_t)(__shfl_sync(0xffffffffu, sp.slot, 0) * PAIR >> 4);
      const uint64_t b = q_desc + (uint64_t)(2 * j * L::QPANEL >> 4);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        issue(d, a + (((kk >> 2) * PANEL + (kk & 3) * 32) >> 4), b + (((kk >> 2) * L::QPANEL + (kk & 3) * 32) >> 4),
              L::IDESC_S, 1u);
      sp.step();
    }
    commit(c.bar(L::SF + (s & 1)));
    if (last) commit(c.bar(L::QE));
    ++s;
  };
  auto pv_products = [&](bool first) {   // P is there
    const uint32_t more = __shfl_sync(0xffffffffu, first ? 0u : 1u, 0);
    const uint64_t b = p_desc + (uint64_t)(__shfl_sync(0xffffffffu, v % L::PBUF, 0) * L::QPANEL >> 4);
    tc_fence_after();
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      const uint64_t a = pair_v + (uint64_t)(__shfl_sync(0xffffffffu, vp.slot, 0) * PAIR >> 4);
      const uint32_t d = tmem + j * N;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        issue(d, a + (kk * 16 * 128 >> 4), b + (kk * 32 >> 4), L::IDESC_O, kk > 0 ? 1u : more);
      commit(c.bar(L::PE + vp.slot));
      vp.step();
    }
    commit(c.bar(L::OD + (v & 1)));
    ++v;
  };
  Part u;
  while (ok && parts.next(&u)) {
    const int n = __shfl_sync(0xffffffffu, u.hi - u.lo, 0);
    const int end = s + n;
    int done = 0;   // P V's of this part
    ok = c.wait_all(L::QF, units & 1);
    ++units;
    while (ok && done < n) {
      // P V(v) when its P is there, else S(s), one tile ahead at most, when its rows are.
      const bool may_s = s < end && s - v < 2, may_pv = s > v;
      bool do_pv = false, do_s = false;
      uint64_t t0 = 0;
      for (uint32_t it = 0; !do_pv && !do_s && ok; ++it) {
        do_pv = may_pv && c.look(L::PR + (v & 1), (v >> 1) & 1);
        do_s = !do_pv && may_s && landed();
        if ((it & 63) == 63 && !do_pv && !do_s) {
          const uint64_t now = global_timer_ns();
          if (t0 == 0) t0 = now;
          const bool late = now - t0 > c.limit;
          if (__any_sync(0xffffffffu, late || *c.abort_flag)) {
            if (late) {
              *c.abort_flag = 1;
              if (c.status) atomicOr(c.status, MLA_DEVSTAT_TIMEOUT);
            }
            ok = false;
          }
        }
      }
      if (do_pv) {
        __syncwarp();
        pv_products(done == 0);
        ++done;
      } else if (do_s) {
        s_products(s + 1 == end);
      }
    }
  }
  commit(c.bar(L::FIN));
  c.drain(L::FIN, 0);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax (warps 4-7)
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t addr, uint32_t* r) {
  if constexpr (N == 64) tmem_ld64_sync(addr, r);
  else if constexpr (N == 32) tmem_ld32_sync(addr, r);
  else tmem_ld16_sync(addr, r);
}
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t addr, const uint32_t* r) {
  if constexpr (N == 64) tmem_st64_sync(addr, r);
  else if constexpr (N == 32) tmem_st32_sync(addr, r);
  else tmem_st16_sync(addr, r);
}

// v[n] reduced over the warp's lanes for every n, by halves: a lane ends with the rows
// lane * N / 32 .. (N = 64: two, 32: one; 16: lanes 2n and 2n + 1 both have row n).  Writes them to out[N].
template <int N, class Op>
__device__ __forceinline__ void reduce_rows(const float* in, float* out, int lane, Op op) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = in[i];
  int off = 16;
#pragma unroll
  for (int half = N / 2; half >= 1 && off >= 1; half /= 2, off /= 2) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
  if constexpr (N == 16) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
  if constexpr (N == 64) *reinterpret_cast<float2*>(out + 2 * lane) = make_float2(v[0], v[1]);
  else if constexpr (N == 32) out[lane] = v[0];
  else out[lane >> 1] = v[0];
}

// Which of the unit's pairs see the key at position pos: bit n for pair n.
template <int N>
__device__ __forceinline__ uint64_t seen_by(const TreeParams& p, const Part& u, int64_t first_pair, int64_t pos) {
  int node = (int)(first_pair / p.num_heads), rem = (int)(first_pair % p.num_heads);
  uint64_t bits = 0;
  bool seen = false;
#pragma unroll 1
  for (int n = 0, look = 1; n < N; ++n) {
    if (look && node < u.q.nodes) seen = visible(p, u, node, pos) & 1;
    if (seen) bits |= 1ull << n;
    look = ++rem == p.num_heads;
    if (look) {
      rem = 0;
      ++node;
    }
  }
  return bits;
}

template <int N>
__device__ void run_softmax(const Ctx<N>& c, const TreeLaunch& p, Parts<N, KEYS> parts, uint32_t tmem, char* ws_slots,
                            uint8_t* smem) {
  using L = Lay<N>;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
  const bool has_key = lane < 16;                    // S^T: 16 keys in each quarter of the lanes
  const int key = 16 * w + (lane & 15);              // of the tile
  const uint32_t lane_addr = tmem + ((uint32_t)(w * 32) << 16);
  float* rows = reinterpret_cast<float*>(smem + L::OFF_XCHG);              // [4][N]
  int* flags = reinterpret_cast<int*>(smem + L::OFF_FLAGS);                // [2][4]
  float* scale = reinterpret_cast<float*>(smem + L::OFF_SCALE);            // [N]
  const float NEG_INF = -__int_as_float(0x7f800000);
  // A pair that has seen no key yet: any finite score exceeds this reference, minus infinity does not.
  constexpr float FRESH = 1e30f;
  const float sc = p.has_cap ? 1.f : p.scale_log2;
  bool ok = true;
  int g = 0, xs = 0;   // tiles and exchanges so far
  // What every warp wrote before, to all four.
  auto exchange = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar(L::XB));
    const bool r = c.wait_all(L::XB, xs & 1);
    ++xs;
    return r;
  };
  Part u;
  while (ok && parts.next(&u)) {
    float neg_m[N], l[N];   // the reference's negative; the sum over this thread's keys
#pragma unroll
    for (int n = 0; n < N; ++n) {
      neg_m[n] = FRESH;
      l[n] = 0.f;
    }
    const int64_t first_pair = u.pair0 - (int64_t)u.q.q0 * p.t.num_heads;   // inside the request
    for (int t = u.lo; t < u.hi; ++t, ++g) {
      const int sb = g & 1;
      float a[N];
      if (!c.wait_all(L::SF + sb, (g >> 1) & 1)) { ok = false; break; }
      tc_fence_after();
      // Once for most tiles; three times where a maximum moves (look, find it, use it).  A loop, so
      // that the code is there once: what runs for the first time waits for its instructions.
#pragma unroll 1
      for (int pass = 0;; ++pass) {
        // Scores in log2 units but for a factor sc; minus infinity where masked.
        tmem_ld_n<N>(lane_addr + L::TM_S + sb * N, reinterpret_cast<uint32_t*>(a));
        if (p.has_cap) {
          // c * tanh(sm_scale * x / c) in log2 units, from tanh(y) = 1 - 2 / (e^(2y) + 1).
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const float r = rcp_approx(ex2_approx(a[n] * p.cap_ex2_scale) + 1.f);
            a[n] = fmaf(r, -2.f * p.cap_log2, p.cap_log2);
          }
        }
        if ((int64_t)t * KEYS + KEYS > min(u.q.ctx, (int64_t)u.q.kv)) {   // nodes, or the end of the keys
          const uint64_t seen = seen_by<N>(p.t, u, first_pair, (int64_t)t * KEYS + key);
#pragma unroll
          for (int n = 0; n < N; ++n)
            if (!((seen >> n) & 1)) a[n] = NEG_INF;
        }
        if (pass == 1) {
#pragma unroll
          for (int n = 0; n < N; ++n) a[n] = has_key ? a[n] * sc : NEG_INF;
          reduce_rows<N>(a, rows + w * N, lane, [](float x, float y) { return fmaxf(x, y); });
          ok = exchange();
          if (!ok) break;
#pragma unroll
          for (int n = 0; n < N; ++n) {   // a: what O and l are scaled by
            const float x = fmaxf(fmax3(rows[n], rows[N + n], rows[2 * N + n]), rows[3 * N + n]);
            a[n] = 1.f;
            if (x + neg_m[n] > TREE_RESCALE_THRESHOLD) {
              a[n] = ex2_approx(-neg_m[n] - x);
              neg_m[n] = -x;
            }
            l[n] *= a[n];
          }
          if (t > u.lo) {
            ok = c.wait_all(L::OD + ((g - 1) & 1), ((g - 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
              float ov[N];
              tmem_ld_n<N>(lane_addr + j * N, reinterpret_cast<uint32_t*>(ov));
#pragma unroll
              for (int n = 0; n < N; ++n) ov[n] *= a[n];
              tmem_st_n<N>(lane_addr + j * N, reinterpret_cast<const uint32_t*>(ov));
            }
          }
          continue;
        }
        float top[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
        for (int n = 0; n < N; n += 2) {
          a[n] = fmaf(a[n], sc, neg_m[n]);
          a[n + 1] = fmaf(a[n + 1], sc, neg_m[n + 1]);
          top[(n >> 1) & 3] = fmax3(top[(n >> 1) & 3], a[n], a[n + 1]);
        }
        if (pass == 2) break;
        const bool above = has_key && fmaxf(fmax3(top[0], top[1], top[2]), top[3]) > TREE_RESCALE_THRESHOLD;
        const int any_above = __any_sync(0xffffffffu, above);
        int* mine = flags + (xs & 1) * 4;   // (written again after the exchange between)
        if (lane == 0) mine[w] = any_above;
        ok = exchange();
        if (!ok) break;
        const int4 f = *reinterpret_cast<const int4*>(mine);
        if (!(f.x | f.y | f.z | f.w)) break;   // no maximum has moved: the same in all four warps
      }
      if (!ok) break;
      // Copied along behind the last key: zero as values (their P is 0, but 0 times what is there
      // need not be).  S, which read them too, is done.
      const int valid = u.q.kv - t * KEYS;
      if (p.grouped && valid > 0 && valid < KEYS) {
#pragma unroll 1
        for (int i = (threadIdx.x & 127); i < (KEYS - valid) * 64; i += 128) {
          const int panel = (i >> 3) & 7, row = valid + (i >> 6);
          const int pair_slot = (4 * g + (panel >> 1)) % L::PAIRS;
          *reinterpret_cast<uint4*>(smem + L::OFF_PAIR + pair_slot * PAIR + (panel & 1) * PANEL + row * 128 +
                                    (i & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
      }
      // P's buffer: the product that read it last is done.
      if (g >= L::PBUF) {
        const int d = g - L::PBUF;
        if (!c.wait_all(L::OD + (d & 1), (d >> 1) & 1)) { ok = false; break; }
      }
      uint8_t* at[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        at[k] = smem + L::OFF_P + (g % L::PBUF) * L::QPANEL + (((key >> 3) ^ k) << 4) + (key & 7) * 2;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float e = ex2_approx(a[n]);
        l[n] += e;                                                         // (lanes without a key: unused)
        if (has_key) *reinterpret_cast<__nv_bfloat16*>(at[n & 7] + n * 128) = __float2bfloat16_rn(e);   // the operand type
      }
      fence_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar(L::PR + sb));
    }
    if (!ok) break;
    // The part's end: the sums over all keys; lane n of warp 0 has row n (and n + 32).
    if (!exchange()) break;   // (rows may still be read by the last tile's third pass)
#pragma unroll
    for (int n = 0; n < N; ++n) l[n] = has_key ? l[n] : 0.f;
    reduce_rows<N>(l, rows + w * N, lane, [](float x, float y) { return x + y; });
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (w == 0 && lane == n % 32) scale[n] = neg_m[n];
    if (!exchange()) break;
    char* slot = ws_slots + (size_t)u.slot * slot_bytes(N);
    if (w == 0) {
#pragma unroll 1
      for (int n = lane; n < N; n += 32) {
        const float sum = (rows[n] + rows[N + n]) + (rows[2 * N + n] + rows[3 * N + n]);
        const bool empty = !(sum > 0.f);
        const float m = empty ? NEG_INF : -scale[n];
        scale[n] = !u.whole ? 1.f : empty ? 0.f : 1.f / sum;
        if (n < u.npairs) {
          float lg;
          asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(sum));
          if (!u.whole) reinterpret_cast<float2*>(slot + slot_ml(N))[n] = make_float2(m, sum);
          else if (p.t.lse) p.t.lse[u.pair0 + n] = empty ? NEG_INF : (m + lg) * 0.6931471805599453f;
        }
      }
    }
    if (!exchange()) break;
    if (!c.wait_all(L::OD + ((g - 1) & 1), ((g - 1) >> 1) & 1)) break;
    tc_fence_after();
    __nv_bfloat16* out = p.t.o + u.pair0 * 512 + 32 * w + lane;
    float* part = reinterpret_cast<float*>(slot) + 32 * w + lane;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      float ov[N];
      tmem_ld_n<N>(lane_addr + j * N, reinterpret_cast<uint32_t*>(ov));
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (n < u.npairs) {
          // (O is finite where l is not 0; a row without a key is 0 whatever is there.)
          const float k = scale[n], x = k == 0.f ? 0.f : ov[n] * k;
          if (u.whole) out[128 * j + n * 512] = __float2bfloat16_rn(x);
          else part[128 * j + n * 512] = x;
        }
      }
    }
    tc_fence_before();   // O has been read: the next part's first P-ready lets it be overwritten
    __syncwarp();
    if (!exchange()) break;   // rows and scale have been read
  }
}

template <int N>
__global__ void __launch_bounds__(NTHREADS, 1)
tree_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c,
                const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_2,
                const __grid_constant__ TreeLaunch p) {
  using L = Lay<N>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ StartRec start;
  __shared__ int64_t count;
  __shared__ JoinRec join;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(smem + L::OFF_MISC + 4);
  const int worker = blockIdx.x;
  const Ctx<N> c{smem_addr(smem), abort_flag, p.t.status, p.wait_limit_ns};
  launch_dependents();   // the join kernel, which waits for this one to end
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NBAR; ++i) mbar_init(c.bar(i), 1);
    mbar_init(c.bar(L::XB), 4);                                  // the four softmax warps
    for (int i = 0; i < 2; ++i) mbar_init(c.bar(L::PR + i), 4);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_c);
    if (p.piece_rows > 0) tma_prefetch_desc(&tm_b);
    if (p.grouped) tma_prefetch_desc(&tm_2);
  }
  if (warp == 2) {
    tmem_alloc(smem_addr(tmem_slot), L::TMEM);
    tmem_relinquish();
  }
  find_piece<N, KEYS, NTHREADS>(p.t, worker, p.workers, blockIdx.x == 0, &start, &count, &join);
  char* ws = static_cast<char*>(p.t.workspace);
  if (threadIdx.x == 0) reinterpret_cast<JoinRec*>(ws)[worker] = join;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const Parts<N, KEYS> parts(p.t, start, count);
  if (warp == 0) {
    run_producer<N>(c, p, parts, &tm_c, &tm_b, &tm_2);
  } else if (warp == 1) {
    run_mma<N>(c, p, parts, tmem);
  } else if (warp == 3) {
    if (lane == 0) run_q<N>(c, parts, &tm_q);
  } else if (warp >= 4) {
    run_softmax<N>(c, p, parts, tmem, ws + WS_SLOTS + (size_t)worker * 2 * slot_bytes(N), smem);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) {
    __syncwarp();
    tmem_dealloc(tmem, L::TMEM);
  }
}

template <int N>
cudaError_t configure() {
  static PerDeviceOnce configured;
  return configured.run([] {
    return cudaFuncSetAttribute(tree_few_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<N>::SMEM);
  });
}

template <int N>
cudaError_t launch(const TreeLaunch& p, const CUtensorMap& tq, const CUtensorMap& tc, const CUtensorMap& tb,
                   const CUtensorMap& t2, cudaStream_t stream) {
  const cudaError_t e = configure<N>();
  if (e != cudaSuccess) return e;
  tree_few_kernel<N><<<p.workers, NTHREADS, Lay<N>::SMEM, stream>>>(tq, tc, tb, t2, p);
  return cudaGetLastError();
}

}  // namespace

int tree_few_workers() {
  const int n = device_sm_count();
  return n < MAX_WORKERS ? n : MAX_WORKERS;
}

cudaError_t launch_tree_few(const TreeLaunch& p, int rows, const CUtensorMap& tq, const CUtensorMap& tc,
                            const CUtensorMap& tb, const CUtensorMap& t2, cudaStream_t stream) {
  switch (rows) {
    case 16: return launch<16>(p, tq, tc, tb, t2, stream);
    case 32: return launch<32>(p, tq, tc, tb, t2, stream);
    case 64: return launch<64>(p, tq, tc, tb, t2, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mla
