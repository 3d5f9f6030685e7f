// What the kernels of tree attention share: the issue of a pair's products, stores to shared memory, logits under a cap.
#pragma once
#include "ptx.cuh"
#include "tree_attn.cuh"

namespace mla {

__device__ __forceinline__ void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The whole warp runs the issue loop and one elected lane (always the same) issues, with every
// operand in a register that the compiler knows to be the same in all lanes (values from memory
// are broadcast by a shuffle first).  With a branch for lane 0 around the loop, or operands that
// may differ by lane, a product took 50-70 clocks to issue; this way an M = 128, N = 128 product
// of the pair takes 32 and an N = 256 one 64, the tensor cores' own rate.  Descriptors are
// passed as low and high words: only the low one moves.
__device__ __forceinline__ void issue_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
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

// c * tanh(y) in log2 units, y = x / c with the logit x.  For |y| < 1/4 x times the series of tanh(y) / y,
// whose next term is 2^-21; from there on c (1 - 2 / (e^(2y) + 1)), which is good to 2^-22 of c and so to
// 2^-20 of the result, where below it would lose the logit's low bits (all of them under a large cap).
// Most logits are far below their cap, so the second is worked out only for the 16 keys of a warp's rows
// in which some logit needs it.  (9 x up to 37 nodes under a cap of 30: 40.6 us, 39.4 with the second form
// alone; both for all keys and a choice: 41.2; tanh(y) / y as a quotient of polynomials: 41.0.)
template <int KEYS_HERE>
__device__ __forceinline__ void cap_scores(const TreeLaunch& p, float* sv) {
  const float2 inv2 = make_float2(p.cap_inv, p.cap_inv), scale2 = make_float2(p.scale_log2, p.scale_log2);
  const float2 e2 = make_float2(2.8853900817779268f, 2.8853900817779268f), one = make_float2(1.f, 1.f);
  const float2 cap2 = make_float2(p.cap_log2, p.cap_log2), m2c = make_float2(-2.f * p.cap_log2, -2.f * p.cap_log2);
  const float2 s1 = make_float2(-1.f / 3.f, -1.f / 3.f), s2 = make_float2(2.f / 15.f, 2.f / 15.f);
  const float2 s3 = make_float2(-17.f / 315.f, -17.f / 315.f);
#pragma unroll
  for (int j = 0; j < KEYS_HERE; j += 16) {
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

}  // namespace mla
