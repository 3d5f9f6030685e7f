// The 4-bit latent entry (layout in include/mla_prefill.h): its sizes, and its codes to bf16 and back.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace mla {

constexpr int FP4_ENTRY = 400;         // bytes: 256 of codes, 128 of rope, 16 of scales
constexpr int FP4_ROPE = 256, FP4_SCALES = 384;
constexpr uint32_t FP4_MAX_SCALE = 252;   // the largest byte with which every code stays finite in bf16

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Bytes of a word of scales above that (in their top bits).
__device__ __forceinline__ uint32_t above252(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x03030303u) & w & 0x80808080u; }

// bf16 of a scale byte, 2^(b - 127), in both halves: b is a bf16's exponent field; 0 stands for the
// subnormal 2^-127, 255 for NaN.
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t b) {
  const uint32_t h = b == 0 ? 0x0040u : b == 255 ? 0x7fc0u : b << 7;
  return h | h << 16;
}

// A word's eight values as four bf16x2, values 2 k and 2 k + 1 in word k, times 2^-126: the code's exponent
// and mantissa bits are moved to where bf16 has them, which makes the value a (sub)normal number of bf16's
// least exponents.
__device__ __forceinline__ void fp4_fields(uint32_t w, uint32_t* r) {
  r[0] = ((w << 12) & 0x80008000u) | ((w << 6) & 0x01c001c0u);
  r[1] = ((w << 8) & 0x80008000u) | ((w << 2) & 0x01c001c0u);
  r[2] = ((w << 4) & 0x80008000u) | ((w >> 2) & 0x01c001c0u);
  r[3] = (w & 0x80008000u) | ((w >> 6) & 0x01c001c0u);
}

// A word's values times a scale byte's, rounded to bf16: exact unless past its largest value (infinite).
__device__ __forceinline__ uint4 fp4_values(uint32_t w, uint32_t scale) {
  uint32_t r[4];
  fp4_fields(w, r);
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = mul_bf16x2(mul_bf16x2(r[k], 0x7e807e80u), scale);   // 2^126, then the scale
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Two fp32 values to two codes, the first in the low nibble: to nearest, ties to the even code.
__device__ __forceinline__ uint32_t fp4_codes(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t fp4_word(const float* v) {
  return fp4_codes(v[0], v[2]) | fp4_codes(v[4], v[6]) << 8 | fp4_codes(v[1], v[3]) << 16 | fp4_codes(v[5], v[7]) << 24;
}

}  // namespace mla
