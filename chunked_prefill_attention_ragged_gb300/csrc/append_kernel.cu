// New tokens into the paged latent cache: y = x rsqrt(mean(x^2) + eps) w over the 512 latents (or y = x), the
// 64 rope values turned by the position's angles, both rounded once to the entry's types and stored by slot;
// the queries' rope turned by the same angles in the same launch.
//
// Memory bound, 128 bytes in and out for each head of a token beside 1152 + 256 in and an entry out for
// its row.  A warp has a token's row (lane l the 16-byte chunks l and 32 + l: a scale group is 4 lanes of
// one load in fp4, 8 in fp8, so that its largest magnitude takes two or three shuffles), or 32 heads of its
// queries: eight lanes a head, four heads a load, eight loads under way.  Both kinds are blocks of one
// grid, so that a decoding step of few tokens has all its latencies side by side.  (Replayed graphs: 8192 bf16 tokens
// with 128 heads 50 us, 290 MB at 5.8 TB/s, 0.86 of a copy's rate; up to 2049 fp8 tokens of 5 requests and the gather of
// them 8 us, data that stay in L2; 64 fp4 tokens with 16 heads 3 us, the three loads that follow one another.)
//
// Roundings: sums, norm and rotation are fp32; each stored value is rounded once.  Squares may leave fp32's range where
// values do not: such a row is scaled by a power of two first.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int WARPS = 4;           // tokens of a block
constexpr int HEADS = 32;          // heads of a warp of queries
constexpr unsigned ALL = 0xffffffffu;

__device__ __forceinline__ void unpack(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// What turns the eight values 8 c .. 8 c + 7 of a rope: lane c of eight.
struct Turn {
  float cos[8], sin[8];   // interleaved: four of each
  int interleaved, c;
  __device__ Turn(const float* row, int which, int lane) : interleaved(which), c(lane & 7) {
    const float4* t = reinterpret_cast<const float4*>(row);
    const int at = interleaved ? c : 2 * (c & 3);
    const float4 a = __ldg(t + at), b = __ldg(t + 8 + at);
    cos[0] = a.x, cos[1] = a.y, cos[2] = a.z, cos[3] = a.w;
    sin[0] = b.x, sin[1] = b.y, sin[2] = b.z, sin[3] = b.w;
    if (!interleaved) {
      const float4 d = __ldg(t + at + 1), e = __ldg(t + 8 + at + 1);
      cos[4] = d.x, cos[5] = d.y, cos[6] = d.z, cos[7] = d.w;
      sin[4] = e.x, sin[5] = e.y, sin[6] = e.z, sin[7] = e.w;
    }
  }
  // (every lane of the warp calls: value i + 32 is with the lane four further)
  __device__ uint4 operator()(const uint4& v) const {
    float x[8], y[8];
    unpack(v, x);
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = x[2 * i] * cos[i] - x[2 * i + 1] * sin[i];
        y[2 * i + 1] = x[2 * i + 1] * cos[i] + x[2 * i] * sin[i];
      }
    } else {
      float o[8];
      unpack(make_uint4(__shfl_xor_sync(ALL, v.x, 4), __shfl_xor_sync(ALL, v.y, 4), __shfl_xor_sync(ALL, v.z, 4),
                        __shfl_xor_sync(ALL, v.w, 4)), o);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = c < 4 ? x[i] * cos[i] - o[i] * sin[i] : x[i] * cos[i] + o[i] * sin[i];
    }
    return pack(y);
  }
};

// The scale byte of a group whose largest magnitude is m: the least power of two with m <= 1.75 * 2^TOP * scale,
// 255 where m is NaN or infinite or the byte would pass MOST.  (Adding 0x1fffff carries a mantissa above 0.75
// into the exponent.)
template <int TOP, int MOST>
__device__ __forceinline__ uint32_t scale_byte(float m) {
  const int e = (int)((__float_as_uint(m) + 0x1fffffu) >> 23) - TOP;
  return !(m <= 3.402823466e38f) || e > MOST ? 255u : (uint32_t)max(e, 0);
}
// 2^(127 - b), by which a value is divided by its scale (0 for 255: the group's codes are zeros).
__device__ __forceinline__ float inverse_scale(uint32_t b) {
  return __uint_as_float(b >= 254 ? (b == 255 ? 0u : 0x00400000u) : (254u - b) << 23);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float largest(const float* x) {   // NaN if one is
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x[i])));
  return m;
}
__device__ __forceinline__ float larger(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}

// The sum of the squares of a row: each lane has sixteen of its values.
__device__ __forceinline__ float squares(const float (*x)[8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += x[0][i] * x[0][i] + x[1][i] * x[1][i];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(ALL, s, d);
  return s;
}

template <int FORMAT>
__global__ void __launch_bounds__(WARPS * 32) append_kernel(const __grid_constant__ AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (t >= p.num_tokens) return;
  const int64_t slot = __ldg(p.slots + t);
  const int pos = __ldg(p.positions + t);
  if (slot < 0) return;
  if (slot >= p.num_slots || pos < 0 || pos >= p.max_positions) {
    if (lane == 0 && p.status) atomicOr(p.status, MLA_DEVSTAT_BAD_INDEX);
    return;
  }
  const float* angles = p.cos_sin + (int64_t)pos * 64;
  if (blockIdx.y > 0) {   // queries
    const int h0 = (int)(blockIdx.y - 1) * HEADS, n = min(HEADS, p.num_heads - h0);
    const Turn turn(angles, p.interleaved, lane);
    const __nv_bfloat16* src = p.q_rope + t * p.q_token + (int64_t)h0 * p.q_head + (lane & 7) * 8;
    __nv_bfloat16* dst = p.q_out + t * p.q_out_token + (int64_t)h0 * p.q_out_head + (lane & 7) * 8;
    uint4 v[HEADS / 4];
#pragma unroll
    for (int i = 0; i < HEADS / 4; ++i) {
      const int h = 4 * i + (lane >> 3);
      v[i] = h < n ? *reinterpret_cast<const uint4*>(src + h * p.q_head) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < HEADS / 4; ++i) {
      const int h = 4 * i + (lane >> 3);
      const uint4 r = turn(v[i]);
      if (h < n) *reinterpret_cast<uint4*>(dst + h * p.q_out_head) = r;
    }
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(p.latent + t * p.latent_stride);
  const uint4 a = __ldg(src + lane), b = __ldg(src + 32 + lane), c = __ldg(src + 64 + (lane & 7));
  const Turn turn(angles, p.interleaved, lane);
  float x[2][8];
  unpack(a, x[0]);
  unpack(b, x[1]);
  if (p.norm_weight) {
    const uint4* w = reinterpret_cast<const uint4*>(p.norm_weight);
    float g[2][8];
    unpack(__ldg(w + lane), g[0]);
    unpack(__ldg(w + 32 + lane), g[1]);
    float s = squares(x), eps = p.norm_eps;   // (the same in every lane)
    // Squares that leave fp32's range: the row by a power of two, which the quotient takes out again.
    if (s > 0x1p120f || s * (1.f / 512.f) + eps < 0x1p-60f) {
      const float f = s > 1.f ? 0x1p-70f : 0x1p80f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[0][i] *= f;
        x[1][i] *= f;
      }
      s = squares(x);
      eps = eps * f * f;   // (the square of the larger f has no fp32)
    }
    const float r = 1.f / sqrtf(s * (1.f / 512.f) + eps);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = x[u][i] * r * g[u][i];
  }
  const uint4 rope = turn(c);
  if constexpr (FORMAT == MLA_ENTRY_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(p.cache + slot * 1152);
    dst[lane] = pack(x[0]);
    dst[32 + lane] = pack(x[1]);
    if (lane < 8) dst[64 + lane] = rope;
  } else if constexpr (FORMAT == MLA_ENTRY_FP8) {
    uint8_t* dst = p.cache + slot * 648;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float m = largest(x[u]);
      m = larger(m, __shfl_xor_sync(ALL, m, 1));
      m = larger(m, __shfl_xor_sync(ALL, m, 2));
      m = larger(m, __shfl_xor_sync(ALL, m, 4));
      const uint32_t s = scale_byte<8, 254>(m);
      const float inv = inverse_scale(s);
      uint32_t w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = s == 255 ? 0.f : x[u][4 * k + i] * inv;
        w[k] = e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16;
      }
      reinterpret_cast<uint2*>(dst)[32 * u + lane] = make_uint2(w[0], w[1]);
      if ((lane & 7) == 0) dst[640 + 4 * u + (lane >> 3)] = (uint8_t)s;
    }
    if (lane < 8) {
      reinterpret_cast<uint2*>(dst + 512)[2 * lane] = make_uint2(rope.x, rope.y);
      reinterpret_cast<uint2*>(dst + 512)[2 * lane + 1] = make_uint2(rope.z, rope.w);
    }
  } else {
    uint8_t* dst = p.cache + slot * FP4_ENTRY;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float m = largest(x[u]);
      m = larger(m, __shfl_xor_sync(ALL, m, 1));
      m = larger(m, __shfl_xor_sync(ALL, m, 2));
      const uint32_t s = scale_byte<2, (int)FP4_MAX_SCALE>(m);
      const float inv = inverse_scale(s);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = s == 255 ? 0.f : x[u][i] * inv;
      reinterpret_cast<uint32_t*>(dst)[32 * u + lane] = fp4_word(y);
      if ((lane & 3) == 0) dst[FP4_SCALES + 8 * u + (lane >> 2)] = (uint8_t)s;
    }
    if (lane < 8) reinterpret_cast<uint4*>(dst + FP4_ROPE)[lane] = rope;
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int format, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  const dim3 grid((unsigned)((p.num_tokens + WARPS - 1) / WARPS), 1 + (p.num_heads + HEADS - 1) / HEADS);
  if (format == MLA_ENTRY_BF16) append_kernel<MLA_ENTRY_BF16><<<grid, WARPS * 32, 0, stream>>>(p);
  else if (format == MLA_ENTRY_FP8) append_kernel<MLA_ENTRY_FP8><<<grid, WARPS * 32, 0, stream>>>(p);
  else append_kernel<MLA_ENTRY_FP4><<<grid, WARPS * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
