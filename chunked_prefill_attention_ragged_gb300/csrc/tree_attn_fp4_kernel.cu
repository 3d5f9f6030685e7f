// Tree attention over a cache of 4-bit entries (include/mla_prefill.h): a plain kernel, one warp for each
// (node, head) pair, which goes over the keys once with the running maximum and sum of its softmax.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "internal.h"
#include "tree_attn.cuh"

namespace mla {
namespace {

constexpr int WARPS = 8;

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__global__ void __launch_bounds__(WARPS * 32) tree_attn_fp4_kernel(const __grid_constant__ TreeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t pair = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  const int64_t row = pair / p.num_heads;
  if (pair >= p.total_rows * p.num_heads) return;
  int r = 0;
  for (; r < p.batch; ++r) {   // the request that has the row
    const Req q = load_req(p, r, pair == 0);
    if (pair > 0 && row >= q.q0 && row < q.q0 + q.nodes) break;
  }
  if (pair == 0)
    for (r = 0; r < p.batch; ++r) {
      const Req q = load_req(p, r, false);
      if (row >= q.q0 && row < q.q0 + q.nodes) break;
    }
  if (r == p.batch) return;
  const Req req = load_req(p, r, false);
  Part u;
  u.q = req;
  u.r = r;
  const int node = (int)(row - req.q0);
  const uint8_t* cache = reinterpret_cast<const uint8_t*>(p.cache);
  const uint4* qv = reinterpret_cast<const uint4*>(p.q + pair * 576);
  float q[2][8], qr[8] = {}, acc[2][8] = {};
  unpack8(qv[lane], q[0]);
  unpack8(qv[32 + lane], q[1]);
  if (lane < 8) unpack8(qv[64 + lane], qr);
  const float NEG_INF = -__int_as_float(0x7f800000);
  float m = NEG_INF, l = 0.f;
  uint64_t bits = 0;
  for (int key = 0; key < req.kv; ++key) {
    if ((key & 63) == 0) bits = visible(p, u, node, key);
    if (!((bits >> (key & 63)) & 1)) continue;
    const int64_t b = __ldg(p.block_table + (int64_t)r * p.max_blocks + key / p.block_size);
    const bool there = b >= 0 && b < p.num_blocks;
    if (!there && lane == 0 && p.status) atomicOr(p.status, MLA_DEVSTAT_BAD_INDEX);
    float c[2][8] = {}, s = 0.f;
    if (there) {
      const uint8_t* e = cache + (b * p.block_size + key % p.block_size) * FP4_ENTRY;
      float rope[8] = {};
      uint32_t most = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sc = __ldg(e + FP4_SCALES + 8 * h + (lane >> 2));
        most = max(most, sc);
        unpack8(fp4_values(__ldg(reinterpret_cast<const uint32_t*>(e) + 32 * h + lane), scale_bf16x2(sc)), c[h]);
      }
      if (lane < 8) unpack8(__ldg(reinterpret_cast<const uint4*>(e + FP4_ROPE) + lane), rope);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += q[0][i] * c[0][i] + q[1][i] * c[1][i] + qr[i] * rope[i];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (__any_sync(0xffffffffu, most > FP4_MAX_SCALE)) s = __int_as_float(0x7fc00000);
    }
    s *= p.sm_scale;
    if (p.soft_cap > 0.f) s = p.soft_cap * tanhf(s / p.soft_cap);
    const float mn = s > m ? s : m;   // (a NaN passes into the sums)
    const float old = m == NEG_INF ? 0.f : expf(m - mn), w = expf(s - mn);
    m = mn;
    l = l * old + w;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[h][i] = acc[h][i] * old + w * c[h][i];
  }
  const bool empty = m == NEG_INF && l == 0.f;
  uint4* o = reinterpret_cast<uint4*>(p.o + pair * 512);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = empty ? 0u : pack_bf16x2(acc[h][2 * i] / l, acc[h][2 * i + 1] / l);
    o[32 * h + lane] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (lane == 0 && p.lse) p.lse[pair] = empty ? NEG_INF : m + logf(l);
}

}  // namespace

cudaError_t launch_tree_attention_fp4(const TreeParams& p, cudaStream_t stream) {
  const int64_t pairs = p.total_rows * p.num_heads;
  tree_attn_fp4_kernel<<<(unsigned)((pairs + WARPS - 1) / WARPS), WARPS * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
