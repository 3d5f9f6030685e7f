// Tree attention over the paged latent cache, absorbed-weight form, with every length on the
// device: O_lat = softmax(sm_scale * q_abs . c^T) c[:, :512] and the per-row LSE.
//
// Plain form: one warp per (token, head), one key at a time.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32) tree_attn_simple(const TreeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t pair = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (pair >= p.total_rows * p.num_heads) return;
  const int64_t t = pair / p.num_heads;
  if (t >= p.qo_indptr[p.batch]) return;
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.qo_indptr[mid] <= t) lo = mid; else hi = mid;
  }
  const int r = lo;
  const int n = p.qo_indptr[r + 1] - p.qo_indptr[r], i = (int)(t - p.qo_indptr[r]);
  if (i < 0 || i >= n) return;
  if (p.qo_indptr[r] < 0 || p.qo_indptr[r + 1] > p.total_rows) {
    if (lane == 0 && p.status) atomicOr(p.status, MLA_DEVSTAT_BAD_INDEX);
    return;
  }
  const int64_t reach = (int64_t)p.max_blocks * p.block_size;
  int64_t kv = p.kv_lens[r];
  const int64_t ctx = kv - n;
  if (kv < 0 || kv > reach) {
    if (lane == 0 && p.status) atomicOr(p.status, MLA_DEVSTAT_BAD_INDEX);
    kv = kv < 0 ? 0 : reach;
  }
  const __nv_bfloat162* q = reinterpret_cast<const __nv_bfloat162*>(p.q + pair * 576);
  float2 qv[9], acc[8];
  for (int k = 0; k < 9; ++k) qv[k] = __bfloat1622float2(q[lane + 32 * k]);
  for (int k = 0; k < 8; ++k) acc[k] = make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  for (int64_t pos = 0; pos < kv; ++pos) {
    if (pos >= ctx) {
      const int64_t j = pos - ctx;
      bool seen = j <= i;
      if (p.mask) seen = (j >> 6) < p.mask_words && ((p.mask[t * p.mask_words + (j >> 6)] >> (j & 63)) & 1);
      if (!seen) continue;
    }
    const int64_t blk = p.block_table[(int64_t)r * p.max_blocks + pos / p.block_size];
    float2 kvv[9];
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0 && p.status) atomicOr(p.status, MLA_DEVSTAT_BAD_INDEX);
      for (int k = 0; k < 9; ++k) kvv[k] = make_float2(0.f, 0.f);
    } else {
      const __nv_bfloat162* c =
          reinterpret_cast<const __nv_bfloat162*>(p.cache + (blk * p.block_size + pos % p.block_size) * 576);
      for (int k = 0; k < 9; ++k) kvv[k] = __bfloat1622float2(c[lane + 32 * k]);
    }
    float s = 0.f;
    for (int k = 0; k < 9; ++k) s += qv[k].x * kvv[k].x + qv[k].y * kvv[k].y;
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.sm_scale;
    if (p.soft_cap > 0.f) s = p.soft_cap * tanhf(s / p.soft_cap);
    const float mn = fmaxf(m, s), a = expf(m - mn), e = expf(s - mn);
    l = l * a + e;
    for (int k = 0; k < 8; ++k) acc[k] = make_float2(acc[k].x * a + e * kvv[k].x, acc[k].y * a + e * kvv[k].y);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(p.o + pair * 512);
  for (int k = 0; k < 8; ++k) o[lane + 32 * k] = __floats2bfloat162_rn(acc[k].x * inv, acc[k].y * inv);
  if (lane == 0 && p.lse) p.lse[pair] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

int64_t tree_workspace_bytes() { return 256; }

cudaError_t launch_tree_attention(const TreeParams& p, cudaStream_t stream) {
  const int64_t pairs = p.total_rows * p.num_heads;
  tree_attn_simple<<<(unsigned)((pairs + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
