// Joins the parts that several workers left of a unit of tree attention: with part k's
// (O_k, m_k, l_k) in fp32 and M = max m_k,
//   O = sum 2^(m_k - M) O_k / sum 2^(m_k - M) l_k,  LSE = ln 2 (M + log2 sum 2^(m_k - M) l_k).
#include "tree_attn.cuh"

namespace mla {
namespace {

// One CTA per eight rows of a unit that a boundary between two workers cuts (the unit's first such
// boundary).  A warp has a row: the parts' (m, l) one per lane, then their O rows, 16 columns per
// lane.  Bound by latency: record, (m, l), O, result, each waits for the one before.
constexpr int JOIN_WARPS = 8;

__global__ void __launch_bounds__(JOIN_WARPS * 32) tree_join_kernel(const __grid_constant__ TreeLaunch p) {
  const char* ws = static_cast<const char*>(p.t.workspace);
  const int b = blockIdx.x + 1;   // the boundary before worker b
  const JoinRec j = reinterpret_cast<const JoinRec*>(ws)[b];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * JOIN_WARPS + warp;
  if (row >= j.npairs || j.parts == 0) return;
  const int64_t pair = j.pair0 + row;
  const int n = j.parts;
  const char* slots = ws + WS_SLOTS + (size_t)2 * (b - 1) * SLOT_BYTES;
  auto slot = [&](int k) { return slots + (size_t)(2 * k + (k == 0 ? j.slot0 : 0)) * SLOT_BYTES; };
  const float NEG_INF = -__int_as_float(0x7f800000);
  float m = NEG_INF;
  for (int k = lane; k < n; k += 32) m = fmaxf(m, reinterpret_cast<const float2*>(slot(k) + SLOT_ML)[row].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float mref = m == NEG_INF ? 0.f : m;
  float4 o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int k0 = 0; k0 < n; k0 += 32) {
    float w = 0.f, wl = 0.f;
    if (k0 + lane < n) {
      const float2 ml = reinterpret_cast<const float2*>(slot(k0 + lane) + SLOT_ML)[row];
      w = ex2_approx(ml.x - mref);
      wl = w * ml.y;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) wl += __shfl_xor_sync(0xffffffffu, wl, d);
    l += wl;
    const int here = min(32, n - k0);
#pragma unroll 4
    for (int k = 0; k < here; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float4* src = reinterpret_cast<const float4*>(slot(k0 + k)) + (size_t)row * 128 + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = src[32 * i];
        o[i].x += wk * x.x;
        o[i].y += wk * x.y;
        o[i].z += wk * x.z;
        o[i].w += wk * x.w;
      }
    }
  }
  const bool empty = l == 0.f;
  const float inv = empty ? 0.f : 1.f / l;
  uint2* d = reinterpret_cast<uint2*>(p.t.o + pair * 512) + lane;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    d[32 * i] = empty ? make_uint2(0u, 0u)
                      : make_uint2(pack_bf16x2(o[i].x * inv, o[i].y * inv), pack_bf16x2(o[i].z * inv, o[i].w * inv));
  if (lane == 0 && p.t.lse) p.t.lse[pair] = empty ? NEG_INF : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_tree_join(const TreeLaunch& p, cudaStream_t stream) {
  if (p.workers < 2) return cudaSuccess;
  // (Launched early, to wait for the other kernel's end on the GPU, it made calls up to 4 us longer:
  // its CTAs take room and issue slots from that kernel's.)
  tree_join_kernel<<<dim3(p.workers - 1, TREE_ROWS / JOIN_WARPS), JOIN_WARPS * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
