// Joins the parts that several workers left of a unit of tree attention: with part k's
// (O_k, m_k, l_k) in fp32 and M = max m_k,
//   O = sum 2^(m_k - M) O_k / sum 2^(m_k - M) l_k,  LSE = ln 2 (M + log2 sum 2^(m_k - M) l_k).
#include "tree_attn.cuh"

namespace mla {
namespace {

// A CTA has 32 rows of a unit that a boundary between two workers cuts (the unit's first such
// boundary) and 64 of the columns, a thread a row and 16 columns: two 32-byte groups of a part, whose
// rows lie one behind the other.  Bound by latency: record, (m, l), result, each waits for the one
// before, with O's loads under way beside the weights'; 6-8 us of a call with the launch.  (128 columns
// a CTA took a call over 16 parts a unit from 72.0 to 73.4 us, 32 columns a thread to 76.8.)
constexpr int JOIN_WARPS = 4, JOIN_COLS = 16;

__global__ void __launch_bounds__(JOIN_WARPS * 32) tree_join_kernel(const __grid_constant__ TreeLaunch p) {
  const char* ws = static_cast<const char*>(p.t.workspace);
  const int b = blockIdx.x + 1;   // the boundary before worker b
  grid_dependency_wait();   // (the other kernel has ended, what it wrote is there)
  const JoinRec j = reinterpret_cast<const JoinRec*>(ws)[b];
  const int row = (blockIdx.y & 3) * 32 + (threadIdx.x & 31);
  const int col = ((blockIdx.y >> 2) * JOIN_WARPS + (threadIdx.x >> 5)) * JOIN_COLS;
  if (row >= j.npairs || j.parts == 0) return;
  const int64_t pair = j.pair0 + row;
  const int n = j.parts;
  const char* slots = ws + WS_SLOTS + (size_t)2 * (b - 1) * SLOT_BYTES;
  auto slot = [&](int k) { return slots + (size_t)(2 * k + (k == 0 ? j.slot0 : 0)) * SLOT_BYTES; };
  const float NEG_INF = -__int_as_float(0x7f800000);
  float m = NEG_INF;
#pragma unroll 4
  for (int k = 0; k < n; ++k) m = fmaxf(m, reinterpret_cast<const float2*>(slot(k) + SLOT_ML)[row].x);
  const float mref = m == NEG_INF ? 0.f : m;
  float o[JOIN_COLS];
#pragma unroll
  for (int i = 0; i < JOIN_COLS; ++i) o[i] = 0.f;
  float l = 0.f;
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    const char* s = slot(k);
    const float2 ml = reinterpret_cast<const float2*>(s + SLOT_ML)[row];
    const float w = ex2_approx(ml.x - mref);
    l += w * ml.y;
#pragma unroll
    for (int i = 0; i < JOIN_COLS; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(s + slot_at(row, col + i) + (i & 4) * 4);
      o[i] += w * x.x;
      o[i + 1] += w * x.y;
      o[i + 2] += w * x.z;
      o[i + 3] += w * x.w;
    }
  }
  const bool empty = l == 0.f;
  const float inv = empty ? 0.f : 1.f / l;
  uint4* d = reinterpret_cast<uint4*>(p.t.o + pair * 512 + col);
#pragma unroll
  for (int i = 0; i < JOIN_COLS; i += 8) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (!empty)
      v = make_uint4(pack_bf16x2(o[i] * inv, o[i + 1] * inv), pack_bf16x2(o[i + 2] * inv, o[i + 3] * inv),
                     pack_bf16x2(o[i + 4] * inv, o[i + 5] * inv), pack_bf16x2(o[i + 6] * inv, o[i + 7] * inv));
    d[i >> 3] = v;
  }
  if (col == 0 && p.t.lse) p.t.lse[pair] = empty ? NEG_INF : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_tree_join(const TreeLaunch& p, cudaStream_t stream) {
  if (p.workers < 2) return cudaSuccess;
  // Launched while the other kernel's CTAs exit, to wait for its end on the GPU: 0.3 to 0.8 us less a
  // call.  (Launched earlier, on the other kernel's word, it made calls up to 4 us longer: its CTAs take
  // room and issue slots from that kernel's.)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.workers - 1, TREE_ROWS / 32 * (512 / (JOIN_WARPS * JOIN_COLS)));
  cfg.blockDim = dim3(JOIN_WARPS * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel, p);
}

}  // namespace mla
