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

// Where units have few pairs (slots row by row): a CTA has a row of a cut unit and threads four columns.  GROUPS = 1:
// 128 threads take its parts one after the other, and there is a CTA for every boundary (mostly a unit is cut in two or
// three).  GROUPS = 4, for calls of few units, which have many parts each: four groups of 128 threads take every fourth
// part, and CTA i looks for the i-th boundary with a unit to join: with a CTA for every boundary their start alone took
// 2 us.  (In replayed graphs, the whole call at 16 heads: 2 requests over 8192 23.5 us, 34.6 with GROUPS = 1 and 27.1 with
// GROUPS = 4 at every boundary; 8 over 8192 30.5, 33.8 and 32.0; 16 over 8192 42.7 with GROUPS = 1, 43.9 with 4.)
template <int GROUPS>
__global__ void __launch_bounds__(GROUPS * 128) tree_join_few_kernel(const __grid_constant__ TreeLaunch p) {
  constexpr int THREADS = GROUPS * 128;
  __shared__ float weight[GROUPS > 1 ? MAX_WORKERS : 1];
  __shared__ float2 part[THREADS / 32];
  __shared__ float4 sum[GROUPS][128];
  const char* ws = static_cast<const char*>(p.t.workspace);
  __shared__ int found[GROUPS > 1 ? THREADS / 32 + 1 : 1];
  const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 31, group = tid >> 7, col = 4 * (tid & 127);
  grid_dependency_wait();   // (the other kernel has ended, what it wrote is there)
  const JoinRec* recs = reinterpret_cast<const JoinRec*>(ws);
  int b = blockIdx.x + 1;   // the boundary before worker b
  if constexpr (GROUPS > 1) {
    const bool is = tid > 0 && tid < p.workers && recs[tid].parts > 0;
    const uint32_t all = __ballot_sync(0xffffffffu, is);
    if (lane == 0) found[tid >> 5] = __popc(all);
    if (tid == 0) found[THREADS / 32] = 0;
    __syncthreads();
    int before = __popc(all & ((1u << lane) - 1));
    for (int w = 0; w < tid >> 5; ++w) before += found[w];
    if (is && before == (int)blockIdx.x) found[THREADS / 32] = tid;
    __syncthreads();
    b = found[THREADS / 32];
    if (b == 0) return;
  }
  const JoinRec j = recs[b];
  const int n = j.parts;
  if (n == 0 || row >= j.npairs) return;
  const char* slots = ws + WS_SLOTS + (size_t)2 * (b - 1) * FEW_SLOT_BYTES;
  auto slot = [&](int k) { return slots + (size_t)(2 * k + (k == 0 ? j.slot0 : 0)) * FEW_SLOT_BYTES; };
  auto state = [&](int k) { return reinterpret_cast<const float2*>(slot(k) + FEW_SLOT_ML)[row]; };
  auto values = [&](int k) { return *reinterpret_cast<const float4*>(slot(k) + ((size_t)row * 512 + col) * 4); };
  const float NEG_INF = -__int_as_float(0x7f800000);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = NEG_INF, l = 0.f;
  auto add = [&](float f, const float4& x) {
    o.x += f * x.x;
    o.y += f * x.y;
    o.z += f * x.z;
    o.w += f * x.w;
  };
  if constexpr (GROUPS == 1) {
#pragma unroll 8
    for (int k = 0; k < n; ++k) m = fmaxf(m, state(k).x);
    const float mref = m == NEG_INF ? 0.f : m;
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float2 ml = state(k);
      const float f = ex2_approx(ml.x - mref);
      l += f * ml.y;
      add(f, values(k));
    }
  } else {
    // The parts' maximum, and the sum of their weighted sums (n <= 256: a thread a part).
    float2 ml = make_float2(NEG_INF, 0.f);
    if (tid < n) ml = state(tid);
    m = ml.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) part[tid >> 5].x = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) m = fmaxf(m, part[w].x);
    const float w = tid < n ? ex2_approx(ml.x - (m == NEG_INF ? 0.f : m)) : 0.f;
    if (tid < n) weight[tid] = w;
    l = tid < n ? w * ml.y : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (lane == 0) part[tid >> 5].y = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) l += part[i].y;
#pragma unroll 8
    for (int k = group; k < n; k += GROUPS) add(weight[k], values(k));
    if (group > 0) sum[group][tid & 127] = o;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) add(1.f, sum[i][tid]);
  }
  const bool empty = l == 0.f;   // (a NaN is passed on)
  const float inv = empty ? 0.f : 1.f / l;
  const int64_t pair = j.pair0 + row;
  *reinterpret_cast<uint2*>(p.t.o + pair * 512 + col) =
      empty ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (col == 0 && p.t.lse) p.t.lse[pair] = empty ? NEG_INF : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_tree_join_few(const TreeLaunch& p, cudaStream_t stream) {
  if (p.workers < 2) return cudaSuccess;
  const int64_t units = (p.t.total_rows * p.t.num_heads + (int64_t)p.t.batch * (TREE_FEW - 1)) / TREE_FEW;   // at most
  const bool wide = units * 8 <= p.workers;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = wide ? dim3((unsigned)units, TREE_FEW) : dim3(p.workers - 1, TREE_FEW);
  cfg.blockDim = dim3(wide ? 512 : 128);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, tree_join_few_kernel<4>, p) : cudaLaunchKernelEx(&cfg, tree_join_few_kernel<1>, p);
}

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
