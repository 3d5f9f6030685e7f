// The cached rows that a call of tree attention reads, 4-bit entries, as bf16 rows of 576 at the same slots of another
// memory: for calls in which so many pairs read a row that it pays (launch_tree_attention_fp4 says when).
//
// Memory bound: 400 bytes read, 1152 written a row.  A warp has a row as in the gather of entries; a request's rows are
// shared out to blocks of its own column of the grid, whose lengths are on the device.  (32 requests of 8192: 62-65 us, 6.3 TB/s.)
// A row with a scale byte above 252 is NaN in its rope, which only the scores see, and zeros in such groups' values.
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int THREADS = 256;

__global__ void __launch_bounds__(THREADS) tree_expand_kernel(const __grid_constant__ TreeParams t, uint8_t* __restrict__ out) {
  const int r = blockIdx.y, lane = threadIdx.x & 31, sh = 8 * ((lane >> 2) & 3);
  grid_launch_dependents();
  const int q0 = __ldg(t.qo_indptr + r), q1 = __ldg(t.qo_indptr + r + 1);
  if (q0 < 0 || q1 <= q0 || q1 > t.total_rows) return;   // (nothing of it is computed)
  const int64_t kv = min((int64_t)__ldg(t.kv_lens + r), (int64_t)t.max_blocks * t.block_size);
  const int32_t* table = t.block_table + (int64_t)r * t.max_blocks;
  const uint8_t* cache = reinterpret_cast<const uint8_t*>(t.cache);
  const int64_t step = (int64_t)gridDim.x * (THREADS / 32);
  for (int64_t pos = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); pos < kv; pos += step) {
    const int page = (int)((uint32_t)pos / (uint32_t)t.block_size);
    const int32_t block = __ldg(table + page);
    if (block < 0 || block >= t.num_blocks) continue;   // (the attention reports it)
    const int64_t slot = (int64_t)block * t.block_size + ((int)pos - page * t.block_size);
    const uint8_t* src = cache + slot * FP4_ENTRY;
    const uint32_t w0 = __ldg(reinterpret_cast<const uint32_t*>(src) + lane), w1 = __ldg(reinterpret_cast<const uint32_t*>(src) + 32 + lane);
    const uint4 sc = __ldg(reinterpret_cast<const uint4*>(src + FP4_SCALES));
    uint4 rope = make_uint4(0, 0, 0, 0);
    if (lane < 8) rope = __ldg(reinterpret_cast<const uint4*>(src + FP4_ROPE) + lane);
    if (above252(sc.x) | above252(sc.y) | above252(sc.z) | above252(sc.w)) rope = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
    const uint32_t s0 = ((lane < 16 ? sc.x : sc.y) >> sh) & 0xffu, s1 = ((lane < 16 ? sc.z : sc.w) >> sh) & 0xffu;
    uint4* dst = reinterpret_cast<uint4*>(out + slot * (576 * 2));
    dst[lane] = fp4_values(s0 > FP4_MAX_SCALE ? 0 : w0, scale_bf16x2(s0 > FP4_MAX_SCALE ? 0 : s0));
    dst[32 + lane] = fp4_values(s1 > FP4_MAX_SCALE ? 0 : w1, scale_bf16x2(s1 > FP4_MAX_SCALE ? 0 : s1));
    if (lane < 8) dst[64 + lane] = rope;
  }
}

}  // namespace

cudaError_t launch_tree_expand(const TreeParams& t, void* out, cudaStream_t stream) {
  const int64_t reach = (int64_t)t.max_blocks * t.block_size, warps = THREADS / 32;
  // Eight times what is resident at once: a warp has several rows where there are many, and short requests beside long
  // ones cost little.
  const int64_t most = std::max<int64_t>(1, (int64_t)std::max(device_sm_count(), 1) * 8 * 8 / t.batch);
  const dim3 grid((unsigned)std::min((reach + warps - 1) / warps, most), (unsigned)t.batch);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, tree_expand_kernel, t, static_cast<uint8_t*>(out));
}

}  // namespace mla
