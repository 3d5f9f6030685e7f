// Paged gather of fp4 latent cache entries, dequantized to bf16 rows of 576 (entry layout in
// include/mla_prefill.h): row t = [e2m1(x_i) * scale_(i / 32) | rope], addressed by the paged slot rule.
//
// Memory bound: 400 bytes read, 1152 written a row.  One warp per row at a time, two rows in flight: lane l
// has words l and 32 + l of the codes (128 contiguous bytes a load, 512 a store), whose scales are bytes
// l / 4 and 8 + l / 4, and lanes 0-7 copy 16 bytes of rope.  One wave of resident warps, as in the gather of
// fp8 entries.
#include "fp4.cuh"
#include "internal.h"
#include "paged.cuh"

namespace mla {
namespace {

constexpr int kRowsPerWarp = 2;
constexpr int kBlocksPerSm = 6;
constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
gather_fp4_kernel(const uint8_t* __restrict__ cache, RowMap m, int64_t total_rows, uint8_t* __restrict__ out,
                  int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
  const int32_t cu_l = m.batch < 32 && lane <= m.batch ? __ldg(m.cu + lane) : 0x7fffffff;
  const int32_t st_l = m.batch < 32 && lane < m.batch ? __ldg(m.starts + lane) : 0;
  for (int64_t base = warp * kRowsPerWarp; base < total_rows; base += nwarps * kRowsPerWarp) {
    uint32_t w[kRowsPerWarp][2];
    uint4 sc[kRowsPerWarp], rope[kRowsPerWarp];
#pragma unroll
    for (int u = 0; u < kRowsPerWarp; ++u) {
      const bool active = base + u < total_rows;
      int64_t slot = 0;
      const bool have = resolve_slot(m, base + u, active, cu_l, st_l, &slot);   // the same row in every lane
      if (active && !have && lane == 0 && status) atomicOr(status, MLA_DEVSTAT_BAD_INDEX);
      w[u][0] = w[u][1] = 0;   // (zeros stay zeros under any scale that is not NaN)
      sc[u] = rope[u] = make_uint4(0, 0, 0, 0);
      if (have) {
        const uint8_t* src = cache + slot * FP4_ENTRY;
        w[u][0] = __ldg(reinterpret_cast<const uint32_t*>(src) + lane);
        w[u][1] = __ldg(reinterpret_cast<const uint32_t*>(src) + 32 + lane);
        sc[u] = __ldg(reinterpret_cast<const uint4*>(src + FP4_SCALES));
        if (lane < 8) rope[u] = __ldg(reinterpret_cast<const uint4*>(src + FP4_ROPE) + lane);
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsPerWarp; ++u) {
      if (base + u >= total_rows) break;
      uint4* dst = reinterpret_cast<uint4*>(out + (base + u) * (576 * 2));
      const int sh = 8 * ((lane >> 2) & 3);
      const uint32_t s0 = ((lane < 16 ? sc[u].x : sc[u].y) >> sh) & 0xffu, s1 = ((lane < 16 ? sc[u].z : sc[u].w) >> sh) & 0xffu;
      dst[lane] = fp4_values(w[u][0], scale_bf16x2(s0));
      dst[32 + lane] = fp4_values(w[u][1], scale_bf16x2(s1));
      if (lane < 8) dst[64 + lane] = rope[u];
    }
  }
}

}  // namespace

cudaError_t launch_gather_fp4(const void* cache, int64_t num_blocks, int block_size, const int32_t* block_table,
                              int max_blocks_per_req, const int32_t* cu_seq_lens, const int32_t* chunk_starts,
                              int batch, int64_t total_tokens, void* out, int32_t* status, cudaStream_t stream) {
  if (total_tokens == 0) return cudaSuccess;
  const int sms = device_sm_count();
  const int64_t warps_needed = (total_tokens + kRowsPerWarp - 1) / kRowsPerWarp;
  const int64_t blocks_needed = (warps_needed + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = (int64_t)(sms > 0 ? sms : 148) * kBlocksPerSm;
  const int grid = (int)(blocks_needed < cap ? blocks_needed : cap);
  RowMap m{cu_seq_lens, chunk_starts, block_table, batch, max_blocks_per_req, block_size, num_blocks};
  gather_fp4_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const uint8_t*>(cache), m, total_tokens,
                                                   static_cast<uint8_t*>(out), status);
  return cudaGetLastError();
}

}  // namespace mla
