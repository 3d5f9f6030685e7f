// Paged gather of fp4 latent cache entries, dequantized to bf16 rows of 576 (entry layout in
// include/mla_prefill.h): row t = [e2m1(x_i) * scale_(i / 32) | rope], addressed by the paged slot rule.
//
// Memory bound: 400 bytes read, 1152 written a row.  A warp has a row: lane l words l and 32 + l of the codes (128
// contiguous bytes a load, 512 a store), whose scales are bytes l / 4 and 8 + l / 4, and lanes 0-7 copy 16 bytes of rope.
// As many warps as rows: a row's latencies, slot then entry, lie beside other rows'.  (4 x 8192 rows 11.6 us in replayed
// graphs, 4.4 TB/s, 3 x 500 2.3; as first measured, 12.1 and 2.7, one wave of warps with two rows in flight each took 12.3
// and 3.4, four rows 14.3 and 4.6.)
#include "fp4.cuh"
#include "internal.h"
#include "paged.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 30;

__global__ void __launch_bounds__(kThreads)
gather_fp4_kernel(const uint8_t* __restrict__ cache, RowMap m, int64_t total_rows, uint8_t* __restrict__ out,
                  int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
  const int32_t cu_l = m.batch < 32 && lane <= m.batch ? __ldg(m.cu + lane) : 0x7fffffff;
  const int32_t st_l = m.batch < 32 && lane < m.batch ? __ldg(m.starts + lane) : 0;
  for (int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; row < total_rows; row += nwarps) {
    int64_t slot = 0;
    const bool have = resolve_slot(m, row, true, cu_l, st_l, &slot);   // the same row in every lane
    if (!have && lane == 0 && status) atomicOr(status, MLA_DEVSTAT_BAD_INDEX);
    uint32_t w0 = 0, w1 = 0;   // (zeros stay zeros under any scale that is not NaN)
    uint4 sc = make_uint4(0, 0, 0, 0), rope = sc;
    if (have) {
      const uint8_t* src = cache + slot * FP4_ENTRY;
      w0 = __ldg(reinterpret_cast<const uint32_t*>(src) + lane);
      w1 = __ldg(reinterpret_cast<const uint32_t*>(src) + 32 + lane);
      sc = __ldg(reinterpret_cast<const uint4*>(src + FP4_SCALES));
      if (lane < 8) rope = __ldg(reinterpret_cast<const uint4*>(src + FP4_ROPE) + lane);
    }
    uint4* dst = reinterpret_cast<uint4*>(out + row * (576 * 2));
    const int sh = 8 * ((lane >> 2) & 3);
    const uint32_t s0 = ((lane < 16 ? sc.x : sc.y) >> sh) & 0xffu, s1 = ((lane < 16 ? sc.z : sc.w) >> sh) & 0xffu;
    dst[lane] = fp4_values(w0, scale_bf16x2(s0));
    dst[32 + lane] = fp4_values(w1, scale_bf16x2(s1));
    if (lane < 8) dst[64 + lane] = rope;
  }
}

}  // namespace

cudaError_t launch_gather_fp4(const void* cache, int64_t num_blocks, int block_size, const int32_t* block_table,
                              int max_blocks_per_req, const int32_t* cu_seq_lens, const int32_t* chunk_starts,
                              int batch, int64_t total_tokens, void* out, int32_t* status, cudaStream_t stream) {
  if (total_tokens == 0) return cudaSuccess;
  const int64_t blocks = (total_tokens + kThreads / 32 - 1) / (kThreads / 32);
  const int grid = (int)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
  RowMap m{cu_seq_lens, chunk_starts, block_table, batch, max_blocks_per_req, block_size, num_blocks};
  gather_fp4_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const uint8_t*>(cache), m, total_tokens,
                                                   static_cast<uint8_t*>(out), status);
  return cudaGetLastError();
}

}  // namespace mla
