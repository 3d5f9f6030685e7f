// C ABI of the entry points for latent cache entries of several formats (declared in
// include/mla_prefill.h): argument checks and launches.
#include <cmath>

#include "internal.h"

using namespace mla;

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline int done(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

}  // namespace

extern "C" {

int mla_cache_append(void* cache, int entry_format, int64_t num_blocks, int block_size, const void* latent,
                     int64_t latent_stride, const void* norm_weight, float norm_eps, const int32_t* positions,
                     const float* cos_sin, int64_t max_positions, int interleaved, const int64_t* slot_mapping,
                     int64_t num_tokens, const void* q_rope, int64_t q_token_stride, int64_t q_head_stride,
                     int num_heads, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                     int32_t* status, void* stream) {
  if (entry_format < MLA_ENTRY_BF16 || entry_format > MLA_ENTRY_FP4 || num_blocks < 0 || block_size < 1 ||
      num_tokens < 0 || max_positions < 0 || num_heads < 0 || latent_stride < 576 || latent_stride % 8 != 0)
    return MLA_ERR_INVALID_ARG;
  if (norm_weight && (!std::isfinite(norm_eps) || norm_eps < 0.f)) return MLA_ERR_INVALID_ARG;
  if (num_heads > 0 && (q_token_stride % 8 != 0 || q_head_stride % 8 != 0 || q_out_token_stride % 8 != 0 ||
                        q_out_head_stride % 8 != 0 || q_token_stride < 0 || q_head_stride < 0 ||
                        q_out_token_stride < 0 || q_out_head_stride < 0))
    return MLA_ERR_INVALID_ARG;
  if (num_tokens > 0x7fffffff || num_heads > 65535 || num_blocks > INT64_MAX / 2048 / block_size ||
      q_token_stride > INT64_MAX >> 36 || q_head_stride > INT64_MAX >> 36 || q_out_token_stride > INT64_MAX >> 36 ||
      q_out_head_stride > INT64_MAX >> 36 || latent_stride > INT64_MAX >> 36)
    return MLA_ERR_UNSUPPORTED;
  if (!aligned(cache, entry_format == MLA_ENTRY_FP8 ? 8 : 16) || !aligned(latent, 16) || !aligned(norm_weight, 16) ||
      !aligned(positions, 4) || !aligned(cos_sin, 16) || !aligned(slot_mapping, 8) || !aligned(q_rope, 16) ||
      !aligned(q_out, 16) || !aligned(status, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (!latent || !positions || !slot_mapping || (max_positions > 0 && !cos_sin) || (num_blocks > 0 && !cache) ||
      (num_heads > 0 && (!q_rope || !q_out)))
    return MLA_ERR_INVALID_ARG;
  // Each value is read before it is written only where the two are the same.
  if (num_heads > 0 && q_rope == q_out && (q_token_stride != q_out_token_stride || q_head_stride != q_out_head_stride))
    return MLA_ERR_INVALID_ARG;
  // No two of the rows that are written share memory.
  if (num_heads > 0) {
    const int64_t heads = (num_heads - 1) * q_out_head_stride + 64, tokens = (num_tokens - 1) * q_out_token_stride + 64;
    if ((num_heads > 1 && q_out_head_stride < 64) || (num_tokens > 1 && q_out_token_stride < 64) ||
        (num_heads > 1 && num_tokens > 1 && q_out_token_stride < heads && q_out_head_stride < tokens))
      return MLA_ERR_INVALID_ARG;
  }
  AppendParams p;
  p.cache = static_cast<uint8_t*>(cache);
  p.num_slots = num_blocks * block_size;
  p.latent = static_cast<const __nv_bfloat16*>(latent);
  p.latent_stride = latent_stride;
  p.norm_weight = static_cast<const __nv_bfloat16*>(norm_weight);
  p.norm_eps = norm_eps;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.max_positions = max_positions;
  p.interleaved = interleaved != 0;
  p.slots = slot_mapping;
  p.num_tokens = num_tokens;
  p.q_rope = static_cast<const __nv_bfloat16*>(q_rope);
  p.q_token = q_token_stride;
  p.q_head = q_head_stride;
  p.num_heads = num_heads;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_out_token = q_out_token_stride;
  p.q_out_head = q_out_head_stride;
  p.status = status;
  return done(launch_append(p, entry_format, as_stream(stream)));
}

int mla_gather_latent_fp4(const void* cache, int64_t num_blocks, int block_size, int entry_bytes,
                          const int32_t* block_table, int max_blocks_per_req, const int32_t* cu_seq_lens,
                          const int32_t* chunk_starts, int batch, int64_t total_tokens, void* out, int32_t* status,
                          void* stream) {
  if (total_tokens < 0 || batch < 0 || num_blocks < 0 || block_size < 1 || max_blocks_per_req < 0)
    return MLA_ERR_INVALID_ARG;
  if (entry_bytes != 400) return MLA_ERR_UNSUPPORTED;
  if (total_tokens == 0) return MLA_OK;
  if (batch == 0) return MLA_ERR_SHAPE;
  if (!cache || !block_table || !cu_seq_lens || !chunk_starts || !out || !aligned(out, 16) || !aligned(cache, 16) ||
      !aligned(block_table, 4) || !aligned(cu_seq_lens, 4) || !aligned(chunk_starts, 4) || !aligned(status, 4))
    return MLA_ERR_INVALID_ARG;
  return done(launch_gather_fp4(cache, num_blocks, block_size, block_table, max_blocks_per_req, cu_seq_lens,
                                chunk_starts, batch, total_tokens, out, status, as_stream(stream)));
}

}  // extern "C"
