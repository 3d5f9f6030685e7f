// C ABI of the entry points for latent cache entries of several formats (declared in
// include/mla_prefill.h): argument checks and launches.
#include <algorithm>
#include <cmath>

#include "internal.h"

using namespace mla;

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline int done(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

// Bytes as a grid of pieces: piece (i, j), i < n[0], j < n[1], is [at + i s[0] + j s[1], + width).
struct Pieces {
  const void* at;
  int64_t n[2], s[2], width;
};
inline Pieces bytes(const void* at, int64_t n) { return {at, {1, 1}, {0, 0}, n}; }

inline int64_t div_down(int64_t a, int64_t b) { return a / b - (a % b < 0); }
// Whether lo < c + k s < hi for some k in [first, last]; s >= 0.
bool reaches(int64_t c, int64_t s, int64_t first, int64_t last, int64_t lo, int64_t hi) {
  if (s == 0) return first <= last && lo < c && c < hi;
  return std::max(first, div_down(lo - c, s) + 1) <= std::min(last, div_down(hi - c - 1, s));
}

// Whether two grids share a byte.  Exact where they have a stride in common (rows of one matrix, or of the same number of
// heads) and few pieces lie close to one another; other grids do if the ranges that they lie in do.
constexpr int64_t MOST_STEPS = 1 << 18;
bool overlap(Pieces a, Pieces b) {
  for (int k = 0; k < 2; ++k) {   // the stride of a single piece is any
    if (a.n[k] == 1) a.s[k] = b.s[k];
    if (b.n[k] == 1) b.s[k] = a.s[k];
  }
  if (!a.at || !b.at || a.width <= 0 || b.width <= 0 || a.n[0] <= 0 || a.n[1] <= 0 || b.n[0] <= 0 || b.n[1] <= 0) return false;
  auto reach = [](const Pieces& p, int k) { return (p.n[k] - 1) * p.s[k]; };
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at));
  if (d >= reach(a, 0) + reach(a, 1) + a.width || -d >= reach(b, 0) + reach(b, 1) + b.width) return false;
  const bool same[2] = {a.s[0] == b.s[0], a.s[1] == b.s[1]};
  if (!same[0] && !same[1]) return true;
  // Pieces k apart in a dimension e with a common stride; in the other one each of a's against all of b's, or, where that
  // stride is common too, one against all differences.
  int e = same[0] ? 0 : 1;
  if (same[0] && same[1] && a.n[1] + b.n[1] < a.n[0] + b.n[0]) e = 1;   // (the fewer steps)
  const int o = 1 - e;
  const int64_t far_a = reach(a, o) + a.width, far_b = reach(b, o) + b.width, s = a.s[e];
  int64_t first = -(a.n[e] - 1), last = b.n[e] - 1;
  if (s > 0) {
    first = std::max(first, div_down(-far_b - d, s) + 1);
    last = std::min(last, div_down(far_a - d - 1, s));
  } else {
    first = last = 0;
  }
  if (last >= first && (last - first + 1) * (same[o] ? 1 : a.n[o]) > MOST_STEPS) return true;
  for (int64_t k = first; k <= last; ++k) {
    if (same[o]) {
      if (reaches(d + k * s, a.s[o], -(a.n[o] - 1), b.n[o] - 1, -b.width, a.width)) return true;
    } else {
      for (int64_t i = 0; i < a.n[o]; ++i)
        if (reaches(d + k * s - i * a.s[o], b.s[o], 0, b.n[o] - 1, -b.width, a.width)) return true;
    }
  }
  return false;
}

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
  // No two of the rows that are written share memory.
  if (num_heads > 0) {
    const int64_t heads = (num_heads - 1) * q_out_head_stride + 64, tokens = (num_tokens - 1) * q_out_token_stride + 64;
    if ((num_heads > 1 && q_out_head_stride < 64) || (num_tokens > 1 && q_out_token_stride < 64) ||
        (num_heads > 1 && num_tokens > 1 && q_out_token_stride < heads && q_out_head_stride < tokens))
      return MLA_ERR_INVALID_ARG;
  }
  // What is written is read by nobody and written by nobody else; but the queries may be rotated in place, where each
  // value is read before it is written.
  const int64_t entry = entry_format == MLA_ENTRY_BF16 ? 1152 : entry_format == MLA_ENTRY_FP8 ? 648 : 400;
  const Pieces rows = bytes(cache, num_blocks * block_size * entry), state = bytes(status, 4);
  const Pieces out = {num_heads > 0 ? q_out : nullptr, {num_tokens, num_heads}, {2 * q_out_token_stride, 2 * q_out_head_stride}, 128};
  const Pieces in = {num_heads > 0 ? q_rope : nullptr, {num_tokens, num_heads}, {2 * q_token_stride, 2 * q_head_stride}, 128};
  const Pieces read[] = {{latent, {num_tokens, 1}, {2 * latent_stride, 0}, 1152}, bytes(norm_weight, 1024),
                         bytes(positions, 4 * num_tokens), bytes(cos_sin, 256 * std::min(max_positions, INT64_MAX >> 16)), bytes(slot_mapping, 8 * num_tokens)};
  for (const Pieces& r : read)
    if (overlap(rows, r) || overlap(out, r) || overlap(state, r)) return MLA_ERR_INVALID_ARG;
  if (overlap(rows, in) || overlap(rows, out) || overlap(rows, state) || overlap(state, in) || overlap(state, out))
    return MLA_ERR_INVALID_ARG;
  const bool in_place = q_rope == q_out && q_token_stride == q_out_token_stride && q_head_stride == q_out_head_stride;
  if (!in_place && overlap(in, out)) return MLA_ERR_INVALID_ARG;
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
