// C ABI of the speculative-decoding entry points (declared in include/mla_prefill.h):
// argument checks and launches.
#include <cmath>

#include "internal.h"

using namespace mla;

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && a_bytes > 0 && b_bytes > 0 && (x < y ? y - x < (uintptr_t)a_bytes : x - y < (uintptr_t)b_bytes);
}
inline int done(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

}  // namespace

extern "C" {

int mla_block_table_update(const int32_t* seq_lens, const int32_t* new_lens, int batch, int block_size,
                           int32_t* block_table, int max_blocks_per_req, int32_t* num_held, int32_t* free_blocks,
                           int32_t free_capacity, int32_t* free_count, int32_t* qo_indptr, int32_t* kv_lens,
                           int64_t* slot_mapping, int64_t num_tokens, int32_t* status, void* stream) {
  if (batch < 0 || block_size < 1 || max_blocks_per_req < 0 || free_capacity < 0 || num_tokens < 0)
    return MLA_ERR_INVALID_ARG;
  if (batch > kMaxTableBatch || (int64_t)batch * max_blocks_per_req > 0x7fffffff || num_tokens > 0x7fffffff)
    return MLA_ERR_UNSUPPORTED;
  if (!aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(num_held, 4) ||
      !aligned(free_blocks, 4) || !aligned(free_count, 4) || !aligned(qo_indptr, 4) || !aligned(kv_lens, 4) ||
      !aligned(slot_mapping, 8) || !aligned(status, 4))
    return MLA_ERR_INVALID_ARG;
  if (!free_count || (num_tokens > 0 && !slot_mapping) || (free_capacity > 0 && !free_blocks))
    return MLA_ERR_INVALID_ARG;
  if (batch > 0 && (!seq_lens || !new_lens || !num_held || (max_blocks_per_req > 0 && !block_table)))
    return MLA_ERR_INVALID_ARG;
  // The lengths are read again after outputs are written.
  struct Written { const void* at; int64_t bytes; };
  const int64_t b = batch;
  const Written written[] = {{block_table, 4 * b * max_blocks_per_req}, {num_held, 4 * b},
                             {free_blocks, 4 * (int64_t)free_capacity}, {free_count, 4},
                             {qo_indptr, 4 * (b + 1)}, {kv_lens, 4 * b}, {slot_mapping, 8 * num_tokens}, {status, 4}};
  for (const Written& w : written)
    if (overlap(seq_lens, 4 * b, w.at, w.bytes) || overlap(new_lens, 4 * b, w.at, w.bytes)) return MLA_ERR_INVALID_ARG;
  TablesParams p;
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.batch = batch;
  p.block_size = block_size;
  p.block_table = block_table;
  p.max_blocks = max_blocks_per_req;
  p.num_held = num_held;
  p.free_blocks = free_blocks;
  p.free_capacity = free_capacity;
  p.free_count = free_count;
  p.qo_indptr = qo_indptr;
  p.kv_lens = kv_lens;
  p.slot_mapping = slot_mapping;
  p.num_tokens = num_tokens;
  p.status = status;
  return done(launch_tables(p, as_stream(stream)));
}

int mla_tree_mask(const int32_t* parents, const int32_t* qo_indptr, const int32_t* kv_lens, int batch,
                  int64_t total_rows, int mask_words, int64_t* tree_mask, int32_t* positions, int32_t* status,
                  void* stream) {
  if (batch < 0 || total_rows < 0 || mask_words < 1) return MLA_ERR_INVALID_ARG;
  if (total_rows > 0x7fffffff || mask_words > kMaxMaskWords) return MLA_ERR_UNSUPPORTED;
  if (!aligned(parents, 4) || !aligned(qo_indptr, 4) || !aligned(kv_lens, 4) || !aligned(tree_mask, 8) ||
      !aligned(positions, 4) || !aligned(status, 4))
    return MLA_ERR_INVALID_ARG;
  if (batch == 0 || total_rows == 0) return MLA_OK;
  if (!parents || !qo_indptr || !tree_mask) return MLA_ERR_INVALID_ARG;
  return done(launch_tree_mask(parents, qo_indptr, kv_lens, batch, total_rows, mask_words, tree_mask, positions, status,
                               as_stream(stream)));
}

int mla_tree_workspace(int64_t total_rows, int num_heads, int64_t* bytes) {
  if (!bytes || total_rows < 0 || num_heads < 1 || num_heads > 65535) return MLA_ERR_INVALID_ARG;
  if (total_rows > kMaxTreePairs || total_rows * num_heads > kMaxTreePairs) return MLA_ERR_UNSUPPORTED;
  const int64_t n = tree_workspace_bytes();
  if (n <= 0) return MLA_ERR_CUDA;
  *bytes = n;
  return MLA_OK;
}

int mla_tree_attention(const void* q_abs, const void* cache, int64_t num_blocks, int block_size,
                       const int32_t* block_table, int max_blocks_per_req, const int32_t* qo_indptr,
                       const int32_t* kv_lens, const int64_t* tree_mask, int mask_words, int batch, int64_t total_rows,
                       int num_heads, float sm_scale, float logits_soft_cap, void* o_lat, float* lse, void* workspace,
                       int64_t workspace_bytes, int32_t* status, void* stream) {
  if (batch < 0 || total_rows < 0 || num_blocks < 0 || block_size < 1 || max_blocks_per_req < 0 || num_heads < 1 ||
      num_heads > 65535 || !std::isfinite(sm_scale) || !(sm_scale > 0.f) || !std::isfinite(logits_soft_cap))
    return MLA_ERR_INVALID_ARG;
  if (tree_mask ? (mask_words < 1) : (mask_words != 0)) return MLA_ERR_INVALID_ARG;
  // Slots are TMA row coordinates (int32), and one past the last slot marks a missing row;
  // so are the (row, head) pairs.
  if (total_rows > kMaxTreePairs || total_rows * num_heads > kMaxTreePairs || mask_words > kMaxMaskWords ||
      num_blocks > 0x7fffffff || num_blocks * (int64_t)block_size >= 0x7fffffff ||
      (int64_t)max_blocks_per_req * block_size > 0x7fffff00)
    return MLA_ERR_UNSUPPORTED;
  if (!aligned(q_abs, 16) || !aligned(cache, 16) || !aligned(o_lat, 16) || !aligned(workspace, 32) ||
      !aligned(block_table, 4) || !aligned(qo_indptr, 4) || !aligned(kv_lens, 4) || !aligned(tree_mask, 8) ||
      !aligned(lse, 4) || !aligned(status, 4))
    return MLA_ERR_INVALID_ARG;
  if (batch == 0 || total_rows == 0) return MLA_OK;
  if (!q_abs || !o_lat || !qo_indptr || !kv_lens || !workspace) return MLA_ERR_INVALID_ARG;
  if (max_blocks_per_req > 0 && num_blocks > 0 && (!cache || !block_table)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < tree_workspace_bytes()) return MLA_ERR_INVALID_ARG;
  TreeParams p;
  p.q = static_cast<const __nv_bfloat16*>(q_abs);
  p.cache = static_cast<const __nv_bfloat16*>(cache);
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.block_table = block_table;
  p.max_blocks = num_blocks > 0 ? max_blocks_per_req : 0;
  p.qo_indptr = qo_indptr;
  p.kv_lens = kv_lens;
  p.mask = tree_mask;
  p.mask_words = mask_words;
  p.batch = batch;
  p.total_rows = total_rows;
  p.num_heads = num_heads;
  p.sm_scale = sm_scale;
  p.soft_cap = logits_soft_cap > 0.f ? logits_soft_cap : 0.f;
  p.o = static_cast<__nv_bfloat16*>(o_lat);
  p.lse = lse;
  p.workspace = workspace;
  p.status = status;
  return done(launch_tree_attention(p, as_stream(stream)));
}

int mla_tree_commit(void* cache, int num_layers, int64_t layer_stride, int64_t num_blocks, int block_size,
                    int entry_dim, const int32_t* block_table, int max_blocks_per_req, const int32_t* seq_lens,
                    const int32_t* accepted, const int32_t* accepted_counts, int batch, int max_accepted,
                    int32_t* status, void* stream) {
  if (num_layers < 0 || num_blocks < 0 || block_size < 1 || entry_dim < 8 || entry_dim % 8 != 0 ||
      max_blocks_per_req < 0 || batch < 0 || max_accepted < 0)
    return MLA_ERR_INVALID_ARG;
  if (num_layers > 1 && (layer_stride % 8 != 0 || layer_stride / entry_dim / block_size < num_blocks))
    return MLA_ERR_INVALID_ARG;
  if (batch > 65535 || (int64_t)num_layers * (entry_dim / 8) > 0x7fffffff || num_blocks > 0x7fffffff)
    return MLA_ERR_UNSUPPORTED;
  if (!aligned(cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(accepted, 4) ||
      !aligned(accepted_counts, 4) || !aligned(status, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_layers == 0 || batch == 0 || max_accepted == 0) return MLA_OK;
  if (!cache || !seq_lens || !accepted || !accepted_counts || (max_blocks_per_req > 0 && !block_table))
    return MLA_ERR_INVALID_ARG;
  CommitParams p;
  p.cache = static_cast<uint4*>(cache);
  p.num_layers = num_layers;
  p.layer_chunks = layer_stride / 8;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.row_chunks = entry_dim / 8;
  p.block_table = block_table;
  p.max_blocks = max_blocks_per_req;
  p.seq_lens = seq_lens;
  p.paths = accepted;
  p.counts = accepted_counts;
  p.max_accept = max_accepted;
  p.status = status;
  return done(launch_tree_commit(p, batch, as_stream(stream)));
}

}  // extern "C"
