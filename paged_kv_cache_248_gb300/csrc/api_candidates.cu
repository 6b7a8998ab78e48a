// api_candidates.cu -- the C entries for requests with several candidate continuations:
// drafted trees, the accepted path, beams and forked tables.  Argument checks and dispatch.
#include <cmath>

#include "api_checks.cuh"
#include "pkv_internal.cuh"

using namespace pkv;

namespace {

constexpr int32_t kMaxSelect = 64, kMaxBeams = 64, kMaxForkRows = 4096, kMaxNewTokens = 65536;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

int check_workspace(const void* ws, int64_t have, size_t need) {
  if (!ws || !aligned(ws, 256) || have < 0) return PKV_ERR_INVALID_ARG;
  return static_cast<size_t>(have) < need ? PKV_ERR_NO_MEMORY : PKV_OK;
}

int check_beams(int32_t num_seqs, int32_t num_beams, int32_t vocab, int32_t num_select) {
  if (num_seqs < 0 || num_beams < 1 || vocab < 1 || num_select < 1) return PKV_ERR_INVALID_ARG;
  if (num_beams > kMaxBeams || num_select > kMaxSelect) return PKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_beams) * vocab >= (int64_t(1) << 31)) return PKV_ERR_UNSUPPORTED;
  // blocks of 1024 logits are numbered in 32 bits
  const int64_t rows = static_cast<int64_t>(num_seqs) * num_beams;
  return rows * (vocab / 1024 + 1) >= (int64_t(1) << 31) ? PKV_ERR_UNSUPPORTED : PKV_OK;
}

int check_tree(const pkv_cache_desc* cache, int32_t num_q_heads, int32_t max_query_len) {
  const int st = check_cache(cache);
  if (st) return st;
  if (num_q_heads <= 0 || num_q_heads % cache->num_kv_heads != 0 || max_query_len <= 0) return PKV_ERR_INVALID_ARG;
  if (num_q_heads / cache->num_kv_heads > 16) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

}  // namespace

extern "C" {

int pkv_tree_mask(const int32_t* parents, const int32_t* query_start_loc, int32_t num_seqs, int64_t num_tokens,
                  uint64_t* mask, int32_t mask_words, int32_t* depths, void* stream) {
  if (num_tokens < 0 || num_seqs < 0 || mask_words < 1) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (num_seqs == 0 || !parents || !query_start_loc || !mask || !aligned(mask, 8)) return PKV_ERR_INVALID_ARG;
  int st = PKV_OK;
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  return launch_tree_mask(parents, query_start_loc, num_seqs, num_tokens, mask, mask_words, depths, ctx->err,
                          as_stream(stream));
}

int pkv_tree_workspace(const pkv_cache_desc* cache, int32_t num_q_heads, int32_t max_query_len, int64_t* bytes) {
  int st = check_tree(cache, num_q_heads, max_query_len);
  if (st) return st;
  if (!bytes) return PKV_ERR_INVALID_ARG;
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  *bytes = static_cast<int64_t>(tree_workspace(*cache, num_q_heads, max_query_len, ctx->num_sms));
  return PKV_OK;
}

int paged_attention_tree(const void* q, const void* k_cache, const void* v_cache, const pkv_cache_desc* cache,
                         const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                         const int32_t* query_start_loc, const uint64_t* tree_mask, int32_t mask_words,
                         int32_t num_seqs, int32_t num_q_heads, int64_t num_tokens, int32_t max_query_len,
                         int32_t max_seq_len, float scale, void* out, void* workspace, int64_t workspace_bytes,
                         void* stream) {
  int st = check_cache(cache);
  if (st) return st;
  if (num_tokens < 0 || num_seqs < 0 || !std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  st = check_tree(cache, num_q_heads, max_query_len);
  if (st) return st;
  if (num_seqs == 0 || max_blocks_per_seq <= 0 || max_seq_len <= 0 || mask_words < 1 ||
      static_cast<int64_t>(mask_words) * 64 < max_query_len)
    return PKV_ERR_INVALID_ARG;
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !query_start_loc || !tree_mask || !out)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned(tree_mask, 8))
    return PKV_ERR_INVALID_ARG;
  if (num_tokens >= (int64_t(1) << 31) || num_seqs >= (1 << 30)) return PKV_ERR_UNSUPPORTED;
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  st = check_workspace(workspace, workspace_bytes, tree_workspace(*cache, num_q_heads, max_query_len, ctx->num_sms));
  if (st) return st;
  const TreeArgs t{{q,        k_cache,    v_cache,         *cache,     block_tables, max_blocks_per_seq, seq_lens, query_start_loc,
                    num_seqs, num_q_heads, num_tokens, max_query_len, max_seq_len,  scale,              out},
                   tree_mask, mask_words};
  return launch_tree_attention(t, workspace, ctx->num_sms, ctx->err, as_stream(stream));
}

int pkv_compact_path(const int32_t* path, int32_t max_path, const int32_t* path_lens, const int32_t* block_tables,
                     int32_t max_blocks_per_seq, const int32_t* seq_lens, const int32_t* query_start_loc,
                     int32_t num_seqs, void* k_cache, void* v_cache, const pkv_cache_desc* cache, int32_t num_layers,
                     int32_t* new_seq_lens, void* stream) {
  int st = check_cache(cache);
  if (st) return st;
  if (num_seqs < 0 || num_layers < 1 || num_layers > 65535 || max_path < 0) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  if (max_blocks_per_seq <= 0 || (max_path > 0 && !path) || !path_lens || !block_tables || !seq_lens ||
      !query_start_loc || !k_cache || !v_cache || !new_seq_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
  const int64_t len_bytes = static_cast<int64_t>(num_seqs) * 4;
  if (overlap(new_seq_lens, len_bytes, seq_lens, len_bytes) || overlap(new_seq_lens, len_bytes, path_lens, len_bytes) ||
      overlap(new_seq_lens, len_bytes, query_start_loc, len_bytes + 4))
    return PKV_ERR_INVALID_ARG;
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  return launch_compact_path(path, max_path, path_lens, block_tables, max_blocks_per_seq, seq_lens, query_start_loc,
                             num_seqs, k_cache, v_cache, *cache, num_layers, new_seq_lens, ctx->err,
                             as_stream(stream));
}

int pkv_beam_workspace(int32_t num_seqs, int32_t num_beams, int32_t vocab, int32_t num_select, int64_t* bytes) {
  int st = check_beams(num_seqs, num_beams, vocab, num_select);
  if (st) return st;
  if (!bytes) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) {
    *bytes = 0;
    return PKV_OK;
  }
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  *bytes = static_cast<int64_t>(beam_workspace(num_seqs, num_beams, vocab, num_select, ctx->num_sms));
  return PKV_OK;
}

int pkv_beam_select(const void* logits, int32_t dtype, int64_t row_stride, const float* cum_scores,
                    const uint8_t* finished, int32_t eos_token, int32_t num_seqs, int32_t num_beams, int32_t vocab,
                    int32_t num_select, float* out_scores, int32_t* out_parents, int32_t* out_tokens, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  int st = check_beams(num_seqs, num_beams, vocab, num_select);
  if (st) return st;
  if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!logits || !cum_scores || !out_scores || !out_parents || !out_tokens || row_stride < vocab ||
      !aligned(logits, dtype == PKV_F32 ? 4 : 2))
    return PKV_ERR_INVALID_ARG;
  if (finished && (eos_token < 0 || eos_token >= vocab)) return PKV_ERR_INVALID_ARG;
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  st = check_workspace(workspace, workspace_bytes,
                       beam_workspace(num_seqs, num_beams, vocab, num_select, ctx->num_sms));
  if (st) return st;
  const BeamArgs a{logits, dtype, row_stride, cum_scores, finished, eos_token, num_seqs, num_beams, vocab,
                   num_select, out_scores, out_parents, out_tokens};
  return launch_beam_select(a, workspace, ctx->num_sms, as_stream(stream));
}

int pkv_fork_workspace(int32_t num_rows, int64_t* bytes) {
  if (num_rows < 0 || !bytes) return PKV_ERR_INVALID_ARG;
  if (num_rows > kMaxForkRows) return PKV_ERR_UNSUPPORTED;
  *bytes = static_cast<int64_t>(fork_workspace(num_rows));
  return PKV_OK;
}

int pkv_fork_tables(const int32_t* block_tables, const int32_t* seq_lens, int32_t num_rows, int32_t max_blocks_per_seq,
                    const int32_t* parents, int32_t num_new, int32_t* ref_counts, int32_t* new_block_tables,
                    int32_t* new_seq_lens, void* k_cache, void* v_cache, const pkv_cache_desc* cache,
                    int32_t num_layers, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st) return st;
  if (num_rows < 0 || num_new < 0 || num_layers < 1) return PKV_ERR_INVALID_ARG;
  if (num_rows == 0) return PKV_OK;
  if (num_rows > kMaxForkRows || num_new > kMaxNewTokens || cache->num_blocks >= (int64_t(1) << 31))
    return PKV_ERR_UNSUPPORTED;
  if (max_blocks_per_seq <= 0 || !block_tables || !seq_lens || !parents || !ref_counts || !new_block_tables ||
      !new_seq_lens || (k_cache == nullptr) != (v_cache == nullptr))
    return PKV_ERR_INVALID_ARG;
  if (max_blocks_per_seq > (1 << 26) || num_layers > 8191) return PKV_ERR_UNSUPPORTED;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
  const int64_t lens = static_cast<int64_t>(num_rows) * 4, tables = lens * max_blocks_per_seq;
  if (overlap(block_tables, tables, new_block_tables, tables) || overlap(seq_lens, lens, new_seq_lens, lens) ||
      overlap(parents, lens, new_seq_lens, lens))
    return PKV_ERR_INVALID_ARG;
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  st = check_workspace(workspace, workspace_bytes, fork_workspace(num_rows));
  if (st) return st;
  return launch_fork_tables(block_tables, seq_lens, num_rows, max_blocks_per_seq, parents, num_new, ref_counts,
                            new_block_tables, new_seq_lens, k_cache, v_cache, *cache, num_layers, workspace,
                            ctx->num_sms, ctx->err, as_stream(stream));
}

}  // extern "C"
