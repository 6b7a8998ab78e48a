// api_step8.cu -- the C entries of a decoding step over a cache that may be held in 8 bits: appending with
// rotation, attention, sampling.  Argument checks and dispatch.
#include <cmath>

#include "api_checks.cuh"
#include "pkv_internal.cuh"

using namespace pkv;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A cache in 8 bits.
int check_cache8(const pkv_cache_desc* c) {
  if (!c) return PKV_ERR_INVALID_ARG;
  if (c->block_size != PKV_BLOCK_SIZE || c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0)
    return PKV_ERR_INVALID_ARG;
  if (c->num_blocks > (int64_t(1) << 40)) return PKV_ERR_INVALID_ARG;
  return c->dtype == PKV_E4M3 && c->head_dim == 128 ? PKV_OK : PKV_ERR_UNSUPPORTED;
}

int check_heads(const pkv_cache_desc* cache, int32_t num_q_heads, int32_t max_query_len) {
  if (num_q_heads <= 0 || num_q_heads % cache->num_kv_heads != 0 || max_query_len <= 0) return PKV_ERR_INVALID_ARG;
  return num_q_heads / cache->num_kv_heads > 16 ? PKV_ERR_UNSUPPORTED : PKV_OK;
}

// `rows` rows of `width` elements, `stride` apart, in bytes.
struct Rows {
  int64_t begin, end, stride, width;
  Rows(const void* p, int64_t rows, int64_t stride_, int64_t width_, int64_t size)
      : begin(static_cast<int64_t>(reinterpret_cast<uintptr_t>(p))), stride(stride_ * size), width(width_ * size) {
    end = begin + (rows - 1) * stride + width;
  }
  // No byte in common: one lies behind the other, or they are different columns of rows of the same length.
  bool apart(const Rows& o) const {
    if (end <= o.begin || o.end <= begin) return true;
    if (stride != o.stride) return false;
    const int64_t at = ((o.begin - begin) % stride + stride) % stride;
    return at >= width && at + o.width <= stride;
  }
};

}  // namespace

extern "C" {

int pkv_rope_append(const void* q, const void* k, const void* v, int32_t dtype, int64_t q_stride, int64_t k_stride,
                    int64_t v_stride, int32_t num_q_heads, const float* cos_sin, int32_t rot_dim, int32_t interleaved,
                    int64_t num_angles, const int32_t* positions, void* k_cache, void* v_cache, float* scales,
                    const pkv_cache_desc* cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                    const int32_t* seq_lens, const int32_t* query_start_loc, int32_t num_seqs, int64_t num_tokens,
                    int32_t max_query_len, void* q_out, int64_t q_out_stride, void* stream) {
  const bool eight = cache && cache->dtype == PKV_E4M3;
  int st = eight ? check_cache8(cache) : check_cache(cache);
  if (st) return st;
  if (num_tokens < 0 || num_seqs < 0) return PKV_ERR_INVALID_ARG;
  if (dtype != (eight ? PKV_BF16 : cache->dtype)) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  const int64_t d = cache->head_dim, size = dtype == PKV_F32 ? 4 : 2;
  if (num_seqs == 0 || max_blocks_per_seq <= 0 || max_query_len <= 0 || rot_dim < 0 || rot_dim > d || num_angles < 0)
    return PKV_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
  if (!k || !v || !k_cache || !v_cache || !block_tables || !seq_lens || !query_start_loc || (rot_dim > 0 && !cos_sin) ||
      (eight != (scales != nullptr)) || ((q == nullptr) != (q_out == nullptr)))
    return PKV_ERR_INVALID_ARG;
  const int64_t kv_width = cache->num_kv_heads * d;
  constexpr int64_t kFar = int64_t(1) << 28;  // (products with tokens fit 64 bits)
  if (num_tokens >= (int64_t(1) << 31) || k_stride > kFar || v_stride > kFar) return PKV_ERR_UNSUPPORTED;
  if (k_stride < kv_width || v_stride < kv_width || k_stride * size % 16 || v_stride * size % 16) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(cos_sin) ||
      !aligned(scales, 8))
    return PKV_ERR_INVALID_ARG;
  if (q) {
    if (num_q_heads <= 0) return PKV_ERR_INVALID_ARG;
    const int64_t q_width = num_q_heads * d;
    if (q_stride > kFar || q_out_stride > kFar) return PKV_ERR_UNSUPPORTED;
    if (q_stride < q_width || q_out_stride < q_width || q_stride * size % 16 || q_out_stride * size % 16 || !aligned16(q) ||
        !aligned16(q_out))
      return PKV_ERR_INVALID_ARG;
    const Rows out(q_out, num_tokens, q_out_stride, q_width, size);
    const bool in_place = q == q_out && q_stride == q_out_stride;
    if ((!in_place && !out.apart(Rows(q, num_tokens, q_stride, q_width, size))) ||
        !out.apart(Rows(k, num_tokens, k_stride, kv_width, size)) || !out.apart(Rows(v, num_tokens, v_stride, kv_width, size)))
      return PKV_ERR_INVALID_ARG;
  }
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  const AppendArgs a{q,       k,       v,      q_stride, k_stride,     v_stride,           q_out_stride, num_q_heads,     cos_sin,
                     rot_dim, interleaved != 0, num_angles, positions, k_cache, v_cache, scales, *cache, block_tables,
                     max_blocks_per_seq, seq_lens, query_start_loc, num_seqs, num_tokens, max_query_len, q_out};
  return launch_append(a, ctx->num_sms, ctx->err, as_stream(stream));
}

int pkv_q8_workspace(const pkv_cache_desc* cache, int32_t num_q_heads, int32_t max_query_len, int64_t* bytes) {
  int st = check_cache8(cache);
  if (!st) st = check_heads(cache, num_q_heads, max_query_len);
  if (st) return st;
  if (!bytes) return PKV_ERR_INVALID_ARG;
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  *bytes = static_cast<int64_t>(q8_workspace(*cache, num_q_heads, max_query_len, ctx->num_sms));
  return PKV_OK;
}

int paged_attention_q8(const void* q, const void* k_cache, const void* v_cache, const float* scales,
                       const pkv_cache_desc* cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                       const int32_t* seq_lens, const int32_t* query_start_loc, int32_t num_seqs, int32_t num_q_heads,
                       int64_t num_tokens, int32_t max_query_len, int32_t max_seq_len, float scale, void* out,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_cache8(cache);
  if (st) return st;
  if (num_tokens < 0 || num_seqs < 0 || !std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  st = check_heads(cache, num_q_heads, max_query_len);
  if (st) return st;
  if (num_seqs == 0 || max_blocks_per_seq <= 0 || max_seq_len <= 0) return PKV_ERR_INVALID_ARG;
  if (!q || !k_cache || !v_cache || !scales || !block_tables || !seq_lens || !query_start_loc || !out)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned(scales, 8))
    return PKV_ERR_INVALID_ARG;
  if (num_tokens >= (int64_t(1) << 31) || num_seqs >= (1 << 30)) return PKV_ERR_UNSUPPORTED;
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  const size_t need = q8_workspace(*cache, num_q_heads, max_query_len, ctx->num_sms);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < 0) return PKV_ERR_INVALID_ARG;
  if (static_cast<size_t>(workspace_bytes) < need) return PKV_ERR_NO_MEMORY;
  const AttnArgs a{q,        k_cache,    v_cache,         *cache,     block_tables, max_blocks_per_seq, seq_lens, query_start_loc,
                   num_seqs, num_q_heads, num_tokens, max_query_len, max_seq_len,  scale,              out};
  return launch_q8(a, scales, workspace, ctx->num_sms, ctx->err, as_stream(stream));
}

int pkv_sample(const void* logits, int32_t dtype, int64_t row_stride, const float* temperature, const int32_t* top_k,
               const float* top_p, const float* min_p, const float* uniform, int32_t num_seqs, int32_t vocab,
               int32_t* out_tokens, float* out_logprobs, void* stream) {
  if (num_seqs < 0 || vocab < 1) return PKV_ERR_INVALID_ARG;
  if (vocab > (1 << 20) || (dtype != PKV_F32 && dtype != PKV_BF16)) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!logits || !uniform || !out_tokens || row_stride < vocab || !aligned(logits, dtype == PKV_F32 ? 4 : 2))
    return PKV_ERR_INVALID_ARG;
  int st = PKV_OK;
  DeviceCtx* ctx = device_ctx(&st);
  if (!ctx) return st;
  const SampleArgs a{logits, dtype, row_stride, temperature, top_p, min_p, uniform, top_k, num_seqs, vocab, out_tokens,
                     out_logprobs};
  return launch_sample(a, ctx->num_sms, ctx->err, as_stream(stream));
}

}  // extern "C"
