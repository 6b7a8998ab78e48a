/*
 * pkv.h -- C ABI of libpkv: the PagedAttention hot path on one GB300 (sm_103a).
 *
 * The KV cache of every request lives in fixed 16-token physical blocks reached
 * through a per-request block table; requests that share a prefix point at the
 * same physical blocks ("vLLM's PagedAttention" teardown, section "PagedAttention:
 * the KV cache is paged, like virtual memory").  One batch mixes chunked prefills
 * and decodes freely (same page, section "Continuous batching").  This library
 * implements the data-parallel steps of that path as CUDA kernels:
 *
 *   pkv_slot_mapping  logical position -> physical slot through the block table
 *   pkv_write         scatter new tokens' K/V rows into their slots
 *   pkv_copy_blocks   copy-on-write block copy ("The 1960s Operating System
 *                     Trick ..." page, Technical Details: Copy-on-Write)
 *   paged_attention   attention for one continuously-batched step: split-KV GQA
 *                     decode with online softmax and a cross-split merge, plus
 *                     causal chunked prefill, gathering K/V through block tables
 *   paged_attention_cascade  the same, reading each shared prompt prefix once
 *   paged_attention_step     slot mapping + K/V scatter + attention in one call
 *   paged_attention_step_cow the same, after the step's copy-on-write block copies
 *
 * and the steps a request with several candidate continuations adds to it:
 *
 *   pkv_tree_mask          who is whose ancestor in a request's tree of drafted tokens
 *   paged_attention_tree   attention of such trees over the paged cache
 *   pkv_compact_path       the accepted path of a tree moved together in the cache
 *   pkv_beam_select        the best continuations of a request's beams
 *   pkv_fork_tables        block tables after the beams they continue: reference
 *                          counts, freed and fresh blocks, copy-on-write
 *
 * and a decoding step over a cache that may be held in 8 bits:
 *
 *   pkv_rope_append        new queries and keys rotated by their positions, keys and values
 *                          put into the cache (of any type, 8 bits among them)
 *   paged_attention_q8     paged_attention over a cache in 8 bits
 *   pkv_sample             tokens drawn from logits: temperature, top-k, min-p, top-p
 *
 * Conventions for every call
 *  - Pointers named as device pointers must point to device memory of the current
 *    CUDA device; `stream` is a cudaStream_t (NULL = legacy default stream).  All
 *    compute calls are asynchronous on `stream`.
 *  - Ownership: the caller owns every buffer it passes.  The library owns only a
 *    per-device workspace for split-KV partials and a per-device error word; both
 *    are created on first use and released by pkv_shutdown().
 *  - Errors: an argument error found on the host returns a non-zero pkv_status
 *    and launches nothing.  Data errors found on the device (a block id outside
 *    [0, num_blocks), a slot past the pool, seq_len < q_len, more blocks than a
 *    table row holds) never trap: they set bits in the device error word, the
 *    affected outputs are zeroed or skipped, and pkv_get_last_error() reports them.
 *  - No call allocates device memory except paged_attention(), which grows the
 *    workspace when a larger batch needs it (never during stream capture).
 *  - A call that takes a `workspace` keeps its scratch there and nowhere else: the
 *    matching *_workspace() call says how many bytes it needs, its contents need no
 *    initialisation and mean nothing afterwards.  Calls that may overlap on the GPU
 *    (two streams, two captured graphs) take one each.
 *
 * Cache layout (a reading where the pages are silent): k_cache and v_cache are
 * each [num_blocks][num_kv_heads][16][head_dim], row-major, so that one
 * (block, kv head) is a contiguous 16 x head_dim tile.
 * Supported element types: fp32 with head_dim 64 or 128; bf16 with head_dim 128.  A cache
 * in 8 bits (PKV_E4M3, head_dim 128) is served by pkv_rope_append and paged_attention_q8; any
 * other call refuses it.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define PKV_API __attribute__((visibility("default")))
#else
#define PKV_API
#endif

typedef enum {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1, /* null pointer, bad size, inconsistent shape */
  PKV_ERR_UNSUPPORTED = 2, /* dtype / head_dim / group size not built */
  PKV_ERR_INDEX = 3,       /* device saw a bad block id, slot or length */
  PKV_ERR_CUDA = 4,        /* a CUDA runtime call failed */
  PKV_ERR_NO_MEMORY = 5,   /* workspace could not be grown */
  PKV_ERR_TIMEOUT = 6      /* a kernel gave up a bounded wait (internal error) */
} pkv_status;

typedef enum {
  PKV_F32 = 0,
  PKV_BF16 = 1,
  PKV_E4M3 = 2 /* 8 bits: sign, 4 of exponent, 3 of mantissa; a value is its code times a scale */
} pkv_dtype;

#define PKV_BLOCK_SIZE 16

/* Shape of the paged KV pool (host struct). */
typedef struct {
  int64_t num_blocks;   /* physical blocks in the pool */
  int32_t block_size;   /* tokens per block; must be 16 */
  int32_t num_kv_heads; /* KV heads */
  int32_t head_dim;     /* elements per head row */
  int32_t dtype;        /* pkv_dtype of the cache, q, k, v and out */
} pkv_cache_desc;

/*
 * Slot mapping ("vLLM's PagedAttention" teardown, section "PagedAttention": the
 * block table maps logical token positions to physical block ids).
 * For request i with q_i = query_start_loc[i+1] - query_start_loc[i] new tokens
 * and context length seq_lens[i] (which counts those new tokens), new token j sits
 * at position p = seq_lens[i] - q_i + j and gets
 *     slot_mapping[query_start_loc[i] + j] = block_tables[i][p / 16] * 16 + p % 16.
 * block_tables    device int32 [num_seqs][max_blocks_per_seq], row-major
 * seq_lens        device int32 [num_seqs]
 * query_start_loc device int32 [num_seqs + 1], non-decreasing, [0] == 0,
 *                 [num_seqs] == num_tokens
 * slot_mapping    device int64 [num_tokens], written
 * Device errors: p / 16 >= max_blocks_per_seq or a negative block id give slot -1
 * and PKV_ERR_INDEX in the error word.
 */
PKV_API int pkv_slot_mapping(const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                     const int32_t* query_start_loc, int32_t num_seqs, int64_t num_tokens,
                     int64_t* slot_mapping, void* stream);

/*
 * KV-slot scatter (same section: new tokens go to the slots their block table
 * names).  For each token t with slot_mapping[t] >= 0 and each kv head h:
 *     k_cache[slot / 16][h][slot % 16][:] = k[t][h][:]   (and v into v_cache)
 * Bit-exact copy.  A negative slot skips the token (padding).
 * k, v            device [num_tokens][num_kv_heads][head_dim], cache dtype, contiguous
 * slot_mapping    device int64 [num_tokens]
 * k_cache,v_cache device pool, layout above
 * Duplicate non-negative slots are a caller error (the surviving row is unspecified).
 * Device errors: slot >= num_blocks * 16 is skipped and flagged PKV_ERR_INDEX.
 */
PKV_API int pkv_write(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens, void* k_cache,
              void* v_cache, const pkv_cache_desc* cache, void* stream);

/*
 * Copy-on-write block copy ("The 1960s Operating System Trick ..." page, Technical
 * Details: samples share blocks until they diverge; only the blocks that change are
 * duplicated).  For i in [0, n): k_cache[dst[i]] = k_cache[src[i]] and the same for
 * v_cache, all heads and all 16 slots, bit-exact.
 * src, dst        device int32 [n]
 * Caller contract: dst entries are distinct and none appears in src, so the pairs
 * are independent and may run in any order.
 * Device errors: an id outside [0, num_blocks) skips the pair and flags PKV_ERR_INDEX.
 */
PKV_API int pkv_copy_blocks(const int32_t* src, const int32_t* dst, int64_t n, void* k_cache, void* v_cache,
                    const pkv_cache_desc* cache, void* stream);

/*
 * Attention for one continuously-batched step ("vLLM's PagedAttention" teardown,
 * sections "PagedAttention" and "Continuous batching": the kernel is handed a
 * per-request block table and gathers K/V from wherever the blocks live; one pass
 * mixes chunked prefills and decodes).
 * For request i (q_i query tokens, context seq_lens[i] including them), query token
 * j at position p = seq_lens[i] - q_i + j and query head h (kv head g = h / G,
 * G = num_q_heads / num_kv_heads):
 *     out[t][h][:] = sum_{u<=p} softmax_u(scale * q[t][h] . K_u) V_u
 * with K_u, V_u = cache[block_tables[i][u / 16]][g][u % 16][:].  Causal masking is
 * bottom-right aligned inside a chunk; a decode token (q_i == 1) sees all seq_lens[i]
 * keys.  Accumulation is fp32; out has the dtype of q.
 * q               device [num_tokens][num_q_heads][head_dim]
 * block_tables    device int32 [num_seqs][max_blocks_per_seq]
 * seq_lens        device int32 [num_seqs]
 * query_start_loc device int32 [num_seqs + 1]
 * max_query_len, max_seq_len  host upper bounds over the batch, used only to plan
 *                 the launch; results never depend on them beyond being bounds
 * out             device [num_tokens][num_q_heads][head_dim], written
 * Device errors: a bad block id, seq_len < q_len or ceil(seq_len/16) >
 * max_blocks_per_seq flags PKV_ERR_INDEX and zeroes the affected output rows.
 */
PKV_API int paged_attention(const void* q, const void* k_cache, const void* v_cache, const pkv_cache_desc* cache,
                    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                    const int32_t* query_start_loc, int32_t num_seqs, int32_t num_q_heads, int64_t num_tokens,
                    int32_t max_query_len, int32_t max_seq_len, float scale, void* out, void* stream);

/*
 * Shared-prefix groups for paged_attention_cascade (host struct of device arrays).
 * Requests that share a prompt prefix point at the same physical blocks ("vLLM's
 * PagedAttention" teardown, section "PagedAttention": a new request whose prefix
 * hashes match reuses the cached blocks), so those blocks need to be read only once
 * per step for all of them.  Group g is a prefix of prefix_num_blocks[g] full blocks
 * (P_g = 16 x that many tokens) whose physical ids are row g of prefix_block_tables;
 * its members are the request indices member_seqs[member_start[g] ..
 * member_start[g + 1]).
 *   prefix_block_tables  device int32 [num_groups][max_prefix_blocks]
 *   prefix_num_blocks    device int32 [num_groups], each in [1, max_prefix_blocks]
 *   member_start         device int32 [num_groups + 1], 0 = first <= ... <= last = num_members
 *   member_seqs          device int32 [num_members]
 */
typedef struct {
  const int32_t* prefix_block_tables;
  int32_t max_prefix_blocks;
  const int32_t* prefix_num_blocks;
  const int32_t* member_start;
  const int32_t* member_seqs;
  int32_t num_groups;
  int32_t num_members;
} pkv_prefix_groups;

/*
 * paged_attention_cascade -- paged_attention() with shared-prefix groups as a hint.
 * The output is paged_attention()'s (up to fp32 rounding order): the groups only
 * change how the work is done.  A member whose request is a decode (one query
 * token), whose context goes past the prefix (seq_len > P_g), which is listed once
 * in all groups, and whose block table starts with the group's prefix blocks has
 * its first P_g keys attended together with the other members of its group: one
 * tensor-core pass per (group, kv head) reads the prefix once and leaves a partial
 * softmax state per member, which the split merge folds with the member's own keys
 * (log-sum-exp merge, prefix first).  Any other listed request -- a prefill chunk,
 * a shorter context, a duplicate, a table that does not match, a malformed group --
 * is attended the ordinary way.  No counterpart on the pages beyond the sharing
 * itself; this is the cascade reading of it.
 * groups: NULL or num_groups == 0 or num_members == 0 = paged_attention().  The fp32
 * path ignores the groups.  Host errors as paged_attention(), plus PKV_ERR_INVALID_ARG
 * for negative counts, null group arrays or max_prefix_blocks < 1.
 */
PKV_API int paged_attention_cascade(const void* q, const void* k_cache, const void* v_cache,
                                    const pkv_cache_desc* cache, const int32_t* block_tables,
                                    int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                    const int32_t* query_start_loc, int32_t num_seqs, int32_t num_q_heads,
                                    int64_t num_tokens, int32_t max_query_len, int32_t max_seq_len, float scale,
                                    const pkv_prefix_groups* groups, void* out, void* stream);

/*
 * paged_attention_step -- the new tokens' slot mapping and K/V scatter, then
 * attention, in one call: pkv_slot_mapping + pkv_write + paged_attention_cascade
 * with the same results, bit for bit ("vLLM's PagedAttention" teardown, section
 * "Continuous batching": every step appends each running request's new tokens to
 * its blocks and attends over them).  On the bf16 path the mapping and the scatter
 * run in extra CTAs of the planning launch, so the step has two launches fewer and
 * no slot array round trip; the kernel boundary orders the writes before every
 * attention read.  On an fp32 cache with max_query_len == 1 (every request brings
 * one token) the attention launch itself stores each token's rows before it reads
 * them, one launch in all; a request with more query tokens than that bound is then
 * flagged (PKV_ERR_INDEX), its rows zeroed and its tokens not written.
 * Copy-on-write copies (pkv_copy_blocks) go before this call.
 * k_new, v_new    device [num_tokens][num_kv_heads][head_dim], cache dtype, required
 * k_cache, v_cache  written at the new tokens' slots, then read
 * groups          NULL for none (see paged_attention_cascade)
 * slot_mapping    optional device int64 [num_tokens]: receives the slots (NULL: not stored)
 * Everything else and the errors: as paged_attention() and pkv_write().
 */
PKV_API int paged_attention_step(const void* q, const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                                 const pkv_cache_desc* cache, const int32_t* block_tables,
                                 int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                 const int32_t* query_start_loc, int32_t num_seqs, int32_t num_q_heads,
                                 int64_t num_tokens, int32_t max_query_len, int32_t max_seq_len, float scale,
                                 const pkv_prefix_groups* groups, int64_t* slot_mapping, void* out, void* stream);

/*
 * paged_attention_step_cow -- pkv_copy_blocks(cow_src, cow_dst, num_cow) followed by
 * paged_attention_step, in one call, with the same results bit for bit.  The copies
 * are the copy-on-write of the "vLLM's PagedAttention" teardown, section
 * "PagedAttention": a request about to write into a block another request still
 * shares gets a fresh copy first.  Taking them in the same call lets the step plan
 * its work while the copies run, instead of after them; only the new tokens' writes,
 * which may land in a copied block, wait for the copies.
 * cow_src, cow_dst  device int32 [num_cow] block ids (as pkv_copy_blocks)
 * num_cow          0: no copies (exactly paged_attention_step)
 * Everything else and the errors: as paged_attention_step() and pkv_copy_blocks().
 */
PKV_API int paged_attention_step_cow(const void* q, const void* k_new, const void* v_new, void* k_cache,
                                     void* v_cache, const pkv_cache_desc* cache, const int32_t* block_tables,
                                     int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                     const int32_t* query_start_loc, int32_t num_seqs, int32_t num_q_heads,
                                     int64_t num_tokens, int32_t max_query_len, int32_t max_seq_len, float scale,
                                     const pkv_prefix_groups* groups, const int32_t* cow_src,
                                     const int32_t* cow_dst, int64_t num_cow, int64_t* slot_mapping, void* out,
                                     void* stream);

/*
 * paged_attention_noalloc -- paged_attention() for callers that cannot let a library
 * allocate device memory.  The pages have no counterpart for this call; it exists
 * for deployment.  paged_attention() grows a workspace with cudaMalloc when a batch
 * needs more split-KV scratch; a caller whose allocator must account for every byte
 * of device memory, or a service that reserves its memory at start-up and forbids
 * allocation afterwards, cannot accept that.  This call computes the same result
 * with its scratch in a fixed 16 MiB static device array that the library holds on
 * every GPU that loads it, until the process exits.
 *  - Same arguments and results as paged_attention(), bf16 with head_dim 128 only.
 *  - error_bits: optional device uint32 the kernels OR their data-error bits into
 *    (the bits of pkv_peek_error_bits); NULL discards them.  The caller clears it.
 *  - A batch whose scratch need exceeds the array returns PKV_ERR_NO_MEMORY and
 *    launches nothing.  The need is about num_seqs * num_kv_heads *
 *    ceil(max_seq_len / 1024) * GP * 520 bytes plus a few arrays per request, GP
 *    being the query-head group size rounded up to 4, 8 or 16.  A batch that
 *    paged_attention() refuses as unsupported (2^31 or more split items) returns
 *    PKV_ERR_UNSUPPORTED here too.
 *  - The first call on a device looks up the array's device address (with that
 *    device current); make it before any stream capture.
 *  - All calls share the array and the library re-zeroes what each call needs, but
 *    calls whose kernels overlap on the GPU race on it: serialise them.
 *  - Calls no cudaMalloc, cudaFree or other allocating routine.
 */
PKV_API int paged_attention_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                    const pkv_cache_desc* cache, const int32_t* block_tables,
                                    int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                    const int32_t* query_start_loc, int32_t num_seqs, int32_t num_q_heads,
                                    int64_t num_tokens, int32_t max_query_len, int32_t max_seq_len, float scale,
                                    void* out, uint32_t* error_bits, void* stream);

/*
 * pkv_tree_mask -- ancestor masks of drafted tokens.  Request i's new tokens
 * query_start_loc[i] .. query_start_loc[i+1] - 1 are the nodes 0 .. q_i - 1 of a tree
 * (a forest: several tokens may continue the context), and parents[t] names the node
 * that token t continues, a smaller index than its own, or -1 for the context itself.
 * Bit u of mask row t (bit u % 64 of word u / 64) is set iff node u is t's own node or
 * one of its ancestors; depths[t] counts the ancestors, so that token t's position is
 * seq_lens[i] - q_i + depths[t].
 * parents         device int32 [num_tokens]
 * mask            device uint64 [num_tokens][mask_words], written
 * depths          optional device int32 [num_tokens], written (NULL: not stored)
 * Device errors: a parent outside [-1, own index) or a node index that the row cannot
 * hold (q_i > 64 * mask_words) flags PKV_ERR_INDEX and gives a zero row and depth 0.
 */
PKV_API int pkv_tree_mask(const int32_t* parents, const int32_t* query_start_loc, int32_t num_seqs,
                          int64_t num_tokens, uint64_t* mask, int32_t mask_words, int32_t* depths, void* stream);

/*
 * paged_attention_tree -- attention of drafted tokens over the paged cache.  The new
 * tokens of a request are candidates that a verification step checks in one pass: node j
 * sees the whole context before the draft and, of the draft, what its mask row says.
 * With c_i = seq_lens[i] - q_i, token t = query_start_loc[i] + j sees key u of its
 * request iff u < c_i, or c_i <= u < seq_lens[i] and bit u - c_i of mask row t is set:
 *     out[t][h][:] = sum_{u seen} softmax_u(scale * q[t][h] . K_u) V_u
 * A row that sees no key is zero.  Keys and values that a row does not see have no part
 * in it, whatever they hold (infinities and NaN among it).  K and V of the new tokens
 * are already in the cache, node j at position c_i + j (pkv_slot_mapping and pkv_write
 * put them there).  Chains, trees and any other mask are served alike, q_i from 1 on.
 * tree_mask       device uint64 [num_tokens][mask_words]; bits past q_i are not read
 * mask_words      64 * mask_words >= max_query_len
 * max_query_len   host bound on q_i: a request with more is flagged (PKV_ERR_INDEX) and
 *                 its rows zeroed
 * query_start_loc rows outside of [0, num_tokens), or a request that ends before it begins, are flagged
 *                 too (PKV_ERR_INDEX); what exists of the request's rows is zeroed
 * max_seq_len     host bound on seq_lens, used only to plan the launch
 * workspace       device memory of at least pkv_tree_workspace() bytes, 256-byte aligned
 * seq_lens        up to 2^31 - 1024 (more is flagged); num_seqs below 2^30, num_tokens below 2^31
 * Everything else, the types and the errors: as paged_attention().  Work is cut along the
 * keys by the batch's sizes, so rounding (not the result) may depend on the batch.
 */
PKV_API int paged_attention_tree(const void* q, const void* k_cache, const void* v_cache,
                                 const pkv_cache_desc* cache, const int32_t* block_tables,
                                 int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                 const int32_t* query_start_loc, const uint64_t* tree_mask, int32_t mask_words,
                                 int32_t num_seqs, int32_t num_q_heads, int64_t num_tokens, int32_t max_query_len,
                                 int32_t max_seq_len, float scale, void* out, void* workspace,
                                 int64_t workspace_bytes, void* stream);
/* Bytes of workspace that paged_attention_tree needs for these sizes (*bytes). */
PKV_API int pkv_tree_workspace(const pkv_cache_desc* cache, int32_t num_q_heads, int32_t max_query_len,
                               int64_t* bytes);

/*
 * pkv_compact_path -- the accepted path of a tree of drafted tokens, moved together.
 * Request i keeps the nodes path[i][0] < path[i][1] < ... (path_lens[i] of them) of the
 * draft that its last q_i positions hold: with c_i = seq_lens[i] - q_i,
 *     K and V at position c_i + a = what was at position c_i + path[i][a],  a < path_lens[i],
 * in every layer, and new_seq_lens[i] = c_i + path_lens[i].  What lies behind that is no
 * longer part of the request; its blocks and bytes stay as they are.
 * k_cache, v_cache  [num_layers] pools of `cache`'s shape, one after the other
 * path            device int32 [num_seqs][max_path], entries past path_lens[i] not read
 * path_lens       device int32 [num_seqs]
 * new_seq_lens    device int32 [num_seqs], written; shares no memory with the inputs
 * Caller contract: the blocks that hold the draft belong to the request alone.
 * Device errors: q_i or seq_lens[i] that do not fit (as in paged_attention), path_lens[i]
 * outside [0, min(max_path, q_i)], a path that does not ascend within [0, q_i), or a bad
 * block id flag PKV_ERR_INDEX; that request's rows stay as they are and its new length
 * is seq_lens[i].
 */
PKV_API int pkv_compact_path(const int32_t* path, int32_t max_path, const int32_t* path_lens,
                             const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                             const int32_t* query_start_loc, int32_t num_seqs, void* k_cache, void* v_cache,
                             const pkv_cache_desc* cache, int32_t num_layers, int32_t* new_seq_lens,
                             void* stream);

/*
 * pkv_beam_select -- beam search's step: the best continuations of each request's beams.
 * Beam w of request n with token v scores
 *     score(w, v) = cum_scores[n][w] + logits[n][w][v] - log sum_u exp(logits[n][w][u]),
 * and a beam with finished[n][w] != 0 stands for itself: its one candidate is
 * (w, eos_token) with score cum_scores[n][w].  The num_select best of all beams are
 * returned, best first; equal scores are taken in order of w * vocab + v.  A score that
 * is not finite (a NaN or infinite beam, a logit of -inf) is no candidate, and where the
 * candidates run out, the score is -inf and beam and token are -1.  Scores are ranked in
 * 64 bits; sums over the vocabulary run in 32, and what their joins round off is kept.
 * logits          device [num_seqs * num_beams] rows of vocab values of `dtype` (pkv_dtype),
 *                 row_stride elements apart (>= vocab), aligned to their type
 * cum_scores      device fp32 [num_seqs][num_beams]
 * finished        optional device uint8 [num_seqs][num_beams] (NULL: none is)
 * num_beams       1 to 64;  num_select  1 to 64;  num_beams * vocab < 2^31
 * out_scores, out_parents, out_tokens  device fp32, int32, int32 [num_seqs][num_select]
 * workspace       device memory of at least pkv_beam_workspace() bytes, 256-byte aligned
 */
PKV_API int pkv_beam_select(const void* logits, int32_t dtype, int64_t row_stride, const float* cum_scores,
                            const uint8_t* finished, int32_t eos_token, int32_t num_seqs, int32_t num_beams,
                            int32_t vocab, int32_t num_select, float* out_scores, int32_t* out_parents,
                            int32_t* out_tokens, void* workspace, int64_t workspace_bytes, void* stream);
PKV_API int pkv_beam_workspace(int32_t num_seqs, int32_t num_beams, int32_t vocab, int32_t num_select,
                               int64_t* bytes);

/*
 * pkv_fork_tables -- block tables after the beams (or samples) they continue, with the
 * pool's reference counts kept on the device ("The 1960s Operating System Trick ..."
 * page, Technical Details: samples share blocks until they diverge, only the block that
 * changes is duplicated, and a block without users is free again).
 * Row b of the new tables continues row parents[b] of the old ones (-1: row b ends).  It
 * holds the first ceil(n / 16) blocks of that row, n = seq_lens[parents[b]], and then
 * whatever num_new more tokens need, all of it its own to write:
 *  - a last block with room in it (n % 16 != 0, num_new > 0) that other rows or other
 *    users hold too is replaced by a copy, in every layer of k_cache and v_cache; if no
 *    one but rows of this call holds it, the lowest of them keeps the block itself;
 *  - ceil((n + num_new) / 16) - ceil(n / 16) fresh blocks follow.
 * Old rows give up all their blocks (every id >= 0 in the row); a block that nobody holds
 * any more is free and may be handed out again by the same call.  Fresh blocks are the
 * lowest free ids, given to rows in order, a row's copy before its other fresh blocks.
 * Entries behind a row's last block are -1, and new_seq_lens[b] = n (0 for an ended row).
 * ref_counts      device int32 [num_blocks], users of each block, 0 = free; updated.  Holds
 *                 one for every row and entry that names the block, plus other holders
 * block_tables, new_block_tables  device int32 [num_rows][max_blocks_per_seq], two arrays
 * seq_lens, new_seq_lens          device int32 [num_rows], two arrays
 * num_rows        1 to 4096;  num_new  0 to 65536
 * k_cache, v_cache  [num_layers] pools of `cache`'s shape, one after the other; both NULL:
 *                 no data is copied (the tables and counts alone)
 * workspace       device memory of at least pkv_fork_workspace() bytes, 256-byte aligned
 * Device errors leave everything as it was (the new tables and lengths equal the old):
 * a parent outside [-1, num_rows), a length past the table's row or a bad block id within
 * it flag PKV_ERR_INDEX, too few free blocks flag PKV_ERR_NO_MEMORY (bit 4).
 */
PKV_API int pkv_fork_tables(const int32_t* block_tables, const int32_t* seq_lens, int32_t num_rows,
                            int32_t max_blocks_per_seq, const int32_t* parents, int32_t num_new,
                            int32_t* ref_counts, int32_t* new_block_tables, int32_t* new_seq_lens, void* k_cache,
                            void* v_cache, const pkv_cache_desc* cache, int32_t num_layers, void* workspace,
                            int64_t workspace_bytes, void* stream);
PKV_API int pkv_fork_workspace(int32_t num_rows, int64_t* bytes);

/*
 * pkv_rope_append -- the new tokens' keys and values into the paged cache, keys (and queries)
 * rotated by their positions on the way: what pkv_slot_mapping and pkv_write do, from a
 * projection's raw output ("vLLM's PagedAttention" teardown, section "PagedAttention": new
 * tokens go to the slots that their block table names).
 * Token j of request i sits at position p = seq_lens[i] - q_i + j, in slot block_tables[i][p / 16] *
 * 16 + p % 16.  Its queries and keys turn by row a = positions[t] (NULL: p) of cos_sin: with half =
 * rot_dim / 2, pair m of a head's first rot_dim elements, (x, y) = elements (m, m + half), or (2m,
 * 2m + 1) where interleaved is not 0, becomes
 *     (x cos_sin[a][m] - y cos_sin[a][half + m],  y cos_sin[a][m] + x cos_sin[a][half + m]).
 * Elements past rot_dim and values stay as they are.  Results are computed in fp32 and rounded once,
 * to the type of q_out and of the cache.
 * An 8-bit cache (PKV_E4M3) holds codes; the value in slot s of block b is code * scales[b][h][0] for K and
 * scales[b][h][1] for V.  Where the call's tokens begin a block (its first position is among them, or the
 * request has none before), its scales are made anew, otherwise they can only grow: to the
 * least power of two s, at least 2^-80, with |x| <= 448 s for all finite new values x of the block and
 * head.  What the block held of the request is then put in the new units (each code rounded again, which
 * changes only those that leave e4m3's normal range where scales are powers of two).  Infinities
 * become +-448 s, NaN stays NaN.
 * q               device [num_tokens][num_q_heads][head_dim], tokens q_stride elements apart; NULL: none
 * k, v            device [num_tokens][num_kv_heads][head_dim], tokens k_stride and v_stride elements apart
 *                 (slices of one projection's output will do); strides of at least a token's elements, 16-byte
 *                 aligned as all of its rows
 * dtype           of q, k, v and q_out: the cache's, PKV_BF16 for an 8-bit cache
 * cos_sin         device fp32 [num_angles][rot_dim], 16-byte aligned; rot_dim a multiple of 16, 0 to head_dim (0:
 *                 nothing turns, cos_sin is not read)
 * positions       optional device int32 [num_tokens]: rows of cos_sin (a drafted tree's tokens turn by
 *                 their depth, not by their slot)
 * scales          device fp32 [num_blocks][num_kv_heads][2] of an 8-bit cache, updated; NULL for others
 * max_query_len   host bound on q_i: a request with more is flagged, its tokens not written
 * q_out           device, as q, tokens q_out_stride apart; written.  May be q itself (same stride); any other
 *                 overlap with q, k or v is refused
 * Rows of tokens behind the last request stay as they are.  A block that the call writes belongs to one request of it.
 * Device errors: a request whose lengths do not fit or a row outside of [0, num_angles) flag PKV_ERR_INDEX, its
 * tokens are not written and their q_out rows are zero; so is a bad block id, whose q_out row stays valid.
 */
PKV_API int pkv_rope_append(const void* q, const void* k, const void* v, int32_t dtype, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, int32_t num_q_heads, const float* cos_sin,
                            int32_t rot_dim, int32_t interleaved, int64_t num_angles, const int32_t* positions,
                            void* k_cache, void* v_cache, float* scales, const pkv_cache_desc* cache,
                            const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                            const int32_t* query_start_loc, int32_t num_seqs, int64_t num_tokens,
                            int32_t max_query_len, void* q_out, int64_t q_out_stride, void* stream);

/*
 * paged_attention_q8 -- paged_attention() over a cache in 8 bits (cache->dtype PKV_E4M3, head_dim 128, up to 16
 * query heads a kv head): the same sum over K_u = code * scales[b][g][0] and V_u = code * scales[b][g][1] of
 * block b = block_tables[i][u / 16].  q and out are bf16.  Chunks and single tokens mix freely.
 * scales          device fp32 [num_blocks][num_kv_heads][2]; positive.  V's are taken as at least 2^-80 and at
 *                 most 2^110
 * max_query_len   host bound on q_i: a request with more is flagged (PKV_ERR_INDEX) and its rows zeroed
 * query_start_loc rows outside of [0, num_tokens) are flagged too; rows that no request has stay as they are
 * workspace       device memory of at least pkv_q8_workspace() bytes, 256-byte aligned
 * A key counts by its weight times V's scale, next to the largest such product that the row sees: where max_query_len is 1, a
 * product is held to 2^-11 of itself down to 2^-29 of the largest, and to 2^-40 of the largest below; otherwise to 2^-21 and
 * 2^-32.  The sum of the weights takes fp32 ones; products below 2^-120 of the largest may be left out there too.
 * What a row does not see (later tokens of its chunk, slots behind the context) has no part in it, whatever its
 * codes are, NaN among them.  A NaN that a row sees makes elements of the row NaN: those of its column at least, of a NaN in K
 * or a query all.  An element of a query counts down to 2^-22 of the largest one among its unit's rows (the heads of a kv
 * head; of a chunk 2^-24, 32 rows).
 * Everything else and the errors: as paged_attention().  Work is cut along the keys by the batch's
 * sizes, so rounding (not the result) may depend on the batch.
 */
PKV_API int paged_attention_q8(const void* q, const void* k_cache, const void* v_cache, const float* scales,
                               const pkv_cache_desc* cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                               const int32_t* seq_lens, const int32_t* query_start_loc, int32_t num_seqs,
                               int32_t num_q_heads, int64_t num_tokens, int32_t max_query_len, int32_t max_seq_len,
                               float scale, void* out, void* workspace, int64_t workspace_bytes, void* stream);
/* Bytes of workspace that paged_attention_q8 needs for these sizes (*bytes). */
PKV_API int pkv_q8_workspace(const pkv_cache_desc* cache, int32_t num_q_heads, int32_t max_query_len,
                             int64_t* bytes);

/*
 * pkv_sample -- one token for each row of logits, drawn with a given random number.  Row n's candidates are its
 * finite logits x, in order: larger ones first, of equal ones the lower index; a candidate's weight is
 * exp((x - max) / temperature[n]).  Kept are, one after the other,
 *     the first top_k[n] of them (0 or less: all),
 *     of these the ones whose weight is at least min_p[n] (that of the first is 1; 0 or less: all),
 *     of these the shortest beginning whose weights are at least top_p[n] of the sum (1 or more: all; one at least).
 * The token is the first of the kept ones whose cumulative weight exceeds uniform[n] times their sum.
 * temperature[n] == 0 takes the first candidate.  Near a border weights are right to 2^-40 (of the largest weight, 2^-44, or
 * vocab 2^-63 where that is more), and sums to 2^-28 of the kept ones (of the largest weight, vocab^2 2^-63 where that is more),
 * or, where a border lies within 2^-25 of a candidate's, exact down to weights of 2^-20 of the largest: tokens are told apart as
 * 64-bit arithmetic does but for borders closer than that.  A call repeats bit by bit.
 * logits          device [num_seqs] rows of vocab values of `dtype` (pkv_dtype: fp32 or bf16), row_stride elements
 *                 apart (>= vocab), aligned to their type; vocab up to 2^20
 * temperature, top_k, top_p, min_p  optional device fp32, int32, fp32, fp32 [num_seqs] (NULL: 1, all, 1, 0)
 * uniform         device fp32 [num_seqs], in [0, 1)
 * out_tokens      device int32 [num_seqs]
 * out_logprobs    optional device fp32 [num_seqs]: log of the token's share of the kept weights, to 2^-22 of itself and of 1
 * Rows are a matter of tens of microseconds, but of a millisecond or two where a border lies among thousands of candidates
 * that cannot be told apart in one look: equal logits, or the end of top_k more than 22 temperatures below the largest logit (a
 * min_p of 1e-9 ends the row before that).
 * A row without a candidate gives token -1 and -inf; so does a setting outside of its range (a temperature that is
 * negative or not finite, uniform outside of [0, 1), top_p below 0, min_p above 1, a NaN), which flags bit 5
 * (PKV_ERR_INDEX).
 */
PKV_API int pkv_sample(const void* logits, int32_t dtype, int64_t row_stride, const float* temperature,
                       const int32_t* top_k, const float* top_p, const float* min_p, const float* uniform,
                       int32_t num_seqs, int32_t vocab, int32_t* out_tokens, float* out_logprobs, void* stream);

/* Synchronises `stream`, returns the device error word of the current device as a
 * pkv_status (PKV_OK, PKV_ERR_INDEX, PKV_ERR_TIMEOUT, or PKV_ERR_NO_MEMORY where a fork
 * that found too few free blocks is all there is) and clears it. */
PKV_API int pkv_get_last_error(void* stream);

/* Raw device error bits of the current device (bit 0 bad block id, bit 1 bad slot,
 * bit 2 bad length, bit 3 wait timeout, bit 4 no free block left, bit 5 a sampling setting out of range); synchronises `stream`; does not clear. */
PKV_API int pkv_peek_error_bits(void* stream, uint32_t* bits);

/* Human-readable name of a pkv_status value (static string). */
PKV_API const char* pkv_status_string(int status);

/* Number of persistent CTAs the attention kernels launch on the current device
 * (a multiple of the SM count); split boundaries depend only on it and the lengths. */
PKV_API int pkv_num_workers(int32_t* workers);

/* Releases the library-owned workspace and error word on every device used. */
PKV_API void pkv_shutdown(void);

/*
 * Launch tracing.  While enabled, every kernel the library launches is bracketed
 * by CUDA events on its stream.  pkv_trace_read() synchronises the device and
 * returns, per kernel kind, the launch count and the summed device time in ms,
 * then resets the counters.  Kinds: 0 slot mapping, 1 write, 2 copy, 3 plan,
 * 4 decode, 5 prefill, 6 generic attention, 7 split merge, 8 shared-prefix (cascade)
 * pass.  Arrays hold PKV_TRACE_KINDS entries.  (The calls for candidate continuations
 * and those of a step over a cache in 8 bits, pkv_tree_mask to pkv_sample, are not traced.)
 */
#define PKV_TRACE_KINDS 9
PKV_API int pkv_trace_enable(int on);
PKV_API int pkv_trace_read(int64_t* launches, double* total_ms);
PKV_API const char* pkv_trace_kind_name(int kind);

/*
 * Diagnostics for the tensor-core operand layouts (no counterpart in the pages).
 * pkv_umma_selftest copies two operand images (a_img, b_img: device bytes, already
 * in shared-memory order) into shared memory, runs k_steps tcgen05 bf16 MMAs with
 * an fp32 accumulator in TMEM, and writes D ([M][N] fp32 row-major) to d_out.
 * params (host int32[29]): M, N, a_mn_major, b_mn_major, a_layout, a_lbo, a_sbo,
 * b_layout, b_lbo, b_sbo, a_bytes, b_bytes, k_steps, a_off[8], b_off[8] -- layouts
 * use the descriptor codes (0 none, 2 128B, 4 64B, 6 32B), offsets are bytes.
 * a_layout = -1 reads A from TMEM instead (M must be 128, A K-major): a_img is then
 * [128 rows][a_bytes / 512] 32-bit columns, two bf16 each, stored to the rows' lanes
 * after the N accumulator columns, and a_off[k] is k step k's first column (a multiple
 * of 8) within them.
 * pkv_umma8_selftest is the same for e4m3 operands (kind::f8f6f4, 32 along K to an MMA),
 * both from shared memory.
 * pkv_tma_selftest loads rows [row0, row0+16) of a bf16 [rows][128] matrix with two
 * 16 x 64 boxes in the 128-byte swizzle and copies the 4 KiB of shared memory they
 * land in to dump.
 */
PKV_API int pkv_umma_selftest(const int32_t* params, const void* a_img, const void* b_img, float* d_out, void* stream);
PKV_API int pkv_umma8_selftest(const int32_t* params, const void* a_img, const void* b_img, float* d_out, void* stream);
PKV_API int pkv_tma_selftest(const void* src, int64_t rows, int32_t row0, void* dump, void* stream);
/*
 * pkv_wait_selftest launches one CTA that waits on an mbarrier nothing arrives on.
 * The bounded wait every kernel of the library uses gives up after its limit (1 s),
 * the CTA sets the timeout bit of the device error word and exits: the next
 * pkv_get_last_error() returns PKV_ERR_TIMEOUT, and the context stays usable.
 */
PKV_API int pkv_wait_selftest(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H_ */
