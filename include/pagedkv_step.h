/*
 * pagedkv_step.h - what surrounds attention in a serving step, and attention for speculative
 * decoding with drafted trees (part of libpagedkv.so).
 *
 *   kv_build_batch             request lengths -> block tables, slots, positions, tree masks
 *   kv_qk_norm_rope            RMS norm of each query and key head, rotary embedding, and the
 *                              write of K and V into the paged cache, in one pass
 *   kv_paged_attention_tree    attention of a tree of drafted tokens over the paged cache
 *
 * One speculative step of one layer calls them in this order; kv_build_batch runs once a step and
 * its outputs serve every layer.  The pages describe the surrounding path ("vLLM의 KV cache 연결
 * 흐름", sections "EngineCore가 하는 일", "GPU worker가 하는 일", "Slot mapping은 왜 필요한가"):
 * tokens per request with speculative tokens, new block ids appended to the request's table row,
 * a slot per token, attention through the block table.  They fix neither the norm and rotation
 * nor the tree; those are this library's own readings, stated below.
 *
 * Conventions (device pointers, caller-owned buffers, stream and capture semantics, d_err bits,
 * host errors returned before any launch, cache layout) are those of pagedkv.h.
 */
#ifndef PAGEDKV_STEP_H
#define PAGEDKV_STEP_H

#include "pagedkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits set in *d_err by device code. */
#define KV_DERR_BAD_POS    64  /* a position >= max_position in kv_qk_norm_rope */
#define KV_DERR_NO_BLOCKS 128  /* kv_build_batch: the list of free blocks holds too few */
#define KV_DERR_BAD_TREE  256  /* kv_build_batch: a parent that is not an earlier token of its tree */

/* Most tokens of one drafted tree (a row's mask is one 64-bit word). */
#define KV_MAX_TREE 64

/*
 * kv_build_batch - the metadata of one step, built on the device from the requests' lengths.
 *
 * Request r holds context_lens[r] = c tokens in the cache and gets new_lens[r] = n more; its row
 * of the block table holds held_blocks[r] = h blocks (NULL: ceil(c / block_size)).  It needs
 *   need = n > 0 ? max(0, ceil((c + n) / block_size) - h) : 0
 * more blocks, taken in request order from the front of the caller's list:
 *   block_table[r][h + k] = free_blocks[*free_start + (blocks taken by requests < r) + k]
 * and, for its i-th new token, t = query_start_loc[r] + i,
 *   query_start_loc[r + 1] = query_start_loc[r] + n          (query_start_loc[0] = 0)
 *   slot_mapping[t] = block_table[r][(c + i) / block_size] * block_size + (c + i) % block_size
 *   positions[t]    = c + i, or c + depth(i) when parents are given
 *   seq_lens[r]     = c + n,     held_out[r] = h + need,     *free_next = *free_start + taken
 * What a request holds beyond its tokens (blocks of rejected drafted tokens) is used before new
 * blocks are taken.
 *
 * Trees: parents[t] is the index, within its own request, of token t's parent, an earlier token,
 * or -1 for a token that follows the context.  depth is the number of ancestors, and
 *   tree_mask[t] bit j = 1 when j is i itself or an ancestor of i
 * (what kv_paged_attention_tree takes).  The K/V of drafted token i belong in slot c + i whatever
 * its depth, while its position, for the rotary embedding, is c + depth.  A parent that is not in
 * [-1, i) sets KV_DERR_BAD_TREE and counts as -1.
 *
 * A request is refused as a whole when a length or held count is negative, c + n needs more than
 * max_blocks_per_seq blocks, h is more than that, its tokens end past num_tokens, or it has more
 * than KV_MAX_TREE tokens and parents are given (KV_DERR_BAD_LEN); or when it needs blocks and the
 * needs of the requests up to it exceed what the list holds (KV_DERR_NO_BLOCKS; requests that need
 * none are still served).  Refused: seq_lens[r] = 0 (attention then writes its rows as 0), positions
 * and slots -1, masks 0, held_out = h, table row untouched; its tokens keep their place in
 * query_start_loc (which never passes num_tokens).  A block id outside [0, num_blocks) that a
 * slot needs gives slot -1, and one in the list is not written (KV_DERR_BAD_BLOCK).
 * Tokens behind the last request (a padded batch) get position and slot -1, mask 0.
 *
 *   context_lens, new_lens  int32 [num_seqs]
 *   held_blocks      int32 [num_seqs] or NULL
 *   parents          int32 [num_tokens] or NULL
 *   block_table      int32 [num_seqs, bt_stride], updated in place
 *   free_blocks      int32 [num_free], distinct ids; free_start: device int32 (NULL: 0) in [0, num_free]
 *   query_start_loc  int32 [num_seqs + 1]; seq_lens, held_out int32 [num_seqs]
 *   positions        int32 [num_tokens]; slot_mapping int64 [num_tokens]
 *   tree_mask        uint64 [num_tokens], given exactly when parents are
 *   free_next        device int32
 * Outputs may not overlap inputs or each other (KV_ERR_INVALID_ARG): a loop keeps two sets and
 * swaps them.  block_size 4, 8, 16 or 32.  Exact integer arithmetic; one launch, whose every CTA reads
 * all lengths (made for batches of up to some thousand requests; num_seqs up to 2^24).
 */
KV_API kv_status kv_build_batch(const int32_t *context_lens, const int32_t *new_lens,
                                const int32_t *held_blocks, const int32_t *parents, int32_t num_seqs,
                                int32_t num_tokens, int32_t *block_table, int64_t bt_stride,
                                int32_t max_blocks_per_seq, int32_t block_size, int32_t num_blocks,
                                const int32_t *free_blocks, int32_t num_free,
                                const int32_t *free_start, int32_t *query_start_loc,
                                int32_t *seq_lens, int32_t *positions, int64_t *slot_mapping,
                                uint64_t *tree_mask, int32_t *held_out, int32_t *free_next,
                                int32_t *d_err, void *stream);

/*
 * kv_qk_norm_rope - norm and rotation of a step's queries and keys, and their cache write.
 *
 * For every token t and head of q and of key, x in float32:
 *   y = x / sqrt(mean(x^2) + eps) * weight         (q_weight / k_weight; NULL: y = x)
 * then the first rotary_dim dims turn by the token's angles, the others stay.  Pair i of
 * rotary_dim / 2 is dims (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved:
 *   (a, b) -> (a cos - b sin, b cos + a sin),
 *   cos = cos_sin[positions[t]][i],  sin = cos_sin[positions[t]][rotary_dim / 2 + i].
 * The result is rounded once: q to q_out; key to k_out (unless NULL) and, when slot_mapping is
 * given, to its slot of k_cache, with value beside it in v_cache, as kv_reshape_and_cache would.
 * 16-bit caches take the same bits as k_out; E4M3 caches round the float32 key divided by k_scale
 * (not its 16-bit rounding).
 * A token with a negative position (padding) is skipped: nothing of it is written.  So is one
 * with a position >= max_position (KV_DERR_BAD_POS).  A slot of -1 leaves the cache alone; one past
 * it sets KV_DERR_BAD_SLOT.  Duplicate slots in one call: undefined.
 *
 *   q, key, value    fp16/bf16 [num_tokens, heads, head_dim], token stride in elements (>= heads *
 *                    head_dim, a multiple of 8), 16-byte aligned: views of one projection will do
 *   q_out, k_out     like q and key; each may be its input (same stride), else overlap nothing
 *                    (KV_ERR_INVALID_ARG; rows of one stride may lie between each other)
 *   q_weight, k_weight  of the same dtype, [head_dim], 16-byte aligned
 *   cos_sin          float32 [max_position, rotary_dim], 16-byte aligned (NULL when rotary_dim 0)
 *   value, caches    as for kv_reshape_and_cache; all NULL when slot_mapping is
 * Supported: head_dim a multiple of 8 up to 256; rotary_dim a multiple of 16 up to head_dim (0: no
 * rotation; positions may then be NULL, else they still mark padding); up to 65535 heads of a kind.  One
 * launch.
 */
KV_API kv_status kv_qk_norm_rope(const void *q, const void *key, const void *value, kv_dtype dtype,
                                 int64_t q_stride, int64_t key_stride, int64_t value_stride,
                                 int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                                 int32_t head_dim, const void *q_weight, const void *k_weight,
                                 float eps, const int32_t *positions, const float *cos_sin,
                                 int32_t max_position, int32_t rotary_dim, int32_t interleaved,
                                 void *q_out, int64_t q_out_stride, void *k_out,
                                 int64_t k_out_stride, const int64_t *slot_mapping, void *k_cache,
                                 void *v_cache, kv_dtype cache_dtype, int32_t num_blocks,
                                 int32_t block_size, float k_scale, float v_scale, int32_t *d_err,
                                 void *stream);

/*
 * kv_paged_attention_tree - attention of drafted trees over the paged cache (speculative decoding:
 * several candidate continuations of each sequence are verified in one step).
 *
 * Sequence b has n_b = query_start_loc[b+1] - query_start_loc[b] drafted tokens (0 allowed, at most
 * KV_MAX_TREE), L_b = seq_lens[b] including them; their K/V sit in the slots of positions
 * c_b .. L_b - 1, c_b = L_b - n_b.  Row i of the sequence sees key j
 *   j < c_b   when window = 0 or j > p_i - window,  p_i = c_b - 1 + (number of its mask bits < n_b)
 *   j >= c_b  when bit j - c_b of tree_mask[row] is set
 * (p_i is the row's position when its mask is itself and its ancestors).  Any mask is taken: a
 * row need not see itself, and a row that sees no key gives out 0, lse -inf.  With GQA and softmax
 * as in kv_paged_attention_decode, and a scale that is finite and not negative (a negative one,
 * which that call takes, is KV_ERR_INVALID_ARG; 0 weighs all keys of a row alike):
 *   out = sum_j softmax_j(scale * q.K_j) V_j,   lse = log(sum_j exp(scale * q.K_j))
 * A key that a row does not see has no part in its result, whatever the cache holds there (NaN and
 * infinities included).
 * Once a path of the tree is accepted, its K/V belong in slots c_b, c_b + 1, ...: kv_reshape_and_cache of
 * the step's rows (k_out of kv_qk_norm_rope, whose positions c_b + depth are the final ones) with a
 * slot mapping that is -1 for the rejected rows puts them there.
 *
 *   q            [num_tokens, num_q_heads, head_dim] fp16/bf16, equal to cache_dtype, 16-byte aligned
 *   query_start_loc int32 [num_seqs + 1], non-decreasing; max_query_len >= every n_b (host bound; 0
 *                says that no sequence has rows: as with no sequences or tokens at all, nothing is
 *                launched, read, checked against the lengths or written)
 *   tree_mask    uint64 [num_tokens] (kv_build_batch writes it; bits from n_b on are ignored)
 *   block_table, seq_lens, max_seq_len, caches: as for kv_paged_attention_decode (entries of blocks
 *                wholly outside every row's window are never read)
 *   workspace    at least kv_paged_attention_tree_workspace_size(...) bytes, 256-byte aligned
 *   out          [num_tokens, num_q_heads, head_dim]; lse_out float32 [num_tokens, num_q_heads] or
 *                NULL.  Rows of no sequence are not written.  Neither they nor the workspace may overlap
 *                an input or each other (KV_ERR_INVALID_ARG)
 * A sequence whose length is rejected (n_b > max_query_len, L_b < n_b, > max_seq_len, > 2^31 - 257 or past
 * the table) sets KV_DERR_BAD_LEN and its rows are 0 (lse -inf).  A bad block id sets KV_DERR_BAD_BLOCK;
 * its keys read as zeros.
 * Supported: head_dim 64 or 128, block_size 8, 16 or 32, num_q_heads / num_kv_heads up to 128,
 * window 0 or >= KV_MAX_TREE.  num_workers as for kv_paged_attention_decode.
 * Two launches: the attention kernel and the merge of the trees that several workers shared.  Calls
 * that may overlap on the GPU need workspaces of their own; captured calls replayed one after the
 * other may share one.
 */
KV_API kv_status kv_paged_attention_tree(
    const void *q, kv_dtype q_dtype, const int32_t *query_start_loc, int32_t num_seqs,
    int32_t num_tokens, int32_t max_query_len, int32_t num_q_heads, const void *k_cache,
    const void *v_cache, kv_dtype cache_dtype, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int32_t num_blocks, const int32_t *block_table, int64_t bt_stride,
    int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t max_seq_len, float scale,
    int32_t window, const uint64_t *tree_mask, int32_t num_workers, void *workspace,
    size_t workspace_bytes, void *out, float *lse_out, int32_t *d_err, void *stream);

/* Workspace bytes of kv_paged_attention_tree for these sizes (SIZE_MAX when they are invalid or
 * unsupported, with the reason in kv_last_error(), or no device can be queried).  More sequences or a larger
 * max_query_len never need less. */
KV_API size_t kv_paged_attention_tree_workspace_size(int32_t num_seqs, int32_t max_query_len,
                                                     int32_t num_q_heads, int32_t num_kv_heads,
                                                     int32_t head_dim, int32_t num_workers);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_STEP_H */
