/*
 * pagedkv_sinks.h - attention with a sliding window and sinks over the paged cache (part of
 * libpagedkv.so).
 *
 *   kv_paged_attention_decode_sinks       decode, 16-bit and E4M3 caches
 *   kv_paged_attention_decode_sinks_int4  decode, INT4 caches
 *   kv_paged_attention_prefill_sinks      chunks of new tokens, 16-bit and E4M3 caches
 *   kv_paged_attention_prefill_sinks_int4 chunks of new tokens, INT4 caches
 *
 * A layer with a sliding window ("vLLM Worker侧GPU KV Cache初始化流程深度解析", section
 * "混合注意力机制") forgets the start of a long sequence, and many models put much of their attention
 * on a few first tokens, whatever those say: the sinks.  Here they stay visible.  The query at position
 * p sees key j when
 *   j <= p  and  (window = 0  or  j > p - window  or  j < num_sinks)
 * With window = 0 every earlier key is seen and num_sinks means nothing; with num_sinks = 0 it is the
 * window alone.  The pages describe the window and have no sinks.
 *
 * Entries of the block table whose blocks no row sees, those between the last sink and the first row's
 * window, are never read (they may hold -1): kv_bm_create_sinks (pagedkv_blocks.h) makes a manager that
 * releases such blocks.  Positions are those of the sequence: a rotation that counts them within the
 * window instead is not applied here.
 *
 * Conventions (device pointers, caller-owned buffers, stream and capture semantics, d_err bits, host
 * errors returned before any launch, cache layouts) are those of pagedkv.h and pagedkv_int4.h.  Outputs
 * and the workspace may not overlap an input or each other (KV_ERR_INVALID_ARG).
 *   - A key that a row does not see has no part in its result, whatever the cache holds there (NaN and
 *     infinities included).  A NaN score that it does see makes its result and log-sum-exp NaN; a NaN
 *     or an infinity in a value that it does see reaches that dim of its result (an infinity as NaN where its
 *     key's weight underflows to 0, in float32 or in the 16 bits of the second product).
 *   - Softmax sums are float32, of the weights before they are rounded to 16 bits for the second product
 *     (INT4 decode: of the rounded weights, whose codes' offset comes out exactly with them; prefill: the
 *     result is divided by a sum that takes the largest weight of each 128 keys as it was rounded).  A row
 *     whose weight lies with one key is that key's value, rounded once.  fp16
 *     weights are formed 2^14 (prefill: 2^7) higher than they are, so that the many small weights beside
 *     a sink that holds nearly all of them keep their digits.
 */
#ifndef PAGEDKV_SINKS_H
#define PAGEDKV_SINKS_H

#include "pagedkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * kv_paged_attention_decode_sinks - kv_paged_attention_decode with sinks: the same arguments, results and
 * supported sizes, and the mask above for each of a sequence's q_len rows at positions L - q_len .. L - 1.
 * The workspace is kv_paged_attention_workspace_size's for the same sizes.
 * A sequence whose length is rejected (as there, or past 2^31 - 65) sets KV_DERR_BAD_LEN; its rows are 0
 * (lse -inf).  A bad block id of a block that some row sees sets KV_DERR_BAD_BLOCK, and its keys are
 * seen by no row.  Two launches: the attention kernel and the log-sum-exp merge.  Calls that may overlap
 * on the GPU need workspaces of their own; captured calls replayed one after the other may share one.
 */
KV_API kv_status kv_paged_attention_decode_sinks(
    const void *q, kv_dtype q_dtype, int32_t num_seqs, int32_t q_len, int32_t num_q_heads,
    const void *k_cache, const void *v_cache, kv_dtype cache_dtype, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t num_blocks, const int32_t *block_table,
    int64_t bt_stride, int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t max_seq_len,
    float scale, int32_t window, int32_t num_sinks, float k_scale, float v_scale,
    int32_t num_workers, void *workspace, size_t workspace_bytes, void *out, float *lse_out,
    int32_t *d_err, void *stream);

/* The same over INT4 caches: the arguments and rounding of kv_paged_attention_decode_int4. */
KV_API kv_status kv_paged_attention_decode_sinks_int4(
    const void *q, kv_dtype q_dtype, int32_t num_seqs, int32_t q_len, int32_t num_q_heads,
    const void *k_cache, const void *v_cache, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int32_t num_blocks, const int32_t *block_table, int64_t bt_stride,
    int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t max_seq_len, float scale,
    int32_t window, int32_t num_sinks, const float *k_scales, const float *v_scales,
    int32_t group_size, int32_t num_workers, void *workspace, size_t workspace_bytes, void *out,
    float *lse_out, int32_t *d_err, void *stream);

/*
 * kv_paged_attention_prefill_sinks - attention of a chunk of new tokens per sequence, as
 * kv_paged_attention_prefill, with the mask above and over every kind of cache.  Sequence b has
 * n_b = query_start_loc[b+1] - query_start_loc[b] rows (0 allowed) at positions L_b - n_b .. L_b - 1,
 * whose K/V are in the cache already.  window = 0 is full attention.
 *   q            [num_tokens, num_q_heads, head_dim] fp16/bf16, 16-byte aligned; a 16-bit cache has its type
 *   query_start_loc int32 [num_seqs + 1], non-decreasing; max_query_len >= every n_b (host bound; 0 says
 *                that no sequence has rows: nothing is launched, read or written)
 *   k_scale, v_scale  of E4M3 caches (else ignored)
 *   num_workers  CTAs that share the key tiles (0: one an SM); results depend on it only through rounding
 *   workspace    at least kv_paged_attention_prefill_sinks_workspace_size(...) bytes, 256-byte aligned
 *   out, lse_out as for kv_paged_attention_prefill.  Rows of no sequence are not written
 * A sequence whose length is rejected (n_b > max_query_len, rows past num_tokens, L_b < n_b, > max_seq_len,
 * > 2^31 - 257 or past the table) sets KV_DERR_BAD_LEN and its rows are 0 (lse -inf).  A bad block id of a
 * block that some row sees sets KV_DERR_BAD_BLOCK; its keys read as zeros.
 * scale finite and not negative; 0 weighs all keys of a row alike.
 * Products take 16-bit operands: over E4M3 caches fp16 queries, rounded after a power of two a row has brought
 * their largest to 2^7 .. 2^8.
 * Supported: head_dim 64 or 128 (E4M3: 128), block_size 8, 16 or 32, num_q_heads / num_kv_heads up to 128.
 * Two launches: the attention kernel, and the merge of the items that several workers shared.  Calls
 * that may overlap on the GPU need workspaces of their own; captured calls replayed one after the other
 * may share one.
 */
KV_API kv_status kv_paged_attention_prefill_sinks(
    const void *q, kv_dtype q_dtype, const int32_t *query_start_loc, int32_t num_seqs,
    int32_t num_tokens, int32_t max_query_len, int32_t num_q_heads, const void *k_cache,
    const void *v_cache, kv_dtype cache_dtype, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int32_t num_blocks, const int32_t *block_table, int64_t bt_stride,
    int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t max_seq_len, float scale,
    int32_t window, int32_t num_sinks, float k_scale, float v_scale, int32_t num_workers,
    void *workspace, size_t workspace_bytes, void *out, float *lse_out, int32_t *d_err,
    void *stream);

/* The same over INT4 caches (pagedkv_int4.h): k_scales, v_scales and group_size as for
 * kv_paged_attention_decode_int4, head_dim 128.  Codes enter the products as the integers they are, queries
 * as q * k_scale rounded to fp16 (after the power of two above), and the V scales multiply the float32
 * result. */
KV_API kv_status kv_paged_attention_prefill_sinks_int4(
    const void *q, kv_dtype q_dtype, const int32_t *query_start_loc, int32_t num_seqs,
    int32_t num_tokens, int32_t max_query_len, int32_t num_q_heads, const void *k_cache,
    const void *v_cache, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
    int32_t num_blocks, const int32_t *block_table, int64_t bt_stride, int32_t max_blocks_per_seq,
    const int32_t *seq_lens, int32_t max_seq_len, float scale, int32_t window, int32_t num_sinks,
    const float *k_scales, const float *v_scales, int32_t group_size, int32_t num_workers,
    void *workspace, size_t workspace_bytes, void *out, float *lse_out, int32_t *d_err,
    void *stream);

/* Workspace bytes of the prefill calls for these sizes (cache_dtype KV_INT4 for the second; SIZE_MAX when they
 * are invalid or unsupported, with the reason in kv_last_error(), or no device can be queried).  A larger
 * max_query_len never needs less; lengths, window and sinks do not matter. */
KV_API size_t kv_paged_attention_prefill_sinks_workspace_size(
    int32_t num_seqs, int32_t max_query_len, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, kv_dtype cache_dtype, int32_t max_seq_len, int32_t window, int32_t num_sinks,
    int32_t num_workers);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_SINKS_H */
