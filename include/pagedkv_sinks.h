/*
 * pagedkv_sinks.h - attention with a sliding window and sinks over the paged cache (part of
 * libpagedkv.so).
 *
 *   kv_paged_attention_decode_sinks       decode, 16-bit and E4M3 caches
 *   kv_paged_attention_decode_sinks_int4  decode, INT4 caches
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
 *     or an infinity in a value that it does see reaches that dim of its result.
 *   - Softmax sums are float32, of the weights before they are rounded to 16 bits for the second product
 *     (INT4 decode: of the rounded weights, whose codes' offset comes out exactly with them).  fp16
 *     weights are formed 2^14 higher than they are, so that the many small weights beside a sink that
 *     holds nearly all of them keep their digits.
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

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_SINKS_H */
