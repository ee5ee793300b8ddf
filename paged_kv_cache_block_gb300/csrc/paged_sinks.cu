// Decode attention with a sliding window and sinks (kv_paged_attention_decode_sinks): the
// instantiations of paged_decode_kernel.cuh for it, and the row merge that keeps NaN.
//
// A row at position p sees key j <= p when j > p - window or j < num_sinks.  The softmax, GQA and
// block-table reads are those of the windowed decode ("vLLM Worker侧GPU KV Cache初始化流程深度解析",
// section "混合注意力机制"; "Understanding PageAttention Memory Optimization", section "Handling
// Softmax Across Blocks"); the pages have no sinks.
//
// What bounds it is what bounds the windowed decode, reading the keys that some row sees; on the
// shortened key axis (SinkAxis) the sinks cost one block a sequence.  What differs from the kernel
// without sinks is compile-time (kSinks), so that kernel's results are as they were.  Times of the call, one
// GB300, blocks of 16:
//   1 sequence of 30000 tokens, window 4096, 4 sinks, 32/8 heads of 128       14.1 us, the host call alone 14.4
//   128 sequences, 4 new tokens each, the same window                          203 us, 5.95 TB/s
//   32 sequences to 131072, window 8192, 64 sinks, 64/8 heads, E4M3             99 us, 5.5 TB/s
//   256 sequences to 8192, window 2048, 16 sinks, 32/8 heads, INT4             118 us, 4.3 TB/s
//   64 sequences to 2048, window 512, 1 sink, 12 heads of 64                  26.4 us, 3.4 TB/s
#include "paged_decode_kernel.cuh"

namespace pkv {

cudaError_t launch_lse_merge_nan(const KernelParams &kp, int num_workers, int q_dtype, cudaStream_t stream) {
    return q_dtype == KV_F16 ? row_merge<__half, 128, true>(kp, num_workers, stream)
                             : row_merge<__nv_bfloat16, 128, true>(kp, num_workers, stream);
}

cudaError_t launch_paged_decode_sinks(const CUtensorMap &tmap_k, const CUtensorMap &tmap_v, const DecodeArgs &a,
                                      const SinkArgs &sinks, const DecodePlan &plan, int q_dtype, int cache_dtype,
                                      cudaStream_t stream) {
    KernelParams kp = make_params(a, plan);
    kp.sinks = sinks;
    const bool f16 = q_dtype == KV_F16;
    if (cache_dtype == KV_FP8_E4M3)
        return f16 ? launch_rows<__half, Fp8E4M3, 128, false, true>(tmap_k, tmap_v, kp, plan, stream)
                   : launch_rows<__nv_bfloat16, Fp8E4M3, 128, false, true>(tmap_k, tmap_v, kp, plan, stream);
    if (a.head_dim == 64)
        return f16 ? launch_rows<__half, __half, 64, false, true>(tmap_k, tmap_v, kp, plan, stream)
                   : launch_rows<__nv_bfloat16, __nv_bfloat16, 64, false, true>(tmap_k, tmap_v, kp, plan, stream);
    return f16 ? launch_rows<__half, __half, 128, false, true>(tmap_k, tmap_v, kp, plan, stream)
               : launch_rows<__nv_bfloat16, __nv_bfloat16, 128, false, true>(tmap_k, tmap_v, kp, plan, stream);
}

}  // namespace pkv
