// Prefill attention with a sliding window and sinks over E4M3 and INT4 caches: the instantiations of
// prefill_sinks.cuh that widen the codes in shared memory.
#include "prefill_sinks.cuh"

namespace pkv {

cudaError_t launch_prefill_sinks_wide(const CUtensorMap &none, const SinkPrefillParams &p, int cache_dtype, int q_dtype,
                                      int dev, cudaStream_t stream) {
    using namespace sinks;
    const bool bf16 = q_dtype == KV_BF16;
    if (cache_dtype == KV_INT4)
        return bf16 ? launch_typed<__nv_bfloat16, 128, kCacheInt4>(none, none, none, p, dev, stream)
                    : launch_typed<__half, 128, kCacheInt4>(none, none, none, p, dev, stream);
    return bf16 ? launch_typed<__nv_bfloat16, 128, kCacheE4M3>(none, none, none, p, dev, stream)
                : launch_typed<__half, 128, kCacheE4M3>(none, none, none, p, dev, stream);
}

}  // namespace pkv
