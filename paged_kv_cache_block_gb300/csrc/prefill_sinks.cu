// Prefill attention with a sliding window and sinks: the plan, the launch, and the instantiations over
// 16-bit caches (those over E4M3 and INT4 caches: prefill_sinks_wide.cu).
#include <algorithm>

#include "prefill_sinks.cuh"

namespace pkv {

namespace {
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
}  // namespace

TreePlan plan_prefill_sinks(int max_query_len, int group, int head_dim, int num_workers, int sm_count) {
    TreePlan t;
    t.workers = num_workers > 0 ? num_workers : sm_count;
    t.heads_per_item = 1;
    t.tokens_per_tile = kTreeRows / group;
    t.key_shift = 7;
    t.rows_per_item = max_query_len > t.tokens_per_tile ? 2 * kTreeRows : kTreeRows;
    t.smem_bytes = head_dim == 128 ? sinks::Tile<128>::smem(true) : sinks::Tile<64>::smem(false);  // (at most)
    const size_t parts = static_cast<size_t>(2) * t.workers * t.rows_per_item;
    t.lse_off = align256(2 * sizeof(int4) * static_cast<size_t>(t.workers));
    t.o_off = t.lse_off + align256(4 * parts);
    t.workspace_bytes = t.o_off + 4 * parts * head_dim;
    return t;
}

cudaError_t launch_prefill_sinks(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                 const SinkPrefillArgs &a, const TreePlan &plan, void *workspace, int head_dim,
                                 int q_dtype, int cache_dtype, int dev, cudaStream_t stream) {
    SinkPrefillParams p;
    p.t.a = a.t;
    p.t.group = a.t.num_q_heads / a.t.num_kv_heads;
    p.t.tokens_per_tile = plan.tokens_per_tile;
    p.t.heads_per_item = 1;
    p.t.key_shift = plan.key_shift;
    p.t.workers = plan.workers;
    p.t.rows_per_item = plan.rows_per_item;
    // max_query_len may be any bound: no accepted sequence has more rows than there are tokens
    const int64_t most = std::min(a.t.max_query_len, a.t.num_tokens);
    const int64_t row_tiles = (most + plan.tokens_per_tile - 1) / plan.tokens_per_tile;
    p.t.items_per_seq = static_cast<int>((row_tiles + 1) / 2 * a.t.num_kv_heads);
    char *ws = static_cast<char *>(workspace);
    p.t.ws_first = reinterpret_cast<int4 *>(ws);
    p.t.ws_lse = reinterpret_cast<float *>(ws + plan.lse_off);
    p.t.ws_o = reinterpret_cast<float4 *>(ws + plan.o_off);
    p.bs_shift = 0;
    while ((1 << p.bs_shift) < a.t.block_size) ++p.bs_shift;
    p.num_sinks = a.num_sinks;
    p.sink_blocks = (a.num_sinks + a.t.block_size - 1) >> p.bs_shift;
    p.q = a.q;
    p.k_cache = a.k_cache;
    p.v_scale = a.v_scale;
    p.k_gscales = a.k_gscales;
    p.v_gscales = a.v_gscales;
    p.group_shift = a.group_shift;
    if (cache_dtype == KV_FP8_E4M3 || cache_dtype == KV_INT4)
        return launch_prefill_sinks_wide(tq, p, cache_dtype, q_dtype, dev, stream);
    using namespace sinks;
    if (q_dtype == KV_BF16)
        return head_dim == 128 ? launch_typed<__nv_bfloat16, 128, kCache16>(tq, tk, tv, p, dev, stream)
                               : launch_typed<__nv_bfloat16, 64, kCache16>(tq, tk, tv, p, dev, stream);
    return head_dim == 128 ? launch_typed<__half, 128, kCache16>(tq, tk, tv, p, dev, stream)
                           : launch_typed<__half, 64, kCache16>(tq, tk, tv, p, dev, stream);
}

}  // namespace pkv
