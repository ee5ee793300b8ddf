// Attention of drafted trees over the paged cache (speculative decoding: "vLLM의 KV cache 연결
// 흐름", section "EngineCore가 하는 일", several tokens a request and step; attention through the
// block table as in its section "Slot mapping은 왜 필요한가").
//
// Row i of a sequence attends the context keys (those inside its window) and the drafted keys of
// its mask:  out = sum_j p_j V_j / sum_j p_j,  p_j = exp2(scale log2(e) q.K_j - m).
// One warp per (row, query head); a lane holds D / 32 dims of q and of the output, keys one after
// another with a running maximum and sum in float32.
#include "common.cuh"
#include "kernels.h"

namespace pkv {
namespace {

template <typename T, int D>
__global__ void __launch_bounds__(256) tree_attention_kernel(const TreeArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t t = w / a.num_q_heads;
    const int hq = static_cast<int>(w - t * a.num_q_heads);
    if (t >= a.num_tokens) return;
    // the sequence: the last b with query_start_loc[b] <= t
    int lo = 0, hi = a.num_seqs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.query_start_loc[mid + 1] <= t) lo = mid + 1;
        else hi = mid;
    }
    const int b = lo;
    if (b >= a.num_seqs || t < a.query_start_loc[b]) return;
    const int q0 = a.query_start_loc[b], n = a.query_start_loc[b + 1] - q0, L = a.seq_lens[b];
    const int64_t row = t * a.num_q_heads + hq;
    T *out = static_cast<T *>(a.out) + row * D + lane * E;
    const bool ok = q0 >= 0 && n <= a.max_query_len && q0 + n <= a.num_tokens && L >= n && L <= a.max_seq_len &&
                    (L + a.block_size - 1) / a.block_size <= a.max_blocks_per_seq;
    float o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    if (!ok) {
        if (lane == 0) report(a.d_err, KV_DERR_BAD_LEN);
    } else {
        const int h = hq / (a.num_q_heads / a.num_kv_heads), ctx = L - n;
        const uint64_t mask = a.tree_mask[t] & (n >= 64 ? ~0ull : (1ull << n) - 1);
        const int pos = ctx - 1 + __popcll(mask);
        const int first = a.window > 0 ? max(0, pos - a.window + 1) : 0;
        float q[E];
        const T *qs = static_cast<const T *>(a.q) + row * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = to_float<T>(qs[e]);
        for (int j = first; j < L; ++j) {
            if (j >= ctx && !((mask >> (j - ctx)) & 1)) continue;
            const int id = a.block_table[b * a.bt_stride + j / a.block_size];
            const bool good = id >= 0 && id < a.num_blocks;
            if (!good && lane == 0) report(a.d_err, KV_DERR_BAD_BLOCK);
            const int64_t at = ((static_cast<int64_t>(good ? id : 0) * a.block_size + j % a.block_size) * a.num_kv_heads + h) * D + lane * E;
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s += q[e] * (good ? to_float<T>(static_cast<const T *>(a.k_cache)[at + e]) : 0.f);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            s *= a.scale_log2;
            const float mn = fmaxf(m, s), f = m == mn ? 1.f : fast_exp2(m - mn), p = fast_exp2(s - mn);
            m = mn;
            l = l * f + p;
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] = o[e] * f + p * (good ? to_float<T>(static_cast<const T *>(a.v_cache)[at + e]) : 0.f);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = from_float<T>(o[e] * inv);
    if (a.lse_out && lane == 0) a.lse_out[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <typename T> cudaError_t launch_typed(const TreeArgs &a, int head_dim, cudaStream_t stream) {
    const int64_t blocks = (static_cast<int64_t>(a.num_tokens) * a.num_q_heads + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (head_dim == 128) tree_attention_kernel<T, 128><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
    else tree_attention_kernel<T, 64><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_attention(const TreeArgs &a, int head_dim, int q_dtype, cudaStream_t stream) {
    if (q_dtype == KV_BF16) return launch_typed<__nv_bfloat16>(a, head_dim, stream);
    return launch_typed<__half>(a, head_dim, stream);
}

}  // namespace pkv
