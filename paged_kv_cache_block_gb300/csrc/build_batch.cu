// The metadata of a step from its requests' lengths: query offsets, positions, slots, new
// block-table entries and tree masks ("vLLM의 KV cache 연결 흐름", sections "GPU worker가 하는 일"
// and "Slot mapping은 왜 필요한가": new block ids appended to the request's row, a slot per token).
//
// Two prefix sums over the requests (tokens, then blocks needed), and from them everything else
// by index.  Integer work on a few bytes a token: below about 100,000 tokens the time is that of
// one launch and its dependent round trips, so there is one launch and no grid-wide step: every
// CTA computes the prefix sums itself (a chunk of kThreads requests at a time, one request a
// thread), then the grid shares out the chunk's tokens and new blocks.
#include "common.cuh"
#include "kernels.h"

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// Inclusive prefix sum over the block's threads; *total receives the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *sums, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int64_t s = sums[w];
        all += s;
        if (w < warp) before += s;
    }
    __syncthreads();
    *total = all;
    return v + before;
}

// The last i in [0, n) with start[i] <= x (start is non-decreasing, start[0] <= x).
__device__ __forceinline__ int last_at_most(const int64_t *start, int n, int64_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) build_batch_kernel(const BatchArgs a) {
    __shared__ int64_t sums[kWarps];
    __shared__ int64_t tok[kThreads];   // first token of each request of the chunk
    __shared__ int64_t blk[kThreads];   // blocks taken before it
    __shared__ int32_t ctx_s[kThreads], held_s[kThreads];
    __shared__ uint8_t served_s[kThreads];
    const int tid = threadIdx.x;
    const bool writer = blockIdx.x == 0;
    const int shift = a.block_shift;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t gtid = static_cast<int64_t>(blockIdx.x) * kThreads + tid;
    const int32_t start = a.free_start ? *a.free_start : 0;
    // a start outside the list: nothing can be taken
    const int64_t avail = start >= 0 && start <= a.num_free ? a.num_free - start : 0;
    int64_t tokens = 0, blocks = 0, taken = 0;  // of the requests before this chunk
    for (int base = 0; base < a.num_seqs; base += kThreads) {
        const int r = base + tid;
        const int count = min(kThreads, a.num_seqs - base);
        int32_t c = 0, n = 0, h = 0;
        if (r < a.num_seqs) {
            c = a.context_lens[r];
            n = a.new_lens[r];
            h = a.held_blocks ? a.held_blocks[r]
                              : static_cast<int32_t>((static_cast<int64_t>(max(c, 0)) + (1 << shift) - 1) >> shift);
        }
        const int64_t len = static_cast<int64_t>(c) + n;
        const int64_t total = (len + (1 << shift) - 1) >> shift;
        bool ok = c >= 0 && n >= 0 && h >= 0 && h <= a.max_blocks_per_seq && total <= a.max_blocks_per_seq &&
                  !(a.parents && n > KV_MAX_TREE);
        int64_t sum;
        const int64_t end = tokens + block_scan(max(n, 0), sums, &sum);
        const int64_t first = end - max(n, 0);
        if (n > 0 && end > a.num_tokens) ok = false;
        if (writer && !ok) report(a.d_err, KV_DERR_BAD_LEN);
        const int64_t need = ok && n > 0 && total > h ? total - h : 0;
        int64_t need_sum;
        const int64_t blk_end = blocks + block_scan(need, sums, &need_sum);
        const bool granted = need == 0 || blk_end <= avail;
        const bool served = ok && granted;
        if (writer && !granted) report(a.d_err, KV_DERR_NO_BLOCKS);
        tok[tid] = first;
        blk[tid] = blk_end - need;
        ctx_s[tid] = c;
        held_s[tid] = h;
        served_s[tid] = served;
        if (writer && r < a.num_seqs) {
            if (r == 0) a.query_start_loc[0] = 0;
            a.query_start_loc[r + 1] = static_cast<int32_t>(end < a.num_tokens ? end : a.num_tokens);
            a.seq_lens[r] = served ? static_cast<int32_t>(len) : 0;
            a.held_out[r] = h + (served ? static_cast<int32_t>(need) : 0);
        }
        // the granted needs are a prefix of the chunk's: what they take in all
        int64_t granted_sum;
        block_scan(granted ? need : 0, sums, &granted_sum);  // ends with a barrier: the tables are written
        taken += granted_sum;

        // new table entries
        for (int64_t e = blocks + gtid; e < blocks + granted_sum; e += stride) {
            const int i = last_at_most(blk, count, e);
            const int32_t id = a.free_blocks[start + e];
            if (id >= 0 && id < a.num_blocks)
                a.block_table[(base + i) * a.bt_stride + held_s[i] + (e - blk[i])] = id;
            else
                report(a.d_err, KV_DERR_BAD_BLOCK);
        }
        // tokens
        const int64_t tok_end = min(tokens + sum, static_cast<int64_t>(a.num_tokens));
        for (int64_t t = tokens + gtid; t < tok_end; t += stride) {
            const int i = last_at_most(tok, count, t);
            const int32_t k = static_cast<int32_t>(t - tok[i]);  // index within the request
            int32_t pos = -1;
            int64_t slot = -1;
            uint64_t mask = 0;
            if (served_s[i]) {
                const int32_t at = ctx_s[i] + k;
                pos = at;
                const int32_t lb = at >> shift;
                const int32_t id = lb < held_s[i] ? a.block_table[(base + i) * a.bt_stride + lb]
                                                  : a.free_blocks[start + blk[i] + (lb - held_s[i])];
                if (id >= 0 && id < a.num_blocks) slot = (static_cast<int64_t>(id) << shift) + (at & ((1 << shift) - 1));
                else report(a.d_err, KV_DERR_BAD_BLOCK);
                if (a.parents) {
                    // up the chain of parents: each an earlier token, so at most k steps
                    int32_t j = k, depth = 0;
                    mask = 1ull << k;
                    for (;;) {
                        const int32_t p = a.parents[tok[i] + j];
                        if (p < -1 || p >= j) {
                            report(a.d_err, KV_DERR_BAD_TREE);
                            break;
                        }
                        if (p < 0) break;
                        mask |= 1ull << p;
                        ++depth;
                        j = p;
                    }
                    pos = ctx_s[i] + depth;
                }
            }
            a.positions[t] = pos;
            a.slot_mapping[t] = slot;
            if (a.tree_mask) a.tree_mask[t] = mask;
        }
        tokens += sum;
        blocks += need_sum;
        __syncthreads();  // the tables are rewritten by the next chunk
    }
    if (writer && tid == 0) {
        if (a.num_seqs == 0) a.query_start_loc[0] = 0;
        *a.free_next = start + static_cast<int32_t>(taken);
    }
    // rows behind the last request
    for (int64_t t = tokens + gtid; t < a.num_tokens; t += stride) {
        a.positions[t] = -1;
        a.slot_mapping[t] = -1;
        if (a.tree_mask) a.tree_mask[t] = 0;
    }
}

}  // namespace

cudaError_t launch_build_batch(const BatchArgs &a, int sm_count, cudaStream_t stream) {
    const int64_t want = (static_cast<int64_t>(a.num_tokens) + kThreads - 1) / kThreads;
    const int grid = static_cast<int>(want < 1 ? 1 : (want < 2 * sm_count ? want : 2 * sm_count));
    build_batch_kernel<<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
