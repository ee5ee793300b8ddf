// The metadata of a step from its requests' lengths: query offsets, positions, slots, new
// block-table entries and tree masks ("vLLM의 KV cache 연결 흐름", sections "GPU worker가 하는 일"
// and "Slot mapping은 왜 필요한가": new block ids appended to the request's row, a slot per token).
//
// Two prefix sums over the requests (tokens, then blocks needed), and from them everything else
// by index.  Integer work on a few bytes a token: below about 100,000 tokens the time is that of
// one launch and its dependent round trips, so there is one launch and no grid-wide step: every
// CTA computes the prefix sums itself (a chunk of kThreads requests at a time, one request a
// thread), then the grid shares out the chunk's new blocks and tokens.  Without trees a thread takes
// one token, or four in a row (one search and mostly one block id, whole-line stores) when there are
// more than the grid has threads: 256 requests of one token 4.5 us with one, 5.9 with four; 512 prompts
// of 557,000 tokens 9.7 and 7.8.  With trees a warp takes a request, whose at most 64 tokens find their
// ancestors by pointer jumping between lanes (128 trees: 5.1 us, 6.8 when each token walked up by itself).
#include "common.cuh"
#include "dependent_launch.cuh"
#include "kernels.h"

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// Inclusive prefix sum over the block's threads; *total receives the sum.  sums is written before and
// read after the barrier inside.
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

// The chunk's requests, in shared memory.
struct Chunk {
    int64_t tok[kThreads + 1];  // first token of each, and the end of the last
    int64_t blk[kThreads];      // blocks taken before it
    int32_t ctx[kThreads], held[kThreads];
    uint8_t served[kThreads];
};

// The block that holds logical block lb of request i (base + i of the batch), or -1.
__device__ __forceinline__ int32_t block_of(const BatchArgs &a, const Chunk &ch, int base, int i, int32_t start, int32_t lb) {
    const int32_t id = lb < ch.held[i] ? a.block_table[(base + i) * a.bt_stride + lb]
                                       : a.free_blocks[start + ch.blk[i] + (lb - ch.held[i])];
    if (id >= 0 && id < a.num_blocks) return id;
    report(a.d_err, KV_DERR_BAD_BLOCK);
    return -1;
}

__device__ __forceinline__ int64_t slot_in(const BatchArgs &a, int32_t id, int32_t at) {
    const int shift = a.block_shift;
    return id < 0 ? -1 : (static_cast<int64_t>(id) << shift) + (at & ((1 << shift) - 1));
}

// Position and slot of token t, along its request.
__device__ __forceinline__ void one_token(const BatchArgs &a, const Chunk &ch, int base, int count, int32_t start, int64_t t) {
    const int i = last_at_most(ch.tok, count, t);
    const bool served = ch.served[i];
    const int32_t at = ch.ctx[i] + static_cast<int32_t>(t - ch.tok[i]);
    a.positions[t] = served ? at : -1;
    a.slot_mapping[t] = served ? slot_in(a, block_of(a, ch, base, i, start, at >> a.block_shift), at) : -1;
}

// Tokens t0 .. t0 + 3 as far as they lie in [lo, hi).
__device__ __forceinline__ void four_tokens(const BatchArgs &a, const Chunk &ch, int base, int count, int32_t start,
                                            int64_t t0, int64_t lo, int64_t hi) {
    int i = last_at_most(ch.tok, count, t0 > lo ? t0 : lo);
    int32_t pos[4];
    int64_t slot[4];
    int32_t lb_i = -1, lb = -1, id = -1;  // the block id at hand: logical block lb of request lb_i
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t t = t0 + k;
        pos[k] = -1;
        slot[k] = -1;
        if (t < lo || t >= hi) continue;
        while (i + 1 < count && ch.tok[i + 1] <= t) ++i;
        if (!ch.served[i]) continue;
        pos[k] = ch.ctx[i] + static_cast<int32_t>(t - ch.tok[i]);
        const int32_t need = pos[k] >> a.block_shift;
        if (need != lb || i != lb_i) {
            lb = need, lb_i = i;
            id = block_of(a, ch, base, i, start, lb);
        }
        slot[k] = slot_in(a, id, pos[k]);
    }
    if (a.aligned && t0 >= lo && t0 + 4 <= hi) {
        *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        reinterpret_cast<longlong2 *>(a.slot_mapping + t0)[0] = make_longlong2(slot[0], slot[1]);
        reinterpret_cast<longlong2 *>(a.slot_mapping + t0)[1] = make_longlong2(slot[2], slot[3]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t t = t0 + k;
        if (t < lo || t >= hi) continue;
        a.positions[t] = pos[k];
        a.slot_mapping[t] = slot[k];
    }
}

// The tree of request i, by one warp: lane l holds tokens l and l + 32.
__device__ __forceinline__ void tree_tokens(const BatchArgs &a, const Chunk &ch, int base, int i, int32_t start) {
    const int lane = threadIdx.x & 31;
    const int64_t t0 = ch.tok[i], t1 = min(ch.tok[i + 1], static_cast<int64_t>(a.num_tokens));
    if (!ch.served[i]) {
        for (int64_t t = t0 + lane; t < t1; t += 32) {
            a.positions[t] = -1;
            a.slot_mapping[t] = -1;
            a.tree_mask[t] = 0;
        }
        return;
    }
    const int n = static_cast<int>(t1 - t0);  // at most 64
    int32_t up[2];      // a token above: the parent, then twice as far each round (-1: past the root)
    uint64_t mask[2];   // the tokens from here up to `up`, without it
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int k = lane + 32 * e;
        up[e] = -1;
        mask[e] = 1ull << k;
        if (k < n) {
            const int32_t p = a.parents[t0 + k];
            if (p >= -1 && p < k) up[e] = p;
            else report(a.d_err, KV_DERR_BAD_TREE);
        }
    }
    // round r covers 2^r ancestors: 6 rounds for 64 tokens, 5 when all lie in the lower half
    const int rounds = n > 32 ? 6 : 5;
    for (int r = 0; r < rounds; ++r) {
        uint64_t m[2];
        int32_t u[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int from = up[e] & 31;
            const uint64_t m0 = __shfl_sync(0xffffffffu, mask[0], from), m1 = __shfl_sync(0xffffffffu, mask[1], from);
            const int32_t u0 = __shfl_sync(0xffffffffu, up[0], from), u1 = __shfl_sync(0xffffffffu, up[1], from);
            m[e] = up[e] < 0 ? 0 : (up[e] < 32 ? m0 : m1);
            u[e] = up[e] < 0 ? -1 : (up[e] < 32 ? u0 : u1);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) mask[e] |= m[e], up[e] = u[e];
        if (!__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) break;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int k = lane + 32 * e;
        if (k >= n) continue;
        a.positions[t0 + k] = ch.ctx[i] + __popcll(mask[e]) - 1;
        const int32_t at = ch.ctx[i] + k;
        a.slot_mapping[t0 + k] = slot_in(a, block_of(a, ch, base, i, start, at >> a.block_shift), at);
        a.tree_mask[t0 + k] = mask[e];
    }
}

__global__ void __launch_bounds__(kThreads) build_batch_kernel(const BatchArgs a) {
    __shared__ int64_t tok_sums[kWarps], blk_sums[kWarps];
    __shared__ Chunk ch;
    __shared__ unsigned long long refused_at;  // blocks taken before the first request without enough
    const int tid = threadIdx.x;
    const bool writer = blockIdx.x == 0;
    const int shift = a.block_shift;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t gtid = static_cast<int64_t>(blockIdx.x) * kThreads + tid;
    previous_kernel_done();
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
        if (tid == 0) refused_at = ~0ull;
        const int64_t len = static_cast<int64_t>(c) + n;
        const int64_t total = (len + (1 << shift) - 1) >> shift;
        bool ok = c >= 0 && n >= 0 && h >= 0 && h <= a.max_blocks_per_seq && total <= a.max_blocks_per_seq &&
                  !(a.parents && n > KV_MAX_TREE);
        int64_t sum;
        const int64_t end = tokens + block_scan(max(n, 0), tok_sums, &sum);
        if (n > 0 && end > a.num_tokens) ok = false;
        if (writer && !ok) report(a.d_err, KV_DERR_BAD_LEN);
        const int64_t need = ok && n > 0 && total > h ? total - h : 0;
        int64_t need_sum;
        const int64_t blk_end = blocks + block_scan(need, blk_sums, &need_sum);
        const bool granted = need == 0 || blk_end <= avail;
        const bool served = ok && granted;
        if (!granted) {
            if (writer) report(a.d_err, KV_DERR_NO_BLOCKS);
            atomicMin(&refused_at, static_cast<unsigned long long>(blk_end - need));
        }
        ch.tok[tid] = end - max(n, 0);
        if (tid == count - 1) ch.tok[count] = end;
        ch.blk[tid] = blk_end - need;
        ch.ctx[tid] = c;
        ch.held[tid] = h;
        ch.served[tid] = served;
        if (writer && r < a.num_seqs) {
            if (r == 0) a.query_start_loc[0] = 0;
            a.query_start_loc[r + 1] = static_cast<int32_t>(end < a.num_tokens ? end : a.num_tokens);
            a.seq_lens[r] = served ? static_cast<int32_t>(len) : 0;
            a.held_out[r] = h + (served ? static_cast<int32_t>(need) : 0);
        }
        __syncthreads();
        // the granted needs are a prefix of the chunk's: up to the first request without enough
        const int64_t blk_stop = static_cast<int64_t>(
            min(refused_at, static_cast<unsigned long long>(blocks + need_sum)));
        taken += blk_stop - blocks;

        // new table entries
        for (int64_t e = blocks + gtid; e < blk_stop; e += stride) {
            const int i = last_at_most(ch.blk, count, e);
            const int32_t id = a.free_blocks[start + e];
            if (id >= 0 && id < a.num_blocks)
                a.block_table[(base + i) * a.bt_stride + ch.held[i] + (e - ch.blk[i])] = id;
            else
                report(a.d_err, KV_DERR_BAD_BLOCK);
        }
        // tokens
        if (a.parents) {
            for (int i = static_cast<int>(gtid >> 5); i < count; i += static_cast<int>(stride >> 5))
                tree_tokens(a, ch, base, i, start);
        } else {
            const int64_t hi = min(tokens + sum, static_cast<int64_t>(a.num_tokens));
            if (a.fours)
                for (int64_t t0 = (tokens / 4 + gtid) * 4; t0 < hi; t0 += 4 * stride)
                    four_tokens(a, ch, base, count, start, t0, tokens, hi);
            else
                for (int64_t t = tokens + gtid; t < hi; t += stride) one_token(a, ch, base, count, start, t);
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

cudaError_t launch_build_batch(const BatchArgs &args, int sm_count, cudaStream_t stream) {
    BatchArgs a = args;
    const int64_t most = 2 * static_cast<int64_t>(sm_count);
    a.fours = a.num_tokens > most * kThreads;
    // a request a warp, or a token or four a thread
    const int64_t threads = a.parents ? 32 * static_cast<int64_t>(a.num_seqs) : (a.fours ? a.num_tokens / 4 + 1 : a.num_tokens);
    const int64_t want = (threads + kThreads - 1) / kThreads;
    return launch_dependent(build_batch_kernel, dim3(static_cast<unsigned>(want < 1 ? 1 : (want < most ? want : most))),
                            dim3(kThreads), 0, stream, a);
}

}  // namespace pkv
