// Pieces shared by the tree attention kernels (tree_attention.cu, tree_packed.cu): the work list of
// (item, key tile) and its equal shares, the masks of drafted trees, the handling of values that
// not every row sees, and the merge of items that lie in several shares.
#pragma once

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace pkv {

constexpr int kTreeRows = 128;         // query rows of a row tile = TMEM lanes
constexpr int kHalf = 128 * 128;       // 128 rows x 64 16-bit elements (one swizzle column)
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;   // a row's reference maximum moves when exceeded by more
constexpr int kItemCost = 2;           // an item's fixed cost in key tiles
constexpr int kMinShare = 3;           // least cost of a share: more than kItemCost, so that it holds a tile
constexpr int kFlags = 8;              // pieces whose odd-value flags are kept

struct TreeParams {
    TreeArgs a;
    int group;            // query heads of a kv head
    int tokens_per_tile;  // drafted tokens of a kv head's rows in a row tile
    int heads_per_item;   // 1: items of two row tiles of a kv head; 2 or 4: of so many kv heads
    int key_shift;        // log2 of the keys of a key tile
    int workers;          // shares at most
    int rows_per_item;    // rows of a partial result
    int4 *ws_first;       // [2 * workers] first piece of each share: (sequence, item of it, key tile of it,
                          // -), (first row, rows, -, -) of the sequence; sequence -1: no share
    float *ws_lse;        // [2 * workers][rows_per_item] log2-sum-exp2 of the partial results
    float *ws_o;          // [2 * workers][rows_per_item][D] partial results, normalised
};

// A sequence's part of the work list.
struct Seq {
    int q0, n, L, ctx, kv_lo;  // first row, rows, length, context, first key any row sees
    int j0, tiles;             // key tiles j0 .. j0 + tiles - 1
    int items, pairs;          // items; of one kv head when items are pairs of row tiles
};

// The sequence's lengths; false when it has no rows, or is rejected (*rejected).
__device__ __forceinline__ bool load_seq(const TreeParams &p, int b, Seq &s, bool *rejected) {
    const TreeArgs &a = p.a;
    s.q0 = a.query_start_loc[b];
    s.n = a.query_start_loc[b + 1] - s.q0;
    s.L = a.seq_lens[b];
    const int bs = a.block_size;
    *rejected = s.n > 0 && !(s.n <= a.max_query_len && s.q0 >= 0 && s.q0 <= a.num_tokens - s.n && s.L >= s.n &&
                             s.L <= a.max_seq_len && (s.L - 1) / bs < a.max_blocks_per_seq);
    if (s.n <= 0 || *rejected) return false;
    s.ctx = s.L - s.n;
    s.kv_lo = a.window > 0 ? max(0, s.ctx - a.window) : 0;
    s.j0 = s.kv_lo >> p.key_shift;
    s.tiles = ((s.L - 1) >> p.key_shift) + 1 - s.j0;
    if (p.heads_per_item == 1) {
        const int row_tiles = (s.n + p.tokens_per_tile - 1) / p.tokens_per_tile;
        s.pairs = (row_tiles + 1) >> 1;
        s.items = s.pairs * a.num_kv_heads;
    } else {
        s.pairs = 1;
        s.items = (a.num_kv_heads + p.heads_per_item - 1) / p.heads_per_item;
    }
    return true;
}

__device__ __forceinline__ int64_t seq_cost(const TreeParams &p, int b) {
    Seq s;
    bool rejected;
    if (!load_seq(p, b, s, &rejected)) return 0;
    return static_cast<int64_t>(s.tiles + kItemCost) * s.items;
}

// The share [x0, x1) of CTA c (x0 == x1: none), and where it starts: sequence, item and the cost
// where that item starts.  Computed by the whole block; b, idx and at are set in shared memory and
// valid after the next __syncthreads.
struct ShareStart {
    int64_t at;
    int b, idx;
};

template <int kThreads>
__device__ __forceinline__ void share_of_cta(const TreeParams &p, int c, int64_t &x0, int64_t &x1, ShareStart &start) {
    __shared__ int64_t warp_sum[kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_seqs = p.a.num_seqs;
    const int per = (num_seqs + kThreads - 1) / kThreads;
    const int b_lo = min(num_seqs, static_cast<int>(threadIdx.x) * per), b_hi = min(num_seqs, b_lo + per);
    int64_t sum = 0;
    for (int b = b_lo; b < b_hi; ++b) sum += seq_cost(p, b);
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    const int64_t most = max(int64_t(1), total / kMinShare);
    const int shares = total == 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(p.workers), most));
    x0 = x1 = 0;
    if (c >= shares) return;
    x0 = total * c / shares;
    x1 = total * (c + 1) / shares;
    if (x0 >= before && x0 < before + sum) {  // one thread
        int64_t at = before;
        for (int b = b_lo; b < b_hi; ++b) {
            const int64_t cost = seq_cost(p, b);
            if (x0 < at + cost) {
                Seq s;
                bool rejected;
                load_seq(p, b, s, &rejected);
                start.b = b;
                start.idx = static_cast<int>((x0 - at) / (s.tiles + kItemCost));
                start.at = at + static_cast<int64_t>(start.idx) * (s.tiles + kItemCost);
                break;
            }
            at += cost;
        }
    }
}

// Rows of rejected sequences are 0 (lse -inf): the CTAs take the sequences in turn.
template <typename T, int D> __device__ __forceinline__ void zero_rejected(const TreeParams &p) {
    const TreeArgs &a = p.a;
    for (int b = blockIdx.x; b < a.num_seqs; b += gridDim.x) {
        Seq s;
        bool rejected;
        load_seq(p, b, s, &rejected);
        if (!rejected) continue;
        if (threadIdx.x == 0) report(a.d_err, KV_DERR_BAD_LEN);
        const int64_t r0 = max(s.q0, 0), r1 = min(static_cast<int64_t>(s.q0) + s.n, static_cast<int64_t>(a.num_tokens));
        const int64_t rows = (r1 - r0) * a.num_q_heads;
        for (int64_t i = threadIdx.x; i < rows * (D / 8); i += blockDim.x)
            reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + r0 * a.num_q_heads * D)[i] = make_uint4(0, 0, 0, 0);
        if (a.lse_out)
            for (int64_t i = threadIdx.x; i < rows; i += blockDim.x) a.lse_out[r0 * a.num_q_heads + i] = -INFINITY;
    }
}

// The pieces of a share, in order: (item, key tiles ja .. jb - 1).  Every warp walks the same ones.
struct Walk {
    int64_t at;       // cost where the item starts
    int64_t x0, x1;   // the share
    Seq cur;          // the piece's sequence,
    int seq, item;    // its number, the item of it
    int ja, jb;       // and key tiles (absolute)
    bool whole;       // the piece is its whole item
    bool begun;

    __device__ __forceinline__ void start(const TreeParams &p, const ShareStart &st, int64_t x0_, int64_t x1_) {
        seq = st.b, item = st.idx, at = st.at, x0 = x0_, x1 = x1_;
        begun = false;
        bool rejected;
        load_seq(p, seq, cur, &rejected);
    }
    __device__ __forceinline__ bool next(const TreeParams &p) {
        for (;;) {
            if (begun) {  // on to the next item
                at += kItemCost + cur.tiles;
                if (at >= x1) return false;
                if (++item == cur.items) {
                    item = 0;
                    bool rejected = false;
                    do {
                        if (++seq >= p.a.num_seqs) return false;
                    } while (!load_seq(p, seq, cur, &rejected));
                }
            }
            begun = true;
            const int64_t first = at + kItemCost;
            ja = static_cast<int>(max(int64_t(0), x0 - first)) + cur.j0;
            jb = static_cast<int>(min(static_cast<int64_t>(cur.tiles), x1 - first)) + cur.j0;
            whole = ja == cur.j0 && jb == cur.j0 + cur.tiles;
            if (ja < jb) return true;
        }
    }
    // The share's first piece, for the merge.
    __device__ __forceinline__ void record(const TreeParams &p, int c) const {
        p.ws_first[2 * c] = make_int4(seq, item, ja - cur.j0, 0);
        p.ws_first[2 * c + 1] = make_int4(cur.q0, cur.n, cur.pairs, 0);
    }
};

// Where the partial result of the piece goes: a share leaves at most one that starts inside its
// item (slot 2c) and one that starts it (2c + 1).
__device__ __forceinline__ int64_t part_row(const TreeParams &p, int c, bool starts, int row) {
    return static_cast<int64_t>(2 * c + (starts ? 1 : 0)) * p.rows_per_item + row;
}

// Whether key tile j holds a key that not every row of the sequence sees.
__device__ __forceinline__ bool mixed_tile(const TreeParams &p, const Seq &s, int j) {
    const int k0 = j << p.key_shift;
    return k0 + (1 << p.key_shift) > s.ctx || (p.a.window > 0 && k0 < s.ctx + s.n - p.a.window);
}

// The keys k0 .. k0 + 31 a row sees (bit i: key k0 + i): context keys from klo, drafted keys of
// the mask word.
__device__ __forceinline__ uint32_t seen32(int k0, int ctx, int klo, uint64_t mask) {
    const int lo = max(klo - k0, 0), hi = min(ctx - k0, 32);
    uint32_t v = 0;
    if (lo < hi) v = (hi == 32 ? 0xffffffffu : (1u << hi) - 1) & ~((1u << lo) - 1);  // lo < 32
    const int d = k0 - ctx;
    if (d >= 0) v |= d < 64 ? static_cast<uint32_t>(mask >> d) : 0u;
    else if (d > -32) v |= static_cast<uint32_t>(mask << -d);
    return v;
}

template <typename T> struct NonFinite;  // exponent bits all ones
template <> struct NonFinite<__half> { static constexpr uint32_t mask = 0x7C00u; };
template <> struct NonFinite<__nv_bfloat16> { static constexpr uint32_t mask = 0x7F80u; };

template <typename T> __device__ __forceinline__ bool non_finite16(uint32_t bits) {
    return (bits & NonFinite<T>::mask) == NonFinite<T>::mask;
}

__device__ __forceinline__ void st_shared_v4(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// One 16-byte chunk of a V tile in shared memory: zeroed, or its non-finite values zeroed (*odd set).
template <typename T> __device__ __forceinline__ void clean_chunk(uint32_t at, bool zero, bool &odd) {
    if (zero) {
        st_shared_v4(at, make_uint4(0, 0, 0, 0));
        return;
    }
    const uint4 v = ld_shared_v4(at);
    uint32_t u[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (non_finite16<T>(u[e])) u[e] &= 0xffff0000u, bad = true;
        if (non_finite16<T>(u[e] >> 16)) u[e] &= 0x0000ffffu, bad = true;
    }
    if (bad) {
        st_shared_v4(at, make_uint4(u[0], u[1], u[2], u[3]));
        odd = true;
    }
}

// Add the non-finite values of V that a row sees among the keys [k0, k1) to its written result
// (out16 of type T, or a float row): they were zeroed for the products.  Rare, so plain.
template <typename T, int D>
static __device__ __noinline__ void add_non_finite(const TreeArgs &a, int b, int h, int k0, int k1, int ctx, int klo,
                                            uint64_t mask, T *out16, float *out32) {
    for (int k = k0; k < k1; ++k) {
        const bool sees = k < ctx ? k >= klo : (mask >> (k - ctx)) & 1;
        const int id = a.block_table[b * a.bt_stride + k / a.block_size];
        if (!sees || id < 0 || id >= a.num_blocks) continue;
        const T *v = static_cast<const T *>(a.v_cache) +
                     ((static_cast<int64_t>(id) * a.block_size + k % a.block_size) * a.num_kv_heads + h) * D;
        for (int d = 0; d < D; ++d) {
            const float f = to_float<T>(v[d]);
            if (isfinite(f)) continue;
            if (out32) out32[d] += f;
            else out16[d] = from_float<T>(to_float<T>(out16[d]) + f);
        }
    }
}

// Add the non-finite values that the row sees in the piece's mixed tiles.
template <typename T, int D>
__device__ __forceinline__ void add_odd_values(const TreeParams &p, const Walk &w, int h, int klo, uint64_t mask, T *out16,
                                               float *out32) {
    const TreeArgs &a = p.a;
    const Seq &s = w.cur;
    const int ka = w.ja << p.key_shift, kb = min(w.jb << p.key_shift, s.L);
    if (a.window > 0)
        add_non_finite<T, D>(a, w.seq, h, max(ka, s.kv_lo), min(min(s.ctx, s.ctx + s.n - a.window), kb), s.ctx, klo, mask,
                             out16, out32);
    add_non_finite<T, D>(a, w.seq, h, max(ka, s.ctx), kb, s.ctx, klo, mask, out16, out32);
}

// Join the partial results of the item that starts in share c and goes on into the next ones: one
// warp a row.  out = sum_i w_i o_i / sum_i w_i, w_i = exp2(lse_i - max).  What it costs is dependent
// round trips: the shares' records, then the lse and the first four partial rows at once.
template <typename T, int D>
static __global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeParams p) {
    constexpr int E = D / 32;
    const TreeArgs &a = p.a;
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    const int rr = blockIdx.y * 8 + (threadIdx.x >> 5);
    // lane i: the first piece of share c + i (none past the last)
    const int4 none = make_int4(-1, 0, 0, 0);
    int4 rec = c + lane < p.workers ? p.ws_first[2 * (c + lane)] : none;
    const int4 sq = p.ws_first[2 * (c + 1) + 1];
    // share c + 1's decides whether c's last item goes on; c's own, whether that item started before
    const int b = __shfl_sync(0xffffffffu, rec.x, 1), idx = __shfl_sync(0xffffffffu, rec.y, 1);
    const bool same = rec.x == b && rec.y == idx && rec.z > 0;  // this share goes on with the item
    uint32_t go = __ballot_sync(0xffffffffu, same);
    if (b < 0 || !(go & 2) || (go & 1)) return;
    // the row's kv head, token and head of the group
    int h, t, hh;
    const int TQ = p.tokens_per_tile;
    if (p.heads_per_item == 1) {
        h = idx / sq.z;
        const int r = rr & 127, tl = r / p.group;
        t = (2 * (idx - h * sq.z) + (rr >> 7)) * TQ + tl;
        hh = r - tl * p.group;
        if (tl >= TQ || t >= sq.y) return;
    } else {
        const int lanes = p.rows_per_item / p.heads_per_item, r = rr % lanes;
        h = idx * p.heads_per_item + rr / lanes;
        t = r / p.group;
        hh = r - t * p.group;
        if (h >= a.num_kv_heads || t >= sq.y) return;
    }
    // pieces: share c's (its last: slot 2c + 1), then those of the next shares (their first: 2c')
    int last = c + __ffs(~(go | 1)) - 2;  // (ffs 0: all 32 go on)
    if (~(go | 1) == 0) last = c + 31;
    while (last >= c + 31) {
        const int e = last + 1 + lane;
        rec = e < p.workers ? p.ws_first[2 * e] : none;
        go = __ballot_sync(0xffffffffu, rec.x == b && rec.y == idx && rec.z > 0);
        if (go == 0xffffffffu) {
            last += 32;
            continue;
        }
        last += __ffs(~go) - 1;
        break;
    }
    auto part = [&](int e) { return part_row(p, e, e == c, rr); };
    float acc[E], wsum = 0.f, mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int base = c; base <= last; base += 32) {
        const int cnt = min(32, last - base + 1);
        const float l = lane < cnt ? p.ws_lse[part(base + lane)] : -INFINITY;
        float v[4][E];
        auto load = [&](int u0) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float *src = p.ws_o + part(base + u0 + u) * D + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) v[u][e] = u0 + u < cnt ? __ldcg(src + e) : 0.f;
            }
        };
        load(0);
        float m = l;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool nan = __any_sync(0xffffffffu, l != l);
        const float mn = fmaxf(mx, m);
        if (mn == -INFINITY && !nan) continue;  // nothing seen so far
        const float f = mx == -INFINITY ? 0.f : fast_exp2(mx - mn);
        mx = mn;
        wsum *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= f;
        const float wl = l == -INFINITY ? 0.f : fast_exp2(l - mx);
        for (int u0 = 0; u0 < cnt; u0 += 4) {
            if (u0) load(u0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float wu = __shfl_sync(0xffffffffu, wl, (u0 + u) & 31);
                if (u0 + u < cnt && wu != 0.f) {  // a piece of weight 0 adds nothing, whatever it holds
                    wsum += wu;
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += wu * v[u][e];
                }
            }
        }
    }
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
    const int64_t row = static_cast<int64_t>(sq.x + t) * a.num_q_heads + h * p.group + hh;
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + row * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<T>(acc[e] * inv, acc[e + 1] * inv);
    if (a.lse_out && lane == 0) a.lse_out[row] = wsum == 0.f ? -INFINITY : (mx + log2f(wsum)) * 0.69314718055994531f;
}

// The attention kernel and, with more than one share, the merge.
template <typename T, int D, typename Kernel>
static cudaError_t launch_tree_kernel(Kernel kernel, int threads, size_t smem, std::atomic<bool> *attr_set,
                                      const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                      const TreeParams &p, int dev, cudaStream_t stream) {
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    kernel<<<p.workers, threads, smem, stream>>>(tq, tk, tv, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.workers < 2) return e;
    tree_merge_kernel<T, D><<<dim3(p.workers - 1, p.rows_per_item / 8), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

// Items of several kv heads (tree_packed.cu): the plan for `rows` query rows a head (heads_per_item
// set), and the launch.
void plan_tree_packed(TreePlan &t, int rows, int group, int head_dim);
cudaError_t launch_tree_packed(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                               int head_dim, int q_dtype, int dev, cudaStream_t stream);

}  // namespace pkv
