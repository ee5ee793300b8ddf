// Pieces shared by the tree attention kernels (tree_attention.cu, tree_packed.cu): the work list of
// (item, key tile) and its equal shares, the masks of drafted trees, the handling of values that
// not every row sees, and the merge of items that lie in several shares.
#pragma once

#include <atomic>
#include <climits>
#include <type_traits>

#include "common.cuh"
#include "dependent_launch.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace pkv {

constexpr int kTreeRows = 128;         // query rows of a row tile = TMEM lanes
constexpr int kHalf = 128 * 128;       // 128 rows x 64 16-bit elements (one swizzle column)
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;   // a row's reference maximum moves when exceeded by more
// log2 of a factor on all weights, sums and O (it leaves with the normaliser, and the lse takes it off).  fp16
// weights below 2^-14 lose digits and those below 2^-25 vanish, which the sum of many such keys shows: 9000
// keys of 2^-20.5 each were 3 % off, of 2^-25.5 lost.  With the largest weight, 2^kRescaleLog2, at 2^15 under
// fp16's 65504, a key is off by at most 2^-32 of its row's largest weight.  bf16 has float's exponents.
template <typename T> constexpr float kWeightLog2 = 0.f;
template <> constexpr float kWeightLog2<__half> = 7.f;
// An item's fixed cost in key tiles (its queries, masked tiles and results), once shares hold kBigShare
// tiles or more.  Smaller ones count tiles alone, down to one: latency is what matters then.
constexpr int kItemCost = 2;
constexpr int kBigShare = 8;
// Workers an item from which a CTA's warps share out the pieces of an item (see the merge kernels).
constexpr int kLongMerge = 32;
constexpr int kFlags = 8;              // pieces whose odd-value flags are kept

struct TreeParams {
    TreeArgs a;
    int group;            // query heads of a kv head
    int tokens_per_tile;  // drafted tokens of a kv head's rows in a row tile
    int heads_per_item;   // 1: items of two row tiles of a kv head; 2 or 4: of so many kv heads
    int key_shift;        // log2 of the keys of a key tile
    int workers;          // shares at most
    int rows_per_item;    // rows of a partial result
    int items_per_seq;    // at most
    int4 *ws_first;       // [2 * workers] first piece of each share: (sequence, item of it, key tile of it,
                          // -), (first row, rows, -, -) of the sequence; sequence -1: no share
    float *ws_lse;        // [2 * workers][rows_per_item] log2-sum-exp2 of the partial results
    float4 *ws_o;         // [2 * workers][D / 4][rows_per_item] partial results, normalised, four dims each: a
                          // warp's rows lie side by side
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

// Where the share of a CTA starts: sequence, item and the cost where that item starts.
struct ShareStart {
    Seq s;
    int64_t at;
    int b, idx;
};

struct ShareScratch {
    int64_t warp_tiles[16], warp_items[16];
    ShareStart start;
};

// The share [x0, x1) of CTA c (x0 == x1: none) and an item's cost.  Computed by the whole block, with
// scratch in shared memory; scratch.start is valid after the next __syncthreads.
template <int kThreads>
__device__ __forceinline__ void share_of_cta(const TreeParams &p, int c, int64_t &x0, int64_t &x1, int &item_cost,
                                             ShareScratch &scratch) {
    static_assert(kThreads <= 16 * 32, "a word a warp");
    int64_t(&warp_tiles)[16] = scratch.warp_tiles;
    int64_t(&warp_items)[16] = scratch.warp_items;
    ShareStart &start = scratch.start;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_seqs = p.a.num_seqs;
    const int per = (num_seqs + kThreads - 1) / kThreads;
    const int b_lo = min(num_seqs, static_cast<int>(threadIdx.x) * per), b_hi = min(num_seqs, b_lo + per);
    Seq s;
    bool rejected;
    int64_t tiles = 0, items = 0;  // of this thread's sequences
    for (int b = b_lo; b < b_hi; ++b) {
        if (!load_seq(p, b, s, &rejected)) continue;
        tiles += static_cast<int64_t>(s.tiles) * s.items;
        items += s.items;
    }
    int64_t it = tiles, ii = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, it, o), i = __shfl_up_sync(0xffffffffu, ii, o);
        if (lane >= o) it += t, ii += i;
    }
    if (lane == 31) warp_tiles[warp] = it, warp_items[warp] = ii;
    __syncthreads();
    int64_t tiles_before = it - tiles, items_before = ii - items, all_tiles = 0, all_items = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) tiles_before += warp_tiles[w], items_before += warp_items[w];
        all_tiles += warp_tiles[w];
        all_items += warp_items[w];
    }
    // a share of cost above item_cost holds a tile at least
    const bool big = all_tiles >= static_cast<int64_t>(kBigShare) * p.workers;
    item_cost = big ? kItemCost : 0;
    const int64_t total = all_tiles + item_cost * all_items;
    const int64_t shares = min(static_cast<int64_t>(p.workers), all_tiles);
    x0 = x1 = 0;
    if (c >= shares) return;
    x0 = total * c / shares;
    x1 = total * (c + 1) / shares;
    const int64_t before = tiles_before + item_cost * items_before;
    if (x0 < before || x0 >= before + tiles + item_cost * items) return;
    int64_t at = before;  // one thread
    for (int b = b_lo; b < b_hi; ++b) {
        if (per > 1 && !load_seq(p, b, s, &rejected)) continue;
        const int64_t cost = static_cast<int64_t>(s.tiles + item_cost) * s.items;
        if (x0 < at + cost) {
            start.b = b;
            start.idx = static_cast<int>((x0 - at) / (s.tiles + item_cost));
            start.at = at + static_cast<int64_t>(start.idx) * (s.tiles + item_cost);
            start.s = s;
            break;
        }
        at += cost;
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
    int item_cost;
    Seq cur;          // the piece's sequence,
    int seq, item;    // its number, the item of it
    int ja, jb;       // and key tiles (absolute)
    bool whole;       // the piece is its whole item
    bool begun;

    __device__ __forceinline__ void start(const ShareStart &st, int64_t x0_, int64_t x1_, int item_cost_) {
        seq = st.b, item = st.idx, at = st.at, x0 = x0_, x1 = x1_, item_cost = item_cost_;
        cur = st.s;
        begun = false;
    }
    __device__ __forceinline__ bool next(const TreeParams &p) {
        for (;;) {
            if (begun) {  // on to the next item
                at += item_cost + cur.tiles;
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
            const int64_t first = at + item_cost;
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

// Where the partial result of a piece goes: a share leaves at most one that starts inside its item
// (slot 2c) and one that starts it (2c + 1).
__device__ __forceinline__ int64_t part_slot(int c, bool starts) { return 2 * c + (starts ? 1 : 0); }
__device__ __forceinline__ float *part_lse(const TreeParams &p, int64_t slot, int row) {
    return p.ws_lse + slot * p.rows_per_item + row;
}
template <int D> __device__ __forceinline__ float4 *part_o(const TreeParams &p, int64_t slot, int row) {
    return p.ws_o + slot * (D / 4) * p.rows_per_item + row;  // four dims on: rows_per_item further
}

// 32 dims of a row a lane (o) to 16-bit rows.  Quads of lanes exchange 16-byte units first, so that a
// store covers 64 bytes of 8 rows instead of 16 bytes of 32.  dst[k]: dims of the row of the quad's
// lane k, at this lane's unit, or null.
template <typename T> __device__ __forceinline__ void store_rows(const float (&o)[32], T *const (&dst)[4], int dim) {
    const int lane = threadIdx.x & 31;
    uint32_t u[4][4];  // unit (8 dims), word
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[k][e] = pack2<T>(o[8 * k + 2 * e], o[8 * k + 2 * e + 1]);
#pragma unroll
    for (int bit = 1; bit <= 2; bit <<= 1) {
        const bool hi = lane & bit;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & bit) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // the lower lane gives its upper unit for the upper lane's lower one
                const uint32_t give = hi ? u[k][e] : u[k | bit][e];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, give, bit);
                if (hi) u[k][e] = got;
                else u[k | bit][e] = got;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (dst[k]) *reinterpret_cast<uint4 *>(dst[k] + dim) = make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
}

// The rows of this lane's quad, at this lane's unit of 8 dims, for store_rows (mine: null for no row).
template <typename T> __device__ __forceinline__ void quad_rows(T *mine, T *(&dst)[4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const unsigned long long q = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), (lane & ~3) | k);
        dst[k] = q ? reinterpret_cast<T *>(q) + 8 * (lane & 3) : nullptr;
    }
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
// (out16 of type T, or a partial result): they were zeroed for the products.  Rare, so plain.
template <typename T, int D>
static __device__ __noinline__ void add_non_finite(const TreeArgs &a, int b, int h, int k0, int k1, int ctx, int klo,
                                            uint64_t mask, T *out16, float4 *part, int part_step) {
    for (int k = k0; k < k1; ++k) {
        const bool sees = k < ctx ? k >= klo : (mask >> (k - ctx)) & 1;
        const int id = a.block_table[b * a.bt_stride + k / a.block_size];
        if (!sees || id < 0 || id >= a.num_blocks) continue;
        const T *v = static_cast<const T *>(a.v_cache) +
                     ((static_cast<int64_t>(id) * a.block_size + k % a.block_size) * a.num_kv_heads + h) * D;
        for (int d = 0; d < D; ++d) {
            const float f = to_float<T>(v[d]);
            if (isfinite(f)) continue;
            if (part) reinterpret_cast<float *>(part + static_cast<int64_t>(d / 4) * part_step)[d % 4] += f;
            else out16[d] = from_float<T>(to_float<T>(out16[d]) + f);
        }
    }
}

// Add the non-finite values that the row sees in the piece's mixed tiles.
template <typename T, int D>
__device__ __forceinline__ void add_odd_values(const TreeParams &p, const Walk &w, int h, int klo, uint64_t mask, T *out16,
                                               float4 *part) {
    const TreeArgs &a = p.a;
    const Seq &s = w.cur;
    const int ka = w.ja << p.key_shift, kb = min(w.jb << p.key_shift, s.L);
    if (a.window > 0)
        add_non_finite<T, D>(a, w.seq, h, max(ka, s.kv_lo), min(min(s.ctx, s.ctx + s.n - a.window), kb), s.ctx, klo, mask,
                             out16, part, p.rows_per_item);
    add_non_finite<T, D>(a, w.seq, h, max(ka, s.ctx), kb, s.ctx, klo, mask, out16, part,
                         p.rows_per_item);
}

// Join the partial results of an item that lies in several shares:
//   out = sum_i w_i o_i / sum_i w_i,  w_i = exp2(lse_i - max)
// A thread takes 8 dims of a row, a warp 32 rows, so that the partial results are read in whole lines.
// What it costs is dependent round trips: the shares' records, then kPieces pieces at a time.
constexpr int kPieces = 4;

struct Joined {
    float acc[8], wsum, mx;
    __device__ __forceinline__ Joined() : wsum(0.f), mx(-INFINITY) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    }
    // Further pieces: their lse (-inf: nothing seen, or no piece) and 8 dims.  kKeep: a piece that saw keys counts at
    // a weight that has underflowed to 0 too, so that a NaN or an infinity that it holds stays (as NaN).
    template <bool kKeep, int N> __device__ __forceinline__ void add(const float (&l)[N], const float4 (&v)[N][2]) {
        float m = mx;
        bool nan = false;
#pragma unroll
        for (int u = 0; u < N; ++u) m = fmaxf(m, l[u]), nan |= l[u] != l[u];
        if (m == -INFINITY && !nan) return;  // nothing seen so far
        const float f = mx == -INFINITY ? 0.f : fast_exp2(mx - m);
        mx = m;
        wsum *= f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= f;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const float w = l[u] == -INFINITY ? 0.f : fast_exp2(l[u] - mx);
            if (kKeep ? l[u] == -INFINITY : w == 0.f) continue;  // it adds nothing, whatever it holds
            wsum += w;
            acc[0] += w * v[u][0].x, acc[1] += w * v[u][0].y, acc[2] += w * v[u][0].z, acc[3] += w * v[u][0].w;
            acc[4] += w * v[u][1].x, acc[5] += w * v[u][1].y, acc[6] += w * v[u][1].z, acc[7] += w * v[u][1].w;
        }
    }
    // Pieces e0, e0 + step, .. up to `last` of the item that starts in share c: row rr, the dims of float4s q, q + 1.
    template <int D, bool kKeep>
    __device__ __forceinline__ void add_pieces(const TreeParams &p, int c, int e0, int step, int last, int rr, int q) {
        for (; e0 <= last; e0 += kPieces * step) {
            float l[kPieces];
            float4 v[kPieces][2];
#pragma unroll
            for (int u = 0; u < kPieces; ++u) {
                const int e = e0 + u * step;
                const bool in = e <= last;
                const int64_t slot = part_slot(e, e == c);
                const float4 *src = part_o<D>(p, slot, rr) + static_cast<int64_t>(q) * p.rows_per_item;
                l[u] = in ? __ldcg(part_lse(p, slot, rr)) : -INFINITY;
                v[u][0] = in ? __ldcg(src) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[u][1] = in ? __ldcg(src + p.rows_per_item) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            add<kKeep>(l, v);
        }
    }
    // The joined result of that row of item idx of a sequence (sq: its second record), if the row exists.
    template <typename T, int D>
    __device__ __forceinline__ void store(const TreeParams &p, const int4 &sq, int idx, int rr, int q) const {
        const int64_t row = row_of(p, sq, idx, rr);
        if (row < 0) return;
        const TreeArgs &a = p.a;
        const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
        *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * D + 4 * q) =
            make_uint4(pack2<T>(acc[0] * inv, acc[1] * inv), pack2<T>(acc[2] * inv, acc[3] * inv),
                       pack2<T>(acc[4] * inv, acc[5] * inv), pack2<T>(acc[6] * inv, acc[7] * inv));
        if (a.lse_out && q == 0) a.lse_out[row] = wsum == 0.f ? -INFINITY : (mx + log2f(wsum)) * 0.69314718055994531f;
    }
    // Row of the output of an item's row rr, or -1: its kv head, token and head of the group.
    static __device__ __forceinline__ int64_t row_of(const TreeParams &p, const int4 &sq, int idx, int rr) {
        int h, t, hh;
        const int TQ = p.tokens_per_tile;
        if (p.heads_per_item == 1) {
            h = idx / sq.z;
            const int r = rr & 127, tl = r / p.group;
            t = (2 * (idx - h * sq.z) + (rr >> 7)) * TQ + tl;
            hh = r - tl * p.group;
            if (tl >= TQ || t >= sq.y) return -1;
        } else {
            const int lanes = p.rows_per_item / p.heads_per_item, r = rr % lanes;
            h = idx * p.heads_per_item + rr / lanes;
            t = r / p.group;
            hh = r - t * p.group;
            if (h >= p.a.num_kv_heads || t >= sq.y) return -1;
        }
        return static_cast<int64_t>(sq.x + t) * p.a.num_q_heads + h * p.group + hh;
    }
};

// A CTA a share c (and 8 units of 8 dims of 32 rows): the item that starts in it and goes on into the next ones.
template <typename T, int D, bool kKeep = false>
static __global__ void __launch_bounds__(256, 4) tree_merge_kernel(const __grid_constant__ TreeParams p) {
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    const int unit = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int rr = unit / (D / 8) * 32 + lane, q = unit % (D / 8) * 2;
    previous_kernel_done();  // the attention kernel's results
    // lane i: the first piece of share c + i (none past the last)
    const int4 none = make_int4(-1, 0, 0, 0);
    int4 rec = c + lane < p.workers ? __ldcg(&p.ws_first[2 * (c + lane)]) : none;
    const int4 sq = __ldcg(&p.ws_first[2 * (c + 1) + 1]);
    // share c + 1's decides whether c's last item goes on; c's own, whether that item started before
    const int b = __shfl_sync(0xffffffffu, rec.x, 1), idx = __shfl_sync(0xffffffffu, rec.y, 1);
    const bool same = rec.x == b && rec.y == idx && rec.z > 0;  // this share goes on with the item
    uint32_t go = __ballot_sync(0xffffffffu, same);
    if (b < 0 || !(go & 2) || (go & 1)) return;
    // pieces: share c's (its last: slot 2c + 1), then those of the next shares (their first: 2c')
    int last = c + 31;
    if (~(go | 1)) last = c + __ffs(~(go | 1)) - 2;
    while (last >= c + 31) {
        const int e = last + 1 + lane;
        rec = e < p.workers ? __ldcg(&p.ws_first[2 * e]) : none;
        go = __ballot_sync(0xffffffffu, rec.x == b && rec.y == idx && rec.z > 0);
        if (go == 0xffffffffu) {
            last += 32;
            continue;
        }
        last += __ffs(~go) - 1;
        break;
    }
    if (Joined::row_of(p, sq, idx, rr) < 0) return;
    Joined x;
    x.add_pieces<D, kKeep>(p, c, c, 1, last, rr, q);
    x.store<T, D>(p, sq, idx, rr, q);
}

// The same when there are few items, of many pieces each: a CTA an item (and a unit), whose 8 warps share
// out its pieces.  One sequence of 32/8 heads takes 15.5 us for 1117 tokens, 17.9 for 4000 and 39 for 30000, and
// 17.0, 22.6 and 46 with the other merge; but with 16 items (8 sequences of 600) it was 25.4 against 20.3, as
// every CTA reads all records and each unit is a CTA.
template <typename T, int D>
static __global__ void __launch_bounds__(256, 4) tree_merge_long_kernel(const __grid_constant__ TreeParams p) {
    __shared__ float lse[8][32];
    __shared__ float4 part[8][2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / p.items_per_seq, idx = blockIdx.x % p.items_per_seq;
    const int rr = blockIdx.y / (D / 8) * 32 + lane, q = blockIdx.y % (D / 8) * 2;
    previous_kernel_done();
    // the shares that begin in the middle of the item: `first` and the next ones
    int mine = INT_MAX, count = 0;
    for (int e = lane; e < p.workers; e += 32) {
        const int4 rec = __ldcg(&p.ws_first[2 * e]);
        if (rec.x == b && rec.y == idx && rec.z > 0) mine = min(mine, e), ++count;
    }
    const int first = __reduce_min_sync(0xffffffffu, mine);
    count = __reduce_add_sync(0xffffffffu, count);
    if (count == 0 || first == 0) return;  // the item is in one share (the first one starts its item)
    const int4 sq = __ldcg(&p.ws_first[2 * first + 1]);
    const int c = first - 1, last = c + count;
    Joined x;  // (a row that does not exist is read as it is, and not stored)
    x.add_pieces<D, false>(p, c, c + warp, 8, last, rr, q);
    // each warp's result as one more piece
    lse[warp][lane] = x.wsum == 0.f ? -INFINITY : x.mx + log2f(x.wsum);
    const float inv = x.wsum == 0.f ? 0.f : 1.f / x.wsum;
    part[warp][0][lane] = make_float4(x.acc[0] * inv, x.acc[1] * inv, x.acc[2] * inv, x.acc[3] * inv);
    part[warp][1][lane] = make_float4(x.acc[4] * inv, x.acc[5] * inv, x.acc[6] * inv, x.acc[7] * inv);
    __syncthreads();
    if (warp) return;
    Joined y;
#pragma unroll
    for (int w0 = 0; w0 < 8; w0 += kPieces) {
        float l[kPieces];
        float4 v[kPieces][2];
#pragma unroll
        for (int u = 0; u < kPieces; ++u) l[u] = lse[w0 + u][lane], v[u][0] = part[w0 + u][0][lane], v[u][1] = part[w0 + u][1][lane];
        y.add<false>(l, v);
    }
    y.store<T, D>(p, sq, idx, rr, q);
}

// The merge, with more than one share.
template <typename T, int D> static cudaError_t launch_tree_merge(const TreeParams &p, cudaStream_t stream) {
    const int units = p.rows_per_item / 32 * (D / 8);
    const int64_t items = static_cast<int64_t>(p.items_per_seq) * p.a.num_seqs;
    if (items * kLongMerge <= p.workers)
        return launch_dependent(tree_merge_long_kernel<T, D>, dim3(static_cast<unsigned>(items), units), dim3(256), 0, stream, p);
    return launch_dependent(tree_merge_kernel<T, D>, dim3(p.workers - 1, units / 8), dim3(256), 0, stream, p);
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
    // The attention kernel waits for the kernel before it once its barriers and TMEM are set up, and lets the
    // merge launch then, whose CTAs wait at once (those that fit beside the attention kernel's; it is launched
    // when all of these are on an SM or done, so that it keeps none of them out).  In a stream of calls that
    // takes 2.5 to 5 us less than launching the merge alone this way, and that 2 us less than plain launches.
    // Letting the next kernel launch at the merge's start: 0.3 us less for one sequence, 1.2 and 2.5 us more
    // for the largest batches.
    const cudaError_t e = launch_dependent(kernel, dim3(p.workers), dim3(threads), smem, stream, tq, tk, tv, p);
    if (e != cudaSuccess || p.workers < 2) return e;
    return launch_tree_merge<T, D>(p, stream);
}

// Items of several kv heads (tree_packed.cu): the plan for `rows` query rows a head (heads_per_item
// set), and the launch.
void plan_tree_packed(TreePlan &t, int rows, int group, int head_dim);
cudaError_t launch_tree_packed(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                               int head_dim, int q_dtype, int dev, cudaStream_t stream);

}  // namespace pkv
