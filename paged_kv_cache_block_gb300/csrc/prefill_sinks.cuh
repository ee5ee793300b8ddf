// Prefill attention with a sliding window and sinks, over 16-bit, E4M3 and INT4 caches, on the
// fifth-generation tensor cores (chunked prefill: "vLLM의 KV cache 연결 흐름", section "EngineCore가
// 하는 일"; windows: "vLLM Worker侧GPU KV Cache初始化流程深度解析", section "混合注意力机制", and its
// section "KV Cache技术背景" for the 8- and 4-bit caches; the pages have no sinks).
//
// The row at position p sees key j <= p when window = 0, j > p - window or j < num_sinks:
//   out = sum_j p_j V_j / sum_j p_j,  p_j = exp2(scale log2(e) q.K_j - m)
// Row tiles are up to 128 rows of a kv head (128 / g tokens x the g heads of its group).  An item is
// (sequence, kv head, two row tiles).  Its keys form an axis of their own, the sequence without the
// blocks that none of its rows sees (those between the last sink's block and the first row's window):
// block c of the axis is block c of the sequence below sink_blocks, and block c + hidden from there on.
// The cache being paged, a tile of 128 keys is any 128 / block_size blocks, so sinks and window share
// tiles and the axis starts at a block, not at a multiple of 128.
//
// Two chains x = 0, 1 of
//   S_x = Q K_j^T   tcgen05.mma, M 128, N 128; fp32 in TMEM
//   P_x = exp2(S_x * scale - m)   one thread a row; 16-bit weights back into TMEM over S_x
//   O_x += P_x V_j  tcgen05.mma, A = P_x in TMEM, fp32 in TMEM across key tiles
// run at once: one row tile each, or, for an item of one row tile, every second key tile each, joined at
// the end.  The flat list of (item, key tile) is cut into equal shares, one a CTA, so that neither the
// batch's lengths nor the triangle of whole prompts matter; items that lie in several shares leave
// partial results, joined by the merge of the tree attention (tree_common.cuh), whose parameters and
// records this kernel shares.
//
// 16-bit caches: a warp copies K and V tiles by TMA, a block and all dims of a head a box, and another
// cleans V tiles that hold keys which not every row sees (a weight of 0 times a NaN or an infinity would not be
// 0): what no row sees is zeroed, and a non-finite value that some rows see is zeroed and added to those
// rows' results afterwards.  E4M3 and INT4 caches (kWide): six warps load codes and write them as fp16
// tiles instead, where the products take them from: INT4 codes as the integers they are, two a lop3 and
// one packed add, their dims in the order (0, 4, 1, 5, 2, 6, 3, 7) of each eight that this leaves them in.  The
// queries follow that order; each row is multiplied by its head's K scales and by the power of two that
// puts its largest product at 2^7 .. 2^8, so that any scale keeps its digits in fp16, and the power comes
// off in the row's softmax scale.  V scales multiply the result.
// Weights are taken against the reference maximum in use; only when a row's maximum exceeds it by
// more than 2^8 are its O and sum rescaled.  The sum is of the weights before their rounding.
// What bounds it: in each chain the scores of a key tile wait for the product before them, whose weights lie
// where they are written (two row tiles of 128 dims leave TMEM no other columns), and both chains come to be in
// phase: about 4,700 clocks a tile of two row tiles, of which the products take 2 x 1,300 and a softmax 1,700.
// Times of the call, one GB300 (32/8 heads of 128 dims and blocks of 16 where not said):
//   16 chunks of 1024 tokens in the middle of 7168 + 1024, window 4096, 4 sinks     969 us, 965 TFLOP/s counted
//   8 ragged prompts up to 2048, 64/8 heads, window 512, 128 sinks                  319 us, 461 (tiles on the
//     diagonal and at the window's edge are half masked)
//   100 tokens after 20000, window 4096, 4 sinks    31 us: start 5, 2.4 a key tile, partial results and merge 10
//   the 16 chunks over an E4M3 cache, the same window                              1368 us, 683
//   the 16 chunks, 40/8 heads of 64 dims                                           1012 us, 577
//   the 16 chunks over an INT4 cache, full attention                               1470 us, 825
//   257 tokens after 8000 over an INT4 cache                                         79 us
// Shares by closed-form costs instead of by items are what the ragged prompts and the single sequences live by.
// Every wait is bounded (2 s): on expiry KV_DERR_TIMEOUT is set, what was issued is drained, TMEM is freed
// and the CTA returns.
#pragma once

#include <cfloat>

#include "tree_common.cuh"

namespace pkv {

enum { kCache16 = 0, kCacheE4M3 = 1, kCacheInt4 = 2 };

struct SinkPrefillParams {
    TreeParams t;          // sizes, outputs and the workspace, for the merge too
    int num_sinks;         // 0 without a window
    int sink_blocks;
    int bs_shift;          // log2(block_size)
    const void *k_cache;   // E4M3 and INT4
    float v_scale;         // E4M3
    const float *k_gscales, *v_gscales;  // INT4: [num_kv_heads, D >> group_shift]
    int group_shift;
    const void *q;         // E4M3 and INT4: [num_tokens, num_q_heads, D]
};

namespace sinks {

constexpr int kBM = kTreeRows;
constexpr int kBN = 128;           // keys of a key tile
template <int kCache> constexpr int kThreads = kCache == kCache16 ? 384 : 512;
constexpr uint32_t kColO = 256;

// E4M3 and INT4 codes come to shared memory in units of 8 KB (an INT4 tile, half an E4M3 one), so many at a time.
constexpr int kUnitBytes = 8192;
constexpr int kUnits = 3;
constexpr int kWideners = 6;       // warps that write them as fp16 tiles

template <int D> struct Tile {
    static constexpr int kHalves = D / 64;
    static constexpr int kBytes = kHalves * kHalf;      // a Q, K or V tile
    static constexpr int kGroup = kHalves * 1024;       // 8 keys of a K or V tile: [64 dims of D][key][dim]
    static constexpr int kStages = D == 128 ? 4 : 8;    // ring entries (128 KB)
    static constexpr int kOffKV = 2 * kBytes;           // after Q_0, Q_1
    static constexpr int kOffJoin = kOffKV + kStages * kBytes;   // chain 1's maxima, sums and excess: 3 x 128 floats
    static constexpr int kOffScratch = kOffJoin + 3 * 128 * 4;   // of the schedule
    static constexpr int kScratchBytes = 512;
    static constexpr int kOffBar = kOffScratch + kScratchBytes;
    static constexpr int kNumBars = 14 + 2 * kStages;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;      // TMEM address, abort flag, flags, cleaned
    static constexpr int kOffUnits = (kOffMisc + 8 + 4 * kWideners * kFlags + 4 * kStages + 15) / 16 * 16;  // kWide: codes
    static constexpr int smem(bool wide) { return kOffUnits + (wide ? kUnits * kUnitBytes : 0) + 1024; }  // + alignment
    // pieces whose V tiles can be in the ring at once, one more that the cleaning warp has begun,
    // and one without mixed tiles (only a share's last)
    static_assert(kFlags >= (kStages + 1) / 2 + 2, "a flag per piece in flight");
};

// mbarrier indices (+ x: one per chain)
enum { kBarQFull = 0, kBarQEmpty = 1, kBarS = 2, kBarP = 4, kBarPv = 6, kBarPd = 8, kBarJoin = 10,
       kBarJoined = 11, kBarDrain = 12, kBarKv = 14 };  // then KvFull[stages], KvEmpty[stages]

// A sequence's part of the work list.  Costs are counted in keys: pair i of a kv head costs
//   c_i = min(keys up to its last token, cap) + item_cost
// where cap is what a window and the sinks leave; it is never above the keys of the pair's axis, so that
// c_i - item_cost <= 128 * (its key tiles).
struct Seq {
    int q0, n, L, ctx;  // first row, rows, length, context
    int pairs;          // of row tiles
};

// a / b for 0 <= a, 0 < b: most are small, and a 64-bit division takes some hundred cycles.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

struct Costs {
    int step;           // tokens of a pair
    int64_t extra;      // of a window: window - 1 + keys of the sinks' blocks (no window: far above any length)
    int64_t item;
    __device__ __forceinline__ Costs(const SinkPrefillParams &p, int64_t item_cost)
        : step(2 * p.t.tokens_per_tile),
          extra(p.t.a.window > 0 ? static_cast<int64_t>(p.t.a.window) - 1 + (p.sink_blocks << p.bs_shift) : int64_t(1) << 40),
          item(item_cost) {}
    __device__ __forceinline__ int64_t of(const Seq &s, int i) const {
        const int last = min(s.n, (i + 1) * step);
        return min(static_cast<int64_t>(s.ctx) + last, extra + (last - i * step)) + item;
    }
    // Of pairs 0 .. k - 1: whole pairs i < m lie below the window's bound ctx + (i + 1) step <= extra + step.
    __device__ __forceinline__ int64_t before(const Seq &s, int k) const {
        const int64_t whole = min(k, s.pairs - 1);
        const int64_t m = min(whole, extra < s.ctx ? int64_t(0) : quotient(extra - s.ctx, step) + 1);
        int64_t sum = m * s.ctx + step * (m * (m + 1) / 2) + (whole - m) * (extra + step) + whole * item;
        if (k == s.pairs) sum += of(s, s.pairs - 1);
        return sum;
    }
};

// The sequence's lengths; false when it has no rows, or is rejected (*rejected).
__device__ __forceinline__ bool load_seq(const SinkPrefillParams &p, int b, Seq &s, bool *rejected) {
    const TreeArgs &a = p.t.a;
    s.q0 = a.query_start_loc[b];
    s.n = a.query_start_loc[b + 1] - s.q0;
    s.L = a.seq_lens[b];
    *rejected = s.n > 0 && !(s.n <= a.max_query_len && s.q0 >= 0 && s.q0 <= a.num_tokens - s.n && s.L >= s.n &&
                             s.L <= a.max_seq_len && ((s.L - 1) >> p.bs_shift) < a.max_blocks_per_seq);
    if (s.n <= 0 || *rejected) return false;
    s.ctx = s.L - s.n;
    s.pairs = (s.n - 1) / (2 * p.t.tokens_per_tile) + 1;
    return true;
}

// Where the share of a CTA starts: sequence, item and the cost where that item starts.
struct ShareStart {
    Seq s;
    int64_t at;
    int b, idx;
};
struct ShareScratch {
    int64_t warp_keys[16], warp_items[16];
    ShareStart start;
};
static_assert(sizeof(ShareScratch) <= 512, "Tile::kScratchBytes");

// The share [x0, x1) of CTA c (x0 == x1: none) and an item's cost.  Computed by the whole block, with
// scratch in shared memory; scratch.start is valid after the next __syncthreads.
template <int kThreads>
__device__ __forceinline__ void share_of_cta(const SinkPrefillParams &p, int c, int64_t &x0, int64_t &x1,
                                             int64_t &item_cost, ShareScratch &scratch) {
    static_assert(kThreads <= 16 * 32, "a word a warp");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_seqs = p.t.a.num_seqs, heads = p.t.a.num_kv_heads;
    const int per = (num_seqs + kThreads - 1) / kThreads;
    const int b_lo = min(num_seqs, static_cast<int>(threadIdx.x) * per), b_hi = min(num_seqs, b_lo + per);
    const Costs free(p, 0);
    Seq s;
    bool rejected;
    int64_t keys = 0, items = 0;  // of this thread's sequences
    for (int b = b_lo; b < b_hi; ++b) {
        if (!load_seq(p, b, s, &rejected)) continue;
        keys += free.before(s, s.pairs) * heads;
        items += static_cast<int64_t>(s.pairs) * heads;
    }
    int64_t ik = keys, ii = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, ik, o), i = __shfl_up_sync(0xffffffffu, ii, o);
        if (lane >= o) ik += t, ii += i;
    }
    if (lane == 31) scratch.warp_keys[warp] = ik, scratch.warp_items[warp] = ii;
    __syncthreads();
    int64_t keys_before = ik - keys, items_before = ii - items, all_keys = 0, all_items = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) keys_before += scratch.warp_keys[w], items_before += scratch.warp_items[w];
        all_keys += scratch.warp_keys[w];
        all_items += scratch.warp_items[w];
    }
    // A share is at least as long as any tile (128 keys of an axis and an item's cost), so that each holds
    // a tile's end, hence a tile: no share between two of an item is empty.
    const bool big = all_keys >= static_cast<int64_t>(kBigShare) * kBN * p.t.workers;
    item_cost = big ? kItemCost * kBN : 0;
    // (With an item's cost, 8 tiles a worker are more than such a length anyway.)
    const int64_t total = all_keys + item_cost * all_items;
    const int64_t most = big ? p.t.workers : min(static_cast<int64_t>(p.t.workers), total / kBN);
    const int64_t shares = most > 0 ? most : (total > 0 ? 1 : 0);
    x0 = x1 = 0;
    if (c >= shares) return;
    x0 = quotient(total * c, shares);
    x1 = quotient(total * (c + 1), shares);
    const int64_t before = keys_before + item_cost * items_before;
    if (x0 < before || x0 >= before + keys + item_cost * items) return;
    const Costs costs(p, item_cost);
    int64_t at = before;  // one thread
    for (int b = b_lo; b < b_hi; ++b) {
        if (per > 1 && !load_seq(p, b, s, &rejected)) continue;
        const int64_t head = costs.before(s, s.pairs);
        if (x0 < at + head * heads) {
            const int64_t h = quotient(x0 - at, head);
            at += h * head;
            int lo = 0, hi = s.pairs - 1;  // the last pair that starts at or before x0
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (at + costs.before(s, mid) <= x0) lo = mid;
                else hi = mid - 1;
            }
            scratch.start.b = b;
            scratch.start.idx = static_cast<int>(h) * s.pairs + lo;
            scratch.start.at = at + costs.before(s, lo);
            scratch.start.s = s;
            break;
        }
        at += head * heads;
    }
}

// Rows of rejected sequences are 0 (lse -inf): the CTAs take the sequences in turn.
template <typename T, int D> __device__ __forceinline__ void zero_rejected(const SinkPrefillParams &p) {
    const TreeArgs &a = p.t.a;
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

// The pieces of a share, in order: (item, key tiles ja .. jb - 1 of its axis).  Every warp walks the same ones.
struct Walk {
    int64_t at, cost;  // cost where the item starts, and of the item
    int64_t x0, x1;    // the share
    int64_t item_cost;
    Seq cur;           // the piece's sequence,
    int seq, item;     // its number, the item of it:
    int h, nt, t0;     // kv head, row tiles, first token
    int pf, pl;        // positions of the item's first and last token, on its axis
    int hidden;        // blocks the axis leaves out
    int tiles;         // of the axis
    int ja, jb;
    bool whole;        // the piece is its whole item
    bool begun;

    __device__ __forceinline__ void start(const ShareStart &st, int64_t x0_, int64_t x1_, int64_t item_cost_) {
        seq = st.b, item = st.idx, at = st.at, x0 = x0_, x1 = x1_, item_cost = item_cost_;
        cur = st.s;
        begun = false;
    }
    // The tile that a cost lies in, of a cost within the item (its end: tiles): a tile belongs to the share
    // that its end lies in.
    __device__ __forceinline__ int tile_at(int64_t x) const { return static_cast<int>(quotient((x - at) * tiles, cost)); }
    __device__ __forceinline__ bool next(const SinkPrefillParams &p) {
        const Costs costs(p, item_cost);
        const TreeArgs &a = p.t.a;
        for (;;) {
            if (begun) {  // on to the next item
                at += cost;
                if (at >= x1) return false;
                if (++item == cur.pairs * a.num_kv_heads) {
                    item = 0;
                    bool rejected = false;
                    do {
                        if (++seq >= a.num_seqs) return false;
                    } while (!load_seq(p, seq, cur, &rejected));
                }
            }
            begun = true;
            h = item / cur.pairs;
            const int pr = item - h * cur.pairs;
            cost = costs.of(cur, pr);
            t0 = pr * costs.step;
            const int count = min(cur.n - t0, costs.step);
            nt = count > p.t.tokens_per_tile ? 2 : 1;
            pf = cur.ctx + t0;
            hidden = a.window > 0 ? max(0, (max(0, pf - a.window + 1) >> p.bs_shift) - p.sink_blocks) : 0;
            pf -= hidden << p.bs_shift;
            pl = pf + count - 1;
            tiles = pl / kBN + 1;
            // (64-bit divisions, which a share's whole items have no need of)
            ja = x0 <= at ? 0 : tile_at(x0);
            jb = x1 >= at + cost ? tiles : tile_at(x1);
            whole = ja == 0 && jb == tiles;
            if (ja < jb) return true;
        }
    }
    // The share's first piece, for the merge.
    __device__ __forceinline__ void record(const SinkPrefillParams &p, int c) const {
        p.t.ws_first[2 * c] = make_int4(seq, item, ja, 0);
        p.t.ws_first[2 * c + 1] = make_int4(cur.q0, cur.n, cur.pairs, 0);
    }
    // First key (on the axis) of the window of the row at axis position pos.
    static __device__ __forceinline__ int window_from(const SinkPrefillParams &p, int pos) {
        return p.t.a.window > 0 ? max(0, pos - p.t.a.window + 1) : 0;
    }
    // Whether key tile j holds a key that not all rows at axis positions first .. last see.
    static __device__ __forceinline__ bool mixed(const SinkPrefillParams &p, int j, int first, int last) {
        const int k1 = j * kBN + kBN - 1;
        return k1 > first || (j * kBN < window_from(p, last) && k1 >= p.num_sinks);
    }
    __device__ __forceinline__ bool mixed(const SinkPrefillParams &p, int j) const { return mixed(p, j, pf, pl); }
    // Block of the sequence that holds block c of the axis.
    __device__ __forceinline__ int block(const SinkPrefillParams &p, int c) const { return c < p.sink_blocks ? c : c + hidden; }
};

// The keys k0 .. k0 + 31 (bit i: key k0 + i) that the row at position pos sees, with a window from klo.
__device__ __forceinline__ uint32_t seen32(int k0, int pos, int klo, int num_sinks) {
    const int hi = pos + 1 - k0, lo = klo - k0, s = num_sinks - k0;
    const uint32_t upto = hi >= 32 ? ~0u : (hi > 0 ? (1u << hi) - 1 : 0u);
    const uint32_t from = lo <= 0 ? ~0u : (lo < 32 ? ~((1u << lo) - 1) : 0u);
    const uint32_t sink = s >= 32 ? ~0u : (s > 0 ? (1u << s) - 1 : 0u);
    return upto & (from | sink);
}

template <typename QT, int kCache> using OperandOf = typename std::conditional<kCache == kCache16, QT, __half>::type;

// The value at byte or element `at` of a 16-bit or E4M3 cache.
template <typename QT, int kCache> __device__ __forceinline__ float cache_value(const void *cache, int64_t at) {
    if constexpr (kCache == kCacheE4M3)
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const __nv_fp8_storage_t *>(cache)[at], __NV_E4M3)));
    else
        return to_float<QT>(static_cast<const QT *>(cache)[at]);
}

// Add the non-finite values of V that a row sees among the axis's keys [k0, k1) to its written result (out of
// type QT, or a partial result): they were zeroed for the products.  Rare, so plain.
template <typename QT, int D, int kCache>
static __device__ __noinline__ void add_non_finite(const SinkPrefillParams &p, int seq, int h, int hidden, int k0, int k1,
                                                   int pos, int klo, QT *out, float4 *part) {
    const TreeArgs &a = p.t.a;
    for (int k = k0; k < k1; ++k) {
        if (k > pos || (k < klo && k >= p.num_sinks)) continue;
        const int c = k >> p.bs_shift;
        const int id = a.block_table[seq * a.bt_stride + (c < p.sink_blocks ? c : c + hidden)];
        if (id < 0 || id >= a.num_blocks) continue;
        const int64_t at = ((static_cast<int64_t>(id) * a.block_size + (k & (a.block_size - 1))) * a.num_kv_heads + h) * D;
        for (int d = 0; d < D; ++d) {
            const float f = cache_value<QT, kCache>(a.v_cache, at + d);
            if (isfinite(f)) continue;
            if (part) reinterpret_cast<float *>(part + static_cast<int64_t>(d / 4) * p.t.rows_per_item)[d % 4] += f;
            else out[d] = from_float<QT>(to_float<QT>(out[d]) + f);
        }
    }
}

// Eight INT4 codes (a 32-bit word) -> their values in fp16, as pairs (0, 4), (1, 5), (2, 6), (3, 7): with u =
// code ^ 8, the fp16 of bits 0x6400 | u is 1024 + u, that of 0x6400 | u << 4 is 1024 + 16 u, both exact.
__device__ __forceinline__ uint4 int4x8_values(uint32_t w) {
    const __half2 off = __half2half2(__ushort_as_half(0xE408));       // -(1024 + 8)
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00)), off16 = __half2half2(__ushort_as_half(0xD480));  // -72
    auto as_h2 = [](uint32_t v) { return *reinterpret_cast<__half2 *>(&v); };
    auto as_u = [](__half2 v) { return *reinterpret_cast<uint32_t *>(&v); };
    const uint32_t w8 = w >> 8;
    uint4 r;
    r.x = as_u(__hadd2(as_h2(and_xor(w, 0x000f000fu, 0x64086408u)), off));
    r.y = as_u(__hfma2(as_h2(and_xor(w, 0x00f000f0u, 0x64806480u)), sixteenth, off16));
    r.z = as_u(__hadd2(as_h2(and_xor(w8, 0x000f000fu, 0x64086408u)), off));
    r.w = as_u(__hfma2(as_h2(and_xor(w8, 0x00f000f0u, 0x64806480u)), sixteenth, off16));
    return r;
}
// Where dim d of each eight stands among such pairs, and the other way round.
__host__ __device__ constexpr int int4_place(int d) { return d < 4 ? 2 * d : 2 * (d - 4) + 1; }

// 16 bytes from global to shared memory, asynchronously (zeros when !there); in groups, of which all but the
// latest N are waited for.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The first tile's weights are formed before its maximum is known, and the reference in use kept while it will do.
// How far (log2) a row's maximum may exceed the reference in use, and how far below the first one, 0, it may
// lie: bf16 has float's exponents; fp16 weights are formed 2^7 higher (kFactor), the largest then at 2^7 .. 2^15.
// (16 chunks / over INT4, us: 967 / 1468; with 8 in the place of 16 for bf16 986 / 1468, with each row's first maximum as
// its first reference, hence a second pass over that tile, 987 / 1485.)
template <typename MT> constexpr float kAbove = 16.f;
template <> constexpr float kAbove<__half> = kRescaleLog2;
template <typename MT> constexpr float kBelow = 16.f;
template <> constexpr float kBelow<__half> = 0.f;
// log2 of a factor on all weights: bf16 weights are formed as much lower, at most 1, so that no value near bf16's
// largest is multiplied beyond float's range (values above 2^111 were, by weights of up to 2^16).
template <typename MT> constexpr float kFactor = -kAbove<MT>;
template <> constexpr float kFactor<__half> = kWeightLog2<__half>;

// The sum is of the weights before their rounding.  With a reference that is not a row's maximum its largest weight is
// not 1 and has a rounding of its own, up to 2^-9 of it in bf16, which stays in the result where that key holds most of
// the row's weight: a sink, or the only key of a row.  So the result is divided by the sum and the `excess`, what the
// rounding added to the largest weight of each tile: six instructions a row and tile.  Worked out in 64 bits, the
// error over that of rounding the result alone, with the excess / with a sum of all rounded weights / without: 1.00 /
// 1.00 / off by the weight's rounding for one key, 1.12 / 1.11 / 1.40 for two, 1.27 / 1.26 / 1.42 for 8, 1.38 / 1.37 /
// 1.40 for 128, 1.02 / 1.02 / 1.41 for 128 with one 2^10 above the others.  The log-sum-exp is the plain sum's.
__device__ __forceinline__ float rounding_of(float x, __half) { return __half2float(__float2half_rn(x)) - x; }
__device__ __forceinline__ float rounding_of(float x, __nv_bfloat16) { return __bfloat162float(__float2bfloat16_rn(x)) - x; }

// The larger magnitudes of two packed pairs.
template <typename T> __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2 m = __hmax2(__habs2(*reinterpret_cast<const T2 *>(&a)), __habs2(*reinterpret_cast<const T2 *>(&b)));
    return *reinterpret_cast<const uint32_t *>(&m);
}

__device__ __forceinline__ void fence_proxy_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <typename QT, int D, int kCache>
__global__ void __launch_bounds__(kThreads<kCache>, 1)
prefill_sinks_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ SinkPrefillParams p) {
    using TL = Tile<D>;
    using MT = OperandOf<QT, kCache>;
    constexpr bool kWide = kCache != kCache16;
    constexpr int kStages = TL::kStages, kTileBytes = TL::kBytes;
    const TreeArgs &a = p.t.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = p.t.group, TQ = p.t.tokens_per_tile, bs = a.block_size;
    const int c = blockIdx.x;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + TL::kOffBar);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + TL::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + TL::kOffMisc + 4);
    // per piece, and per widening warp
    volatile int *odd_flag = reinterpret_cast<volatile int *>(smem + TL::kOffMisc + 8);  // [kWideners][kFlags]
    int32_t *cleaned = reinterpret_cast<int32_t *>(smem + TL::kOffMisc + 8 + 4 * kWideners * kFlags);  // [kStages]: entry + 1
    float *join = reinterpret_cast<float *>(smem + TL::kOffJoin);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto bar_full = [&](int s) { return smem_u32(&bars[kBarKv + s]); };
    auto bar_empty = [&](int s) { return smem_u32(&bars[kBarKv + kStages + s]); };

    if (!kWide && threadIdx.x == 32) {
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    if (threadIdx.x == 0) {
        mbar_init(bar(kBarQFull), kWide ? 256 : 1);
        mbar_init(bar(kBarQEmpty), 2);
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(kBarS + x), 1);
            mbar_init(bar(kBarP + x), 128);
            mbar_init(bar(kBarPv + x), 1);
            mbar_init(bar(kBarPd + x), 1);
            mbar_init(bar(kBarDrain + x), 1);
        }
        mbar_init(bar(kBarJoin), 128);
        mbar_init(bar(kBarJoined), 128);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar_full(s), kWide ? kWideners : 1);
            mbar_init(bar_empty(s), kWide ? 2 : 3);  // released by both chains, and the cleaning warp
        }
        *abort_flag = 0;
        for (int i = 0; i < kWideners * kFlags; ++i) odd_flag[i] = 0;
        for (int i = 0; i < kStages; ++i) cleaned[i] = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    ShareScratch &scratch = *reinterpret_cast<ShareScratch *>(smem + TL::kOffScratch);
    int64_t x0, x1, item_cost;
    previous_kernel_done();
    let_next_kernel_launch();
    share_of_cta<kThreads<kCache>>(p, c, x0, x1, item_cost, scratch);
    zero_rejected<QT, D>(p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (x0 == x1) {
        // no share: nothing but the record that says so
        if (threadIdx.x == 0) p.t.ws_first[2 * c] = make_int4(-1, 0, 0, 0);
    } else if (warp >= 8) {
        // (kWide: 512 threads start with 128 registers each, of which the softmax's two warpgroups take 168 and
        // the others keep 88)
        if constexpr (kWide) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        Walk w;
        w.start(scratch.start, x0, x1, item_cost);
        if (!kWide && warp == 8) {
            // ============================================================ TMA producer
            const int bpt = kBN / bs;  // blocks of a key tile
            const uint32_t q_bytes = static_cast<uint32_t>(TL::kHalves) * TQ * g * 128;
            int entry = 0;  // ring entries filled
            int piece = 0;
            bool stop = false;
            while (!stop && w.next(p)) {
                const Seq s = w.cur;
                if (piece == 0 && lane == 0) w.record(p, c);
                // block ids of key tile j: lane l holds block j * bpt + l of the axis
                const int nblk = (w.pl >> p.bs_shift) + 1;
                auto entry_of = [&](int j) {  // (read before it is needed, checked when it is)
                    const int lb = j * bpt + lane;
                    return lane < bpt && lb < nblk ? a.block_table[static_cast<int64_t>(w.seq) * a.bt_stride + w.block(p, lb)]
                                                   : a.num_blocks;  // one past the pool: the copy reads zeros
                };
                int next_id = entry_of(w.ja);
                bool ok = true;
                if (lane == 0) {
                    // Q of the item, once the piece before has formed its last scores
                    if (piece > 0) ok = mbar_wait_sleep(bar(kBarQEmpty), (piece - 1) & 1);
                    if (ok) {
                        mbar_arrive_expect_tx(bar(kBarQFull), w.nt * q_bytes);
                        for (int x = 0; x < w.nt; ++x)
                            for (int hf = 0; hf < TL::kHalves; ++hf)
                                tma_load_3d(smem_u32(smem + x * kTileBytes + hf * kHalf), &tmap_q, bar(kBarQFull), 64 * hf,
                                            w.h * g, s.q0 + w.t0 + x * TQ);
                    }
                }
                if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) {
                    if (lane == 0) {
                        report(a.d_err, KV_DERR_TIMEOUT);
                        *abort_flag = 1;
                    }
                    break;
                }
                ++piece;
                for (int j = w.ja; j < w.jb && !stop; ++j) {
                    int my_id = next_id;
                    if (j + 1 < w.jb) next_id = entry_of(j + 1);
                    if (my_id < 0 || my_id > a.num_blocks || (my_id == a.num_blocks && lane < bpt && j * bpt + lane < nblk)) {
                        report(a.d_err, KV_DERR_BAD_BLOCK);
                        my_id = a.num_blocks;
                    }
                    for (int is_v = 0; is_v < 2; ++is_v) {
                        const int slot = entry % kStages;
                        int quit = 0;
                        if (lane == 0) {
                            if (entry >= kStages && !mbar_wait_sleep(bar_empty(slot), (entry / kStages - 1) & 1)) {
                                quit = 1;
                                report(a.d_err, KV_DERR_TIMEOUT);
                                *abort_flag = 1;
                            } else if (*abort_flag) {
                                quit = 1;
                            }
                            if (!quit) mbar_arrive_expect_tx(bar_full(slot), kTileBytes);
                        }
                        if (__shfl_sync(0xffffffffu, quit, 0)) {
                            stop = true;
                            break;
                        }
                        const CUtensorMap *m = is_v ? &tmap_v : &tmap_k;
                        uint8_t *dst = smem + TL::kOffKV + slot * kTileBytes;
                        for (int jb = 0; jb < bpt; ++jb) {
                            const int id = __shfl_sync(0xffffffffu, my_id, jb);
                            if (lane == 0)
                                tma_load_5d(smem_u32(dst + jb * bs * TL::kHalves * 128), m, bar_full(slot), 0, 0,
                                            w.h * TL::kHalves, 0, id);
                        }
                        ++entry;
                    }
                }
            }
            // never leave with copies in flight into this CTA's shared memory
            if (lane == 0) {
                if (piece > 0 && !mbar_wait_sleep(bar(kBarQFull), (piece - 1) & 1)) report(a.d_err, KV_DERR_TIMEOUT);
                for (int i = max(0, entry - kStages); i < entry; ++i)
                    if (!mbar_wait_sleep(bar_full(i % kStages), (i / kStages) & 1)) report(a.d_err, KV_DERR_TIMEOUT);
            }
        } else if (warp == 9 || warp == 10) {
            // ============================================================ MMA issue, one lane a chain
            // Chain x, key tile by key tile: S_x once the product that read the columns it overwrites has
            // completed; O_x once the softmax has written P_x and the V tile has landed (and been
            // cleaned).  The other chain's tiles are released as soon as they have landed: everyone who
            // waits for a ring entry passes all of them in order, so that no phase of its barrier can be
            // mistaken.
            const int x = warp - 9;
            constexpr uint32_t ab = AbFormat<MT>::value;
            constexpr uint32_t idesc_s = mma_idesc(ab, false, kBM, kBN);
            constexpr uint32_t idesc_pv = mma_idesc(ab, true, kBM, D);
            if (lane == 0) {
                const uint64_t dkv = smem_desc(smem_u32(smem + TL::kOffKV), 16, TL::kGroup);
                const uint64_t dv0 = smem_desc(smem_u32(smem + TL::kOffKV), 1024, TL::kGroup);
                const uint32_t t_s = tmem + x * 128, t_o = tmem + kColO + x * 128;
                auto full = [&](int e) { return mbar_wait_bounded(bar_full(e % kStages), (e / kStages) & 1); };
                int base = 0;  // key tiles of the pieces before
                int npv = 0;   // products O_x committed
                bool dead = false;
                for (int piece = 0; !dead && w.next(p); ++piece) {
                    if (*abort_flag != 0) break;
                    if (!mbar_wait_bounded(bar(kBarQFull), piece & 1)) {
                        dead = true;
                        break;
                    }
                    const int nt = w.nt;
                    const uint64_t dq = smem_desc(smem_u32(smem + (nt == 2 ? x * kTileBytes : 0)), 16, 1024);
                    const int step = nt == 2 ? 1 : 2;
                    const int first = w.ja + (nt == 2 ? 0 : x);
                    if (first >= w.jb) mbar_arrive(bar(kBarQEmpty));  // no tile for this chain
                    for (int j = w.ja; j < w.jb; ++j) {
                        const bool last = j + step >= w.jb;
                        const int ek = 2 * (base + j - w.ja), ev = ek + 1;
                        const int sk = ek % kStages, sv = ev % kStages;
                        if (nt == 1 && ((j - w.ja) & 1) != x) {
                            bool landed = full(ek);
                            if (landed) mbar_arrive(bar_empty(sk));
                            landed = landed && full(ev);
                            if (landed) mbar_arrive(bar_empty(sv));
                            if (!landed) {
                                dead = true;
                                break;
                            }
                            continue;
                        }
                        if ((npv > 0 && !mbar_wait_bounded(bar(kBarPd + x), (npv - 1) & 1)) || !full(ek)) {
                            dead = true;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t dk = dkv + static_cast<uint64_t>((sk * kTileBytes) >> 4);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const int in = (k & 3) * 32;
                            mma_f16(t_s, dq + (((k >> 2) * kHalf + in) >> 4), dk + (((k >> 2) * 1024 + in) >> 4), idesc_s, k > 0);
                        }
                        mma_commit(bar(kBarS + x));
                        mma_commit(bar_empty(sk));
                        if (last) mma_commit(bar(kBarQEmpty));
                        if (!full(ev) || (!kWide && w.mixed(p, j) && !wait_at_least_bounded(&cleaned[sv], ev + 1)) ||
                            !mbar_wait_bounded(bar(kBarP + x), npv & 1)) {
                            dead = true;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t dv = dv0 + static_cast<uint64_t>((sv * kTileBytes) >> 4);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_f16_ts(t_o, t_s + k * 8, dv + ((k * 2 * TL::kGroup) >> 4), idesc_pv, j > first || k > 0);
                        mma_commit(bar(kBarPd + x));
                        mma_commit(bar_empty(sv));
                        if (last) mma_commit(bar(kBarPv + x));
                        ++npv;
                    }
                    base += w.jb - w.ja;
                }
                if (dead) {
                    report(a.d_err, KV_DERR_TIMEOUT);
                    *abort_flag = 1;
                }
                // every MMA this lane issued has completed before TMEM is freed
                mma_commit(bar(kBarDrain + x));
                if (!mbar_wait_bounded(bar(kBarDrain + x), 0)) report(a.d_err, KV_DERR_TIMEOUT);
            }
            __syncwarp();
        } else if (!kWide && warp == 11) {
            // ============================================================ cleaning of V tiles
            int base = 0;
            bool dead = false;
            for (int piece = 0; !dead && w.next(p); ++piece) {
                if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
                if (lane == 0) odd_flag[piece % kFlags] = 0;
                __syncwarp();
                for (int e = 0; e < 2 * (w.jb - w.ja); ++e) {
                    const int j = w.ja + (e >> 1);
                    const int ev = 2 * base + e, sv = ev % kStages;
                    if (!__all_sync(0xffffffffu, mbar_wait_sleep(bar_full(sv), (ev / kStages) & 1))) {
                        dead = true;
                        break;
                    }
                    if (!(e & 1) || !w.mixed(p, j)) {
                        if (lane == 0) mbar_arrive(bar_empty(sv));
                        continue;
                    }
                    const uint32_t tile = smem_u32(smem + TL::kOffKV + sv * kTileBytes);
                    const int k0 = j * kBN;
                    bool odd = false;
                    auto clean = [&](int lo, int hi, bool zero) {
                        lo = max(lo, k0) - k0;
                        hi = min(hi, k0 + kBN) - k0;
                        if (lo >= hi) return;  // (either may lie 2^31 from the tile: sinks past any length)
                        for (int i = lo * 8 + lane; i < hi * 8; i += 32)
                            for (int hf = 0; hf < TL::kHalves; ++hf)
                                clean_chunk<MT>(tile + (i >> 6) * TL::kGroup + hf * 1024 + (i & 63) * 16, zero, odd);
                    };
                    // keys no row sees: between the sinks and the first row's window, and behind the last row;
                    // keys some rows do not see: up to the last row's window, and the item's own behind its first
                    const int from = max(w.window_from(p, w.pf), p.num_sinks), to = w.window_from(p, w.pl);
                    if (a.window > 0) {
                        clean(p.num_sinks, w.window_from(p, w.pf), true);
                        clean(from, min(to, w.pf + 1), false);
                    }
                    clean(w.pf + 1, w.pl + 1, false);
                    clean(w.pl + 1, ((w.pl >> p.bs_shift) + 1) << p.bs_shift, true);
                    if (__any_sync(0xffffffffu, odd) && lane == 0) odd_flag[piece % kFlags] = 1;
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        st_release_cta(&cleaned[sv], ev + 1);
                        mbar_arrive(bar_empty(sv));
                    }
                    __syncwarp();
                }
                base += w.jb - w.ja;
            }
            if (dead && lane == 0) {
                report(a.d_err, KV_DERR_TIMEOUT);
                *abort_flag = 1;
            }
        } else if (kWide && warp >= 8) {
            // ============================================================ codes to fp16 tiles
            // Each of the six warps takes every sixth group of 8 keys; lane l holds 16 bytes of key l & 7 (E4M3:
            // 16 of each half of it).  A lane fetches what it will convert itself, two units ahead.
            if constexpr (kWide) {
                constexpr int kRow = kCache == kCacheInt4 ? D / 2 : D;  // bytes of a key of a head
                constexpr int kParts = kRow / 64;                       // 64-byte parts of it = units of a tile
                constexpr int kAll = kBN / 8 / kParts;                  // groups of a unit,
                constexpr int kGroups = (kAll + kWideners - 1) / kWideners;  // of a warp at most
                const int wi = warp == 8 ? 0 : warp - 10;
                const int bpt = kBN / bs;
                const int row = lane & 7, quarter = lane >> 3;
                const uint32_t token = static_cast<uint32_t>(a.num_kv_heads) * kRow;  // bytes of a slot,
                const uint32_t block = token << p.bs_shift;                           // and of a block (below 2^32)
                uint8_t *codes = smem + TL::kOffUnits + lane * 16;
                // ---- the fetching side: its own walk over the units
                Walk f = w;
                int fj = 0, fpart = 0, fslot = 0;  // key tile, unit of its K (below kParts) and V, place
                int ids = -1, next_ids = -1;       // lane l: block l of tiles fj and fj + 1 (-1: zeros)
                bool more = f.next(p);
                int64_t at = 0;                    // this lane's bytes of a block's first key
                auto load_ids = [&](int j) {
                    const int lb = j * bpt + lane;
                    if (lane >= bpt || lb > f.pl >> p.bs_shift) return -1;
                    const int e = a.block_table[static_cast<int64_t>(f.seq) * a.bt_stride + f.block(p, lb)];
                    if (e >= 0 && e < a.num_blocks) return e;
                    if (wi == 0) report(a.d_err, KV_DERR_BAD_BLOCK);
                    return -1;
                };
                auto begin = [&]() {  // a piece
                    fj = f.ja, fpart = 0;
                    ids = load_ids(fj);
                    at = f.h * kRow + quarter * 16 + static_cast<int64_t>(row) * token;
                };
                auto fetch = [&]() {
                    if (more) {
                        if (fpart == 0 && fj + 1 < f.jb) next_ids = load_ids(fj + 1);
                        const bool is_v = fpart >= kParts;
                        const int base = is_v ? fpart - kParts : fpart;
                        const uint8_t *mine = static_cast<const uint8_t *>(is_v ? a.v_cache : p.k_cache) + at;
                        const uint32_t dst = smem_u32(codes + fslot * kUnitBytes);
#pragma unroll
                        for (int i = 0; i < kGroups; ++i) {
                            const int grp = i * kWideners + wi;          // of the unit
                            if (grp >= kAll) break;
                            const int k = (base * kAll + grp) * 8;  // its first key, in the tile
                            const int id = __shfl_sync(0xffffffffu, ids, k >> p.bs_shift);
                            const uint8_t *src = mine + (k & (bs - 1)) * token + static_cast<uint64_t>(static_cast<uint32_t>(max(id, 0))) * block;
#pragma unroll
                            for (int u = 0; u < kParts; ++u) copy16_async(dst + (grp * kParts + u) * 512, src + 64 * u, id >= 0);
                        }
                        if (++fpart == 2 * kParts) {
                            fpart = 0;
                            ids = next_ids;
                            if (++fj == f.jb) {
                                more = f.next(p);
                                if (more) begin();
                            }
                        }
                    }
                    copies_commit();
                    if (++fslot == kUnits) fslot = 0;
                };
                if (more) begin();
#pragma unroll
                for (int i = 0; i < kUnits - 1; ++i) fetch();
                // ---- the converting side
                int entry = 0, cslot = 0;
                bool dead = false;
                for (int piece = 0; !dead && w.next(p); ++piece) {
                    if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
                    if (piece == 0 && wi == 0 && lane == 0) w.record(p, c);
                    if (lane == 0) odd_flag[wi * kFlags + piece % kFlags] = 0;
                    __syncwarp();
                    for (int e = 0; e < 2 * (w.jb - w.ja); ++e, ++entry) {
                        const int j = w.ja + (e >> 1);
                        const bool is_v = e & 1;
                        const int slot = entry % kStages;
                        if (entry >= kStages &&
                            !__all_sync(0xffffffffu, mbar_wait_sleep(bar_empty(slot), (entry / kStages - 1) & 1))) {
                            dead = true;
                            break;
                        }
                        if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
                        uint8_t *tile = smem + TL::kOffKV + slot * kTileBytes + row * 128;
                        const bool mixed = kCache == kCacheE4M3 && is_v && w.mixed(p, j);
                        bool odd = false;
#pragma unroll 1
                        for (int part = 0; part < kParts; ++part) {
                            fetch();  // (into the place of the unit before this one)
                            copies_wait<kUnits - 1>();
                            const uint8_t *unit = codes + cslot * kUnitBytes;
                            if (++cslot == kUnits) cslot = 0;
#pragma unroll
                            for (int i = 0; i < kGroups; ++i) {
                                const int in = i * kWideners + wi, grp = part * kAll + in;  // in the unit, in the tile
                                if (in >= kAll) break;
                                uint8_t *dst = tile + grp * TL::kGroup;
                                if constexpr (kCache == kCacheInt4) {
                                    const uint4 held = *reinterpret_cast<const uint4 *>(unit + in * 512);
                                    const uint32_t words[4] = {held.x, held.y, held.z, held.w};
                                    // 32 dims: four chunks of one half of the head
#pragma unroll
                                    for (int u = 0; u < 4; ++u)
                                        *reinterpret_cast<uint4 *>(dst + (quarter >> 1) * 1024 +
                                                                   ((((quarter & 1) * 4 + u) ^ row) << 4)) = int4x8_values(words[u]);
                                } else {
                                    const int k = j * kBN + grp * 8 + row;
                                    const bool none = mixed && (k > w.pl || (k >= p.num_sinks && k < w.window_from(p, w.pf)));
                                    const bool some = mixed && (k > w.pf || (k >= p.num_sinks && k < w.window_from(p, w.pl)));
#pragma unroll
                                    for (int u = 0; u < kParts; ++u) {
                                        const uint4 held = *reinterpret_cast<const uint4 *>(unit + (in * kParts + u) * 512);
                                        uint32_t words[4] = {held.x, held.y, held.z, held.w};
                                        if (mixed) {
#pragma unroll
                                            for (int q4 = 0; q4 < 4; ++q4) {
                                                // bytes that are NaN (there are no infinities)
                                                const uint32_t nan = some ? __vcmpeq4(words[q4] & 0x7f7f7f7fu, 0x7f7f7f7fu) : 0u;
                                                odd |= nan != 0 && !none;
                                                words[q4] &= none ? 0u : ~nan;
                                            }
                                        }
                                        // 16 dims: two chunks of half u of the head
                                        uint32_t v[8];
#pragma unroll
                                        for (int q4 = 0; q4 < 4; ++q4) e4m3x4_to_h2x2(words[q4], v[2 * q4], v[2 * q4 + 1]);
                                        *reinterpret_cast<uint4 *>(dst + u * 1024 + (((quarter * 2) ^ row) << 4)) =
                                            make_uint4(v[0], v[1], v[2], v[3]);
                                        *reinterpret_cast<uint4 *>(dst + u * 1024 + (((quarter * 2 + 1) ^ row) << 4)) =
                                            make_uint4(v[4], v[5], v[6], v[7]);
                                    }
                                }
                            }
                        }
                        if (__any_sync(0xffffffffu, odd) && lane == 0) odd_flag[wi * kFlags + piece % kFlags] = 1;
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_full(slot));
                    }
                }
                copies_wait<0>();  // never leave with copies in flight into this CTA's shared memory
                if (dead && lane == 0) {
                    report(a.d_err, KV_DERR_TIMEOUT);
                    *abort_flag = 1;
                }
            }
        }
    } else {
        // ============================================================ softmax and results
        if constexpr (kWide) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        Walk w;
        w.start(scratch.start, x0, x1, item_cost);
        const int x = warp >> 2;                // chain
        const int r = threadIdx.x & 127;        // query row in the tile = TMEM lane
        const int tl = r / g, hh = r - tl * g;  // its token in the tile and head in the group
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t t_s = trow + x * 128, t_o = trow + kColO + x * 128;
        bool dead = false;
        // waits are decided for the whole warp: its lanes take the warp-collective TMEM
        // loads and stores together
        auto wait_all = [&](uint32_t b, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait_sleep(b, parity));
        };
        int ns = 0, npv = 0, njoin = 0;  // phases taken of S, Pv, Join
        for (int piece = 0; !dead && w.next(p); ++piece) {
            const Seq s = w.cur;
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
            const int nt = w.nt;
            const int tok0 = w.t0 + (nt == 2 ? x : 0) * TQ;         // first token of the row tile
            const int nq = min(TQ, s.n - tok0);                     // its tokens (the tile exists)
            const bool valid = tl < nq;
            const int64_t token = s.q0 + tok0 + (valid ? tl : 0);
            const int64_t row = token * a.num_q_heads + w.h * g + hh;
            const int first_pos = w.pf + (nt == 2 ? x : 0) * TQ, last_pos = first_pos + nq - 1;  // of the tile, on the axis
            const int pos = first_pos + (valid ? tl : 0);
            const int klo = w.window_from(p, pos);
            const bool warp_valid = __any_sync(0xffffffffu, valid);
            float c2 = a.scale_log2;
            if constexpr (kWide) {
                // the row's queries, times the K scales and a power of two, into the tile (once, where both chains
                // share it)
                uint4 raw[D / 8];
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const QT *>(p.q) + row * D);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) raw[i] = valid ? src[i] : make_uint4(0, 0, 0, 0);
                float ks[D / 8];  // a scale for each 8 dims
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    ks[i] = kCache == kCacheInt4 ? p.k_gscales[w.h * (D >> p.group_shift) + ((8 * i) >> p.group_shift)] : 1.f;
                float most = 0.f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const float2 v = unpack2<QT>(max2<QT>(max2<QT>(raw[i].x, raw[i].y), max2<QT>(raw[i].z, raw[i].w)));
                    most = fmaxf(most, fmaxf(v.x, v.y) * ks[i]);
                }
                // 2^up with 2^7 <= most * 2^up < 2^8, as far as floats go (2^up and 2^-up are normal ones)
                const int exponent = static_cast<int>(__float_as_uint(most) >> 23) - 127;  // (-127: 0 or subnormal)
                const int up = most > 0.f && exponent < 128 ? min(7 - exponent, 126) : 0;  // (-120 at least)
                const float factor = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                // (a scale that underflows, or of 0, as the least normal number: an unseen score of -inf times it
                // has to stay -inf)
                c2 = fmaxf(c2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23), FLT_MIN);
                if (piece > 0 && !wait_all(bar(kBarQEmpty), (piece - 1) & 1)) {  // the piece before has formed its last scores
                    dead = true;
                    break;
                }
                if (nt == 2 || x == 0) {
                    uint8_t *dst = smem + (nt == 2 ? x * kTileBytes : 0) + r * 128;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 v2 = unpack2<QT>(u[e]);
                            v[2 * e] = v2.x * ks[i] * factor, v[2 * e + 1] = v2.y * ks[i] * factor;
                        }
                        const uint4 h8 = kCache == kCacheInt4
                                             ? make_uint4(pack2<MT>(v[0], v[4]), pack2<MT>(v[1], v[5]), pack2<MT>(v[2], v[6]),
                                                          pack2<MT>(v[3], v[7]))
                                             : make_uint4(pack2<MT>(v[0], v[1]), pack2<MT>(v[2], v[3]), pack2<MT>(v[4], v[5]),
                                                          pack2<MT>(v[6], v[7]));
                        *reinterpret_cast<uint4 *>(dst + (i >> 3) * kHalf + (((i & 7) ^ (r & 7)) << 4)) = h8;
                    }
                    fence_proxy_async_shared();
                }
                mbar_arrive(bar(kBarQFull));
            }
            const float2 cc = make_float2(c2, c2);
            float m_used = -INFINITY;  // the reference maximum of O and the sums, in log2 units
            float2 sum = make_float2(0.f, 0.f);  // sum of the weights
            float excess = 0.f;                  // what the largest weights' rounding adds to it
            const int step = nt == 2 ? 1 : 2;
            const int first = w.ja + (nt == 2 ? 0 : x);
            uint32_t wt[64];
            for (int j = first; j < w.jb; j += step) {
                if (!wait_all(bar(kBarS + x), ns & 1)) {
                    dead = true;
                    break;
                }
                ++ns;
                tc_fence_after();
                if (warp_valid) {  // (a warp without rows leaves its lanes of P as they are)
                    if (w.mixed(p, j, first_pos, last_pos)) {
                        // (scale > 0: an unseen score of -inf gets weight 0.  Apart from the pass below, whose
                        // unrolled code the warps would fetch anew each time.  32 keys that the warp's rows all see
                        // are left as they are: 967 us and not 970 for the 16 chunks, 1468 and not 1494 over INT4.)
#pragma unroll 1
                        for (int ch = 0; ch < 4; ++ch) {
                            const uint32_t seen = valid ? seen32(j * kBN + ch * 32, pos, klo, p.num_sinks) : 0u;
                            if (__all_sync(0xffffffffu, seen == ~0u)) continue;
                            uint32_t v[32];
                            tmem_ld32_async(t_s + 32 * ch, v);
                            tmem_wait_regs(v);
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[k] = (seen >> k) & 1 ? v[k] : 0xff800000u;
                            tmem_st32u(t_s + 32 * ch, v);
                        }
                        tmem_wait_st();
                    }
                    float2 part_sum;
                    float part_excess;
                    // One pass over the tile's S: weights against the reference in use (0 at first), the tile
                    // maximum tracked alongside, 32 columns at a time with the next load in flight.  A second one
                    // when the reference has to move.
#pragma unroll 1
                    for (bool again = false;; again = true) {
                        const bool none = m_used == -INFINITY;  // no key seen so far
                        const float nref = kFactor<MT> - (none ? 0.f : m_used);
                        const float2 ref2 = make_float2(nref, nref);
                        float mraw = -INFINITY;
                        part_sum = make_float2(0.f, 0.f);
                        uint32_t buf[2][32];
                        tmem_ld32_async(t_s, buf[0]);
#pragma unroll
                        for (int ch = 0; ch < 4; ++ch) {
                            uint32_t(&v)[32] = buf[ch & 1];
                            tmem_wait_regs(v);
                            if (ch < 3) tmem_ld32_async(t_s + 32 * (ch + 1), buf[(ch + 1) & 1]);
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float s0 = __uint_as_float(v[2 * k]), s1 = __uint_as_float(v[2 * k + 1]);
                                const float2 e = fma2(make_float2(s0, s1), cc, ref2);
                                const float2 x2 = make_float2(fast_exp2(e.x), fast_exp2(e.y));
                                mraw = fmaxf(mraw, fmaxf(s0, s1));
                                wt[ch * 16 + k] = pack2<MT>(x2.x, x2.y);
                                part_sum = add2(part_sum, x2);
                            }
                        }
                        part_excess = rounding_of(fast_exp2(fmaf(mraw, c2, nref)), MT());  // (as the pass formed it)
                        if (again) break;
                        // scale > 0, so the scaled maximum is the maximum of the scaled scores
                        const float mt = mraw == -INFINITY ? -INFINITY : mraw * c2;
                        bool moved = valid && mt > (none ? 0.f : m_used) + kAbove<MT>;
                        if (none && mt != -INFINITY && !moved) {
                            if (mt >= -kBelow<MT>) m_used = 0.f;
                            else moved = valid;
                        }
                        if (!__any_sync(0xffffffffu, moved)) break;
                        const bool rescale = moved && !none;  // O and the sums hold earlier tiles
                        const float f = rescale ? fast_exp2(m_used - mt) : 1.f;
                        if (moved) {
                            m_used = mt;
                            sum.x *= f, sum.y *= f;
                            excess *= f;
                        }
                        if (__any_sync(0xffffffffu, rescale)) {
                            // the warp loads and stores O together; rows that keep their maximum scale by 1
#pragma unroll 1
                            for (int ch = 0; ch < D / 32; ++ch) {
                                float o[32];
                                tmem_ld32(t_o + ch * 32, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] *= f;
                                tmem_st32(t_o + ch * 32, o);
                            }
                            tmem_wait_st();
                        }
                    }
                    sum = add2(sum, part_sum);
                    excess += part_excess;
                    // P_x into TMEM: 128 keys of 16-bit weights = 64 columns over the S_x just read
                    tmem_st32u(t_s, wt);
                    tmem_st32u(t_s + 32, wt + 32);
                    tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(bar(kBarP + x));
            }
            if (dead) break;
            if (first < w.jb && !wait_all(bar(kBarPv + x), npv++ & 1)) {  // the last product has landed
                dead = true;
                break;
            }
            tc_fence_after();
            float m = m_used, l = sum.x + sum.y;
            float f0 = 1.f, f1 = 0.f;  // weights of O_0 (O_x with two row tiles) and O_1 in the result
            bool seen0 = false, seen1 = false, use1 = false;
            if (nt == 1) {
                if (x == 1) {
                    // hand the maximum and sums to chain 0's thread of the same row, which joins the two
                    join[r] = m;
                    join[128 + r] = l;
                    join[256 + r] = excess;
                    tc_fence_before();
                    mbar_arrive(bar(kBarJoin));
                    if (!wait_all(bar(kBarJoined), njoin++ & 1)) {
                        dead = true;
                        break;
                    }
                    tc_fence_after();
                    continue;
                }
                if (!wait_all(bar(kBarJoin), njoin++ & 1)) {
                    dead = true;
                    break;
                }
                tc_fence_after();
                const float m1 = join[r], l1 = join[128 + r];
                const float mm = fmaxf(m, m1);
                f0 = m == -INFINITY ? 0.f : fast_exp2(m - mm);
                f1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - mm);
                // a chain that saw keys counts at a weight that underflows to 0 too (a NaN or an infinity in its O
                // stays, as NaN)
                seen0 = m != -INFINITY;
                seen1 = m1 != -INFINITY;
                use1 = w.jb - w.ja > 1;
                m = mm;
                // (no guard: a chain whose scores are all NaN has no maximum, hence weight 0, and a sum of NaN,
                // which has to come through; an empty one has a sum of 0)
                l = l * f0 + l1 * f1;
                excess = excess * f0 + join[256 + r] * f1;
            }
            const float inv = l == 0.f ? 0.f : (kCache == kCacheE4M3 ? p.v_scale : 1.f) / (l + excess);
            f0 *= inv;
            f1 *= inv;
            seen0 |= f0 != 0.f;
            seen1 |= f1 != 0.f;
            QT *out16 = static_cast<QT *>(a.out) + row * D;
            const int prow = (nt == 2 ? x * 128 : 0) + r;
            const int64_t slot = part_slot(c, w.ja == 0);
            float4 *part = part_o<D>(p.t, slot, prow);
            QT *rows[4];
            if (w.whole) quad_rows<QT>(valid ? out16 : nullptr, rows);
            if (warp_valid) {
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    float o[32];
                    tmem_ld32(t_o + ch * 32, o);
                    tmem_wait_ld();
                    // a row that sees no key in a chain has nothing there, whatever O holds
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = seen0 ? o[k] * f0 : 0.f;
                    if (use1) {
                        float o1[32];
                        tmem_ld32(trow + kColO + 128 + ch * 32, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] += seen1 ? o1[k] * f1 : 0.f;
                    }
                    if constexpr (kCache == kCacheInt4) {
                        // times the V scales, the dims of each eight back in order
                        const float *vs = p.v_gscales + w.h * (D >> p.group_shift);
#pragma unroll
                        for (int k8 = 0; k8 < 4; ++k8) {
                            const float f = vs[(ch * 32 + 8 * k8) >> p.group_shift];
                            float t[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) t[e] = o[8 * k8 + int4_place(e)] * f;
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[8 * k8 + e] = t[e];
                        }
                    }
                    if (w.whole) {
                        store_rows<QT>(o, rows, ch * 32);
                    } else if (valid) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            part[static_cast<int64_t>(ch * 8 + k) * p.t.rows_per_item] =
                                make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                }
            }
            if (nt == 1) {
                tc_fence_before();
                mbar_arrive(bar(kBarJoined));  // O_1 has been read
            }
            __syncwarp();  // (a row is written by the lanes of its quad)
            if (valid) {
                const float lse2 = l == 0.f ? -INFINITY : m + (log2f(l) - kFactor<MT>);
                if (!w.whole) *part_lse(p.t, slot, prow) = lse2;
                else if (a.lse_out) a.lse_out[row] = lse2 * 0.69314718055994531f;
                if constexpr (kCache != kCacheInt4) {
                    int odd = 0;
#pragma unroll
                    for (int i = 0; i < (kWide ? kWideners : 1); ++i) odd |= odd_flag[i * kFlags + piece % kFlags];
                    if (odd) {
                        const int ka = w.ja * kBN, kb = min(w.jb * kBN, w.pl + 1);
                        const int edge = max(w.window_from(p, w.pf), p.num_sinks);
                        float4 *mine = w.whole ? nullptr : part;
                        if (a.window > 0)
                            add_non_finite<QT, D, kCache>(p, w.seq, w.h, w.hidden, max(ka, edge),
                                                          min(min(w.window_from(p, w.pl), w.pf + 1), kb), pos, klo, out16, mine);
                        add_non_finite<QT, D, kCache>(p, w.seq, w.h, w.hidden, max(ka, w.pf + 1), kb, pos, klo, out16, mine);
                    }
                }
            }
        }
        if (dead) {
            if (lane == 0) report(a.d_err, KV_DERR_TIMEOUT);
            *abort_flag = 1;
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// The merge of tree_common.cuh with a row of CTAs an item instead of one a share: most of that one's CTAs find that no
// item starts in their share, after a round trip, but this one's have to look for their item first.  With partial
// results of 256 rows of 128 dims (16 CTAs a share or item) and 152 workers the whole call takes, in us with this /
// that merge: 8 items 31.6 / 29.5, 16: 30.2 / 31.7 to 33.7, 24: 37.8 / 39.0, 32: 41.6 / 42.3, 48: 51.0 / 50.5, 64: 62.1 /
// 59.1, 96: 84 / 77.  With half as many CTAs the other is faster everywhere: 128 rows 24.9 / 22.3 (8 items), 36.1 / 34.9
// (32); 64 dims 26.5 / 26.1 (16 items), 46.3 / 45.0 (64).
static bool merge_by_items(int64_t items, const TreeParams &p) {  // (128 dims)
    return p.rows_per_item == 2 * kTreeRows && items * 4 <= p.workers && items * 16 > p.workers;
}
template <typename T, int D>
static __global__ void __launch_bounds__(256, 4) merge_items_kernel(const __grid_constant__ TreeParams p) {
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.x / p.items_per_seq, idx = blockIdx.x % p.items_per_seq;
    const int unit = blockIdx.y * 8 + (threadIdx.x >> 5);  // of 8 dims of 32 rows
    const int rr = unit / (D / 8) * 32 + lane, q = unit % (D / 8) * 2;
    previous_kernel_done();  // the attention kernel's results
    // the shares that begin in the middle of the item: `first` and the next ones
    int mine = INT_MAX, count = 0;
#pragma unroll 4
    for (int e = lane; e < p.workers; e += 32) {
        const int4 rec = __ldcg(&p.ws_first[2 * e]);
        if (rec.x == b && rec.y == idx && rec.z > 0) mine = min(mine, e), ++count;
    }
    const int first = __reduce_min_sync(0xffffffffu, mine);
    count = __reduce_add_sync(0xffffffffu, count);
    if (count == 0) return;  // the item is in one share, or there is no such item
    const int4 sq = __ldcg(&p.ws_first[2 * first + 1]);
    if (Joined::row_of(p, sq, idx, rr) < 0) return;
    Joined x;
    x.add_pieces<D, true>(p, first - 1, first - 1, 1, first - 1 + count, rr, q);
    x.store<T, D>(p, sq, idx, rr, q);
}

// The attention kernel and, with more than one share, the merge (launched as in tree_common.cuh).
template <typename QT, int D, int kCache>
static cudaError_t launch_typed(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                const SinkPrefillParams &p, int dev, cudaStream_t stream) {
    static std::atomic<bool> attr_set[64];
    constexpr int kSmem = Tile<D>::smem(kCache != kCache16);
    static_assert(kSmem <= 227 * 1024, "shared memory");
    auto kernel = prefill_sinks_kernel<QT, D, kCache>;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    const cudaError_t e = launch_dependent(kernel, dim3(p.t.workers), dim3(kThreads<kCache>), kSmem, stream, tq, tk, tv, p);
    if (e != cudaSuccess || p.t.workers < 2) return e;
    const int64_t items = static_cast<int64_t>(p.t.items_per_seq) * p.t.a.num_seqs;
    const unsigned ctas = p.t.rows_per_item / 32 * (D / 8) / 8;  // a share or item
    if constexpr (D == 128) {
        if (merge_by_items(items, p.t))
            return launch_dependent(merge_items_kernel<QT, D>, dim3(static_cast<unsigned>(items), ctas), dim3(256), 0, stream, p.t);
    }
    return launch_dependent(tree_merge_kernel<QT, D, true>, dim3(p.t.workers - 1, ctas), dim3(256), 0, stream, p.t);
}

}  // namespace sinks

// The launches over E4M3 and INT4 caches (prefill_sinks_wide.cu).
cudaError_t launch_prefill_sinks_wide(const CUtensorMap &tmap, const SinkPrefillParams &p, int cache_dtype, int q_dtype,
                                      int dev, cudaStream_t stream);

}  // namespace pkv
