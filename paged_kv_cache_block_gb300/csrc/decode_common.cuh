// Pieces shared by the decode kernels (paged_decode_kernel.cuh, paged_decode_int4.cu): launch
// parameters, the stream-K schedule over (head group, sequence, stage) and the log-sum-exp merge
// of sequences whose stages were split between workers ("Understanding PageAttention Memory
// Optimization", section "Handling Softmax Across Blocks": the softmax needs every block, so
// partial results carry their own maximum and sum and are combined exactly).
#pragma once

#include "common.cuh"
#include "dependent_launch.cuh"
#include "kernels.h"

namespace pkv {

struct KernelParams {
    DecodeArgs a;
    StepArgs f;            // fused decode step only: the slot mapping and cache write inputs
    int heads_per_cta;     // HG
    int warps_per_head;    // ceil(group * q_len / rows_per_warp)
    int blocks_per_stage;  // BPS
    int num_stages;        // NS
    int box_bytes, box_stride;
    int num_items;         // (num_kv_heads / HG) * num_seqs
    int rows_per_item;     // HG * group * q_len
    int sets_per_cta;      // INT4 kernel: independent warp sets (stream-K workers) per CTA
    int num_workers;       // INT4 kernel: stream-K workers in all (the shares the stages are cut in)
    int tile_ws;           // 16-bit / E4M3 kernel: partial results as fragment tiles (every row of a
                           // consumer warp's tile is a query row); else one workspace row per query row
    int item_cost;         // 16-bit / E4M3 kernel: a piece's fixed cost in quarter stages (shares are cut
                           // by stages plus this per item); 0: equal stage counts
    int lens_smem;         // 16-bit / E4M3 kernel: the length table is in shared memory (it fits
                           // without costing the ring a stage); else lengths are read from seq_lens
    SinkArgs sinks;        // kernels with sinks
};

// The CTA that owns flat stage s when S stages are split into G equal shares
// (CTA c owns [c*S/G, (c+1)*S/G)).
__host__ __device__ __forceinline__ int owner_cta(long long s, long long S, int G) {
    return static_cast<int>(((s + 1) * G - 1) / S);
}

// Shares actually cut from S stages by G workers: at most G, and few enough that a share holds
// at least kMinShareStages stages (one when S is smaller).  Small batches are then cut into a few
// pieces of several stages rather than one per stage (each piece costs its own output and a
// place in the merge), no share is empty and the merge never walks empty shares.
constexpr int kMinShareStages = 4;
__host__ __device__ __forceinline__ int active_shares(long long S, int G) {
    const long long by_work = S >= kMinShareStages ? S / kMinShareStages : (S > 0 ? 1 : 0);
    return by_work < G ? static_cast<int>(by_work) : G;
}

// First stage of worker w's share (S for a worker without one); its share ends where worker
// w + 1's begins.
__host__ __device__ __forceinline__ long long share_begin(long long S, int A, int w) {
    return w < A ? S * w / A : S;
}

// The first stage at or past cost position x when item i costs h quarter stages of fixed cost
// followed by its stages at 4 quarters each (item i starts at cost 4 * P[i] + h * i): the number
// of stages whose start cost lies below x.  P is the stage prefix of NI items.
__device__ __forceinline__ long long stage_at_cost(long long x, const int32_t *P, int NI, int h) {
    int lo = 0, hi = NI;  // the last item starting at or before x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (4LL * P[mid] + static_cast<long long>(h) * mid <= x) lo = mid;
        else hi = mid - 1;
    }
    if (lo == NI) return P[NI];
    const long long past = x - (4LL * P[lo] + static_cast<long long>(h) * lo) - h;
    const long long k = past <= 0 ? 0 : (past + 3) / 4;
    const long long n = P[lo + 1] - P[lo];
    return P[lo] + (k < n ? k : n);
}

// The share [*b, *e) of worker w of G over the S stages of the NI items: equal costs of stages
// plus item_cost quarter stages a piece (no share empty), or, when shares that small could be
// empty (or an item has no stages), min(G, S) equal stage counts.
__device__ __forceinline__ void share_of(int w, int G, const int32_t *P, int NI, int item_cost, bool any_empty,
                                         long long *b, long long *e) {
    const long long S = P[NI];
    const long long C = 4 * S + static_cast<long long>(item_cost) * NI;
    if (item_cost > 0 && !any_empty && C / G >= item_cost + 8) {
        *b = stage_at_cost(C * w / G, P, NI, item_cost);
        *e = stage_at_cost(C * (w + 1) / G, P, NI, item_cost);
    } else {
        const int A = active_shares(S, G);
        *b = share_begin(S, A, w);
        *e = share_begin(S, A, w + 1);
    }
}

// The length of sequence b when it is accepted (at least q_len, at most max_seq_len, within the
// block table), else -1.
__device__ __forceinline__ int checked_len(const DecodeArgs &a, int b) {
    const int L = a.seq_lens[b];
    const bool ok = L >= a.q_len && L <= a.max_seq_len &&
                    (L + a.block_size - 1) / a.block_size <= a.max_blocks_per_seq;
    return ok ? L : -1;
}

// The keys that a sequence of length L attends, as the axis the stages are cut from.  Without sinks
// the axis is the positions themselves and starts at the window's first block.  With sinks it is the
// sequence without the blocks that no row sees, those between the last sink's block and the window's
// first: block c of the axis is block c of the sequence below sink_blocks, and block c + hidden from
// there on, and all lengths and positions behind the gap are smaller by hidden * block_size.  The
// kernel runs on that axis as on an ordinary sequence that starts at block 0, so a window's keys and
// its sinks share stages and no stage is spent on the gap.
struct SinkAxis {
    int hidden;  // blocks left out
    int len;     // length on the axis
};
__device__ __forceinline__ int sink_blocks(const KernelParams &kp, int bs_shift) {
    return (kp.sinks.num_sinks + kp.a.block_size - 1) >> bs_shift;
}
__device__ __forceinline__ SinkAxis sink_axis(const KernelParams &kp, int L, int bs_shift) {
    const DecodeArgs &a = kp.a;
    const int first = a.window > 0 ? max(0, L - a.q_len - a.window + 1) >> bs_shift : 0;
    const int hidden = max(0, first - sink_blocks(kp, bs_shift));
    return SinkAxis{hidden, L - (hidden << bs_shift)};
}

// Per-CTA schedule, computed by every thread of the block (it contains __syncthreads):
//   Ls[b]  the length of sequence b, or -1 when it is rejected (KV_DERR_BAD_LEN, reported once);
//          without kLens there is no table: lengths are read from seq_lens (checked_len);
//   (returns whether some length was rejected)
//   P[i]   the number of stages of items 0 .. i-1 (an item is (head group, sequence), group-major;
//          a stage is BPS consecutive cache blocks of the attended range), P[0] = 0.
// (kp: kSinks)
template <bool kLens = true, bool kSinks = false>
__device__ __forceinline__ bool build_schedule(const KernelParams &kp, const DecodeArgs &a, int NI, int BPS, int32_t *Ls,
                                               int32_t *P, int32_t *warp_sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = a.num_seqs, q_len = a.q_len, bs = a.block_size;
    int rejected = 0;
    for (int i = threadIdx.x; i < B; i += blockDim.x) {
        const int L = checked_len(a, i);
        if (L < 0 && blockIdx.x == 0) report(a.d_err, KV_DERR_BAD_LEN);
        rejected |= L < 0 ? 1 : 0;
        if constexpr (kLens) Ls[i] = L;
    }
    const bool any_rejected = __syncthreads_or(rejected) != 0;
    // stage counts of the items (group-major, then sequence), inclusive scan into P[1..NI]
    {
        const int T = blockDim.x;
        const int per = (NI + T - 1) / T;
        const int lo = min(NI, static_cast<int>(threadIdx.x) * per), hi = min(NI, lo + per);
        // block_size and BPS are powers of two: shifts, not divisions
        const int bs_shift = __ffs(bs) - 1, bps_shift = __ffs(BPS) - 1;
        auto stages_of = [&](int seq) {  // of an item of sequence seq
            int L;
            if constexpr (kLens) L = Ls[seq];
            else L = checked_len(a, seq);
            if (L < 0) return 0;
            if constexpr (kSinks) {
                return (((sink_axis(kp, L, bs_shift).len + bs - 1) >> bs_shift) + BPS - 1) >> bps_shift;
            } else {
                const int lo_key = a.window > 0 ? max(0, L - q_len - a.window + 1) : 0;
                const int nb = ((L + bs - 1) >> bs_shift) - (lo_key >> bs_shift);
                return (nb + BPS - 1) >> bps_shift;
            }
        };
        int sum = 0;
        const int seq_lo = lo % B;
        for (int i = lo, sq = seq_lo; i < hi; ++i, sq = sq + 1 == B ? 0 : sq + 1) sum += stages_of(sq);
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            const int nw = (T + 31) >> 5;
            int w = lane < nw ? warp_sums[lane] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += v;
            }
            if (lane < nw) warp_sums[lane] = w;
        }
        __syncthreads();
        int run = incl - sum + (warp > 0 ? warp_sums[warp - 1] : 0);
        if (threadIdx.x == 0) P[0] = 0;
        for (int i = lo, sq = seq_lo; i < hi; ++i, sq = sq + 1 == B ? 0 : sq + 1) {
            run += stages_of(sq);
            P[i + 1] = run;
        }
    }
    __syncthreads();
    return any_rejected;  // (an item without stages is one of a rejected length)
}

// Whether a sum of weights w counts: one of 0 (no key seen) gives nothing.  kNan: one that is NaN (a score that
// its row sees was NaN) counts, so that the NaN stays.
template <bool kNan> __device__ __forceinline__ bool counts(float w) { return kNan ? w != 0.f : w > 0.f; }
// The same of a piece in a merge, with its lse.  kNan: every piece that saw a key counts, at a weight that has
// underflowed to 0 too: a NaN or an infinity that it holds stays (as NaN), as it would in one piece with the others.
template <bool kNan> __device__ __forceinline__ bool counts(float w, float lse) { return kNan ? lse != -INFINITY : w > 0.f; }

// One warp per (item, row): combine the pieces of a sequence that several CTAs shared, and
// write zeros (lse -inf) for sequences whose length was rejected.  P is the stage prefix.
template <typename QT, int D, bool kNan = false>
__device__ __forceinline__ void merge_row(const KernelParams &kp, const int32_t *P, int num_ctas,
                                          int64_t w, int lane) {
    const DecodeArgs &a = kp.a;
    const int item = static_cast<int>(w / kp.rows_per_item);
    const int rr = static_cast<int>(w - static_cast<int64_t>(item) * kp.rows_per_item);
    const int B = a.num_seqs;
    const int g = a.num_q_heads / a.num_kv_heads;
    const int R = g * a.q_len;
    const int seq = item % B, grp = item / B;
    const int h_loc = rr / R, r = rr % R;
    const int64_t tokq = static_cast<int64_t>(seq) * a.q_len + r / g;
    const int64_t rowid = tokq * a.num_q_heads + (grp * kp.heads_per_cta + h_loc) * g + r % g;
    const long long p0 = P[item], p1 = P[item + 1], S = P[kp.num_items];
    num_ctas = active_shares(S, num_ctas);
    constexpr int kPer = D / 32;
    constexpr int kFewPieces = 8;  // rows split into at most this many pieces take the short path
    QT *orow = static_cast<QT *>(a.out) + rowid * D + lane * kPer;
    if (p1 == p0) {  // rejected length: defined output
#pragma unroll
        for (int e = 0; e < kPer; ++e) orow[e] = from_float<QT>(0.f);
        if (a.lse_out && lane == 0) a.lse_out[rowid] = -INFINITY;
        return;
    }
    // the shares holding the item's first and last stage: written by the kernel, or (equal
    // stage counts) computed
    const bool owners = a.ws_pieces != nullptr;
    const int c_lo = owners ? a.ws_pieces[2 * item] : owner_cta(p0, S, num_ctas);
    const int c_hi = owners ? a.ws_pieces[2 * item + 1] : owner_cta(p1 - 1, S, num_ctas);
    if (c_lo == c_hi) return;  // one CTA covered it and wrote the output
    // with min(workers, stages) shares none is empty; kept as a guard for equal stage counts
    auto empty_share = [&](int c) { return !owners && S * c / num_ctas == S * (c + 1) / num_ctas; };
    float acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    float wsum = 0.f, mx = -INFINITY;
    const int n = c_hi - c_lo + 1;
    if (n <= kFewPieces) {
        // the common case: the pieces' lse (lane u holds piece u) and partial rows are all loaded
        // at once, before the weights are known, so a row costs two round trips through L2 (the
        // prefix, then everything else).  Empty shares wrote nothing and rows of weight 0 may
        // hold anything: they are selected away, never multiplied.
        const bool has = lane < n && !empty_share(c_lo + lane);
        const float lv = has ? __ldcg(a.ws_lse + static_cast<int64_t>(item + c_lo + lane) * kp.rows_per_item + rr)
                             : -INFINITY;
        float v[kFewPieces][kPer];
#pragma unroll
        for (int u = 0; u < kFewPieces; ++u) {
            const float *src = a.ws_o + (static_cast<int64_t>(item + c_lo + u) * kp.rows_per_item + rr) * D + lane * kPer;
#pragma unroll
            for (int e = 0; e < kPer; ++e) v[u][e] = u < n ? __ldcg(src + e) : 0.f;
        }
        mx = lv;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float wl = kNan ? (has && lv != -INFINITY ? expf(lv - (mx == -INFINITY ? 0.f : mx)) : 0.f)
                              : (has && mx != -INFINITY ? expf(lv - mx) : 0.f);
        wsum = wl;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
#pragma unroll
        for (int u = 0; u < kFewPieces; ++u) {
            const float wu = __shfl_sync(0xffffffffu, wl, u), lu = kNan ? __shfl_sync(0xffffffffu, lv, u) : 0.f;
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] += counts<kNan>(wu, lu) ? wu * v[u][e] : 0.f;
        }
    } else {
        for (int c = c_lo + lane; c <= c_hi; c += 32)
            if (!empty_share(c)) mx = fmaxf(mx, __ldcg(a.ws_lse + static_cast<int64_t>(item + c) * kp.rows_per_item + rr));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float ref = kNan && mx == -INFINITY ? 0.f : mx;
        if (kNan || mx != -INFINITY) {
            // pieces 32 at a time: lane i weighs piece base + i; the partial rows are then loaded
            // four pieces at a time, every load issued before the sums use them
            for (int base = c_lo; base <= c_hi; base += 32) {
                const int c = base + lane;
                float wl = 0.f, ll = -INFINITY;
                if (c <= c_hi && !empty_share(c)) {
                    ll = __ldcg(a.ws_lse + static_cast<int64_t>(item + c) * kp.rows_per_item + rr);
                    wl = expf(ll - ref);
                }
                float wsb = wl;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) wsb += __shfl_xor_sync(0xffffffffu, wsb, o);
                wsum += wsb;
                const int nb = min(32, c_hi - base + 1);
                for (int u0 = 0; u0 < nb; u0 += 4) {
                    float w[4], vv[4][kPer];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        w[u] = __shfl_sync(0xffffffffu, wl, (u0 + u) & 31);
                        const float lu = kNan ? __shfl_sync(0xffffffffu, ll, (u0 + u) & 31) : 0.f;
                        const bool ok = u0 + u < nb && counts<kNan>(w[u], lu);  // a piece without keys adds nothing
                        const float *src =
                            a.ws_o + (static_cast<int64_t>(item + base + u0 + u) * kp.rows_per_item + rr) * D + lane * kPer;
#pragma unroll
                        for (int e = 0; e < kPer; ++e) vv[u][e] = ok ? __ldcg(src + e) : 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int e = 0; e < kPer; ++e) acc[e] += w[u] * vv[u][e];
                }
            }
        }
    }
    const float inv = counts<kNan>(wsum) ? 1.f / wsum : 0.f;
#pragma unroll
    for (int e = 0; e < kPer; e += 2)
        *reinterpret_cast<uint32_t *>(orow + e) = pack2<QT>(acc[e] * inv, acc[e + 1] * inv);
    if (a.lse_out && lane == 0) a.lse_out[rowid] = counts<kNan>(wsum) ? mx + logf(wsum) : -INFINITY;
}

// Items at most, as a share of the workers, for the merges below that take a CTA where the others take a warp:
// with few items each is in many pieces, and a warp's round trips through L2, one for every 4 or 8 pieces, add
// up; with many the CTAs themselves do.  The whole call on 152 SMs, sequences of 4100 seen keys, in us by CTAs / by
// warps (both as programmatic dependents):
//   32/8 heads, 1 row, items 1, 4, 8, 12, 16, 32   14.2 / 26.1, 22.5 / 30.6, 32.1 / 36.5, 42.2 / 45.9, 52.8 / 55.0, 93.8 / 92.1
//   the same, 4 rows, items 1, 4, 8, 16            21.5 / 36.7, 29.2 / 36.4, 43.3 / 41.7, 71.2 / 60.5
//   12 heads of 64, items 1, 8, 16, 32             12.7 / 23.5, 25.7 / 29.4, 41.2 / 43.1, 71.0 / 70.9
//   INT4, 32/8 heads, 8 or 16, 32 sequences        25.0 / 32.4, 29.9 / 32.8, 46.5 / 45.8
// The two cross between 8 and 32 items of 152 workers, 9 with this share.
constexpr int kLongMergeShare = 16;

// The merge of one row's pieces by a CTA of 8 warps: each takes every eighth piece, then their sums are joined.
// (Kernels with sinks: NaN stays.)
template <typename QT, int D>
__global__ void __launch_bounds__(256) lse_merge_long_kernel(const __grid_constant__ KernelParams kp, int num_ctas) {
    constexpr int kPer = D / 32, kG = 4, kWarps = 8;
    __shared__ float part[kWarps][32 * kPer], part_m[kWarps], part_sum[kWarps];
    const DecodeArgs &a = kp.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int item = static_cast<int>(blockIdx.x / kp.rows_per_item), rr = static_cast<int>(blockIdx.x % kp.rows_per_item);
    const int B = a.num_seqs, g = a.num_q_heads / a.num_kv_heads, R = g * a.q_len;
    const int seq = item % B, grp = item / B, h_loc = rr / R, r = rr % R;
    const int64_t rowid = (static_cast<int64_t>(seq) * a.q_len + r / g) * a.num_q_heads + (grp * kp.heads_per_cta + h_loc) * g + r % g;
    QT *orow = static_cast<QT *>(a.out) + rowid * D + lane * kPer;
    previous_kernel_done();  // the attention kernel's results
    const int32_t *P = a.ws_prefix;
    const long long p0 = P[item], p1 = P[item + 1], S = P[kp.num_items];
    float acc[kPer], mx = -INFINITY, wsum = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    if (p1 > p0) {
        num_ctas = active_shares(S, num_ctas);
        const bool owners = a.ws_pieces != nullptr;
        const int c_lo = owners ? a.ws_pieces[2 * item] : owner_cta(p0, S, num_ctas);
        const int c_hi = owners ? a.ws_pieces[2 * item + 1] : owner_cta(p1 - 1, S, num_ctas);
        if (c_lo == c_hi) return;  // one worker covered it and wrote the output (every warp of the CTA alike)
        for (int base = c_lo + warp; base <= c_hi; base += kG * kWarps) {
            float l[kG], v[kG][kPer];
#pragma unroll
            for (int u = 0; u < kG; ++u) {
                const int c = base + u * kWarps;
                const int64_t row = static_cast<int64_t>(item + c) * kp.rows_per_item + rr;
                l[u] = c <= c_hi ? __ldcg(a.ws_lse + row) : -INFINITY;
#pragma unroll
                for (int e = 0; e < kPer; ++e) v[u][e] = c <= c_hi ? __ldcg(a.ws_o + row * D + lane * kPer + e) : 0.f;
            }
            float m = mx;
#pragma unroll
            for (int u = 0; u < kG; ++u) m = fmaxf(m, l[u]);
            const float ref = m == -INFINITY ? 0.f : m, f = mx == -INFINITY ? 1.f : expf(mx - ref);
            mx = m;
            wsum *= f;  // (all zero, or NaN, while there is no maximum)
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] *= f;
#pragma unroll
            for (int u = 0; u < kG; ++u) {
                const float w = expf(l[u] - ref);
                if (!counts<true>(w, l[u])) continue;
                wsum += w;
#pragma unroll
                for (int e = 0; e < kPer; ++e) acc[e] += w * v[u][e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) part[warp][e * 32 + lane] = acc[e];
    if (lane == 0) part_m[warp] = mx, part_sum[warp] = wsum;
    __syncthreads();
    if (warp) return;
    float top = -INFINITY, total = 0.f, out[kPer];
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, part_m[i]);
#pragma unroll
    for (int e = 0; e < kPer; ++e) out[e] = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const float f = part_m[i] == -INFINITY ? 1.f : expf(part_m[i] - top);
        if (part_sum[i] == 0.f) continue;
        total += part_sum[i] * f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) out[e] += part[i][e * 32 + lane] * f;
    }
    const float inv = counts<true>(total) ? 1.f / total : 0.f;
#pragma unroll
    for (int e = 0; e < kPer; e += 2) *reinterpret_cast<uint32_t *>(orow + e) = pack2<QT>(out[e] * inv, out[e + 1] * inv);
    if (a.lse_out && lane == 0)
        a.lse_out[rowid] = counts<true>(total) ? (top == -INFINITY ? 0.f : top) + logf(total) : -INFINITY;
}

template <typename QT, int D, bool kNan>
__global__ void lse_merge_kernel(const __grid_constant__ KernelParams kp, int num_ctas) {
    if constexpr (kNan) previous_kernel_done();
    const int64_t rows = static_cast<int64_t>(kp.num_items) * kp.rows_per_item;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (w >= rows) return;
    merge_row<QT, D, kNan>(kp, kp.a.ws_prefix, num_ctas, w, threadIdx.x & 31);
}

template <typename QT, int D, bool kNan = false>
static cudaError_t row_merge(const KernelParams &kp, int num_workers, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(kp.num_items) * kp.rows_per_item;
    const int threads = 256;
    const int64_t blocks = (rows * 32 + threads - 1) / threads;
    if constexpr (kNan) {  // kernels with sinks: as a programmatic dependent of theirs
        if (static_cast<int64_t>(kp.num_items) * kLongMergeShare <= num_workers)
            return launch_dependent(lse_merge_long_kernel<QT, D>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, stream, kp,
                                    num_workers);
        return launch_dependent(lse_merge_kernel<QT, D, true>, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, stream, kp,
                                num_workers);
    } else {
        lse_merge_kernel<QT, D, false><<<static_cast<unsigned>(blocks), threads, 0, stream>>>(kp, num_workers);
        return cudaGetLastError();
    }
}

// The row merge for a finished INT4 decode launch (defined in paged_attention.cu): one warp per
// (item, row) over num_items * rows_per_item rows, num_workers the shares the stages were cut in.
// (The 16-bit and E4M3 decode kernels write their partial results as fragment tiles and have
// their own tile merge, in paged_decode_kernel.cuh.)
cudaError_t launch_lse_merge(const KernelParams &kp, int num_workers, int q_dtype, cudaStream_t stream);
// The same for the INT4 kernel with sinks, whose pieces may hold NaN (paged_sinks.cu).
cudaError_t launch_lse_merge_nan(const KernelParams &kp, int num_workers, int q_dtype, cudaStream_t stream);

}  // namespace pkv
