// Attention of drafted trees over the paged cache, on the fifth-generation tensor cores
// (speculative decoding: "vLLM의 KV cache 연결 흐름", section "EngineCore가 하는 일", several tokens
// a request and step; attention through the block table as in its section "Slot mapping은 왜
// 필요한가").
//
// Row i of a sequence attends the context keys (those inside its window) and the drafted keys of
// its mask word:  out = sum_j p_j V_j / sum_j p_j,  p_j = exp2(scale log2(e) q.K_j - m).
//
// The n drafted tokens x g heads of a kv head's group are its query rows, in tiles of up to 128
// rows (whole tokens: 128 / g tokens, row r = token r / g, head r % g).  An item is (sequence, kv
// head, two row tiles); its keys go in tiles of 128.  Two chains x = 0, 1 of
//   S_x = Q K_j^T   tcgen05.mma, M 128, N 128; fp32 in TMEM
//   P_x = exp2(S_x * scale - m)   one thread a row; 16-bit weights back into TMEM over S_x
//   O_x += P_x V_j  tcgen05.mma, A = P_x in TMEM, fp32 in TMEM across key tiles
// run at once, so that one chain's softmax overlaps the other's products.  An item with two row
// tiles gives each chain one of them and both read every key tile.  An item with one row tile
// (few drafted tokens, the case that is bound by reading the cache) gives chain x every second
// key tile, and the chains' results are joined at the end.
//
// The flat list of (item, key tile) is cut into equal shares, one a CTA (an item costs kItemCost
// tiles more), so the batch's lengths do not matter; an item that lies in several shares leaves a
// partial result from each, joined by a second, small kernel.
//
// Warps (384 threads): 0-3 softmax of chain 0, 4-7 of chain 1 (thread = TMEM lane = query row), 8
// TMA producer (Q once an item, K and V tiles through a ring), 9 and 10 issue the chains' MMAs, 11
// cleans V tiles that hold keys which not every row sees: a weight of 0 times a NaN or an
// infinity would not be 0, so values that no row sees are zeroed in shared memory, and non-finite
// values that some rows see are zeroed and added afterwards to the rows that do see them.
// Weights are taken against the reference maximum in use; only when a row's maximum exceeds it by
// more than 2^8 are its O and sum rescaled.
// The matrix instructions take 16-bit operands, so the weights are rounded (half a step of each) for the
// second product; float32 weights would be two such products.  On normal scores that makes the output's
// error 1.35 to 1.4 times that of rounding the result alone (bf16 2.3e-3 of its rms, fp16 2.9e-4).  The sum is of
// the weights before that rounding: with a second sum, of the rounded ones, as normaliser a batch of 38
// trees of 256 rows took 7 % longer, with the same error on normal scores; only where most weights of a
// row are equal, so that one rounding is common to them all, would it cancel (1.0 times instead of 1.35).
// Every wait is bounded (2 s): on expiry
// KV_DERR_TIMEOUT is set, what was issued is drained, TMEM is freed and the CTA returns.
#include "tree_common.cuh"

namespace pkv {
namespace {

constexpr int kBM = kTreeRows;
constexpr int kBN = 128;           // keys of a key tile
constexpr int kThreads = 384;
constexpr uint32_t kColO = 256;

template <int D> struct Tile {
    static constexpr int kHalves = D / 64;
    static constexpr int kBytes = kHalves * kHalf;      // a Q, K or V tile
    static constexpr int kGroup = kHalves * 1024;       // 8 keys of a K or V tile: [64 dims of D][key][dim]
    static constexpr int kStages = D == 128 ? 4 : 8;    // ring entries (128 KB)
    static constexpr int kOffKV = 2 * kBytes;           // after Q_0, Q_1
    static constexpr int kOffJoin = kOffKV + kStages * kBytes;   // chain 1's maxima and sums: 2 x 128 floats
    static constexpr int kOffScratch = kOffJoin + 2 * 128 * 4;   // of the schedule
    static constexpr int kOffBar = kOffScratch + sizeof(ShareScratch);
    static constexpr int kNumBars = 14 + 2 * kStages;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;      // TMEM address, abort flag, flags, cleaned
    static constexpr int kSmem = kOffMisc + 8 + 4 * kFlags + 4 * kStages + 1024;  // + alignment
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(sizeof(ShareScratch) % 8 == 0, "the barriers behind it");
    // pieces whose V tiles can be in the ring at once, one more that the cleaning warp has begun,
    // and one without mixed tiles (only a share's last)
    static_assert(kFlags >= (kStages + 1) / 2 + 2, "a flag per piece in flight");
};

// mbarrier indices (+ x: one per chain)
enum { kBarQFull = 0, kBarQEmpty = 1, kBarS = 2, kBarP = 4, kBarPv = 6, kBarPd = 8, kBarJoin = 10,
       kBarJoined = 11, kBarDrain = 12, kBarKv = 14 };  // then KvFull[stages], KvEmpty[stages]

// Row tiles of pair pr: 2, or 1 when the tree ends in its first.
__device__ __forceinline__ int row_tiles(const TreeParams &p, const Seq &s, int pr) {
    return s.n > (2 * pr + 1) * p.tokens_per_tile ? 2 : 1;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
tree_attention_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ TreeParams p) {
    using TL = Tile<D>;
    constexpr int kStages = TL::kStages, kTileBytes = TL::kBytes;
    const TreeArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = p.group, TQ = p.tokens_per_tile, bs = a.block_size;
    const int c = blockIdx.x;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + TL::kOffBar);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + TL::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + TL::kOffMisc + 4);
    volatile int *odd_flag = reinterpret_cast<volatile int *>(smem + TL::kOffMisc + 8);  // [kFlags], per piece
    int32_t *cleaned = reinterpret_cast<int32_t *>(smem + TL::kOffMisc + 8 + 4 * kFlags);  // [kStages]: entry + 1
    float *join = reinterpret_cast<float *>(smem + TL::kOffJoin);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto bar_full = [&](int s) { return smem_u32(&bars[kBarKv + s]); };
    auto bar_empty = [&](int s) { return smem_u32(&bars[kBarKv + kStages + s]); };

    if (threadIdx.x == 32) {
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    if (threadIdx.x == 0) {
        mbar_init(bar(kBarQFull), 1);
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
            mbar_init(bar_full(s), 1);
            mbar_init(bar_empty(s), 3);  // released by both chains and the cleaning warp
        }
        *abort_flag = 0;
        for (int i = 0; i < kFlags; ++i) odd_flag[i] = 0;
        for (int i = 0; i < kStages; ++i) cleaned[i] = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // (memory of its own: chain 1 may write `join` while other warps still read the share's start)
    ShareScratch &scratch = *reinterpret_cast<ShareScratch *>(smem + TL::kOffScratch);
    int64_t x0, x1;
    int item_cost;
    previous_kernel_done();
    let_next_kernel_launch();
    share_of_cta<kThreads>(p, c, x0, x1, item_cost, scratch);
    zero_rejected<T, D>(p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    Walk w;
    w.start(scratch.start, x0, x1, item_cost);

    if (x0 == x1) {
        // no share: nothing but the record that says so
        if (threadIdx.x == 0) p.ws_first[2 * c] = make_int4(-1, 0, 0, 0);
    } else if (warp == 8) {
        // ============================================================ TMA producer
        const int bpt = kBN / bs;  // blocks of a key tile
        const uint32_t q_bytes = static_cast<uint32_t>(TL::kHalves) * TQ * g * 128;
        int entry = 0;  // ring entries filled
        int piece = 0;
        bool stop = false;
        while (!stop && w.next(p)) {
            const Seq s = w.cur;
            const int h = w.item / s.pairs, pr = w.item - h * s.pairs, nt = row_tiles(p, s, pr);
            if (piece == 0 && lane == 0) w.record(p, c);
            // block ids of key tile j: lane l holds block j * bpt + l
            const int nblk = (s.L - 1) / bs + 1, first_blk = s.kv_lo / bs;
            auto entry_of = [&](int j) {  // (read before it is needed, checked when it is)
                const int lb = j * bpt + lane;
                return lane < bpt && lb >= first_blk && lb < nblk
                           ? a.block_table[static_cast<int64_t>(w.seq) * a.bt_stride + lb]
                           : a.num_blocks;  // one past the pool: the copy reads zeros
            };
            int next_id = entry_of(w.ja);
            bool ok = true;
            if (lane == 0) {
                // Q of the item, once the piece before has formed its last scores
                if (piece > 0) ok = mbar_wait_sleep(bar(kBarQEmpty), (piece - 1) & 1);
                if (ok) {
                    mbar_arrive_expect_tx(bar(kBarQFull), nt * q_bytes);
                    for (int x = 0; x < nt; ++x)
                        for (int hf = 0; hf < TL::kHalves; ++hf)
                            tma_load_3d(smem_u32(smem + x * kTileBytes + hf * kHalf), &tmap_q, bar(kBarQFull), 64 * hf,
                                        h * g, s.q0 + (2 * pr + x) * TQ);
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
                if (my_id < 0 || my_id > a.num_blocks || (my_id == a.num_blocks && j * bpt + lane < nblk && lane < bpt &&
                                                          j * bpt + lane >= first_blk)) {
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
                                        h * TL::kHalves, 0, id);
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
        constexpr uint32_t ab = AbFormat<T>::value;
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
                const Seq s = w.cur;
                const int nt = row_tiles(p, s, w.item % s.pairs);
                if (*abort_flag != 0) break;
                if (!mbar_wait_bounded(bar(kBarQFull), piece & 1)) {
                    dead = true;
                    break;
                }
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
                    if (!full(ev) || (mixed_tile(p, s, j) && !wait_at_least_bounded(&cleaned[sv], ev + 1)) ||
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
    } else if (warp == 11) {
        // ============================================================ cleaning of V tiles
        int base = 0;
        bool dead = false;
        for (int piece = 0; !dead && w.next(p); ++piece) {
            const Seq s = w.cur;
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
                if (!(e & 1) || !mixed_tile(p, s, j)) {
                    if (lane == 0) mbar_arrive(bar_empty(sv));
                    continue;
                }
                const uint32_t tile = smem_u32(smem + TL::kOffKV + sv * kTileBytes);
                const int k0 = j * kBN;
                bool odd = false;
                // keys no row sees: [block start, kv_lo) and [L, block end); keys some rows may not
                // see: [kv_lo, ctx + n - window) of the context, the drafted [ctx, L)
                auto clean = [&](int lo, int hi, bool zero) {
                    lo = max(lo, k0) - k0;
                    hi = min(hi, k0 + kBN) - k0;
                    if (lo >= hi) return;  // (either may lie far from the tile)
                    for (int i = lo * 8 + lane; i < hi * 8; i += 32)
                        for (int hf = 0; hf < TL::kHalves; ++hf)
                            clean_chunk<T>(tile + (i >> 6) * TL::kGroup + hf * 1024 + (i & 63) * 16, zero, odd);
                };
                if (a.window > 0) {
                    clean(s.kv_lo / bs * bs, s.kv_lo, true);
                    clean(s.kv_lo, min(s.ctx, s.ctx + s.n - a.window), false);
                }
                clean(s.ctx, s.L, false);
                clean(s.L, (s.L + bs - 1) / bs * bs, true);
                if (__any_sync(0xffffffffu, odd) && lane == 0) odd_flag[piece % kFlags] = 1;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
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
    } else {
        // ============================================================ softmax and results
        const int x = warp >> 2;                // chain
        const int r = threadIdx.x & 127;        // query row in the tile = TMEM lane
        const int tl = r / g, hh = r - tl * g;  // its token in the tile and head in the group
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t t_s = trow + x * 128, t_o = trow + kColO + x * 128;
        const float c2 = a.scale_log2;
        const float2 cc = make_float2(c2, c2);
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
            const int h = w.item / s.pairs, pr = w.item - h * s.pairs, nt = row_tiles(p, s, pr);
            const int t0 = (2 * pr + (nt == 2 ? x : 0)) * TQ;       // first token of the row tile
            const int nq = min(TQ, s.n - t0);                       // its tokens (the tile exists)
            const bool valid = tl < nq;
            const int64_t token = s.q0 + t0 + (valid ? tl : 0);
            uint64_t mask = 0;
            if (valid) mask = a.tree_mask[token] & (s.n >= 64 ? ~0ull : (1ull << s.n) - 1);
            const int pos = s.ctx - 1 + __popcll(mask);
            const int klo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
            const bool warp_valid = __any_sync(0xffffffffu, valid);
            float m_used = -INFINITY;  // the reference maximum of O and the sums, in log2 units
            float2 sum = make_float2(0.f, 0.f);  // sum of the weights
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
                    if (mixed_tile(p, s, j)) {
                        // (scale > 0: an unseen score of -inf gets weight 0.  Apart from the pass below, whose
                        // unrolled code the warps fetch anew each time: 38 trees of 256 rows took 348 us instead
                        // of 317 with the masks in it.)
#pragma unroll 1
                        for (int ch = 0; ch < 4; ++ch) {
                            uint32_t v[32];
                            tmem_ld32_async(t_s + 32 * ch, v);
                            tmem_wait_regs(v);
                            const uint32_t seen = valid ? seen32(j * kBN + ch * 32, s.ctx, klo, mask) : 0u;
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[k] = (seen >> k) & 1 ? v[k] : 0xff800000u;
                            tmem_st32u(t_s + 32 * ch, v);
                        }
                        tmem_wait_st();
                    }
                    float2 part_sum;
                    // One pass over the tile's S: weights against the reference in use, the tile maximum
                    // tracked alongside, 32 columns at a time with the next load in flight.  A second one
                    // when the reference has to move.  (One copy of the code: a CTA's first tile pays for
                    // fetching it.)
#pragma unroll 1
                    for (bool again = false;; again = true) {
                        const float nref = m_used == -INFINITY ? 0.f : kWeightLog2<T> - m_used;
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
                                wt[ch * 16 + k] = pack2<T>(x2.x, x2.y);
                                part_sum = add2(part_sum, x2);
                            }
                        }
                        if (again) break;
                        // scale > 0, so the scaled maximum is the maximum of the scaled scores
                        const float mt = mraw == -INFINITY ? -INFINITY : mraw * c2;
                        const bool moved = valid && mt > m_used + kRescaleLog2;  // also the first finite maximum
                        if (!__any_sync(0xffffffffu, moved)) break;
                        const bool rescale = moved && m_used != -INFINITY;  // O and the sums hold earlier tiles
                        const float f = moved ? fast_exp2(m_used - mt) : 1.f;
                        if (moved) {
                            m_used = mt;
                            sum.x *= f, sum.y *= f;
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
            bool use1 = false;
            if (nt == 1) {
                if (x == 1) {
                    // hand the maximum and sum to chain 0's thread of the same row, which joins the two
                    join[r] = m;
                    join[128 + r] = l;
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
                use1 = w.jb - w.ja > 1;
                m = mm;
                // (no guard: a chain whose scores are all NaN has no maximum, hence weight 0, and a sum of NaN,
                // which has to come through; an empty one has a sum of 0)
                l = l * f0 + l1 * f1;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            f0 *= inv;
            f1 *= inv;
            const int64_t row = token * a.num_q_heads + h * g + hh;
            T *out16 = static_cast<T *>(a.out) + row * D;
            const int prow = (nt == 2 ? x * 128 : 0) + r;
            const int64_t slot = part_slot(c, w.ja == s.j0);
            float4 *part = part_o<D>(p, slot, prow);
            T *rows[4];
            if (w.whole) quad_rows<T>(valid ? out16 : nullptr, rows);
            if (warp_valid) {
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    float o[32];
                    tmem_ld32(t_o + ch * 32, o);
                    tmem_wait_ld();
                    // a row of weight 0 in a chain has nothing there, whatever O holds
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = f0 != 0.f ? o[k] * f0 : 0.f;
                    if (use1) {
                        float o1[32];
                        tmem_ld32(trow + kColO + 128 + ch * 32, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] += f1 != 0.f ? o1[k] * f1 : 0.f;
                    }
                    if (w.whole) {
                        store_rows<T>(o, rows, ch * 32);
                    } else if (valid) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            part[static_cast<int64_t>(ch * 8 + k) * p.rows_per_item] =
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
                const float lse2 = l == 0.f ? -INFINITY : m + (log2f(l) - kWeightLog2<T>);
                if (!w.whole) *part_lse(p, slot, prow) = lse2;
                else if (a.lse_out) a.lse_out[row] = lse2 * 0.69314718055994531f;
                if (odd_flag[piece % kFlags])
                    add_odd_values<T, D>(p, w, h, klo, mask, out16, w.whole ? nullptr : part);
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

template <typename T, int D>
cudaError_t launch_typed(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                         int dev, cudaStream_t stream) {
    static std::atomic<bool> attr_set[64];
    return launch_tree_kernel<T, D>(tree_attention_kernel<T, D>, kThreads, Tile<D>::kSmem, attr_set, tq, tk, tv, p, dev,
                                    stream);
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

// Trees of up to 128 rows a kv head go by groups of heads (tree_packed.cu, which has the times of both);
// wider ones, and a single kv head, take the kernel of this file.  A single head, us here and as the first of
// two packed ones (whose boxes carry it alone, the other half zeros), 38 sequences of 8000 tokens and 304:
//   16/1 heads of 128 dims, 64 rows      47, 243   packed 53, 320   (blocks of 8: 59, 341 against 67, 435)
//   5/1 heads of 64 dims, 60 rows        43, 238   packed 42, 231   (blocks of 8: 58, 346 against 56, 335)
//                         125 rows       44, 238   packed 45, 235
// (64 dims are within 5 % either way, so that one rule serves both).
TreePlan plan_tree(int num_seqs, int max_query_len, int group, int num_kv_heads, int head_dim, int num_workers, int sm_count) {
    TreePlan t;
    const int rows = max_query_len * group;
    t.workers = num_workers > 0 ? num_workers : sm_count;
    t.heads_per_item = num_kv_heads == 1 || rows > kTreeRows ? 1 : 2;
    if (head_dim == 64 && num_kv_heads >= 3) {
        const int64_t items = static_cast<int64_t>(num_seqs) * ((num_kv_heads + 3) / 4);
        if (rows <= 32 || (rows <= 64 && 4 * items >= t.workers)) t.heads_per_item = 4;
    }
    if (t.heads_per_item > 1) {
        plan_tree_packed(t, rows, group, head_dim);
    } else {
        t.tokens_per_tile = kTreeRows / group;
        t.key_shift = 7;
        t.rows_per_item = max_query_len > t.tokens_per_tile ? 2 * kTreeRows : kTreeRows;
        t.smem_bytes = head_dim == 128 ? Tile<128>::kSmem : Tile<64>::kSmem;
    }
    const size_t parts = static_cast<size_t>(2) * t.workers * t.rows_per_item;
    t.lse_off = align256(2 * sizeof(int4) * static_cast<size_t>(t.workers));
    t.o_off = t.lse_off + align256(4 * parts);
    t.workspace_bytes = t.o_off + 4 * parts * head_dim;
    return t;
}

cudaError_t launch_tree_attention(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                  const TreeArgs &a, const TreePlan &plan, void *workspace, int head_dim, int q_dtype,
                                  int dev, cudaStream_t stream) {
    TreeParams p;
    p.a = a;
    p.group = a.num_q_heads / a.num_kv_heads;
    p.tokens_per_tile = plan.tokens_per_tile;
    p.heads_per_item = plan.heads_per_item;
    p.key_shift = plan.key_shift;
    p.workers = plan.workers;
    p.rows_per_item = plan.rows_per_item;
    const int row_tiles = (a.max_query_len + p.tokens_per_tile - 1) / p.tokens_per_tile;
    p.items_per_seq = p.heads_per_item == 1 ? (row_tiles + 1) / 2 * a.num_kv_heads
                                            : (a.num_kv_heads + p.heads_per_item - 1) / p.heads_per_item;
    char *ws = static_cast<char *>(workspace);
    p.ws_first = reinterpret_cast<int4 *>(ws);
    p.ws_lse = reinterpret_cast<float *>(ws + plan.lse_off);
    p.ws_o = reinterpret_cast<float4 *>(ws + plan.o_off);
    if (p.heads_per_item > 1) return launch_tree_packed(tq, tk, tv, p, head_dim, q_dtype, dev, stream);
    if (q_dtype == KV_BF16)
        return head_dim == 128 ? launch_typed<__nv_bfloat16, 128>(tq, tk, tv, p, dev, stream)
                               : launch_typed<__nv_bfloat16, 64>(tq, tk, tv, p, dev, stream);
    return head_dim == 128 ? launch_typed<__half, 128>(tq, tk, tv, p, dev, stream)
                           : launch_typed<__half, 64>(tq, tk, tv, p, dev, stream);
}

}  // namespace pkv
