// Tree attention, two or four kv heads of a sequence at a time.
//
// Reading the cache bounds small trees, and one head at a time cannot read it fast enough: a TMA box of 2 KB
// (16 tokens of 64 dims of one head) costs about 130 clocks plus two a row, 13 bytes a clock and SM, where
// HBM gives 23; a box of 4 KB moves 21, one of 8 KB 32.  So a box takes all dims of a block of several
// heads.  The tensor map splits tokens into groups of 8 and heads into parts of 64 dims, and a box lands as
// [group of 8 tokens][head][part][token][64 dims]: the swizzle atoms of one part of one head lie a constant
// distance apart over all blocks of a key tile, which is what a matrix descriptor can say.  (A box a part
// took 3 % longer on the Mistral-shaped window layer, 8 % on 38 sequences of 8000 tokens and 64 rows.)
//
// Two heads of up to 64 rows share the 128 TMEM lanes of a row tile, those of up to 128 rows have one each.
// Heads of 64 dims go by four, in one row tile (up to 32 rows) or two (up to 64, when the batch gives the
// workers items enough).  us for 38 sequences of 8000 tokens, and for 152 of 1000:
//   32/8 heads of 128 dims, 28 rows    two heads 200, 117   one 239, 168
//                           64 rows    two 201, 121         one 239, 169
//                           128 rows   two 225, 151         one 240, 202
//   12/12 heads of 64 dims, 24 rows    four 159, 90         two 182, 104   one 346, 201
//                           64 rows    four 167, 105        two 186, 118   (one sequence of 1117: 18.5, two 15.0)
// Four heads of 128 dims and up to 32 rows (16 KB a box) took as long as two on long contexts, 112 us instead of
// 122 on the 152 of 1000, and 69 instead of 62 on 38 of 2000, 30 instead of 26 on 38 of 500: they go by two.
// Above 128 rows two row tiles of one head are faster than two heads (405 against 505 us at 256 rows when both
// were tried, 317 now): tree_attention.cu.
//
// Per key tile and head h (64 keys, or 128 of two heads of 64 dims: 32 KB of K and of V; with 128 keys
// of two heads of 128 dims the ring has three entries instead of six, and the window layer took 235 us
// instead of 208; with 64 of two heads of 64 dims 64 rows took 255 instead of 216):
//   S_h = Q K_h^T    all 128 rows, of which the lanes of head h are read
//   P_h = exp2(S_h * scale - m)    one thread a row; P_h has TMEM columns of its own
//   O  += P_h V_h    for the lanes of head h alone (the other lanes are switched off), so that
//                    heads that share a row tile share the columns of O
// S_h is free as soon as the softmax has read it, so the next tile's scores are formed before
// O += P_h V_h when its keys are there, and after it when they are not.
// For the work list, the masks, cleaned V tiles and bounded waits see tree_attention.cu.
//
// Warps: 0 .. softmax, four a row tile (thread = TMEM lane = query row), then a TMA producer, one that
// cleans V tiles, and one a head (of it one lane) that issues the MMAs: a commit takes the issuing
// thread some 120 clocks and a wait about as much, so that one warp for all heads was the bound (6,400
// clocks a key tile of 4 heads and 64 dims, of which 2,050 on the tensor cores).
#include "tree_common.cuh"

namespace pkv {
namespace {

// PH heads in MT row tiles.
template <int D, int PH, int MT> struct Pack {
    static constexpr int kHalves = D / 64;
    static constexpr int kKeys = PH == 4 || D == 128 ? 64 : 128;  // keys of a key tile
    static constexpr int kLanes = MT * kTreeRows / PH;       // lanes of a head
    static constexpr int kColP = PH * kKeys;                 // TMEM: S, P, O
    static constexpr int kColO = kColP + PH * kKeys / 2;
    static_assert(kColO + MT * D <= static_cast<int>(kTmemCols), "TMEM columns");
    static constexpr int kSoftmax = 4 * MT;                  // warps
    static constexpr int kThreads = (kSoftmax + 2 + PH) * 32;
    static constexpr int kQBytes = kHalves * kHalf;          // Q of a row tile
    static constexpr int kGroup = PH * kHalves * 1024;       // 8 keys: [head][64 dims of D][key][dim]
    static constexpr int kEntry = kKeys / 8 * kGroup;        // a key tile
    static constexpr int kOffKV = MT * kQBytes;
    static constexpr int kFit = (224 * 1024 - kOffKV) / kEntry;  // ring entries, 160 or 192 KB
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kOffBar = kOffKV + kStages * kEntry;
    static constexpr int kNumBars = 2 + 4 * PH + 2 * kStages;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // TMEM address, abort flag, flags, cleaned
    static constexpr int kSmem = kOffMisc + 8 + 4 * kFlags + 4 * kStages + 1024;  // + alignment
    static_assert(kSmem + 512 <= 227 * 1024, "shared memory, with the kernel's static part");
    static_assert(kFlags >= (kStages + 1) / 2 + 2, "a flag per piece in flight");
};

template <typename T, int D, int PH, int MT>
__global__ void __launch_bounds__((4 * MT + 2 + PH) * 32, 1)
tree_packed_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ TreeParams p) {
    using PK = Pack<D, PH, MT>;
    constexpr int kStages = PK::kStages, kKeys = PK::kKeys, kLanes = PK::kLanes;
    constexpr int kPerTile = PH / MT;  // heads of a row tile
    constexpr int kProducer = PK::kSoftmax, kCleaner = kProducer + 1, kIssuer = kCleaner + 1;  // warps
    constexpr int kBarQFull = 0, kBarQEmpty = 1, kBarS = 2, kBarP = kBarS + PH, kBarPd = kBarP + PH,
                  kBarDrain = kBarPd + PH, kBarFull = kBarDrain + PH, kBarEmpty = kBarFull + kStages;
    const TreeArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = p.group, TQ = p.tokens_per_tile, bs = a.block_size;
    const int c = blockIdx.x;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + PK::kOffBar);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + PK::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + PK::kOffMisc + 4);
    volatile int *odd_flag = reinterpret_cast<volatile int *>(smem + PK::kOffMisc + 8);  // [kFlags], per piece
    int32_t *cleaned = reinterpret_cast<int32_t *>(smem + PK::kOffMisc + 8 + 4 * kFlags);  // [kStages]: entry + 1
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    if (threadIdx.x == 32) {
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    if (threadIdx.x == 0) {
        mbar_init(bar(kBarQFull), 1);
        mbar_init(bar(kBarQEmpty), PH);
        for (int h = 0; h < PH; ++h) {
            mbar_init(bar(kBarS + h), 1);
            mbar_init(bar(kBarP + h), kLanes);
            mbar_init(bar(kBarPd + h), 1);
            mbar_init(bar(kBarDrain + h), 1);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(kBarFull + s), 1);
            mbar_init(bar(kBarEmpty + s), PH + 1);  // released by the MMA warps and the cleaning warp
        }
        *abort_flag = 0;
        for (int i = 0; i < kFlags; ++i) odd_flag[i] = 0;
        for (int i = 0; i < kStages; ++i) cleaned[i] = 0;
        fence_barrier_init();
    }
    if (warp == kCleaner) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __shared__ ShareScratch scratch;
    int64_t x0, x1;
    int item_cost;
    previous_kernel_done();
    let_next_kernel_launch();
    share_of_cta<PK::kThreads>(p, c, x0, x1, item_cost, scratch);
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
    } else if (warp == kProducer) {
        // ============================================================ TMA producer
        const int bpt = kKeys / bs;  // blocks of a key tile
        const uint32_t q_bytes = static_cast<uint32_t>(PH * PK::kHalves) * TQ * g * 128;
        int entry = 0;  // ring entries filled
        int piece = 0;
        bool stop = false;
        while (!stop && w.next(p)) {
            const Seq s = w.cur;
            const int h0 = w.item * PH;
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
                // Q of the item (heads past the last read zeros), once the piece before has formed
                // its last scores
                if (piece > 0) ok = mbar_wait_sleep(bar(kBarQEmpty), (piece - 1) & 1);
                if (ok) {
                    mbar_arrive_expect_tx(bar(kBarQFull), q_bytes);
                    for (int h = 0; h < PH; ++h)
                        for (int hf = 0; hf < PK::kHalves; ++hf)
                            tma_load_3d(smem_u32(smem + h / kPerTile * PK::kQBytes + hf * kHalf + h % kPerTile * kLanes * 128),
                                        &tmap_q, bar(kBarQFull), 64 * hf, (h0 + h) * g, s.q0);
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
                        if (entry >= kStages && !mbar_wait_sleep(bar(kBarEmpty + slot), (entry / kStages - 1) & 1)) {
                            quit = 1;
                            report(a.d_err, KV_DERR_TIMEOUT);
                            *abort_flag = 1;
                        } else if (*abort_flag) {
                            quit = 1;
                        }
                        if (!quit) mbar_arrive_expect_tx(bar(kBarFull + slot), PK::kEntry);
                    }
                    if (__shfl_sync(0xffffffffu, quit, 0)) {
                        stop = true;
                        break;
                    }
                    const CUtensorMap *m = is_v ? &tmap_v : &tmap_k;
                    uint8_t *dst = smem + PK::kOffKV + slot * PK::kEntry;
                    for (int jb = 0; jb < bpt; ++jb) {
                        const int id = __shfl_sync(0xffffffffu, my_id, jb);
                        if (lane == 0)
                            tma_load_5d(smem_u32(dst + bs / 8 * jb * PK::kGroup), m, bar(kBarFull + slot), 0, 0,
                                        h0 * PK::kHalves, 0, id);
                    }
                    ++entry;
                }
            }
        }
        // never leave with copies in flight into this CTA's shared memory
        if (lane == 0) {
            if (piece > 0 && !mbar_wait_sleep(bar(kBarQFull), (piece - 1) & 1)) report(a.d_err, KV_DERR_TIMEOUT);
            for (int i = max(0, entry - kStages); i < entry; ++i)
                if (!mbar_wait_sleep(bar(kBarFull + i % kStages), (i / kStages) & 1)) report(a.d_err, KV_DERR_TIMEOUT);
        }
    } else if (warp >= kIssuer) {
        // ============================================================ MMA issue, one lane a head
        const int h = warp - kIssuer;
        constexpr uint32_t ab = AbFormat<T>::value;
        constexpr uint32_t idesc_s = mma_idesc(ab, false, kTreeRows, kKeys);
        constexpr uint32_t idesc_pv = mma_idesc(ab, true, kTreeRows, D);
        if (lane == 0) {
            const uint64_t dq = smem_desc(smem_u32(smem + h / kPerTile * PK::kQBytes), 16, 1024);
            // a head's swizzle atoms (8 keys x 64 dims, 1 KB): those of the next keys are kGroup bytes on
            const uint32_t kv = smem_u32(smem + PK::kOffKV) + h * PK::kHalves * 1024;
            const uint64_t dk0 = smem_desc(kv, 16, PK::kGroup);
            const uint64_t dv0 = smem_desc(kv, 1024, PK::kGroup);
            const uint32_t t_s = tmem + h * kKeys, t_p = tmem + PK::kColP + h * (kKeys / 2);
            const uint32_t t_o = tmem + PK::kColO + h / kPerTile * D;
            uint32_t off[4];  // the other heads' lanes
#pragma unroll
            for (int i = 0; i < 4; ++i) off[i] = i * 32 / kLanes == h % kPerTile ? 0u : 0xffffffffu;
            // scores against the keys in ring entry e
            auto scores = [&](int e) {
                const int sk = e % kStages;
                const uint64_t dk = dk0 + static_cast<uint64_t>((sk * PK::kEntry) >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_f16(t_s, dq + (((k >> 2) * kHalf + (k & 3) * 32) >> 4),
                            dk + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), idesc_s, k > 0);
                mma_commit(bar(kBarS + h));
                mma_commit(bar(kBarEmpty + sk));
            };
            auto full = [&](int e) { return mbar_wait_bounded(bar(kBarFull + e % kStages), (e / kStages) & 1); };
            int done = 0;  // key tiles of the pieces before
            bool dead = false;
            for (int piece = 0; !dead && w.next(p); ++piece) {
                const Seq s = w.cur;
                if (*abort_flag != 0) break;
                if (!mbar_wait_bounded(bar(kBarQFull), piece & 1) || !full(2 * done)) {
                    dead = true;
                    break;
                }
                tc_fence_after();
                const int n = w.jb - w.ja;
                scores(2 * done);
                for (int t = 0; t < n; ++t, ++done) {
                    const int ev = 2 * done + 1, sv = ev % kStages, ek = ev + 1;
                    const bool more = t + 1 < n;
                    if (!more) mma_commit(bar(kBarQEmpty));  // the piece's last scores have been issued
                    if (!full(ev) ||
                        (mixed_tile(p, s, w.ja + t) && !wait_at_least_bounded(&cleaned[sv], ev + 1)) ||
                        !mbar_wait_bounded(bar(kBarP + h), done & 1)) {
                        dead = true;
                        break;
                    }
                    const bool keys = more && mbar_test(bar(kBarFull + ek % kStages), (ek / kStages) & 1);
                    tc_fence_after();
                    if (keys) scores(ek);
                    const uint64_t dv = dv0 + static_cast<uint64_t>((sv * PK::kEntry) >> 4);
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k) {
                        const uint64_t db = dv + ((k * 2 * PK::kGroup) >> 4);
                        if constexpr (kPerTile == 1) mma_f16_ts(t_o, t_p + k * 8, db, idesc_pv, t > 0 || k > 0);
                        else mma_f16_ts_rows(t_o, t_p + k * 8, db, idesc_pv, t > 0 || k > 0, off);
                    }
                    mma_commit(bar(kBarPd + h));
                    mma_commit(bar(kBarEmpty + sv));
                    if (more && !keys) {
                        if (!full(ek)) {
                            dead = true;
                            break;
                        }
                        tc_fence_after();
                        scores(ek);
                    }
                }
            }
            if (dead) {
                report(a.d_err, KV_DERR_TIMEOUT);
                *abort_flag = 1;
            }
            // every MMA this lane issued has completed before TMEM is freed
            mma_commit(bar(kBarDrain + h));
            if (!mbar_wait_bounded(bar(kBarDrain + h), 0)) report(a.d_err, KV_DERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kCleaner) {
        // ============================================================ cleaning of V tiles
        int done = 0;
        bool dead = false;
        for (int piece = 0; !dead && w.next(p); ++piece) {
            const Seq s = w.cur;
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
            if (lane == 0) odd_flag[piece % kFlags] = 0;
            __syncwarp();
            for (int e = 0; e < 2 * (w.jb - w.ja); ++e) {
                const int j = w.ja + (e >> 1);
                const int ev = 2 * done + e, sv = ev % kStages;
                if (!__all_sync(0xffffffffu, mbar_wait_sleep(bar(kBarFull + sv), (ev / kStages) & 1))) {
                    dead = true;
                    break;
                }
                if (!(e & 1) || !mixed_tile(p, s, j)) {
                    if (lane == 0) mbar_arrive(bar(kBarEmpty + sv));
                    continue;
                }
                const uint32_t tile = smem_u32(smem + PK::kOffKV + sv * PK::kEntry);
                const int k0 = j * kKeys;
                bool odd = false;
                // keys no row sees: [block start, kv_lo) and [L, block end); keys some rows may not
                // see: [kv_lo, ctx + n - window) of the context, the drafted [ctx, L)
                auto clean = [&](int lo, int hi, bool zero) {
                    lo = max(lo, k0) - k0;
                    hi = min(hi, k0 + kKeys) - k0;
                    if (lo >= hi) return;  // (either may lie far from the tile)
                    // 16-byte chunks: 8 of a key's 64 dims, of every head and side
                    for (int i = lo * 8 + lane; i < hi * 8; i += 32) {
                        const int key = i >> 3;
                        const uint32_t at0 = tile + (key >> 3) * PK::kGroup + (key & 7) * 128 + (i & 7) * 16;
                        for (int u = 0; u < PH * PK::kHalves; ++u) clean_chunk<T>(at0 + u * 1024, zero, odd);
                    }
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
                    mbar_arrive(bar(kBarEmpty + sv));
                }
                __syncwarp();
            }
            done += w.jb - w.ja;
        }
        if (dead && lane == 0) {
            report(a.d_err, KV_DERR_TIMEOUT);
            *abort_flag = 1;
        }
    } else {
        // ============================================================ softmax and results
        const int r = threadIdx.x;                       // query row (128 a row tile) = TMEM lane
        const int hi = r / kLanes, rr = r % kLanes;      // head of the item (one a warp), row of it
        const int tl = rr / g, hh = rr - tl * g;         // token, head of the group
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t t_s = trow + hi * kKeys, t_p = trow + PK::kColP + hi * (kKeys / 2);
        const uint32_t t_o = trow + PK::kColO + hi / kPerTile * D;
        const float c2 = a.scale_log2;
        const float2 cc = make_float2(c2, c2);
        bool dead = false;
        // waits are decided for the whole warp: its lanes take the warp-collective TMEM
        // loads and stores together
        auto wait_all = [&](uint32_t b, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait_sleep(b, parity));
        };
        int done = 0, pd = 0;  // key tiles taken; of those, products O known to have completed
        auto settled = [&] {   // O and P_h are free: the products of all tiles taken have completed
            while (pd < done)
                if (!wait_all(bar(kBarPd + hi), pd++ & 1)) return false;
            tc_fence_after();
            return true;
        };
        for (int piece = 0; !dead && w.next(p); ++piece) {
            const Seq s = w.cur;
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
            const int h = w.item * PH + hi;
            const bool valid = tl < s.n && h < a.num_kv_heads;
            const int64_t token = s.q0 + (valid ? tl : 0);
            uint64_t mask = 0;
            if (valid) mask = a.tree_mask[token] & (s.n >= 64 ? ~0ull : (1ull << s.n) - 1);
            const int pos = s.ctx - 1 + __popcll(mask);
            const int klo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
            const bool warp_valid = __any_sync(0xffffffffu, valid);
            float m_used = -INFINITY;  // the reference maximum of O and the sums, in log2 units
            float2 sum = make_float2(0.f, 0.f);  // sum of the weights
            uint32_t wt[kKeys / 2];
            for (int j = w.ja; j < w.jb; ++j) {
                if (!wait_all(bar(kBarS + hi), done & 1)) {
                    dead = true;
                    break;
                }
                tc_fence_after();
                if (warp_valid) {
                    if (mixed_tile(p, s, j)) {
                        // (scale > 0: an unseen score of -inf gets weight 0.  Apart from the pass below, whose
                        // unrolled code the warps fetch anew each time: 128 rows 225 us instead of 233.)
#pragma unroll 1
                        for (int ch = 0; ch < kKeys / 32; ++ch) {
                            uint32_t v[32];
                            tmem_ld32_async(t_s + 32 * ch, v);
                            tmem_wait_regs(v);
                            const uint32_t seen = valid ? seen32(j * kKeys + ch * 32, s.ctx, klo, mask) : 0u;
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
                        for (int ch = 0; ch < kKeys / 32; ++ch) {
                            uint32_t(&v)[32] = buf[ch & 1];
                            tmem_wait_regs(v);
                            if (ch + 1 < kKeys / 32) tmem_ld32_async(t_s + 32 * (ch + 1), buf[(ch + 1) & 1]);
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float s0 = __uint_as_float(v[2 * k]), s1 = __uint_as_float(v[2 * k + 1]);
                                const float2 e = fma2(make_float2(s0, s1), cc, ref2);
                                const float2 x = make_float2(fast_exp2(e.x), fast_exp2(e.y));
                                mraw = fmaxf(mraw, fmaxf(s0, s1));
                                wt[ch * 16 + k] = pack2<T>(x.x, x.y);
                                part_sum = add2(part_sum, x);
                            }
                        }
                        if (again) break;
                        // scale > 0, so the scaled maximum is the maximum of the scaled scores
                        const float mt = mraw == -INFINITY ? -INFINITY : mraw * c2;
                        const bool moved = valid && mt > m_used + kRescaleLog2;  // also the first finite maximum
                        const bool any_moved = __any_sync(0xffffffffu, moved);
                        if (!settled()) {
                            dead = true;
                            break;
                        }
                        if (!any_moved) break;
                        const bool rescale = moved && m_used != -INFINITY;  // O and the sums hold earlier tiles
                        const float f = moved ? fast_exp2(m_used - mt) : 1.f;
                        if (moved) {
                            m_used = mt;
                            sum.x *= f, sum.y *= f;
                        }
                        if (__any_sync(0xffffffffu, rescale)) {
                            // the warp loads and stores its lanes of O together; rows that keep their
                            // maximum scale by 1
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
                    if (dead) break;
                    sum = add2(sum, part_sum);
                    tmem_st32u(t_p, wt);
                    if constexpr (kKeys == 128) tmem_st32u(t_p + 32, wt + 32);
                    tmem_wait_st();
                } else if (!settled()) {  // a warp without rows passes every phase all the same
                    dead = true;
                    break;
                }
                tc_fence_before();
                mbar_arrive(bar(kBarP + hi));
                ++done;
            }
            if (dead) break;
            if (!settled()) {
                dead = true;
                break;
            }
            if (!warp_valid) continue;
            const float l = sum.x + sum.y;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int64_t row = token * a.num_q_heads + h * g + hh;
            T *out16 = static_cast<T *>(a.out) + row * D;
            const int64_t slot = part_slot(c, w.ja == s.j0);
            float4 *part = part_o<D>(p, slot, r);
            T *rows[4];
            if (w.whole) quad_rows<T>(valid ? out16 : nullptr, rows);
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
                float o[32];
                tmem_ld32(t_o + ch * 32, o);
                tmem_wait_ld();
                // a row that saw nothing is 0
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = inv != 0.f ? o[k] * inv : 0.f;
                if (w.whole) {
                    store_rows<T>(o, rows, ch * 32);
                } else if (valid) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        part[static_cast<int64_t>(ch * 8 + k) * p.rows_per_item] =
                            make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            }
            __syncwarp();  // (a row is written by the lanes of its quad)
            if (valid) {
                const float lse2 = l == 0.f ? -INFINITY : m_used + (log2f(l) - kWeightLog2<T>);
                if (!w.whole) *part_lse(p, slot, r) = lse2;
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
    if (warp == kCleaner)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

template <typename T, int D, int PH, int MT>
cudaError_t launch_heads(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                         int dev, cudaStream_t stream) {
    static std::atomic<bool> attr_set[64];
    return launch_tree_kernel<T, D>(tree_packed_kernel<T, D, PH, MT>, Pack<D, PH, MT>::kThreads, Pack<D, PH, MT>::kSmem,
                                    attr_set, tq, tk, tv, p, dev, stream);
}

template <typename T, int D>
cudaError_t launch_typed(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                         int dev, cudaStream_t stream) {
    if constexpr (D == 64)
        if (p.heads_per_item == 4)
            return p.rows_per_item == kTreeRows ? launch_heads<T, D, 4, 1>(tq, tk, tv, p, dev, stream)
                                                : launch_heads<T, D, 4, 2>(tq, tk, tv, p, dev, stream);
    return p.rows_per_item == kTreeRows ? launch_heads<T, D, 2, 1>(tq, tk, tv, p, dev, stream)
                                        : launch_heads<T, D, 2, 2>(tq, tk, tv, p, dev, stream);
}

template <typename PK> void set_plan(TreePlan &t, int group) {
    t.rows_per_item = PK::kSoftmax * 32;
    t.tokens_per_tile = PK::kLanes / group;
    t.key_shift = PK::kKeys == 64 ? 6 : 7;
    t.smem_bytes = PK::kSmem;
}

template <int D> void plan_heads(TreePlan &t, int rows, int group) {
    if constexpr (D == 64)
        if (t.heads_per_item == 4) return rows <= 32 ? set_plan<Pack<D, 4, 1>>(t, group) : set_plan<Pack<D, 4, 2>>(t, group);
    if (rows <= 64) set_plan<Pack<D, 2, 1>>(t, group);
    else set_plan<Pack<D, 2, 2>>(t, group);
}

}  // namespace

void plan_tree_packed(TreePlan &t, int rows, int group, int head_dim) {
    if (head_dim == 128) plan_heads<128>(t, rows, group);
    else plan_heads<64>(t, rows, group);
}

cudaError_t launch_tree_packed(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                               int head_dim, int q_dtype, int dev, cudaStream_t stream) {
    if (q_dtype == KV_BF16)
        return head_dim == 128 ? launch_typed<__nv_bfloat16, 128>(tq, tk, tv, p, dev, stream)
                               : launch_typed<__nv_bfloat16, 64>(tq, tk, tv, p, dev, stream);
    return head_dim == 128 ? launch_typed<__half, 128>(tq, tk, tv, p, dev, stream)
                           : launch_typed<__half, 64>(tq, tk, tv, p, dev, stream);
}

}  // namespace pkv
