// RMS norm of every query and key head, rotary embedding, and the write of K and V into the paged
// cache, in one pass over a step's projections ("vLLM의 KV cache 연결 흐름", section "Slot
// mapping은 왜 필요한가": the new tokens' K/V go to their slots; the norm and the rotation that
// come before it are in no section of the pages).
//
// Per head of D dims:  y = x * w / sqrt(mean(x^2) + eps),  then pairs turn by the token's angles.
// A lane holds 8 elements of a head as two pieces of 4, chosen so that both halves of its pairs
// are its own: dims 4c .. and rotary_dim / 2 + 4c .. of the turning part, 8c .. and 8c + 4 .. of the
// rest (and everywhere when pairs are adjacent).  D / 8 lanes make a head, rounded up to a power of
// two; the squares are summed over them by shuffles.  A lane's cos and sin (4 pairs) and weights stay
// in registers for all heads that its warp takes of a token.
//
// About 2 bytes move per element each way and some 5 instructions are spent on it: the bound is
// HBM.  A warp takes several heads, all loaded before the first is used, once there are
// tokens enough to fill the GPU; fewer heads a warp below that (see heads_a_warp).
#include "common.cuh"
#include "kernels.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // loads in flight a lane

// Four 16-bit elements (one piece) to float32 and back.
template <typename T> __device__ __forceinline__ void widen4(uint2 raw, float *x) {
    const float2 a = unpack2<T>(raw.x), b = unpack2<T>(raw.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
template <typename T> __device__ __forceinline__ uint2 narrow4(const float *x) {
    return make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
}

// Four float32 values -> four E4M3 bytes of x / scale (correctly rounded division, round to nearest
// even, saturating).
__device__ __forceinline__ uint32_t quantise4(const float *x, float scale) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)),
                                                 __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ uint2 ld_piece(const void *p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

// LP lanes a head; a warp takes 32 / LP heads at a time, of one token.  An output may be its
// input: a piece is read and then written by one lane, and no other lane touches it.
template <typename T, int LP, bool kAdjacent>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int HPW = 32 / LP;
    const int lane = threadIdx.x & 31;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int64_t t = w / a.parts;
    const int part = static_cast<int>(w - t * a.parts);
    if (t >= a.num_tokens) return;
    const int32_t pos = a.positions ? a.positions[t] : 0;
    int64_t slot = a.slot_mapping ? a.slot_mapping[t] : -1;
    const int c = lane & (LP - 1);
    const bool has = 8 * c < a.head_dim;
    const int half = a.rotary_dim >> 1;
    const bool turns = 8 * c < a.rotary_dim;
    const int d0 = kAdjacent || !turns ? 8 * c : 4 * c;   // the two pieces
    const int d1 = kAdjacent || !turns ? 8 * c + 4 : half + 4 * c;
    const int heads = a.num_q_heads + a.num_kv_heads * (a.slot_mapping ? 2 : 1);
    const int first = part * a.heads_a_warp, last = min(heads, first + a.heads_a_warp);

    auto source = [&](int hd) -> const T * {
        if (hd < a.num_q_heads) return static_cast<const T *>(a.q) + t * a.q_stride + static_cast<int64_t>(hd) * a.head_dim;
        hd -= a.num_q_heads;
        if (hd < a.num_kv_heads)
            return static_cast<const T *>(a.key) + t * a.key_stride + static_cast<int64_t>(hd) * a.head_dim;
        return static_cast<const T *>(a.value) + t * a.value_stride + static_cast<int64_t>(hd - a.num_kv_heads) * a.head_dim;
    };
    uint2 raw[kBatch][2];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int hd = h0 + i * HPW + lane / LP;
            raw[i][0] = raw[i][1] = make_uint2(0, 0);
            if (has && hd < last) {
                const T *src = source(hd);
                raw[i][0] = ld_piece(src + d0);
                raw[i][1] = ld_piece(src + d1);
            }
        }
    };
    load(first);  // needs no position: on the way while the token's position, angles and weights come

    if (pos < 0) return;
    if (a.rotary_dim > 0 && pos >= a.max_position) {
        if (part == 0 && lane == 0) report(a.d_err, KV_DERR_BAD_POS);
        return;
    }
    if (slot >= a.total_slots) {
        if (a.slot_mapping && part == 0 && lane == 0) report(a.d_err, KV_DERR_BAD_SLOT);
        slot = -1;
    }
    float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turns) {
        const float *row = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim + 4 * c;
        cs = __ldg(reinterpret_cast<const float4 *>(row));
        sn = __ldg(reinterpret_cast<const float4 *>(row + half));
    }
    uint2 wq[2] = {}, wk[2] = {};
    if (has && a.q_weight) {
        wq[0] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const T *>(a.q_weight) + d0));
        wq[1] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const T *>(a.q_weight) + d1));
    }
    if (has && a.k_weight) {
        wk[0] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const T *>(a.k_weight) + d0));
        wk[1] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const T *>(a.k_weight) + d1));
    }
    const float inv_d = 1.f / static_cast<float>(a.head_dim);
    for (int h0 = first; h0 < last; h0 += kBatch * HPW) {
        if (h0 > first) load(h0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (h0 + i * HPW >= last) break;  // the same for the warp
            int h = h0 + i * HPW + lane / LP;
            const bool in = has && h < last;
            int kind = 0;  // q, key, value
            if (h >= a.num_q_heads) kind = 1, h -= a.num_q_heads;
            if (kind && h >= a.num_kv_heads) kind = 2, h -= a.num_kv_heads;
            float x[8];
            widen4<T>(raw[i][0], x);
            widen4<T>(raw[i][1], x + 4);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = LP / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!in) continue;
            const int64_t at = (slot * a.num_kv_heads + h) * a.head_dim;  // in the caches, once slot >= 0
            if (kind == 2) {
                if (slot < 0) continue;
                if (a.cache_fp8) {
                    uint8_t *dst = static_cast<uint8_t *>(a.v_cache) + at;
                    *reinterpret_cast<uint32_t *>(dst + d0) = quantise4(x, a.v_scale);
                    *reinterpret_cast<uint32_t *>(dst + d1) = quantise4(x + 4, a.v_scale);
                } else {
                    T *dst = static_cast<T *>(a.v_cache) + at;
                    *reinterpret_cast<uint2 *>(dst + d0) = raw[i][0];
                    *reinterpret_cast<uint2 *>(dst + d1) = raw[i][1];
                }
                continue;
            }
            if (kind == 0 ? a.q_weight != nullptr : a.k_weight != nullptr) {
                const float rs = rsqrtf(fmaf(ss, inv_d, a.eps));
                float wt[8];
                widen4<T>(kind == 0 ? wq[0] : wk[0], wt);
                widen4<T>(kind == 0 ? wq[1] : wk[1], wt + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= rs * wt[e];
            }
            if (turns) {
                const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, sc[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float &p = kAdjacent ? x[2 * e] : x[e], &q = kAdjacent ? x[2 * e + 1] : x[4 + e];
                    const float u = fmaf(-q, sc[e], p * cc[e]), v = fmaf(p, sc[e], q * cc[e]);
                    p = u;
                    q = v;
                }
            }
            const uint2 r0 = narrow4<T>(x), r1 = narrow4<T>(x + 4);
            const int64_t off = static_cast<int64_t>(h) * a.head_dim;
            auto store = [&](T *dst) {
                *reinterpret_cast<uint2 *>(dst + d0) = r0;
                *reinterpret_cast<uint2 *>(dst + d1) = r1;
            };
            if (kind == 0) {
                store(static_cast<T *>(a.q_out) + t * a.q_out_stride + off);
                continue;
            }
            if (a.k_out) store(static_cast<T *>(a.k_out) + t * a.k_out_stride + off);
            if (slot < 0) continue;
            if (a.cache_fp8) {
                uint8_t *dst = static_cast<uint8_t *>(a.k_cache) + at;
                *reinterpret_cast<uint32_t *>(dst + d0) = quantise4(x, a.k_scale);
                *reinterpret_cast<uint32_t *>(dst + d1) = quantise4(x + 4, a.k_scale);
            } else {
                store(static_cast<T *>(a.k_cache) + at);
            }
        }
    }
}

template <typename T, int LP>
cudaError_t launch_lanes(RopeArgs a, int sm_count, cudaStream_t stream) {
    constexpr int HPW = 32 / LP;
    const int heads = a.num_q_heads + a.num_kv_heads * (a.slot_mapping ? 2 : 1);
    // heads a warp: as many as leave each SM 32 warps (what a lane reads ahead, times 32 warps, covers
    // the memory's latency), between one load and four batches of them
    int n = 4 * kBatch;
    while (n > 1 && static_cast<int64_t>(a.num_tokens) * ((heads + n * HPW - 1) / (n * HPW)) < 32ll * sm_count) n /= 2;
    a.heads_a_warp = n * HPW;
    a.parts = (heads + a.heads_a_warp - 1) / a.heads_a_warp;
    const int64_t blocks = (static_cast<int64_t>(a.num_tokens) * a.parts + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(blocks);
    if (a.interleaved) qk_norm_rope_kernel<T, LP, true><<<grid, kThreads, 0, stream>>>(a);
    else qk_norm_rope_kernel<T, LP, false><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_typed(const RopeArgs &a, int sm_count, cudaStream_t stream) {
    const int chunks = a.head_dim / 8;
    if (chunks <= 2) return launch_lanes<T, 2>(a, sm_count, stream);
    if (chunks <= 4) return launch_lanes<T, 4>(a, sm_count, stream);
    if (chunks <= 8) return launch_lanes<T, 8>(a, sm_count, stream);
    if (chunks <= 16) return launch_lanes<T, 16>(a, sm_count, stream);
    return launch_lanes<T, 32>(a, sm_count, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs &a, int dtype, int sm_count, cudaStream_t stream) {
    if (dtype == KV_BF16) return launch_typed<__nv_bfloat16>(a, sm_count, stream);
    return launch_typed<__half>(a, sm_count, stream);
}

}  // namespace pkv
