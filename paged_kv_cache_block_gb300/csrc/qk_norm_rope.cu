// RMS norm of every query and key head, rotary embedding, and the write of K and V into the paged
// cache, in one pass over a step's projections ("vLLM의 KV cache 연결 흐름", section "Slot
// mapping은 왜 필요한가": the new tokens' K/V go to their slots; the norm and the rotation that
// come before it are in no section of the pages).
//
// Per head of D dims:  y = x * w / sqrt(mean(x^2) + eps),  then pairs turn by the token's angles.
// A lane holds 8 elements of a head as two pieces of 4, chosen so that both halves of its pairs
// are its own: dims 4c .. and rotary_dim / 2 + 4c .. of the turning part, 8c .. and 8c + 4 .. of the
// rest (and everywhere when pairs are adjacent).  D / 8 lanes make a head, rounded up to a power of
// two; the squares are summed over them by shuffles.  A warp takes heads of one token and one kind
// (query, key or value), so that the weights, multiplied by cos and sin once, stay in registers:
//   u = r (p wp cos - q wq sin),  v = r (q wq cos + p wp sin),  r = 1 / sqrt(mean + eps)
// in packed pairs of floats.
//
// INT4 caches (kInt4) take a key's four codes of a piece, its float32 values divided by the scale of
// their group, as 16 bits; a piece never crosses a group, whose size is at least 8.
// 16384 tokens of 64 + 16 heads take 119 us (5.3 TB/s): 107 at HBM's rate, which is what codes that are neither
// divided nor clamped take (5.9 TB/s; the 16-bit form 6.1), and 12 of the codes' instructions.  121 with one reciprocal
// for a piece's four quotients and two exact steps, 122 with that and 3 blocks an SM (no spills).
//
// About 2 bytes move per element each way: the bound is HBM, once the instructions per element are
// few (packed arithmetic, pointers advanced by a constant).  A warp takes several heads, loaded four
// at a time before the first is used, once there are tokens enough to fill the GPU; fewer heads a
// warp below that (see launch_lanes).
#include "common.cuh"
#include "dependent_launch.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
// Loads in flight a lane, batches of them a warp at most, blocks an SM.  16384 tokens of 64 + 16 heads
// take 111 us so (6.1 TB/s); 121, 115 us with 2 and 4 batches, 119 with 5 loads, 128 us with 3 blocks
// (80 registers: fewer warps), 132 with 5 (48: spills; and 2 loads, 4 batches).
constexpr int kBatch = 4;
constexpr int kRounds = 8;
constexpr int kBlocksAnSm = 4;

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Eight 16-bit elements (two pieces) as four pairs: p01 p23 (first piece), q01 q23 (second).
struct Eight {
    float2 p[2], q[2];
};
template <typename T> __device__ __forceinline__ Eight widen(uint2 r0, uint2 r1) {
    Eight x;
    x.p[0] = unpack2<T>(r0.x), x.p[1] = unpack2<T>(r0.y);
    x.q[0] = unpack2<T>(r1.x), x.q[1] = unpack2<T>(r1.y);
    return x;
}

// Four float32 values -> four E4M3 bytes of x / scale (correctly rounded division, round to nearest
// even, saturating).
__device__ __forceinline__ uint32_t quantise4(const float2 (&x)[2], float scale) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[0].x, scale), __fdiv_rn(x[0].y, scale)),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[1].x, scale), __fdiv_rn(x[1].y, scale)),
                                                 __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// Four float32 values -> four INT4 codes (the rounding of kv_reshape_and_cache_int4).
__device__ __forceinline__ uint16_t quantise4_int4(const float2 (&x)[2], float scale) {
    return static_cast<uint16_t>(int4_code(x[0].x, scale) | (int4_code(x[0].y, scale) << 4) |
                                 (int4_code(x[1].x, scale) << 8) | (int4_code(x[1].y, scale) << 12));
}

__device__ __forceinline__ uint2 ld_piece(const void *p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

// LP lanes a head; a warp takes 32 / LP heads at a time.  kD is the head size, or 0 for one only known
// at run time (64 and 128, the sizes the attention calls take, get their addresses as constants).
// An output may be its input: a piece is read and then written by one lane, and no other lane
// touches it.
template <typename T, int LP, bool kAdjacent, int kD, bool kInt4>
__global__ void __launch_bounds__(kThreads, kBlocksAnSm) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int HPW = 32 / LP;
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    int part = blockIdx.y;
    previous_kernel_done();
    if (t >= a.num_tokens) return;
    const bool reports = part == 0 && lane == 0;
    const int32_t pos = a.positions ? a.positions[t] : 0;
    int64_t slot = a.slot_mapping ? a.slot_mapping[t] : -1;
    // the warp's kind and heads
    int kind = 0;
    if (part >= a.q_parts) part -= a.q_parts, kind = 1;
    if (kind && part >= a.kv_parts) part -= a.kv_parts, kind = 2;
    const int heads = kind == 0 ? a.num_q_heads : a.num_kv_heads;
    const int first = part * a.heads_a_warp, last = min(heads, first + a.heads_a_warp);
    const int c = lane & (LP - 1), mine = first + lane / LP;  // chunk of the head, first head
    const int D = kD ? kD : a.head_dim;
    const bool has = kD ? true : 8 * c < D;
    const int half = a.rotary_dim >> 1;
    const bool turns = 8 * c < a.rotary_dim;
    const int d0 = kAdjacent || !turns ? 8 * c : 4 * c;   // the two pieces
    const int d1 = kAdjacent || !turns ? 8 * c + 4 : half + 4 * c;
    const T *src = kind == 0 ? static_cast<const T *>(a.q) + t * a.q_stride
                             : (kind == 1 ? static_cast<const T *>(a.key) + t * a.key_stride
                                          : static_cast<const T *>(a.value) + t * a.value_stride);
    src += static_cast<int64_t>(mine) * D;
    const int step = HPW * D;
    const int n = has ? (last - mine + HPW - 1) / HPW : 0;  // this lane's heads (those past last: none)
    const int rounds = (last - first + HPW - 1) / HPW;      // the warp's
    uint2 raw[kBatch][2];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            raw[i][0] = raw[i][1] = make_uint2(0, 0);
            if (i0 + i < n) {
                raw[i][0] = ld_piece(src + i * step + d0);
                raw[i][1] = ld_piece(src + i * step + d1);
            }
        }
        src += kBatch * step;
    };
    load(0);  // needs no position: on the way while the token's position, angles and weights come

    if (pos < 0) return;
    if (a.rotary_dim > 0 && pos >= a.max_position) {
        if (reports) report(a.d_err, KV_DERR_BAD_POS);
        return;
    }
    if (slot >= a.total_slots) {
        if (a.slot_mapping && reports) report(a.d_err, KV_DERR_BAD_SLOT);
        slot = -1;
    }
    const int64_t at = (slot * a.num_kv_heads + mine) * D;  // in the caches, once slot >= 0
    if (kind == 2) {
        if (slot < 0) return;
        if constexpr (kInt4) {
            uint8_t *dst = static_cast<uint8_t *>(a.v_cache) + (at >> 1);
            const float *sc = a.v_gscales + static_cast<int64_t>(mine) * (D >> a.group_shift);
            const int s0 = d0 >> a.group_shift, s1 = d1 >> a.group_shift, next = step >> a.group_shift;
            for (int i0 = 0; i0 < rounds; i0 += kBatch) {
                if (i0) load(i0);
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (i0 + i >= n) continue;
                    const Eight x = widen<T>(raw[i][0], raw[i][1]);
                    *reinterpret_cast<uint16_t *>(dst + ((i * step + d0) >> 1)) = quantise4_int4(x.p, sc[i * next + s0]);
                    *reinterpret_cast<uint16_t *>(dst + ((i * step + d1) >> 1)) = quantise4_int4(x.q, sc[i * next + s1]);
                }
                dst += kBatch * step / 2;
                sc += kBatch * next;
            }
        } else if (a.cache_fp8) {
            uint8_t *dst = static_cast<uint8_t *>(a.v_cache) + at;
            for (int i0 = 0; i0 < rounds; i0 += kBatch) {
                if (i0) load(i0);
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (i0 + i >= n) continue;
                    const Eight x = widen<T>(raw[i][0], raw[i][1]);
                    *reinterpret_cast<uint32_t *>(dst + i * step + d0) = quantise4(x.p, a.v_scale);
                    *reinterpret_cast<uint32_t *>(dst + i * step + d1) = quantise4(x.q, a.v_scale);
                }
                dst += kBatch * step;
            }
        } else {
            T *dst = static_cast<T *>(a.v_cache) + at;
            for (int i0 = 0; i0 < rounds; i0 += kBatch) {
                if (i0) load(i0);
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (i0 + i >= n) continue;
                    *reinterpret_cast<uint2 *>(dst + i * step + d0) = raw[i][0];
                    *reinterpret_cast<uint2 *>(dst + i * step + d1) = raw[i][1];
                }
                dst += kBatch * step;
            }
        }
        return;
    }
    // the lane's coefficients: weights of the two pieces, times cos and sin of its four pairs
    const T *weight = static_cast<const T *>(kind == 0 ? a.q_weight : a.k_weight);
    const bool norm = weight != nullptr;
    Eight wt;
    wt.p[0] = wt.p[1] = wt.q[0] = wt.q[1] = make_float2(1.f, 1.f);
    if (norm && has)
        wt = widen<T>(*reinterpret_cast<const uint2 *>(weight + d0), *reinterpret_cast<const uint2 *>(weight + d1));
    float2 pc[2], ps[2], qc[2], qs[2];  // p -> p wp cos, p wp sin; q -> q wq cos, -q wq sin
    if (kAdjacent) {
        // pair e is elements 2e and 2e + 1: regroup the eight as evens (p) and odds (q)
        const Eight g = wt;
        wt.p[0] = make_float2(g.p[0].x, g.p[1].x), wt.p[1] = make_float2(g.q[0].x, g.q[1].x);
        wt.q[0] = make_float2(g.p[0].y, g.p[1].y), wt.q[1] = make_float2(g.q[0].y, g.q[1].y);
    }
    if (turns) {
        const float *row = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim + 4 * c;
        const float4 cs = *reinterpret_cast<const float4 *>(row);
        const float4 sn = *reinterpret_cast<const float4 *>(row + half);
        const float2 c2[2] = {make_float2(cs.x, cs.y), make_float2(cs.z, cs.w)};
        const float2 s2[2] = {make_float2(sn.x, sn.y), make_float2(sn.z, sn.w)};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            pc[i] = mul2(wt.p[i], c2[i]);
            ps[i] = mul2(wt.p[i], s2[i]);
            qc[i] = mul2(wt.q[i], c2[i]);
            qs[i] = mul2(wt.q[i], make_float2(-s2[i].x, -s2[i].y));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) pc[i] = wt.p[i], qc[i] = wt.q[i], ps[i] = qs[i] = make_float2(0.f, 0.f);
    }
    T *dst = kind == 0 ? static_cast<T *>(a.q_out) + t * a.q_out_stride
                       : (a.k_out ? static_cast<T *>(a.k_out) + t * a.k_out_stride : nullptr);
    if (dst) dst += static_cast<int64_t>(mine) * D;
    const bool to_cache = kind == 1 && slot >= 0;
    const int esize = a.cache_fp8 ? 1 : 2;
    uint8_t *cdst = to_cache ? static_cast<uint8_t *>(a.k_cache) + (kInt4 ? at >> 1 : at * esize) : nullptr;
    const float *sc = kInt4 ? a.k_gscales + static_cast<int64_t>(mine) * (D >> a.group_shift) : nullptr;
    const float inv_d = 1.f / static_cast<float>(D);
    for (int i0 = 0; i0 < rounds; i0 += kBatch) {
        if (i0) load(i0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (i0 + i >= rounds) break;  // the same for the warp
            Eight x = widen<T>(raw[i][0], raw[i][1]);
            float r = 1.f;
            if (norm) {
                float2 s2 = mul2(x.p[0], x.p[0]);
                s2 = fma2(x.p[1], x.p[1], s2);
                s2 = fma2(x.q[0], x.q[0], s2);
                s2 = fma2(x.q[1], x.q[1], s2);
                float ss = s2.x + s2.y;
#pragma unroll
                for (int o = LP / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                r = rsqrtf(fmaf(ss, inv_d, a.eps));
            }
            if (kAdjacent) {
                const Eight g = x;
                x.p[0] = make_float2(g.p[0].x, g.p[1].x), x.p[1] = make_float2(g.q[0].x, g.q[1].x);
                x.q[0] = make_float2(g.p[0].y, g.p[1].y), x.q[1] = make_float2(g.q[0].y, g.q[1].y);
            }
            const float2 r2 = make_float2(r, r);
            float2 u[2], v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                u[e] = mul2(x.p[e], pc[e]);
                v[e] = mul2(x.q[e], qc[e]);
                if (turns) {  // (a product with 0 would spread an infinity)
                    u[e] = fma2(x.q[e], qs[e], u[e]);
                    v[e] = fma2(x.p[e], ps[e], v[e]);
                }
                if (norm) u[e] = mul2(u[e], r2), v[e] = mul2(v[e], r2);
            }
            if (kAdjacent) {
                const float2 a0 = u[0], a1 = u[1], b0 = v[0], b1 = v[1];
                u[0] = make_float2(a0.x, b0.x), u[1] = make_float2(a0.y, b0.y);
                v[0] = make_float2(a1.x, b1.x), v[1] = make_float2(a1.y, b1.y);
            }
            const uint2 r0 = make_uint2(pack2<T>(u[0].x, u[0].y), pack2<T>(u[1].x, u[1].y));
            const uint2 r1 = make_uint2(pack2<T>(v[0].x, v[0].y), pack2<T>(v[1].x, v[1].y));
            if (i0 + i < n) {
                if (dst) {
                    *reinterpret_cast<uint2 *>(dst + i * step + d0) = r0;
                    *reinterpret_cast<uint2 *>(dst + i * step + d1) = r1;
                }
                if (to_cache) {
                    if constexpr (kInt4) {
                        const float c0 = sc[(i * step + d0) >> a.group_shift], c1 = sc[(i * step + d1) >> a.group_shift];
                        *reinterpret_cast<uint16_t *>(cdst + ((i * step + d0) >> 1)) = quantise4_int4(u, c0);
                        *reinterpret_cast<uint16_t *>(cdst + ((i * step + d1) >> 1)) = quantise4_int4(v, c1);
                    } else if (a.cache_fp8) {
                        *reinterpret_cast<uint32_t *>(cdst + i * step + d0) = quantise4(u, a.k_scale);
                        *reinterpret_cast<uint32_t *>(cdst + i * step + d1) = quantise4(v, a.k_scale);
                    } else {
                        *reinterpret_cast<uint2 *>(cdst + 2 * (i * step + d0)) = r0;
                        *reinterpret_cast<uint2 *>(cdst + 2 * (i * step + d1)) = r1;
                    }
                }
            }
        }
        if (dst) dst += kBatch * step;
        if constexpr (kInt4) {
            if (to_cache) cdst += kBatch * step / 2, sc += (kBatch * step) >> a.group_shift;
        } else {
            if (to_cache) cdst += kBatch * step * esize;
        }
    }
}

template <typename T, int LP, int kD, bool kInt4 = false>
cudaError_t launch_lanes(RopeArgs a, int sm_count, cudaStream_t stream) {
    constexpr int HPW = 32 / LP;
    // heads a warp: as many as leave each SM 32 warps (what a lane reads ahead, times 32 warps, covers
    // the memory's latency), between one load and kRounds batches of them
    int n = kRounds * kBatch;
    auto parts = [&](int heads) { return (heads + n * HPW - 1) / (n * HPW); };
    auto all = [&] { return parts(a.num_q_heads) + parts(a.num_kv_heads) * (a.slot_mapping ? 2 : 1); };
    while (n > 1 && static_cast<int64_t>(a.num_tokens) * all() < 32ll * sm_count) n /= 2;
    a.heads_a_warp = n * HPW;
    a.q_parts = parts(a.num_q_heads);
    a.kv_parts = parts(a.num_kv_heads);
    // a warp a token, the parts of its heads along y (fewer than 65536: n is halved only below 32 warps an
    // SM, and 65535 heads of each kind make at most 6144 parts at first)
    const dim3 grid((static_cast<unsigned>(a.num_tokens) + kThreads / 32 - 1) / (kThreads / 32), all());
    return launch_dependent(a.interleaved ? qk_norm_rope_kernel<T, LP, true, kD, kInt4>
                                          : qk_norm_rope_kernel<T, LP, false, kD, kInt4>,
                            grid, dim3(kThreads), 0, stream, a);
}

template <typename T> cudaError_t launch_typed(const RopeArgs &a, int sm_count, cudaStream_t stream) {
    const int chunks = a.head_dim / 8;
    if (a.cache_int4) return launch_lanes<T, 16, 128, true>(a, sm_count, stream);  // (head_dim 128)
    if (a.head_dim == 128) return launch_lanes<T, 16, 128>(a, sm_count, stream);
    if (a.head_dim == 64) return launch_lanes<T, 8, 64>(a, sm_count, stream);
    if (chunks <= 2) return launch_lanes<T, 2, 0>(a, sm_count, stream);
    if (chunks <= 4) return launch_lanes<T, 4, 0>(a, sm_count, stream);
    if (chunks <= 8) return launch_lanes<T, 8, 0>(a, sm_count, stream);
    if (chunks <= 16) return launch_lanes<T, 16, 0>(a, sm_count, stream);
    return launch_lanes<T, 32, 0>(a, sm_count, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs &a, int dtype, int sm_count, cudaStream_t stream) {
    if (dtype == KV_BF16) return launch_typed<__nv_bfloat16>(a, sm_count, stream);
    return launch_typed<__half>(a, sm_count, stream);
}

}  // namespace pkv
