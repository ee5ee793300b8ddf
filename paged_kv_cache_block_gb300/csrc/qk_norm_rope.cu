// RMS norm of every query and key head, rotary embedding, and the write of K and V into the paged
// cache, in one pass over a step's projections ("vLLM의 KV cache 연결 흐름", section "Slot
// mapping은 왜 필요한가": the new tokens' K/V go to their slots; the norm and the rotation that
// come before it are in no section of the pages).
//
// Per head of D dims:  y = x * w / sqrt(mean(x^2) + eps),  then pairs turn by the token's angles.
// A head is read once into registers (8 elements a lane, D / 8 lanes a head, rounded up to a power
// of two), the squares are summed over those lanes by shuffles, a lane gets its pair's other
// half from the lane that holds it, and the result is rounded once.  About 2 bytes moved per
// element each way: the bound is HBM.
#include "common.cuh"
#include "kernels.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

// Eight float32 values -> eight E4M3 bytes of x / scale (correctly rounded division, round to
// nearest even, saturating).
__device__ __forceinline__ uint2 quantise8f(const float (&x)[8], float scale) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <typename T> __device__ __forceinline__ void widen8(uint4 raw, float (&x)[8]) {
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T>(u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// LP lanes a head; a warp takes 32 / LP heads at a time, of one token.
template <typename T, int LP>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int HPW = 32 / LP;
    const int lane = threadIdx.x & 31;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int64_t t = w / a.parts;
    const int part = static_cast<int>(w - t * a.parts);
    if (t >= a.num_tokens) return;
    const int32_t pos = a.positions ? a.positions[t] : 0;
    if (pos < 0) return;
    if (a.rotary_dim > 0 && pos >= a.max_position) {
        if (part == 0 && lane == 0) report(a.d_err, KV_DERR_BAD_POS);
        return;
    }
    int64_t slot = a.slot_mapping ? a.slot_mapping[t] : -1;
    if (slot >= a.total_slots) {
        if (part == 0 && lane == 0) report(a.d_err, KV_DERR_BAD_SLOT);
        slot = -1;
    }
    const int c = lane & (LP - 1);       // chunk of 8 dims
    const int d0 = 8 * c;
    const bool has = d0 < a.head_dim;
    const int half = a.rotary_dim >> 1;
    const bool turns = d0 < a.rotary_dim;
    // cos and sin of this lane's dims: 8 pairs (halves) or 4 (adjacent), the same for every head
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
    int partner = lane;
    if (turns) {
        const float *row = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim;
        if (a.interleaved) {
            const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row + d0 / 2));
            const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + half + d0 / 2));
            cs[0] = cs[1] = c4.x, cs[2] = cs[3] = c4.y, cs[4] = cs[5] = c4.z, cs[6] = cs[7] = c4.w;
            sn[0] = -s4.x, sn[1] = s4.x, sn[2] = -s4.y, sn[3] = s4.y;
            sn[4] = -s4.z, sn[5] = s4.z, sn[6] = -s4.w, sn[7] = s4.w;
        } else {
            const bool second = d0 >= half;
            const int p0 = second ? d0 - half : d0;
            const float sign = second ? 1.f : -1.f;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row + p0) + q);
                const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + half + p0) + q);
                cs[4 * q] = c4.x, cs[4 * q + 1] = c4.y, cs[4 * q + 2] = c4.z, cs[4 * q + 3] = c4.w;
                sn[4 * q] = sign * s4.x, sn[4 * q + 1] = sign * s4.y, sn[4 * q + 2] = sign * s4.z,
                       sn[4 * q + 3] = sign * s4.w;
            }
            partner = second ? lane - half / 8 : lane + half / 8;
        }
    }
    const int heads = a.num_q_heads + a.num_kv_heads * (a.slot_mapping ? 2 : 1);
    const float inv_d = 1.f / static_cast<float>(a.head_dim);
    for (int h0 = part * HPW; h0 < heads; h0 += a.parts * HPW) {  // the warp's lanes stay together
        const int hd = h0 + lane / LP;
        const bool in = has && hd < heads;
        const int kind = hd < a.num_q_heads ? 0 : (hd < a.num_q_heads + a.num_kv_heads ? 1 : 2);
        const int h = kind == 0 ? hd : (kind == 1 ? hd - a.num_q_heads : hd - a.num_q_heads - a.num_kv_heads);
        const T *src = kind == 0 ? static_cast<const T *>(a.q) + t * a.q_stride
                                 : (kind == 1 ? static_cast<const T *>(a.key) + t * a.key_stride
                                              : static_cast<const T *>(a.value) + t * a.value_stride);
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (in) raw = *reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(h) * a.head_dim + d0);
        float x[8];
        widen8<T>(raw, x);
        const T *weight = static_cast<const T *>(kind == 0 ? a.q_weight : a.k_weight);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
        for (int o = LP / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (kind < 2 && weight && in) {
            const float rs = rsqrtf(ss * inv_d + a.eps);
            float wt[8];
            widen8<T>(__ldg(reinterpret_cast<const uint4 *>(weight + d0)), wt);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= rs * wt[i];
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the other half of the pair: the neighbouring element, or the same element of a lane
            const float other = __shfl_sync(0xffffffffu, x[i], partner);
            const float o = a.interleaved ? x[i ^ 1] : other;
            y[i] = turns ? fmaf(o, sn[i], x[i] * cs[i]) : x[i];
        }
        if (!in) continue;
        if (kind == 2) {
            if (slot < 0) continue;
            const int64_t at = (slot * a.num_kv_heads + h) * a.head_dim + d0;
            if (a.cache_fp8) *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.v_cache) + at) = quantise8<T>(raw, a.v_scale);
            else *reinterpret_cast<uint4 *>(static_cast<T *>(a.v_cache) + at) = raw;
            continue;
        }
        const uint4 r = make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
        const int64_t off = static_cast<int64_t>(h) * a.head_dim + d0;
        if (kind == 0) {
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.q_out) + t * a.q_out_stride + off) = r;
        } else {
            if (a.k_out) *reinterpret_cast<uint4 *>(static_cast<T *>(a.k_out) + t * a.k_out_stride + off) = r;
            if (slot >= 0) {
                const int64_t at = (slot * a.num_kv_heads + h) * a.head_dim + d0;
                if (a.cache_fp8) *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.k_cache) + at) = quantise8f(y, a.k_scale);
                else *reinterpret_cast<uint4 *>(static_cast<T *>(a.k_cache) + at) = r;
            }
        }
    }
}

template <typename T, int LP>
cudaError_t launch_lanes(RopeArgs a, int sm_count, cudaStream_t stream) {
    const int heads = a.num_q_heads + a.num_kv_heads * (a.slot_mapping ? 2 : 1);
    a.parts = (heads + 32 / LP - 1) / (32 / LP);
    const int64_t blocks = (static_cast<int64_t>(a.num_tokens) * a.parts + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    (void)sm_count;
    qk_norm_rope_kernel<T, LP><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
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
