// Per-head norms of queries and keys, rotary positions and the append of keys
// and values, one pass over a layer's q, k, v projections.
//
// Per head row x of a token: y = x / sqrt(mean(x^2) + eps) * weight, then
// (a, b) -> (a cos - b sin, a sin + b cos) for each rotated pair of y, in
// fp32 with one rounding to bf16 at the end (as separate kernels the norm and
// the rotation would each read, round and write the rows again). Bound by
// bandwidth: every value is read once and written once.
//
// A row of head_dim values is held by a group of lanes, 8 values (16 bytes)
// each, so every access is a whole 32-byte sector or more, the sum of squares
// is a shuffle reduction, and a half-split pair's other half sits in a fixed
// partner lane. A group walks the heads of one token, so the token's angles
// are loaded once, into registers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace qkw {

constexpr int kThreads = 256;

struct Params {
    const __nv_bfloat16 *q, *k, *v, *q_weight, *k_weight;
    long long q_stride, k_stride, v_stride;
    const float* cos_sin;
    const int32_t* positions;
    const int64_t* slots;
    __nv_bfloat16 *q_out, *k_cache, *v_cache;
    uint32_t* err;
    long long slot_limit;
    float eps;
    int max_positions, rot, num_tokens, hq, hkv, dim, bt;
    int head_chunks;  // blocks per token
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}

// kLanes: lanes per head row (a power of two, at least head_dim / 8).
template <int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) qk_write_kernel(const Params p) {
    constexpr int kGroups = kThreads / kLanes;
    const int lane = threadIdx.x & (kLanes - 1);
    const int tok = blockIdx.x / p.head_chunks;
    const int chunk = blockIdx.x - tok * p.head_chunks;
    const bool live = lane * 8 < p.dim;  // lanes past a head_dim that is no power of two hold nothing

    const long long slot = __ldg(p.slots + tok);
    const bool store_kv = slot >= 0 && slot < p.slot_limit;
    uint32_t bad = slot >= p.slot_limit ? PKV_DEVERR_SLOT : 0u;
    const bool turned = lane * 8 < p.rot;
    const int half_lanes = p.rot >> 4;                       // lanes of the first half of the rotated values
    const bool upper = !kInterleaved && lane >= half_lanes;  // this lane holds the pairs' second values
    float c[8], s[8];
    if (p.rot > 0) {
        int pos = __ldg(p.positions + tok);
        if (pos < 0 || pos >= p.max_positions) {
            if (slot >= 0) bad |= PKV_DEVERR_POSITION;
            pos = min(max(pos, 0), p.max_positions - 1);
        }
        if (turned) {
            const float* row = p.cos_sin + static_cast<long long>(pos) * p.rot;
            const int a0 = kInterleaved ? lane * 4 : (upper ? lane - half_lanes : lane) * 8;
#pragma unroll
            for (int i = 0; i < (kInterleaved ? 4 : 8); i += 4) {
                const float4 cv = __ldg(reinterpret_cast<const float4*>(row + a0 + i));
                const float4 sv = __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1) + a0 + i));
                c[i] = cv.x; c[i + 1] = cv.y; c[i + 2] = cv.z; c[i + 3] = cv.w;
                s[i] = sv.x; s[i + 1] = sv.y; s[i + 2] = sv.z; s[i + 3] = sv.w;
            }
        }
    }
    if (bad && p.err && chunk == 0 && threadIdx.x == 0) atomicOr(p.err, bad);

    const long long blk = store_kv ? slot / p.bt : 0;
    const int in_blk = store_kv ? static_cast<int>(slot - blk * p.bt) : 0;
    const int heads = p.hq + 2 * p.hkv;
    // every lane of a warp takes the same number of turns (shuffles below)
    for (int h0 = chunk * kGroups; h0 < heads; h0 += p.head_chunks * kGroups) {
        const int h = h0 + threadIdx.x / kLanes;
        const bool is_q = h < p.hq, is_k = !is_q && h < p.hq + p.hkv, is_v = !is_q && !is_k;
        const int hh = is_q ? h : is_k ? h - p.hq : h - p.hq - p.hkv;
        const bool here = live && h < heads;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (here) {
            const __nv_bfloat16* src = is_q ? p.q + tok * p.q_stride : is_k ? p.k + tok * p.k_stride : p.v + tok * p.v_stride;
            u = __ldg(reinterpret_cast<const uint4*>(src + static_cast<long long>(hh) * p.dim + lane * 8));
        }
        float x[8];
        unpack8(u, x);
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq += x[i] * x[i];
#pragma unroll
        for (int d = kLanes / 2; d; d >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, d, kLanes);
        const __nv_bfloat16* weight = is_q ? p.q_weight : p.k_weight;
        if (!is_v && weight && live) {
            const float r = rsqrtf(sq / static_cast<float>(p.dim) + p.eps);
            float w[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(weight + lane * 8)), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
        }
        if (kInterleaved) {
            if (turned) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = x[2 * i], b = x[2 * i + 1];
                    x[2 * i] = a * c[i] - b * s[i];
                    x[2 * i + 1] = a * s[i] + b * c[i];
                }
            }
        } else {
            const int partner = turned ? (upper ? lane - half_lanes : lane + half_lanes) : lane;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = __shfl_sync(0xFFFFFFFFu, x[i], partner, kLanes);
                if (turned) x[i] = upper ? y * s[i] + x[i] * c[i] : x[i] * c[i] - y * s[i];
            }
        }
        if (!here) continue;
        if (!is_v) u = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        if (is_q) {
            *reinterpret_cast<uint4*>(p.q_out + (static_cast<long long>(tok) * p.hq + hh) * p.dim + lane * 8) = u;
        } else if (store_kv) {
            __nv_bfloat16* cache = is_k ? p.k_cache : p.v_cache;
            *reinterpret_cast<uint4*>(cache + ((blk * p.hkv + hh) * p.bt + in_blk) * p.dim + lane * 8) = u;
        }
    }
}

using KernelFn = void (*)(Params);

KernelFn kernel_for(int lanes, bool interleaved) {
    switch (lanes) {
        case 4: return interleaved ? qk_write_kernel<4, true> : qk_write_kernel<4, false>;
        case 8: return interleaved ? qk_write_kernel<8, true> : qk_write_kernel<8, false>;
        case 16: return interleaved ? qk_write_kernel<16, true> : qk_write_kernel<16, false>;
        default: return interleaved ? qk_write_kernel<32, true> : qk_write_kernel<32, false>;
    }
}

}  // namespace qkw
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                   int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                                   const float* cos_sin, int max_positions, int rotary_dim, int interleaved,
                                   const int32_t* positions, const int64_t* slot_mapping, int num_tokens,
                                   int num_q_heads, int num_kv_heads, int head_dim, void* q_out, void* k_cache,
                                   void* v_cache, int num_blocks, int block_tokens, uint32_t* device_error,
                                   void* stream) {
    if (block_tokens != 8 && block_tokens != 16 && block_tokens != 32 && block_tokens != 64) return PKV_EUNSUPPORTED;
    if (num_tokens < 0 || num_q_heads < 1 || num_kv_heads < 1 || num_blocks < 1 || head_dim < 1 || rotary_dim < 0 ||
        max_positions < 0 || !std::isfinite(eps) || eps < 0.f)
        return PKV_EINVAL;
    if (head_dim % 8 != 0 || head_dim > PKV_ROPE_MAX_HEAD_DIM || rotary_dim % 16 != 0 || rotary_dim > head_dim)
        return PKV_EUNSUPPORTED;
    if (num_q_heads > (1 << 16) || num_kv_heads > (1 << 16)) return PKV_ERANGE;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k || !v || !slot_mapping || !q_out || !k_cache || !v_cache ||
        (rotary_dim > 0 && (!cos_sin || !positions || max_positions < 1)))
        return PKV_EINVAL;
    if (q_stride < static_cast<int64_t>(num_q_heads) * head_dim || k_stride < static_cast<int64_t>(num_kv_heads) * head_dim ||
        v_stride < static_cast<int64_t>(num_kv_heads) * head_dim || q_stride % 8 || k_stride % 8 || v_stride % 8)
        return PKV_EINVAL;
    for (const void* ptr : {q, k, v, q_weight, k_weight, static_cast<const void*>(cos_sin), static_cast<const void*>(q_out),
                            static_cast<const void*>(k_cache), static_cast<const void*>(v_cache)})
        if (!aligned16(ptr)) return PKV_EINVAL;
    int lanes = 4;
    while (lanes * 8 < head_dim) lanes *= 2;
    qkw::Params p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
    p.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.slots = slot_mapping;
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.k_cache = static_cast<__nv_bfloat16*>(k_cache);
    p.v_cache = static_cast<__nv_bfloat16*>(v_cache);
    p.err = device_error;
    p.slot_limit = static_cast<long long>(num_blocks) * block_tokens;
    p.eps = eps;
    p.max_positions = max_positions;
    p.rot = rotary_dim;
    p.num_tokens = num_tokens;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.dim = head_dim;
    p.bt = block_tokens;
    p.head_chunks = 1;
    qkw::kernel_for(lanes, interleaved != 0)<<<num_tokens, qkw::kThreads, 0, as_stream(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return PKV_ECUDA;
    }
    return PKV_OK;
}

}  // extern "C"
