// Decode attention over a paged cache held in 4 bits (layout: pkv_int4.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkv_decode_kernel.cuh"
#include "pkv_int4.cuh"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace kv4 {

struct Decode {
    const __nv_bfloat16* q;
    const uint8_t* cache;
    const int32_t* tables;
    const int32_t* context_lens;
    __nv_bfloat16* out;
    int width, cap, hq, hkv, group, num_blocks, bt;
    float scale_log2;
    uint32_t* err;
};

// One CTA per sequence and KV head, one warp per token in turn; lane l owns
// dims 4 l .. + 3 of all query heads of the group.
template <int kGroups>
__global__ void __launch_bounds__(128) decode_kernel(const Decode p) {
    using U = Unit<kGroups>;
    constexpr int kMaxG = PKV_ATTN_MAX_GROUP;
    const int s = blockIdx.y, head = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float sm_o[4][kMaxG][kDim], sm_m[4][kMaxG], sm_l[4][kMaxG];
    int n = __ldg(p.context_lens + s);
    if (n > p.cap) {
        n = p.cap;
        if (threadIdx.x == 0) atomicOr(p.err, PKV_DEVERR_CONTEXT);
    }
    const __nv_bfloat16* q = p.q + (static_cast<size_t>(s) * p.hq + head * p.group) * kDim + 4 * lane;
    float qf[kMaxG][4], o[kMaxG][4], mx[kMaxG], l[kMaxG];
#pragma unroll
    for (int h = 0; h < kMaxG; ++h) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            qf[h][e] = h < p.group ? __bfloat162float(q[h * kDim + e]) * p.scale_log2 : 0.f;
            o[h][e] = 0.f;
        }
        mx[h] = -INFINITY;
        l[h] = 0.f;
    }
    const int part = lane >> 1, w = part >> 2, c = part & 3, r = 2 * c + (lane & 1), g = lane / (32 / kGroups);
    for (int j = warp; j < n; j += 4) {
        int blk = __ldg(p.tables + static_cast<size_t>(s) * p.width + j / p.bt);
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
            blk = 0;
        }
        const int t = j & 7;
        const uint8_t* unit = p.cache + ((static_cast<size_t>(blk) * p.hkv + head) * (p.bt / kUnit) + j % p.bt / kUnit) * U::kBytes;
        const uint32_t kc = *reinterpret_cast<const uint16_t*>(unit + key_word(t, w, c) + 2 * (lane & 1));
        const uint32_t vc = *reinterpret_cast<const uint16_t*>(unit + value_piece(t, w, r));
        const __half2 kp = *reinterpret_cast<const __half2*>(unit + U::kKeyParams + (t * kGroups + g) * 4);
        const float ks = __low2float(kp), km = __high2float(kp);
        const float vs = __half2float(*reinterpret_cast<const __half*>(unit + U::kValueScales + (g * kUnit + t) * 2));
        const float vm = __half2float(*reinterpret_cast<const __half*>(unit + U::kValueMins + (g * kUnit + t) * 2));
#pragma unroll
        for (int h = 0; h < kMaxG; ++h) {
            if (h >= p.group) break;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) x = fmaf(qf[h][e], fmaf(ks, static_cast<float>((kc >> (4 * e)) & 15u), km), x);
#pragma unroll
            for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            const float top = fmaxf(mx[h], x), a = ex2(mx[h] - top), pr = ex2(x - top);
            mx[h] = top;
            l[h] = l[h] * a + pr;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[h][e] = o[h][e] * a + pr * fmaf(vs, static_cast<float>((vc >> (4 * e)) & 15u), vm);
        }
    }
#pragma unroll
    for (int h = 0; h < kMaxG; ++h) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sm_o[warp][h][4 * lane + e] = o[h][e];
        if (lane == 0) {
            sm_m[warp][h] = mx[h];
            sm_l[warp][h] = l[h];
        }
    }
    __syncthreads();
    for (int h = 0; h < p.group; ++h) {
        const float top = fmaxf(fmaxf(sm_m[0][h], sm_m[1][h]), fmaxf(sm_m[2][h], sm_m[3][h]));
        float sum = 0.f, acc = 0.f;
        for (int i = 0; i < 4 && n > 0; ++i) {
            const float f = sm_l[i][h] > 0.f || sm_l[i][h] != sm_l[i][h] ? ex2(sm_m[i][h] - top) : 0.f;
            if (f == 0.f) continue;
            sum += f * sm_l[i][h];
            acc += f * sm_o[i][h][threadIdx.x];
        }
        p.out[(static_cast<size_t>(s) * p.hq + head * p.group + h) * kDim + threadIdx.x] =
            __float2bfloat16_rn(n > 0 ? acc / sum : 0.f);
    }
}

}  // namespace kv4
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_attn_decode_int4(const void* q, const void* cache, const int32_t* block_tables,
                                           int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                                           int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                                           int block_tokens, int group_dims, float scale, int num_ctas, void* workspace,
                                           size_t workspace_bytes, void* out, void* stream) {
    if (!kv4::block_tokens_ok(block_tokens) || !kv4::groups_of(group_dims)) return PKV_EUNSUPPORTED;
    if (!q || !cache || !block_tables || !context_lens || !workspace || !out) return PKV_EINVAL;
    if (num_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1 || num_blocks < 1 || max_blocks_per_seq < 1 ||
        num_ctas < 0 || num_ctas > PKV_ATTN_MAX_CTAS || !std::isfinite(scale))
        return PKV_EINVAL;
    if (num_seqs > PKV_ATTN_MAX_SEQS || head_dim != kv4::kDim || num_q_heads % num_kv_heads != 0 ||
        num_q_heads / num_kv_heads > PKV_ATTN_MAX_GROUP)
        return PKV_EUNSUPPORTED;
    if (static_cast<long long>(num_blocks) * num_kv_heads * block_tokens >= (1ll << 31) ||
        static_cast<long long>(num_seqs) * max_blocks_per_seq >= (1ll << 31) ||
        static_cast<long long>(max_blocks_per_seq) * block_tokens >= (1ll << 31))
        return PKV_ERANGE;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PKV_EINVAL;
    if (workspace_bytes < attn::workspace_bytes(std::max(num_ctas, 1))) return PKV_EINVAL;
    kv4::Decode p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.cache = static_cast<const uint8_t*>(cache);
    p.tables = block_tables;
    p.context_lens = context_lens;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.width = max_blocks_per_seq;
    p.cap = max_blocks_per_seq * block_tokens;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.num_blocks = num_blocks;
    p.bt = block_tokens;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err = static_cast<uint32_t*>(workspace);
    const dim3 grid(num_kv_heads, num_seqs);
    switch (kv4::groups_of(group_dims)) {
        case 1: kv4::decode_kernel<1><<<grid, 128, 0, as_stream(stream)>>>(p); break;
        case 2: kv4::decode_kernel<2><<<grid, 128, 0, as_stream(stream)>>>(p); break;
        default: kv4::decode_kernel<4><<<grid, 128, 0, as_stream(stream)>>>(p); break;
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return PKV_ECUDA;
    }
    return PKV_OK;
}
