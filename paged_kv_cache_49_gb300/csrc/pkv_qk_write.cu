// Per-head norms of queries and keys, rotary positions and the append of keys
// and values, one pass over a layer's q, k, v projections.
//
// Per head row x of a token: y = x / sqrt(mean(x^2) + eps) * weight, then
// (a, b) -> (a cos - b sin, a sin + b cos) for each rotated pair of y, in
// fp32 with one rounding to bf16 at the end (as separate kernels the norm and
// the rotation would each read, round and write the rows again). Bound by
// bandwidth: every value is read once and written once.
//
// A row of head_dim values is held by a group of lanes, 16 values each: of the
// rotated values the 8 first halves and the 8 second halves of the same pairs
// (so a pair never crosses lanes), elsewhere 16 in a row. The groups of a
// resident grid take the (token, head) rows in turn and read the next turn's
// row, position and slot before they work on this one's, so that a turn waits
// for memory once. 16,411 tokens of 64 + 16 heads of 128: 127 us, 5.4 TB/s
// (211 us with a block per token and nothing read ahead, 175 us with three
// heads read together; two or three heads a turn, two or four blocks an SM,
// streaming stores: 127-147 us). What bounds it now is the bytes under way, 24
// KB an SM. Three turns ahead through shared memory gives 119 us there but
// takes 8.3 us for 6.1 where the rows come from L2 (5,003 tokens of 24 heads
// of 64), as they do behind a projection of a usual step. 64 tokens of 32 + 16
// heads: 2.4 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <vector>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace qkw {

constexpr int kThreads = 256;

struct Params {
    const __nv_bfloat16 *q, *k, *v, *q_weight, *k_weight;
    int q_stride, k_stride, v_stride;
    const float* cos_sin;
    const int32_t* positions;
    const int64_t* slots;
    __nv_bfloat16 *q_out, *k_out, *k_cache, *v_cache;
    uint32_t* err;
    long long slot_limit;
    float eps, inv_dim;
    int max_positions, rot, num_tokens, hq, hkv, dim, bt_shift;
    int step_tok, step_head;  // the grid's groups, as tokens and heads
};

// 16 bytes that are read once
__device__ __forceinline__ uint4 ld_streaming(const __nv_bfloat16* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// 8 bf16 values as four pairs of floats
__device__ __forceinline__ void unpack8(const uint4& u, uint64_t (&x)[4]) {
    x[0] = pair(bf16_lo(u.x), bf16_hi(u.x));
    x[1] = pair(bf16_lo(u.y), bf16_hi(u.y));
    x[2] = pair(bf16_lo(u.z), bf16_hi(u.z));
    x[3] = pair(bf16_lo(u.w), bf16_hi(u.w));
}

__device__ __forceinline__ uint32_t pack_pair(uint64_t x) {
    float lo, hi;
    unpair(x, lo, hi);
    return pack_bf16x2(lo, hi);
}

constexpr int kBlocksPerSm = 3;

// kLanes: lanes per head row (a power of two, at least head_dim / 16).
template <int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) qk_write_kernel(const Params p) {
    griddep_launch_dependents();  // an attention launched early behind this one sets itself up, then waits
    constexpr int kGroups = kThreads / kLanes;
    const int lane = threadIdx.x & (kLanes - 1);
    const int heads = p.hq + 2 * p.hkv;

    // this lane's two runs of 8 values
    const bool turned = lane * 16 < p.rot;
    const int at0 = kInterleaved || !turned ? lane * 16 : lane * 8;
    const int at1 = kInterleaved || !turned ? at0 + 8 : at0 + (p.rot >> 1);
    const bool live0 = at0 < p.dim, live1 = at1 < p.dim;  // a head_dim that is no multiple of 16 lanes' values

    // this group's (token, head), heads of q, k and v in a row
    const long long gid = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / kLanes;
    int tok = static_cast<int>(gid / heads), h = static_cast<int>(gid - static_cast<long long>(tok) * heads);
    uint4 ahead0, ahead1;
    long long slot_ahead = -1;
    int pos_ahead = 0;
    auto read_ahead = [&](int t, int hd) {
        ahead0 = ahead1 = make_uint4(0, 0, 0, 0);
        if (t >= p.num_tokens) return;
        const bool is_q = hd < p.hq, is_k = hd < p.hq + p.hkv;
        const int hh = is_q ? hd : is_k ? hd - p.hq : hd - p.hq - p.hkv;
        const __nv_bfloat16* row = (is_q ? p.q : is_k ? p.k : p.v) + hh * p.dim;
        row += static_cast<long long>(t) * (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride);
        if (live0) ahead0 = ld_streaming(row + at0);
        if (live1) ahead1 = ld_streaming(row + at1);
        slot_ahead = __ldg(p.slots + t);
        if (p.rot > 0) pos_ahead = __ldg(p.positions + t);
    };
    read_ahead(tok, h);

    // every lane of a warp takes the same number of turns (shuffles below)
    while (__any_sync(0xFFFFFFFFu, tok < p.num_tokens)) {
        const bool mine = tok < p.num_tokens;
        uint4 u[2] = {ahead0, ahead1};
        const long long slot = slot_ahead;
        int pos = pos_ahead;
        int tok2 = tok + p.step_tok, h2 = h + p.step_head;
        if (h2 >= heads) {
            h2 -= heads;
            ++tok2;
        }
        read_ahead(tok2, h2);
        const bool store_kv = mine && slot >= 0 && slot < p.slot_limit;
        uint32_t bad = mine && slot >= p.slot_limit ? PKV_DEVERR_SLOT : 0u;
        uint64_t c[4], s[4];  // of eight angles
        if (p.rot > 0) {
            if (pos < 0 || pos >= p.max_positions) {
                if (mine && slot >= 0) bad |= PKV_DEVERR_POSITION;
                pos = min(max(pos, 0), p.max_positions - 1);
            }
            if (turned && mine && h < p.hq + p.hkv) {
                const float* row = p.cos_sin + static_cast<long long>(pos) * p.rot + lane * 8;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 cv = __ldg(reinterpret_cast<const float4*>(row + 4 * i));
                    const float4 sv = __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1) + 4 * i));
                    c[2 * i] = pair(cv.x, cv.y);
                    c[2 * i + 1] = pair(cv.z, cv.w);
                    s[2 * i] = pair(sv.x, sv.y);
                    s[2 * i + 1] = pair(sv.z, sv.w);
                }
            }
        }
        if (bad && p.err && lane == 0 && h == 0) atomicOr(p.err, bad);
        const long long blk = store_kv ? slot >> p.bt_shift : 0;
        const int in_blk = static_cast<int>(slot) & ((1 << p.bt_shift) - 1);

        const bool is_q = h < p.hq, is_k = !is_q && h < p.hq + p.hkv, is_v = !is_q && !is_k;
        uint64_t x[2][4];
        unpack8(u[0], x[0]);
        unpack8(u[1], x[1]);
        const __nv_bfloat16* weight = is_q ? p.q_weight : is_k ? p.k_weight : nullptr;
        if (p.q_weight || p.k_weight) {
            uint64_t sq2 = mul2(x[0][0], x[0][0]);
#pragma unroll
            for (int e = 1; e < 8; ++e) sq2 = fma2(x[e >> 2][e & 3], x[e >> 2][e & 3], sq2);
            float sq, odd;
            unpair(sq2, sq, odd);
            sq += odd;
#pragma unroll
            for (int d = kLanes / 2; d; d >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, d, kLanes);
            if (weight) {
                const float r = rsqrtf(sq * p.inv_dim + p.eps);
                const uint64_t r2 = pair(r, r);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!(half ? live1 : live0)) continue;
                    uint64_t w[4];
                    unpack8(__ldg(reinterpret_cast<const uint4*>(weight + (half ? at1 : at0))), w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[half][e] = mul2(mul2(x[half][e], r2), w[e]);
                }
            }
        }
        if (!is_v) {
            if (turned) {
                if (kInterleaved) {
                    // angle e turns the e-th pair of the lane's 16 values
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float a, b, c0, c1, s0, s1;
                        unpair(x[e >> 2][e & 3], a, b);
                        unpair(c[e >> 1], c0, c1);
                        unpair(s[e >> 1], s0, s1);
                        const float ce = e & 1 ? c1 : c0, se = e & 1 ? s1 : s0;
                        x[e >> 2][e & 3] = pair(a * ce - b * se, a * se + b * ce);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint64_t a = x[0][e], b = x[1][e];
                        x[0][e] = sub2(mul2(a, c[e]), mul2(b, s[e]));
                        x[1][e] = fma2(a, s[e], mul2(b, c[e]));
                    }
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half)
                u[half] = make_uint4(pack_pair(x[half][0]), pack_pair(x[half][1]), pack_pair(x[half][2]), pack_pair(x[half][3]));
        }
        __nv_bfloat16* dst = nullptr;
        if (is_q) {
            if (mine) dst = p.q_out + (static_cast<long long>(tok) * p.hq + h) * p.dim;
        } else if (store_kv) {
            const int hh = is_k ? h - p.hq : h - p.hq - p.hkv;
            dst = (is_k ? p.k_cache : p.v_cache) + (((blk * p.hkv + hh) << p.bt_shift) + in_blk) * p.dim;
        }
        if (dst && live0) *reinterpret_cast<uint4*>(dst + at0) = u[0];
        if (dst && live1) *reinterpret_cast<uint4*>(dst + at1) = u[1];
        if (p.k_out && is_k && mine) {
            dst = p.k_out + (static_cast<long long>(tok) * p.hkv + (h - p.hq)) * p.dim;
            if (live0) *reinterpret_cast<uint4*>(dst + at0) = u[0];
            if (live1) *reinterpret_cast<uint4*>(dst + at1) = u[1];
        }
        tok = tok2;
        h = h2;
    }
}

using KernelFn = void (*)(Params);

KernelFn kernel_for(int lanes, bool interleaved) {
    switch (lanes) {
        case 4: return interleaved ? qk_write_kernel<4, true> : qk_write_kernel<4, false>;
        case 8: return interleaved ? qk_write_kernel<8, true> : qk_write_kernel<8, false>;
        default: return interleaved ? qk_write_kernel<16, true> : qk_write_kernel<16, false>;
    }
}

// Blocks that run at once on the current device (as many on an SM as the
// kernel's launch bounds leave registers for), its SMs read once per device.
int resident_blocks() {
    static std::mutex mu;
    static std::vector<int> cache;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (static_cast<int>(cache.size()) <= dev) cache.resize(dev + 1);
    if (cache[dev] > 0) return cache[dev];
    const cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return 0;
    }
    return cache[dev] = sms * kBlocksPerSm;
}

}  // namespace qkw
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_qk_norm_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                   int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                                   const float* cos_sin, int max_positions, int rotary_dim, int interleaved,
                                   const int32_t* positions, const int64_t* slot_mapping, int num_tokens,
                                   int num_q_heads, int num_kv_heads, int head_dim, void* q_out, void* k_out, void* k_cache,
                                   void* v_cache, int num_blocks, int block_tokens, uint32_t* device_error,
                                   void* stream) {
    if (block_tokens != 8 && block_tokens != 16 && block_tokens != 32 && block_tokens != 64) return PKV_EUNSUPPORTED;
    if (num_tokens < 0 || num_q_heads < 1 || num_kv_heads < 1 || num_blocks < 1 || head_dim < 1 || rotary_dim < 0 ||
        max_positions < 0 || !std::isfinite(eps) || eps < 0.f)
        return PKV_EINVAL;
    if (head_dim % 8 != 0 || head_dim > PKV_ROPE_MAX_HEAD_DIM || rotary_dim % 16 != 0 || rotary_dim > head_dim)
        return PKV_EUNSUPPORTED;
    if (num_q_heads > (1 << 16) || num_kv_heads > (1 << 16) || num_tokens > (1 << 30)) return PKV_ERANGE;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k || !v || !slot_mapping || !q_out || !k_cache || !v_cache ||
        (rotary_dim > 0 && (!cos_sin || !positions || max_positions < 1)))
        return PKV_EINVAL;
    if (q_stride < static_cast<int64_t>(num_q_heads) * head_dim || k_stride < static_cast<int64_t>(num_kv_heads) * head_dim ||
        v_stride < static_cast<int64_t>(num_kv_heads) * head_dim || q_stride % 8 || k_stride % 8 || v_stride % 8)
        return PKV_EINVAL;
    if (q_stride > INT32_MAX || k_stride > INT32_MAX || v_stride > INT32_MAX) return PKV_ERANGE;
    for (const void* ptr : {q, k, v, q_weight, k_weight, static_cast<const void*>(cos_sin), static_cast<const void*>(q_out), static_cast<const void*>(k_out),
                            static_cast<const void*>(k_cache), static_cast<const void*>(v_cache)})
        if (!aligned16(ptr)) return PKV_EINVAL;
    int lanes = 4;
    while (lanes * 16 < head_dim) lanes *= 2;
    qkw::Params p = {};
    p.bt_shift = 3;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
    p.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
    p.q_stride = static_cast<int>(q_stride);
    p.k_stride = static_cast<int>(k_stride);
    p.v_stride = static_cast<int>(v_stride);
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.slots = slot_mapping;
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.k_out = static_cast<__nv_bfloat16*>(k_out);
    p.k_cache = static_cast<__nv_bfloat16*>(k_cache);
    p.v_cache = static_cast<__nv_bfloat16*>(v_cache);
    p.err = device_error;
    p.slot_limit = static_cast<long long>(num_blocks) * block_tokens;
    p.eps = eps;
    p.inv_dim = 1.f / static_cast<float>(head_dim);
    p.max_positions = max_positions;
    p.rot = rotary_dim;
    p.num_tokens = num_tokens;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.dim = head_dim;
    while ((8 << (p.bt_shift - 3)) < block_tokens) ++p.bt_shift;
    const int heads = num_q_heads + 2 * num_kv_heads, groups = qkw::kThreads / lanes;
    const long long blocks = (static_cast<long long>(num_tokens) * heads + groups - 1) / groups;
    const int resident = qkw::resident_blocks();
    if (resident < 1) return PKV_ECUDA;
    const int grid = static_cast<int>(std::min<long long>(blocks, resident));
    const long long step = static_cast<long long>(grid) * groups;
    p.step_tok = static_cast<int>(step / heads);
    p.step_head = static_cast<int>(step % heads);
    qkw::kernel_for(lanes, interleaved != 0)<<<grid, qkw::kThreads, 0, as_stream(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return PKV_ECUDA;
    }
    return PKV_OK;
}

}  // extern "C"
