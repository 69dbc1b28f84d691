// Ways into and out of a cache held in 4 bits (layout and formulas:
// pkv_int4.cuh): the quantising append, pages back as bf16 pages, and copies of
// whole blocks. All are data movement with a few operations a value.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "pkv_int4.cuh"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace kv4 {

constexpr int kThreads = 256;
constexpr float kHalfMax = 65504.f;

struct Append {
    const uint4* k;
    const uint4* v;
    int64_t k_stride, v_stride;  // of a token, in 8-value vectors
    const int64_t* slots;
    long long rows;  // tokens * heads
    int hkv, bt;
    long long slot_limit;
    uint8_t* cache;
    uint32_t* err;
};

// 16 lanes a row, 8 values a lane; the lanes of a group find its range by
// shuffles.
template <int kGroups>
__global__ void __launch_bounds__(kThreads) append_kernel(const Append p) {
    using U = Unit<kGroups>;
    constexpr int kLanes = 16 / kGroups;
    const long long stride = static_cast<long long>(gridDim.x) * (kThreads / 16);
    const int part = threadIdx.x & 15;
    const int w = part >> 2, c = part & 3;
    for (long long i0 = static_cast<long long>(blockIdx.x) * (kThreads / 16); i0 < 2 * p.rows; i0 += stride) {
        const long long i = i0 + threadIdx.x / 16;
        const bool live = i < 2 * p.rows;
        const bool is_v = i >= p.rows;
        const long long row = !live ? 0 : is_v ? i - p.rows : i;
        const long long tok = row / p.hkv;
        const int head = static_cast<int>(row - tok * p.hkv);
        const uint4 raw = is_v ? __ldg(p.v + tok * p.v_stride + head * 16 + part)
                               : __ldg(p.k + tok * p.k_stride + head * 16 + part);
        const long long slot = live ? __ldg(p.slots + tok) : -1;
        float x[8] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y),
                      bf16_lo(raw.z), bf16_hi(raw.z), bf16_lo(raw.w), bf16_hi(raw.w)};
        float lo = x[0], hi = x[0];
        bool nan = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo = fminf(lo, x[e]);
            hi = fmaxf(hi, x[e]);
            nan |= x[e] != x[e];
        }
#pragma unroll
        for (int d = kLanes / 2; d; d >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
        }
        const unsigned lane = threadIdx.x & 31;
        const unsigned mine = ((1u << kLanes) - 1) << (lane / kLanes * kLanes);
        nan = (__ballot_sync(0xffffffffu, nan) & mine) != 0;
        lo = fminf(fmaxf(lo, -kHalfMax), kHalfMax);
        hi = fminf(fmaxf(hi, -kHalfMax), kHalfMax);
        __half m = __float2half_rn(lo);
        __half s = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
        const float mf = __half2float(m), sf = __half2float(s);
        uint32_t word = 0;
        if (!nan && sf > 0.f) {
            // The quotient by a reciprocal is off by less than 2^-18 of a step
            // within the range, so where it is not near a half it rounds as the
            // true one does; there the division itself decides.
            const float r = __frcp_rn(sf);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = __fsub_rn(x[e], mf);
                float q = t * r, n = rintf(q);
                if (fabsf(fabsf(q - n) - 0.5f) < 0x1p-12f) n = rintf(__fdiv_rn(t, sf));
                word |= static_cast<uint32_t>(fminf(fmaxf(n, 0.f), 15.f)) << (4 * e);
            }
        }
        if (nan) s = m = __ushort_as_half(0x7fff);
        if (slot < 0) continue;
        if (slot >= p.slot_limit) {
            if (p.err && part == 0 && head == 0 && !is_v) atomicOr(p.err, PKV_DEVERR_SLOT);
            continue;
        }
        const long long blk = slot / p.bt;
        const int pos = static_cast<int>(slot - blk * p.bt), t = pos & 7;
        uint8_t* unit = p.cache + ((blk * p.hkv + head) * (p.bt / kUnit) + pos / kUnit) * U::kBytes;
        const int g = part / kLanes;
        if (!is_v) {
            *reinterpret_cast<uint32_t*>(unit + key_word(t, w, c)) = word;
            if (part % kLanes == 0)
                *reinterpret_cast<__half2*>(unit + U::kKeyParams + (t * kGroups + g) * 4) = __halves2half2(s, m);
        } else {
            *reinterpret_cast<uint16_t*>(unit + value_piece(t, w, 2 * c)) = static_cast<uint16_t>(word);
            *reinterpret_cast<uint16_t*>(unit + value_piece(t, w, 2 * c + 1)) = static_cast<uint16_t>(word >> 16);
            if (part % kLanes == 0) {
                *reinterpret_cast<__half*>(unit + U::kValueScales + (g * kUnit + t) * 2) = s;
                *reinterpret_cast<__half*>(unit + U::kValueMins + (g * kUnit + t) * 2) = m;
            }
        }
    }
}

struct Load {
    const uint8_t* cache;
    const int32_t* pairs;
    uint4* k;
    uint4* v;
    long long vectors;  // 8 values each, of the keys: pairs * heads * block tokens * 16
    int per_block;      // vectors of a block
    int num_src, num_dst;
    int hkv, bt;
    uint32_t* err;
};

// One thread per 8 values of one token and head.
template <int kGroups>
__global__ void __launch_bounds__(kThreads) load_kernel(const Load p) {
    using U = Unit<kGroups>;
    const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < 2 * p.vectors; i += stride) {
        const bool is_v = i >= p.vectors;
        const long long j = is_v ? i - p.vectors : i;
        const long long pr = j / p.per_block;
        const int at = static_cast<int>(j - pr * p.per_block);  // (head * bt + position) * 16 + part
        const int src = __ldg(p.pairs + 2 * pr), dst = __ldg(p.pairs + 2 * pr + 1);
        if (src < 0 || src >= p.num_src || dst < 0 || dst >= p.num_dst) {
            if (p.err && at == 0 && !is_v) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
            continue;
        }
        const int part = at & 15, w = part >> 2, c = part & 3, t = (at >> 4) & 7, g = part / (16 / kGroups);
        const uint8_t* unit = p.cache + (static_cast<long long>(src) * (p.per_block / 128) + (at >> 7)) * U::kBytes;
        uint32_t word;
        __half s, m;
        if (!is_v) {
            word = __ldg(reinterpret_cast<const uint32_t*>(unit + key_word(t, w, c)));
            const __half2 sm = __ldg(reinterpret_cast<const __half2*>(unit + U::kKeyParams + (t * kGroups + g) * 4));
            s = __low2half(sm);
            m = __high2half(sm);
        } else {
            word = __ldg(reinterpret_cast<const uint16_t*>(unit + value_piece(t, w, 2 * c))) |
                   static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(unit + value_piece(t, w, 2 * c + 1)))) << 16;
            s = __ldg(reinterpret_cast<const __half*>(unit + U::kValueScales + (g * kUnit + t) * 2));
            m = __ldg(reinterpret_cast<const __half*>(unit + U::kValueMins + (g * kUnit + t) * 2));
        }
        const float sf = __half2float(s), mf = __half2float(m);
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = pack_bf16x2(fmaf(sf, static_cast<float>((word >> (8 * e)) & 15u), mf),
                               fmaf(sf, static_cast<float>((word >> (8 * e + 4)) & 15u), mf));
        (is_v ? p.v : p.k)[static_cast<long long>(dst) * p.per_block + at] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// grid.y = pair; blocks stride over one block's 16-byte vectors.
__global__ void __launch_bounds__(kThreads)
copy_kernel(uint4* __restrict__ cache, const int32_t* __restrict__ pairs, int num_blocks, int vec_per_block, uint32_t* err) {
    const int src = __ldg(pairs + 2 * blockIdx.y), dst = __ldg(pairs + 2 * blockIdx.y + 1);
    if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
        if (err && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, PKV_DEVERR_BLOCK_ID);
        return;
    }
    const uint4* s = cache + static_cast<long long>(src) * vec_per_block;
    uint4* d = cache + static_cast<long long>(dst) * vec_per_block;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < vec_per_block; i += gridDim.x * kThreads) d[i] = s[i];
}

int block_bytes(int hkv, int bt, int groups) { return hkv * (bt / kUnit) * (2 * kCodeBytes + 64 * groups); }

// Shape checks that the calls share.
pkv_status check(int num_blocks, int hkv, int head_dim, int bt, int group_dims) {
    if (num_blocks < 1 || hkv < 1) return PKV_EINVAL;
    if (head_dim != kDim || !block_tokens_ok(bt) || !groups_of(group_dims)) return PKV_EUNSUPPORTED;
    if (hkv > (1 << 16) || static_cast<long long>(num_blocks) * hkv * bt >= (1ll << 31)) return PKV_ERANGE;
    return PKV_OK;
}

pkv_status launched() {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return PKV_OK;
    record_cuda_error(e);
    return PKV_ECUDA;
}

}  // namespace kv4
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_int4_block_bytes(int num_kv_heads, int block_tokens, int group_dims) {
    if (kv4::check(1, num_kv_heads, kv4::kDim, block_tokens, group_dims) != PKV_OK) return 0;
    return static_cast<size_t>(kv4::block_bytes(num_kv_heads, block_tokens, kv4::groups_of(group_dims)));
}

pkv_status pkv_append_int4(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const int64_t* slot_mapping, int num_tokens, void* cache, int num_blocks, int num_kv_heads,
                           int head_dim, int block_tokens, int group_dims, uint32_t* device_error, void* stream) {
    const pkv_status st = kv4::check(num_blocks, num_kv_heads, head_dim, block_tokens, group_dims);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return PKV_EINVAL;
    if (num_tokens > (1 << 30)) return PKV_ERANGE;
    if (num_tokens == 0) return PKV_OK;
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (!k || !v || !slot_mapping || !cache || k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8)
        return PKV_EINVAL;
    if (k_stride > INT32_MAX || v_stride > INT32_MAX) return PKV_ERANGE;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache)) return PKV_EINVAL;
    kv4::Append p = {};
    p.k = static_cast<const uint4*>(k);
    p.v = static_cast<const uint4*>(v);
    p.k_stride = k_stride / 8;
    p.v_stride = v_stride / 8;
    p.slots = slot_mapping;
    p.rows = static_cast<long long>(num_tokens) * num_kv_heads;
    p.hkv = num_kv_heads;
    p.bt = block_tokens;
    p.slot_limit = static_cast<long long>(num_blocks) * block_tokens;
    p.cache = static_cast<uint8_t*>(cache);
    p.err = device_error;
    const int grid = static_cast<int>(std::min<long long>((2 * p.rows + 15) / 16, 65535));
    switch (kv4::groups_of(group_dims)) {
        case 1: kv4::append_kernel<1><<<grid, kv4::kThreads, 0, as_stream(stream)>>>(p); break;
        case 2: kv4::append_kernel<2><<<grid, kv4::kThreads, 0, as_stream(stream)>>>(p); break;
        default: kv4::append_kernel<4><<<grid, kv4::kThreads, 0, as_stream(stream)>>>(p); break;
    }
    return kv4::launched();
}

pkv_status pkv_load_int4(const void* cache, const int32_t* src_dst_pairs, int num_pairs, void* k_cache, void* v_cache,
                         int num_blocks, int num_dst_blocks, int num_kv_heads, int head_dim, int block_tokens,
                         int group_dims, uint32_t* device_error, void* stream) {
    pkv_status st = kv4::check(num_blocks, num_kv_heads, head_dim, block_tokens, group_dims);
    if (st == PKV_OK) st = kv4::check(num_dst_blocks, num_kv_heads, head_dim, block_tokens, group_dims);
    if (st != PKV_OK) return st;
    if (num_pairs < 0) return PKV_EINVAL;
    if (num_pairs == 0) return PKV_OK;
    if (!cache || !src_dst_pairs || !k_cache || !v_cache) return PKV_EINVAL;
    if (!aligned16(cache) || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_EINVAL;
    kv4::Load p = {};
    p.cache = static_cast<const uint8_t*>(cache);
    p.pairs = src_dst_pairs;
    p.k = static_cast<uint4*>(k_cache);
    p.v = static_cast<uint4*>(v_cache);
    p.per_block = num_kv_heads * block_tokens * 16;
    p.vectors = static_cast<long long>(num_pairs) * p.per_block;
    p.num_src = num_blocks;
    p.num_dst = num_dst_blocks;
    p.hkv = num_kv_heads;
    p.bt = block_tokens;
    p.err = device_error;
    const int grid = static_cast<int>(std::min<long long>((2 * p.vectors + kv4::kThreads - 1) / kv4::kThreads, 65535));
    switch (kv4::groups_of(group_dims)) {
        case 1: kv4::load_kernel<1><<<grid, kv4::kThreads, 0, as_stream(stream)>>>(p); break;
        case 2: kv4::load_kernel<2><<<grid, kv4::kThreads, 0, as_stream(stream)>>>(p); break;
        default: kv4::load_kernel<4><<<grid, kv4::kThreads, 0, as_stream(stream)>>>(p); break;
    }
    return kv4::launched();
}

pkv_status pkv_block_copy_int4(void* cache, const int32_t* src_dst_pairs, int num_pairs, int num_blocks,
                               int num_kv_heads, int head_dim, int block_tokens, int group_dims,
                               uint32_t* device_error, void* stream) {
    const pkv_status st = kv4::check(num_blocks, num_kv_heads, head_dim, block_tokens, group_dims);
    if (st != PKV_OK) return st;
    if (num_pairs < 0) return PKV_EINVAL;
    if (num_pairs == 0) return PKV_OK;
    if (num_pairs > 65535) return PKV_ERANGE;
    if (!cache || !src_dst_pairs || !aligned16(cache)) return PKV_EINVAL;
    const int vec = kv4::block_bytes(num_kv_heads, block_tokens, kv4::groups_of(group_dims)) / 16;
    const dim3 grid(std::min((vec + kv4::kThreads - 1) / kv4::kThreads, 64), num_pairs);
    kv4::copy_kernel<<<grid, kv4::kThreads, 0, as_stream(stream)>>>(static_cast<uint4*>(cache), src_dst_pairs, num_blocks,
                                                                     vec, device_error);
    return kv4::launched();
}

}  // extern "C"
