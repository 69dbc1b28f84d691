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

// Read once: not kept in L1.
__device__ __forceinline__ uint4 ld_streaming(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

struct Append {
    const uint4* k;
    const uint4* v;
    int64_t k_stride, v_stride;  // of a token, in 8-value vectors
    const int64_t* slots;
    long long tokens;
    int hkv, bt_shift;
    long long slot_limit;
    uint8_t* cache;
    uint32_t* err;
};

// A row's 8 values of this lane as codes (value e in bits 4 e .. + 3), and its
// group's scale and minimum, over which the group's kLanes lanes agree.
//
// Rounding is by adding 1.5 * 2^23, whose last bit counts ones: t / s by the
// reciprocal and one rounding. That is off by less than 2^-18 of a step within
// the range, so where the quotient is not near a half it rounds as the true one
// does; near one (one lane in 3,000 values) the division itself decides.
template <int kLanes>
__device__ __forceinline__ uint32_t quantise(const uint4& raw, __half& s, __half& m) {
    constexpr float kOne = 12582912.f;
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t lo2 = u[0], hi2 = u[0], nan = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo2 = min_bf16x2(lo2, u[i]);
        hi2 = max_bf16x2(hi2, u[i]);
        // a NaN's magnitude is above 0x7f80: its sum with 0x7f carries into the sign's place
        nan |= ((u[i] & 0x7fff7fffu) + 0x007f007fu) & 0x80008000u;
    }
    float lo = fminf(bf16_lo(lo2), bf16_hi(lo2)), hi = fmaxf(bf16_lo(hi2), bf16_hi(hi2));
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
    }
    const unsigned lane = threadIdx.x & 31, group = ((1u << kLanes) - 1) << (lane / kLanes * kLanes);
    const bool none = (__ballot_sync(0xffffffffu, nan != 0) & group) != 0;
    lo = fminf(fmaxf(lo, -kHalfMax), kHalfMax);
    hi = fminf(fmaxf(hi, -kHalfMax), kHalfMax);
    m = __float2half_rn(lo);
    s = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float mf = __half2float(m), sf = __half2float(s);
    const float r = sf > 0.f ? __frcp_rn(sf) : 0.f;
    uint32_t word = 0;
    float off = 0.f;  // the largest distance from a whole number
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = __fsub_rn(e & 1 ? bf16_hi(u[e / 2]) : bf16_lo(u[e / 2]), mf);
        const float y = __fmaf_rn(t, r, kOne);
        off = fmaxf(off, fabsf(__fmaf_rn(t, r, -__fsub_rn(y, kOne))));
        word |= static_cast<uint32_t>(__vimin_s32_relu(__float_as_int(y) - __float_as_int(kOne), 15)) << (4 * e);
    }
    if (off > 0.5f - 0x1p-14f) {
        word = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float t = __fsub_rn(e & 1 ? bf16_hi(u[e / 2]) : bf16_lo(u[e / 2]), mf);
            word |= static_cast<uint32_t>(fminf(fmaxf(rintf(__fdiv_rn(t, sf)), 0.f), 15.f)) << (4 * e);
        }
    }
    if (!(sf > 0.f)) word = 0;
    if (none) {
        s = m = __ushort_as_half(0x7fff);
        word = 0;
    }
    return word;
}

// Half a warp a pair of tokens and head: 8 values of the key and of the value of
// both a lane, so four loads in flight. Tokens next to one another in a unit
// (a prompt's) share the 4-byte words of its values' codes and parameters.
template <int kGroups>
__global__ void __launch_bounds__(kThreads) append_kernel(const Append p) {
    using U = Unit<kGroups>;
    constexpr int kLanes = 16 / kGroups;
    const int part = threadIdx.x & 15, w = part >> 2, c = part & 3, g = part / kLanes;
    const long long i = static_cast<long long>(blockIdx.x) * (kThreads / 16) + threadIdx.x / 16;
    const long long pr = i / p.hkv;
    const int head = static_cast<int>(i - pr * p.hkv);
    const long long tok = 2 * pr;
    uint4 raw[2][2] = {};  // [key, value][token]
    long long slot[2] = {-1, -1};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (tok + j >= p.tokens) continue;
        raw[0][j] = ld_streaming(p.k + (tok + j) * p.k_stride + head * 16 + part);
        raw[1][j] = ld_streaming(p.v + (tok + j) * p.v_stride + head * 16 + part);
        slot[j] = __ldg(p.slots + tok + j);
    }
    __half s[2][2], m[2][2];
    uint32_t word[2][2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int j = 0; j < 2; ++j) word[kv][j] = quantise<kLanes>(raw[kv][j], s[kv][j], m[kv][j]);
    uint8_t* unit[2];
    int t[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (slot[j] >= p.slot_limit) {
            if (p.err && part == 0 && head == 0) atomicOr(p.err, PKV_DEVERR_SLOT);
            slot[j] = -1;
        }
        const long long blk = slot[j] >> p.bt_shift;
        const int pos = static_cast<int>(slot[j] & ((1 << p.bt_shift) - 1));
        t[j] = pos & 7;
        unit[j] = p.cache + (((blk * p.hkv + head) << (p.bt_shift - 3)) + (pos >> 3)) * U::kBytes;
        if (slot[j] < 0) continue;
        *reinterpret_cast<uint32_t*>(unit[j] + key_word(t[j], w, c)) = word[0][j];
        if (part % kLanes == 0)
            *reinterpret_cast<__half2*>(unit[j] + U::kKeyParams + (t[j] * kGroups + g) * 4) = __halves2half2(s[0][j], m[0][j]);
    }
    if (slot[0] >= 0 && slot[1] == slot[0] + 1 && (slot[0] & 1) == 0) {
        *reinterpret_cast<uint32_t*>(unit[0] + value_piece(t[0], w, 2 * c)) = __byte_perm(word[1][0], word[1][1], 0x5410);
        *reinterpret_cast<uint32_t*>(unit[0] + value_piece(t[0], w, 2 * c + 1)) = __byte_perm(word[1][0], word[1][1], 0x7632);
        if (part % kLanes == 0) {
            *reinterpret_cast<__half2*>(unit[0] + U::kValueScales + (g * kUnit + t[0]) * 2) = __halves2half2(s[1][0], s[1][1]);
            *reinterpret_cast<__half2*>(unit[0] + U::kValueMins + (g * kUnit + t[0]) * 2) = __halves2half2(m[1][0], m[1][1]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (slot[j] < 0) continue;
        *reinterpret_cast<uint16_t*>(unit[j] + value_piece(t[j], w, 2 * c)) = static_cast<uint16_t>(word[1][j]);
        *reinterpret_cast<uint16_t*>(unit[j] + value_piece(t[j], w, 2 * c + 1)) = static_cast<uint16_t>(word[1][j] >> 16);
        if (part % kLanes == 0) {
            *reinterpret_cast<__half*>(unit[j] + U::kValueScales + (g * kUnit + t[j]) * 2) = s[1][j];
            *reinterpret_cast<__half*>(unit[j] + U::kValueMins + (g * kUnit + t[j]) * 2) = m[1][j];
        }
    }
}

struct Load {
    const uint8_t* cache;
    const int32_t* pairs;
    uint8_t* k;
    uint8_t* v;
    long long units;  // pairs * heads * block tokens / 8
    int per_block;    // units of a block
    int num_src, num_dst;
    uint32_t* err;
};

// Four values of a 16-bit piece (or eight of a word, its halves' in turn): codes
// as subnormal fp16 numbers by one AND a pair, 2^24 of which the scale makes up
// for: s c + m with one rounding, then that to bf16.
__device__ __forceinline__ uint32_t values2(uint32_t codes, float s24, float m0, float s24b, float m1) {
    const __half2 h = reinterpret_cast<const __half2&>(codes);
    return pack_bf16x2(fmaf(__low2float(h), s24, m0), fmaf(__high2float(h), s24b, m1));
}

// A warp a unit, lane 4 r + c: of the keys, token r's dims 32 w + 8 c .. + 7; of
// the values, dims 32 w + 4 r .. + 3 of tokens 2 c and 2 c + 1.
template <int kGroups>
__global__ void __launch_bounds__(kThreads) load_kernel(const Load p) {
    using U = Unit<kGroups>;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const long long i = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    if (i >= p.units) return;
    const long long pr = i / p.per_block;
    const int at = static_cast<int>(i - pr * p.per_block);
    const int src = __ldg(p.pairs + 2 * pr), dst = __ldg(p.pairs + 2 * pr + 1);
    if (src < 0 || src >= p.num_src || dst < 0 || dst >= p.num_dst) {
        if (p.err && at == 0 && lane == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
        return;
    }
    const uint8_t* unit = p.cache + (static_cast<long long>(src) * p.per_block + at) * U::kBytes;
    const long long out = (static_cast<long long>(dst) * p.per_block + at) * (kUnit * kDim * 2);
    const uint4 kc = ld_streaming(reinterpret_cast<const uint4*>(unit) + lane);
    const uint4 vc = ld_streaming(reinterpret_cast<const uint4*>(unit + U::kValues) + lane);
    __half2 kp[kGroups], vs[kGroups], vm[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        kp[g] = __ldg(reinterpret_cast<const __half2*>(unit + U::kKeyParams) + r * kGroups + g);
        vs[g] = __ldg(reinterpret_cast<const __half2*>(unit + U::kValueScales) + g * 4 + c);
        vm[g] = __ldg(reinterpret_cast<const __half2*>(unit + U::kValueMins) + g * 4 + c);
    }
    const uint32_t kw[4] = {kc.x, kc.y, kc.z, kc.w}, vw[4] = {vc.x, vc.y, vc.z, vc.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int g = w * kGroups / 4;
        const float s = __low2float(kp[g]) * 0x1p24f, m = __high2float(kp[g]);
        // pairs (j, j + 4) of the word's eight codes, put in order behind the rounding
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = values2(kw[w] >> (4 * j) & 0x000f000fu, s, m, s, m);
        *reinterpret_cast<uint4*>(p.k + out + r * (2 * kDim) + (32 * w + 8 * c) * 2) =
            make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410), __byte_perm(o[0], o[1], 0x7632),
                       __byte_perm(o[2], o[3], 0x7632));
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int g = w * kGroups / 4;
        const float s0 = __low2float(vs[g]) * 0x1p24f, s1 = __high2float(vs[g]) * 0x1p24f;
        const float m0 = __low2float(vm[g]), m1 = __high2float(vm[g]);
        uint32_t o[4];  // dim j of both tokens
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = values2(vw[w] >> (4 * j) & 0x000f000fu, s0, m0, s1, m1);
        uint8_t* row = p.v + out + 2 * c * (2 * kDim) + (32 * w + 4 * r) * 2;
        *reinterpret_cast<uint2*>(row) = make_uint2(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410));
        *reinterpret_cast<uint2*>(row + 2 * kDim) = make_uint2(__byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632));
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
    p.tokens = num_tokens;
    p.hkv = num_kv_heads;
    p.bt_shift = block_tokens == 8 ? 3 : block_tokens == 16 ? 4 : block_tokens == 32 ? 5 : 6;
    p.slot_limit = static_cast<long long>(num_blocks) * block_tokens;
    p.cache = static_cast<uint8_t*>(cache);
    p.err = device_error;
    const long long pairs = (static_cast<long long>(num_tokens) + 1) / 2 * num_kv_heads;
    const long long blocks = (pairs + kv4::kThreads / 16 - 1) / (kv4::kThreads / 16);
    if (blocks > INT32_MAX) return PKV_ERANGE;
    const int grid = static_cast<int>(blocks);
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
    p.k = static_cast<uint8_t*>(k_cache);
    p.v = static_cast<uint8_t*>(v_cache);
    p.per_block = num_kv_heads * (block_tokens / kv4::kUnit);
    p.units = static_cast<long long>(num_pairs) * p.per_block;
    p.num_src = num_blocks;
    p.num_dst = num_dst_blocks;
    p.err = device_error;
    const long long blocks = (p.units + kv4::kThreads / 32 - 1) / (kv4::kThreads / 32);
    if (blocks > INT32_MAX) return PKV_ERANGE;
    const int grid = static_cast<int>(blocks);
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
