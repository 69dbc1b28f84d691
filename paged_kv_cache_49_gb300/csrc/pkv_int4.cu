// Ways into and out of a cache held in 4 bits (layout and formulas:
// pkv_int4.cuh): the quantising append, pages back as bf16 pages, and copies of
// whole blocks. All are data movement with a few operations a value. Of 16,411
// tokens of 8 heads the append reads 67 MB and writes 19: 19 us, 4.5 TB/s, bound by
// its operations (13 warp instructions for 32 values, 64% of the issue slots) and by
// what the blocks of a wave wait for their first loads; loading them again takes
// 14 us, 6.1 TB/s. A load of 0.47 GB in and out takes 72 us, 6.5 TB/s.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "pkv_int4.cuh"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "pkv_tcgen05.cuh"

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
// 1 / x to the last bit but one.
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Of both halves; NaN where either is.
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

struct Append {
    const uint4* k;
    const uint4* v;
    uint32_t k_stride, v_stride;  // of a token, in 8-value vectors
    const int64_t* slots;
    uint32_t tokens, magic;  // (i * magic) >> (32 + magic_shift) is i / hkv
    int magic_shift, hkv;
    bool blocks_of_8;
    long long slot_limit;
    uint8_t* cache;
    uint32_t* err;
};

// Of both 16-bit halves, as whole numbers.
__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

constexpr float kMargin = 0x1p-14f;  // 4 of a quotient's 2^16 parts
constexpr uint32_t kNear = 8;        // parts: twice the margin

__device__ __forceinline__ float value_of(const uint4& raw, int e) {
    const uint32_t u = e < 4 ? (e < 2 ? raw.x : raw.y) : (e < 6 ? raw.z : raw.w);
    return e & 1 ? bf16_hi(u) : bf16_lo(u);
}

// All eight codes (value e in bits 4 e .. + 3) by the definition: one difference,
// one division, one rounding.
__device__ __noinline__ uint32_t divided(uint4 raw, float m, float s) {
    uint32_t word = 0;
#pragma unroll 1
    for (int e = 7; e >= 0; --e) {
        const float q = rintf(__fdiv_rn(__fsub_rn(value_of(raw, e), m), s));
        word = word << 4 | static_cast<uint32_t>(fminf(fmaxf(q, 0.f), 15.f));
    }
    return word;
}

// The codes whose sums y = x r + from (see below) are near a half: code c was
// rounded up from about h = c - 1/2, and stays where t / s > h, or = h and c is
// even. t and s h are fp32 numbers (s has 11 bits, h 5), and where they differ the
// quotient differs from h by more than half a step, so t <=> s h decides as the
// rounded division would.
__device__ __noinline__ uint32_t corrected(uint32_t word, uint4 raw, float m, float s, float r, float from) {
    unsigned which = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if ((__float_as_uint(__fmaf_rn(value_of(raw, e), r, from)) & 0xffffu) < kNear) which |= 1u << e;
    for (; which; which &= which - 1) {
        const int e = __ffs(static_cast<int>(which)) - 1;
        // one too many at the most, and 16 at the most: 15.25 is not near a half
        const uint32_t code = word >> (4 * e) & 15u;
        const float over = __fmaf_rn(0.5f - static_cast<float>(code), s, __fsub_rn(value_of(raw, e), m));
        if (code && (over < 0.f || (over == 0.f && (code & 1)))) word -= 1u << (4 * e);
    }
    return word;
}

// A row's 16 values of this lane as codes, and its group's scale and minimum, over
// which the group's kLanes lanes agree. What bounds the append is the number of
// its operations (21 warp instructions for 32 values before the steps below), so
//  * least and greatest value go through the reduction as one pair of bf16
//    numbers, the greatest negated, and NaN goes with them;
//  * (hi - lo) / 15 is by Markstein's correction of a product with 1 / 15, which
//    rounds as the division does;
//  * a code comes from one fused product and sum with r = 1 / s,
//      y = x r + (192.5 + margin - m r),
//    in [192, 256), whose last bit counts 2^-16: the upper half of its bits is a
//    constant and the code, the lower half how far the quotient is above the half
//    (less the margin) that it was rounded up from. y is off by less than the
//    margin: 2^-17 of its own rounding, 2^-15 of the sum's in brackets while
//    |m r| < 512, 2^-19 of r's error, 2^-20 of the definition's own difference.
//    A quotient within the margin of a half is looked at again (one lane in 170:
//    bf16 values lie on few points), and where saturated values leave the range,
//    or |m r| is 512 or more (groups all of whose values are within 3% of one
//    number), the division itself decides.
template <int kLanes>
__device__ __forceinline__ void quantise(const uint4 (&raw)[2], uint32_t (&word)[2], __half& s, __half& m) {
    uint32_t lo2[2], hi2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        lo2[i] = min_bf16x2(min_bf16x2(raw[i].x, raw[i].y), min_bf16x2(raw[i].z, raw[i].w));
        hi2[i] = max_bf16x2(max_bf16x2(raw[i].x, raw[i].y), max_bf16x2(raw[i].z, raw[i].w));
    }
    const uint32_t lows = min_bf16x2(lo2[0], lo2[1]), highs = max_bf16x2(hi2[0], hi2[1]) ^ 0x80008000u;
    uint32_t range = min_bf16x2(__byte_perm(lows, highs, 0x5410), __byte_perm(lows, highs, 0x7632));  // (lo, -hi)
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) range = min_bf16x2(range, __shfl_xor_sync(0xffffffffu, range, d));
    const float least = bf16_lo(range), most = -bf16_hi(range);
    const float lo = fminf(fmaxf(least, -kHalfMax), kHalfMax), span = fminf(fmaxf(most, -kHalfMax), kHalfMax) - lo;
    const float third = span * (1.f / 15.f);
    m = __float2half_rn(lo);
    s = __float2half_rn(__fmaf_rn(__fmaf_rn(-15.f, third, span), 1.f / 15.f, third));
    const float mf = __half2float(m), sf = __half2float(s);
    const float r = sf > 0.f ? rcp(sf) : 0.f;
    const float from = __fmaf_rn(-mf, r, 192.5f + kMargin);
    const uint64_t by = pair(r, r), add = pair(from, from);
    const bool inside = __fmaf_rn(least, r, from) > 192.25f && __fmaf_rn(most, r, from) < 207.75f && fabsf(mf * r) < 512.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t near = 0xffffffffu;
        word[i] = 0;
#pragma unroll
        for (int j = 3; j >= 0; --j) {  // values j and j + 4
            const uint32_t a = u[j / 2], b = u[j / 2 + 2];
            float y0, y1;
            unpair(fma2(j & 1 ? pair(bf16_hi(a), bf16_hi(b)) : pair(bf16_lo(a), bf16_lo(b)), by, add), y0, y1);
            near = min_u16x2(near, __byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x5410));
            word[i] = word[i] * 16u + __byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x7632);
        }
        // less what the upper halves' constant 0x4340 is, at each of eight places
        word[i] -= 0x43404340u * 0x1111u;
        if (!(sf > 0.f)) word[i] = 0;
        else if (!inside) word[i] = divided(raw[i], mf, sf);
        else if (min(near & 0xffffu, near >> 16) < kNear) word[i] = corrected(word[i], raw[i], mf, sf, r, from);
    }
    if (least != least) {  // a NaN
        s = m = __ushort_as_half(0x7fff);
        word[0] = word[1] = 0;
    }
}

// A quarter of a warp a pair of tokens and head: 16 values of the key and of the
// value of both a lane, so eight loads in flight. Tokens next to one another in a
// unit (a prompt's) share the 4-byte words of its values' codes and parameters.
constexpr int kTeam = 8;  // lanes
constexpr int kAppendThreads = 128;  // (16,411 tokens: 19 us, 20 with 256 threads a block)

template <int kGroups>
__global__ void __launch_bounds__(kAppendThreads, 8) append_kernel(const Append p) {
    using U = Unit<kGroups>;
    constexpr int kLanes = kTeam / kGroups;
    griddep_launch_dependents();
    griddep_wait();
    const int part = threadIdx.x % kTeam, w = part >> 1, c = 2 * (part & 1), g = part / kLanes;  // (words c and c + 1)
    const uint32_t i = blockIdx.x * (kAppendThreads / kTeam) + threadIdx.x / kTeam;
    const uint32_t pr = p.magic ? __umulhi(i, p.magic) >> p.magic_shift : i;  // i / hkv
    const int head = static_cast<int>(i - pr * p.hkv);
    const uint32_t tok = 2 * pr;
    uint4 raw[2][2][2] = {};  // [key, value][token][half]
    int slot[2] = {-1, -1};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (tok + j >= p.tokens) continue;
        const uint4* k = p.k + static_cast<uint64_t>(tok + j) * p.k_stride + (head * 16 + 2 * part);
        const uint4* v = p.v + static_cast<uint64_t>(tok + j) * p.v_stride + (head * 16 + 2 * part);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            raw[0][j][h] = __ldg(k + h);
            raw[1][j][h] = __ldg(v + h);
        }
        const long long at = __ldg(p.slots + tok + j);
        if (at >= p.slot_limit && p.err && part == 0 && head == 0) atomicOr(p.err, PKV_DEVERR_SLOT);
        slot[j] = at >= 0 && at < p.slot_limit ? static_cast<int>(at) : -1;
    }
    auto unit_at = [&](int at) { return p.cache + static_cast<size_t>(unit_of(at, head, p.hkv, p.blocks_of_8)) * U::kBytes; };
    const bool first = part % kLanes == 0;
    __half s[2], m[2];
    uint32_t word[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        quantise<kLanes>(raw[0][j], word[j], s[0], m[0]);
        if (slot[j] < 0) continue;
        uint8_t* unit = unit_at(slot[j]);
        const int t = slot[j] & 7;
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<uint32_t*>(unit + key_word(t, w, c + h)) = word[j][h];
        if (first) *reinterpret_cast<__half2*>(unit + U::kKeyParams + (t * kGroups + g) * 4) = __halves2half2(s[0], m[0]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) quantise<kLanes>(raw[1][j], word[j], s[j], m[j]);
    if (slot[0] >= 0 && slot[1] == slot[0] + 1 && (slot[0] & 1) == 0) {
        uint8_t* unit = unit_at(slot[0]);
        const int t = slot[0] & 7;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            *reinterpret_cast<uint32_t*>(unit + value_piece(t, w, 2 * (c + h))) = __byte_perm(word[0][h], word[1][h], 0x5410);
            *reinterpret_cast<uint32_t*>(unit + value_piece(t, w, 2 * (c + h) + 1)) = __byte_perm(word[0][h], word[1][h], 0x7632);
        }
        if (first) {
            *reinterpret_cast<__half2*>(unit + U::kValueScales + (g * kUnit + t) * 2) = __halves2half2(s[0], s[1]);
            *reinterpret_cast<__half2*>(unit + U::kValueMins + (g * kUnit + t) * 2) = __halves2half2(m[0], m[1]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (slot[j] < 0) continue;
        uint8_t* unit = unit_at(slot[j]);
        const int t = slot[j] & 7;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            *reinterpret_cast<uint16_t*>(unit + value_piece(t, w, 2 * (c + h))) = static_cast<uint16_t>(word[j][h]);
            *reinterpret_cast<uint16_t*>(unit + value_piece(t, w, 2 * (c + h) + 1)) = static_cast<uint16_t>(word[j][h] >> 16);
        }
        if (first) {
            *reinterpret_cast<__half*>(unit + U::kValueScales + (g * kUnit + t) * 2) = s[j];
            *reinterpret_cast<__half*>(unit + U::kValueMins + (g * kUnit + t) * 2) = m[j];
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
    int slab_units;   // of one head
    int num_src, num_dst, hkv;
    uint32_t* err;
};

// Four values of a 16-bit piece (or eight of a word, its halves' in turn): codes
// as subnormal fp16 numbers by one AND a pair, 2^24 of which the scale makes up
// for: s c + m with one rounding, then that to bf16.
__device__ __forceinline__ uint32_t values2(uint32_t codes, float s24, float m0, float s24b, float m1) {
    const __half2 h = reinterpret_cast<const __half2&>(codes);
    return pack_bf16x2(fmaf(__low2float(h), s24, m0), fmaf(__high2float(h), s24b, m1));
}

// A warp a unit, which is 1,024 bytes of codes in two loads a lane and 4,096 of
// rows out; lane 4 r + c: of the keys, token r's dims 32 w + 8 c .. + 7; of
// the values, dims 32 w + 4 r .. + 3 of tokens 2 c and 2 c + 1.
template <int kGroups>
__global__ void __launch_bounds__(kThreads) load_kernel(const Load p) {
    using U = Unit<kGroups>;
    griddep_launch_dependents();
    griddep_wait();
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
    // where its 8 rows are in a bf16 block: [head][position]
    const int per_slab = p.slab_units * p.hkv, slab = at / per_slab, rest = at - slab * per_slab;
    const int head = rest / p.slab_units, first = slab * p.slab_units + rest % p.slab_units;
    const long long out = (static_cast<long long>(dst) * p.per_block + head * (p.per_block / p.hkv) + first) * (kUnit * kDim * 2);
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

pkv_status launched(cudaError_t e) {
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) return PKV_OK;
    record_cuda_error(e);
    return PKV_ECUDA;
}

// Launched early (programmatic stream serialization): the kernel's blocks take
// their places while the one before it ends, then wait for it.
template <class P>
pkv_status launch(void (*kernel)(P), int grid, int threads, const P& p, void* stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = as_stream(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched(cudaLaunchKernelEx(&cfg, kernel, p));
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
    p.k_stride = static_cast<uint32_t>(k_stride / 8);
    p.v_stride = static_cast<uint32_t>(v_stride / 8);
    p.slots = slot_mapping;
    p.tokens = static_cast<uint32_t>(num_tokens);
    p.hkv = num_kv_heads;
    p.blocks_of_8 = block_tokens == 8;
    p.slot_limit = static_cast<long long>(num_blocks) * block_tokens;
    p.cache = static_cast<uint8_t*>(cache);
    p.err = device_error;
    const long long pairs = (static_cast<long long>(num_tokens) + 1) / 2 * num_kv_heads;
    if (pairs >= (1ll << 31) - kv4::kThreads) return PKV_ERANGE;
    // i / hkv for i < 2^31: with 2^shift < hkv <= 2^(shift + 1), the magic number
    // ceil(2^(32 + shift) / hkv) is off by less than one part in 2^31 (0: hkv is 1; Granlund
    // and Montgomery's division by an invariant)
    while ((2ll << p.magic_shift) < num_kv_heads) ++p.magic_shift;
    p.magic = static_cast<uint32_t>(((1ull << (32 + p.magic_shift)) + num_kv_heads - 1) / num_kv_heads);
    const long long blocks = (pairs + kv4::kAppendThreads / kv4::kTeam - 1) / (kv4::kAppendThreads / kv4::kTeam);
    const int groups = kv4::groups_of(group_dims);
    return kv4::launch(groups == 1 ? kv4::append_kernel<1> : groups == 2 ? kv4::append_kernel<2> : kv4::append_kernel<4>,
                       static_cast<int>(blocks), kv4::kAppendThreads, p, stream);
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
    p.slab_units = block_tokens == 8 ? 1 : 2;
    p.hkv = num_kv_heads;
    p.num_src = num_blocks;
    p.num_dst = num_dst_blocks;
    p.err = device_error;
    const long long blocks = (p.units + kv4::kThreads / 32 - 1) / (kv4::kThreads / 32);
    if (blocks > INT32_MAX) return PKV_ERANGE;
    const int groups = kv4::groups_of(group_dims);
    return kv4::launch(groups == 1 ? kv4::load_kernel<1> : groups == 2 ? kv4::load_kernel<2> : kv4::load_kernel<4>,
                       static_cast<int>(blocks), kv4::kThreads, p, stream);
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
    return kv4::launched(cudaSuccess);
}

}  // extern "C"
