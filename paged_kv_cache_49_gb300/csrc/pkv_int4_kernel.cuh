// Decode attention over a paged cache held in 4 bits: the device code (layout
// and formulas of the cache: pkv_int4.cuh), included by pkv_int4_attn.cu.
//
// With q a query row, a key k_t = s c + m by groups g of its dims, and a value
// likewise:
//   x_t = scale * sum_g (s_tg <q, c_t>_g + m_tg sum_g q)
//   out = sum_t p_t v_t,  out_g = sum_t (p_t s_tg) c_t + sum_t p_t m_tg
// so the codes go into the matrix products as whole numbers, the keys' scales
// are applied to each group's sums and the values' scales to the weights: no
// code is ever turned into the value that it stands for.
//
//  * A code becomes an fp16 operand by one AND: bits 0000 0000 0000 cccc are
//    the subnormal number c * 2^-24, which the tensor core takes at full rate
//    and in full precision, and bits cccc 0000 are c * 2^-20; so a word of 8
//    codes is four registers of two (the bits 0-3, 4-7 of each half, and of
//    the word shifted by 8), 5 operations. The 16 of the odd nibbles is taken
//    off the queries' side (keys) and off the results (values).
//  * S^T[16 tokens x 8 heads] = K Q^T and O^T[128 dims x 8 heads] += V^T P^T by
//    mma.sync m16n8k16, whose N = 8 is a whole group of query heads; a unit's
//    codes lie in shared memory as the lanes hold them (one 16-byte load each).
//    The queries are scaled by a power of two per head so that fp16 holds them
//    without loss.
//  * Weights are 2^(x - max + 10), so what fp16 drops of them is below 2^-35 of
//    the largest; where a value's scale is 32 or more, 2^(x - max + 2), for
//    weight times scale to stay in range. A third product with rows of the
//    values' minima and of ones gives sum p m and the softmax's denominator.
//
// Work: as the bf16 cache's decode kernel (pkv_decode_kernel.cuh): all
// (sequence, KV head) runs laid end to end in tiles of kTile tokens, cut into
// gridDim.x ranges of equal cost. A producer warp copies tiles
// into a ring; consumer warp i takes every kWarps-th, whatever piece it
// belongs to. A helper warp goes with them, so that none waits for another: it
// has the next piece's queries ready as the products take them, and combines the
// states that the consumers leave of a piece; pieces of a run that is cut among
// CTAs are combined by whichever helper finishes last.
#pragma once

#include "pkv_decode_kernel.cuh"
#include "pkv_int4.cuh"

namespace pkv {
namespace kv4 {

constexpr int kMaxG = PKV_ATTN_MAX_GROUP;
constexpr int kTile = 64;   // tokens
constexpr int kWarps = 4;   // consumers
constexpr int kStages = 8;
static_assert(kStages % kWarps == 0, "each stage is always the same warp's");
constexpr int kProducers = 2;  // producer i copies every tile whose place in the stream is i modulo their number
constexpr int kHelper = kWarps + kProducers;
constexpr int kThreads = (kHelper + 1) * 32;
static_assert(kStages % kProducers == 0, "each stage is always the same producer's");
constexpr int kSubs = kTile / 16;
// Work partition: what a run costs beyond its tiles, in tiles.
constexpr int kRunCost = 3;
// Runs of more pieces than this are combined in two levels.
constexpr int kMergeGroup = 16;
constexpr int kMaxCtas = attn::kMaxCtas;

constexpr int kORow = attn::kORow;
constexpr int kStateFloats = kWarps * kMaxG * kORow;  // output, max and sum of every warp's heads
constexpr int kQSlots = 2;

// Shared memory: the ring, queries, states of one or two pieces (one where two
// would keep a second CTA off the SM), barriers, the plan.
template <int kGroups>
struct Smem {
    static constexpr int kStage = kTile / kUnit * Unit<kGroups>::kBytes;
    static constexpr int kQueries = kStages * kStage;
    static constexpr int kQBytes = (16 + 2 + 2 * kGroups) * 32 * 4;
    static constexpr int kBars = kQueries + kQSlots * kQBytes;
    static constexpr int kNumBars = 2 * kStages + 2 * kQSlots + 4;
    static constexpr int kMisc = kBars + kNumBars * 8;
    static constexpr int kStates = (kMisc + 64 + 15) / 16 * 16;
    static __host__ __device__ constexpr int scan(int slots) { return kStates + slots * kStateFloats * 4; }
    static constexpr size_t bytes(int num_seqs, int slots) { return 128 + scan(slots) + 4 * static_cast<size_t>(num_seqs); }
};

struct Decode {
    const __nv_bfloat16* q;
    const uint8_t* cache;
    const int32_t* tables;
    const int32_t* context_lens;
    __nv_bfloat16* out;
    int num_seqs, width, cap, hq, hkv, group, num_blocks, bt_shift;
    float scale_log2;
    uint32_t* err;
    int* counters;        // [kMaxCtas]: pieces counted of the cut run whose first piece is the CTA's
    int* group_counters;  // [kMaxCtas]: likewise, of a group of its pieces
    float* partials;      // [grid][2][kMaxG][kORow]
    int slots;            // pieces whose states fit in shared memory
};

// True in one thread of the warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one = 0;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t@p mov.u32 %0, 1;\n\t}" : "+r"(one));
    return one != 0;
}

// Products and transposes that the compiler may schedule among others.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint32_t lds32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float half_lo(uint32_t v) { return __half2float(__ushort_as_half(static_cast<unsigned short>(v))); }
__device__ __forceinline__ float half_hi(uint32_t v) { return __half2float(__ushort_as_half(static_cast<unsigned short>(v >> 16))); }
__device__ __forceinline__ uint32_t word(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

constexpr uint32_t kEven = 0x000f000fu, kOdd = 0x00f000f0u;

// A consumer warp's queries: B operands of the 8 steps of 16 dims (pairs of
// dims as the codes' registers pair them, the odd nibbles' divided by 16), and
// for the lane's two heads 2 c, 2 c + 1 the factor from sums to scores and the
// sums of the queries by group (in units of 2^-24 of a sum, as the products).
template <int kGroups>
struct Queries {
    uint32_t b[16];
    float factor[2];
    float sum[kGroups][2];

    __device__ __forceinline__ void load(const Decode& p, int s, int g, int r, int c) {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (static_cast<size_t>(s) * p.hq + static_cast<size_t>(g) * p.group + r) * kDim) + c;
        uint4 u[4];
        uint32_t top = 0;  // the head's largest magnitude, as bits
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            u[w] = r < p.group ? __ldg(src + 4 * w) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                top = max(top, max(word(u[w], i) & 0x7fffu, (word(u[w], i) >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // times 2^up the largest lies in [2^14, 2^15)
        const int up = 14 + 127 - max(static_cast<int>(top >> 7), 15);
        const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        float sums[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) sums[i] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_lo(word(u[w], i)) * by;
                x[2 * i + 1] = bf16_hi(word(u[w], i)) * by;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[4 * w + j] = pack_f16x2(x[j] * (j & 1 ? 0.0625f : 1.f), x[j + 4] * (j & 1 ? 0.0625f : 1.f));
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) t += x[i];
            sums[w * kGroups / 4] += t;
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], 1);
            sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], 2);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int lane = (2 * c + h) * 4;
            const int e = 24 - __shfl_sync(0xffffffffu, up, lane);
            factor[h] = fmaxf(fminf(ldexpf(p.scale_log2, e), 3e38f), -3e38f);
#pragma unroll
            for (int i = 0; i < kGroups; ++i) sum[i][h] = __shfl_sync(0xffffffffu, sums[i], lane) * 0x1p-24f;
        }
    }

    // Into and out of shared memory, as the lanes hold them.
    __device__ __forceinline__ void store(uint8_t* slot, int lane) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<uint4*>(slot)[i * 32 + lane] = make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
        float2* rest = reinterpret_cast<float2*>(slot + 2048) + lane;
        rest[0] = make_float2(factor[0], factor[1]);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) rest[32 * (i + 1)] = make_float2(sum[i][0], sum[i][1]);
    }
    __device__ __forceinline__ void fetch(const uint8_t* slot, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 u = reinterpret_cast<const uint4*>(slot)[i * 32 + lane];
            b[4 * i] = u.x, b[4 * i + 1] = u.y, b[4 * i + 2] = u.z, b[4 * i + 3] = u.w;
        }
        const float2* rest = reinterpret_cast<const float2*>(slot + 2048) + lane;
        factor[0] = rest[0].x, factor[1] = rest[0].y;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) sum[i][0] = rest[32 * (i + 1)].x, sum[i][1] = rest[32 * (i + 1)].y;
    }
};

// A warp's softmax state of a piece. Lane 4 r + c holds heads 2 c, 2 c + 1:
// o[2 w + j / 2][2 (j & 1) + head] dim 32 w + 4 r + j, e the third product's
// rows r (minima's sums by group, then the denominator).
template <int kGroups>
struct State {
    float base[2];  // max less the weights' exponent offset
    float max[2];
    float o[8][4];
    float e[4];
    float offset;

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int h = 0; h < 2; ++h) base[h] = max[h] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        e[0] = e[1] = e[2] = e[3] = 0.f;
        offset = 10.f;
    }

    // What the codes' sums stand for: four dims from 32 w + 4 r on of head 2 c + h.
    __device__ __forceinline__ float4 row(int w, int h, const float (&mins)[kGroups][2]) const {
        const float m = mins[w * kGroups / 4][h];
        return make_float4(fmaf(o[2 * w][h], 0x1p24f, m), fmaf(o[2 * w][h + 2], 0x1p20f, m),
                           fmaf(o[2 * w + 1][h], 0x1p24f, m), fmaf(o[2 * w + 1][h + 2], 0x1p20f, m));
    }

    // The third product's rows for the lane's heads.
    __device__ __forceinline__ void rows(int c, float (&mins)[kGroups][2], float (&sum)[2]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) mins[g][h] = __shfl_sync(0xffffffffu, e[h], 4 * g + c);
            sum[h] = __shfl_sync(0xffffffffu, e[h], 4 * kGroups + c);
        }
    }
};

// One tile into a warp's state; `valid` of its tokens count.
template <int kGroups>
__device__ __forceinline__ void add_tile(uint8_t* tile, int valid, const Queries<kGroups>& q, State<kGroups>& st, int lane) {
    using U = Unit<kGroups>;
    const int r = lane >> 2, c = lane & 3;
    if (valid < kTile) {
        // scales and minima behind the context, which may be anything, are zeros to the values' products
        for (int t = valid + lane; t < kTile; t += 32) {
            uint8_t* unit = tile + t / kUnit * U::kBytes;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                *reinterpret_cast<uint16_t*>(unit + U::kValueScales + (g * kUnit + t % kUnit) * 2) = 0;
                *reinterpret_cast<uint16_t*>(unit + U::kValueMins + (g * kUnit + t % kUnit) * 2) = 0;
            }
        }
        __syncwarp();
    }

    // ---- scores ----
    float x[kSubs][4];
#pragma unroll
    for (int i = 0; i < kSubs; ++i) {
        const uint8_t* u0 = tile + 2 * i * U::kBytes;
        const uint8_t* u1 = u0 + U::kBytes;
        const uint4 k0 = lds128(u0 + lane * 16), k1 = lds128(u1 + lane * 16);
        // two chains of products a group (one for four groups)
        constexpr int kChains = kGroups == 4 ? 1 : 2;
        float acc[kGroups][kChains][4];
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int j = 0; j < kChains; ++j) acc[g][j][0] = acc[g][j][1] = acc[g][j][2] = acc[g][j][3] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t a = word(k0, w), b = word(k1, w), ah = a >> 8, bh = b >> 8;
            const int g = w * kGroups / 4;
            mma(acc[g][0], a & kEven, b & kEven, a & kOdd, b & kOdd, q.b[4 * w], q.b[4 * w + 1]);
            mma(acc[g][kChains - 1], ah & kEven, bh & kEven, ah & kOdd, bh & kOdd, q.b[4 * w + 2], q.b[4 * w + 3]);
        }
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const uint32_t p0 = lds32(u0 + U::kKeyParams + (r * kGroups + g) * 4);
            const uint32_t p1 = lds32(u1 + U::kKeyParams + (r * kGroups + g) * 4);
            float d[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) d[h] = kChains == 2 ? acc[g][0][h] + acc[g][kChains - 1][h] : acc[g][0][h];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                t[h] = fmaf(half_lo(p0), d[h], fmaf(half_hi(p0), q.sum[g][h], t[h]));
                t[h + 2] = fmaf(half_lo(p1), d[h + 2], fmaf(half_hi(p1), q.sum[g][h], t[h + 2]));
            }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) x[i][h] = t[h] * q.factor[h & 1];
    }
    if (valid < kTile) {
#pragma unroll
        for (int i = 0; i < kSubs; ++i) {
            if (16 * i + r >= valid) x[i][0] = x[i][1] = -INFINITY;
            if (16 * i + 8 + r >= valid) x[i][2] = x[i][3] = -INFINITY;
        }
    }

    // ---- running maximum, and the scale of the weights ----
    float top[2] = {st.max[0], st.max[1]};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < kSubs; ++i) top[h] = fmaxf(top[h], fmaxf(x[i][h], x[i][h + 2]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], d));
    }
    bool large = false;
    constexpr int kWords = kTile / kUnit * kGroups * 4;
#pragma unroll
    for (int i = 0; i < (kWords + 31) / 32; ++i) {
        const int at = i * 32 + lane;
        if (kWords % 32 == 0 || at < kWords) {
            const uint32_t v = lds32(tile + at / (kGroups * 4) * U::kBytes + U::kValueScales + at % (kGroups * 4) * 4);
            large |= (v & 0xffffu) >= 0x5000u || (v >> 16) >= 0x5000u;  // 32 in fp16
        }
    }
    if (__any_sync(0xffffffffu, large)) st.offset = 2.f;
    const float base[2] = {top[0] - st.offset, top[1] - st.offset};
    if (__any_sync(0xffffffffu, base[0] != st.base[0] || base[1] != st.base[1])) {
        const float f[2] = {ex2(st.base[0] - base[0]), ex2(st.base[1] - base[1])};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int h = 0; h < 4; ++h) st.o[i][h] *= f[h & 1];
        }
        st.e[0] *= f[0];
        st.e[1] *= f[1];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        st.max[h] = top[h];
        st.base[h] = base[h];
    }

    // ---- values ----
#pragma unroll
    for (int i = 0; i < kSubs; ++i) {
        const uint8_t* u0 = tile + 2 * i * U::kBytes;
        const uint8_t* u1 = u0 + U::kBytes;
        const uint32_t p0 = transposed(pack_f16x2(ex2(x[i][0] - base[0]), ex2(x[i][1] - base[1])));
        const uint32_t p1 = transposed(pack_f16x2(ex2(x[i][2] - base[0]), ex2(x[i][3] - base[1])));
        uint32_t m0 = 0, m1 = 0;
        if (r < kGroups) {
            m0 = lds32(u0 + U::kValueMins + (r * kUnit + 2 * c) * 2);
            m1 = lds32(u1 + U::kValueMins + (r * kUnit + 2 * c) * 2);
        } else if (r == kGroups) {
            m0 = m1 = 0x3c003c00u;  // ones
        }
        mma(st.e, m0, 0u, m1, 0u, p0, p1);
        const uint4 v0 = lds128(u0 + U::kValues + lane * 16), v1 = lds128(u1 + U::kValues + lane * 16);
        uint32_t b0 = 0, b1 = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w % (4 / kGroups) == 0) {
                const int g = w * kGroups / 4;
                b0 = hmul2(p0, lds32(u0 + U::kValueScales + (g * kUnit + 2 * c) * 2));
                b1 = hmul2(p1, lds32(u1 + U::kValueScales + (g * kUnit + 2 * c) * 2));
            }
            const uint32_t a = word(v0, w), b = word(v1, w), ah = a >> 8, bh = b >> 8;
            mma(st.o[2 * w], a & kEven, a & kOdd, b & kEven, b & kOdd, b0, b1);
            mma(st.o[2 * w + 1], ah & kEven, ah & kOdd, bh & kEven, bh & kOdd, b0, b1);
        }
    }
}

// A run's pieces leave their partial results with their CTAs: slot 0 for the
// run's last, slot 1 for the others (a CTA holds at most two pieces of cut runs,
// one that goes on in the next CTA and the end of one from an earlier CTA).
__device__ __forceinline__ float* partial(const Decode& p, int cta, int last, int h) {
    return p.partials + ((static_cast<size_t>(cta) * 2 + (cta == last ? 0 : 1)) * kMaxG + h) * kORow;
}

// `count` partial results, `stride` CTAs apart from CTA `first` on, combined by
// head; emit(h, four dims from 4 lane on, max, sum). Four heads and four partial
// results are on their way at a time.
template <class Emit>
__device__ __forceinline__ void combine(const Decode& p, int first, int stride, int count, int last, int lane, Emit emit) {
#pragma unroll 1
    for (int h0 = 0; h0 < p.group; h0 += 4) {
        float M[4], L[4];
        float4 acc[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            M[h] = -INFINITY;
            L[h] = 0.f;
            acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int n = 0; n < count; n += 4) {
            float m[4][4], l[4][4];
            float4 o[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const bool live = n + k < count && h0 + h < p.group;
                    const float* src = partial(p, live ? first + (n + k) * stride : first, last, live ? h0 + h : h0);
                    m[k][h] = live ? __ldcg(src + kDim) : -INFINITY;
                    l[k][h] = live ? __ldcg(src + kDim + 1) : 0.f;
                    o[k][h] = live ? __ldcg(reinterpret_cast<const float4*>(src + 4 * lane)) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                float top = M[h];
#pragma unroll
                for (int k = 0; k < 4; ++k) top = fmaxf(top, m[k][h]);
                const float a = ex2(M[h] - top);
                acc[h] = make_float4(acc[h].x * a, acc[h].y * a, acc[h].z * a, acc[h].w * a);
                L[h] *= a;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float f = ex2(m[k][h] - top);
                    L[h] = fmaf(f, l[k][h], L[h]);
                    acc[h] = make_float4(fmaf(f, o[k][h].x, acc[h].x), fmaf(f, o[k][h].y, acc[h].y), fmaf(f, o[k][h].z, acc[h].z),
                                         fmaf(f, o[k][h].w, acc[h].w));
                }
                M[h] = top;
            }
        }
        __syncwarp();  // every lane's reads, before what emit() may put in their place
#pragma unroll
        for (int h = 0; h < 4; ++h)
            if (h0 + h < p.group) emit(h0 + h, acc[h], M[h], L[h]);
    }
}

__device__ __forceinline__ uint2 rounded(float4 o, float inv) {
    return make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

template <int kGroups>
__global__ void __launch_bounds__(kThreads, 2) decode_kernel(const Decode p) {
    using U = Unit<kGroups>;
    using L = Smem<kGroups>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = p.num_seqs, hkv = p.hkv;
    int* scan = reinterpret_cast<int*>(smem + L::scan(p.slots));
    int* misc = reinterpret_cast<int*>(smem + L::kMisc);
    volatile int* abort_flag = misc;
    int* ends = misc + 1;
    int* unknown = misc + 3;  // the walk's first piece: left to its search
    int* warp_total = misc + 4;
    static_assert(4 + kThreads / 32 <= 16, "the warps' totals fit");
    const uint32_t bar0 = smem_u32(smem + L::kBars);
    auto full_bar = [&](int i) { return bar0 + 8u * i; };
    auto empty_bar = [&](int i) { return bar0 + 8u * (kStages + i); };
    auto qfull_bar = [&](int i) { return bar0 + 8u * (2 * kStages + i); };
    auto qempty_bar = [&](int i) { return bar0 + 8u * (2 * kStages + kQSlots + i); };
    auto mfull_bar = [&](int i) { return bar0 + 8u * (2 * kStages + 2 * kQSlots + i); };
    auto mempty_bar = [&](int i) { return bar0 + 8u * (2 * kStages + 2 * kQSlots + 2 + i); };
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full_bar(i), 1);
            mbar_init(empty_bar(i), 1);
        }
        for (int i = 0; i < kQSlots; ++i) {
            mbar_init(qfull_bar(i), 1);
            mbar_init(qempty_bar(i), kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(mfull_bar(i), kWarps);
            mbar_init(mempty_bar(i), 1);
        }
        misc[0] = 0;
        *unknown = -1;
        fence_barrier_init();
    }

    // ---- plan: prefix sums of the runs' tiles, then this CTA's range ----
    // Tile x of run i = s * hkv + g sits at cost position x + kRunCost * i; a
    // CTA takes the tiles of an equal share of positions. An end of its range is
    // found by the thread that holds the sequence.
    const int per = (B + kThreads - 1) / kThreads;
    const int lo = min(B, tid * per), hi = min(B, lo + per);
    int local = 0;
    for (int s = lo; s < hi; ++s) {
        const int n = __ldg(p.context_lens + s);
        if (n > p.cap) atomicOr(p.err, PKV_DEVERR_CONTEXT);
        local += (max(min(n, p.cap), 0) + kTile - 1) / kTile;
        scan[s] = local;
    }
    int sum = local;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += n;
    }
    if (lane == 31) warp_total[warp] = sum;
    __syncthreads();
    int before = sum - local, tiles = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int t = warp_total[w];
        tiles += t;
        if (w < warp) before += t;
    }
    const int cost = hkv * (tiles + kRunCost * B);
    const int share = (cost + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    for (int s = lo, start = before; s < hi; ++s) {
        const int end = before + scan[s], nb = end - start;
        scan[s] = end;
        const int c0 = hkv * (start + kRunCost * s), c1 = c0 + hkv * (nb + kRunCost);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int y = (static_cast<int>(blockIdx.x) + i) * share;
            if (y < c0 || y >= c1) continue;
            const int g = attn::div_small(y - c0, nb + kRunCost);
            ends[i] = hkv * start + g * nb + min(y - c0 - g * (nb + kRunCost), nb);
        }
        start = end;
    }
    if (tid < 2 && (static_cast<int>(blockIdx.x) + tid) * share >= cost) ends[tid] = hkv * tiles;
    __syncthreads();
    const int range_lo = ends[0], range_hi = ends[1];

    // sequences without a context: zero rows
    for (int s = blockIdx.x; s < B; s += gridDim.x) {
        if (attn::run_blocks(scan, s) != 0) continue;
        uint4* row = reinterpret_cast<uint4*>(p.out + static_cast<size_t>(s) * p.hq * kDim);
        for (int i = tid; i < p.hq * kDim / 8; i += kThreads) row[i] = make_uint4(0, 0, 0, 0);
    }
    if (range_lo >= range_hi) return;

    const int r = lane >> 2, c = lane & 3;
    float* states = reinterpret_cast<float*>(smem + L::kStates);
    attn::PieceWalk walk(scan, B, hkv, range_lo, range_hi, unknown);
    attn::Piece pc;
    if (warp >= kWarps && warp < kHelper) {
        // ====================== producer warps =======================
        // A copy costs the warp that issues it 100 to 150 cycles, and one producer
        // took 860 a tile of four: more than the tile's time in HBM.
        const uint64_t policy = policy_evict_first();
        const int bt = 1 << p.bt_shift;
        const int tokens = min(bt, kTile);  // of one copy
        const int copies = kTile / tokens;  // of one tile
        const int ahead = 32 / copies;      // tiles whose copies' places the lanes hold
        const uint32_t copy_bytes = tokens / kUnit * U::kBytes;
        constexpr int kMaxCopies = kTile / 8;
        int gi = 0, last_issued = -1;
        while (walk.next(pc)) {
            const int ctx = min(__ldg(p.context_lens + pc.s), p.cap);
            const int32_t* row = p.tables + static_cast<size_t>(pc.s) * p.width;
            for (int j0 = 0; j0 < pc.len; j0 += ahead) {
                const int n = min(ahead, pc.len - j0);
                const int token = (pc.blk + j0) * kTile + lane * tokens;
                uint64_t src = 0;
                if (lane < n * copies && token < ctx) {
                    int id = __ldg(row + (token >> p.bt_shift));
                    if (id < 0 || id >= p.num_blocks) {
                        atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
                        id = 0;  // a valid block in its place; the output is flagged invalid
                    }
                    src = reinterpret_cast<uint64_t>(p.cache) +
                          (((static_cast<size_t>(id) * hkv + pc.g) << (p.bt_shift - 3)) + (token & (bt - 1)) / kUnit) * U::kBytes;
                }
                for (int j = 0; j < n; ++j, ++gi) {
                    if (gi % kProducers != warp - kWarps) continue;
                    const int st = gi % kStages;
                    const int left = min(kTile, ctx - (pc.blk + j0 + j) * kTile);
                    const uint32_t bytes = (left + kUnit - 1) / kUnit * U::kBytes;
                    const uint32_t full = full_bar(st), dst = smem_u32(smem + st * L::kStage);
                    const bool ok = mbar_wait(empty_bar(st), static_cast<uint32_t>((gi / kStages) & 1) ^ 1u, abort_flag, p.err);
                    if (!__all_sync(0xffffffffu, ok)) continue;
                    last_issued = gi;
                    uint64_t from[kMaxCopies];
#pragma unroll
                    for (int i = 0; i < kMaxCopies; ++i)
                        if (i < copies) from[i] = __shfl_sync(0xffffffffu, src, j * copies + i);
                    if (elect_one()) {
                        mbar_arrive_expect_tx(full, bytes);
#pragma unroll
                        for (int i = 0; i < kMaxCopies; ++i) {
                            const uint32_t at = i * copy_bytes;
                            if (at >= bytes) break;
                            bulk_load(dst + at, reinterpret_cast<const void*>(from[i]), min(bytes - at, copy_bytes), full, policy);
                        }
                    }
                }
            }
        }
        // No copy may land after the CTA has ended. Without an abort every copy
        // was waited for by its consumer and these waits return at once; after
        // one (a wait that ran out) the copies issued need not be a prefix, so
        // a grace period far longer than any copy takes comes first.
        if (lane == 0) {
            if (*abort_flag) {
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < attn::kDrainGraceNs) {
                }
            }
            volatile int never = 0;
            for (int i = last_issued; i > last_issued - kStages && i >= 0; i -= kProducers)
                mbar_wait(full_bar(i % kStages), static_cast<uint32_t>((i / kStages) & 1), &never, nullptr);
        }
        return;
    }

    if (warp == kHelper) {
        // ======================== helper warp ========================
        // The next piece's queries, then this one's results. Consumers that have
        // few tiles of a piece read its queries themselves.
        int slot = 0, qslot = 0;
        uint32_t phase = 0, qphase = 0;
        int turn = 0;  // the consumer that has the piece's first tile
        auto prepare = [&](const attn::Piece& piece) {
            if (piece.len < kWarps) return;
            Queries<kGroups> q;
            q.load(p, piece.s, piece.g, r, c);
            if (mbar_wait(qempty_bar(qslot), qphase ^ 1u, abort_flag, p.err)) q.store(smem + L::kQueries + qslot * L::kQBytes, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull_bar(qslot));
            if (++qslot == kQSlots) {
                qslot = 0;
                qphase ^= 1u;
            }
        };
        attn::Piece next;
        bool more = walk.next(next);
        prepare(next);
        while (more) {
            pc = next;
            more = walk.next(next);
            if (more) prepare(next);
            const int s = pc.s, g = pc.g, nb = pc.nb, some = min(kWarps, pc.len), from = turn;
            turn = (turn + pc.len) % kWarps;
            if (nb == 1) continue;  // its consumer writes the rows
            const int seg = hkv * (scan[s] - nb) + g * nb + kRunCost * (s * hkv + g);
            const int i0 = seg / share, i1 = (seg + nb - 1) / share, pieces = i1 - i0 + 1;
            const int cta = static_cast<int>(blockIdx.x);
            uint2* out = reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(s) * p.hq + static_cast<size_t>(g) * p.group) * kDim) + lane;
            auto finish = [&](int h, float4 o, float, float l) { out[h * (kDim / 4)] = rounded(o, 1.f / l); };
            auto leave = [&](float* dst, float4 o, float m, float l) {
                *reinterpret_cast<float4*>(dst + 4 * lane) = o;
                if (lane == 0) {
                    dst[kDim] = m;
                    dst[kDim + 1] = l;
                }
            };
            mbar_wait(mfull_bar(slot), phase, abort_flag, p.err);
            const float* held = states + slot * kStateFloats;
#pragma unroll 2
            for (int h = 0; h < p.group; ++h) {
                float m[kWarps], M = -INFINITY, l = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {  // consumers from, from + 1, ... hold tiles of the piece
                    const int w = from + k < kWarps ? from + k : from + k - kWarps;
                    m[k] = k < some ? held[(w * kMaxG + h) * kORow + kDim] : -INFINITY;
                    M = fmaxf(M, m[k]);
                }
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    if (k >= some) continue;
                    const int w = from + k < kWarps ? from + k : from + k - kWarps;
                    const float* src = held + (w * kMaxG + h) * kORow;
                    const float f = ex2(m[k] - M);
                    const float4 v = *reinterpret_cast<const float4*>(src + 4 * lane);
                    l = fmaf(f, src[kDim + 1], l);
                    o = make_float4(fmaf(f, v.x, o.x), fmaf(f, v.y, o.y), fmaf(f, v.z, o.z), fmaf(f, v.w, o.w));
                }
                if (pieces == 1) finish(h, o, M, l);
                else leave(partial(p, cta, i1, h), o, M, l);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(mempty_bar(slot));
            if (++slot == p.slots) {
                slot = 0;
                phase ^= 1u;
            }
            if (pieces == 1) continue;
            // true for the last of `count` that come here
            auto last = [&](int* ctr, int count) {
                __syncwarp();  // every lane's stores, before lane 0's release
                int old = 0;
                if (lane == 0) {
                    old = atom_add_acq_rel_gpu(ctr, 1);
                    if (old == count - 1) *ctr = 0;  // ready for the next launch
                }
                old = __shfl_sync(0xffffffffu, old, 0);
                __syncwarp();
                return old == count - 1;
            };
            int stride = 1;
            if (pieces > kMergeGroup) {
                stride = kMergeGroup;
                const int base = i0 + (cta - i0) / kMergeGroup * kMergeGroup;
                const int count = min(kMergeGroup, i1 - base + 1);
                if (count > 1) {  // else a lone piece, its group's result already
                    if (!last(p.group_counters + base, count)) continue;
                    combine(p, base, 1, count, i1, lane,
                            [&](int h, float4 o, float m, float l) { leave(partial(p, base, i1, h), o, m, l); });
                }
            }
            const int count = (pieces + stride - 1) / stride;
            if (last(p.counters + i0, count)) combine(p, i0, stride, count, i1, lane, finish);
        }
        return;
    }

    // ======================= consumer warps =======================
    int gidx = 0, slot = 0, qslot = 0;
    uint32_t phase = 0, qphase = 0;
    while (walk.next(pc)) {
        const int s = pc.s, g = pc.g;
        const int ctx = min(__ldg(p.context_lens + s), p.cap);
        const int turn = gidx % kWarps;
        const int first = warp >= turn ? warp - turn : warp + kWarps - turn;
        const bool mine = first < pc.len;
        Queries<kGroups> q;
        if (pc.len >= kWarps) {
            const bool landed = mbar_wait(qfull_bar(qslot), qphase, abort_flag, p.err);
            q.fetch(smem + L::kQueries + qslot * L::kQBytes, lane);
            __syncwarp();
            if (lane == 0 && landed) mbar_arrive(qempty_bar(qslot));
            if (++qslot == kQSlots) {
                qslot = 0;
                qphase ^= 1u;
            }
        } else if (mine) {
            q.load(p, s, g, r, c);
        }
        State<kGroups> st;
        st.clear();
        for (int j = first; j < pc.len; j += kWarps) {
            const int gi = gidx + j, stage = gi % kStages;
            const bool landed = mbar_wait(full_bar(stage), static_cast<uint32_t>((gi / kStages) & 1), abort_flag, p.err);
            add_tile<kGroups>(smem + stage * L::kStage, min(kTile, ctx - (pc.blk + j) * kTile), q, st, lane);
            fence_proxy_async_shared();  // this lane's accesses of the stage, before the copy that will replace it
            __syncwarp();
            if (lane == 0 && landed) mbar_arrive(empty_bar(stage));
        }
        gidx += pc.len;
        if (pc.nb == 1) {  // a run of one tile: its warp writes the rows
            if (!mine) continue;
            float mins[kGroups][2], sums[2];
            st.rows(c, mins, sums);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (2 * c + h >= p.group) continue;
                const float inv = 1.f / sums[h];
                __nv_bfloat16* row = p.out + (static_cast<size_t>(s) * p.hq + static_cast<size_t>(g) * p.group + 2 * c + h) * kDim;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    *reinterpret_cast<uint2*>(row + 32 * w + 4 * r) = rounded(st.row(w, h, mins), inv);
            }
            continue;
        }
        mbar_wait(mempty_bar(slot), phase ^ 1u, abort_flag, p.err);
        if (mine) {
            float mins[kGroups][2], sums[2];
            st.rows(c, mins, sums);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* dst = states + slot * kStateFloats + (warp * kMaxG + 2 * c + h) * kORow;
#pragma unroll
                for (int w = 0; w < 4; ++w) *reinterpret_cast<float4*>(dst + 32 * w + 4 * r) = st.row(w, h, mins);
                if (r == 0) {
                    dst[kDim] = st.base[h];
                    dst[kDim + 1] = sums[h];
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(mfull_bar(slot));
        if (++slot == p.slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
}

}  // namespace kv4
}  // namespace pkv
