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
//    (Register operands: tcgen05 would have the codes' fp16 numbers, four times
//    their bytes, written back to shared or tensor memory for each product.)
//    The queries are scaled by a power of two per head so that fp16 holds them
//    without loss.
//  * Weights are 2^(x - max + 10), so what fp16 drops of them is below 2^-35 of
//    the largest (less room where fp32 holds no max - 10, from 2^24 on); where a
//    value's scale is 32 or more, 2^(x - max + 2), for weight times scale to stay
//    in range. Where all scales are below 2^-6, they are lifted by 2^11, exactly, so
//    that what fp16 drops of weight times scale is below 2^-29 of the largest weight
//    times the largest scale (from scales of 2^-17 on). A third product with rows of
//    the values' minima and of ones gives sum p m and the softmax's denominator.
//
// Work. A run is one sequence and up to 4 of its KV heads (the most of 4, 2, 1
// that divide their number), in tiles of 16 tokens a consumer warp: with 4 heads a
// warp has a head of its own, with fewer the warps of a head share its tokens. A
// tile's bytes are one copy then, or few, since a slab holds its heads' rows next
// to one another -- with a copy a block and head, issuing them (100 to 150 cycles
// each) was what bounded the kernel. All runs are laid end to end, as in the bf16
// cache's decode kernel (pkv_decode_kernel.cuh), and cut into gridDim.x ranges of
// equal cost, one a CTA, two CTAs an SM. Producer warps copy tiles into a ring;
// the consumers take up to four tiles at a time. At the end of a piece a warp has
// its head's result; warps that share a head combine theirs through shared memory
// first. Pieces of a run that is cut among CTAs are combined by whichever warp (of
// those with the same rows) finishes last.
//
// What bounds it: of 256 sequences of 11,200 tokens on average and 8 heads (3.3 GB)
// the reading, 547 us, 6.0 TB/s; of 64 of 1,500 (111 MB, 32 us, 3.5 TB/s) the start
// (5 us until the first tiles land) and the unequal ends of the ranges; the matrix
// products and what feeds them, 2,300 cycles for 64 tokens of 4 heads, fill three
// quarters of the time between.
#pragma once

#include <algorithm>
#include <type_traits>

#include "pkv_decode_kernel.cuh"
#include "pkv_int4.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace kv4 {

constexpr int kMaxG = PKV_ATTN_MAX_GROUP;
// With both sides measured, each as the kernel was then, in us for one sequence / 64 /
// 256 / 200 of one KV head:
// 8 warps and heads take 128 registers a thread at most and spill (10.5 / 34.3 /
// 558 / 22.9 with 4, 13.3 / 52.9 / 965 / 29.7 with 8); two tiles at a time overlap
// less (10.5 / 33.8 / 594 / 21.5); a second producer gives 10.4 / 33.5 / 542 / 21.9;
// a ring of 12 tiles leaves one CTA an SM (10.0 / 39.2 / 764 / 25.9).
constexpr int kWarps = 4;      // consumers, and heads of a run at most
constexpr int kTok = 16;       // tokens of a tile, a warp
constexpr int kSubs = 4;       // tiles a warp takes at a time
constexpr int kStages = 8;     // tiles of the ring
constexpr int kProducers = 2;  // producer i copies every tile whose place in the stream is i modulo their number
static_assert(kStages % kSubs == 0 && kStages % kProducers == 0, "each stage is always the same producer's");
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + kProducers * 32;
// Work partition: what a run costs beyond its tiles, in tiles (for 64 sequences /
// 256 / 200 of one KV head 32.9 / 551 / 21.2 us with 4, 32.9 / 546 / 20.4 with 6,
// 32.0 / 547 / 20.5 with 10, 33.9 / 550 / 21.6 with 14).
constexpr int kRunCost = 10;
// Runs of more pieces than this are combined in two levels, each of up to 32.
constexpr int kMergeGroup = 16;
// Counters of a launch, 64 bits with one byte a warp, in the workspace's region
// of counters: per CTA one for the cut run, and one for the group of its pieces,
// whose first piece is the CTA's (at most one: the last run of its range).
constexpr int kMaxCtas = 32 * kMergeGroup;
static_assert(2 * kMaxCtas * 8 <= static_cast<int>(attn::kWsCounterBytes), "the counters fit their region");

constexpr int kORow = attn::kORow;
// Turns of kSubs tiles after which a warp puts its sums by in shared memory, where fp32
// additions join them, and begins anew: the tensor core cuts off what it adds to a sum, so
// that one of N products of a sign loses about N 2^-28 of itself, and an output is the
// small difference of two such sums. (A piece of 131,072 tokens, error of the output's
// scale: 0.036 without, 0.0029 with 32 turns, 0.0018 with 8, of which rounding to bf16
// is 0.00165. 128 sequences of 8,000 tokens: 225 us with 32, 229 with 8.)
constexpr int kHold = 8;
constexpr int kKeptFloats = 36;  // of a lane
// Output, max and sum of every warp's rows, or the warps' kept states.
constexpr int kStateFloats = std::max(kWarps * kMaxG * kORow, kWarps * kKeptFloats * 32);

template <int kGroups>
struct Smem {
    static constexpr int kStage = kWarps * 2 * Unit<kGroups>::kBytes;
    static constexpr int kStates = kStages * kStage;
    static constexpr int kBars = kStates + kStateFloats * 4;
    static constexpr int kMisc = kBars + 2 * kStages * 8;
    static constexpr int kWalks = kMisc + 64;
    static constexpr int kScan = kWalks + kWarps * 64;
    static constexpr size_t bytes(int num_seqs) { return 128 + kScan + 4 * static_cast<size_t>(num_seqs); }
};

// A CTA's partial results: two pieces, up to 32 rows each.
constexpr int kRows = kWarps * kMaxG;
constexpr size_t partial_bytes(int rows) { return 2 * static_cast<size_t>(rows) * kORow * 4; }

struct Decode {
    const __nv_bfloat16* q;
    const uint8_t* cache;
    const int32_t* tables;
    const int32_t* context_lens;
    __nv_bfloat16* out;
    int num_seqs, width, cap, hq, hkv, group, num_blocks, bt_shift;  // (log2 of block tokens)
    int heads, runs, rows;    // KV heads of a run, runs of a sequence, query rows of a run
    int copy_tokens, copies;  // of a copy, and copies of a tile
    float scale_log2;
    uint32_t* err;
    unsigned long long* counters;        // [kMaxCtas]
    unsigned long long* group_counters;  // [kMaxCtas]
    float* partials;                     // [grid][2][rows][kORow]
};

// For tests of the bounded waits: CTA 0 copies no tiles from stop_tiles on.
struct StoppedDecode : Decode {
    int stop_tiles;
};
__device__ __forceinline__ bool stopped(const Decode&, int) { return false; }
__device__ __forceinline__ bool stopped(const StoppedDecode& p, int tile) { return blockIdx.x == 0 && tile >= p.stop_tiles; }

__device__ __forceinline__ uint64_t atom_add_acq_rel_gpu(unsigned long long* addr, uint64_t v) {
    uint64_t old;
    asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], %2;" : "=l"(old) : "l"(addr), "l"(v) : "memory");
    return old;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}
// Two floats -> f16x2 (round to nearest even); lo in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
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
// The larger of two non-negative fp16 numbers, of both halves (a NaN is larger).
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
__device__ __forceinline__ float half_lo(uint32_t v) { return __half2float(__ushort_as_half(static_cast<unsigned short>(v))); }
__device__ __forceinline__ float half_hi(uint32_t v) { return __half2float(__ushort_as_half(static_cast<unsigned short>(v >> 16))); }
__device__ __forceinline__ uint32_t word(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

constexpr uint32_t kEven = 0x000f000fu, kOdd = 0x00f000f0u;

// Values' scales that are all below kSmall (fp16 bits: 2^-6) are multiplied by kLift,
// which leaves them below 32.
constexpr uint32_t kSmall = 0x2400u;
constexpr uint32_t kLift2 = 0x68006800u;  // in both halves
constexpr float kLift = 0x1p11f;
__device__ __forceinline__ bool all_small(uint32_t scales) {
    return !__any_sync(0xffffffffu, (scales & 0xffffu) >= kSmall || (scales >> 16) >= kSmall);
}

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
};

// A warp's softmax state of a piece. Lane 4 r + c holds heads 2 c, 2 c + 1:
// o[2 w + j / 2][2 (j & 1) + head] dim 32 w + 4 r + j, e the third product's
// rows r (minima's sums by group, then the denominator).
template <int kGroups>
struct State {
    float base[2];  // the maximum less the weights' exponent offset, rounded up
    float o[8][4];
    float e[2];
    uint32_t scales;  // the largest of the values', a lane's two tokens at a time

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int h = 0; h < 2; ++h) base[h] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        e[0] = e[1] = 0.f;
        scales = 0;
    }

    // What was summed with lifted scales, without.
    __device__ __forceinline__ void unlift() {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < 4; ++h) o[i][h] *= 1.f / kLift;
    }

    // The sums with what was kept of them, which counts from an earlier base; and the sums
    // kept for later.
    __device__ __forceinline__ void add_kept(const float4* kept) {
        const float4 more = kept[8 * 32];
        const float f[2] = {ex2(more.z - base[0]), ex2(more.w - base[1])};
        e[0] = fmaf(more.x, f[0], e[0]);
        e[1] = fmaf(more.y, f[1], e[1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 x = kept[i * 32];
            o[i][0] = fmaf(x.x, f[0], o[i][0]);
            o[i][1] = fmaf(x.y, f[1], o[i][1]);
            o[i][2] = fmaf(x.z, f[0], o[i][2]);
            o[i][3] = fmaf(x.w, f[1], o[i][3]);
        }
    }
    __device__ __forceinline__ void keep(float4* kept) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            kept[i * 32] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
            o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        }
        kept[8 * 32] = make_float4(e[0], e[1], base[0], base[1]);
        e[0] = e[1] = 0.f;
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

// Lifts the values' scales of tiles, as add_tiles() takes them, where they lie; false,
// and none lifted, where one is not small.
template <int kGroups>
__device__ __forceinline__ bool lift_tiles(uint8_t* const (&at)[kSubs], const int (&valid)[kSubs], int second, int lane) {
    constexpr int kWords = kUnit * kGroups / 2;  // of a unit; a lane has one of either unit
    static_assert(2 * kWords <= 32, "a lane has one word");
    const int token = lane / kWords * kUnit + lane % 4 * 2;
    uint32_t w[kSubs], most = 0;
#pragma unroll
    for (int i = 0; i < kSubs; ++i) {
        w[i] = 0;
        if (lane < 2 * kWords && token < valid[i])
            w[i] = lds32(at[i] + lane / kWords * second + Unit<kGroups>::kValueScales + lane % kWords * 4);
        if (token + 1 >= valid[i]) w[i] &= 0xffffu;  // (what lies behind the context may be anything)
        most = max_u16x2(most, w[i]);
    }
    if (!all_small(most)) return false;
#pragma unroll
    for (int i = 0; i < kSubs; ++i)
        if (lane < 2 * kWords && token < valid[i])
            *reinterpret_cast<uint32_t*>(at[i] + lane / kWords * second + Unit<kGroups>::kValueScales + lane % kWords * 4) =
                hmul2(w[i], kLift2);
    __syncwarp();
    return true;
}

// Up to kSubs tiles into a warp's state: unit 0 of tile i at `at[i]`, unit 1 `second`
// bytes behind it; valid[i] of its 16 tokens count, and at least one in all.
// kWhole: all of them do, and with no branch between them the tiles' products and
// loads overlap.
template <int kGroups, bool kWhole>
__device__ __forceinline__ void add_tiles(uint8_t* const (&at)[kSubs], const int (&valid)[kSubs], int second,
                                          const Queries<kGroups>& q, State<kGroups>& st, int lane) {
    using U = Unit<kGroups>;
    const int r = lane >> 2, c = lane & 3;
    float x[kSubs][4];
#pragma unroll
    for (int i = 0; i < kSubs; ++i) {
        x[i][0] = x[i][1] = x[i][2] = x[i][3] = -INFINITY;
        if (!kWhole && valid[i] <= 0) continue;
        uint8_t* u0 = at[i];
        uint8_t* u1 = u0 + second;
        if (!kWhole && valid[i] < kTok) {
            // scales and minima behind the context, which may be anything, are zeros to the values' products
            if (lane >= valid[i] && lane < kTok) {
                uint8_t* unit = lane < kUnit ? u0 : u1;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    *reinterpret_cast<uint16_t*>(unit + U::kValueScales + (g * kUnit + lane % kUnit) * 2) = 0;
                    *reinterpret_cast<uint16_t*>(unit + U::kValueMins + (g * kUnit + lane % kUnit) * 2) = 0;
                }
            }
            __syncwarp();
        }
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
            st.scales = max_u16x2(st.scales, max_u16x2(lds32(u0 + U::kValueScales + (g * kUnit + 2 * c) * 2),
                                                 lds32(u1 + U::kValueScales + (g * kUnit + 2 * c) * 2)));
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) x[i][h] = t[h] * q.factor[h & 1];
        if (!kWhole && valid[i] < kTok) {
            if (r >= valid[i]) x[i][0] = x[i][1] = -INFINITY;
            if (kUnit + r >= valid[i]) x[i][2] = x[i][3] = -INFINITY;
        }
    }

    // ---- running maximum, and the scale of the weights ----
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < kSubs; ++i) top[h] = fmaxf(top[h], fmaxf(x[i][h], x[i][h + 2]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], d));
    }
    // the first scale of 32 (in fp16) makes the weights smaller, those before it too
    float offset = 10.f, less = 0.f;
    if (__any_sync(0xffffffffu, (st.scales & 0xffffu) >= 0x5000u || (st.scales >> 16) >= 0x5000u)) {
        offset = 2.f;
        if (__any_sync(0xffffffffu, ~st.scales != 0u)) less = 8.f;
        st.scales = ~0u;  // from now on
    }
    // rounded up: where fp32 numbers are 16 apart (tops of 2^27 and more), one below the
    // difference would have the largest weight 2^16, which is none in fp16
    const float base[2] = {fmaxf(__fadd_ru(st.base[0], less), __fsub_ru(top[0], offset)),
                           fmaxf(__fadd_ru(st.base[1], less), __fsub_ru(top[1], offset))};
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
    st.base[0] = base[0];
    st.base[1] = base[1];

    // ---- values ----
#pragma unroll
    for (int i = 0; i < kSubs; ++i) {
        if (!kWhole && valid[i] <= 0) continue;
        const uint8_t* u0 = at[i];
        const uint8_t* u1 = u0 + second;
        const uint32_t p0 = transposed(pack_f16x2(ex2(x[i][0] - base[0]), ex2(x[i][1] - base[1])));
        const uint32_t p1 = transposed(pack_f16x2(ex2(x[i][2] - base[0]), ex2(x[i][3] - base[1])));
        uint32_t m0 = 0, m1 = 0;
        if (r < kGroups) {
            m0 = lds32(u0 + U::kValueMins + (r * kUnit + 2 * c) * 2);
            m1 = lds32(u1 + U::kValueMins + (r * kUnit + 2 * c) * 2);
        } else if (r == kGroups) {
            m0 = m1 = 0x3c003c00u;  // ones
        }
        float e[4] = {st.e[0], st.e[1], 0.f, 0.f};  // (rows 8 to 15 are zeros)
        mma(e, m0, 0u, m1, 0u, p0, p1);
        st.e[0] = e[0];
        st.e[1] = e[1];
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
__device__ __forceinline__ float* partial(const Decode& p, int cta, int last, int row) {
    return p.partials + ((static_cast<size_t>(cta) * 2 + (cta == last ? 0 : 1)) * p.rows + row) * kORow;
}

// `count` (at most 32) partial results of rows row, row + step, ... (`rows` of them),
// `stride` CTAs apart from CTA `first` on, combined; emit(row, four dims from 4 lane
// on, max, sum). Lane k holds partial result k's maxima and sums of all rows, which
// come first; then six results of four rows are on their way at a time (256
// sequences: 546 us, 553 with four, which leaves the kernel's other values less room
// in registers).
template <class Emit>
__device__ __forceinline__ void combine(const Decode& p, int first, int stride, int count, int last, int row, int step, int rows,
                                        int lane, Emit emit) {
    constexpr int kAhead = 6, kAbreast = 4;
    const int cta = first + min(lane, count - 1) * stride;
#pragma unroll 1
    for (int j = 0; j < rows; j += kAbreast) {
        float2 ml[kAbreast];
#pragma unroll
        for (int h = 0; h < kAbreast; ++h)
            ml[h] = __ldcg(reinterpret_cast<const float2*>(partial(p, cta, last, row + min(j + h, rows - 1) * step) + kDim));
        float M[kAbreast], L[kAbreast], weight[kAbreast];
        float4 acc[kAbreast];
#pragma unroll
        for (int h = 0; h < kAbreast; ++h) {
            M[h] = lane < count ? ml[h].x : -INFINITY;
#pragma unroll
            for (int d = 16; d; d >>= 1) M[h] = fmaxf(M[h], __shfl_xor_sync(0xffffffffu, M[h], d));
            weight[h] = lane < count ? ex2(ml[h].x - M[h]) : 0.f;
            L[h] = lane < count ? weight[h] * ml[h].y : 0.f;
#pragma unroll
            for (int d = 16; d; d >>= 1) L[h] += __shfl_xor_sync(0xffffffffu, L[h], d);
            acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int n = 0; n < count; n += kAhead) {
            float4 o[kAhead][kAbreast];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
#pragma unroll
                for (int h = 0; h < kAbreast; ++h)
                    o[k][h] = __ldcg(reinterpret_cast<const float4*>(partial(p, first + min(n + k, count - 1) * stride, last,
                                                                             row + min(j + h, rows - 1) * step) + 4 * lane));
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (n + k >= count) break;
#pragma unroll
                for (int h = 0; h < kAbreast; ++h) {
                    const float f = __shfl_sync(0xffffffffu, weight[h], n + k);
                    acc[h] = make_float4(fmaf(f, o[k][h].x, acc[h].x), fmaf(f, o[k][h].y, acc[h].y), fmaf(f, o[k][h].z, acc[h].z),
                                         fmaf(f, o[k][h].w, acc[h].w));
                }
            }
        }
        __syncwarp();  // every lane's reads, before what emit() may put in their place
#pragma unroll
        for (int h = 0; h < kAbreast; ++h)
            if (j + h < rows) emit(row + (j + h) * step, acc[h], M[h], L[h]);
    }
}

// A row from the results of the warps that share its head, `stride` floats apart:
// four dims from 4 lane on. (All loads at once: 200 sequences of one KV head 18.3 us,
// 18.9 one after the other.)
struct Row {
    float4 o;
    float max, sum;
};
__device__ __forceinline__ Row of_parts(const float* state, int stride, int parts, int lane) {
    float2 ml[kWarps];
    float4 v[kWarps];
    Row x = {make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
        const float* src = state + min(k, parts - 1) * stride;
        ml[k] = *reinterpret_cast<const float2*>(src + kDim);
        v[k] = *reinterpret_cast<const float4*>(src + 4 * lane);
        x.max = fmaxf(x.max, ml[k].x);
    }
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
        if (k >= parts || ml[k].y == 0.f) continue;  // a part without tokens
        const float f = ex2(ml[k].x - x.max);
        x.sum = fmaf(f, ml[k].y, x.sum);
        x.o = make_float4(fmaf(f, v[k].x, x.o.x), fmaf(f, v[k].y, x.o.y), fmaf(f, v[k].z, x.o.z), fmaf(f, v[k].w, x.o.w));
    }
    return x;
}

__device__ __forceinline__ uint2 rounded(float4 o, float inv) {
    return make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

// kShared: runs of fewer than kWarps heads, whose warps share them. (Compiled apart, since
// either takes the registers that the other would have: 200 sequences of one KV head 19.4
// us, 20.5 in one kernel, 64 of two 26.0 and 27.1; 256 of 8 heads 547 in both.)
template <int kGroups, bool kShared, class Params>
__global__ void __launch_bounds__(kThreads, 2) decode_kernel(const Params p) {
    using U = Unit<kGroups>;
    using L = Smem<kGroups>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = p.num_seqs, runs = p.runs;
    const int heads = kShared ? p.heads : kWarps;
    const int parts = kWarps / heads, tile_tokens = kTok * parts;  // warps of a head, tokens of a tile
    int* scan = reinterpret_cast<int*>(smem + L::kScan);
    int* misc = reinterpret_cast<int*>(smem + L::kMisc);
    volatile int* abort_flag = misc;
    int* ends = misc + 1;
    int* first_piece = misc + 3;  // sequence (or -1), run, tile, place on the line
    int* warp_total = misc + 7;
    static_assert(7 + kThreads / 32 <= 16, "the warps' totals fit");
    const uint32_t bar0 = smem_u32(smem + L::kBars);
    auto full_bar = [&](int i) { return bar0 + 8u * i; };
    auto empty_bar = [&](int i) { return bar0 + 8u * (kStages + i); };
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full_bar(i), 1);
            mbar_init(empty_bar(i), kWarps);
        }
        misc[0] = 0;
        first_piece[0] = -1;
        fence_barrier_init();
    }
    // Launched early, behind kernels that may write what is read from here on.
    griddep_launch_dependents();
    griddep_wait();

    // ---- plan: prefix sums of the runs' tiles, then this CTA's range ----
    // Tile x of run i = s * runs + g sits at cost position x + kRunCost * i; a
    // CTA takes the tiles of an equal share of positions. An end of its range is
    // found by the thread that holds the sequence.
    const int per = (B + kThreads - 1) / kThreads;
    const int lo = min(B, tid * per), hi = min(B, lo + per);
    const int tile_shift = 31 - __clz(tile_tokens);
    int local = 0;
    for (int s = lo; s < hi; ++s) {
        const int n = __ldg(p.context_lens + s);
        if (n > p.cap) atomicOr(p.err, PKV_DEVERR_CONTEXT);
        local += (max(min(n, p.cap), 0) + tile_tokens - 1) >> tile_shift;
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
    const int cost = runs * (tiles + kRunCost * B);
    const int share = (cost + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    for (int s = lo, start = before; s < hi; ++s) {
        const int end = before + scan[s], nb = end - start;
        scan[s] = end;
        const int c0 = runs * (start + kRunCost * s), c1 = c0 + runs * (nb + kRunCost);
        const int y0 = static_cast<int>(blockIdx.x) * share, y1 = y0 + share;
        // the first tile at or behind cost position y, within this sequence: its run and its place in it
        auto tile_at = [&](int y, int& g) {
            g = attn::div_small(y - c0, nb + kRunCost);
            return min(y - c0 - g * (nb + kRunCost), nb);
        };
        int g, at;
        if (y0 >= c0 && y0 < c1) {
            at = tile_at(y0, g);
            ends[0] = runs * start + g * nb + at;
        }
        if (y1 >= c0 && y1 < c1) {
            at = tile_at(y1, g);
            const int end_tile = runs * start + g * nb + at;
            ends[1] = end_tile;
            // The walk's first piece is the part of the range in the run that holds
            // its last tile; where that is this sequence's, nobody searches for it.
            if (at == 0) --g;
            if (nb > 0 && g >= 0) {
                const int seg = runs * start + g * nb;
                int split = seg, g0;
                if (y0 >= c0) {
                    const int in_run = tile_at(y0, g0);
                    split = max(seg, runs * start + g0 * nb + in_run);
                }
                if (split < end_tile) {
                    first_piece[0] = s;
                    first_piece[1] = g;
                    first_piece[2] = split - seg;
                    first_piece[3] = split;
                }
            }
        }
        start = end;
    }
    if (tid < 2 && (static_cast<int>(blockIdx.x) + tid) * share >= cost) ends[tid] = runs * tiles;
    __syncthreads();
    const int range_lo = ends[0], range_hi = ends[1];

    // sequences without a context: zero rows
    for (int s = blockIdx.x; s < B; s += gridDim.x) {
        if (attn::run_blocks(scan, s) != 0) continue;
        uint4* row = reinterpret_cast<uint4*>(p.out + static_cast<size_t>(s) * p.hq * kDim);
        for (int i = tid; i < p.hq * kDim / 8; i += kThreads) row[i] = make_uint4(0, 0, 0, 0);
    }
    if (range_lo >= range_hi) return;

    attn::Piece pc;
    const bool blocks_of_8 = p.bt_shift == 3;
    if (warp >= kWarps) {
        // ====================== producer warps =======================
        // Lanes look up where a round of copies come from, each tile's then go out
        // from one thread, chosen by elect.sync: knowing it to be one, the compiler
        // hands a copy its operands at once.
        attn::PieceWalk walk(scan, B, runs, range_lo, range_hi, first_piece);
        const uint64_t policy = policy_evict_first();
        const int ahead = 32 / p.copies;  // tiles whose copies' places the lanes hold
        const uint32_t unit_row = static_cast<uint32_t>(heads) * U::kBytes;  // a unit of every head of the run
        int gi = 0, last_issued = -1;
        while (walk.next(pc)) {
            const int ctx = min(__ldg(p.context_lens + pc.s), p.cap);
            const int32_t* row = p.tables + static_cast<size_t>(pc.s) * p.width;
            for (int j0 = 0; j0 < pc.len; j0 += ahead) {
                const int n = min(ahead, pc.len - j0);
                const int token = (pc.blk + j0) * tile_tokens + lane * p.copy_tokens;
                uint64_t src = 0;
                if (lane < n * p.copies && token < ctx) {
                    int id = __ldg(row + (token >> p.bt_shift));
                    if (id < 0 || id >= p.num_blocks) {
                        atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
                        id = 0;  // a valid block in its place; the output is flagged invalid
                    }
                    const long long slot = (static_cast<long long>(id) << p.bt_shift) + (token & ((1 << p.bt_shift) - 1));
                    src = reinterpret_cast<uint64_t>(p.cache) + unit_of(slot, pc.g * heads, p.hkv, blocks_of_8) * U::kBytes;
                }
                for (int j = 0; j < n; ++j, ++gi) {
                    if (gi % kProducers != warp - kWarps || stopped(p, gi)) continue;
                    const int st = gi % kStages;
                    // whole slabs: 16 tokens (8 in blocks of 8)
                    const int left = min(tile_tokens, ctx - (pc.blk + j0 + j) * tile_tokens);
                    const uint32_t slabs = blocks_of_8 ? (left + 7) >> 3 : (left + 15) >> 4;
                    const uint32_t slab_bytes = blocks_of_8 ? unit_row : 2 * unit_row;
                    const uint32_t bytes = slabs * slab_bytes, copy_bytes = p.copy_tokens / 8 * unit_row;
                    const uint32_t full = full_bar(st), dst = smem_u32(smem + st * L::kStage);
                    const bool ok = mbar_wait(empty_bar(st), static_cast<uint32_t>((gi / kStages) & 1) ^ 1u, abort_flag, p.err);
                    if (!__all_sync(0xffffffffu, ok)) continue;
                    last_issued = gi;
                    if (elect_one()) mbar_arrive_expect_tx(full, bytes);
                    for (uint32_t at = 0, i = j * p.copies; at < bytes; at += copy_bytes, ++i) {
                        const uint64_t a = __shfl_sync(0xffffffffu, src, i);
                        if (elect_one()) bulk_load(dst + at, reinterpret_cast<const void*>(a), min(bytes - at, copy_bytes), full, policy);
                    }
                }
            }
        }
        // No copy may land after the CTA has ended. Without an abort every copy
        // was waited for by its consumers and these waits return at once; after
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

    // ======================= consumer warps =======================
    // The walk stays in shared memory between pieces: the registers are the sums'. (128
    // sequences of 8,000 tokens, 32 turns held: 224 us, 227 without.)
    attn::PieceWalk* place = reinterpret_cast<attn::PieceWalk*>(smem + L::kWalks + warp * 64);
    static_assert(sizeof(attn::PieceWalk) <= 64, "a walk fits its place");
    {
        const attn::PieceWalk walk(scan, B, runs, range_lo, range_hi, first_piece);
        if (lane == 0) *place = walk;
        __syncwarp();
    }
    const int r = lane >> 2, c = lane & 3;
    const int head = warp & (heads - 1), part = warp / heads;
    // the warp's two units in a stage
    const int second = blocks_of_8 ? heads * U::kBytes : U::kBytes;
    const int own = blocks_of_8 ? (part * 2 * heads + head) * U::kBytes : (part * heads + head) * 2 * U::kBytes;
    float* states = reinterpret_cast<float*>(smem + L::kStates);
    float4* kept = reinterpret_cast<float4*>(states + warp * kKeptFloats * 32) + lane;
    const int cta = static_cast<int>(blockIdx.x);
    int gidx = 0;
    while (true) {
        attn::PieceWalk walk = *place;
        __syncwarp();
        if (!walk.next(pc)) break;  // (the whole warp)
        if (lane == 0) *place = walk;
        __syncwarp();
        const int s = pc.s, nb = pc.nb;
        const int ctx = min(__ldg(p.context_lens + s), p.cap);
        Queries<kGroups> q;
        q.load(p, s, pc.g * heads + head, r, c);
        State<kGroups> st;
        st.clear();
        const int left = ctx - pc.blk * tile_tokens - part * kTok;  // of the context, from the warp's first token on
        bool some = false;  // whether the warp has tokens of the piece
        // The piece's tiles from j to `stop`; false, with the last ones not yet given back,
        // where they are for the other kind of turn: the first ones, if their scales are all small,
        // are taken again with lifted scales (`lift`), until there is one that is not. (One
        // loop for both, with a branch: 256 sequences 565 us, 547 with two.)
        int j = 0, stop = 0;
        auto tiles = [&](auto lift) {
            for (; j < stop; j += kSubs) {
                const int n = min(kSubs, stop - j);
                uint8_t* at[kSubs];
                int valid[kSubs];
                bool landed = true, any = false, whole = true;
#pragma unroll
                for (int i = 0; i < kSubs; ++i) {
                    const int gi = gidx + j + i;
                    at[i] = smem + gi % kStages * L::kStage + own;
                    valid[i] = i < n ? min(kTok, left - (j + i) * tile_tokens) : 0;
                    any |= valid[i] > 0;
                    whole &= valid[i] == kTok;
                    if (i < n) landed &= mbar_wait(full_bar(gi % kStages), static_cast<uint32_t>((gi / kStages) & 1), abort_flag, p.err);
                }
                const bool first = any && !some;
                some |= any;
                if (decltype(lift)::value) {
                    if (any) {
                        if (!lift_tiles<kGroups>(at, valid, second, lane)) return false;
                        add_tiles<kGroups, false>(at, valid, second, q, st, lane);
                    }
                } else if (any) {
                    if (whole) add_tiles<kGroups, true>(at, valid, second, q, st, lane);
                    else add_tiles<kGroups, false>(at, valid, second, q, st, lane);
                    if (first && all_small(st.scales)) return false;
                }
                fence_proxy_async_shared();  // this lane's accesses of the stages, before the copies that will replace them
                __syncwarp();
                if (lane < n && landed) mbar_arrive(empty_bar((gidx + j + lane) % kStages));
            }
            return true;
        };
        bool lifted = false;
        while (true) {
            stop = min(stop + kHold * kSubs, pc.len);
            while (lifted ? !tiles(std::true_type()) : !tiles(std::false_type())) {
                if (lifted) st.unlift();
                else st.clear();
                lifted = !lifted;
            }
            if (__builtin_expect(lifted, 0)) st.unlift();
            if (__builtin_expect(stop > kHold * kSubs, 0)) st.add_kept(kept);
            if (__builtin_expect(stop == pc.len, 1)) break;
            if (stop == kHold * kSubs && kShared) named_barrier_sync(1, kConsumers);  // all have read the last piece's states
            st.keep(kept);
        }
        gidx += pc.len;

        // ---- the piece's result, row by row ----
        const int seg = runs * (scan[s] - nb) + pc.g * nb + kRunCost * (s * runs + pc.g);
        const int i0 = seg / share, i1 = (seg + nb - 1) / share, pieces = i1 - i0 + 1;
        __nv_bfloat16* out = p.out + (static_cast<size_t>(s) * p.hq + static_cast<size_t>(pc.g) * p.rows) * kDim;
        // rows of this warp from here on: its head's, or every fourth of the run's
        int row = head * p.group, step = 1, rows = p.group;
        float mins[kGroups][2], sums[2];
        st.rows(c, mins, sums);
        if (!kShared) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (2 * c + h >= p.group) continue;
                const int mine = row + 2 * c + h;
                if (pieces == 1) {
                    const float inv = 1.f / sums[h];
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        *reinterpret_cast<uint2*>(out + mine * kDim + 32 * w + 4 * r) = rounded(st.row(w, h, mins), inv);
                } else {
                    float* dst = partial(p, cta, i1, mine);
#pragma unroll
                    for (int w = 0; w < 4; ++w) *reinterpret_cast<float4*>(dst + 32 * w + 4 * r) = st.row(w, h, mins);
                    if (r == 0) {
                        dst[kDim] = st.base[h];
                        dst[kDim + 1] = sums[h];
                    }
                }
            }
        } else {
            // the warps of a head through shared memory; all have read the last piece's states
            named_barrier_sync(1, kConsumers);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* dst = states + (warp * kMaxG + 2 * c + h) * kORow;
#pragma unroll
                for (int w = 0; w < 4; ++w) *reinterpret_cast<float4*>(dst + 32 * w + 4 * r) = st.row(w, h, mins);
                if (r == 0) {
                    dst[kDim] = some ? st.base[h] : -INFINITY;
                    dst[kDim + 1] = some ? sums[h] : 0.f;
                }
            }
            named_barrier_sync(1, kConsumers);
            row = warp;
            step = kWarps;
            rows = (p.rows - warp + kWarps - 1) / kWarps;
            for (int j = 0; j < rows; ++j) {
                const int mine = row + j * step, of = mine / p.group, h = mine - of * p.group;
                const Row x = of_parts(states + (of * kMaxG + h) * kORow, heads * kMaxG * kORow, parts, lane);
                if (pieces == 1) {
                    reinterpret_cast<uint2*>(out + mine * kDim)[lane] = rounded(x.o, 1.f / x.sum);
                } else {
                    float* dst = partial(p, cta, i1, mine);
                    *reinterpret_cast<float4*>(dst + 4 * lane) = x.o;
                    if (lane == 0) {
                        dst[kDim] = x.max;
                        dst[kDim + 1] = x.sum;
                    }
                }
            }
        }
        if (pieces == 1) continue;

        // ---- a run that is cut: the last of the warps with these rows combines them ----
        auto last = [&](unsigned long long* ctr, int count) {
            __syncwarp();  // every lane's stores, before lane 0's release
            uint64_t old = 0;
            if (lane == 0) {
                old = atom_add_acq_rel_gpu(ctr, uint64_t(1) << (8 * warp));
                old = (old >> (8 * warp)) & 255u;
                if (static_cast<int>(old) == count - 1)  // ready for the next launch
                    atomicAdd(ctr, 0ull - (static_cast<unsigned long long>(count) << (8 * warp)));
            }
            const int seen = __shfl_sync(0xffffffffu, static_cast<int>(old), 0);
            __syncwarp();
            return seen == count - 1;
        };
        int stride = 1;
        if (pieces > kMergeGroup) {
            stride = kMergeGroup;
            const int base = i0 + (cta - i0) / kMergeGroup * kMergeGroup;
            const int count = min(kMergeGroup, i1 - base + 1);
            if (count > 1) {  // else a lone piece, its group's result already
                if (!last(p.group_counters + base, count)) continue;
                combine(p, base, 1, count, i1, row, step, rows, lane, [&](int i, float4 o, float m, float l) {
                    float* dst = partial(p, base, i1, i);
                    *reinterpret_cast<float4*>(dst + 4 * lane) = o;
                    if (lane == 0) {
                        dst[kDim] = m;
                        dst[kDim + 1] = l;
                    }
                });
            }
        }
        const int count = (pieces + stride - 1) / stride;
        if (!last(p.counters + i0, count)) continue;
        combine(p, i0, stride, count, i1, row, step, rows, lane, [&](int i, float4 o, float, float l) {
            reinterpret_cast<uint2*>(out + i * kDim)[lane] = rounded(o, 1.f / l);
        });
    }
}

}  // namespace kv4
}  // namespace pkv
