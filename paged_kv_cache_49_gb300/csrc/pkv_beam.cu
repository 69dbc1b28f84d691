// Beam selection: of every group of beams, the best continuations over the
// vocabulary, and the beams' token histories behind them.
//
// For beam k of a group, with running score s_k and logits x_k:
//   candidate (k, v) has the score s_k + x_kv - log sum_v exp x_kv
// (a finished beam: the one candidate (k, eos) with score s_k), and the best n of
// a group's are taken, equal ones in the order of k * vocab + v.
//
// Two launches. The scan reads each logit once: a CTA holds a chunk of a row in
// registers, and leaves its maximum, the sum of its exponentials and its n
// largest logits. These come without a sort: of the 8 warps' threads' maxima,
// each warp's ceil(n / 8)-th largest is known after as many warp reductions; at
// least n logits of the chunk reach the least of these 8, and hardly more do, so
// those that reach it go into a list whose entries are ranked by comparing them
// all. (A list that overflows, as of equal logits, is replaced by n rounds over
// the chunk.) The join merges the chunks' lists of a group by scores of twice
// fp32's precision: neighbours of the last one taken may differ by less than
// fp32 holds. The exponentials bound the scan from the other side:
// at 16 a cycle and SM they take two thirds of the time of reading bf16 logits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace beam {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBeams = PKV_BEAM_MAX_BEAMS;
constexpr int kMaxCandidates = PKV_BEAM_MAX_CANDIDATES;
constexpr int kList = 512;     // candidates that are ranked
constexpr int kMaxVectors = 8;  // 16-byte vectors a thread holds
// Chunks are made smaller (fewer vectors a thread) while this many CTAs are not reached.
constexpr int kWantCtas = 304;

struct Params {
    const void* logits;
    int64_t row_stride;  // elements
    const float* scores;
    const uint8_t* finished;
    const int32_t* history;
    const int32_t* lengths;
    float* scores_out;
    int32_t* tokens_out;
    int32_t* parents_out;
    uint8_t* finished_out;
    int32_t* lengths_out;
    int32_t* history_out;
    float2* stats;  // [rows][chunks][kWarps]: maximum, sum of exponentials from it on
    uint2* lists;   // [rows][chunks][n]: logit bits, token (or -1)
    uint32_t* err;
    int eos, beams, n, vocab, max_length, chunks;
};

constexpr float kLog2e = 1.4426950408889634f;

// A beam that is read: neither finished nor without a score.
__device__ __forceinline__ bool row_done(const Params& p, int row) { return p.finished && p.finished[row] != 0; }
__device__ __forceinline__ bool row_live(const Params& p, int row) { return !row_done(p, row) && p.scores[row] > -INFINITY; }

// Numbers that compare as unsigned integers as the keys do as floats (-0 as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }
// A number as the sum of two, the second below half a step of the first: 48 bits
// or more from fp32 operations (64-bit ones run at 1/64 of their rate here).
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair add(Pair a, float b) {
    const Pair s = two_sum(a.hi, b);
    return two_sum(s.hi, __fadd_rn(s.lo, a.lo));
}
__device__ __forceinline__ Pair add(Pair a, Pair b) { return add(add(a, b.hi), b.lo); }
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    const float p = __fmul_rn(a.hi, b.hi);
    return two_sum(p, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.hi, -p))));
}

// ---- selection from a chunk ------------------------------------------------------

// A candidate: its key in order, and its index; of equal keys the lower index
// comes first.
struct Candidate {
    uint64_t key;
    int at;
    int pad;
};

__device__ __forceinline__ bool before(uint64_t ka, int ia, uint64_t kb, int ib) { return ka > kb || (ka == kb && ia < ib); }

struct Selection {
    Candidate list[kList];
    uint32_t warp_key[kWarps];
    Candidate warp_best[kWarps];
    int count;
};

// The least, over the warps, of each warp's ceil(n / 8)-th largest thread key:
// at least n keys of the block reach it (or all that are above -inf).
__device__ __forceinline__ float threshold(Selection& sel, float best, int n) {
    uint32_t mine = ordered(best), top = 0;
    for (int i = 0; i < (n + kWarps - 1) / kWarps; ++i) {
        top = __reduce_max_sync(0xffffffffu, mine);
        const unsigned holders = __ballot_sync(0xffffffffu, mine == top);
        if ((threadIdx.x & 31) == __ffs(holders) - 1) mine = 0;
    }
    if (threadIdx.x == 0) sel.count = 0;
    if ((threadIdx.x & 31) == 0) sel.warp_key[threadIdx.x >> 5] = max(top, ordered(-INFINITY));
    __syncthreads();
    uint32_t t = sel.warp_key[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) t = min(t, sel.warp_key[w]);
    return unordered(t);
}

__device__ __forceinline__ void offer(Selection& sel, uint64_t key, int at) {
    const int i = atomicAdd(&sel.count, 1);
    if (i < kList) *reinterpret_cast<uint4*>(&sel.list[i]) = make_uint4(static_cast<uint32_t>(key), static_cast<uint32_t>(key >> 32), at, 0);
}

// Writes the n first of the list in order to put(rank, key, at), the missing
// ones as (0, -1); where the list overflowed, finds them by n rounds over items
// 0 .. items - 1, item(i, key, at) being false for no candidate.
template <class Item, class Put>
__device__ __forceinline__ void finish(Selection& sel, int n, int items, Item item, Put put) {
    __syncthreads();
    const int count = sel.count;
    if (count <= kList) {
        for (int i = threadIdx.x; i < count; i += kThreads) {
            const Candidate c = sel.list[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < count; ++j) {
                const uint4 u = *reinterpret_cast<const uint4*>(&sel.list[j]);
                rank += before(static_cast<uint64_t>(u.y) << 32 | u.x, static_cast<int>(u.z), c.key, c.at);
            }
            if (rank < n) put(rank, c.key, c.at);
        }
        for (int i = count + threadIdx.x; i < n; i += kThreads) put(i, uint64_t(0), -1);
        return;
    }
    uint64_t last = ~uint64_t(0);
    int last_at = -1;
    for (int j = 0; j < n; ++j) {
        uint64_t best = 0;
        int best_at = INT_MAX;
        for (int i = threadIdx.x; i < items; i += kThreads) {
            uint64_t k;
            int at;
            if (item(i, k, at) && before(last, last_at, k, at) && before(k, at, best, best_at)) {
                best = k;
                best_at = at;
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const uint64_t k = __shfl_xor_sync(0xffffffffu, best, d);
            const int at = __shfl_xor_sync(0xffffffffu, best_at, d);
            if (before(k, at, best, best_at)) {
                best = k;
                best_at = at;
            }
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sel.warp_best[threadIdx.x >> 5] = {best, best_at, 0};
        __syncthreads();
        last = sel.warp_best[0].key;
        last_at = sel.warp_best[0].at;
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            if (before(sel.warp_best[w].key, sel.warp_best[w].at, last, last_at)) {
                last = sel.warp_best[w].key;
                last_at = sel.warp_best[w].at;
            }
        if (threadIdx.x == 0) put(j, last, last_at);  // kList > n candidates are there
    }
}

// ---- scan -----------------------------------------------------------------------

template <class T>
struct Vector;  // 16 bytes of logits
template <>
struct Vector<__nv_bfloat16> {
    static constexpr int kN = 8;
    uint32_t u[4];
    __device__ __forceinline__ void fill() { u[0] = u[1] = u[2] = u[3] = 0xff80ff80u; }  // -inf
    __device__ __forceinline__ void set(int e, __nv_bfloat16 x) {
        const uint32_t v = __bfloat16_as_ushort(x);
        u[e / 2] = e & 1 ? (u[e / 2] & 0xffffu) | v << 16 : (u[e / 2] & 0xffff0000u) | v;
    }
    __device__ __forceinline__ float get(int e) const { return e & 1 ? bf16_hi(u[e / 2]) : bf16_lo(u[e / 2]); }
    // the largest value (NaN passed over), pairs at a time
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ __forceinline__ float largest() const {
        const uint32_t m = max2(max2(u[0], u[1]), max2(u[2], u[3]));
        return fmaxf(bf16_lo(m), bf16_hi(m));
    }
};
template <>
struct Vector<float> {
    static constexpr int kN = 4;
    uint32_t u[4];
    __device__ __forceinline__ void fill() { u[0] = u[1] = u[2] = u[3] = 0xff800000u; }
    __device__ __forceinline__ void set(int e, float x) { u[e] = __float_as_uint(x); }
    __device__ __forceinline__ float get(int e) const { return __uint_as_float(u[e]); }
    __device__ __forceinline__ float largest() const { return fmaxf(fmaxf(get(0), get(1)), fmaxf(get(2), get(3))); }
};

// kN logits from token `at` on, -inf behind the row's end. Which logits a thread
// sums is a matter of their tokens alone, so rows that are alike have the same
// sums wherever they lie: a row that does not begin on a 16-byte boundary is read
// in words (for bf16 rows on odd places, shifted by half a word); logits whose
// words reach beyond the row are read one by one.
template <class T>
__device__ __forceinline__ Vector<T> load(const T* row, int at, int vocab, unsigned shift) {
    constexpr int kN = Vector<T>::kN;
    Vector<T> v;
    if (shift == 0 && at + kN <= vocab) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + at));
        v.u[0] = u.x, v.u[1] = u.y, v.u[2] = u.z, v.u[3] = u.w;
    } else if (shift != 0 && shift % 4 == 0 && at + kN <= vocab) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v.u[i] = __ldg(reinterpret_cast<const uint32_t*>(row + at) + i);
    } else if (shift % 4 != 0 && at >= kN && at + kN < vocab) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(row + at - 1);
        uint32_t w[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = __ldg(src + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.u[i] = __funnelshift_r(w[i], w[i + 1], 16);
    } else {
        v.fill();
#pragma unroll
        for (int e = 0; e < kN; ++e)
            if (at + e < vocab) v.set(e, row[at + e]);
    }
    return v;
}

// CTA (row, chunk).
template <class T, int kVectors>
__global__ void __launch_bounds__(kThreads, 4) scan_kernel(const Params p) {
    constexpr int kN = Vector<T>::kN;
    const int row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks;
    if (!row_live(p, row)) return;
    __shared__ Selection sel;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T* logits = static_cast<const T*>(p.logits) + row * p.row_stride;
    const unsigned shift = static_cast<unsigned>(reinterpret_cast<uintptr_t>(logits) & 15u);
    const int first = (chunk * kVectors * kThreads + threadIdx.x) * kN;  // token of the thread's first logit
    Vector<T> v[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) v[i] = load(logits, first + i * kThreads * kN, p.vocab, shift);
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVectors; ++i) best = fmaxf(best, v[i].largest());
    // Each warp sums from its own largest logit on, with no barrier before it:
    // sum 2^(x log2(e) - from), whose only error beside the sum's is that of the
    // fp32 constant, by which the join divides again. A NaN makes the row's sum
    // NaN, and then none of its scores is a number.
    const int lo = chunk * kVectors * kThreads * kN, hi = min(lo + kVectors * kThreads * kN, p.vocab);
    const float top = unordered(__reduce_max_sync(0xffffffffu, ordered(best)));
    const float from = top > -INFINITY ? top * kLog2e : 0.f;
    float sum = 0.f;
    if (fabsf(from) < INFINITY || fabsf(top) == INFINITY) {
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
#pragma unroll
            for (int e = 0; e < kN; ++e) part[e % 4] += ex2(fmaf(v[i].get(e), kLog2e, -from));
        sum = (part[0] + part[1]) + (part[2] + part[3]);
    } else {  // logits of more than 2e38
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
#pragma unroll 1
            for (int e = 0; e < kN; ++e) {
                const int at = first + i * kThreads * kN + e;
                if (at < p.vocab) sum += ex2((static_cast<float>(logits[at]) - top) * kLog2e);
            }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const size_t out = static_cast<size_t>(row) * p.chunks + chunk;
    if (lane == 0) p.stats[out * kWarps + warp] = make_float2(top, sum);
    const float cut = threshold(sel, best, p.n);
    if (best >= cut && best > -INFINITY) {
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            if (!(v[i].largest() >= cut)) continue;
            // the vector's logits that reach the cut, as bits, and then one by one
            unsigned hits = 0;
#pragma unroll
            for (int e = 0; e < kN; ++e)
                if (v[i].get(e) >= cut) hits |= 1u << e;
#pragma unroll 1
            for (; hits; hits &= hits - 1) {
                const int at = first + i * kThreads * kN + __ffs(static_cast<int>(hits)) - 1;
                const float x = at < p.vocab ? static_cast<float>(logits[at]) : -INFINITY;
                if (x > -INFINITY) offer(sel, ordered(x), at);
            }
        }
    }
    griddep_launch_dependents();  // the join's CTAs need not take room before
    uint2* list = p.lists + out * p.n;
    finish(
        sel, p.n, hi - lo,
        [&](int i, uint64_t& k, int& at) {
            at = lo + i;
            const float x = static_cast<float>(logits[at]);
            k = ordered(x);
            return x > -INFINITY;
        },
        [&](int rank, uint64_t k, int at) {
            list[rank] = make_uint2(__float_as_uint(unordered(static_cast<uint32_t>(k))), static_cast<uint32_t>(at));
        });
}

// ---- join -----------------------------------------------------------------------

// CTA (group, share): every share of a group finds its best n candidates, and
// writes the results of every gridDim.y-th. The chunks' lists are in order, so
// the candidates are merged: in each of n rounds the best of the lists' first
// remaining entries is taken. (A cut as in the scan's does not bound the list:
// where one beam leads, the best n are in a few chunks, and the other chunks'
// first entries say nothing about them.)
__global__ void __launch_bounds__(kThreads) join_kernel(const Params p) {
    // In quarters, so that no sum of finite ones overflows: the beams' scores and
    // the logarithms of their sums.
    __shared__ float score[kMaxBeams];
    __shared__ Pair lse[kMaxBeams];
    __shared__ bool done[kMaxBeams];
    __shared__ uint4 warp_best[2][kWarps];
    __shared__ float won_score[kMaxCandidates];
    __shared__ int won_at[kMaxCandidates];
    const int group = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = group * p.beams;
    griddep_wait();
    for (int k = warp; k < p.beams; k += kWarps) {
        const int row = row0 + k, parts = p.chunks * kWarps;
        const bool live = row_live(p, row);
        if (lane == 0) {
            score[k] = 0.25f * p.scores[row];
            done[k] = row_done(p, row);
        }
        if (!live) continue;
        const float2* stats = p.stats + static_cast<size_t>(row) * parts;
        float top = -INFINITY;
#pragma unroll 4
        for (int i = lane; i < parts; i += 32) top = fmaxf(top, stats[i].x);
        top = unordered(__reduce_max_sync(0xffffffffu, ordered(top)));
        // a part's sum counts from its largest logit, times the scan's fp32 log2(e)
        const bool large = fabsf(top * kLog2e) == INFINITY;
        float sum = 0.f;
#pragma unroll 4
        for (int i = lane; i < parts; i += 32) {
            const float2 s = stats[i];
            sum += s.y * exp2f(large ? (s.x - top) * kLog2e : __fmul_rn(s.x, kLog2e) - __fmul_rn(top, kLog2e));
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) {
            // log2 of the sum by its exponent and the rest, then by 1 / kLog2e
            const int e = ilogbf(sum);
            const float rest = log2f(ldexpf(sum, -e));
            const Pair by = {0x1.62e43p-1f, 0x1.f8ff94p-28f};
            Pair l;
            if (large) l = two_sum(top, 0.f);
            else l = mul(add(two_sum(__fmul_rn(top, kLog2e), static_cast<float>(e)), rest), by);
            if (!(sum < INFINITY) || !(fabsf(top) < INFINITY)) l.hi = l.lo = NAN;
            lse[k] = {0.25f * l.hi, 0.25f * l.lo};
        }
    }
    __syncthreads();
    // Entry j of list i (a chunk of a beam): its key, 0 for none, and index. A
    // finished beam has one entry in all, whose score is the beam's.
    const int lists = p.beams * p.chunks;
    auto raw = [&](int i, int k, int j) {
        if (!(score[k] > -INFINITY) || j >= p.n) return make_uint2(0u, 0xffffffffu);
        if (done[k]) return make_uint2(0u, i == k * p.chunks && j == 0 ? static_cast<uint32_t>(p.eos) : 0xffffffffu);
        return p.lists[(static_cast<size_t>(row0) * p.chunks + i) * p.n + j];
    };
    auto key_of = [&](int k, uint2 c, int& at) {
        at = k * p.vocab + static_cast<int>(c.y);
        if (static_cast<int>(c.y) < 0) return uint64_t(0);
        const Pair l = lse[k];
        const Pair s = done[k] ? Pair{score[k], 0.f}
                               : add(add(two_sum(0.25f * __uint_as_float(c.x), -l.hi), -l.lo), score[k]);
        if (!(s.hi > -INFINITY && s.hi < INFINITY)) return uint64_t(0);  // (none for NaN)
        return static_cast<uint64_t>(ordered(s.hi)) << 32 | ordered(s.lo);
    };
    // The thread's list with its first remaining entry, and the one behind it;
    // where it has more lists, how far each was taken is counted again from the
    // last one taken, since its own entries are in order.
    uint64_t key = 0, next_key = 0;
    int at = INT_MAX, next_at = INT_MAX, taken = 0;
    const bool single = lists <= kThreads;
    const int list = min(static_cast<int>(threadIdx.x), lists - 1), beam = list / p.chunks;
    if (single && list == threadIdx.x) {
        const uint2 c0 = raw(list, beam, 0), c1 = raw(list, beam, 1);
        key = key_of(beam, c0, at);
        next_key = key_of(beam, c1, next_at);
    }
    uint64_t last = ~uint64_t(0);
    int last_at = -1;
    auto search = [&] {  // the best entry of the thread's lists behind the last one taken
        key = 0;
        at = INT_MAX;
        for (int i = threadIdx.x; i < lists; i += kThreads) {
            const int k = i / p.chunks;
            for (int j = 0; j < p.n; ++j) {
                int a;
                const uint64_t e = key_of(k, raw(i, k, j), a);
                if (e == 0) break;
                if (!before(last, last_at, e, a)) continue;
                if (before(e, a, key, at)) {
                    key = e;
                    at = a;
                }
                break;
            }
        }
    };
    if (!single) search();
    // the first of the warp's keys, and where it is
    auto first_of = [](uint64_t k, int i) {
        const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(k >> 32));
        const bool top = static_cast<uint32_t>(k >> 32) == hi;
        const uint32_t lo = __reduce_max_sync(0xffffffffu, top ? static_cast<uint32_t>(k) : 0u);
        const int first = __reduce_min_sync(0xffffffffu, top && static_cast<uint32_t>(k) == lo ? i : INT_MAX);
        return make_uint4(lo, hi, static_cast<uint32_t>(first), 0u);
    };
    for (int j = 0; j < p.n; ++j) {
        const uint4 u = first_of(key, at);
        if (lane == 0) warp_best[j & 1][warp] = u;
        __syncthreads();
        const uint4 w = warp_best[j & 1][lane % kWarps];
        const uint4 best = first_of(static_cast<uint64_t>(w.y) << 32 | w.x, static_cast<int>(w.z));
        last = static_cast<uint64_t>(best.y) << 32 | best.x;
        last_at = static_cast<int>(best.z);
        if (threadIdx.x == 0) {
            won_score[j] = last ? 4.f * (unordered(best.y) + unordered(best.x)) : -INFINITY;
            won_at[j] = last ? last_at : -1;
        }
        if (last && key == last && at == last_at) {
            if (single) {
                key = next_key;
                at = next_at;
                ++taken;
                next_key = key_of(beam, raw(list, beam, taken + 1), next_at);
            } else {
                search();
            }
        }
    }
    __syncthreads();
    for (int j = blockIdx.y; j < p.n; j += gridDim.y) {
        const int at = won_at[j];
        const bool some = at >= 0;
        const int k = some ? at / p.vocab : -1, token = some ? at - k * p.vocab : -1;
        const int row = row0 + max(k, 0);
        const bool ended = some && done[k];
        const size_t out = static_cast<size_t>(group) * p.n + j;
        int length = 0;
        if (some && p.lengths) {
            const int given = p.lengths[row];
            length = min(max(given, 0), p.max_length);
            if ((given != length || (!ended && length == p.max_length)) && p.err && threadIdx.x == 0)
                atomicOr(p.err, PKV_DEVERR_CONTEXT);
        }
        const bool grows = some && !ended && length < p.max_length;
        if (threadIdx.x == 0) {
            p.scores_out[out] = won_score[j];
            p.tokens_out[out] = token;
            p.parents_out[out] = k;
            p.finished_out[out] = ended || (some && token == p.eos);
            if (p.lengths) p.lengths_out[out] = length + (grows ? 1 : 0);
            if (p.lengths && grows) p.history_out[out * p.max_length + length] = token;
        }
        if (p.lengths) {
            const int32_t* src = p.history + static_cast<size_t>(row) * p.max_length;
            int32_t* dst = p.history_out + out * p.max_length;
#pragma unroll 4
            for (int i = threadIdx.x; i < length; i += kThreads) dst[i] = src[i];
        }
    }
}

// Vectors a thread holds, of a row's `vectors`: as many as leave kWantCtas CTAs.
int vectors_for(long long rows, long long vectors) {
    int v = kMaxVectors;
    while (v > 1 && rows * ((vectors + v * kThreads - 1) / (v * kThreads)) < kWantCtas) v /= 2;
    return v;
}

// Chunks of a row of `vocab` logits of `size` bytes.
int chunks_for(long long rows, int vocab, int size, int* vectors) {
    const int n = 16 / size;
    const long long most = (static_cast<long long>(vocab) + n - 1) / n;
    *vectors = vectors_for(rows, most);
    return static_cast<int>((most + *vectors * kThreads - 1) / (*vectors * kThreads));
}

template <class T>
void (*scan_for(int vectors))(Params) {
    switch (vectors) {
        case 1: return scan_kernel<T, 1>;
        case 2: return scan_kernel<T, 2>;
        case 4: return scan_kernel<T, 4>;
        default: return scan_kernel<T, 8>;
    }
}

pkv_status check(int groups, int beams, int candidates, int vocab) {
    if (groups < 1 || beams < 1 || candidates < 1 || vocab < 1) return PKV_EINVAL;
    if (beams > kMaxBeams || candidates > kMaxCandidates) return PKV_EUNSUPPORTED;
    if (static_cast<long long>(beams) * vocab >= INT_MAX || vocab > (1 << 30) || groups > (1 << 20)) return PKV_ERANGE;
    int v;
    if (static_cast<long long>(groups) * beams * chunks_for(static_cast<long long>(groups) * beams, vocab, 4, &v) > INT_MAX)
        return PKV_ERANGE;
    return PKV_OK;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

size_t workspace_for(long long rows, int candidates, int chunks) {
    return align256(static_cast<size_t>(rows) * chunks * kWarps * sizeof(float2)) +
           align256(static_cast<size_t>(rows) * chunks * candidates * sizeof(uint2));
}

}  // namespace beam
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_beam_workspace_size(int num_groups, int num_beams, int num_candidates, int vocab) {
    if (beam::check(num_groups, num_beams, num_candidates, vocab) != PKV_OK) return 0;
    const long long rows = static_cast<long long>(num_groups) * num_beams;
    int v;
    return std::max(beam::workspace_for(rows, num_candidates, beam::chunks_for(rows, vocab, 2, &v)),
                    beam::workspace_for(rows, num_candidates, beam::chunks_for(rows, vocab, 4, &v)));
}

pkv_status pkv_beam_select(const void* logits, int64_t row_stride, int logits_bytes, const float* scores,
                           const uint8_t* finished, int eos, int num_groups, int num_beams, int num_candidates, int vocab,
                           const int32_t* history, const int32_t* lengths, int max_length, float* scores_out,
                           int32_t* tokens_out, int32_t* parents_out, uint8_t* finished_out, int32_t* lengths_out,
                           int32_t* history_out, void* workspace, size_t workspace_bytes, uint32_t* device_error,
                           void* stream) {
    const pkv_status st = beam::check(num_groups, num_beams, num_candidates, vocab);
    if (st != PKV_OK) return st;
    if (logits_bytes != 2 && logits_bytes != 4) return PKV_EUNSUPPORTED;
    if (!logits || !scores || !scores_out || !tokens_out || !parents_out || !finished_out || !workspace || row_stride < vocab ||
        eos < -1 || eos >= vocab || (finished && eos < 0) || max_length < 0)
        return PKV_EINVAL;
    const bool told = history || lengths || history_out || lengths_out;
    if (told && (!history || !lengths || !history_out || !lengths_out || max_length < 1)) return PKV_EINVAL;
    if (reinterpret_cast<uintptr_t>(logits) % logits_bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return PKV_EINVAL;
    const long long rows = static_cast<long long>(num_groups) * num_beams;
    int vectors;
    beam::Params p = {};
    p.chunks = beam::chunks_for(rows, vocab, logits_bytes, &vectors);
    if (workspace_bytes < beam::workspace_for(rows, num_candidates, p.chunks)) return PKV_EINVAL;
    p.logits = logits;
    p.row_stride = row_stride;
    p.scores = scores;
    p.finished = finished;
    p.history = history;
    p.lengths = lengths;
    p.scores_out = scores_out;
    p.tokens_out = tokens_out;
    p.parents_out = parents_out;
    p.finished_out = finished_out;
    p.lengths_out = lengths_out;
    p.history_out = history_out;
    p.stats = static_cast<float2*>(workspace);
    p.lists = reinterpret_cast<uint2*>(static_cast<uint8_t*>(workspace) +
                                       beam::align256(static_cast<size_t>(rows) * p.chunks * beam::kWarps * sizeof(float2)));
    p.err = device_error;
    p.eos = eos;
    p.beams = num_beams;
    p.n = num_candidates;
    p.vocab = vocab;
    p.max_length = max_length;
    const auto scan = logits_bytes == 2 ? beam::scan_for<__nv_bfloat16>(vectors) : beam::scan_for<float>(vectors);
    scan<<<static_cast<unsigned>(rows * p.chunks), beam::kThreads, 0, as_stream(stream)>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        // launched early: it waits for the scan before it reads anything
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(num_groups, static_cast<unsigned>(std::max(1, std::min(num_candidates, beam::kWantCtas / num_groups))));
        cfg.blockDim = dim3(beam::kThreads);
        cfg.stream = as_stream(stream);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, beam::join_kernel, p);
    }
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return PKV_ECUDA;
    }
    return PKV_OK;
}

}  // extern "C"
