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
// the chunk.) The join does the same with the chunks' candidates of a group,
// whose scores it forms in 64 bits: neighbours of the last one taken may differ
// by less than fp32 holds. The exponentials bound the scan from the other side:
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
    float2* stats;  // [rows][chunks]: maximum, sum of exponentials
    uint2* lists;   // [rows][chunks][n]: logit bits, token (or -1)
    uint32_t* err;
    int eos, beams, n, vocab, max_length, chunks;
};

// A beam that is read: neither finished nor without a score.
__device__ __forceinline__ bool row_done(const Params& p, int row) { return p.finished && p.finished[row] != 0; }
__device__ __forceinline__ bool row_live(const Params& p, int row) { return !row_done(p, row) && p.scores[row] > -INFINITY; }

// ---- selection shared by both kernels -----------------------------------------

template <class Key>
__device__ __forceinline__ bool before(Key ka, int ia, Key kb, int ib) {
    return ka > kb || (ka == kb && ia < ib);
}

template <class Key>
struct Selection {
    Key key[kList];
    int at[kList];
    Key warp_key[kWarps];
    int warp_at[kWarps];
    int count;
};

// The least, over the warps, of each warp's ceil(n / 8)-th largest thread key:
// at least n keys of the block reach it (or all that are above -inf).
template <class Key>
__device__ __forceinline__ Key threshold(Selection<Key>& sel, Key best, int n) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Key mine = best, top = -INFINITY;
    for (int i = 0; i < (n + kWarps - 1) / kWarps; ++i) {
        top = mine;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const unsigned holders = __ballot_sync(0xffffffffu, mine == top);
        if (lane == __ffs(holders) - 1) mine = -INFINITY;
    }
    if (threadIdx.x == 0) sel.count = 0;
    if (lane == 0) sel.warp_key[warp] = top;
    __syncthreads();
    Key t = sel.warp_key[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) t = min(t, sel.warp_key[w]);
    return t;
}

template <class Key>
__device__ __forceinline__ void offer(Selection<Key>& sel, Key key, int at) {
    const int i = atomicAdd(&sel.count, 1);
    if (i < kList) {
        sel.key[i] = key;
        sel.at[i] = at;
    }
}

// Writes the n first of the list in order to put(rank, key, at), the missing
// ones as (-inf, -1); where the list overflowed, finds them by n rounds over
// items 0 .. items - 1, item(i, key, at) being false for no candidate.
template <class Key, class Item, class Put>
__device__ __forceinline__ void finish(Selection<Key>& sel, int n, int items, Item item, Put put) {
    __syncthreads();
    const int count = sel.count;
    if (count <= kList) {
        for (int i = threadIdx.x; i < count; i += kThreads) {
            const Key k = sel.key[i];
            const int at = sel.at[i];
            int rank = 0;
            for (int j = 0; j < count; ++j) rank += before(sel.key[j], sel.at[j], k, at);
            if (rank < n) put(rank, k, at);
        }
        for (int i = count + threadIdx.x; i < n; i += kThreads) put(i, Key(-INFINITY), -1);
        return;
    }
    Key last = INFINITY;
    int last_at = -1;
    for (int j = 0; j < n; ++j) {
        Key best = -INFINITY;
        int best_at = INT_MAX;
        for (int i = threadIdx.x; i < items; i += kThreads) {
            Key k;
            int at;
            if (item(i, k, at) && before(last, last_at, k, at) && before(k, at, best, best_at)) {
                best = k;
                best_at = at;
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const Key k = __shfl_xor_sync(0xffffffffu, best, d);
            const int at = __shfl_xor_sync(0xffffffffu, best_at, d);
            if (before(k, at, best, best_at)) {
                best = k;
                best_at = at;
            }
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            sel.warp_key[threadIdx.x >> 5] = best;
            sel.warp_at[threadIdx.x >> 5] = best_at;
        }
        __syncthreads();
        last = sel.warp_key[0];
        last_at = sel.warp_at[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            if (before(sel.warp_key[w], sel.warp_at[w], last, last_at)) {
                last = sel.warp_key[w];
                last_at = sel.warp_at[w];
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
};
template <>
struct Vector<float> {
    static constexpr int kN = 4;
    uint32_t u[4];
    __device__ __forceinline__ void fill() { u[0] = u[1] = u[2] = u[3] = 0xff800000u; }
    __device__ __forceinline__ void set(int e, float x) { u[e] = __float_as_uint(x); }
    __device__ __forceinline__ float get(int e) const { return __uint_as_float(u[e]); }
};

// kN logits from token `at` on, -inf behind the row's end. Which logits a thread
// sums is a matter of their tokens alone, so rows that are alike have the same
// sums wherever they lie: a row that does not begin on a 16-byte boundary is read
// as neighbouring aligned vectors, shifted; its first and last logits, whose
// vectors reach beyond the row, one by one.
template <class T>
__device__ __forceinline__ Vector<T> load(const T* row, int at, int vocab, unsigned shift) {
    constexpr int kN = Vector<T>::kN;
    Vector<T> v;
    if (shift == 0 && at + kN <= vocab) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + at));
        v.u[0] = u.x, v.u[1] = u.y, v.u[2] = u.z, v.u[3] = u.w;
    } else if (shift != 0 && at >= kN && at + 2 * kN <= vocab) {
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(row + at) - shift);
        const uint4 a = __ldg(src), b = __ldg(src + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const unsigned bits = shift % 4 * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = shift < 4 ? w[i] : shift < 8 ? w[i + 1] : shift < 12 ? w[i + 2] : w[i + 3];
            const uint32_t hi = shift < 4 ? w[i + 1] : shift < 8 ? w[i + 2] : shift < 12 ? w[i + 3] : w[i + 4];
            v.u[i] = __funnelshift_r(lo, hi, bits);
        }
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
__global__ void __launch_bounds__(kThreads) scan_kernel(const Params p) {
    constexpr int kN = Vector<T>::kN;
    griddep_launch_dependents();
    const int row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks;
    if (!row_live(p, row)) return;
    __shared__ Selection<float> sel;
    __shared__ float warp_max[kWarps], warp_sum[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T* logits = static_cast<const T*>(p.logits) + row * p.row_stride;
    const unsigned shift = static_cast<unsigned>(reinterpret_cast<uintptr_t>(logits) & 15u);
    const int first = (chunk * kVectors * kThreads + threadIdx.x) * kN;  // token of the thread's first logit
    Vector<T> v[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) v[i] = load(logits, first + i * kThreads * kN, p.vocab, shift);
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
#pragma unroll
        for (int e = 0; e < kN; ++e) best = fmaxf(best, v[i].get(e));
    float top = best;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0) warp_max[warp] = top;
    const float cut = threshold(sel, best, p.n);  // behind its barrier the warps' maxima are there
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, warp_max[w]);
    const float from = top > -INFINITY ? top : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
#pragma unroll
        for (int e = 0; e < kN; ++e) sum += ex2((v[i].get(e) - from) * 1.4426950408889634f);
    // a NaN makes the row's sum NaN, and then none of its scores is a number
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) warp_sum[warp] = sum;
    if (best >= cut && best > -INFINITY) {
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const float x = v[i].get(e);
                if (x >= cut && x > -INFINITY) offer(sel, x, first + i * kThreads * kN + e);
            }
    }
    const size_t out = static_cast<size_t>(row) * p.chunks + chunk;
    uint2* list = p.lists + out * p.n;
    const int lo = chunk * kVectors * kThreads * kN, hi = min(lo + kVectors * kThreads * kN, p.vocab);
    finish(
        sel, p.n, hi - lo,
        [&](int i, float& k, int& at) {
            at = lo + i;
            k = static_cast<float>(logits[at]);
            return k > -INFINITY;
        },
        [&](int rank, float k, int at) { list[rank] = make_uint2(__float_as_uint(k), static_cast<uint32_t>(at)); });
    if (threadIdx.x == 0) {
        float all = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all += warp_sum[w];
        p.stats[out] = make_float2(top, all);
    }
}

// ---- join -----------------------------------------------------------------------

// CTA (group, share): every share of a group finds its best n candidates, and
// writes the results of every gridDim.y-th.
__global__ void __launch_bounds__(kThreads) join_kernel(const Params p) {
    __shared__ Selection<double> sel;
    __shared__ double lse[kMaxBeams];
    __shared__ double won_key[kMaxCandidates];
    __shared__ int won_at[kMaxCandidates];
    const int group = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = group * p.beams;
    griddep_wait();
    for (int k = warp; k < p.beams; k += kWarps) {
        const int row = row0 + k;
        if (!row_live(p, row)) continue;
        const float2* stats = p.stats + static_cast<size_t>(row) * p.chunks;
        float top = -INFINITY;
        for (int i = lane; i < p.chunks; i += 32) top = fmaxf(top, stats[i].x);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        double sum = 0.;
        for (int i = lane; i < p.chunks; i += 32)
            sum += static_cast<double>(stats[i].y) * exp(static_cast<double>(stats[i].x) - static_cast<double>(top));
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) lse[k] = static_cast<double>(top) + log(sum);
    }
    __syncthreads();
    // candidate i: entry i % (chunks * n) of beam i / (chunks * n)
    const int per_row = p.chunks * p.n, items = p.beams * per_row;
    auto item = [&](int i, double& key, int& at) {
        const int k = i / per_row, j = i - k * per_row, row = row0 + k;
        const float s = p.scores[row];
        if (row_done(p, row)) {
            key = s;
            at = k * p.vocab + p.eos;
            return j == 0 && s > -INFINITY;
        }
        if (!(s > -INFINITY)) return false;
        const uint2 c = p.lists[static_cast<size_t>(row) * per_row + j];
        key = static_cast<double>(s) + (static_cast<double>(__uint_as_float(c.x)) - lse[k]);
        at = k * p.vocab + static_cast<int>(c.y);
        return static_cast<int>(c.y) >= 0 && key > -INFINITY;  // (false for NaN)
    };
    double best = -INFINITY;
    for (int i = threadIdx.x; i < items; i += kThreads) {
        double key;
        int at;
        if (item(i, key, at)) best = max(best, key);
    }
    const double cut = threshold(sel, best, p.n);
    if (best >= cut && best > -INFINITY)
        for (int i = threadIdx.x; i < items; i += kThreads) {
            double key;
            int at;
            if (item(i, key, at) && key >= cut) offer(sel, key, at);
        }
    finish(sel, p.n, items, item, [&](int rank, double key, int at) {
        won_key[rank] = key;
        won_at[rank] = at;
    });
    __syncthreads();
    for (int j = blockIdx.y; j < p.n; j += gridDim.y) {
        const int at = won_at[j];
        const bool some = at >= 0;
        const int k = some ? at / p.vocab : -1, token = some ? at - k * p.vocab : -1;
        const int row = row0 + max(k, 0);
        const bool done = some && row_done(p, row);
        const size_t out = static_cast<size_t>(group) * p.n + j;
        int length = 0;
        if (some && p.lengths) {
            const int given = p.lengths[row];
            length = min(max(given, 0), p.max_length);
            if ((given != length || (!done && length == p.max_length)) && p.err && threadIdx.x == 0)
                atomicOr(p.err, PKV_DEVERR_CONTEXT);
        }
        const bool grows = some && !done && length < p.max_length;
        if (threadIdx.x == 0) {
            p.scores_out[out] = static_cast<float>(won_key[j]);
            p.tokens_out[out] = token;
            p.parents_out[out] = k;
            p.finished_out[out] = done || (some && token == p.eos);
            if (p.lengths) p.lengths_out[out] = length + (grows ? 1 : 0);
            if (p.lengths && grows) p.history_out[out * p.max_length + length] = token;
        }
        if (p.lengths) {
            const int32_t* src = p.history + static_cast<size_t>(row) * p.max_length;
            int32_t* dst = p.history_out + out * p.max_length;
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
    return align256(static_cast<size_t>(rows) * chunks * sizeof(float2)) +
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
                                       beam::align256(static_cast<size_t>(rows) * p.chunks * sizeof(float2)));
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
