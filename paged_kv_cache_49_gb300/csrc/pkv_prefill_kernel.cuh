// Attention of many query rows per sequence over the paged cache, on the
// fifth-generation tensor cores: causal prompt chunks and draft trees.
//
// A tile is 128 query rows of one KV head -- 128 / group tokens with all
// their query heads, so a K or V byte serves the whole group -- against 128
// keys: S = Q K^T into tensor memory, an online softmax in registers, P as
// bf16 back into tensor memory over S, O += P V in tensor memory.
//
// An item is up to two tiles of one (sequence, KV head) against all their
// keys. Its two streams (one accumulator and one softmax warpgroup each) run
// in turn on the tensor core, so that one multiplies while the other takes
// exponentials:
//   - two tiles: each stream has its own query tile, both share every K and V
//     tile;
//   - one tile: the streams share the query tile and take the even and the
//     odd key tiles; their states are joined at the end.
//
// The items of the batch, laid end to end by cost, are cut into one range per
// CTA (one persistent CTA per SM; three one after the other where that keeps
// the contexts in L2), planned by every CTA from the lengths on the device. A
// cut near an item's end moves there; any other leaves fp32 partial results that
// merge_kernel joins in a fixed order.
//
// What no row sees never enters a sum: masked scores are replaced before the
// softmax, and of the value tiles that only some rows see in full, a warp
// pair zeroes the rows past the end and the non-finite values before the
// product; those are added to the rows that do see them at the end.
//
// A group of G heads and T rows do G T operations a byte of K and V: prompts
// are bound by the tensor core (16,411 tokens of 64 / 8 heads: 2.6 to 2.9 ms,
// 1.5 to 1.7 PFLOP/s of a measured 1.7 under the power cap to 1.9; chunks of
// 1,000 tokens on 9,000 cached ones 2.0 ms, 1.43 PFLOP/s), trees by bandwidth
// (64 trees of 16 drafts on 1,024 tokens: 98 us, 4.6 of 6.8 TB/s), short items
// by their starts and ends (16 packed prompts of 512 tokens: 99 us, 0.62
// PFLOP/s). A K or V byte is read once for an item's 256 rows: a tree of more
// than 32 drafts at 8 heads is two items and reads its context twice.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cfloat>
#include <cstdint>

#include "pkv_ptx.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace prefill {

constexpr int kDim = PKV_ATTN_HEAD_DIM;
constexpr int kRows = 128;    // query rows of a tile
constexpr int kKeys = 128;    // keys of a tile
constexpr int kThreads = 384;
constexpr int kSoftmaxWarps = 8;
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpClean = 10;  // and 11
// Registers: what the block is launched with, moved from the third warpgroup to the softmax's two.
constexpr int kRegsLaunch = 168, kRegsSoftmax = 208, kRegsOther = 88;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * kRegsLaunch, "register split");
constexpr int kCleanBars = 8;  // more than the ring can hold

constexpr int kMaxStages = 5;
constexpr uint32_t kTileBytes = kKeys * kDim * 2;
constexpr uint32_t kTmemColumns = 512;
constexpr uint32_t kTmemO = 256;  // S0, S1, O0, O1 of 128 columns each

// Cost units of the work line: one key of an item's two tiles is 8 (3,400
// cycles for a key tile). One tile alone costs 2,300 where the products bound
// it, but as much as two where its keys' bytes do, as over the long contexts
// of trees. An item's fixed work is 7,000 cycles (of a tree 4,800).
constexpr int kCostTwo = 8;
__host__ __device__ constexpr int cost_one(bool tree) { return tree ? 8 : 6; }
__host__ __device__ constexpr int cost_item(bool tree) { return tree ? 8 * 200 : 8 * 290; }
constexpr int kSnap = 8 * 256;      // a cut this near an item's end moves there
constexpr int kWhole = 8 * 768;     // an item of this cost is never cut
constexpr int kMinRange = 8 * 256;  // least cost of a CTA's range
constexpr int kPieces = 4;          // pieces described ahead

constexpr size_t kWsHeader = 256;
constexpr int kMaxGrid = 1024;
// Ranges of a CTA, one after the other: more than one where many items each
// read the same long contexts, all heads' contexts at once would exceed L2, and
// there are items enough (rounds_of). The CTAs then share a third of the heads
// at a time.
constexpr int kRounds = 3;
constexpr float kRoundBytes = 96.f * (1 << 20);  // of L2's 129 MB
constexpr float kRoundReads = 16.f;

struct Params {
    __nv_bfloat16* out;
    const __nv_bfloat16* v_cache;
    const __nv_bfloat16* v_draft;
    const int64_t* masks;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_starts;
    uint32_t* err;
    struct Split* splits;   // [ranges], as are:
    float2* part_ml;        // [2 * ranges][256]
    float* part_o;          // [2 * ranges][256][128]
    int* rounds;            // of this call, for the join
    int grid, one;          // CTAs; items of one query tile only
    int max_rounds;         // kRounds where the call may take them, else 1
    int num_seqs, num_tokens, hq, hkv, group, tpt;  // tpt: tokens of a tile
    int max_blocks, num_blocks, bt;
    float scale_log2;
    unsigned long long item_magic;  // ceil(2^36 / tokens of an item)
};

// An item cut among CTAs, described by the CTA that has its first piece.
struct Split {
    long long start, cost;  // the item's place and length on the cost line
    long long chunk;        // the length of a range
    int ntiles;             // 0: nothing to join
    int tok0, ntok, head0;
};

struct Seq {
    int n, ctx, tok0;  // query rows, tokens in the cache, first row
    int full, rest;    // full items, tokens of the last, smaller one
};

// A CTA's piece of an item, as the loader describes it to the other warps.
struct __align__(16) Piece {
    int count;          // key tiles; below zero: no more pieces
    int ta;             // the first of them
    int cnt[2];         // key tiles of each stream
    int two;            // two query tiles, or one
    int whole;          // the piece is its whole item
    int tok0, ntok;     // rows of q / out
    int pos0;           // prefill: position of the first row
    int first_masked;   // first tile that not every row sees in full
    int kend, nct;      // keys in the cache it needs; their tiles
    int s, h;           // sequence, KV head
    int seq_n, seq_tok0, ctx;  // query rows and first row of the sequence, its tokens in the cache
    int slot;           // of its partial results
    int any_bad;        // set by the cleaning warps: values were taken out
};

struct __align__(16) Misc {
    uint64_t q_full, q_empty;
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
    uint64_t part_full[kCleanBars], clean[kCleanBars];  // value tiles to be cleaned: landed, cleaned
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t join[2];         // one-tile items: both streams' states are there; both accumulators are read
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    Piece piece[kPieces];
    uint32_t bad[kPieces][4][4];  // [piece][masked tile][key / 32]: non-finite values taken out
    uint32_t tmem;
    int abort;
    union {
        struct {  // the plan; the loader has read it before it describes the first piece
            long long scan[kThreads / 32];
            float keys[kThreads / 32], items[kThreads / 32];
            int cut[kRounds][2][4];  // sequence, head, item, tile of the ranges' ends
            Seq cut_seq;             // the first one's first sequence
            int rounds;
        };
        float2 ml[2][kRows];  // one-tile items: the streams' row states
    };
};

// Shared memory of a kernel whose items have one query tile at most, or two.
// The room of the second one is a fifth stage of the ring: with four, a stream
// of one-tile items over long contexts waits for its loads (a K tile is held
// for 600 cycles after it lands, a V tile for 2,500, and a load takes 3,300).
constexpr uint32_t kOutBytes = 32 * 128;  // a softmax warp's staging: 32 rows of 128 bytes
template <bool kOne>
struct Smem {
    static constexpr int kStages = kOne ? 5 : 4;  // K or V tiles in flight
    static constexpr uint32_t kQ = 0, kRing = (kOne ? 1 : 2) * kTileBytes, kOut = kRing + kStages * kTileBytes;
    static constexpr uint32_t kMisc = kOut + kSoftmaxWarps * kOutBytes;
    static constexpr size_t kBytes = kMisc + sizeof(Misc);
    static_assert(kBytes <= 232448, "shared memory of one CTA");
};

// ---- the work line -----------------------------------------------------------

template <bool kOne>
__device__ __forceinline__ int item_tokens(int tpt) { return kOne ? tpt : 2 * tpt; }

template <bool kTree, bool kOne>
__device__ __forceinline__ Seq load_seq(const Params& p, int s, uint32_t* bad) {
    const int a = __ldg(p.query_starts + s), b = __ldg(p.query_starts + s + 1);
    int ctx = __ldg(p.context_lens + s);
    Seq q;
    q.tok0 = min(max(a, 0), p.num_tokens);
    const int end = min(max(b, 0), p.num_tokens);
    q.n = max(end - q.tok0, 0);
    if (bad && (a != q.tok0 || b != end || end < q.tok0)) *bad |= PKV_DEVERR_QUERY;
    if (kTree && q.n > PKV_TREE_MAX_DRAFTS) {
        q.n = PKV_TREE_MAX_DRAFTS;
        if (bad) *bad |= PKV_DEVERR_QUERY;
    }
    const long long cap = static_cast<long long>(p.max_blocks) * p.bt;
    if (ctx > cap) {
        ctx = static_cast<int>(cap);
        if (bad) *bad |= PKV_DEVERR_CONTEXT;
    }
    q.ctx = max(ctx, 0);
    if (bad && !kTree && q.n > q.ctx) *bad |= PKV_DEVERR_CONTEXT;
    // n / tokens by the host's ceil(2^36 / tokens): exact below 2^28, then corrected
    const int tokens = item_tokens<kOne>(p.tpt);
    q.full = static_cast<int>((static_cast<unsigned long long>(q.n) * p.item_magic) >> 36);
    if (q.full * tokens > q.n) --q.full;
    q.rest = q.n - q.full * tokens;
    return q;
}

// Costs of one head of a sequence: of the first i items, all full, i * (a + b i);
// of the smaller one behind them, last.
struct Cost {
    long long a, last;
    int b;
    __device__ __forceinline__ long long first(int i) const { return i * (a + static_cast<long long>(b) * i); }
};

template <bool kTree, bool kOne>
__device__ __forceinline__ Cost cost_of(const Seq& q, int tpt) {
    constexpr int kOneCost = cost_one(kTree), kFull = kOne ? kOneCost : kCostTwo, kItemCost = cost_item(kTree);
    Cost c;
    // keys of item i of a prompt: ctx - n + (i + 1) * its tokens; of a chunk longer
    // than its context, all of ctx for every item. So none costs more than the keys
    // of its table row would, by which the host leaves out the join.
    const bool flat = kTree || q.n > q.ctx;
    const long long keys = kTree ? q.ctx + static_cast<long long>(kKeys) : flat ? q.ctx : q.ctx - q.n;
    c.b = flat ? 0 : kFull * item_tokens<kOne>(tpt) / 2;
    c.a = kFull * keys + kItemCost + c.b;
    c.last = q.rest ? (q.rest > tpt ? kCostTwo : kOneCost) * (kTree ? keys : static_cast<long long>(q.ctx)) + kItemCost : 0;
    return c;
}

// Tiles of an item that belong to ranges before a cut `off` cost units into
// it; any monotone rule does that every reader computes alike.
__device__ __forceinline__ int cut_tile(long long off, long long cost, int ntiles) {
    if (off <= kSnap || (cost <= kWhole && 2 * off < cost)) return 0;
    if (cost - off <= kSnap || cost <= kWhole) return ntiles;
    const int t = static_cast<int>(__ll2float_rn(off) / __ll2float_rn(cost) * ntiles + 0.5f);
    return min(max(t, 0), ntiles);
}

// One item: the i-th of one (sequence, KV head).
struct Item {
    int s, h, i;
    Seq q;
    int tok0, ntok;   // rows of q / out
    int pos0;         // prefill: position of the first row
    int kend;         // keys in the cache it may need
    int nct, nt;      // tiles of the cache; with the draft tile
    int first_masked; // first tile that not every row sees in full
    bool two;

    __device__ __forceinline__ int cut_tiles() const { return max(nt, 1); }
};

template <bool kTree, bool kOne>
__device__ __forceinline__ void set_item(const Params& p, Item& it) {
    const int off = it.i * item_tokens<kOne>(p.tpt);
    it.tok0 = it.q.tok0 + off;
    it.ntok = min(item_tokens<kOne>(p.tpt), it.q.n - off);
    it.two = !kOne && it.ntok > p.tpt;
    it.pos0 = it.q.ctx - it.q.n + off;
    it.kend = kTree ? it.q.ctx : max(it.pos0 + it.ntok, 0);
    it.nct = (it.kend + kKeys - 1) / kKeys;
    it.nt = it.nct + (kTree ? 1 : 0);
    it.first_masked = (kTree ? it.q.ctx : max(it.pos0 + 1, 0)) / kKeys;
}

// The loader's walk over its CTA's range: next() yields the pieces in order.
template <bool kTree, bool kOne>
struct Walk {
    const Params& p;
    Item it;
    Seq ahead;           // the sequence after it.s, read early
    int s1, h1, i1, t1;  // the range's end
    int ta, tb;          // tiles of the piece
    bool first;
    int cuts, round, rounds;  // lane i: the i-th number of the ranges' ends

    __device__ __forceinline__ Walk(const Params& prm, const Misc& m) : p(prm), round(0), rounds(m.rounds) {
        const int lane = threadIdx.x & 31;
        cuts = lane < kRounds * 8 ? (&m.cut[0][0][0])[lane] : 0;
        it.q = m.cut_seq;
        open();
    }
    __device__ __forceinline__ void open() {
        auto get = [&](int i) { return __shfl_sync(0xFFFFFFFFu, cuts, round * 8 + i); };
        it.s = get(0);
        it.h = get(1);
        it.i = get(2);
        ta = get(3);
        s1 = get(4);
        h1 = get(5);
        i1 = get(6);
        t1 = get(7);
        first = true;
    }
    __device__ __forceinline__ bool next() {
        if (next_of_range()) return true;
#pragma unroll 1
        while (round + 1 < rounds) {
            ++round;
            open();
            if (it.s < p.num_seqs) it.q = load_seq<kTree, kOne>(p, it.s, nullptr);
            if (next_of_range()) return true;
        }
        return false;
    }
    __device__ __forceinline__ bool next_of_range() {
        bool enter = first, step = !first;  // a sequence was entered; go on to another item
        if (first) {
            if (it.s >= p.num_seqs) return false;
            set_item<kTree, kOne>(p, it);
            step = ta >= it.cut_tiles();  // the range starts behind this item
            first = false;
        }
#pragma unroll 1
        while (enter || step) {
            if (enter) {
                if (it.s + 1 < p.num_seqs) ahead = load_seq<kTree, kOne>(p, it.s + 1, nullptr);
                enter = false;
            }
            if (step) {
                step = false;
                ta = 0;
                ++it.i;
                if (it.i * item_tokens<kOne>(p.tpt) >= it.q.n) {
                    it.i = 0;
                    if (it.q.n == 0 || ++it.h == p.hkv) {
                        it.h = 0;
                        if (++it.s >= p.num_seqs) return false;
                        it.q = ahead;
                        enter = true;
                        step = it.q.n == 0;
                    }
                }
            }
        }
        set_item<kTree, kOne>(p, it);
        if (it.s > s1 || (it.s == s1 && (it.h > h1 || (it.h == h1 && it.i > i1)))) return false;
        const bool last = it.s == s1 && it.h == h1 && it.i == i1;
        if (last && t1 <= ta) return false;
        tb = last ? t1 : it.cut_tiles();
        return true;
    }
    __device__ __forceinline__ void describe(Piece& d) const {
        d.ta = ta;
        const int c = max(min(tb, it.nt) - ta, 0);
        d.count = c;
        if (!it.two) {
            d.cnt[0] = (c + 1) >> 1;
            d.cnt[1] = c >> 1;
        } else {
            // the first tile's rows see no tile past their own last token's
            const int own = kTree ? it.nt : (max(it.pos0 + p.tpt, 0) + kKeys - 1) / kKeys;
            d.cnt[0] = max(min(own - ta, c), 0);
            d.cnt[1] = c;
        }
        d.two = it.two;
        d.whole = ta == 0 && tb == it.cut_tiles();
        d.tok0 = it.tok0;
        d.ntok = it.ntok;
        d.pos0 = it.pos0;
        d.first_masked = it.first_masked;
        d.kend = it.kend;
        d.nct = it.nct;
        d.s = it.s;
        d.h = it.h;
        d.seq_n = it.q.n;
        d.seq_tok0 = it.q.tok0;
        d.ctx = it.q.ctx;
        d.slot = 2 * (round * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x)) + (ta == 0 ? 1 : 0);
        d.any_bad = 0;
    }
};

// The ring's entries of a piece in the order of their use: K0 V0 K1 V1 ... for
// two query tiles, K0 K1 V0 K2 V1 ... for one, whose streams take turns; and
// the places of the j-th K and V tile in it.
struct RingEntry {
    bool is_v;
    int j;
};
__device__ __forceinline__ RingEntry ring_entry(bool two, int pos, int count) {
    if (two || pos == 0 || pos == 2 * count - 1) return {(pos & 1) != 0, pos >> 1};
    return (pos & 1) ? RingEntry{false, (pos >> 1) + 1} : RingEntry{true, (pos >> 1) - 1};
}
__device__ __forceinline__ int ring_k(bool two, int j) { return two ? 2 * j : max(2 * j - 1, 0); }
__device__ __forceinline__ int ring_v(bool two, int j, int count) { return two || j == count - 1 ? 2 * j + 1 : 2 * j + 2; }

template <bool kTree, bool kOne>
__host__ __device__ constexpr int rounds_max() { return kTree || kOne ? 1 : kRounds; }  // others read their contexts a few times at the most

// The rounds of a call: keys that it reads and items that it has (of all KV
// heads), and their cost. Chunks of 1,000 tokens on 9,000 cached ones, 64 / 8
// heads, 0.5 GB of inputs, read 9 GB from memory in one round, which slows the
// products where power bounds the clocks: call after call 2,210 us in one
// round, 2,140 in two, 2,000 in three or four. Items read by few others gain
// nothing, and each cut more costs a join.
__device__ __forceinline__ int rounds_of(float keys, float items, float cost, int grid) {
    const bool many = cost >= kRoundReads * kCostTwo * keys && items >= 4.f * grid;
    return many && keys * (4 * kDim) > kRoundBytes ? kRounds : 1;
}

// Every thread of the CTA: the ends of this CTA's range, and the description
// of the item that its end cuts. Each half of the threads goes over all
// sequences and finds one end.
template <bool kTree, bool kOne>
__device__ void plan(const Params& p, Misc& m) {
    constexpr int kHalf = kThreads / 2, kHalfWarps = kHalf / 32;
    const int e = threadIdx.x >= kHalf, tid = threadIdx.x - e * kHalf, lane = tid & 31, warp = tid >> 5;
    const int per = (p.num_seqs + kHalf - 1) / kHalf;
    const int s0 = min(tid * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
    long long sum = 0;
    float keys = 0.f, items = 0.f;  // read at least once; the same in every CTA
    uint32_t bad = 0;
    Seq seq0 = {};
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
        const Seq q = load_seq<kTree, kOne>(p, s, &bad);
        if (s == s0) seq0 = q;
        const Cost c = cost_of<kTree, kOne>(q, p.tpt);
        sum += (c.first(q.full) + c.last) * p.hkv;
        if (rounds_max<kTree, kOne>() > 1 && p.max_rounds > 1 && q.n > 0) {
            keys += static_cast<float>(q.ctx);
            items += static_cast<float>(q.full + (q.rest != 0));
        }
    }
    if (bad && blockIdx.x == 0) atomicOr(p.err, bad);
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) m.scan[e * kHalfWarps + warp] = incl;
    if (rounds_max<kTree, kOne>() > 1 && p.max_rounds > 1) {
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            keys += __shfl_xor_sync(0xFFFFFFFFu, keys, d);
            items += __shfl_xor_sync(0xFFFFFFFFu, items, d);
        }
        if (lane == 0) {
            m.keys[e * kHalfWarps + warp] = keys;
            m.items[e * kHalfWarps + warp] = items;
        }
    }
    if (tid < 4 * kRounds) m.cut[tid >> 2][e][tid & 3] = (tid & 3) == 0 ? p.num_seqs : 0;
    if (threadIdx.x < p.max_rounds) p.splits[threadIdx.x * gridDim.x + blockIdx.x].ntiles = 0;
    __syncthreads();
    long long before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kHalfWarps; ++w) {
        const long long v = m.scan[e * kHalfWarps + w];
        if (w < warp) before += v;
        total += v;
    }
    int rounds = 1;
    if (rounds_max<kTree, kOne>() > 1 && p.max_rounds > 1) {
        keys = items = 0.f;
#pragma unroll
        for (int w = 0; w < kHalfWarps; ++w) {
            keys += m.keys[e * kHalfWarps + w];
            items += m.items[e * kHalfWarps + w];
        }
        rounds = rounds_of(keys * p.hkv, items * p.hkv, static_cast<float>(total), gridDim.x);
    }
    if (threadIdx.x == 0) {
        m.rounds = rounds;
        if (p.max_rounds > 1 && blockIdx.x == 0) *p.rounds = rounds;
    }
    const int ranges = static_cast<int>(min(static_cast<long long>(gridDim.x) * rounds, max(total / kMinRange, 1ll)));
    // a range's length, no less than its share (by some 2^-20 more)
    const long long chunk = static_cast<long long>(__ll2float_ru(total) / ranges * 1.000001f) + 1;
#pragma unroll 1
    for (int r = 0; r < rounds; ++r) {
        const int b = r * gridDim.x + blockIdx.x;
        const long long x = chunk * (b + e);
        if (x < before || x >= before + sum) continue;  // at or past the line's end: behind the last sequence
        long long at = before;
#pragma unroll 1
        for (int s = s0; s < s1; ++s) {
            Item it;
            it.q = s == s0 ? seq0 : load_seq<kTree, kOne>(p, s, nullptr);
            const Cost c = cost_of<kTree, kOne>(it.q, p.tpt);
            const long long hc = c.first(it.q.full) + c.last;
            if (x >= at + hc * p.hkv) {
                at += hc * p.hkv;
                continue;
            }
            it.s = s;
            // estimates, then the exact head and item
            long long off = x - at;
            it.h = min(static_cast<int>(__ll2float_rn(off) / __ll2float_rn(hc)), p.hkv - 1);
            off -= hc * it.h;
            if (off < 0) {
                off += hc;
                --it.h;
            } else if (off >= hc) {
                off -= hc;
                ++it.h;
            }
            const float fa = __ll2float_rn(c.a), fo = __ll2float_rn(off);
            it.i = min(static_cast<int>(2.f * fo / (fa + sqrtf(fa * fa + 4.f * c.b * fo))), it.q.full - (it.q.rest == 0));
#pragma unroll 1
            while (c.first(it.i) > off) --it.i;
#pragma unroll 1
            while (it.i < it.q.full - (it.q.rest == 0) && c.first(it.i + 1) <= off) ++it.i;
            set_item<kTree, kOne>(p, it);
            const long long start = x - off + c.first(it.i);
            const long long cost = it.i < it.q.full ? c.first(it.i + 1) - c.first(it.i) : c.last;
            const int t = cut_tile(x - start, cost, it.cut_tiles());
            m.cut[r][e][0] = s;
            m.cut[r][e][1] = it.h;
            m.cut[r][e][2] = it.i;
            m.cut[r][e][3] = t;
            if (e == 0 && r == 0) m.cut_seq = it.q;
            // this CTA has the item's first piece and not its last
            if (e == 1 && t > 0 && t < it.cut_tiles() &&
                (x - chunk <= start || cut_tile(x - chunk - start, cost, it.cut_tiles()) == 0)) {
                Split sp;
                sp.start = start;
                sp.cost = cost;
                sp.chunk = chunk;
                sp.ntiles = it.cut_tiles();
                sp.tok0 = it.tok0;
                sp.ntok = it.ntok;
                sp.head0 = it.h * p.group;
                p.splits[b] = sp;
            }
            break;
        }
    }
}

// ---- the kernel ---------------------------------------------------------------

__device__ __forceinline__ uint32_t non_finite2(uint32_t w) {  // a set sign bit for each non-finite bf16 half
    return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

// One 128-byte half of a row of a value tile in the ring: non-finite values
// become zero, a row behind the last (live false) becomes zero whole. Whether
// a live row had non-finite values.
__device__ __forceinline__ bool clean_half_row(uint8_t* half, int lane, bool live) {
    uint4 v[8];
    uint32_t any = 0;
    // lanes start at different 16-byte chunks of their rows: no bank conflicts
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const uint4*>(half + ((i + lane) & 7) * 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= non_finite2(v[i].x) | non_finite2(v[i].y) | non_finite2(v[i].z) | non_finite2(v[i].w);
    if (any == 0 && live) return false;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        uint4* const at = reinterpret_cast<uint4*>(half + ((i + lane) & 7) * 16);
        auto finite = [live](uint32_t w) { return live ? w & ~((non_finite2(w) >> 15) * 0xFFFFu) : 0u; };
        const uint4 u = *at;
        *at = make_uint4(finite(u.x), finite(u.y), finite(u.z), finite(u.w));
    }
    return live;
}

// The keys of a masked tile that a row sees, as four words of 32.
template <bool kTree>
__device__ __forceinline__ void seen_words(const Piece& it, int tile, int vis, uint64_t draft_mask, uint32_t (&w)[4]) {
    if (kTree && tile == it.nct) {
        if (it.seq_n < 64) draft_mask &= (1ull << it.seq_n) - 1ull;
        w[0] = static_cast<uint32_t>(draft_mask);
        w[1] = static_cast<uint32_t>(draft_mask >> 32);
        w[2] = w[3] = 0;
        return;
    }
    const int limit = vis - tile * kKeys;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int l = limit - 32 * k;
        w[k] = l <= 0 ? 0u : l >= 32 ? 0xFFFFFFFFu : (1u << l) - 1u;
    }
}

// Adds to columns [lo, hi) of a finished row -- bf16 in out, or fp32 in part --
// the non-finite values that were taken out of the product for keys the row
// sees (their weights are positive, so each weighted value is the value
// itself). bad: the words of tiles t_lo ..
template <bool kTree>
__device__ __forceinline__ void add_non_finite(const Params& p, const Piece& it, int t_lo, int t_hi, const uint32_t (*bad)[4],
                                               int vis, uint64_t draft_mask, int lo, int hi, __nv_bfloat16* out, float* part) {
#pragma unroll 1
    for (int kk = 0; kk < 4 * (t_hi - t_lo); ++kk) {
        const int t = t_lo + (kk >> 2), k = kk & 3;
        uint32_t bits = bad[kk >> 2][k];
#pragma unroll 1
        for (; bits; bits &= bits - 1) {
            const int key = __ffs(bits) - 1 + 32 * k;
            const __nv_bfloat16* row;
            if (kTree && t == it.nct) {
                if (!(draft_mask >> key & 1)) continue;
                row = p.v_draft + (static_cast<long long>(it.seq_tok0 + key) * p.hkv + it.h) * kDim;
            } else {
                const int pos = t * kKeys + key;
                if (pos >= vis) continue;
                int blk = __ldg(p.block_tables + static_cast<long long>(it.s) * p.max_blocks + pos / p.bt);
                if (blk < 0 || blk >= p.num_blocks) blk = 0;
                row = p.v_cache + ((static_cast<long long>(blk) * p.hkv + it.h) * p.bt + pos % p.bt) * kDim;
            }
#pragma unroll 1
            for (int c = lo; c < hi; ++c) {
                const float v = __bfloat162float(row[c]);
                if (isfinite(v)) continue;
                if (out) out[c] = __float2bfloat16(__bfloat162float(out[c]) + v);
                else part[c] += v;
            }
        }
    }
}

template <bool kTree, bool kOne>
__global__ void __launch_bounds__(kThreads, 1)
rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kd,
            const __grid_constant__ CUtensorMap tm_vd, const __grid_constant__ Params p) {
    using L = Smem<kOne>;
    constexpr int kStages = L::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    Misc& m = *reinterpret_cast<Misc*>(smem + L::kMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem_base = smem_u32(smem);
    volatile int* abort_flag = &m.abort;

    griddep_launch_dependents();
    if (smem_base & 1023) {  // the swizzle atoms need it; dynamic shared memory starts so, with no static beside it
        griddep_wait();
        if (tid == 0) {
            for (int r = 0; r < p.max_rounds; ++r) p.splits[r * gridDim.x + blockIdx.x].ntiles = 0;
            if (blockIdx.x == 0) *p.rounds = 1;
            atomicOr(p.err, PKV_DEVERR_TIMEOUT);
        }
        return;
    }
    if (tid == 0) {
        m.abort = 0;
        mbar_init(smem_u32(&m.q_full), 1);
        mbar_init(smem_u32(&m.q_empty), 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&m.kv_full[i]), 1);
            mbar_init(smem_u32(&m.kv_empty[i]), 1);
        }
        for (int i = 0; i < kCleanBars; ++i) {
            mbar_init(smem_u32(&m.part_full[i]), 1);
            mbar_init(smem_u32(&m.clean[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&m.s_full[i]), 1);
            mbar_init(smem_u32(&m.p_full[i]), 4);
            mbar_init(smem_u32(&m.o_full[i]), 1);
            mbar_init(smem_u32(&m.join[i]), kSoftmaxWarps);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(smem_u32(&m.piece_full[i]), 1);
            mbar_init(smem_u32(&m.piece_empty[i]), kSoftmaxWarps + 3);
        }
        fence_barrier_init();
    }
    if (tid == kWarpLoad * 32) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        if (kTree) {
            prefetch_tensormap(&tm_kd);
            prefetch_tensormap(&tm_vd);
        }
    }
    // Launched early: behind this wait are the earlier kernels' results and the
    // last call's partial results. The tensor memory too is taken only here: an
    // earlier kernel may still be about to take its own, and this one would hold
    // all of it while it waits for that kernel's end.
    griddep_wait();
    if (warp == kWarpMma) tmem_alloc(smem_u32(&m.tmem), kTmemColumns);
    tc_fence_before();
    plan<kTree, kOne>(p, m);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m.tmem;
    // A reader of the pieces: the n-th, or null when there are no more (or the pipeline broke).
    auto get_piece = [&](uint32_t n) -> const Piece* {
        const bool ok = wait_for(smem_u32(&m.piece_full[n % kPieces]), (n / kPieces) & 1, abort_flag, p.err);
        const Piece& d = m.piece[n % kPieces];
        return __all_sync(0xFFFFFFFFu, ok) && d.count >= 0 ? &d : nullptr;
    };
    auto done_piece = [&](uint32_t n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&m.piece_empty[n % kPieces]));
    };

    if (warp < kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---- softmax and epilogue: thread = row of the stream's tile
        const int stream = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 tensor-memory lanes
        const uint32_t t_s = tmem + lanes + stream * 128, t_o = tmem + lanes + kTmemO + stream * 128;
        const int row_tok = row / p.group, row_head = row - row_tok * p.group;
        const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);
        uint32_t n_s = 0, n_o = 0, n_join = 0, n_item = 0;
        // one-tile items: a meeting of both warpgroups
        auto meet = [&](int k) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&m.join[k]));
            const bool met = wait_for(smem_u32(&m.join[k]), n_join & 1, abort_flag, p.err);
            tc_fence_after();
            return __all_sync(0xFFFFFFFFu, met) != 0;
        };
        for (;; ++n_item) {
            const Piece* const piece = get_piece(n_item);
            if (!piece) break;
            const Piece& it = *piece;
            const int tile_tok = it.two ? stream * p.tpt : 0;
            const int tok = it.tok0 + tile_tok + row_tok;
            const bool valid = row_tok < p.tpt && tile_tok + row_tok < it.ntok;
            const bool warp_valid = __any_sync(0xFFFFFFFFu, valid);
            const int vis = kTree ? it.ctx : valid ? it.pos0 + tile_tok + row_tok + 1 : 0;
            uint64_t draft_mask = 0;
            if (kTree && valid) {
                draft_mask = static_cast<uint64_t>(__ldg(reinterpret_cast<const long long*>(p.masks) + tok));
            }
            const int count = it.cnt[stream];
            const int first_masked = it.first_masked, tile0 = it.two ? it.ta : it.ta + stream, tile_step = it.two ? 1 : 2;
            float mx = -INFINITY;  // reference of the exponentials, unscaled
            float l = 0.f;
            bool any = false;
            bool ok = true;
            for (int i = 0; i < count; ++i) {
                const int tile = tile0 + i * tile_step;
                ok = wait_for(smem_u32(&m.s_full[stream]), n_s & 1, abort_flag, p.err);
                ++n_s;
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                tc_fence_after();
                if (warp_valid) {
                    uint32_t s[4][32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_ld32(s[k], t_s + 32 * k);
                    tmem_wait_ld(s[0]);
                    hold(s[1]);
                    hold(s[2]);
                    hold(s[3]);
                    if (tile >= first_masked) {
                        uint32_t w[4];
                        seen_words<kTree>(it, tile, vis, draft_mask, w);
                        any |= (w[0] | w[1] | w[2] | w[3]) != 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (__all_sync(0xFFFFFFFFu, w[k] == 0xFFFFFFFFu)) continue;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(w[k] >> c & 1)) s[k][c] = 0xFF800000u;
                        }
                    } else {
                        any = true;
                    }
                    float m4[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        m4[k] = fmaxf(__uint_as_float(s[k][0]), __uint_as_float(s[k][1]));
#pragma unroll
                        for (int c = 2; c < 32; c += 2)
                            m4[k] = fmaxf(m4[k], fmaxf(__uint_as_float(s[k][c]), __uint_as_float(s[k][c + 1])));
                    }
                    const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    // The reference only has to keep the exponentials in range: it
                    // follows the maximum when that has grown by more than 8 (a
                    // factor of 256 in the sums), which spares most rescalings of O.
                    float factor = 1.f;
                    const bool grow = mx == -INFINITY ? top != -INFINITY : (top - mx) * p.scale_log2 > 8.f;
                    if (grow) {
                        factor = mx == -INFINITY ? 0.f : ex2((mx - top) * p.scale_log2);
                        mx = top;
                    }
                    const float ref = mx == -INFINITY ? 0.f : -mx * p.scale_log2;
                    const uint64_t ref2 = pair(ref, ref);
                    uint64_t sum2[4] = {pair(l * factor, 0.f), pair(0.f, 0.f), pair(0.f, 0.f), pair(0.f, 0.f)};
                    // S of this tile being complete, so is the stream's previous product
                    if (i > 0 && __any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            uint32_t o[32];
                            tmem_ld32(o, t_o + 32 * k);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * factor);
                            tmem_st32(t_o + 32 * k, o);
                        }
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t pk[32];
#pragma unroll
                        for (int c = 0; c < 64; c += 2) {
                            const uint32_t* sk = s[2 * half + (c >> 5)];
                            float a, b;
                            unpair(fma2(pair(__uint_as_float(sk[c & 31]), __uint_as_float(sk[(c & 31) + 1])), scale2, ref2), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            sum2[(c >> 1) & 3] = add2(sum2[(c >> 1) & 3], pair(a, b));
                            // the weights enter the product as bf16, as the tensor
                            // core takes them; their sum is of the unrounded ones.
                            // (The sum of the rounded ones, as decode takes it, has
                            // no better a bound than 2^-8 of the weighted values, for two
                            // more operations a pair in the loop that the long
                            // prompts wait for.)
                            pk[c >> 1] = pack_bf16x2(a, b);
                        }
                        tmem_st32(t_s + 32 * half, pk);
                    }
                    float s0, s1;
                    unpair(add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3])), s0, s1);
                    l = s0 + s1;
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&m.p_full[stream]));
            }
            if (!ok) break;
            if (count > 0) {
                ok = wait_for(smem_u32(&m.o_full[stream]), n_o & 1, abort_flag, p.err);
                ++n_o;
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                tc_fence_after();
            }

            // the row's state: maximum (log2 units; any finite value says that the row sees a key) and sum
            float2 st = make_float2(any ? (mx == -INFINITY ? -FLT_MAX : mx * p.scale_log2) : -INFINITY, l);
            const bool whole = it.whole;
            const int t_lo = max(first_masked, it.ta), t_hi = it.ta + it.count;
            const uint32_t(*bad)[4] = m.bad[n_item % kPieces];
            const long long slot = it.slot;

            // what the sum is divided by; no key seen: zeros; only keys of weight zero: NaN, as 0 / 0
            auto inverse = [](const float2& v) {
                return v.y == 0.f ? (v.x == -INFINITY ? 0.f : __int_as_float(0x7FC00000)) : 1.f / v.y;
            };
            // The row's result is acc0 * f0 + acc1 * f1: of two tiles this stream's
            // accumulator; of one tile both streams' accumulators joined, half of the
            // columns in each warpgroup.
            int col_lo = 0, col_hi = kDim, t_end = t_hi, prow = row;  // t_end: end of the tiles that it holds
            uint32_t acc0 = t_o, acc1 = t_o;
            float f0 = 1.f, f1 = 0.f;
            bool has0 = count > 0, has1 = false;
            if (!kOne && it.two) {
                t_end = min(t_hi, it.ta + count);
                prow += stream * kRows;
            } else {
                col_lo = stream * 64;
                col_hi = col_lo + 64;
                m.ml[stream][row] = st;
                if (!meet(0)) break;
                const float2 s0 = m.ml[0][row], s1 = m.ml[1][row];
                st.x = fmaxf(s0.x, s1.x);
                f0 = s0.x == st.x ? 1.f : ex2(s0.x - st.x);
                f1 = s1.x == st.x ? 1.f : ex2(s1.x - st.x);
                st.y = s0.y * f0 + s1.y * f1;
                acc0 = tmem + lanes + kTmemO;
                acc1 = acc0 + 128;
                has0 = it.cnt[0] > 0;
                has1 = it.cnt[1] > 0;
            }
            const int out_row = valid ? tok * p.hq + it.h * p.group + row_head : -1;  // below 2^31: 256 bytes each
            const long long part_row0 = slot * 2 * kRows + (prow - lane);
            if (warp_valid) {
                if (whole) {
                    const float inv = inverse(st);
                    f0 *= inv;
                    f1 *= inv;
                } else if (valid && (it.two || stream == 0)) {
                    p.part_ml[part_row0 + lane] = st;
                }
                // The results leave through shared memory, 128 bytes of each of the warp's
                // 32 rows at a time, so that a store covers whole lines of 4 rows where one
                // from the accumulator's rows would touch 32 lines. 64 columns a turn: the
                // turns' latencies are what an item's end waits for.
                uint8_t* const staging = smem + L::kOut + warp * kOutBytes;
                auto chunk = [&](int r, int c) { return reinterpret_cast<uint4*>(staging + r * 128 + ((c ^ (r & 7)) << 4)); };
                const int r0 = lane >> 3, c0 = lane & 7;  // the lane's rows r0 + 4 k and its 16 bytes of each
                const uint64_t f0x2 = pair(f0, f0), f1x2 = pair(f1, f1);
#pragma unroll 1
                for (int col = col_lo; col < col_hi; col += 64) {
                    uint32_t r[2][32];
                    tmem_ld32(r[0], acc0 + col);
                    tmem_ld32(r[1], acc0 + col + 32);
                    tmem_wait_ld(r[0]);
                    hold(r[1]);
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        uint32_t* const x = &r[c >> 5][c & 31];
                        float a, b;
                        unpair(mul2(pair(__uint_as_float(x[0]), __uint_as_float(x[1])), f0x2), a, b);
                        x[0] = __float_as_uint(a);
                        x[1] = __float_as_uint(b);
                    }
                    if (has1) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t r1[32];
                            tmem_ld32(r1, acc1 + col + 32 * h);
                            tmem_wait_ld(r1);
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                float a, b;
                                unpair(fma2(pair(__uint_as_float(r1[c]), __uint_as_float(r1[c + 1])), f1x2,
                                            pair(__uint_as_float(r[h][c]), __uint_as_float(r[h][c + 1]))), a, b);
                                r[h][c] = __float_as_uint(a);
                                r[h][c + 1] = __float_as_uint(b);
                            }
                        }
                    }
                    if (!has0) {
#pragma unroll
                        for (int c = 0; c < 64; ++c) r[c >> 5][c & 31] = 0u;
                    }
                    if (whole) {
                        auto two = [&](int c) { return pack_bf16x2(__uint_as_float(r[c >> 5][c & 31]), __uint_as_float(r[c >> 5][(c & 31) + 1])); };
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *chunk(lane, c) = make_uint4(two(8 * c), two(8 * c + 2), two(8 * c + 4), two(8 * c + 6));
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint4 v = *chunk(r0 + 4 * k, c0);
                            const int orow = __shfl_sync(0xFFFFFFFFu, out_row, r0 + 4 * k);
                            if (orow >= 0) *reinterpret_cast<uint4*>(p.out + static_cast<long long>(orow) * kDim + col + c0 * 8) = v;
                        }
                        __syncwarp();
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                *chunk(lane, c) = make_uint4(r[h][4 * c], r[h][4 * c + 1], r[h][4 * c + 2], r[h][4 * c + 3]);
                            __syncwarp();
                            float* const dst = p.part_o + (part_row0 + r0) * kDim + col + 32 * h + c0 * 4;
#pragma unroll
                            for (int k = 0; k < 8; ++k)  // rows that are none are written too: they are the workspace's
                                *reinterpret_cast<uint4*>(dst + 4 * k * kDim) = *chunk(r0 + 4 * k, c0);
                            __syncwarp();
                        }
                    }
                }
            }
            if (!it.two) {
                // both accumulators are read before either is written again
                if (!meet(1)) break;
                ++n_join;
            }
            if (*const_cast<const volatile int*>(&it.any_bad) && valid && t_lo < t_end) {
                add_non_finite<kTree>(p, it, t_lo, t_end, bad, vis, draft_mask, col_lo, col_hi,
                                      whole ? p.out + static_cast<long long>(out_row) * kDim : nullptr,
                                      p.part_o + (part_row0 + lane) * kDim);
            }
            done_piece(n_item);
        }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
      if (warp == kWarpLoad) {
        // ---- loader: query tiles, then K and V tiles in the order of their use
        uint32_t stage = 0, phase = 0, n_q = 0, n_clean = 0, n_item = 0;
        Walk<kTree, kOne> walk(p, m);
        const int bt_shift = 31 - __clz(p.bt), tile_shift = 7 - bt_shift;
        const int blocks_per_tile = 1 << tile_shift, block_rows = p.hkv << (bt_shift - 3);  // row groups of a block
        bool ok = true;
        // One piece is described ahead of the one that is loaded, and its query rows
        // are brought into L2 meanwhile.
        auto describe = [&](bool more) {
            ok = wait_for(smem_u32(&m.piece_empty[n_item % kPieces]), ((n_item / kPieces) & 1) ^ 1, abort_flag, p.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) return;
            if (lane == 0) {
                if (more) walk.describe(m.piece[n_item % kPieces]);
                else m.piece[n_item % kPieces].count = -1;
                mbar_arrive(smem_u32(&m.piece_full[n_item % kPieces]));
            }
            __syncwarp();
            ++n_item;
        };
        bool more = walk.next();
        describe(more);
        while (ok && more) {
            const Piece& it = m.piece[(n_item - 1) % kPieces];  // only this warp replaces it, kPieces later
            more = walk.next();
            describe(more);
            if (!ok) break;
            if (more && lane < 4 && (walk.it.two || lane < 2))
                tma_prefetch_5d(&tm_q, 0, 0, walk.it.tok0 + (lane >> 1) * p.tpt, lane & 1, walk.it.h);
            const int ta = it.ta, count = it.count;
            if (count == 0) continue;
            // What a load needs, in registers: at 1,500 cycles a load, as a plain loop
            // took, the loader bounds the kernel (two loads a key tile).
            const bool two = !kOne && it.two;
            const int masked0 = max(it.first_masked, ta) - ta;  // first masked tile of the piece
            const int head = it.h, draft_tile = kTree ? it.nct - ta : count, draft_row = it.seq_tok0 + lane * 8;
            const int blocks = min(count, it.nct - ta) > 0 ? (it.kend - ta * kKeys + p.bt - 1) >> bt_shift : 0;  // from the piece's first on
            const int draft_boxes = (it.seq_n + 7) >> 3, head_row = head << (bt_shift - 3);
            const int32_t* const table = p.block_tables + static_cast<long long>(it.s) * p.max_blocks + (ta << tile_shift);
            // this lane's block of a tile, read from the table a tile early; and its
            // box's last coordinate in the map
            auto table_entry = [&](int j) {
                const int idx = (j << tile_shift) + lane;
                return j < count && lane < blocks_per_tile && idx < blocks ? __ldg(table + idx) : 0;
            };
            auto coordinate = [&](int j, int blk) {
                if (kTree && j == draft_tile) return draft_row;
                if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
                    atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
                    blk = 0;
                }
                return blk * block_rows + head_row;
            };
            int blk_next = table_entry(0), coord_k = 0, coord_v = 0;  // of K's tile; of the V tile to come
#pragma unroll 1
            for (int pos = 0; pos < 2 * count; ++pos) {
                const RingEntry en = ring_entry(two, pos, count);
                if (!en.is_v) {
                    const int c = coordinate(en.j, blk_next);
                    blk_next = table_entry(en.j + 1);
                    coord_v = two || pos == 0 ? c : coord_k;
                    coord_k = c;
                }
                const int coord = en.is_v ? coord_v : coord_k;
                if (en.is_v) coord_v = coord_k;
                const bool draft = kTree && en.j == draft_tile;
                const int boxes = draft ? draft_boxes : min(blocks - (en.j << tile_shift), blocks_per_tile);
                const uint32_t box_shift = draft ? 11 : bt_shift + 8;
                uint32_t full = smem_u32(&m.kv_full[stage]);
                ok = wait_for(smem_u32(&m.kv_empty[stage]), phase ^ 1, abort_flag, p.err);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (en.is_v && en.j >= masked0) {
                    // a value tile to be cleaned lands on a barrier of its own: the
                    // cleaning warps see no other tile, and could not follow the
                    // ring's phases
                    if (lane == 0) mbar_arrive(full);
                    full = smem_u32(&m.part_full[n_clean % kCleanBars]);
                    ++n_clean;
                }
                if (lane == 0) mbar_arrive_expect_tx(full, boxes << box_shift);
                if (lane < boxes) {
                    const uint32_t dst = smem_base + L::kRing + stage * kTileBytes + (lane << box_shift);
                    if (draft) tma_load_4d(dst, en.is_v ? &tm_vd : &tm_kd, 0, coord, 0, head, full);
                    else tma_load_4d(dst, en.is_v ? &tm_v : &tm_k, 0, 0, 0, coord, full);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
                if (pos == 0) {
                    ok = wait_for(smem_u32(&m.q_empty), (n_q & 1) ^ 1, abort_flag, p.err);
                    ++n_q;
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const int halves = two ? 4 : 2;
                    if (lane == 0) mbar_arrive_expect_tx(smem_u32(&m.q_full), halves * 128 * p.group * p.tpt);
                    if (lane < halves)
                        tma_load_5d(smem_base + L::kQ + lane * (kTileBytes / 2), &tm_q, 0, 0, it.tok0 + (lane >> 1) * p.tpt, lane & 1,
                                    head, smem_u32(&m.q_full));
                }
            }
        }
    } else if (warp == kWarpMma) {
        // ---- tensor core: one elected thread issues every product, P V of a
        // stream's key tile and S of its next one in one go. The tensor core queues
        // only two or three products, so whatever the issuer waits for between them
        // shows as idle time; and issued from one place the streams take turns, one
        // multiplying while the other takes exponentials (an issuer for each let
        // both do the same at the same time). The warp stays converged and its
        // counters provably uniform: in one diverged lane, issuing the 8 products of
        // a tile took 620-900 cycles against the 512 they run for.
        constexpr uint32_t kIdescS = mma_idesc(kRows, kKeys, false), kIdescO = mma_idesc(kRows, kDim, true);
        const uint32_t tm = uniform(tmem), base = uniform(smem_base);
        uint32_t ring = 0, n_q = 0, n_clean = 0, n_p0 = 0, n_p1 = 0;  // n_p: tiles of each stream so far
        bool ok = true;
        for (uint32_t n_item = 0; ok; ++n_item) {
            const Piece* const piece = get_piece(n_item);
            if (!piece) break;
            const int count = uniform(piece->count);
            const bool two = !kOne && uniform(piece->two) != 0;
            const int cnt0 = uniform(piece->cnt[0]), cnt1 = uniform(piece->cnt[1]);
            const int masked0 = uniform(max(piece->first_masked - piece->ta, 0));  // first masked tile of the piece
            done_piece(n_item);
            if (count == 0) continue;
            struct Step {
                bool has_v, has_k, last_k;
                uint32_t st_v, st_k, bar_v, bar_k, bar_p, par_v, par_k, par_p;
            };
            auto step_at = [&](int turn) {
                const int stream = turn & 1, i = turn >> 1, n = stream ? cnt1 : cnt0;
                const int jv = two ? i : 2 * i + stream, jk = two ? i + 1 : jv + 2;
                const uint32_t at_v = ring + ring_v(two, jv, count), at_k = ring + ring_k(two, jk), c = n_clean + (jv - masked0);
                Step x;
                x.has_v = i >= 0 && i < n;
                x.has_k = i + 1 < n;
                x.last_k = jk == count - 1;
                x.st_v = at_v % kStages;
                x.st_k = at_k % kStages;
                const bool cleaned = jv >= masked0;
                x.bar_v = cleaned ? smem_u32(&m.clean[c % kCleanBars]) : smem_u32(&m.kv_full[x.st_v]);
                x.par_v = cleaned ? (c / kCleanBars) & 1 : (at_v / kStages) & 1;
                x.bar_k = smem_u32(&m.kv_full[x.st_k]);
                x.par_k = (at_k / kStages) & 1;
                x.bar_p = smem_u32(&m.p_full[stream]);
                x.par_p = ((stream ? n_p1 : n_p0) + i) & 1;
                return x;
            };
            ok = wait_for(smem_u32(&m.q_full), n_q & 1, abort_flag, p.err);
            ++n_q;
            // S of each stream's first tile, then P V of tile i with S of tile i + 1,
            // the streams in turn. A step waits for its V and K tile and its P.
            const int turns = 2 * max(cnt0, cnt1);
            auto issue_s = [&](uint32_t t_s, uint32_t dq, uint32_t dk, int k) {
                mma_ss<desc_high(1024), desc_high(2048), kIdescS>(t_s, dq + (((k >> 2) * (kTileBytes / 2) + (k & 3) * 32) >> 4),
                       dk + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), k > 0);
            };
            auto issue_o = [&](uint32_t t_s, uint32_t dv, int k, bool accumulate) {
                mma_ts<desc_high(2048), kIdescO>(t_s + kTmemO, t_s + k * 8, dv + ((k * 4096) >> 4), accumulate);
            };
            auto tile_at = [&](uint32_t at) { return base + L::kRing + (at % kStages) * kTileBytes; };
            const uint32_t dq0 = desc_low(base + L::kQ, 16), dq1 = two ? desc_low(base + L::kQ + kTileBytes, 16) : dq0;
            // Two query tiles, both with a tile to come that every row sees in full: the
            // same steps in as little as it takes, since a scalar instruction of this
            // warp costs up to 10 cycles beside the softmax warps', and what is not
            // hidden behind the two or three queued products (a look at the next
            // barriers before a step's last three) leaves the tensor core idle.
            const int fast = two ? min(cnt0 - 1, masked0) : 0;
            ok = __all_sync(0xFFFFFFFFu, ok);
#pragma unroll 1
            for (int turn = -2; ok && turn < turns; ++turn) {
                if (!kOne && turn == 0 && fast > 0) {
                    const uint32_t p0 = smem_u32(&m.p_full[0]), p1 = smem_u32(&m.p_full[1]);
                    bool ready = false;
#pragma unroll 1
                    for (int i = 0; i < fast; ++i) {
                        const uint32_t at = ring + 2 * i + 1;  // V of tile i, then K of tile i + 1
                        const uint32_t dv = desc_low(tile_at(at), 1024), dk = desc_low(tile_at(at + 1), 16);
                        if (!ready) {
                            ok = wait_for(smem_u32(&m.kv_full[at % kStages]), (at / kStages) & 1, abort_flag, p.err);
                            if (ok) ok = wait_for(smem_u32(&m.kv_full[(at + 1) % kStages]), ((at + 1) / kStages) & 1, abort_flag, p.err);
                            if (ok) ok = wait_for(p0, (n_p0 + i) & 1, abort_flag, p.err);
                            ok = __all_sync(0xFFFFFFFFu, ok);
                            if (!ok) break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) issue_o(tm, dv, k, i > 0 || k > 0);
#pragma unroll
                            for (int k = 0; k < 5; ++k) issue_s(tm, dq0, dk, k);
                        }
                        __syncwarp();
                        ready = __all_sync(0xFFFFFFFFu, mbar_test(p1, (n_p1 + i) & 1));
                        if (elect_one()) {
#pragma unroll
                            for (int k = 5; k < 8; ++k) issue_s(tm, dq0, dk, k);
                            mma_commit(smem_u32(&m.s_full[0]));
                        }
                        __syncwarp();
                        if (!ready) {
                            ok = __all_sync(0xFFFFFFFFu, wait_for(p1, (n_p1 + i) & 1, abort_flag, p.err));
                            if (!ok) break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) issue_o(tm + 128, dv, k, i > 0 || k > 0);
                            mma_commit(smem_u32(&m.kv_empty[at % kStages]));
#pragma unroll
                            for (int k = 0; k < 5; ++k) issue_s(tm + 128, dq1, dk, k);
                        }
                        __syncwarp();
                        ready = mbar_test(p0, (n_p0 + i + 1) & 1) & mbar_test(smem_u32(&m.kv_full[(at + 2) % kStages]), ((at + 2) / kStages) & 1) &
                                mbar_test(smem_u32(&m.kv_full[(at + 3) % kStages]), ((at + 3) / kStages) & 1);
                        ready = __all_sync(0xFFFFFFFFu, ready) && i + 1 < fast;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 5; k < 8; ++k) issue_s(tm + 128, dq1, dk, k);
                            mma_commit(smem_u32(&m.s_full[1]));
                            mma_commit(smem_u32(&m.kv_empty[(at + 1) % kStages]));
                            if (i + 2 == count) mma_commit(smem_u32(&m.q_empty));
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    turn = 2 * fast;
                }
                const Step now = step_at(turn);
                if (!now.has_v && !now.has_k) continue;
                const uint32_t t_s = tm + (turn & 1) * 128;
                const bool last_user = !two || (turn & 1);  // of a key tile
                if (now.has_v) {
                    ok = wait_for(now.bar_v, now.par_v, abort_flag, p.err);
                    // (one-tile items are bound by their loads: there the product that
                    // frees a stage does not wait for the next key tile)
                    if (!kOne && ok && now.has_k) ok = wait_for(now.bar_k, now.par_k, abort_flag, p.err);
                    if (ok) ok = wait_for(now.bar_p, now.par_p, abort_flag, p.err);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t dv = desc_low(base + L::kRing + now.st_v * kTileBytes, 1024);
#pragma unroll
                        for (int k = 0; k < 8; ++k) issue_o(t_s, dv, k, turn >= 2 || k > 0);
                        if (last_user) mma_commit(smem_u32(&m.kv_empty[now.st_v]));
                        if (!now.has_k) mma_commit(smem_u32(&m.o_full[turn & 1]));
                    }
                    __syncwarp();
                }
                if (now.has_k) {
                    if (kOne || !now.has_v) {
                        ok = __all_sync(0xFFFFFFFFu, wait_for(now.bar_k, now.par_k, abort_flag, p.err));
                        if (!ok) break;
                        tc_fence_after();
                    }
                    if (elect_one()) {
                        const uint32_t dk = desc_low(base + L::kRing + now.st_k * kTileBytes, 16), dq = turn & 1 ? dq1 : dq0;
#pragma unroll
                        for (int k = 0; k < 8; ++k) issue_s(t_s, dq, dk, k);
                        mma_commit(smem_u32(&m.s_full[turn & 1]));
                        if (last_user) mma_commit(smem_u32(&m.kv_empty[now.st_k]));
                        if (last_user && now.last_k) mma_commit(smem_u32(&m.q_empty));
                    }
                    __syncwarp();
                }
            }
            n_p0 += cnt0;
            n_p1 += cnt1;
            ring += 2 * count;
            n_clean += max(count - masked0, 0);
        }
    } else {
        // ---- value tiles that not every row sees in full
        const int half = warp - kWarpClean;
        uint32_t n_clean = 0;
        bool ok = true;
        for (uint32_t n_item = 0, ring = 0; ok; ++n_item) {
            const Piece* const piece = get_piece(n_item);
            if (!piece) break;
            const int count = piece->count;
            const int masked0 = max(piece->first_masked - piece->ta, 0);
#pragma unroll 1
            for (int j = masked0; ok && j < count; ++j, ++n_clean) {
                const uint32_t st = (ring + ring_v(piece->two, j, count)) % kStages;
                const int t = piece->ta + j;
                const int valid = kTree && t == piece->nct ? piece->seq_n : min(kKeys, piece->kend - t * kKeys);
                ok = __all_sync(0xFFFFFFFFu, wait_for(smem_u32(&m.part_full[n_clean % kCleanBars]),
                                                       (n_clean / kCleanBars) & 1, abort_flag, p.err));
                if (!ok) break;
                uint8_t* tile = smem + L::kRing + st * kTileBytes;
#pragma unroll 1
                for (int r = 0; r < 2; ++r) {
                    const int row = half * 64 + r * 32 + lane;
                    uint8_t* const row_at = tile + (row >> 3) * 2048 + (row & 7) * 128;
                    bool bad = false;
#pragma unroll 1
                    for (int side = 0; side < 2; ++side) bad |= clean_half_row(row_at + side * 1024, lane, row < valid);
                    const uint32_t word = __ballot_sync(0xFFFFFFFFu, bad);
                    if (lane == 0) {
                        m.bad[n_item % kPieces][j - masked0][half * 2 + r] = word;
                        if (word) atomicOr(&m.piece[n_item % kPieces].any_bad, 1);
                    }
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&m.clean[n_clean % kCleanBars]));
            }
            ring += 2 * count;
            done_piece(n_item);
        }
      }
    }
    __syncthreads();
    if (*abort_flag) {
        // copies and products of a broken pipeline may still be under way
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {}
        __syncthreads();
    }
    if (warp == kWarpMma) tmem_free(tmem, kTmemColumns);
}

// Joins the pieces of the items that cuts split: kEvery, block x serves the item
// that CTA x describes, if it does; else, where there are fewer items than CTAs,
// the x-th of them (and every gridDim.x-th behind it), so that more blocks can
// share its rows (y). A warp takes
// kMergeRows rows of all pieces, read kMergeAhead at a time (one row of one
// piece at a time, the kernel was as long as their latencies: 13 us behind the
// ragged prompts' 65); of an item in more than kMergeShare pieces -- few rows on
// a long context -- the warps share the pieces instead and join their results.
// 8 drafts on 60,000 keys of one head, 150 pieces: 25 us for both kernels, 118
// when one warp read all pieces of its rows; where there are two or three pieces
// an item the search costs 1 to 2 us. The order of the sums is the same in every
// run.
constexpr int kMergeWarps = 8, kMergeRows = 4, kMergeAhead = 2, kMergeShare = 8;

struct RowSums {
    float m, l;  // maximum (log2 units), sum of weights
    float4 o;    // this lane's 4 columns

    __device__ __forceinline__ void add(float m2, float l2, const float4& o2) {
        if (m2 == -INFINITY) return;  // sees no key of the piece, or is not a row
        const float top = fmaxf(m, m2);
        const float fa = m == top ? 1.f : ex2(m - top), fb = m2 == top ? 1.f : ex2(m2 - top);
        m = top;
        l = l * fa + l2 * fb;
        o.x = o.x * fa + o2.x * fb;
        o.y = o.y * fa + o2.y * fb;
        o.z = o.z * fa + o2.z * fb;
        o.w = o.w * fa + o2.w * fb;
    }
};

template <bool kEvery, bool kLoop>
__global__ void __launch_bounds__(kMergeWarps * 32, kEvery && !kLoop ? 3 : 2) merge_kernel(const Params p) {
    __shared__ int slots[kMaxGrid];  // of the ranges from the first piece's on; -1: no piece in it
    __shared__ int last, item, marks[kMergeWarps];
    __shared__ float4 shared_o[kMergeWarps][kMergeRows][32];
    __shared__ float2 shared_ml[kMergeWarps][kMergeRows];
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) last = kMaxGrid;
    __syncthreads();
    griddep_wait();
    // the CTA that describes this block's item
    int c0 = blockIdx.x, ranges = p.grid;
    if (kLoop) {
        ranges *= *const_cast<const volatile int*>(p.rounds);
    }
    int rank = blockIdx.x, found = 0;  // !kEvery: of the item among the split ones; how many those are
    auto find = [&] {
        found = 0;
        for (int base = 0; base < p.grid; base += kMergeWarps * 32) {
            const int c = base + threadIdx.x;
            const bool split = c < p.grid && p.splits[c].ntiles != 0;
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, split);
            if (lane == 0) marks[warp] = __popc(mask);
            __syncthreads();
            int at = found + __popc(mask & ((1u << lane) - 1u));
            for (int w = 0; w < kMergeWarps; ++w) {
                if (w < warp) at += marks[w];
                found += marks[w];
            }
            if (split && at == rank) item = c;
            __syncthreads();
        }
        return rank < found ? item : ranges;
    };
    auto next = [&] {
        if (kEvery) return c0 + (kLoop ? static_cast<int>(gridDim.x) : ranges);
        // one turn, but where query_starts lays sequences over the same rows: then
        // there are more items than the host counted
        rank += gridDim.x;
        return rank < found ? find() : ranges;
    };
    if (!kEvery) c0 = find();
#pragma unroll 1
    for (; c0 < ranges; c0 = next()) {
        const Split sp = p.splits[c0];
        if (sp.ntiles == 0) continue;
        const int block_rows = (p.one ? 1 : 2) * kRows / gridDim.y;
        auto row_token = [&](int r) { return (r >> 7) * p.tpt + (r & 127) / p.group; };  // the second query tile starts at row 128
        if (row_token(blockIdx.y * block_rows) >= sp.ntok) continue;
        auto tiles_before = [&](int c) {  // tiles of the item in the ranges up to c0 + c
            const long long end = sp.chunk * (c0 + c + 1) - sp.start;
            return end >= sp.cost ? sp.ntiles : cut_tile(end, sp.cost, sp.ntiles);
        };
        // the piece in the c-th range from the first piece's on, -1 if there is none
        auto slot_of = [&](int c, bool& ends) {
            const int t = tiles_before(c), before = c == 0 ? 0 : tiles_before(c - 1);
            ends = t == sp.ntiles || c0 + c == ranges - 1;
            return t > before ? 2 * (c0 + c) + (c == 0 ? 1 : 0) : -1;
        };

        RowSums sums[kMergeRows];
        auto gather = [&](int first, int from, int to, auto slot_at) {
#pragma unroll
            for (int i = 0; i < kMergeRows; ++i) sums[i] = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
            for (int c = from; c < to; c += kMergeAhead) {
                float2 st[kMergeAhead][kMergeRows];
                float4 v[kMergeAhead][kMergeRows];
#pragma unroll
                for (int a = 0; a < kMergeAhead; ++a) {
                    const int slot = c + a < to ? slot_at(c + a) : -1;
#pragma unroll
                    for (int i = 0; i < kMergeRows; ++i) {
                        st[a][i] = make_float2(-INFINITY, 0.f);
                        v[a][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (slot < 0) continue;
                        const long long row = static_cast<long long>(slot) * 2 * kRows + first + i;
                        st[a][i] = p.part_ml[row];
                        v[a][i] = *reinterpret_cast<const float4*>(p.part_o + row * kDim + lane * 4);
                    }
                }
#pragma unroll
                for (int a = 0; a < kMergeAhead; ++a)
#pragma unroll
                    for (int i = 0; i < kMergeRows; ++i) sums[i].add(st[a][i].x, st[a][i].y, v[a][i]);
            }
        };
        auto store = [&](int row, const RowSums& x) {
            const int r = row & 127, row_tok = r / p.group, tok = row_token(row);
            if (row_tok >= p.tpt || tok >= sp.ntok) return;
            const float inv = x.l != 0.f ? 1.f / x.l : x.m == -INFINITY ? 0.f : __int_as_float(0x7FC00000);
            const int head = sp.head0 + r - row_tok * p.group;
            *reinterpret_cast<uint2*>(p.out + (static_cast<long long>(sp.tok0 + tok) * p.hq + head) * kDim + lane * 4) =
                make_uint2(pack_bf16x2(x.o.x * inv, x.o.y * inv), pack_bf16x2(x.o.z * inv, x.o.w * inv));
        };
        bool ends;
        const int mine = slot_of(lane, ends);
        const int few = __ffs(__ballot_sync(0xFFFFFFFFu, ends));
        if (few != 0 && few <= kMergeShare) {
            for (int g = warp; g < block_rows / kMergeRows; g += kMergeWarps) {
                const int first = blockIdx.y * block_rows + g * kMergeRows;
                gather(first, 0, few, [&](int c) { return __shfl_sync(0xFFFFFFFFu, mine, c); });
#pragma unroll
                for (int i = 0; i < kMergeRows; ++i) store(first + i, sums[i]);
            }
            continue;
        }
        for (int c = threadIdx.x; c0 + c < ranges; c += blockDim.x) {
            slots[c] = slot_of(c, ends);
            if (ends) atomicMin(&last, c);
        }
        __syncthreads();
        const int pieces = last + 1;
        for (int g = 0; g < block_rows / kMergeRows; ++g) {
            const int first = blockIdx.y * block_rows + g * kMergeRows;
            if (row_token(first) >= sp.ntok) break;
            gather(first, pieces * warp / kMergeWarps, pieces * (warp + 1) / kMergeWarps,
                   [&](int c) { return slots[c]; });
#pragma unroll
            for (int i = 0; i < kMergeRows; ++i) {
                shared_o[warp][i][lane] = sums[i].o;
                if (lane == 0) shared_ml[warp][i] = make_float2(sums[i].m, sums[i].l);
            }
            __syncthreads();
            if (warp < kMergeRows) {
                RowSums x = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
                for (int w = 0; w < kMergeWarps; ++w) x.add(shared_ml[w][warp].x, shared_ml[w][warp].y, shared_o[w][warp][lane]);
                store(first + warp, x);
            }
            __syncthreads();
        }
        if (kEvery && !kLoop) return;
        if (threadIdx.x == 0) last = kMaxGrid;  // every warp has read it
        __syncthreads();
    }
}

}  // namespace prefill
}  // namespace pkv
