// Attention of many query rows per sequence over the paged cache: causal
// prompt attention (pkv_attn_prefill) and draft-tree attention
// (pkv_attn_tree).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace prefill {

constexpr int kDim = PKV_ATTN_HEAD_DIM;
constexpr size_t kWsHeader = 256;

struct Params {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_cache;
    const __nv_bfloat16* v_cache;
    const __nv_bfloat16* k_draft;  // null: prefill
    const __nv_bfloat16* v_draft;
    const int64_t* masks;
    __nv_bfloat16* out;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_starts;
    uint32_t* err;
    int num_seqs, num_tokens, hq, hkv, group, max_blocks, num_blocks, bt;
    float scale_log2;
};

constexpr int kWarps = 8;

// One warp per (token, query head), four head dims per lane, one key at a
// time with the running maximum and sum of the softmax.
template <bool kTree>
__global__ void __launch_bounds__(kWarps * 32) rows_kernel(const Params p) {
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int tok = static_cast<int>(w / p.hq);
    if (tok >= p.num_tokens) return;
    const int h = static_cast<int>(w - static_cast<long long>(tok) * p.hq);
    const int g = h / p.group;
    // last sequence that starts at or before the token
    int lo = 0, hi = p.num_seqs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.query_starts + mid + 1) > tok) hi = mid; else lo = mid + 1;
    }
    const int s = lo;
    if (s >= p.num_seqs) return;
    const int start = __ldg(p.query_starts + s), end = __ldg(p.query_starts + s + 1);
    if (tok < start) return;
    uint32_t bad = 0;
    if (start < 0 || end > p.num_tokens) bad |= PKV_DEVERR_QUERY;
    const int first = max(start, 0), last = min(end, p.num_tokens);
    const int n = last - first, i = tok - first;
    if (kTree && n > PKV_TREE_MAX_DRAFTS) bad |= PKV_DEVERR_QUERY;
    if (kTree && i >= PKV_TREE_MAX_DRAFTS) return;
    int ctx = __ldg(p.context_lens + s);
    const long long cap = static_cast<long long>(p.max_blocks) * p.bt;
    if (ctx > cap) {
        bad |= PKV_DEVERR_CONTEXT;
        ctx = static_cast<int>(cap);
    }
    ctx = max(ctx, 0);
    if (!kTree && n > ctx) bad |= PKV_DEVERR_CONTEXT;
    const int seen = kTree ? ctx : max(0, ctx - n + i + 1);

    float q[4];
    const uint2 qv = *reinterpret_cast<const uint2*>(p.q + (static_cast<long long>(tok) * p.hq + h) * kDim + lane * 4);
    q[0] = bf16_lo(qv.x); q[1] = bf16_hi(qv.x); q[2] = bf16_lo(qv.y); q[3] = bf16_hi(qv.y);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    bool any = false;
    auto add = [&](const __nv_bfloat16* kr, const __nv_bfloat16* vr) {
        const uint2 kv = *reinterpret_cast<const uint2*>(kr + lane * 4);
        const uint2 vv = *reinterpret_cast<const uint2*>(vr + lane * 4);
        float x = q[0] * bf16_lo(kv.x) + q[1] * bf16_hi(kv.x) + q[2] * bf16_lo(kv.y) + q[3] * bf16_hi(kv.y);
#pragma unroll
        for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
        x *= p.scale_log2;
        const float m2 = fmaxf(m, x);
        const float ref = m2 == -INFINITY ? 0.f : m2;
        const float a = exp2f(m - ref), e = exp2f(x - ref);
        m = m2;
        l = l * a + e;
        o[0] = o[0] * a + e * bf16_lo(vv.x);
        o[1] = o[1] * a + e * bf16_hi(vv.x);
        o[2] = o[2] * a + e * bf16_lo(vv.y);
        o[3] = o[3] * a + e * bf16_hi(vv.y);
        any = true;
    };
    for (int j = 0; j < seen; ++j) {
        int blk = __ldg(p.block_tables + static_cast<long long>(s) * p.max_blocks + j / p.bt);
        if (blk < 0 || blk >= p.num_blocks) {
            bad |= PKV_DEVERR_BLOCK_ID;
            blk = 0;
        }
        const long long row = (static_cast<long long>(blk) * p.hkv + g) * p.bt + j % p.bt;
        add(p.k_cache + row * kDim, p.v_cache + row * kDim);
    }
    if (kTree) {
        const uint64_t bits = static_cast<uint64_t>(__ldg(reinterpret_cast<const long long*>(p.masks) + tok));
        for (int j = 0; j < min(n, PKV_TREE_MAX_DRAFTS); ++j)
            if (bits >> j & 1) {
                const long long row = static_cast<long long>(first + j) * p.hkv + g;
                add(p.k_draft + row * kDim, p.v_draft + row * kDim);
            }
    }
    const float inv = any ? 1.f / l : 0.f;
    uint2 r;
    r.x = pack_bf16x2(o[0] * inv, o[1] * inv);
    r.y = pack_bf16x2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(p.out + (static_cast<long long>(tok) * p.hq + h) * kDim + lane * 4) = r;
    if (bad && lane == 0) atomicOr(p.err, bad);
}

pkv_status run(const Params& p0, const void* q, const void* k_cache, const void* v_cache, const void* k_draft,
               const void* v_draft, const int64_t* masks, bool tree, const int32_t* block_tables, int max_blocks_per_seq,
               const int32_t* context_lens, const int32_t* query_starts, int num_seqs, int num_tokens, int num_q_heads,
               int num_kv_heads, int head_dim, int num_blocks, int block_tokens, float scale, void* workspace,
               size_t workspace_bytes, void* out, cudaStream_t stream) {
    if (block_tokens != 8 && block_tokens != 16 && block_tokens != 32 && block_tokens != 64) return PKV_EUNSUPPORTED;
    if (num_tokens < 0 || num_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1 || num_blocks < 1 ||
        max_blocks_per_seq < 1 || !std::isfinite(scale) || scale < 0.f)
        return PKV_EINVAL;
    if (num_seqs > PKV_ATTN_MAX_SEQS || head_dim != kDim || num_q_heads % num_kv_heads != 0 ||
        num_q_heads / num_kv_heads > PKV_ATTN_MAX_GROUP)
        return PKV_EUNSUPPORTED;
    if (static_cast<long long>(num_blocks) * num_kv_heads * block_tokens >= (1ll << 31) ||
        static_cast<long long>(num_seqs) * max_blocks_per_seq >= (1ll << 31) ||
        static_cast<long long>(max_blocks_per_seq) * block_tokens >= (1ll << 31))
        return PKV_ERANGE;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !query_starts || !workspace || !out ||
        (tree && (!k_draft || !v_draft || !masks)))
        return PKV_EINVAL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(k_draft) ||
        !aligned16(v_draft) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PKV_EINVAL;
    if (workspace_bytes < kWsHeader) return PKV_EINVAL;
    Params p = p0;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
    p.v_cache = static_cast<const __nv_bfloat16*>(v_cache);
    p.k_draft = static_cast<const __nv_bfloat16*>(k_draft);
    p.v_draft = static_cast<const __nv_bfloat16*>(v_draft);
    p.masks = masks;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_starts = query_starts;
    p.err = static_cast<uint32_t*>(workspace);
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.bt = block_tokens;
    p.scale_log2 = scale * 1.4426950408889634f;
    const long long warps = static_cast<long long>(num_tokens) * num_q_heads;
    const long long grid = (warps + kWarps - 1) / kWarps;
    if (grid >= (1ll << 31)) return PKV_ERANGE;
    if (tree) rows_kernel<true><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(p);
    else rows_kernel<false><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return PKV_ECUDA;
    }
    return PKV_OK;
}

}  // namespace prefill
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_attn_prefill_workspace_size(void) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    return prefill::kWsHeader;
}

pkv_status pkv_attn_prefill(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                            int max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_starts,
                            int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                            int num_blocks, int block_tokens, float scale, void* workspace, size_t workspace_bytes,
                            void* out, void* stream) {
    return prefill::run({}, q, k_cache, v_cache, nullptr, nullptr, nullptr, false, block_tables, max_blocks_per_seq,
                        context_lens, query_starts, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                        num_blocks, block_tokens, scale, workspace, workspace_bytes, out, as_stream(stream));
}

pkv_status pkv_attn_tree(const void* q, const void* k_draft, const void* v_draft, const int64_t* tree_masks,
                         const void* k_cache, const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                         const int32_t* context_lens, const int32_t* query_starts, int num_seqs, int num_tokens,
                         int num_q_heads, int num_kv_heads, int head_dim, int num_blocks, int block_tokens,
                         float scale, void* workspace, size_t workspace_bytes, void* out, void* stream) {
    return prefill::run({}, q, k_cache, v_cache, k_draft, v_draft, tree_masks, true, block_tables, max_blocks_per_seq,
                        context_lens, query_starts, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                        num_blocks, block_tokens, scale, workspace, workspace_bytes, out, as_stream(stream));
}

}  // extern "C"
