// Attention of many query rows per sequence over the paged cache: causal
// prompt attention (pkv_attn_prefill) and draft-tree attention
// (pkv_attn_tree).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <vector>

#include "pkv_internal.h"
#include "pkv_prefill_kernel.cuh"

namespace pkv {
namespace prefill {

using KernelFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, Params);

KernelFn kernel_for(bool tree, bool one) {
    if (one) return tree ? rows_kernel<true, true> : rows_kernel<false, true>;
    return tree ? rows_kernel<true, false> : rows_kernel<false, false>;
}

size_t smem_for(bool one) { return one ? Smem<true>::kBytes : Smem<false>::kBytes; }

// Per device, once: its SMs, and leave for the kernels' shared memory.
struct DeviceInfo {
    bool ok = false;
    int grid = 0;
};

DeviceInfo device_info() {
    static std::mutex mu;
    static std::vector<DeviceInfo> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return {};
    std::lock_guard<std::mutex> lock(mu);
    if (static_cast<int>(cache.size()) <= dev) cache.resize(dev + 1);
    DeviceInfo& d = cache[dev];
    if (d.ok) return d;
    int sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    for (const bool tree : {false, true})
        for (const bool one : {false, true}) {
            const KernelFn fn = kernel_for(tree, one);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem_for(one)));
            // the kernels move registers between their warpgroups: a launch with
            // fewer than they count on would wait for ever
            cudaFuncAttributes at = {};
            if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, fn);
            if (e == cudaSuccess && at.numRegs < kRegsLaunch) e = cudaErrorInvalidDeviceFunction;
        }
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return {};
    }
    d.grid = std::min(sms, kMaxGrid / kRounds);
    d.ok = true;
    return d;
}

// Workspace: header (error word), split items, then each range's two slots of
// 256 row states and 256 rows of 128 fp32 values.
constexpr size_t kWsRounds = 64, kWsSplits = kWsHeader, kWsStates = kWsSplits + sizeof(Split) * kMaxGrid;
static_assert(kWsStates % 256 == 0, "alignment of the partial results");

size_t workspace_bytes(int grid) {
    return kWsStates + static_cast<size_t>(grid) * kRounds * 2 * 2 * kRows * (sizeof(float2) + kDim * sizeof(float));
}

bool encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    const auto enc = tensor_map_encoder();
    return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows: {64 columns, group heads, tokens, 2 column halves, KV heads};
// a box is one half of a tile's tokens with their heads, one 128-byte row each.
bool query_map(CUtensorMap* map, const void* q, int tokens, int hq, int hkv, int tpt) {
    const cuuint64_t g = hq / hkv;
    const cuuint64_t dims[5] = {64, g, static_cast<cuuint64_t>(tokens), 2, static_cast<cuuint64_t>(hkv)};
    const cuuint64_t strides[4] = {256, static_cast<cuuint64_t>(hq) * 256, 128, g * 256};
    const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(g), static_cast<cuuint32_t>(tpt), 1, 1};
    return encode(map, q, 5, dims, strides, box);
}

// A cache as groups of 8 rows: {64 columns, 8 rows, 2 column halves, groups}.
// A box is one block of one KV head; each of its row groups lands as its two
// halves, one 1024-byte swizzle atom each.
bool cache_map(CUtensorMap* map, const void* cache, int num_blocks, int hkv, int bt) {
    const cuuint64_t dims[4] = {64, 8, 2, static_cast<cuuint64_t>(num_blocks) * hkv * (bt / 8)};
    const cuuint64_t strides[3] = {256, 128, 2048};
    const cuuint32_t box[4] = {64, 8, 2, static_cast<cuuint32_t>(bt / 8)};
    return encode(map, cache, 4, dims, strides, box);
}

// Drafted keys or values, 8 tokens of one KV head a box, landing likewise.
bool draft_map(CUtensorMap* map, const void* rows, int tokens, int hkv) {
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(tokens), 2, static_cast<cuuint64_t>(hkv)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(hkv) * 256, 128, 256};
    const cuuint32_t box[4] = {64, 8, 2, 1};
    return encode(map, rows, 4, dims, strides, box);
}

pkv_status run(const void* q, const void* k_cache, const void* v_cache, const void* k_draft, const void* v_draft,
               const int64_t* masks, bool tree, const int32_t* block_tables, int max_blocks_per_seq,
               const int32_t* context_lens, const int32_t* query_starts, int num_seqs, int num_tokens, int num_q_heads,
               int num_kv_heads, int head_dim, int num_blocks, int block_tokens, float scale, void* workspace,
               size_t ws_bytes, void* out, cudaStream_t stream) {
    if (block_tokens != 8 && block_tokens != 16 && block_tokens != 32 && block_tokens != 64) return PKV_EUNSUPPORTED;
    if (num_tokens < 0 || num_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1 || num_blocks < 1 ||
        max_blocks_per_seq < 1 || !std::isfinite(scale) || scale < 0.f)
        return PKV_EINVAL;
    if (num_seqs > PKV_ATTN_MAX_SEQS || head_dim != kDim || num_q_heads % num_kv_heads != 0 ||
        num_q_heads / num_kv_heads > PKV_ATTN_MAX_GROUP)
        return PKV_EUNSUPPORTED;
    if (static_cast<long long>(num_blocks) * num_kv_heads * block_tokens >= (1ll << 31) ||
        static_cast<long long>(num_seqs) * max_blocks_per_seq >= (1ll << 31) ||
        static_cast<long long>(max_blocks_per_seq) * block_tokens >= (1ll << 31) || num_tokens >= (1 << 28) ||
        static_cast<long long>(num_tokens) * num_q_heads >= (1ll << 31))
        return PKV_ERANGE;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !query_starts || !workspace || !out ||
        (tree && (!k_draft || !v_draft || !masks)))
        return PKV_EINVAL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(k_draft) ||
        !aligned16(v_draft) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PKV_EINVAL;
    if (ws_bytes < workspace_bytes(1)) return PKV_EINVAL;
    const DeviceInfo d = device_info();
    if (!d.ok) return PKV_ECUDA;
    const size_t per_cta = workspace_bytes(1) - workspace_bytes(0);
    const int grid = static_cast<int>(std::min<size_t>(d.grid, (ws_bytes - workspace_bytes(0)) / per_cta));
    Params p = {};
    p.out = static_cast<__nv_bfloat16*>(out);
    p.v_cache = static_cast<const __nv_bfloat16*>(v_cache);
    p.v_draft = static_cast<const __nv_bfloat16*>(v_draft);
    p.masks = masks;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_starts = query_starts;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.err = reinterpret_cast<uint32_t*>(ws);
    p.splits = reinterpret_cast<Split*>(ws + kWsSplits);
    p.part_ml = reinterpret_cast<float2*>(ws + kWsStates);
    p.part_o = reinterpret_cast<float*>(ws + kWsStates + static_cast<size_t>(grid) * kRounds * 2 * 2 * kRows * sizeof(float2));
    p.rounds = reinterpret_cast<int*>(ws + kWsRounds);
    p.grid = grid;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.tpt = kRows / p.group;
    // Sequences of one query tile each on the average (decode rows, small trees):
    // the kernel of one-tile items, whose ring is deeper.
    const bool one = static_cast<long long>(num_tokens) * p.group <= static_cast<long long>(num_seqs) * kRows;
    p.one = one;
    const int tokens = (one ? 1 : 2) * p.tpt;
    p.item_magic = ((1ull << 36) + tokens - 1) / tokens;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.bt = block_tokens;
    // a scale of zero weighs every seen key alike: as does any scale this
    // small, without 0 * -infinity at the masked ones
    p.scale_log2 = std::max(scale * 1.4426950408889634f, 1e-30f);
    CUtensorMap tm_q, tm_k, tm_v, tm_kd, tm_vd;
    if (!query_map(&tm_q, q, num_tokens, num_q_heads, num_kv_heads, p.tpt) ||
        !cache_map(&tm_k, k_cache, num_blocks, num_kv_heads, block_tokens) ||
        !cache_map(&tm_v, v_cache, num_blocks, num_kv_heads, block_tokens))
        return PKV_ECUDA;
    if (tree) {
        if (!draft_map(&tm_kd, k_draft, num_tokens, num_kv_heads) || !draft_map(&tm_vd, v_draft, num_tokens, num_kv_heads))
            return PKV_ECUDA;
    } else {
        tm_kd = tm_k;  // not read
        tm_vd = tm_v;
    }
    const long long most_keys = static_cast<long long>(max_blocks_per_seq) * block_tokens + (tree ? kKeys : 0);
    // no more items than tiles of tokens and sequences allow
    const long long items = (num_tokens / tokens + static_cast<long long>(num_seqs)) * num_kv_heads;
    // The device takes rounds where the lengths ask for them; the join of a call
    // that may take them is slower by 2 us, so a call of few items a sequence
    // does not.
    p.max_rounds = !tree && !one && num_tokens / tokens >= kRoundReads * num_seqs && items >= 4 * grid &&
                           num_seqs * most_keys * num_kv_heads * (4ll * kDim) > kRoundBytes
                       ? kRounds
                       : 1;
    // Both kernels are launched early (programmatic stream serialization) and
    // wait for the one before, so that they are set up when it ends.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_for(one);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel_for(tree, one), tm_q, tm_k, tm_v, tm_kd, tm_vd, p);
    // an item costs no more than the keys of a table row (cost_of): where that is
    // too little to be cut, there is nothing to join
    if (e == cudaSuccess && kCostTwo * most_keys + cost_item(tree) > kWhole) {
        // where there can be fewer split items than CTAs, 4 to 32 rows a block, for
        // 3 to 6 blocks an SM, else 32 (2,000 rows of 8 heads, 64 items: 27.5 us with
        // 32 rows, 30.5 with 16; 16 items of 9 pieces: 72 us with 8 rows, 78 with 16)
        const int most = static_cast<int>(std::min<long long>(items, grid)), rows = (one ? 1 : 2) * kRows;
        int parts = rows / (kMergeWarps * kMergeRows);
        while (parts < rows / kMergeRows && most < grid && parts * most <= 3 * grid) parts *= 2;
        cfg.gridDim = dim3(most, parts);
        cfg.blockDim = dim3(kMergeWarps * 32);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, most < grid ? merge_kernel<false, false> : p.max_rounds > 1 ? merge_kernel<true, true> : merge_kernel<true, false>, p);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
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
    const prefill::DeviceInfo d = prefill::device_info();
    return d.ok ? prefill::workspace_bytes(d.grid) : 0;
}

pkv_status pkv_attn_prefill(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                            int max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_starts,
                            int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                            int num_blocks, int block_tokens, float scale, void* workspace, size_t workspace_bytes,
                            void* out, void* stream) {
    return prefill::run(q, k_cache, v_cache, nullptr, nullptr, nullptr, false, block_tables, max_blocks_per_seq,
                        context_lens, query_starts, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                        num_blocks, block_tokens, scale, workspace, workspace_bytes, out, as_stream(stream));
}

pkv_status pkv_attn_tree(const void* q, const void* k_draft, const void* v_draft, const int64_t* tree_masks,
                         const void* k_cache, const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                         const int32_t* context_lens, const int32_t* query_starts, int num_seqs, int num_tokens,
                         int num_q_heads, int num_kv_heads, int head_dim, int num_blocks, int block_tokens,
                         float scale, void* workspace, size_t workspace_bytes, void* out, void* stream) {
    return prefill::run(q, k_cache, v_cache, k_draft, v_draft, tree_masks, true, block_tables, max_blocks_per_seq,
                        context_lens, query_starts, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                        num_blocks, block_tokens, scale, workspace, workspace_bytes, out, as_stream(stream));
}

}  // extern "C"
