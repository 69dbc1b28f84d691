// Decode attention over a paged cache held in 4 bits: the launch and the C ABI
// around decode_kernel (pkv_int4_kernel.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <vector>

#include "pkv_int4_kernel.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace kv4 {

using KernelFn = void (*)(Decode);

// shared: runs of fewer heads than warps.
KernelFn kernel_for(int groups, bool shared) {
    if (shared)
        return groups == 1 ? decode_kernel<1, true, Decode> : groups == 2 ? decode_kernel<2, true, Decode> : decode_kernel<4, true, Decode>;
    return groups == 1 ? decode_kernel<1, false, Decode> : groups == 2 ? decode_kernel<2, false, Decode> : decode_kernel<4, false, Decode>;
}

size_t smem_for(int groups, int num_seqs) {
    return groups == 1 ? Smem<1>::bytes(num_seqs) : groups == 2 ? Smem<2>::bytes(num_seqs) : Smem<4>::bytes(num_seqs);
}
// CTAs that fit at once on the current device; 0 on error. Kept per device, group
// count and shared memory (in steps of 64 sequences).
int resident_ctas(int groups, int num_seqs) {
    struct Entry {
        int dev, groups;
        size_t smem;
        int ctas;
    };
    static std::mutex mu;
    static std::vector<Entry> cache;
    int dev = 0, sms = 0, per_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const size_t smem = smem_for(groups, (num_seqs + 63) / 64 * 64);
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry& e : cache)
        if (e.dev == dev && e.groups == groups && e.smem == smem) return e.ctas;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    for (const bool shared : {false, true}) {  // (two CTAs an SM of either, as they are compiled for)
        const KernelFn fn = kernel_for(groups, shared);
        int here = 0;
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(smem_for(groups, PKV_ATTN_MAX_SEQS)));
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&here, fn, kThreads, smem);
        per_sm = shared ? std::min(per_sm, here) : here;
    }
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return 0;
    }
    cache.push_back({dev, groups, smem, std::min(sms * per_sm, kMaxCtas)});
    return cache.back().ctas;
}

// stop_tiles: none where negative, else the stopped kernel of two groups.
pkv_status decode(const void* q, const void* cache, const int32_t* block_tables, int max_blocks_per_seq,
                  const int32_t* context_lens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                  int block_tokens, int group_dims, float scale, int num_ctas, void* workspace, size_t workspace_bytes, void* out,
                  int stop_tiles, void* stream) {
    const int groups = groups_of(group_dims);
    if (!block_tokens_ok(block_tokens) || !groups) return PKV_EUNSUPPORTED;
    if (!q || !cache || !block_tables || !context_lens || !workspace || !out) return PKV_EINVAL;
    if (num_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1 || num_blocks < 1 || max_blocks_per_seq < 1 ||
        num_ctas < 0 || num_ctas > kMaxCtas || !std::isfinite(scale))
        return PKV_EINVAL;
    if (num_seqs > PKV_ATTN_MAX_SEQS || head_dim != kDim || num_q_heads % num_kv_heads != 0 ||
        num_q_heads / num_kv_heads > PKV_ATTN_MAX_GROUP)
        return PKV_EUNSUPPORTED;
    Decode p = {};
    p.heads = kWarps;
    while (num_kv_heads % p.heads) p.heads /= 2;
    p.runs = num_kv_heads / p.heads;
    p.group = num_q_heads / num_kv_heads;
    p.rows = p.heads * p.group;
    const int tile_tokens = kTok * (kWarps / p.heads);
    const long long cap = static_cast<long long>(max_blocks_per_seq) * block_tokens;
    const long long cost = static_cast<long long>(p.runs) * num_seqs * ((cap + tile_tokens - 1) / tile_tokens + kRunCost);
    if (static_cast<long long>(num_blocks) * num_kv_heads * block_tokens >= (1ll << 31) ||
        static_cast<long long>(num_seqs) * max_blocks_per_seq >= (1ll << 31) || cap >= (1ll << 31) - tile_tokens ||
        cost >= (1ll << 30))
        return PKV_ERANGE;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PKV_EINVAL;
    const int resident = resident_ctas(groups, num_seqs);
    if (resident < 1) return PKV_ECUDA;
    // No more CTAs than leave each the tiles that its consumers take at a time (one
    // sequence of 417 tokens: 9.4 us, 14.3 with a CTA a tile, whose joins cost more).
    int grid = num_ctas > 0 ? num_ctas : static_cast<int>(std::min<long long>(resident, (cost + kSubs - 1) / kSubs));
    const size_t each = partial_bytes(p.rows);
    if (workspace_bytes < attn::kWsFixed + each) return PKV_EINVAL;
    const size_t fit = (workspace_bytes - attn::kWsFixed) / each;
    if (static_cast<size_t>(grid) > fit) {
        if (num_ctas > 0) return PKV_EINVAL;
        grid = static_cast<int>(fit);
    }
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.cache = static_cast<const uint8_t*>(cache);
    p.tables = block_tables;
    p.context_lens = context_lens;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.num_seqs = num_seqs;
    p.width = max_blocks_per_seq;
    p.cap = static_cast<int>(cap);
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.num_blocks = num_blocks;
    p.bt_shift = block_tokens == 8 ? 3 : block_tokens == 16 ? 4 : block_tokens == 32 ? 5 : 6;
    // a copy's tokens lie next to one another: a slab's, or the block's where the
    // run has all its heads
    p.copy_tokens = p.runs == 1 ? std::min(block_tokens, tile_tokens) : std::min(block_tokens, 16);
    p.copies = tile_tokens / p.copy_tokens;
    p.scale_log2 = scale * 1.4426950408889634f;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.err = reinterpret_cast<uint32_t*>(ws);
    p.counters = reinterpret_cast<unsigned long long*>(ws + attn::kWsHeader);
    p.group_counters = p.counters + kMaxCtas;
    p.partials = reinterpret_cast<float*>(ws + attn::kWsFixed);
    // Launched early (programmatic stream serialization): the kernel sets itself up
    // while the one before it ends, then waits for it.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_for(groups, num_seqs);
    cfg.stream = as_stream(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaSuccess;
    const bool shared = p.heads < kWarps;
    if (stop_tiles < 0) {
        e = cudaLaunchKernelEx(&cfg, kernel_for(groups, shared), p);
    } else {
        StoppedDecode stopped;
        static_cast<Decode&>(stopped) = p;
        stopped.stop_tiles = stop_tiles;
        const auto fn = shared ? decode_kernel<2, true, StoppedDecode> : decode_kernel<2, false, StoppedDecode>;
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(cfg.dynamicSmemBytes));
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, fn, stopped);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return PKV_ECUDA;
    }
    return PKV_OK;
}

}  // namespace kv4
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_attn_int4_workspace_size(void) {
    const int ctas = kv4::resident_ctas(2, 1);
    return ctas < 1 ? 0 : attn::kWsFixed + static_cast<size_t>(ctas) * kv4::partial_bytes(kv4::kRows);
}

pkv_status pkv_attn_decode_int4(const void* q, const void* cache, const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* context_lens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                int num_blocks, int block_tokens, int group_dims, float scale, int num_ctas, void* workspace,
                                size_t workspace_bytes, void* out, void* stream) {
    return kv4::decode(q, cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim,
                       num_blocks, block_tokens, group_dims, scale, num_ctas, workspace, workspace_bytes, out, -1, stream);
}

pkv_status pkv_attn_decode_int4_wait_test(const void* q, const void* cache, const int32_t* block_tables,
                                          int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int num_q_heads,
                                          int num_kv_heads, int head_dim, int num_blocks, int block_tokens, int group_dims,
                                          float scale, int num_ctas, void* workspace, size_t workspace_bytes, void* out,
                                          int stop_tiles, void* stream) {
    if (stop_tiles < 0) return PKV_EINVAL;
    if (group_dims != 64) return PKV_EUNSUPPORTED;
    return kv4::decode(q, cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim,
                       num_blocks, block_tokens, group_dims, scale, num_ctas, workspace, workspace_bytes, out, stop_tiles,
                       stream);
}

}  // extern "C"
