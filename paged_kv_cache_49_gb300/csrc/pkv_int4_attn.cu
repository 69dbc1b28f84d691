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

KernelFn kernel_for(int groups) { return groups == 1 ? decode_kernel<1> : groups == 2 ? decode_kernel<2> : decode_kernel<4>; }

size_t smem_for(int groups, int num_seqs, int slots) {
    return groups == 1 ? Smem<1>::bytes(num_seqs, slots) : groups == 2 ? Smem<2>::bytes(num_seqs, slots) : Smem<4>::bytes(num_seqs, slots);
}

// A launch's shape: every CTA that fits at once, with room for the states of two
// pieces, or of one where that keeps two CTAs on an SM.
struct Shape {
    int dev = -1, groups = 0, num_seqs = 0;
    int ctas = 0, slots = 0;  // ctas 0 on error
    size_t smem = 0;
};

// Kept per device, group count and number of sequences.
Shape shape_for(int groups, int num_seqs) {
    static std::mutex mu;
    static std::vector<Shape> cache;
    Shape s;
    if (cudaGetDevice(&s.dev) != cudaSuccess) return s;
    s.groups = groups;
    s.num_seqs = (num_seqs + 63) / 64 * 64;
    std::lock_guard<std::mutex> lock(mu);
    for (const Shape& e : cache)
        if (e.dev == s.dev && e.groups == groups && e.num_seqs == s.num_seqs) return e;
    const KernelFn fn = kernel_for(groups);
    int sms = 0, best = 0;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem_for(groups, PKV_ATTN_MAX_SEQS, 2)));
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, s.dev);
    for (int slots = 2; slots >= 1 && e == cudaSuccess; --slots) {
        int per_sm = 0;
        const size_t smem = smem_for(groups, s.num_seqs, slots);
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, kThreads, smem);
        if (e == cudaSuccess && per_sm > best) {
            best = per_sm;
            s.slots = slots;
            s.smem = smem;
        }
    }
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return s;
    }
    s.ctas = std::min(sms * best, kMaxCtas);
    cache.push_back(s);
    return s;
}

}  // namespace kv4
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_attn_decode_int4(const void* q, const void* cache, const int32_t* block_tables,
                                           int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                                           int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                                           int block_tokens, int group_dims, float scale, int num_ctas, void* workspace,
                                           size_t workspace_bytes, void* out, void* stream) {
    const int groups = kv4::groups_of(group_dims);
    if (!kv4::block_tokens_ok(block_tokens) || !groups) return PKV_EUNSUPPORTED;
    if (!q || !cache || !block_tables || !context_lens || !workspace || !out) return PKV_EINVAL;
    if (num_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1 || num_blocks < 1 || max_blocks_per_seq < 1 ||
        num_ctas < 0 || num_ctas > kv4::kMaxCtas || !std::isfinite(scale))
        return PKV_EINVAL;
    if (num_seqs > PKV_ATTN_MAX_SEQS || head_dim != kv4::kDim || num_q_heads % num_kv_heads != 0 ||
        num_q_heads / num_kv_heads > PKV_ATTN_MAX_GROUP)
        return PKV_EUNSUPPORTED;
    const long long cap = static_cast<long long>(max_blocks_per_seq) * block_tokens;
    const long long cost = static_cast<long long>(num_kv_heads) * num_seqs * ((cap + kv4::kTile - 1) / kv4::kTile + kv4::kRunCost);
    if (static_cast<long long>(num_blocks) * num_kv_heads * block_tokens >= (1ll << 31) ||
        static_cast<long long>(num_seqs) * max_blocks_per_seq >= (1ll << 31) || cap >= (1ll << 31) || cost >= (1ll << 30))
        return PKV_ERANGE;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return PKV_EINVAL;
    const kv4::Shape shape = kv4::shape_for(groups, num_seqs);
    if (shape.ctas < 1) return PKV_ECUDA;
    // No more CTAs than the tables can hold work for: a run's cost each.
    int grid = num_ctas > 0 ? num_ctas
                            : static_cast<int>(std::max<long long>(1, std::min<long long>(shape.ctas, cost / (kv4::kRunCost + 1))));
    if (workspace_bytes < attn::workspace_bytes(1)) return PKV_EINVAL;
    const long long fit = static_cast<long long>((workspace_bytes - attn::kWsFixed) / attn::kWsPerCta);
    if (grid > fit) {
        if (num_ctas > 0) return PKV_EINVAL;
        grid = static_cast<int>(fit);
    }
    kv4::Decode p = {};
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
    p.group = num_q_heads / num_kv_heads;
    p.num_blocks = num_blocks;
    p.bt_shift = block_tokens == 8 ? 3 : block_tokens == 16 ? 4 : block_tokens == 32 ? 5 : 6;
    p.scale_log2 = scale * 1.4426950408889634f;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.err = reinterpret_cast<uint32_t*>(ws);
    p.counters = reinterpret_cast<int*>(ws + attn::kWsHeader);
    p.group_counters = p.counters + kv4::kMaxCtas;
    p.partials = reinterpret_cast<float*>(ws + attn::kWsFixed);
    p.slots = shape.slots;
    kv4::kernel_for(groups)<<<grid, kv4::kThreads, shape.smem, as_stream(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return PKV_ECUDA;
    }
    return PKV_OK;
}
