// The layout of a cache held in 4 bits, and the conversions between its units
// and values, shared by the kernels that write and read it.
//
// Per row of 128 values (the key or the value of one token and KV head), in
// groups of G = 32, 64 or 128 values, all in fp32 with one rounding per step:
//   lo, hi = the group's least and greatest value, held to +-65504
//   m = fp16(lo), s = fp16((hi - lo) / 15)
//   c = rint((x - m) / s), held to 0 .. 15 (0 where s is 0)
// and the row stands for s c + m. s and m are fp16 because they feed the fp16
// matrix products of the attention as they are; bf16 keys and values convert to
// m without loss from 2^-14 on. A NaN in a group makes its s and m NaN.
//
// A block is slabs of 16 tokens (of 8 where it has but 8), one after the other; a
// slab has its KV heads' rows one after the other, so that the rows of a slab of
// several heads are one contiguous copy; and a head's part of a slab is one or
// two units of 8 tokens. A unit (1,024 + 64 * 128 / G bytes) holds, in this
// order,
//   512 bytes  key codes: token t at 64 t; its 16 words in the order 4 c + w,
//              word (w, c) the dims 32 w + 8 c .. + 7, lowest dim lowest
//   512 bytes  value codes: 16-bit pieces of 4 dims at
//              ((r * 4 + t / 2) * 4 + w) * 2 + t % 2 for dims 32 w + 4 r .. + 3
//   32 * 128/G bytes  keys' (s, m): token t, group g at 4 (128/G t + g)
//   16 * 128/G bytes  values' s: group g, token t at 2 (8 g + t)
//   16 * 128/G bytes  values' m, likewise
// which is the order in which the lanes of a warp hold the operands of
// mma.m16n8k16: lane 4 r + c loads 16 consecutive bytes of key codes (token r,
// a quarter of its dims) and 16 of value codes (tokens 2 c and 2 c + 1, 16
// dims), both without bank conflicts.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstddef>
#include <cstdint>

#include "../../include/pkv.h"

namespace pkv {
namespace kv4 {

constexpr int kDim = 128;
constexpr int kUnit = 8;  // tokens
constexpr int kCodeBytes = kUnit * kDim / 2;  // of the keys, and of the values, of a unit

template <int kGroups>  // groups of a row: 1, 2 or 4
struct Unit {
    static constexpr int kGroupDims = kDim / kGroups;
    static constexpr int kKeys = 0;
    static constexpr int kValues = kCodeBytes;
    static constexpr int kKeyParams = 2 * kCodeBytes;
    static constexpr int kValueScales = kKeyParams + kUnit * kGroups * 4;
    static constexpr int kValueMins = kValueScales + kUnit * kGroups * 2;
    static constexpr int kBytes = kValueMins + kUnit * kGroups * 2;
};

// Groups of a row for a group size, 0 for one that is not offered.
inline int groups_of(int group_dims) { return group_dims == 32 ? 4 : group_dims == 64 ? 2 : group_dims == 128 ? 1 : 0; }

inline bool block_tokens_ok(int bt) { return bt == 8 || bt == 16 || bt == 32 || bt == 64; }

// The unit that holds a slot's token (slot = block * block tokens + position).
__host__ __device__ __forceinline__ long long unit_of(long long slot, int head, int hkv, bool blocks_of_8) {
    return blocks_of_8 ? (slot >> 3) * hkv + head : ((slot >> 4) * hkv + head) * 2 + ((slot >> 3) & 1);
}

// Byte of token t's key word (w, c), and of its value piece (w, r), in a unit.
__device__ __forceinline__ int key_word(int t, int w, int c) { return t * 64 + (4 * c + w) * 4; }
__device__ __forceinline__ int value_piece(int t, int w, int r) {
    return kCodeBytes + (((r * 4 + (t >> 1)) * 4 + w) * 2 + (t & 1)) * 2;
}

}  // namespace kv4
}  // namespace pkv
