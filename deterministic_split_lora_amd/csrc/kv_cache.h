// The paged key / value cache in 8 bits, as its kernels see it.
//
// A page holds page_size tokens (whole blocks of kKvBlock) of every head.  A block
// of kKvBlock tokens of a head has one E8M0 scale for its keys and one for its values.
//   k  [page][head][token][D]            E4M3 codes
//   v  [page][head][block][D][kKvBlock]  E4M3 codes
// A lane's 16-byte load of k is 16 consecutive d of a token, one of v the block's
// tokens of one d: either way the dimension that the matrix cores reduce lies
// within the load, so both go from memory to an operand without passing through LDS.
#pragma once

#include "device.h"
#include "step_kernels.h"

namespace lora {

__device__ __forceinline__ float pow2_of_scale(uint32_t byte)
{
    return __builtin_bit_cast(float, byte << 23);
}

// The run of new tokens of a sequence, from its entries in the batch's tables;
// `n` 0 where they make no sense.
struct KvSequence {
    int64_t first;                           // row of the first new token
    int64_t n;                               // new tokens
    int64_t len;                             // tokens with them
};

__device__ __forceinline__ KvSequence kv_sequence(int64_t first, int64_t end, int64_t len, int64_t T)
{
    return {first, first >= 0 && end > first && end <= T ? end - first : 0, len};
}

__device__ __forceinline__ KvSequence kv_sequence(const KvCacheView& c, int64_t b, int64_t T)
{
    return kv_sequence(c.cu_tokens[b], c.cu_tokens[b + 1], c.seq_lens[b], T);
}

// Sequences have slots in a row, `total` in all: those of j begin at at(j, cu_tokens[j]),
// which does not fall with j.  The one that slot w (the same in the whole wave, every
// lane of which is active) belongs to, and its entries; -1 where w lies behind them all.
// A lane looks at a sequence and reads all that is needed of it, so where the sequences
// have about as many slots each, one round of loads finds it; else the range is cut to a
// 64th each round.
struct KvFound {
    int64_t b;
    KvSequence s;
};

template <class F>
__device__ __forceinline__ KvFound kv_find(const KvCacheView& c, int64_t T, int64_t w, int64_t total, F at)
{
    KvFound f{-1, {0, 0, 0}};
    const int lane = threadIdx.x & 63, n = (int)c.n_seqs;
    int base = min(max((int)((float)w / (float)total * (float)n) - 32, 0), n - 1);
#pragma unroll 1
    for (int from = 0, size = n;;) {
        const int j = base + lane, i = min(j, n - 1);
        const int32_t first = c.cu_tokens[i], end = c.cu_tokens[i + 1], len = c.seq_lens[i];
        const uint64_t hit =
            __ballot(j < n && at((int64_t)j, (int64_t)first) <= w && at((int64_t)j + 1, (int64_t)end) > w);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            f.b = base + l;
            f.s = kv_sequence(__builtin_amdgcn_readlane(first, l), __builtin_amdgcn_readlane(end, l),
                              __builtin_amdgcn_readlane(len, l), T);
            return f;
        }
        if (size <= 64 && base <= from && base + 64 >= from + size)
            return f;                        // looked at every one that is left
        // the first of 64 parts of the range whose last sequence ends behind w
        while (size > 64) {
            const int part = (size + 63) / 64, k = min(from + (lane + 1) * part, from + size);
            const uint64_t behind = __ballot(at((int64_t)k, (int64_t)c.cu_tokens[k]) > w);
            if (behind == 0)
                return f;
            from += __builtin_ctzll(behind) * part;
            size = min(part, n - from);
            if (size <= 0)
                return f;
        }
        base = from;
    }
}

// The page that holds a sequence's tokens [p, p + kKvBlock), or -1 if there is none;
// p is not negative.  The table is read through the constant address space: a scalar
// load where p is the same in the whole wave.
__device__ __forceinline__ int32_t kv_page(const KvCacheView& c, int64_t b, int64_t p)
{
    typedef __attribute__((address_space(4))) const int32_t constant_i32;
    const int64_t i = p >> c.page_shift;
    const int32_t page = *(constant_i32*)(c.page_table + b * c.ld_table + min(i, c.max_pages - 1));
    return i < c.max_pages && page >= 0 && page < c.n_pages ? page : -1;
}

}  // namespace lora
