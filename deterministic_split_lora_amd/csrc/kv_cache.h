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

__device__ __forceinline__ KvSequence kv_sequence(const KvCacheView& c, int64_t b, int64_t T)
{
    KvSequence s;
    s.first = c.cu_tokens[b];
    const int64_t end = c.cu_tokens[b + 1];
    s.len = c.seq_lens[b];
    s.n = s.first >= 0 && end > s.first && end <= T ? end - s.first : 0;
    return s;
}

// Sequences have slots in a row: those of j begin at at(j, cu_tokens[j]), which does
// not fall with j.  The one that slot w (the same in the whole wave, every lane of
// which is active) belongs to; n_seqs where w lies behind them.
// Every lane of the wave looks at entries of its own: one round of loads for 64.
template <class F>
__device__ __forceinline__ int64_t kv_find(const KvCacheView& c, int64_t w, F at)
{
    int64_t b = 0;
    const int lane = threadIdx.x & 63;
    for (int64_t base = 1; base <= c.n_seqs; base += 64) {
        const int64_t j = base + lane;
        b += __popcll(__ballot(j <= c.n_seqs && at(j, (int64_t)c.cu_tokens[min(j, c.n_seqs)]) <= w));
    }
    return b;
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
