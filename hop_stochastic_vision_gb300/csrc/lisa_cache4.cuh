// lisa_cache4.cuh -- how a page of the 4-bit cache is laid out, shared by the
// kernels that fill, read and attend over it.
//
// A page of one key head is one block: the keys' codes, the values' codes, the
// keys' scales, the values' scales.  Codes are held plus 8, so 0x4300 | code is
// the bf16 number 136 + code and a pair of codes 4 bits wide becomes a pair of
// bf16 operands with one shift and one logic operation.  The codes stand in the
// order in which the lanes (g = lane / 4, q = lane % 4) of the warp-level product
// m16n8k16 want them as its left side:
//   keys    rows are tokens; lane (g, q) supplies elements 8 q .. 8 q + 7 of every
//           group for token g, one 32-bit word per group.  Within the word the pairs
//           (i, i + 4) are columns 2 q, 2 q + 1 of a product (the queries' elements
//           are taken in the same order).  Token t: word (q, group) at
//           t D / 2 + (q G + group) 4.
//   values  rows are elements; lane (g, q) supplies elements 4 g .. 4 g + 3 of every
//           group for tokens 2 q, 2 q + 1, one word per group: the even token's four
//           codes below the odd one's, so the same shift gives the pair.  Tokens 2 t,
//           2 t + 1: word (g, group) at t 32 G + (g G + group) 4.
// Both are read as consecutive words of a warp, without bank conflicts.  A byte
// belongs to one token, so tokens are stored without reading their neighbours.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "lisa_prompt.h"

namespace lisa {
namespace cache4 {

constexpr int kPage = LISA_CACHE4_PAGE;
constexpr int kGroup = 32;   // elements that share a scale

template <int D>
struct Block {
    static constexpr int G = D / kGroup;
    static constexpr int kCodes = kPage * D / 2;       // bytes of the keys' codes, and of the values'
    static constexpr int kScales = kPage * G * 2;
    static constexpr int off_v = kCodes, off_ks = 2 * kCodes, off_vs = 2 * kCodes + kScales;
    static constexpr int kBytes = 2 * kCodes + 2 * kScales;
    __host__ __device__ static constexpr int key_word(int t, int q, int group) { return t * (D / 2) + (q * G + group) * 4; }
    // the 16 bits of one token; the word of the pair is at the even token's
    __host__ __device__ static constexpr int value_half(int t, int g, int group) {
        return (t >> 1) * (32 * G) + (g * G + group) * 4 + (t & 1) * 2;
    }
};
constexpr size_t block_bytes(int d) { return d == 64 ? Block<64>::kBytes : Block<32>::kBytes; }

struct Cache {
    uint8_t *store;
    const int *table;
    long long table_stride;
    int pages, kv_heads, sequences, width;
};

// The page of token `position` of sequence `s`, or -1 where there is none.
__device__ __forceinline__ int page_of(const Cache &c, int s, int position) {
    if (s < 0 || s >= c.sequences || position < 0 || position >= c.width * kPage) return -1;
    const int page = c.table[s * c.table_stride + position / kPage];
    return page >= 0 && page < c.pages ? page : -1;
}

}  // namespace cache4
}  // namespace lisa
