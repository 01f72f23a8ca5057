// lisa_packed_tc.cuh -- what the tensor-core kernels of the packed prompts share:
// the walk over a worker's items, tiles of a sequence, the join of parts.
#pragma once

#include <algorithm>

#include "lisa_attn_tc.cuh"
#include "lisa_packed.h"

namespace lisa {
namespace packed {
namespace {

using namespace lisa::attn;
using namespace lisa::sm100;
using lisa::packed::Problem;

// One (item, head) pair.
struct Work {
    int h, row0, len, first, t0, t1, part, steps;
};
// A worker's pairs begin .. end - 1 in the order list.
struct Walk {
    const Item *items;
    const int *order;
    int begin, end;
    FastDiv div_heads;
    __device__ __forceinline__ Work at(int k) const {
        Work w;
        int pair = order[k];
        const int4 *it = reinterpret_cast<const int4 *>(items + split_off(pair));
        const int4 a = it[0], b = it[1];
        w.h = pair;
        w.row0 = a.x;
        w.len = a.y;
        w.first = a.z;
        w.t0 = a.w;
        w.t1 = b.x;
        w.part = b.y;
        w.steps = b.z;
        return w;
    }
    // pair / heads, and pair becomes pair % heads
    __device__ __forceinline__ int split_off(int &pair) const { return split(pair, div_heads); }
};
static_assert(sizeof(Item) == 32, "an item is two 16-byte loads");

__device__ __forceinline__ Walk walk_of(const Lists &l, const FastDiv &div_heads) {
    return Walk{l.items, l.order, l.starts[blockIdx.x], l.starts[blockIdx.x + 1], div_heads};
}

// Valid rows of the tile of 128 from row `at` of a sequence, and the columns its products cover.
__device__ __forceinline__ int tile_rows(int len, int at) { return min(kRows, len - at); }
__device__ __forceinline__ int tile_cols(int rows) { return (rows + 15) & ~15; }

// 4-D map of a packed tensor [heads][tokens][d] (lisa_attn_tc.cuh's, of a batch of one).
inline bool make_packed_map(CUtensorMap *m, MapUse *u, const Tensor &t, int heads, int tokens, int d) {
    return make_map(m, u, Tensor{t.p, 0, t.sh, t.st}, 1, heads, tokens, d);
}

// Workers with anything to do: the first ones.
inline unsigned workers(const Lists &l, int heads) {
    return (unsigned)std::min<long long>(kSms, (long long)l.n_items * heads);
}

}  // namespace
}  // namespace packed
}  // namespace lisa
