// lisa_args.h -- argument checks that the C entry points of the attention
// operators share: alignment, strides, extents and overlaps.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "lisa_attention.h"

namespace lisa {
namespace attn {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Strides of a [B][heads][tokens][d] tensor: multiples of 16 bytes, tokens of a
// head apart, extents within 63 bits.  `out`: no two elements in one place.
inline bool good_strides(const lisa_strides *s, int B, int heads, int tokens, int d, size_t esz, bool out) {
    if (!s) return false;
    const long long q = 16 / (long long)esz, most = 1LL << 38;
    for (const long long x : {s->batch, s->head, s->token})
        if (x < 0 || x > most || x % q != 0) return false;
    if (tokens > 1 && s->token < d) return false;
    if (!out) return true;
    // the axes from the narrowest stride up: each steps over all of the ones below
    struct Axis { long long stride; int count; } ax[3] = {{s->batch, B}, {s->head, heads}, {s->token, tokens}};
    std::sort(ax, ax + 3, [](const Axis &a, const Axis &b) { return a.stride < b.stride; });
    long long inner = d;
    for (const Axis &a : ax) {
        if (a.count <= 1) continue;
        if (a.stride < inner) return false;
        inner += a.stride * (a.count - 1);
    }
    return true;
}

// Bytes from the first to behind the last element.
inline size_t extent(const lisa_strides *s, int B, int heads, int tokens, int d, size_t esz) {
    return ((size_t)s->batch * (size_t)(B - 1) + (size_t)s->head * (size_t)(heads - 1) +
            (size_t)s->token * (size_t)(tokens - 1) + (size_t)d) * esz;
}

struct Span {
    uintptr_t lo, hi;
    Span() : lo(0), hi(0) {}
    Span(const void *p, size_t bytes) : lo(reinterpret_cast<uintptr_t>(p)), hi(lo + bytes) {}
    bool meets(const Span &o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
};

inline lisa_status status_of(cudaError_t e) { return e == cudaSuccess ? LISA_OK : LISA_ERR_CUDA; }

}  // namespace attn
}  // namespace lisa
