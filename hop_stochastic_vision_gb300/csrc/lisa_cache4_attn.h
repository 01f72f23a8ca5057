// lisa_cache4_attn.h -- the attention over the 4-bit cache as its launcher gets it.
#pragma once

#include <cuda_runtime.h>

#include "lisa_attn.h"
#include "lisa_cache4.cuh"

namespace lisa {
namespace cache4 {

struct AttnProblem {
    Cache c;
    attn::Tensor Q, O;
    float *lse;
    const int *lens;
    int B, heads, group, n;
    float scale;
};

cudaError_t launch_attention(const AttnProblem &p, int d, cudaStream_t s);

}  // namespace cache4
}  // namespace lisa
