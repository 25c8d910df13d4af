// mix_grad.cuh -- what the two backward paths of the gated mix share.
#pragma once

#include "common.cuh"

namespace duo {

// The gradient of one gate: its shares (mix_grad.cu: one per query head and 128
// rows of a sequence; tiled_attn.cu: one per 32 rows) added in a fixed order by
// one warp, in fp64.
__device__ __forceinline__ void sum_shares(const float* part, int n, float* out, int lane) {
    double sum = 0.0;
    for (int i = lane; i < n; i += 32) sum += part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) *out = (float)sum;
}

}  // namespace duo
