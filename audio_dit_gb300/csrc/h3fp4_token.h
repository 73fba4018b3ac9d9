// Internal declarations of a token's way through a block: the norms around a
// block, the linear of a few rows, the paged 4-bit cache and its attention.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "h3fp4_heads.h"
#include "h3fp4_internal.h"

namespace h3fp4 {

constexpr int kBlockNormMaxK = 32768;

struct BlockNormJob {
    const __nv_bfloat16* x;   // [M][K]
    const __nv_bfloat16* y;   // [M][K] or null
    __nv_bfloat16* x_out;     // [M][K] or null
    __nv_bfloat16* out;       // [M][K] or null
    const float* y_weight;    // [nseg][K] or null, as all vectors
    const float* gate;
    const float* weight;
    const float* shift;
    const float* scale;
    float x_scale, eps;
    bool post, layer;
    float* amax;              // device fp32 or null
    int64_t M;
    int K;
    Segments seg;
};

cudaError_t launch_block_norm(const BlockNormJob& job, cudaStream_t s);

}  // namespace h3fp4
