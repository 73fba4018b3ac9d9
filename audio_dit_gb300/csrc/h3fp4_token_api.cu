// C ABI of a token's way through a block (h3fp4_block_norm): argument validation
// and job set-up.  Nothing here allocates device memory or synchronises.
#include <cmath>
#include <cstdint>

#include "h3fp4_token.h"

namespace h3fp4 {
namespace {

bool overlap(const void* a, const void* b, int64_t bytes)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + (uint64_t)bytes && y < x + (uint64_t)bytes;
}

}  // namespace
}  // namespace h3fp4

using namespace h3fp4;

extern "C" {

h3fp4_status h3fp4_block_norm(const void* x, const void* y, int64_t M, int64_t K, const float* y_weight,
                              const float* gate, float x_scale, const float* weight, const float* shift,
                              const float* scale, const int64_t* seg_off, int nseg, float eps, void* x_out, void* out,
                              float* out_amax, int flags, cudaStream_t stream)
{
    if (M < 0 || M > INT32_MAX || K < 8 || K > kBlockNormMaxK || K % 8 != 0) return H3FP4_ERR_SHAPE;
    if (flags & ~(H3FP4_NORM_POST | H3FP4_NORM_LAYER)) return H3FP4_ERR_INVALID;
    if (!(eps >= 0.0f) || std::isinf(eps) || !std::isfinite(x_scale)) return H3FP4_ERR_INVALID;
    if (M > 0) {
        if (!x || (!out && !x_out)) return H3FP4_ERR_INVALID;
        if (!out && (weight || shift || scale || out_amax || (flags & H3FP4_NORM_LAYER))) return H3FP4_ERR_INVALID;
        if (!y && (x_out || y_weight || gate || (flags & H3FP4_NORM_POST))) return H3FP4_ERR_INVALID;
        if (y_weight && !(flags & H3FP4_NORM_POST)) return H3FP4_ERR_INVALID;
    }
    for (const void* p : {x, y, static_cast<const void*>(y_weight), static_cast<const void*>(gate),
                          static_cast<const void*>(weight), static_cast<const void*>(shift),
                          static_cast<const void*>(scale), static_cast<const void*>(x_out),
                          static_cast<const void*>(out)})
        if (!aligned16(p)) return H3FP4_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(out_amax) & 3u) return H3FP4_ERR_ALIGN;
    // an output is an input itself or apart from it, and apart from the other output
    const int64_t bytes = M * K * 2;
    if (overlap(x_out, out, bytes)) return H3FP4_ERR_INVALID;
    for (const void* o : {static_cast<const void*>(x_out), static_cast<const void*>(out)})
        for (const void* i : {x, y})
            if (o != i && overlap(o, i, bytes)) return H3FP4_ERR_INVALID;
    BlockNormJob job{};
    h3fp4_status st = make_segments(seg_off, seg_off == nullptr && nseg <= 0 ? 1 : nseg, M, &job.seg);
    if (st != H3FP4_OK) return st;
    if ((st = check_device()) != H3FP4_OK) return st;
    job.x = static_cast<const __nv_bfloat16*>(x);
    job.y = static_cast<const __nv_bfloat16*>(y);
    job.x_out = static_cast<__nv_bfloat16*>(x_out);
    job.out = static_cast<__nv_bfloat16*>(out);
    job.y_weight = y_weight;
    job.gate = gate;
    job.weight = weight;
    job.shift = shift;
    job.scale = scale;
    job.x_scale = x_scale;
    job.eps = eps;
    job.post = (flags & H3FP4_NORM_POST) != 0;
    job.layer = (flags & H3FP4_NORM_LAYER) != 0;
    job.amax = out_amax;
    job.M = M;
    job.K = (int)K;
    return launch_block_norm(job, stream) == cudaSuccess ? H3FP4_OK : H3FP4_ERR_CUDA;
}

}  // extern "C"
