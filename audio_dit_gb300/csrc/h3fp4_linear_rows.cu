// The linear of a few rows over NVFP4 weights, activations as they are (bf16).
//
//     out[m][n] = bf16( R[m][n] + g[m][n] * (s_w * sum_k x[m][k] W[n][k] + b[n]) )
//
// or the SwiGLU of gate and up rows.  It has to read the weights, 9/16 byte an element.
// A warp takes a row of W (with SwiGLU its gate and up row), a lane a block of 16 at a time.
#include <cstdint>

#include <cuda_bf16.h>

#include "act_prologue.cuh"
#include "h3fp4_token.h"
#include "nvfp4_encode.cuh"
#include "ptx_sm103.cuh"

namespace h3fp4 {
namespace {

constexpr int kThreads = 128;
constexpr int kRowsAtOnce = 8;

struct RowsParams {
    LinearRowsJob j;
};

__device__ __forceinline__ float2 e2m1_pair(uint32_t byte)
{
    float lo, hi;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .b32 h2;\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {a, b, c, d}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 h2, a;\n\t"
        "mov.b32 {l, h}, h2;\n\t"
        "cvt.f32.f16 %0, l;\n\t"
        "cvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(byte));
    return make_float2(lo, hi);
}

__device__ __forceinline__ float silu_f32(float g)
{
    const float t = ex2_approx(-fabsf(g) * 1.4426950408889634f);
    const float r = rcp_approx(1.0f + t);
    return g * (g >= 0.0f ? r : t * r);
}

__global__ void __launch_bounds__(kThreads) linear_rows_kernel(const __grid_constant__ RowsParams p)
{
    const LinearRowsJob& j = p.j;
    const int lane = threadIdx.x & 31;
    const long long warp = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const long long outs = j.swiglu ? j.N / 2 : j.N;
    if (warp >= outs) return;
    griddep_wait();
    const float alpha = *j.w_gscale;
    for (int m0 = 0; m0 < j.M; m0 += kRowsAtOnce) {
        float res[2][kRowsAtOnce];
        for (int part = 0; part < (j.swiglu ? 2 : 1); ++part) {
            const long long n = j.swiglu ? warp / 128 * 256 + warp % 128 + 128 * part : warp;
            float acc[kRowsAtOnce] = {};
            for (int b = lane; b < j.K / 16; b += 32) {
                const uint2 w = *reinterpret_cast<const uint2*>(j.w_codes + n * (j.K / 2) + 8 * b);
                const long long off = ((n >> 7) * (j.K / 64) + (b >> 2)) * 512 + (n & 31) * 16 + ((n & 127) >> 5) * 4 + (b & 3);
                const float S = e4m3_value(j.w_sf[off]);
                float f[16];
                for (int k = 0; k < 8; ++k) {
                    const float2 q = e2m1_pair(((k < 4 ? w.x : w.y) >> (8 * (k & 3))) & 0xFFu);
                    f[2 * k] = q.x * S;
                    f[2 * k + 1] = q.y * S;
                }
                for (int i = 0; i < kRowsAtOnce; ++i) {
                    if (m0 + i >= j.M) break;
                    const __nv_bfloat16* x = j.x + (m0 + i) * j.K + 16 * b;
                    for (int k = 0; k < 16; ++k) acc[i] = fmaf(__bfloat162float(x[k]), f[k], acc[i]);
                }
            }
            for (int i = 0; i < kRowsAtOnce; ++i) {
                for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
                res[part][i] = fmaf(alpha, acc[i], j.bias ? __bfloat162float(j.bias[n]) : 0.0f);
            }
        }
        for (int i = 0; i < kRowsAtOnce && m0 + i < j.M; ++i) {
            if (lane != 0) continue;
            const long long m = m0 + i;
            float v = res[0][i];
            if (j.swiglu)
                v = silu_f32(__bfloat162float(__float2bfloat16_rn(v))) * __bfloat162float(__float2bfloat16_rn(res[1][i]));
            if (j.gate) v = fmaf(j.gate[m * j.gate_stride + warp], v, __bfloat162float(j.resid[m * j.N + warp]));
            j.out[m * outs + warp] = __float2bfloat16_rn(v);
        }
    }
}

}  // namespace

size_t linear_rows_workspace_bytes(int64_t, int64_t, int64_t) { return 256; }

cudaError_t launch_linear_rows(const LinearRowsJob& job, cudaStream_t s)
{
    RowsParams p{job};
    const long long outs = job.swiglu ? job.N / 2 : job.N;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((outs + 3) / 4));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_rows_kernel, p);
}

}  // namespace h3fp4
