// The norms around a block with its gate and residual, one pass over the rows.
//
//     y' = y * rsqrt(mean(y^2) + eps) * y_weight[seg]        (post; else y' = y)
//     r  = x_scale * x + gate[seg] * y'                       x_out = bf16(r)
//     z  = (r - mean(r)) * rsqrt(var(r) + eps)                (layer; else r * rsqrt(mean(r^2) + eps))
//     out = bf16(z * weight[seg] * (1 + scale[seg]) + shift[seg]),   amax = max |out|
//
// Memory-bound: 8 bytes move per element (x, y, x_out, out), 4 without y.  A row
// is held in registers by the threads of its group (8 elements of 16 bytes per
// vector, kVec vectors a thread), so each byte moves once; all sums are fp32 over
// fp32 values, the variance of the layer norm about the mean itself (a second
// sum over the registers), and each output is rounded once.  The fp32 vectors of
// a segment (up to five of K) are read for every row from L1, which the blocks of
// an SM share.
#include <cstdint>

#include <cuda_bf16.h>

#include "act_prologue.cuh"
#include "h3fp4_token.h"
#include "ptx_sm103.cuh"

namespace h3fp4 {
namespace {

struct BlockNormParams {
    const __nv_bfloat16* x;
    const __nv_bfloat16* y;
    __nv_bfloat16* x_out;
    __nv_bfloat16* out;
    const float* y_weight;
    const float* gate;
    const float* weight;
    const float* shift;
    const float* scale;
    float x_scale, eps, inv_k;
    int post, layer;
    unsigned int* amax;
    long long M;
    int K;
    Segments seg;
};

__device__ __forceinline__ void load_f8(const float* p, float (&f)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

__device__ __forceinline__ void unpack_bf8(const uint4& v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack_bf8(const float (&f)[8])
{
    return make_uint4(cvt_bf16x2(f2(f[0], f[1])), cvt_bf16x2(f2(f[2], f[3])), cvt_bf16x2(f2(f[4], f[5])),
                      cvt_bf16x2(f2(f[6], f[7])));
}

// Sum over the threads of a row.  Rows of several warps meet in shared memory;
// consecutive sums use different halves of `part`, so one barrier each is enough.
template <int kRow>
__device__ __forceinline__ float row_sum(float v, float (&part)[2][32], uint32_t& turn)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (kRow > 32) {
        constexpr int kWarps = kRow / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) part[turn][warp] = v;
        __syncthreads();
        v = lane < kWarps ? part[turn][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        turn ^= 1u;
    }
    return v;
}

// kRow threads per row (32: four rows to a block of 128 threads, which never wait
// for one another; else one row to a block), kVec vectors of eight elements each.
template <int kRow, int kVec>
__global__ void __launch_bounds__(kRow < 128 ? 128 : kRow) block_norm_kernel(const __grid_constant__ BlockNormParams p)
{
    constexpr int kRows = kRow < 128 ? 128 / kRow : 1;  // rows of a block
    __shared__ float part[2][32];
    const int t = threadIdx.x % kRow;
    const int nv = p.K >> 3;
    uint32_t turn = 0, top = 0;
    griddep_wait();
    for (long long r = (long long)blockIdx.x * kRows + threadIdx.x / kRow; r < p.M; r += (long long)gridDim.x * kRows) {
        const long long row = r * p.K;
        uint4 vx[kVec], vy[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = t + i * kRow;
            vx[i] = vy[i] = make_uint4(0, 0, 0, 0);
            if (v < nv) {
                vx[i] = *reinterpret_cast<const uint4*>(p.x + row + 8 * v);
                if (p.y) vy[i] = *reinterpret_cast<const uint4*>(p.y + row + 8 * v);
            }
        }
        const long long at = (long long)segment_of(p.seg, r) * p.K;
        float f[kVec][8];
#pragma unroll
        for (int i = 0; i < kVec; ++i) unpack_bf8(vx[i], f[i]);
        if (p.y) {
            float rs = 1.0f;
            if (p.post) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    float y[8];
                    unpack_bf8(vy[i], y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = fmaf(y[j], y[j], sum);
                }
                rs = rsqrtf(fmaf(row_sum<kRow>(sum, part, turn), p.inv_k, p.eps));
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = t + i * kRow;
                if (v >= nv) continue;
                float y[8], w[8];
                unpack_bf8(vy[i], y);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] *= rs;
                if (p.y_weight) {
                    load_f8(p.y_weight + at + 8 * v, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] *= w[j];
                }
                if (p.gate) {
                    load_f8(p.gate + at + 8 * v, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] *= w[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] = fmaf(p.x_scale, f[i][j], y[j]);
                if (p.x_out) *reinterpret_cast<uint4*>(p.x_out + row + 8 * v) = pack_bf8(f[i]);
            }
        }
        if (!p.out) continue;
        float mean = 0.0f;
        if (p.layer) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += f[i][j];  // (places past the row hold zeros)
            mean = row_sum<kRow>(sum, part, turn) * p.inv_k;
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            if (t + i * kRow >= nv) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[i][j] -= mean;
                sum = fmaf(f[i][j], f[i][j], sum);
            }
        }
        const float rs = rsqrtf(fmaf(row_sum<kRow>(sum, part, turn), p.inv_k, p.eps));
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = t + i * kRow;
            if (v >= nv) continue;
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] *= rs;
            if (p.weight) {
                load_f8(p.weight + at + 8 * v, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] *= w[j];
            }
            if (p.scale) {
                load_f8(p.scale + at + 8 * v, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] *= 1.0f + w[j];
            }
            if (p.shift) {
                load_f8(p.shift + at + 8 * v, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] += w[j];
            }
            const uint4 o = pack_bf8(f[i]);
            *reinterpret_cast<uint4*>(p.out + row + 8 * v) = o;
            if (p.amax) {
                // magnitudes of bf16 values in the order of their bits (a NaN is above all)
                const uint32_t words[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    top = max(top, max((words[j] << 16) & 0x7FFF0000u, words[j] & 0x7FFF0000u));
            }
        }
    }
    if (p.amax) {
        top = __reduce_max_sync(0xffffffffu, top);
        // the largest of all, in whatever order they come
        if ((threadIdx.x & 31) == 0 && top != 0) atomicMax(p.amax, top);
    }
}

template <int kRow, int kVec>
cudaError_t launch(const BlockNormParams& p, cudaStream_t s)
{
    constexpr int kThreads = kRow < 128 ? 128 : kRow, kRows = kThreads / kRow;
    const long long blocks = (p.M + kRows - 1) / kRows;
    // as many blocks as an SM can hold at 64 registers a thread, which then take the next rows
    const long long most = (long long)sm_count_current_device() * (1024 / kThreads);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, block_norm_kernel<kRow, kVec>, p);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormJob& job, cudaStream_t s)
{
    if (job.amax) {
        const cudaError_t e = cudaMemsetAsync(job.amax, 0, sizeof(float), s);
        if (e != cudaSuccess) return e;
    }
    if (job.M == 0) return cudaSuccess;
    BlockNormParams p{};
    p.x = job.x;
    p.y = job.y;
    p.x_out = job.x_out;
    p.out = job.out;
    p.y_weight = job.y_weight;
    p.gate = job.gate;
    p.weight = job.weight;
    p.shift = job.shift;
    p.scale = job.scale;
    p.x_scale = job.x_scale;
    p.eps = job.eps;
    p.inv_k = 1.0f / (float)job.K;
    p.post = job.post;
    p.layer = job.layer;
    p.amax = reinterpret_cast<unsigned int*>(job.amax);
    p.M = job.M;
    p.K = job.K;
    p.seg = job.seg;
    const int nv = job.K / 8;
    if (nv <= 32) return launch<32, 1>(p, s);
    if (nv <= 64) return launch<32, 2>(p, s);
    if (nv <= 128) return launch<32, 4>(p, s);
    if (nv <= 256) return launch<128, 2>(p, s);
    if (nv <= 384) return launch<128, 3>(p, s);
    if (nv <= 512) return launch<128, 4>(p, s);
    if (nv <= 768) return launch<256, 3>(p, s);
    if (nv <= 1024) return launch<256, 4>(p, s);
    if (nv <= 2048) return launch<1024, 2>(p, s);
    return launch<1024, 4>(p, s);
}

}  // namespace h3fp4
