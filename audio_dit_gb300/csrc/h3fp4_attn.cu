// Attention of packed query rows to an encoder's states and to a shared context.
//
//     out[r][h] = sum_j p_j v_j / l,  p_j = exp(scale q_r.k_j - m),  l = sum_j p_j
// over the context's keys and the keys of r's own segment, in one pass with a
// running maximum m: when m grows, the sums so far are scaled by exp(m_old - m).
//
// A CTA takes 64 query rows of one head and walks its keys 32 at a time
// through shared memory; four threads share a row (eight scores each, then a
// quarter of the output's columns each).  All arithmetic is fp32.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>

#include "h3fp4_heads.h"
#include "ptx_sm103.cuh"

namespace h3fp4 {
namespace {

constexpr int kRows = 64, kKeys = 32, kThreads = 256;

struct AttnParams {
    HeadsIn q, k, v, kc, vc;
    __nv_bfloat16* out;
    long long out_row, out_head;
    float* lse;
    int C, Hq, group, D, nseg;
    const uint8_t* key_mask;
    const uint8_t* ctx_mask;
    float scale_log2;
    int q_off[H3FP4_ATTN_MAX_SEGMENTS + 1];
    int kv_off[H3FP4_ATTN_MAX_SEGMENTS + 1];
    int tiles[H3FP4_ATTN_MAX_SEGMENTS + 1];  // row tiles before each segment
};

__global__ void __launch_bounds__(kThreads) attn_kernel(const __grid_constant__ AttnParams p)
{
    griddep_wait();
    __shared__ __nv_bfloat16 sq[kRows][kAttnMaxD + 2];
    __shared__ __nv_bfloat16 sk[kKeys][kAttnMaxD + 2];
    __shared__ __nv_bfloat16 sv[kKeys][kAttnMaxD];
    __shared__ uint8_t keep[kKeys];
    __shared__ float sp[kRows][kKeys + 1];
    const int tid = threadIdx.x, row = tid >> 2, c = tid & 3;
    const int h = blockIdx.y, hk = h / p.group;
    int seg = 0;
    while (seg + 1 < p.nseg && (int)blockIdx.x >= p.tiles[seg + 1]) ++seg;
    const int r0 = p.q_off[seg] + ((int)blockIdx.x - p.tiles[seg]) * kRows;
    const int rows = min(kRows, p.q_off[seg + 1] - r0);
    for (int i = tid; i < kRows * p.D; i += kThreads) {
        const int r = i / p.D, d = i - r * p.D;
        sq[r][d] = r < rows ? p.q.p[(r0 + r) * p.q.row + h * p.q.head + d] : __float2bfloat16(0.0f);
    }
    float m = -INFINITY, l = 0.0f, acc[kAttnMaxD / 4];
#pragma unroll
    for (int i = 0; i < kAttnMaxD / 4; ++i) acc[i] = 0.0f;

    for (int part = 0; part < 2; ++part) {  // the context, then the segment's own keys
        const HeadsIn& K = part ? p.k : p.kc;
        const HeadsIn& V = part ? p.v : p.vc;
        const uint8_t* mask = part ? p.key_mask : p.ctx_mask;
        const int k0 = part ? p.kv_off[seg] : 0, k1 = part ? p.kv_off[seg + 1] : p.C;
        for (int t = k0; t < k1; t += kKeys) {
            __syncthreads();
            if (tid < kKeys) keep[tid] = t + tid < k1 && (!mask || mask[t + tid]);
            __syncthreads();
            for (int i = tid; i < kKeys * p.D; i += kThreads) {
                const int j = i / p.D, d = i - j * p.D;
                const long long at = (long long)(t + j);
                sk[j][d] = keep[j] ? K.p[at * K.row + hk * K.head + d] : __float2bfloat16(0.0f);
                sv[j][d] = keep[j] ? V.p[at * V.row + hk * V.head + d] : __float2bfloat16(0.0f);
            }
            __syncthreads();
            float z[kKeys / 4], top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kKeys / 4; ++i) z[i] = 0.0f;
            for (int d = 0; d < p.D; ++d) {
                const float x = __bfloat162float(sq[row][d]);
#pragma unroll
                for (int i = 0; i < kKeys / 4; ++i) z[i] = fmaf(x, __bfloat162float(sk[c + 4 * i][d]), z[i]);
            }
#pragma unroll
            for (int i = 0; i < kKeys / 4; ++i) {
                if (!keep[c + 4 * i]) z[i] = -INFINITY;
                top = fmaxf(top, z[i]);
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float m_new = fmaxf(m, top);
            const float base = m_new == -INFINITY ? 0.0f : m_new * p.scale_log2;
            const float f = exp2f(fmaf(m, p.scale_log2, -base));
            l *= f;
#pragma unroll
            for (int i = 0; i < kKeys / 4; ++i) {
                const float e = exp2f(fmaf(z[i], p.scale_log2, -base));
                l += e;
                sp[row][c + 4 * i] = e;
            }
#pragma unroll
            for (int i = 0; i < kAttnMaxD / 4; ++i) acc[i] *= f;
            m = m_new;
            __syncwarp();
            for (int j = 0; j < kKeys; ++j) {
                const float e = sp[row][j];
#pragma unroll
                for (int i = 0; i < kAttnMaxD / 4; ++i)
                    if (c + 4 * i < p.D) acc[i] = fmaf(e, __bfloat162float(sv[j][c + 4 * i]), acc[i]);
            }
        }
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (row >= rows) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row without a key: zeros
    __nv_bfloat16* o = p.out + (long long)(r0 + row) * p.out_row + h * p.out_head;
#pragma unroll
    for (int i = 0; i < kAttnMaxD / 4; ++i)
        if (c + 4 * i < p.D) o[c + 4 * i] = __float2bfloat16_rn(acc[i] * inv);
    if (p.lse && c == 0)
        p.lse[(long long)(r0 + row) * p.Hq + h] =
            l == 0.0f ? -INFINITY : (m * p.scale_log2 + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

size_t attn_workspace_bytes(const AttnJob& job)
{
    (void)job;
    return 256;  // the status word
}

cudaError_t launch_attn(const AttnJob& job, cudaStream_t s)
{
    AttnParams p{};
    p.q = job.q;
    p.k = job.k;
    p.v = job.v;
    p.kc = job.kc;
    p.vc = job.vc;
    p.out = job.out;
    p.out_row = job.out_row;
    p.out_head = job.out_head;
    p.lse = job.lse;
    p.C = (int)job.C;
    p.Hq = job.Hq;
    p.group = job.Hq / job.Hkv;
    p.D = job.D;
    p.nseg = job.nseg;
    p.key_mask = job.key_mask;
    p.ctx_mask = job.ctx_mask;
    p.scale_log2 = job.scale * 1.4426950408889634f;
    for (int i = 0; i <= job.nseg; ++i) {
        p.q_off[i] = (int)job.q_off[i];
        p.kv_off[i] = (int)job.kv_off[i];
        if (i < job.nseg) p.tiles[i + 1] = p.tiles[i] + (int)((job.q_off[i + 1] - job.q_off[i] + kRows - 1) / kRows);
    }
    attn_kernel<<<dim3((unsigned)p.tiles[job.nseg], (unsigned)job.Hq), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace h3fp4
