// Per-head RMS norm with rotation of the queries and keys, one pass.
//
//     y = x * rsqrt(mean_d(x^2) + eps) * w[seg(row)]
//     (a, b) -> (a cos - b sin, b cos + a sin)  over rot / 2 pairs of elements
//     out = bf16(y)
//
// Memory-bound: 4 bytes move per element, the angle table (4 rot bytes per
// row) is shared by all heads of a row.  Sums and the rotation are fp32; the
// only rounding is the one to bf16 at the end.
//
// A head of n = D/8 sixteen-byte chunks is held by a group of lanes, two
// chunks per lane.  With pairs (i, i + rot/2) lane c < rot/16 holds chunks c
// and c + rot/16, so both halves of its eight pairs are in its own registers
// and the rotation exchanges nothing; the chunks past rot, and all chunks when
// adjacent elements form the pairs, are dealt out two by two.
#include <cstdint>

#include <cuda_bf16.h>

#include "act_prologue.cuh"
#include "h3fp4_heads.h"
#include "ptx_sm103.cuh"

namespace h3fp4 {
namespace {

constexpr int kThreads = 128;

struct NormRopeParams {
    NormTensor t[2];
    long long M;
    int D, rot, half;
    float inv_d, eps;
    const float* cos;
    const float* sin;
    Segments seg;
};

__device__ __forceinline__ void load8(const float* p, float (&f)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(cvt_bf16x2(f2(f[0], f[1])), cvt_bf16x2(f2(f[2], f[3])), cvt_bf16x2(f2(f[4], f[5])),
                      cvt_bf16x2(f2(f[6], f[7])));
}

// kLanes lanes per head (a power of two, at least half the head's chunks).
template <int kLanes, bool kPairs>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeParams p)
{
    griddep_wait();
    constexpr int kGroups = 32 / kLanes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = lane & (kLanes - 1), g = lane / kLanes;
    const long long r = (long long)blockIdx.x * (kThreads / 32) + warp;
    if (r >= p.M) return;
    const int n = p.D >> 3, hc = p.rot >> 4;
    int ca, cb;  // this lane's chunks
    if (kPairs) {
        ca = 2 * c;
        cb = 2 * c + 1;
    } else if (c < hc) {
        ca = c;
        cb = c + hc;
    } else {
        ca = 2 * c;
        cb = 2 * c + 1;
    }
    const bool has_a = ca < n, has_b = cb < n;
    const int s = segment_of(p.seg, r);

    // The angles of this lane's pairs: eight for the split halves (shared by
    // both chunks), four per chunk for adjacent pairs.
    float co[8], si[8];
    bool turn_a = false, turn_b = false;
    if (p.rot > 0) {
        const float* cr = p.cos + r * p.half;
        const float* sr = p.sin + r * p.half;
        if (kPairs) {
            turn_a = 8 * ca < p.rot;  // rot is a multiple of 16: both chunks of a lane or none
            turn_b = turn_a;
            if (turn_a) {
                load8(cr + 4 * ca, co);
                load8(sr + 4 * ca, si);
            }
        } else if (c < hc) {
            turn_a = turn_b = true;
            load8(cr + 8 * c, co);
            load8(sr + 8 * c, si);
        }
    }
#pragma unroll 1
    for (int ti = 0; ti < 2; ++ti) {
        const NormTensor& t = p.t[ti];
        float wa[8], wb[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) wa[i] = wb[i] = 1.0f;
        if (t.weight) {
            if (has_a) load8(t.weight + (long long)s * p.D + 8 * ca, wa);
            if (has_b) load8(t.weight + (long long)s * p.D + 8 * cb, wb);
        }
#pragma unroll 1
        for (int h0 = 0; h0 < t.heads; h0 += kGroups) {
            const int h = h0 + g;
            const bool on = h < t.heads;
            uint4 va = make_uint4(0, 0, 0, 0), vb = va;
            const __nv_bfloat16* x = t.x + r * t.x_row + (long long)h * t.x_head;
            if (on && has_a) va = *reinterpret_cast<const uint4*>(x + 8 * ca);
            if (on && has_b) vb = *reinterpret_cast<const uint4*>(x + 8 * cb);
            float a[8], b[8];
            unpack8(va, a);
            unpack8(vb, b);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
            for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            const float rs = rsqrtf(fmaf(sum, p.inv_d, p.eps));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] *= rs * wa[i];
                b[i] *= rs * wb[i];
            }
            if (turn_a) {
                if (kPairs) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
                        a[2 * i] = a0 * co[i] - a1 * si[i];
                        a[2 * i + 1] = a1 * co[i] + a0 * si[i];
                        b[2 * i] = b0 * co[4 + i] - b1 * si[4 + i];
                        b[2 * i + 1] = b1 * co[4 + i] + b0 * si[4 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a0 = a[i], b0 = b[i];
                        a[i] = a0 * co[i] - b0 * si[i];
                        b[i] = b0 * co[i] + a0 * si[i];
                    }
                }
            }
            __nv_bfloat16* y = t.y + r * t.y_row + (long long)h * t.y_head;
            if (on && has_a) *reinterpret_cast<uint4*>(y + 8 * ca) = pack8(a);
            if (on && has_b) *reinterpret_cast<uint4*>(y + 8 * cb) = pack8(b);
        }
    }
}

template <int kLanes>
cudaError_t launch_lanes(const NormRopeParams& p, bool pairs, cudaStream_t s)
{
    const unsigned blocks = (unsigned)((p.M + kThreads / 32 - 1) / (kThreads / 32));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return pairs ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<kLanes, true>, p)
                 : cudaLaunchKernelEx(&cfg, norm_rope_kernel<kLanes, false>, p);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeJob& job, cudaStream_t s)
{
    NormRopeParams p{};
    p.t[0] = job.t[0];
    p.t[1] = job.t[1];
    p.M = job.M;
    p.D = job.D;
    p.rot = job.rot;
    p.half = job.rot / 2;
    p.inv_d = 1.0f / (float)job.D;
    p.eps = job.eps;
    p.cos = job.cos;
    p.sin = job.sin;
    p.seg = job.seg;
    const int need = (job.D / 8 + 1) / 2;  // lanes per head, two chunks each
    if (need <= 1) return launch_lanes<1>(p, job.pairs, s);
    if (need <= 2) return launch_lanes<2>(p, job.pairs, s);
    if (need <= 4) return launch_lanes<4>(p, job.pairs, s);
    if (need <= 8) return launch_lanes<8>(p, job.pairs, s);
    return launch_lanes<16>(p, job.pairs, s);
}

}  // namespace h3fp4
