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
//
// A warp takes kUnroll heads per group of one tensor (a part of the row's heads)
// for every so many rows: its weights stay in registers, and all of a row's loads
// are issued before the first is used, which is what memory latency asks for.
//
// Measured (24 + 24 heads of 128, all rotated; calls back to back): 31744 rows
// 120 us (6.6 TB/s of 6.8 that a copy reaches), 8192 rows 34 us (6.1 TB/s), one
// row 2 us.  31744 rows with flushed caches: three heads in flight and five
// blocks per SM 126 us, two and eight 144, six and three 130; a whole row per
// warp 136.
#include <cstdint>
#include <numeric>

#include <cuda_bf16.h>

#include "act_prologue.cuh"
#include "h3fp4_heads.h"
#include "ptx_sm103.cuh"

namespace h3fp4 {
namespace {

constexpr int kThreads = 128;

constexpr int kUnroll = 3;  // heads of a group in flight: 24 heads of 128 are two parts
constexpr int kBlocksPerSm = 5;

struct NormRopeParams {
    NormTensor t[2];
    int parts[2];       // of a row's heads, per tensor
    long long M;
    int D, rot, half;
    float inv_d, eps;
    const float* cos;
    const float* sin;
    Segments seg;
};

__device__ __forceinline__ void load8(const float* p, float (&f)[8])
{
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
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
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) norm_rope_kernel(const __grid_constant__ NormRopeParams p)
{
    constexpr int kGroups = 32 / kLanes;
    const int lane = threadIdx.x & 31;
    const int c = lane & (kLanes - 1), g = lane / kLanes;
    // this warp's tensor, part of its heads, first row and step
    const unsigned all_parts = p.parts[0] + p.parts[1];
    const unsigned warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kThreads / 32);
    const int part = warp % all_parts;
    const bool second = part >= p.parts[0];
    const NormTensor& t = p.t[second ? 1 : 0];
    const int h0 = (second ? part - p.parts[0] : part) * (kGroups * kUnroll) + g;
    const unsigned step = warps / all_parts;  // the grid is a multiple of the parts
    const int n = p.D >> 3, hc = p.rot >> 4;
    int ca = 2 * c, cb = 2 * c + 1;  // this lane's chunks
    if (!kPairs && c < hc) {
        ca = c;
        cb = c + hc;
    }
    const bool has_a = ca < n, has_b = cb < n;
    // Pairs of adjacent elements: rot is a multiple of 16, both chunks of a lane turn or none.
    const bool turn = kPairs ? 8 * ca < p.rot : c < hc;
    const int angle = kPairs ? 4 * ca : 8 * c;
    const __nv_bfloat16* xa = t.x + 8 * ca;
    const __nv_bfloat16* xb = t.x + 8 * cb;
    __nv_bfloat16* ya = t.y + 8 * ca;
    __nv_bfloat16* yb = t.y + 8 * cb;
    griddep_wait();
    float wa[8], wb[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wa[i] = wb[i] = 1.0f;
    long long seg_end = 0;  // the weights are those of the rows before it
    for (long long r = warp / all_parts; r < p.M; r += step) {
        uint4 va[kUnroll], vb[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int h = h0 + k * kGroups;
            const long long at = r * t.x_row + (long long)h * t.x_head;
            va[k] = vb[k] = make_uint4(0, 0, 0, 0);
            if (h < t.heads && has_a) va[k] = *reinterpret_cast<const uint4*>(xa + at);
            if (h < t.heads && has_b) vb[k] = *reinterpret_cast<const uint4*>(xb + at);
        }
        // The angles of this lane's pairs: eight that both chunks share, or four per chunk.
        float co[8], si[8];
        if (turn) {
            load8(p.cos + r * p.half + angle, co);
            load8(p.sin + r * p.half + angle, si);
        }
        if (r >= seg_end) {
            const int s = segment_of(p.seg, r);
            seg_end = p.seg.off[s + 1];
            if (t.weight) {
                if (has_a) load8(t.weight + (long long)s * p.D + 8 * ca, wa);
                if (has_b) load8(t.weight + (long long)s * p.D + 8 * cb, wb);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            float a[8], b[8];
            unpack8(va[k], a);
            unpack8(vb[k], b);
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
            if (turn) {
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
            const int h = h0 + k * kGroups;
            const long long at = r * t.y_row + (long long)h * t.y_head;
            if (h < t.heads && has_a) *reinterpret_cast<uint4*>(ya + at) = pack8(a);
            if (h < t.heads && has_b) *reinterpret_cast<uint4*>(yb + at) = pack8(b);
        }
    }
}

template <int kLanes>
cudaError_t launch_lanes(NormRopeParams& p, bool pairs, cudaStream_t s)
{
    constexpr int kHeads = 32 / kLanes * kUnroll, kWarps = kThreads / 32;
    for (int i = 0; i < 2; ++i) p.parts[i] = (p.t[i].heads + kHeads - 1) / kHeads;
    // Warps for as many rows as are resident at once, which then take the next rows; up to
    // four times as many where a warp has few rows, so that blocks in waiting even out the
    // end (4099 rows of 25 heads of 80: 17 against 21 us; 31744 rows of 48 heads of 128:
    // 128 against 126 us).  Either way a whole number of rows' warps.
    const long long parts = p.parts[0] + p.parts[1], most = (long long)sm_count_current_device() * kBlocksPerSm * kWarps;
    long long rows = most / parts;
    if (p.M <= 16 * rows) rows *= 4;
    rows = rows < 1 ? 1 : rows < p.M ? rows : p.M;
    const long long whole = parts / std::gcd(parts, (long long)kWarps);  // blocks whose warps are whole rows
    const long long blocks = ((rows * parts + kWarps - 1) / kWarps + whole - 1) / whole * whole;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)blocks);
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
