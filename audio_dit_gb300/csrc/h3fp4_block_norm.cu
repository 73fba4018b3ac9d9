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
// sum over the registers), and each output is rounded once.
//
// Rows of up to 512 by parts of a warp, the next one on its way; up to 8192 by a block that
// copies rows ahead into a ring of three (each thread its own columns, so that no barrier guards
// it), keeps a segment's vectors for its columns folded to three in registers and computes in
// pairs; wider ones by a block that reads the vectors when they are needed.
//
// Measured, of the measured 6793 GB/s: 31744 rows of 3072 with gate and modulation 123 us (6320
// GB/s), 4099 of 5192 with both norms 38.5 us (4430; two block sums a row, one after the other,
// and rows that end inside a sector: 8192 rows of 5192 take 65 us, where as many of 6144 take
// 63), 8192 of 3072 33 us, 170000 of 256 60 us (5790), of 512 108 us (6450), one row 2.1 us (a
// launch).  8192 rows of 8192 take 90 us, as few as 82 with less ahead: whole tensors a power of
// two apart.  Of wider ones 2048 rows of 16384 take 86 us with all vectors (3140 GB/s: 2.5 bytes
// of vectors from L2 for each of the row), 57 with one.
// In single values, with the warps' sums joined by shuffles, the first took 135 us and the
// second 43; vectors read for each row took 74 us of 170000 rows of 256.  The second norm's sum
// behind one barrier with the next row's first: 42 for that 43, but 146 for the 135 without a
// first norm.  Rings of two: 131 and 40 us.  Clusters of two and four blocks to a wide row: 78 us
// for that 86, but 68 for 57 with one vector, and 296 for 158 of 32768.
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

// Eight bf16 values as pairs of fp32, and back.
__device__ __forceinline__ void unpack_pairs(const uint4& v, uint64_t (&f)[4])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(bf16_lo(w[i]), bf16_hi(w[i]));
}

__device__ __forceinline__ uint4 pack_pairs(const uint64_t (&f)[4])
{
    return make_uint4(cvt_bf16x2(f[0]), cvt_bf16x2(f[1]), cvt_bf16x2(f[2]), cvt_bf16x2(f[3]));
}

__device__ __forceinline__ float both(uint64_t v)
{
    float lo, hi;
    unf2(v, lo, hi);
    return lo + hi;
}

// A segment's vectors of eight columns from `at` on, in pairs: what y and the normed r are multiplied with, and
// what is added.
__device__ __forceinline__ void fold_vectors(const BlockNormParams& p, long long at, uint64_t (&va)[4], uint64_t (&vb)[4],
                                             uint64_t (&vc)[4])
{
    float a[8], b[8], c[8], w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = b[j] = 1.0f, c[j] = 0.0f;
    if (p.gate) load_f8(p.gate + at, a);
    if (p.y_weight) {
        load_f8(p.y_weight + at, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] *= w[j];
    }
    if (p.weight) load_f8(p.weight + at, b);
    if (p.scale) {
        load_f8(p.scale + at, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] *= 1.0f + w[j];
    }
    if (p.shift) load_f8(p.shift + at, c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        va[j] = f2(a[2 * j], a[2 * j + 1]);
        vb[j] = f2(b[2 * j], b[2 * j + 1]);
        vc[j] = f2(c[2 * j], c[2 * j + 1]);
    }
}

// max |.| of bf16 values, as fp32 bits (a NaN is above all).
__device__ __forceinline__ uint32_t top_of(uint32_t top, const uint4& o)
{
    const uint32_t words[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, max((words[j] << 16) & 0x7FFF0000u, words[j] & 0x7FFF0000u));
    return top;
}

// Narrow rows: kRow lanes each, kVec vectors a lane, the next row on its way.  Vectors stay in registers while the
// segment does.
template <int kRow, int kVec>
__global__ void __launch_bounds__(128, kVec == 1 ? 6 : 4) block_norm_narrow_kernel(const __grid_constant__ BlockNormParams p)
{
    constexpr int kRows = 32 / kRow;   // rows of a warp
    const int lane = threadIdx.x & 31, t = lane % kRow, nv = p.K >> 3;
    const long long step = (long long)gridDim.x * (4 * kRows);
    griddep_wait();
    auto sum_of = [&](float v) {
#pragma unroll
        for (int o = kRow / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    uint4 x[kVec], y[kVec];
    auto load = [&](long long r) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = t + i * kRow;
            x[i] = y[i] = make_uint4(0, 0, 0, 0);
            if (r < p.M && v < nv) {
                x[i] = *reinterpret_cast<const uint4*>(p.x + r * p.K + 8 * v);
                if (p.y) y[i] = *reinterpret_cast<const uint4*>(p.y + r * p.K + 8 * v);
            }
        }
    };
    uint64_t va[kVec][4], vb[kVec][4], vc[kVec][4];
    long long seg_end = 0;
    uint32_t top = 0;
    // the warp's first row; a lane's is `lane / kRow` on (past the last one: zeros, nothing is written)
    long long r0 = ((long long)blockIdx.x * 4 + (threadIdx.x >> 5)) * kRows;
    load(r0 + lane / kRow);
    for (; r0 < p.M; r0 += step) {
        const long long r = r0 + lane / kRow, row = r * p.K;
        const bool mine = r < p.M;
        if (mine && r >= seg_end) {
            const int sg = segment_of(p.seg, r);
            seg_end = p.seg.off[sg + 1];
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                fold_vectors(p, (long long)sg * p.K + 8 * min(t + i * kRow, nv - 1), va[i], vb[i], vc[i]);
        }
        uint64_t f[kVec][4], g[kVec][4];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            unpack_pairs(x[i], f[i]);
            unpack_pairs(y[i], g[i]);
        }
        load(r + step);
        if (p.y) {
            if (p.post) {
                uint64_t sum = 0;
#pragma unroll
                for (int i = 0; i < kVec; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum = fma2(g[i][j], g[i][j], sum);
                const float rs = rsqrtf(fmaf(sum_of(both(sum)), p.inv_k, p.eps));
#pragma unroll
                for (int i = 0; i < kVec; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) g[i][j] = mul2(g[i][j], f2(rs, rs));
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = t + i * kRow;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[i][j] = fma2(f2(p.x_scale, p.x_scale), f[i][j], mul2(g[i][j], va[i][j]));
                if (p.x_out && mine && v < nv) *reinterpret_cast<uint4*>(p.x_out + row + 8 * v) = pack_pairs(f[i]);
            }
        }
        if (!p.out) continue;
        if (p.layer) {
            uint64_t sum = 0;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (t + i * kRow < nv) sum = add2(sum, f[i][j]);
            const float mean = sum_of(both(sum)) * p.inv_k;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = add2(f[i][j], f2(-mean, -mean));
        }
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t + i * kRow < nv) sum = fma2(f[i][j], f[i][j], sum);
        const float rs = rsqrtf(fmaf(sum_of(both(sum)), p.inv_k, p.eps));
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = t + i * kRow;
            if (!mine || v >= nv) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) f[i][j] = fma2(mul2(f[i][j], f2(rs, rs)), vb[i][j], vc[i][j]);
            const uint4 o = pack_pairs(f[i]);
            *reinterpret_cast<uint4*>(p.out + row + 8 * v) = o;
            if (p.amax) top = top_of(top, o);
        }
    }
    if (p.amax) {
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0 && top != 0) atomicMax(p.amax, top);
    }
}

__device__ __forceinline__ void copy16(void* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Wide rows: a block of kWide threads each, rows copied ahead (each thread its own columns), the vectors read when
// they are needed.
constexpr int kWide = 1024;

template <int kVec>
constexpr int kWideRing = kVec == 2 ? 3 : 1;   // rows ahead: what shared memory holds

template <int kVec>
__global__ void __launch_bounds__(kWide) block_norm_wide_kernel(const __grid_constant__ BlockNormParams p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float part[2][kWide / 32];
    constexpr int kAhead = kWideRing<kVec>, kSlot = 2 * kVec;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, nv = p.K >> 3;
    uint32_t turn = 0, top = 0;
    // a sum over the block: consecutive ones use different halves of `part`, so one barrier each is enough
    auto block_sum = [&](float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) part[turn][warp] = v;
        __syncthreads();
        v = part[turn][lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        turn ^= 1u;
        return v;
    };
    auto times = [](uint64_t (&f)[4], const float* p) {
        float w[8];
        load_f8(p, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = mul2(f[j], f2(w[2 * j], w[2 * j + 1]));
    };
    uint4* ring = reinterpret_cast<uint4*>(smem) + t;   // [row][x, y][vector of the thread][thread]
    auto copy = [&](long long r, int slot, bool y) {
        const __nv_bfloat16* from = (y ? p.y : p.x) + r * p.K;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = t + i * kWide;
            if (r < p.M && v < nv) copy16(ring + (slot * kSlot + (y ? kVec : 0) + i) * kWide, from + 8 * v);
        }
    };
    auto load = [&](long long r, int slot) {
        copy(r, slot, false);
        if (p.y) copy(r, slot, true);
        asm volatile("cp.async.commit_group;" ::: "memory");   // (also where there is nothing: groups are counted)
    };
    griddep_wait();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(blockIdx.x + (long long)i * gridDim.x, i);
    int slot = 0;
    for (long long r = blockIdx.x; r < p.M; r += gridDim.x) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const long long row = r * p.K;
        auto got = [&](int i, bool y) {
            return t + i * kWide < nv ? ring[(slot * kSlot + (y ? kVec : 0) + i) * kWide] : make_uint4(0, 0, 0, 0);
        };
        const long long at = (long long)segment_of(p.seg, r) * p.K;
        uint64_t f[kVec][4];
#pragma unroll
        for (int i = 0; i < kVec; ++i) unpack_pairs(got(i, false), f[i]);
        if (p.y) {
            float rs = 1.0f;
            if (p.post) {
                uint64_t sum = 0;
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    uint64_t y[4];
                    unpack_pairs(got(i, true), y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum = fma2(y[j], y[j], sum);
                }
                rs = rsqrtf(fmaf(block_sum(both(sum)), p.inv_k, p.eps));
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = t + i * kWide;
                if (v >= nv) continue;
                uint64_t y[4];
                unpack_pairs(got(i, true), y);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], f2(rs, rs));
                if (p.y_weight) times(y, p.y_weight + at + 8 * v);
                if (p.gate) times(y, p.gate + at + 8 * v);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = fma2(f2(p.x_scale, p.x_scale), f[i][j], y[j]);
                if (p.x_out) *reinterpret_cast<uint4*>(p.x_out + row + 8 * v) = pack_pairs(f[i]);
            }
        }
        load(r + (long long)kAhead * gridDim.x, slot);   // (the thread has read what is its own)
        slot = slot + 1 == kAhead ? 0 : slot + 1;
        if (!p.out) continue;
        if (p.layer) {
            uint64_t sum = 0;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = add2(sum, f[i][j]);   // (places past the row hold zeros)
            const float mean = block_sum(both(sum)) * p.inv_k;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = add2(f[i][j], f2(-mean, -mean));
        }
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            if (t + i * kWide >= nv) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum = fma2(f[i][j], f[i][j], sum);
        }
        const float rs = rsqrtf(fmaf(block_sum(both(sum)), p.inv_k, p.eps));
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = t + i * kWide;
            if (v >= nv) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) f[i][j] = mul2(f[i][j], f2(rs, rs));
            if (p.weight) times(f[i], p.weight + at + 8 * v);
            if (p.scale) {
                float w[8];
                load_f8(p.scale + at + 8 * v, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = mul2(f[i][j], add2(f2(w[2 * j], w[2 * j + 1]), f2(1.0f, 1.0f)));
            }
            if (p.shift) {
                float w[8];
                load_f8(p.shift + at + 8 * v, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = add2(f[i][j], f2(w[2 * j], w[2 * j + 1]));
            }
            const uint4 o = pack_pairs(f[i]);
            *reinterpret_cast<uint4*>(p.out + row + 8 * v) = o;
            if (p.amax) top = top_of(top, o);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (p.amax) {
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0 && top != 0) atomicMax(p.amax, top);
    }
}

// The same for many rows: a block keeps its columns' vectors in registers, folded into three
// (y_weight gate, weight (1 + scale), shift), and takes rows one after the other.  Its threads copy their
// columns of the next rows to shared memory ahead of time (each for itself, nothing waits for others), so
// that enough bytes are on their way whatever the sums wait for.
constexpr int kRing = 3;   // rows ahead

template <int kVec, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks)
    block_norm_ring_kernel(const __grid_constant__ BlockNormParams p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kWarps = kThreads / 32;
    __shared__ __align__(16) float part[2][kWarps];   // of warps that there are not: zeros
    static_assert(kThreads % 128 == 0, "four sums a load");
    const int t = threadIdx.x, threads = blockDim.x, warp = t >> 5, lane = t & 31;
    const int nv = p.K >> 3;
    uint4* ring = reinterpret_cast<uint4*>(smem) + t;   // [row][x, y][vector of the thread][thread]
    constexpr int kY = kVec, kSlot = 2 * kVec;
    for (int i = t; i < 2 * kWarps; i += threads) (&part[0][0])[i] = 0.0f;
    __syncthreads();
    griddep_wait();
    auto load = [&](long long r, int slot) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = t + i * threads;
            if (r < p.M && v < nv) {
                copy16(ring + (slot * kSlot + i) * threads, p.x + r * p.K + 8 * v);
                if (p.y) copy16(ring + (slot * kSlot + kY + i) * threads, p.y + r * p.K + 8 * v);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");   // (also where there is nothing: groups are counted)
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) load(blockIdx.x + (long long)i * gridDim.x, i);
    uint32_t turn = 0, top = 0;
    // a sum over the block: consecutive ones use different halves of `part`, so one barrier each is enough
    auto block_sum = [&](float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) part[turn][warp] = v;
        __syncthreads();
        // (all warps' sums by each thread: fewer steps one after another than by shuffles)
        constexpr int kFours = kWarps / 4;
        float four[kFours];
#pragma unroll
        for (int i = 0; i < kFours; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(&part[turn][4 * i]);
            four[i] = (x.x + x.y) + (x.z + x.w);
        }
        turn ^= 1u;
        v = four[0];
#pragma unroll
        for (int i = 1; i < kFours; ++i) v += four[i];
        return v;
    };
    uint64_t va[kVec][4], vb[kVec][4], vc[kVec][4];   // pairs, as all below
    long long seg_end = 0;
    int slot = 0;
    for (long long r = blockIdx.x; r < p.M; r += gridDim.x) {
        if (r >= seg_end) {
            const int sg = segment_of(p.seg, r);
            seg_end = p.seg.off[sg + 1];
            const long long at = (long long)sg * p.K;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = min(t + i * threads, nv - 1);
                fold_vectors(p, at + 8 * v, va[i], vb[i], vc[i]);
            }
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        uint64_t f[kVec][4], y[kVec][4];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const bool real = t + i * threads < nv;
            unpack_pairs(real ? ring[(slot * kSlot + i) * threads] : zero, f[i]);
            if (p.y) unpack_pairs(real ? ring[(slot * kSlot + kY + i) * threads] : zero, y[i]);
        }
        const long long row = r * p.K;
        if (p.y) {
            if (p.post) {
                uint64_t sum = 0;
#pragma unroll
                for (int i = 0; i < kVec; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum = fma2(y[i][j], y[i][j], sum);
                const float rs = rsqrtf(fmaf(block_sum(both(sum)), p.inv_k, p.eps));
#pragma unroll
                for (int i = 0; i < kVec; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[i][j] = mul2(y[i][j], f2(rs, rs));
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = t + i * threads;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[i][j] = fma2(f2(p.x_scale, p.x_scale), f[i][j], mul2(y[i][j], va[i][j]));
                if (p.x_out && v < nv) *reinterpret_cast<uint4*>(p.x_out + row + 8 * v) = pack_pairs(f[i]);
            }
        }
        if (p.layer) {
            uint64_t sum = 0;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = add2(sum, f[i][j]);   // (places past the row hold zeros)
            const float mean = block_sum(both(sum)) * p.inv_k;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = add2(f[i][j], f2(-mean, -mean));
        }
        uint64_t pairs = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            if (t + i * threads >= nv) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) pairs = fma2(f[i][j], f[i][j], pairs);
        }
        const float sum = block_sum(both(pairs));
        // (the sum has used what the thread read of the slot)
        load(r + (long long)kRing * gridDim.x, slot);
        if (p.out) {
            const float rs = rsqrtf(fmaf(sum, p.inv_k, p.eps));
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = t + i * threads;
                if (v >= nv) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = fma2(mul2(f[i][j], f2(rs, rs)), vb[i][j], vc[i][j]);
                const uint4 o = pack_pairs(f[i]);
                *reinterpret_cast<uint4*>(p.out + row + 8 * v) = o;
                if (p.amax) top = top_of(top, o);
            }
        }
        slot = slot + 1 == kRing ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (p.amax) {
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0 && top != 0) atomicMax(p.amax, top);
    }
}

template <int kVec, int kThreads, int kBlocks>
cudaError_t launch_ring(const BlockNormParams& p, cudaStream_t s)
{
    const int nv = p.K / 8, threads = ((nv + kVec - 1) / kVec + 31) / 32 * 32;
    const int bytes = kRing * 2 * kVec * 16 * threads;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(block_norm_ring_kernel<kVec, kThreads, kBlocks>),
                                              kRing * 2 * kVec * 16 * kThreads);
    if (e != cudaSuccess) return e;
    // as many as are resident at the registers that kThreads leave
    const long long most = (long long)sm_count_current_device() * (kThreads * kBlocks / threads);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(p.M < most ? p.M : most));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, block_norm_ring_kernel<kVec, kThreads, kBlocks>, p);
}

template <int kRow, int kVec>
cudaError_t launch_narrow(const BlockNormParams& p, cudaStream_t s)
{
    constexpr int kRows = 4 * (32 / kRow);
    const long long blocks = (p.M + kRows - 1) / kRows, most = (long long)sm_count_current_device() * (kVec == 1 ? 6 : 4);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, block_norm_narrow_kernel<kRow, kVec>, p);
}

template <int kVec>
cudaError_t launch_wide(const BlockNormParams& p, cudaStream_t s)
{
    constexpr int bytes = kWideRing<kVec> * 2 * kVec * 16 * kWide;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(block_norm_wide_kernel<kVec>), bytes);
    if (e != cudaSuccess) return e;
    const long long most = sm_count_current_device();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(p.M < most ? p.M : most));
    cfg.blockDim = dim3(kWide);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, block_norm_wide_kernel<kVec>, p);
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
    // Rows of up to 64 vectors by parts of a warp, wider ones by a block and from its ring: so also single
    // rows, whose vectors it fetches while the sums are made (128 rows of 3072 2.5 us against 4.0 for blocks
    // that read the vectors when they need them, 8192 rows 33 against 48).
    if (nv <= 8) return launch_narrow<8, 1>(p, s);
    if (nv <= 16) return launch_narrow<16, 1>(p, s);
    if (nv <= 32) return launch_narrow<32, 1>(p, s);
    if (nv <= 64) return launch_narrow<32, 2>(p, s);
    if (nv <= 384) return launch_ring<1, 384, 2>(p, s);
    if (nv <= 512) return launch_ring<1, 512, 2>(p, s);
    if (nv <= 1024) return launch_ring<2, 512, 1>(p, s);
    if (nv <= 2048) return launch_wide<2>(p, s);
    return launch_wide<4>(p, s);
}

}  // namespace h3fp4
