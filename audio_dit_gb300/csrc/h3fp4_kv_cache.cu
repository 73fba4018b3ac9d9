// Rows into the 4-bit cache and back.
//
//     S = e4m3(max |x| (1/6) / s),  q = e2m1(x / (S s))   per 16 elements of a head
//     x' = bf16(q S s)                                     on the way back
//
// s the head's global scale, each step one rounding to fp32.  As the activations' quantiser
// (nvfp4_encode.cuh) but for the sixth, which is a product with RN(1/6) as in the elementary
// form of this format, where that one divides: the two are one step of fp32 apart at most, and
// their codes differ only where that step crosses a tie of E4M3.  Which blocks do depends on the
// head's global scale: of scales f amax / 2688 with amax in bf16, those with f = 1 and a mantissa
// of amax of 1.09375, 1.203125, 1.53125 or 1.75 have 0.7 to 2.1 % of such block maxima, with f =
// 1.25 that of 1.75 has 0.7 %, with f = 1.5 none has any; of 20000 scales at random one has.
// A NaN in a block makes its scale NaN and so all of it.
// Memory-bound: 4 bytes of bf16 per pair of K and V elements and 9/8 of the cache.
// A warp takes a run of rows.  Measured, 8 heads of 128: 16384 rows in 22 us (3940 GB/s: the
// loads' latency beside 55 % of the issue slots; loading ahead needs registers that take the
// warps away, 26.7 us), 25385 rows out 25.5 us (5230 GB/s; with more warps an SM 27 to 35, with
// fewer instructions for a code, but more registers, 27); 64 rows 4.2 and 3.2 us (a launch).
#include <cstdint>

#include <cuda_bf16.h>

#include "act_prologue.cuh"
#include "h3fp4_token.h"
#include "kv_cache.cuh"
#include "nvfp4_encode.cuh"
#include "ptx_sm103.cuh"

namespace h3fp4 {
namespace {

constexpr int kThreads = 128;

// Two E2M1 codes -> fp32 (the low four bits first).
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

// Four codes (16 bits) to the low halves of four bytes, and back.
__device__ __forceinline__ uint32_t spread(uint32_t x)
{
    x &= 0xFFFFu;
    x = (x | (x << 8)) & 0x00FF00FFu;
    return (x | (x << 4)) & 0x0F0F0F0Fu;
}

__device__ __forceinline__ uint32_t gather(uint32_t x)
{
    x &= 0x0F0F0F0Fu;
    x = (x | (x >> 4)) & 0x00FF00FFu;
    return (x | (x >> 8)) & 0xFFFFu;
}

// Sixteen bf16 values.
__device__ __forceinline__ V16 load16(const __nv_bfloat16* x)
{
    V16 v;
    *reinterpret_cast<uint4*>(v.w) = *reinterpret_cast<const uint4*>(x);
    *reinterpret_cast<uint4*>(v.w + 4) = *reinterpret_cast<const uint4*>(x + 8);
    return v;
}

// Codes (eight of 16 elements in each word) and scale of a block.
__device__ __forceinline__ uint32_t encode(const V16& v, float s, uint32_t (&w)[2])
{
    float f[16];
    unpack16(v, f);
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; k += 2) top = max3_nan(top, fabsf(f[k]), fabsf(f[k + 1]));   // (a NaN stays: E4M3's scale is NaN)
    const uint32_t S = cvt_e4m3(__fdiv_rn(__fmul_rn(top, 1.0f / 6.0f), s));
    const float rcp = block_rcp(S, s);
#pragma unroll
    for (int k = 0; k < 16; k += 2) unf2(mul2(f2(f[k], f[k + 1]), f2(rcp, rcp)), f[k], f[k + 1]);
    w[0] = e2m1x8(reinterpret_cast<const float(&)[8]>(f[0]));
    w[1] = e2m1x8(reinterpret_cast<const float(&)[8]>(f[8]));
    return S;
}

__device__ __forceinline__ uint4 decode(uint32_t w, uint32_t code, float s)
{
    const float S = e4m3_value(code);
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 q = e2m1_pair((w >> (8 * k)) & 0xFFu);
        o[k] = cvt_bf16x2(f2(q.x * S * s, q.y * S * s));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The 16 bytes that two tokens' values share.
template <int W>
struct Shared16 {
    static constexpr int kSecond = W == 64 ? 32 : 8;
    uint32_t w[4];
    __device__ __forceinline__ void load(const uint8_t* p)
    {
        const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(p + kSecond);
        w[0] = a.x, w[1] = a.y, w[2] = b.x, w[3] = b.y;
    }
    __device__ __forceinline__ void store(uint8_t* p) const
    {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(p + kSecond) = make_uint2(w[2], w[3]);
    }
};

// The rows of a warp, one after the other: the sequence of each, and its place.
struct Rows {
    int s = -1;
    long long first = 0, end = 0, len = 0, n = 0;   // the sequence's rows, tokens that there is room for, its length

    // Position of row r, or -1 where it has none: one warp, all lanes.
    __device__ __forceinline__ long long place(const CacheView& c, long long r, int lane)
    {
        if (s < 0 || r >= end) {
            s = cache_sequence(c, r, lane);
            if (s < 0) return -1;
            first = c.row_off ? c.row_off[s] : r;
            end = c.row_off ? c.row_off[s + 1] : r + 1;
            n = c.length[s];
            len = cache_length(c, s);
        }
        const long long pos = n - (end - r);
        return pos < len ? pos : -1;
    }
};

// A lane takes a block of 16 elements of a head at a time.
template <int W>
__global__ void __launch_bounds__(kThreads, 7) cache_append_kernel(const __grid_constant__ CacheRowsJob p, int rows_per_warp)
{
    using L = CacheLayout<W>;
    constexpr int kHeads = 32 / L::kBlocks;   // heads of a warp at a time
    const int lane = threadIdx.x & 31, b = lane % L::kBlocks, h0 = lane / L::kBlocks;
    const CacheView& c = p.c;
    const bool real = 16 * b < c.D;
    const long long head_bytes = (long long)(c.page / kCacheGroup) * L::kGroupBytes;
    griddep_wait();
    const long long warp = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const long long r0 = warp * rows_per_warp, r1 = min((long long)p.M, r0 + rows_per_warp);
    Rows rows;
    for (long long r = r0; r < r1; ++r) {
        const long long pos = rows.place(c, r, lane);
        if (pos < 0) continue;
        uint8_t* base = cache_group<W>(c, rows.s, pos, 0);
        if (!base) continue;
        const int t = (int)((uint32_t)pos % (uint32_t)c.page) % kCacheGroup, shift = 4 * (t & 1);
        // Two tokens share V's bytes: the row of the first writes both where the call has both, else a row
        // keeps the other token's bits.
        const bool with_next = !(t & 1) && r + 1 < min(rows.end, (long long)p.M) && pos + 1 < rows.len;
        const bool with_last = (t & 1) && r > rows.first && r > 0;
        const __nv_bfloat16* kp = p.k.p + r * p.k.row + h0 * p.k.head + 16 * b;
        const __nv_bfloat16* vp = p.v.p + r * p.v.row + h0 * p.v.head + 16 * b;
        uint8_t* g = base + h0 * head_bytes;
        for (int h = h0; h < c.Hkv; h += kHeads, kp += kHeads * p.k.head, vp += kHeads * p.v.head, g += kHeads * head_bytes) {
            // (blocks past the head are zeros under a scale of zero)
            V16 k = {}, v = {}, v2 = {};
            if (real) {
                k = load16(kp);
                if (!with_last) v = load16(vp);
                if (with_next) v2 = load16(vp + p.v.row);
            }
            uint32_t w[2];
            const uint32_t S = encode(k, c.k_gscale ? c.k_gscale[h] : 1.0f, w);
            *reinterpret_cast<uint2*>(g + L::k_codes(t, b)) = make_uint2(w[0], w[1]);
            g[L::k_scale(t, b)] = (uint8_t)S;
            if (with_last) continue;
            const float gs = c.v_gscale ? c.v_gscale[h] : 1.0f;
            Shared16<W> m = {};
            if (!with_next) m.load(g + L::v_codes(t, b));
            const uint32_t keep = 0xF0F0F0F0u >> shift;
            g[L::v_scale(t, b)] = (uint8_t)encode(v, gs, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) m.w[i] = (m.w[i] & keep) | (spread(w[i >> 1] >> (16 * (i & 1))) << shift);
            if (with_next) {
                g[L::v_scale(t + 1, b)] = (uint8_t)encode(v2, gs, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) m.w[i] |= spread(w[i >> 1] >> (16 * (i & 1))) << 4;
            }
            m.store(g + L::v_codes(t, b));
        }
    }
}

// A lane takes half a block, so that whole lines of bf16 are written.
template <int W>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheRowsJob p, int rows_per_warp)
{
    using L = CacheLayout<W>;
    constexpr int kLanes = 2 * L::kBlocks;    // of a head
    constexpr int kHeads = 32 / kLanes;       // heads of a warp at a time
    constexpr int kBatch = 4;                 // and how many of them it has in flight
    const int lane = threadIdx.x & 31, b = lane % kLanes >> 1, half = lane & 1, h0 = lane / kLanes;
    const CacheView& c = p.c;
    const int d = 16 * b + 8 * half;
    const long long head_bytes = (long long)(c.page / kCacheGroup) * L::kGroupBytes;
    griddep_wait();
    const long long warp = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const long long r0 = warp * rows_per_warp, r1 = min((long long)p.M, r0 + rows_per_warp);
    Rows rows;
    for (long long r = r0; r < r1; ++r) {
        const long long pos = rows.place(c, r, lane);
        if (pos < 0) continue;
        const uint8_t* base = cache_group<W>(c, rows.s, pos, 0);
        if (!base || d >= c.D) continue;
        const int t = (int)((uint32_t)pos % (uint32_t)c.page) % kCacheGroup, shift = 4 * (t & 1);
        for (int h1 = h0; h1 < c.Hkv; h1 += kHeads * kBatch) {
            uint32_t k[kBatch], sk[kBatch], sv[kBatch];
            uint2 v[kBatch];
            float gk[kBatch], gv[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int h = h1 + u * kHeads;
                if (h >= c.Hkv) continue;
                const uint8_t* g = base + h * head_bytes;
                k[u] = *reinterpret_cast<const uint32_t*>(g + L::k_codes(t, b) + 4 * half);
                v[u] = *reinterpret_cast<const uint2*>(g + L::v_codes(t, b) + half * Shared16<W>::kSecond);
                sk[u] = g[L::k_scale(t, b)];
                sv[u] = g[L::v_scale(t, b)];
                gk[u] = c.k_gscale ? c.k_gscale[h] : 1.0f;
                gv[u] = c.v_gscale ? c.v_gscale[h] : 1.0f;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int h = h1 + u * kHeads;
                if (h >= c.Hkv) continue;
                const uint32_t codes = gather(v[u].x >> shift) | (gather(v[u].y >> shift) << 16);
                *reinterpret_cast<uint4*>(p.k_out + r * p.k.row + h * p.k.head + d) = decode(k[u], sk[u], gk[u]);
                *reinterpret_cast<uint4*>(p.v_out + r * p.v.row + h * p.v.head + d) = decode(codes, sv[u], gv[u]);
            }
        }
    }
}

template <int W>
constexpr void (*kernel_of(bool read))(CacheRowsJob, int)
{
    return read ? cache_read_kernel<W> : cache_append_kernel<W>;
}

cudaError_t launch(const CacheRowsJob& job, bool read, cudaStream_t s)
{
    if (job.M == 0) return cudaSuccess;
    // each warp with a run of rows: on the way in as many as are resident, on the way out half as many again (25.5
    // us of 25385 rows; 26.0 with fewer, 27.4 with twice as many)
    const long long most = (long long)sm_count_current_device() * (read ? 96 : 28);
    const int per_warp = (int)((job.M + most - 1) / most);
    const long long warps = (job.M + per_warp - 1) / per_warp;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int w = cache_width(job.c.D);
    return cudaLaunchKernelEx(&cfg, w == 64 ? kernel_of<64>(read) : w == 128 ? kernel_of<128>(read) : kernel_of<256>(read), job,
                              per_warp);
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowsJob& job, cudaStream_t s) { return launch(job, false, s); }

cudaError_t launch_cache_read(const CacheRowsJob& job, cudaStream_t s) { return launch(job, true, s); }

}  // namespace h3fp4
