// Rows into the 4-bit cache and back.
//
//     S = e4m3(max |x| / 6 / s),  q = e2m1(x / (S s))     per 16 elements of a head
//     x' = bf16(q S s)                                     on the way back
//
// with the quantiser's own arithmetic (nvfp4_encode.cuh), s the head's global scale.
// Memory-bound: 4 bytes of bf16 per pair of K and V elements and 9/8 of the cache.
// A warp takes one row; a lane one block of 16 elements at a time.
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

// Codes (eight of 16 elements in each word) and scale of a block.
__device__ __forceinline__ void encode(const __nv_bfloat16* x, float s, uint32_t (&w)[2], uint32_t& S)
{
    V16 v;
    *reinterpret_cast<uint4*>(v.w) = *reinterpret_cast<const uint4*>(x);
    *reinterpret_cast<uint4*>(v.w + 4) = *reinterpret_cast<const uint4*>(x + 8);
    float f[16];
    unpack16(v, f);
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(f[k]));
    S = block_scale_code(top, s);
    const float rcp = block_rcp(S, s);
#pragma unroll
    for (int k = 0; k < 16; ++k) f[k] = __fmul_rn(f[k], rcp);
    w[0] = e2m1x8(reinterpret_cast<const float(&)[8]>(f[0]));
    w[1] = e2m1x8(reinterpret_cast<const float(&)[8]>(f[8]));
}

__device__ __forceinline__ void decode(const uint32_t (&w)[2], uint32_t code, float s, __nv_bfloat16* y)
{
    const float S = e4m3_value(code);
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 q = e2m1_pair((w[k >> 2] >> (8 * (k & 3))) & 0xFFu);
        o[k] = cvt_bf16x2(f2(q.x * S * s, q.y * S * s));
    }
    *reinterpret_cast<uint4*>(y) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(y + 8) = make_uint4(o[4], o[5], o[6], o[7]);
}

// The 16 bytes that two tokens' values share.
template <int W>
struct Shared16 {
    uint32_t w[4];
    __device__ __forceinline__ void load(const uint8_t* p)
    {
        constexpr int kSecond = W == 64 ? 32 : 8;
        const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(p + kSecond);
        w[0] = a.x, w[1] = a.y, w[2] = b.x, w[3] = b.y;
    }
    __device__ __forceinline__ void store(uint8_t* p) const
    {
        constexpr int kSecond = W == 64 ? 32 : 8;
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(p + kSecond) = make_uint2(w[2], w[3]);
    }
};

template <int W, bool kRead>
__global__ void __launch_bounds__(kThreads) cache_rows_kernel(const __grid_constant__ CacheRowsJob p)
{
    using L = CacheLayout<W>;
    const int lane = threadIdx.x & 31;
    const CacheView& c = p.c;
    griddep_wait();
    const long long warps = (long long)gridDim.x * (kThreads / 32);
    for (long long r = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < p.M; r += warps) {
        const int s = cache_sequence(c, r, lane);
        if (s < 0) continue;
        const long long first = c.row_off ? c.row_off[s] : r, end = c.row_off ? c.row_off[s + 1] : r + 1;
        const long long pos = (long long)c.length[s] - (end - r), len = cache_length(c, s);
        if (pos < 0 || pos >= len) continue;
        uint8_t* base = cache_group<W>(c, s, pos, 0);
        if (!base) continue;
        const int t = (int)(pos % c.page) % kCacheGroup;
        const long long head_bytes = (long long)(c.page / kCacheGroup) * L::kGroupBytes;
        // Two tokens share V's bytes: the row of the first writes both where the call has both, else a
        // row keeps the other token's bits.
        const bool with_next = !(t & 1) && r + 1 < min(end, (long long)p.M) && pos + 1 < len;
        const bool with_last = (t & 1) && r > first && r > 0;
        const int blocks = 2 * c.Hkv * L::kBlocks;  // K's, then V's
        for (int i = lane; i < blocks; i += 32) {
            const bool is_v = i >= blocks / 2;
            const int j = is_v ? i - blocks / 2 : i;
            const int h = j / L::kBlocks, b = j % L::kBlocks;
            uint8_t* g = base + h * head_bytes;
            const HeadsIn& x = is_v ? p.v : p.k;
            const float* gs = is_v ? c.v_gscale : c.k_gscale;
            const float sc = gs ? gs[h] : 1.0f;
            const long long at = r * x.row + (long long)h * x.head + 16 * b;
            const bool real = 16 * b < c.D;
            if constexpr (kRead) {
                if (!real) continue;
                uint32_t w[2];
                if (is_v) {
                    Shared16<W> m;
                    m.load(g + L::v_codes(t, b));
                    const int shift = 4 * (t & 1);
                    w[0] = gather(m.w[0] >> shift) | (gather(m.w[1] >> shift) << 16);
                    w[1] = gather(m.w[2] >> shift) | (gather(m.w[3] >> shift) << 16);
                } else {
                    const uint2 m = *reinterpret_cast<const uint2*>(g + L::k_codes(t, b));
                    w[0] = m.x, w[1] = m.y;
                }
                decode(w, g[is_v ? L::v_scale(t, b) : L::k_scale(t, b)], sc, (is_v ? p.v_out : p.k_out) + at);
            } else {
                if (is_v && with_last) continue;
                uint32_t w[2] = {0, 0}, S = 0;
                if (real) encode(x.p + at, sc, w, S);
                if (!is_v) {
                    *reinterpret_cast<uint2*>(g + L::k_codes(t, b)) = make_uint2(w[0], w[1]);
                    g[L::k_scale(t, b)] = (uint8_t)S;
                    continue;
                }
                Shared16<W> m;
                if (!with_next) m.load(g + L::v_codes(t, b));
                const int shift = 4 * (t & 1);
                const uint32_t keep = 0xF0F0F0F0u >> shift;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t mine = spread(w[k >> 1] >> (16 * (k & 1))) << shift;
                    m.w[k] = with_next ? mine : (m.w[k] & keep) | mine;
                }
                g[L::v_scale(t, b)] = (uint8_t)S;
                if (with_next) {
                    w[0] = w[1] = S = 0;
                    if (real) encode(x.p + at + x.row, sc, w, S);
#pragma unroll
                    for (int k = 0; k < 4; ++k) m.w[k] |= spread(w[k >> 1] >> (16 * (k & 1))) << 4;
                    g[L::v_scale(t + 1, b)] = (uint8_t)S;
                }
                m.store(g + L::v_codes(t, b));
            }
        }
    }
}

template <bool kRead>
cudaError_t launch(const CacheRowsJob& job, cudaStream_t s)
{
    if (job.M == 0) return cudaSuccess;
    const long long blocks = (job.M + kThreads / 32 - 1) / (kThreads / 32);
    const long long most = (long long)sm_count_current_device() * 16;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int w = cache_width(job.c.D);
    if (w == 64) return cudaLaunchKernelEx(&cfg, cache_rows_kernel<64, kRead>, job);
    if (w == 128) return cudaLaunchKernelEx(&cfg, cache_rows_kernel<128, kRead>, job);
    return cudaLaunchKernelEx(&cfg, cache_rows_kernel<256, kRead>, job);
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowsJob& job, cudaStream_t s) { return launch<false>(job, s); }

cudaError_t launch_cache_read(const CacheRowsJob& job, cudaStream_t s) { return launch<true>(job, s); }

}  // namespace h3fp4
