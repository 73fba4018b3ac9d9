// Attention of a few rows of each sequence to a paged cache held in four bits.
//
//     out[r][h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q_r . k_j - m_r),  k = e2m1 * S * s_k, v likewise
//
// What it has to read is the cache, 9/8 bytes per element pair of K and V, each element for
// up to 16 query columns (rows x query heads of a kv head): bound by HBM where the lanes can
// unpack that fast.  An element costs half a conversion (two codes to f16x2), half a
// multiplication by its block scale (exact in f16: six significant bits) and its share of the
// matrix products, about 1 instruction in all; the 47 G (token, head) pairs a second that HBM
// delivers at heads of 128 leave 1.5.
//
// A unit of work is (sequence, kv head, 8 or 16 columns); its keys come in tiles of 128, four
// warps taking 32 each.  All units' tiles are one row of work that is cut evenly over the CTAs,
// from the lengths on the device: the same launch serves any lengths, so it can be captured.
// Every warp has a ring of steps of 32 tokens that bulk copies fill, its own running maximum,
// sum and output; the four are joined at a unit's end.  A unit that was cut leaves partial sums
// in the workspace, which a second kernel joins.  All orders are fixed: the same call gives
// the same bits.
//
// Measured, calls back to back over three caches, of the measured 6793 GB/s: 64 tokens of 64
// sequences over 524288 keys, 32 heads on 8 of 128, 113 us (5340 GB/s; the products, scores and
// unpacking of two thirds of the issue slots beside the loads), one token over 131072 keys
// 35.1 us (4310 GB/s: 3 us until the first keys are there, 4 us for the second kernel), 31 rows
// of 6 sequences over 4433 keys, 28 heads on 4 of 64, 12.2 us (launches and latencies; the
// bytes take 0.2).  Two CTAs of eight warps in place of four of four take 121 us for the first,
// three CTAs an SM 117; shares by the order in which an SM's CTAs issue (the first ended at 86,
// the last at 101 us) change nothing, as the bytes come no faster.
//
// S = Q K^T: m16n8k16; with 16 columns they are the rows of A and the tokens the columns of B,
// with 8 the tokens are A's rows: what a lane unpacks of a token is its fragment either way.
// O = P V: P stays where S was (the accumulator layout is A's, or a transposition away from
// B's), V's bytes hold two tokens as its fragment does.
// Q is scaled per column by a power of two to f16's range (exact for elements within 2^31 of
// the column's largest).  The reference of the exponent follows the true maximum only when
// that passed it by 2^14: p lies in f16's upper range, and those below 2^-30 of the largest
// vanish.  Scores, sums and O are fp32.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "h3fp4_token.h"
#include "kv_cache.cuh"
#include "ptx_sm103.cuh"

namespace h3fp4 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 2 * kCacheGroup;        // tokens that a warp takes at a time
constexpr int kTile = kStep * kWarps;         // tokens of a tile
constexpr int kPartCols = 16;                 // query columns of a unit at most
constexpr uint32_t kSmemOfSm = 228 * 1024;
constexpr int kMaxCtas = 608;                 // of a launch: the workspace is made for as many
constexpr long long kNear = 2;                // tiles that a cut is moved by at most
constexpr float kRaise = 14.0f, kStart = 6.0f;  // in powers of two: see above
// No key yet; and the lowest score that counts: where a column's largest is there, it left fp32's range.
constexpr float kNone = -3.4e38f, kLowest = -3.0e38f;

// What the joining kernel has to know about a unit that was cut, written by the CTA that began it.
struct Cut {
    int first;                // packed row of the unit's sequence's first
    int head, col, cols;      // kv head, the unit's first column and how many
    int cta, count;           // the CTA that began the unit, and of how many CTAs it takes partials (0: not cut)
};

// Partial sums: per CTA one of a unit that began before it, one of a unit that goes on after it.
template <int W>
struct Part {
    static constexpr long long kFloats = kPartCols * (W + 2);
};

constexpr size_t kUnitsOff = 128;   // int: units of the last call
constexpr size_t kCutOff = 256;
constexpr size_t kPartOff = kCutOff + (kMaxCtas * sizeof(Cut) + 255) / 256 * 256;

struct AttnParams {
    CacheView c;
    HeadsIn q;
    __nv_bfloat16* out;
    long long out_row, out_head;
    float* lse;
    long long M;
    int Hq, group, causal, stall;
    int by_unit;          // there are few units: a cut stands at its unit's number, else at its CTA's
    float scale_log2;
    uint8_t* ws;
    unsigned long long wait_ns;
};

// The rows of a sequence and its units.  Row offsets may hold anything: they are kept inside
// the M rows that there are.
struct Seq {
    int first, rows, len;   // packed rows [first, first + rows), tokens that the table has room for
    int start;              // position of the first row
};

__device__ __forceinline__ Seq sequence(const AttnParams& p, int s)
{
    long long a = s, b = s + 1;
    if (p.c.row_off) {
        a = p.c.row_off[s];
        b = p.c.row_off[s + 1];
    }
    const long long n = p.c.length[s], room = p.c.max_pages * p.c.page;
    long long start = n - (b - a);
    if (a < 0) {
        start -= a;
        a = 0;
    }
    b = min(b, p.M);
    Seq q;
    q.first = (int)a;
    q.rows = b > a ? (int)(b - a) : 0;
    q.len = (int)max(0ll, min(n, room));
    q.start = (int)max(start, -(1ll << 30));
    return q;
}

// Units of a kv head, tiles of a unit.
template <int kCols>
__device__ __forceinline__ int col_tiles(const AttnParams& p, const Seq& q)
{
    return (int)(((long long)q.rows * p.group + kCols - 1) / kCols);
}

__device__ __forceinline__ int key_tiles(const Seq& q) { return (int)(((long long)q.len + kTile - 1) / kTile); }

template <int W, int kCols>
struct Config {
    static constexpr int kSlots = W == 64 ? 3 : 2;                     // steps in flight per warp
    static constexpr int kCtasPerSm = W == 256 ? 2 : kCols == 16 ? 3 : 4;
    static constexpr int kMergeRegs = W * kCols / 32 + 4;              // a lane's state: O, two maxima, two sums
    static constexpr uint32_t kSlot = 2 * CacheLayout<W>::kGroupBytes;
    static constexpr uint32_t kRing = kWarps * kSlots * kSlot;
    static constexpr uint32_t kMerge = kWarps / 2 * kMergeRegs * 32 * 4;
    static constexpr uint32_t kBars = kWarps * kSlots * 8;
    static constexpr uint32_t kFixed = kRing + kMerge + kBars;
    static_assert(kFixed % 16 == 0, "the sequences' table behind it");
    // with the tiles before each sequence and the sequences
    static uint32_t smem(int nseq) { return kFixed + (uint32_t)nseq * (sizeof(Seq) + 8) + 8; }
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four bytes of two E2M1 codes each -> four f16x2 (the low code in the low half).
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&o)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}

// Two E4M3 codes -> f16x2 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w)
{
    uint32_t o;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(o) : "r"(w));
    return o;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t o;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
    return o;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t o;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(hi), "f"(lo));
    return o;
}

// The larger one, NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float o;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
    return o;
}

// A column's outputs per unit of O: zero without a key, NaN where the largest score left fp32's range.
__device__ __forceinline__ float norm(float m, float l, float s)
{
    return l == 0.0f ? 0.0f : m < 0.99f * kLowest ? __int_as_float(0x7FFFFFFF) : s / l;
}

__device__ __forceinline__ float log_sum(float m, float l)
{
    return l == 0.0f ? -INFINITY : m < 0.99f * kLowest ? __int_as_float(0x7FFFFFFF) : (m + log2f(l)) * 0.6931471805599453f;
}

// a / b of non-negative values, in 32 bits where they fit (which costs a fifth).
__device__ __forceinline__ long long div(long long a, long long b)
{
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// How the tiles of a call are cut over its CTAs: shares that differ by one at most (shares of the rounded-up mean
// left CTAs idle: one token over 131072 keys 37.3 -> 35.0 us), none empty but where there are fewer tiles.  A second
// unit costs a CTA more than some tiles do (its keys' places, queries and first copies come one after another), so a
// cut up to kNear tiles from a unit's edge is moved there: 31 rows of 6 sequences 14.1 -> 12.2 us, 10 of 5 over 50000
// keys, heads of 64, 17.5 -> 14.8, the batch 113.3 -> 112.1 (and 114.7 with three tiles for two, where shares differ).
struct Shares {
    long long total;
    int ctas;

    // CTA b's first tile, before it is moved
    __device__ __forceinline__ long long raw(int b) const
    {
        return total < ctas ? min(total, (long long)b) : div(total * b, ctas);
    }
    // where the cut before CTA b goes that lies inside a unit from `first` to `last`: of the two cuts around a unit's
    // edge the nearer one is moved
    __device__ __forceinline__ long long moved(int b, long long x, long long first, long long last) const
    {
        const long long up = last - x, down = x - first;
        if (total < ctas || down == 0) return x;
        if (up <= kNear) {
            const long long next = raw(b + 1);
            if (next > last && up <= next - last) return last;
        }
        if (down > kNear) return x;
        const long long before = raw(b - 1);
        return before < first && down < first - before ? first : x;
    }
    // the CTA that has the last tile of a unit
    __device__ __forceinline__ int owner_of_last(long long first, long long last) const
    {
        if (total < ctas) return (int)(last - 1);
        const int c = (int)div(last * ctas + total - 1, total) - 1;
        const long long x = raw(c);
        return x > first && moved(c, x, first, last) == last ? c - 1 : c;
    }
};

// 2^x for an integer x in the normal range.
__device__ __forceinline__ float pow2i(int x) { return __uint_as_float((uint32_t)(x + 127) << 23); }

template <int N>
__device__ __forceinline__ void ld_words(const uint8_t* p, uint32_t (&w)[N])
{
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// The state of a warp over the tokens it has seen, of the lane's two columns: the exponents'
// reference, the lane's part of the sums, and O.
//   16 columns: columns g and g + 8, O[j]: elements n W/8 + j of n = 2 c, 2 c + 1
//    8 columns: columns 2 c and 2 c + 1, O[j]: elements g W/8 + 2 j and the next one
template <int W, int kCols>
struct State {
    static constexpr int kO = kCols == 16 ? W / 8 : W / 16;
    float m[2], l[2];
    float o[kO][4];
};

// Which of the lane's two columns value i of a fragment belongs to.
template <int kCols>
__device__ __forceinline__ constexpr int column_of(int i) { return kCols == 16 ? i >> 1 : i & 1; }

template <int W, int kCols>
__device__ __forceinline__ void rescale(State<W, kCols>& st, int col, float to)
{
    const float f = exp2f(st.m[col] - to);
    st.m[col] = to;
    st.l[col] *= f;
#pragma unroll
    for (int j = 0; j < State<W, kCols>::kO; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (column_of<kCols>(i) == col) st.o[j][i] *= f;
}

// A sum or a maximum over the lanes that share columns.
template <int kCols, class F>
__device__ __forceinline__ float over_lanes(float v, F f)
{
#pragma unroll
    for (int o = kCols == 16 ? 1 : 4; o < (kCols == 16 ? 4 : 32); o <<= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, __half2 b)
{
    const __half2 o = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
    return *reinterpret_cast<const uint32_t*>(&o);
}

// Scores of one group: two of the lane's columns by four tokens (16 columns: tokens 8 half + 2 c + (0, 1),
// 8 columns: tokens g, g + 8, two chains of sums).
template <int W, int kCols>
__device__ __forceinline__ void scores(float (&s)[2][4], const uint8_t* gp, int lane, const uint32_t (&qf)[W / 16][kCols / 4])
{
    using L = CacheLayout<W>;
    uint32_t sc[W == 256 ? 2 : 1];   // the lane's scales of tokens g (low half) and g + 8
    if constexpr (W == 256) ld_words<2>(gp + L::kKScale + lane * 8, sc);
    else if constexpr (W == 128) sc[0] = *reinterpret_cast<const uint32_t*>(gp + L::kKScale + lane * 4);
    else sc[0] = *reinterpret_cast<const uint16_t*>(gp + L::kKScale + lane * 2);
    constexpr int kRuns = W == 256 ? 2 : 1, kWords = W == 64 ? 2 : 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.0f;
#pragma unroll
    for (int run = 0; run < kRuns; ++run) {
        uint32_t w[2][kWords];   // both tokens: codes, their two scales
        __half2 x[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            ld_words<kWords>(W == 64 ? gp + half * 256 + lane * 8 : gp + run * 1024 + half * 512 + lane * 16, w[half]);
            uint32_t pair;
            if constexpr (W == 64) pair = e4m3x2_f16(half ? sc[0] >> 8 : sc[0]);   // (its first half counts)
            else if constexpr (W == 128) pair = e4m3x2_f16(half ? sc[0] >> 16 : sc[0]);
            else pair = e4m3x2_f16(run ? sc[half] >> 16 : sc[half]);
            x[half] = *reinterpret_cast<const __half2*>(&pair);
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            uint32_t f[2][4];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const __half2 by = W == 64 || 2 * i < kWords ? __low2half2(x[half]) : __high2half2(x[half]);
                e2m1x8_f16(w[half][i], f[half]);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[half][j] = mul_half2(f[half][j], by);
            }
            const int step = run * 8 + 2 * i;
            if constexpr (kCols == 16) {
                // Q's 16 columns are A's rows, the tokens B's columns
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    mma_f16(s[half], qf[step], f[half][0], f[half][1]);
                    mma_f16(s[half], qf[step + 1], f[half][2], f[half][3]);
                }
            } else {
                // the tokens are A's rows, Q's 8 columns B's
                const uint32_t a0[4] = {f[0][0], f[1][0], f[0][1], f[1][1]};
                const uint32_t a1[4] = {f[0][2], f[1][2], f[0][3], f[1][3]};
                mma_f16(s[0], a0, qf[step][0], qf[step][1]);
                mma_f16(s[1], a1, qf[step + 1][0], qf[step + 1][1]);
            }
        }
    }
    if constexpr (kCols == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[0][i] += s[1][i];
    }
}

// NaN into the outputs of the columns that see a token whose block of V is NaN, of a group in the pool: of the lane's
// two columns, `lim` tokens of it each.
template <int W, int kCols>
__device__ __forceinline__ void nan_values(State<W, kCols>& st, const uint8_t* gp, int lane, const int (&lim)[2])
{
    constexpr int kRuns = kCols == 16 ? 2 : 1, kVBlocks = W == 256 ? 2 : 1;   // of the lane's elements, of a run
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int run = 0; run < kRuns; ++run)
#pragma unroll
        for (int b = 0; b < kVBlocks; ++b) {
            const int block = ((kCols == 16 ? 2 * c + run : g) * (W / 8) >> 4) + b;
            const uint8_t* scale = gp + CacheLayout<W>::kVScale + block * 16;   // 16 tokens'
            int first = kCacheGroup;                                           // the first that is NaN
#pragma unroll 1
            for (int t = kCacheGroup - 1; t >= 0; --t)
                if ((scale[((t & 7) >> 1) * 4 + (t >> 3) * 2 + (t & 1)] & 0x7Fu) == 0x7Fu) first = t;
#pragma unroll
            for (int j = 0; j < State<W, kCols>::kO; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((kCols == 8 || (i & 1) == run) && (kCols == 16 ? j >> 4 : j >> 3) == b &&
                        first < min(kCacheGroup, lim[column_of<kCols>(i)]))
                        st.o[j][i] = __int_as_float(0x7FFFFFFF);
        }
}

constexpr uint32_t kSawNan = 1u << 31;   // a masked step left out blocks of V that are NaN

// O += P V of one group, token pairs 8 half + 2 c + (0, 1).  kMasked: `left` tokens of it hold anything; blocks that
// are NaN count as zeros and are reported.
template <int W, int kCols, bool kMasked>
__device__ __forceinline__ void values(State<W, kCols>& st, const uint8_t* gp, int lane, const uint32_t (&pf)[kCols / 4], int left,
                                       uint32_t& flags)
{
    using L = CacheLayout<W>;
    const int g = lane >> 2, c = lane & 3;
    constexpr int kVBlocks = W == 256 ? 2 : 1;      // scale blocks of a lane
    uint32_t vs[2][kVBlocks];
#pragma unroll
    for (int b = 0; b < kVBlocks; ++b) {
        const int block = W == 64 ? g >> 1 : W == 128 ? g : 2 * g + b;
        const uint32_t four = *reinterpret_cast<const uint32_t*>(gp + L::kVScale + (block * 4 + c) * 4);
        vs[0][b] = e4m3x2_f16(four);
        vs[1][b] = e4m3x2_f16(four >> 16);
    }
    if (kMasked) {
        // tokens without data: their scales may be anything, NaN too
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int b = 0; b < kVBlocks; ++b) {
                const int t = 8 * half + 2 * c;
                vs[half][b] &= (t < left ? 0xFFFFu : 0u) | (t + 1 < left ? 0xFFFF0000u : 0u);
            }
        // (a product of NaN with a p of zero would be NaN for columns that do not see the token)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int b = 0; b < kVBlocks; ++b) {
                const uint32_t v = vs[half][b] & 0x7FFF7FFFu;
                const uint32_t bad = (v & 0xFFFFu) > 0x7C00u ? 0xFFFFu : 0u, bad2 = v > 0x7C00FFFFu ? 0xFFFF0000u : 0u;
                if (bad | bad2) flags |= kSawNan;
                vs[half][b] &= ~(bad | bad2);
            }
    }
    uint32_t w[2][4 * kVBlocks];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if constexpr (W == 64) {
            uint32_t two[2];
            ld_words<2>(gp + L::kV + half * 256 + lane * 8, two);
            w[half][0] = two[0], w[half][1] = two[1];
        } else {
#pragma unroll
            for (int b = 0; b < kVBlocks; ++b)
                ld_words<4>(gp + L::kV + half * (8 * W / 2) + b * 512 + lane * 16, reinterpret_cast<uint32_t(&)[4]>(w[half][4 * b]));
        }
    }
#pragma unroll
    for (int i = 0; i < W / 32; ++i) {
        uint32_t f[2][4];   // elements 4 i .. 4 i + 3
        const int blk = i >> 2;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            e2m1x8_f16(w[half][i], f[half]);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[half][j] = mul_f16x2(f[half][j], vs[half][blk]);
        }
        if constexpr (kCols == 16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_f16(st.o[4 * i + j], pf, f[0][j], f[1][j]);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t a[4] = {f[0][2 * j], f[0][2 * j + 1], f[1][2 * j], f[1][2 * j + 1]};
                mma_f16(st.o[2 * i + j], a, pf[0], pf[1]);
            }
        }
    }
}

// Two groups of 16 tokens.  kMasked: of group e `left[e]` tokens hold anything and `lim[e]` are
// attended to by the lane's two columns; scores that leave fp32's range downwards stay finite.
template <int W, int kCols, bool kMasked>
__device__ __forceinline__ void step(State<W, kCols>& st, const uint8_t* gp, int lane, const uint32_t (&qf)[W / 16][kCols / 4],
                                     const float (&factor)[2], const int (&left)[2], const int (&lim)[2][2],
                                     uint32_t& flags)
{
    constexpr int kF = kCols / 8;   // fragments of four scores a group
    const int g = lane >> 2, c = lane & 3;
    float s[2][2][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) scores<W, kCols>(s[e], gp + e * CacheLayout<W>::kGroupBytes, lane, qf);
    float top[2] = {kNone, kNone};
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int h = 0; h < kF; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = column_of<kCols>(i);
                float& v = s[e][h][i];
                v *= factor[col];
                if (kMasked) {
                    const int token = kCols == 16 ? 8 * h + 2 * c + (i & 1) : g + 8 * (i >> 1);
                    v = token < lim[e][col] ? max_nan(v, kLowest) : -INFINITY;
                }
            }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int h = 0; h < kF; ++h)
#pragma unroll
            for (int col = 0; col < 2; ++col)
                top[col] = max3(top[col], s[e][h][kCols == 16 ? 2 * col : col], s[e][h][kCols == 16 ? 2 * col + 1 : 2 + col]);
    if (__any_sync(0xffffffffu, top[0] > st.m[0] + kRaise || top[1] > st.m[1] + kRaise)) {
#pragma unroll
        for (int col = 0; col < 2; ++col) {
            const float t = over_lanes<kCols>(top[col], [](float a, float b) { return fmaxf(a, b); });
            if (t > st.m[col] + kRaise) rescale<W, kCols>(st, col, t - kStart);
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint32_t pf[kCols / 4];   // P as the second product's A (16 columns) or, transposed, its B
#pragma unroll
        for (int h = 0; h < kF; ++h) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = column_of<kCols>(i);
                x[i] = ex2_approx_ftz(s[e][h][i] - st.m[col]);
                st.l[col] += x[i];
            }
            pf[2 * h] = pack_f16x2(x[0], x[1]);
            pf[2 * h + 1] = pack_f16x2(x[2], x[3]);
        }
        if constexpr (kCols == 8) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(pf[h]));
        }
        values<W, kCols, kMasked>(st, gp + e * CacheLayout<W>::kGroupBytes, lane, pf, left[e], flags);
    }
}

// The larger reference of two states, and what their sums are scaled with.
__device__ __forceinline__ void join_scale(float a, float b, float& m, float& fa, float& fb)
{
    m = fmaxf(a, b);
    fa = exp2f(a - m);
    fb = exp2f(b - m);
}

template <int W, int kCols>
__global__ void __launch_bounds__(kThreads, Config<W, kCols>::kCtasPerSm)
    cache_attn_kernel(const __grid_constant__ AttnParams p)
{
    using L = CacheLayout<W>;
    using C = Config<W, kCols>;
    using S = State<W, kCols>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + warp * (C::kSlots * C::kSlot);
    float* merge = reinterpret_cast<float*>(smem + C::kRing);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kRing + C::kMerge) + warp * C::kSlots;
    const int nseq = p.c.nseq;
    Seq* seqs = reinterpret_cast<Seq*>(smem + C::kFixed);
    long long* prefix = reinterpret_cast<long long*>(seqs + nseq);
    __shared__ long long warp_sum[kWarps];
    unsigned int* status = reinterpret_cast<unsigned int*>(p.ws);
    if (lane == 0) {
        for (int i = 0; i < C::kSlots; ++i) mbar_init(&bars[i], 1);
        fence_mbarrier_init();
    }
    griddep_wait();
    griddep_launch_dependents();

    // ------------------------------------------------------------ tiles before each sequence
    {
        // each thread's run of sequences
        const int per = (nseq + kThreads - 1) / kThreads, s0 = min(nseq, (int)threadIdx.x * per), s1 = min(nseq, s0 + per);
        auto tiles = [&](const Seq& q) { return (long long)p.c.Hkv * col_tiles<kCols>(p, q) * key_tiles(q); };
        long long mine = 0;
#pragma unroll 4
        for (int s = s0; s < s1; ++s) {
            const Seq q = sequence(p, s);
            seqs[s] = q;
            mine += tiles(q);
        }
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) warp_sum[warp] = upto;
        __syncthreads();
        for (int w = 0; w < warp; ++w) upto += warp_sum[w];
        long long before = upto - mine;
        for (int s = s0; s < s1; ++s) {
            prefix[s] = before;
            before += tiles(seqs[s]);
        }
        if (threadIdx.x == kThreads - 1) prefix[nseq] = upto;
        __syncthreads();
    }
    const long long total = prefix[nseq];
    const Shares shares{total, (int)gridDim.x};
    // the sequence whose tiles hold x < total (the last one that begins there or before), by a warp: in steps of 32
    auto holder = [&](long long x) {
        int lo = 0, each = 1;
        while (each * 32 < nseq) each *= 32;
        for (; each > 0; each /= 32) {
            const int i = lo + lane * each;
            lo += (__popc(__ballot_sync(0xffffffffu, i < nseq && prefix[i] <= x)) - 1) * each;
        }
        return lo;
    };
    // this CTA's tiles: two warps look for their ends
    __shared__ long long ends[2];
    if (warp < 2) {
        const int b = blockIdx.x + warp;
        long long x = shares.raw(b);
        if (x < total) {
            const int s = holder(x), tiles = key_tiles(seqs[s]);
            const long long first = prefix[s] + div(x - prefix[s], tiles) * tiles;
            x = shares.moved(b, x, first, first + tiles);
        }
        if (lane == 0) ends[warp] = x;
    }
    __syncthreads();
    const long long begin = ends[0], end = ends[1];

    // rows of sequences that hold nothing
    for (int s = blockIdx.x; s < nseq; s += gridDim.x) {
        const Seq q = seqs[s];
        if (q.len > 0) continue;
        const int vecs = p.c.D / 8;
        const long long of_row = (long long)p.Hq * vecs;   // (past 32 bits from 2^26 heads of 256 on)
        for (long long i = threadIdx.x; i < q.rows * of_row; i += kThreads) {
            const long long r = q.first + i / of_row;
            const int h = (int)(i / vecs % p.Hq), v = (int)(i % vecs);
            *reinterpret_cast<uint4*>(p.out + r * p.out_row + (long long)h * p.out_head + 8 * v) = make_uint4(0, 0, 0, 0);
            if (p.lse && v == 0) p.lse[r * p.Hq + h] = -INFINITY;
        }
    }
    // Cuts.  By unit: units in the order of their sequences, empty ones have no number.
    Cut* cuts = reinterpret_cast<Cut*>(p.ws + kCutOff);
    auto units_before = [&](int s) {   // by a warp
        int n = 0;
        for (int i = lane; i < s; i += 32)
            n += seqs[i].len > 0 ? (int)min((long long)kMaxCtas, (long long)p.c.Hkv * col_tiles<kCols>(p, seqs[i])) : 0;
        return __reduce_add_sync(0xffffffffu, n);   // (more than there can be where row offsets overlap)
    };
    if (warp == 0) {
        const int units = p.by_unit && blockIdx.x == 0 ? units_before(nseq) : 0;
        if (lane == 0) {
            if (!p.by_unit) cuts[blockIdx.x].count = 0;
            else if (blockIdx.x == 0) *reinterpret_cast<int*>(p.ws + kUnitsOff) = min(kMaxCtas, units);
        }
    }

    // ------------------------------------------------------------ units
    uint32_t phases = 0;    // of the ring's barriers, one bit each
    bool lost = false;      // a wait ran out: nothing more is loaded or computed
    const int per_page = p.c.page / kCacheGroup;
    // Of short units, of which this CTA has four and more whole ones, each warp takes some by itself (`solo`): their
    // latencies, one after another, are what they cost (1024 sequences of 64 keys 159 -> 57 us).  Units of eight columns
    // only: with 16 the registers that this takes cost more (10 % of 256 rows over 262144 keys).
    constexpr bool kSolo = kCols == 8;
    long long run_end = begin, next = begin;   // of a run of such units, and the warp's next one
    for (long long at = begin; at < end;) {
        const bool solo = kSolo && at < run_end;
        if (solo && next >= run_end) {
            at = run_end;
            continue;
        }
        const long long here = solo ? next : at;
        const int s = holder(here);
        const Seq q = seqs[s];
        const int coltiles = col_tiles<kCols>(p, q), tiles = key_tiles(q);
        const long long unit = div(here - prefix[s], tiles);
        if (kSolo && !solo && here == prefix[s] + unit * tiles && (long long)kWarps * tiles <= end - here) {
            int to = s;   // sequences of as many tiles
            while (to + 1 < nseq && prefix[to + 1] < end && key_tiles(seqs[to + 1]) == tiles) ++to;
            const long long units = div(min(end, prefix[to + 1]) - here, tiles);
            if (units >= kWarps) {
                run_end = here + units * tiles;
                next = here + (long long)warp * tiles;
                continue;
            }
        }
        if (solo) next += (long long)kWarps * tiles;
        const int h = (int)div(unit, coltiles), ct = (int)(unit - (long long)h * coltiles);
        const long long ubegin = prefix[s] + unit * tiles, uend = ubegin + tiles;
        const int t0 = (int)(here - ubegin), t1 = (int)(min(end, uend) - ubegin);
        const bool begins = here == ubegin, whole = begins && uend <= end;
        // what each column attends to
        // (rows times heads of a call are below 2^31)
        const int cols = min(kCols, q.rows * p.group - ct * kCols);
        auto limit = [&](int col) { return p.causal ? max(0, min(q.len, q.start + (ct * kCols + col) / p.group + 1)) : q.len; };
        // the lane's two columns
        int mycol[2], mylim[2];
        const int least = limit(0), most = limit(cols - 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mycol[i] = kCols == 16 ? g + 8 * i : 2 * c + i;
            mylim[i] = mycol[i] < cols ? limit(mycol[i]) : most;
        }

        // Q: the lane's elements of columns g (and g + 8)
        uint2 raw[kCols / 8][W / 16];
#pragma unroll
        for (int half = 0; half < kCols / 8; ++half) {
            const int col = g + 8 * half, id = ct * kCols + col;
            const __nv_bfloat16* src = nullptr;
            if (col < cols)
                src = p.q.p + (long long)(q.first + id / p.group) * p.q.row + (long long)(h * p.group + id % p.group) * p.q.head;
#pragma unroll
            for (int t = 0; t < W / 16; ++t) {
                const int d = W == 64 ? 16 * c + 4 * t : (t >> 3) * 128 + 32 * c + 4 * (t & 7);
                raw[half][t] = make_uint2(0, 0);
                if (src && d < p.c.D) raw[half][t] = *reinterpret_cast<const uint2*>(src + d);
            }
        }
        const float kg = p.c.k_gscale ? p.c.k_gscale[h] : 1.0f, vg = p.c.v_gscale ? p.c.v_gscale[h] : 1.0f;

        // this warp's steps of 32 tokens: tile t's is 4 t + warp, up to the last token that any column sees
        const int steps = most > 0 ? (most - 1) / kStep + 1 : 0;
        const int every = solo ? 1 : kWarps, g0 = solo ? 0 : kWarps * t0 + warp;   // the first, and the stride
        int n = 0;
        if (solo) n = steps;
        else if (steps > g0) n = min(t1 - t0, (steps - g0 + kWarps - 1) / kWarps);
        const int32_t* table = p.c.table + (long long)s * p.c.max_pages;
        // where the groups of the next 16 steps lie, one per lane, and which of them the pool has
        const uint8_t* where = nullptr;
        uint32_t has = 0;
        auto look = [&](int i) {
            const int gi = 2 * (g0 + every * (i + (lane >> 1))) + (lane & 1);
            int pg = -1;
            if ((uint32_t)gi * kCacheGroup < (uint32_t)most) pg = table[gi / per_page];
            const bool ok = pg >= 0 && pg < p.c.n_pages;
            if (ok) where = p.c.pool + (((long long)pg * p.c.Hkv + h) * per_page + gi % per_page) * L::kGroupBytes;
            has = __ballot_sync(0xffffffffu, ok);
        };
        uint32_t there = 0;   // which groups of the slots exist, two bits each, and kSawNan
        auto load = [&](int i, int slot) {
            if ((i & 15) == 0) look(i);
            const int first = 2 * (i & 15);
            const uint32_t two = (has >> first) & 3u;
            there = (there & ~(3u << (2 * slot))) | (two << (2 * slot));
            if (lane - first == 0 || lane - first == 1) {
                // (a copy may end before its bytes are expected: the arrival holds the phase open)
                if (p.stall) return;
                if (lane == first) {
                    if (two) mbar_arrive_expect_tx(&bars[slot], __popc(two) * L::kGroupBytes);
                    else mbar_arrive(&bars[slot]);
                }
                if ((two >> (lane - first)) & 1u)
                    bulk_load(ring + slot * C::kSlot + (lane - first) * L::kGroupBytes, where, L::kGroupBytes, &bars[slot]);
            }
        };
        int loaded = 0;
        if (lost) n = 0;
        for (; loaded < min(n, C::kSlots); ++loaded) load(loaded, loaded);

        // ... scaled to f16's range
        uint32_t qf[W / 16][kCols / 4];
        float factor[2], mine[kCols / 8];
#pragma unroll
        for (int half = 0; half < kCols / 8; ++half) {
            uint32_t top = 0;
#pragma unroll
            for (int t = 0; t < W / 16; ++t)
                top = max(top, max(max(raw[half][t].x & 0x7FFFu, (raw[half][t].x >> 16) & 0x7FFFu),
                                   max(raw[half][t].y & 0x7FFFu, (raw[half][t].y >> 16) & 0x7FFFu)));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the largest to [2^14, 2^15), by a power of two in the normal range
            const int e = min(126, max(-126, 14 - ((int)(top >> 7) - 127)));
            const float up = pow2i(e);
            mine[half] = p.scale_log2 * kg * pow2i(-e);
#pragma unroll
            for (int t = 0; t < W / 16; ++t) {
                auto f16 = [&](uint32_t w) {
                    return pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
                };
                qf[t][kCols == 16 ? half : 0] = f16(raw[half][t].x);
                qf[t][kCols == 16 ? 2 + half : 1] = f16(raw[half][t].y);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            factor[i] = kCols == 16 ? mine[i % (kCols / 8)] : __shfl_sync(0xffffffffu, mine[0], 4 * (2 * c + i));

        S st;
        st.m[0] = st.m[1] = kNone;
        st.l[0] = st.l[1] = 0.0f;
#pragma unroll
        for (int j = 0; j < S::kO; ++j) st.o[j][0] = st.o[j][1] = st.o[j][2] = st.o[j][3] = 0.0f;
        // steps that all columns see whole, with scores that cannot leave fp32's range (a raw one is below 2^36)
        const bool tame = __all_sync(0xffffffffu, fabsf(factor[0]) < 1e26f && fabsf(factor[1]) < 1e26f);
        const int whole_steps = max(0, least / kStep - g0);
        const int plain = tame ? min(n, solo ? whole_steps : (whole_steps + kWarps - 1) / kWarps) : 0;
        int slot = 0;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            {
                const bool ok = mbar_wait(&bars[slot], (phases >> slot) & 1u, p.wait_ns, status, kStatusTimeoutMma);
                if (!__all_sync(0xffffffffu, ok)) {
                    lost = true;
                    // copies in flight land before the CTA may end
                    if (!p.stall)
                        for (int k = i; k < loaded; ++k) {
                            (void)mbar_wait(&bars[slot], (phases >> slot) & 1u, p.wait_ns, status, kStatusTimeoutMma);
                            slot = slot + 1 == C::kSlots ? 0 : slot + 1;
                        }
                    break;
                }
                phases ^= 1u << slot;
                const uint32_t two = (there >> (2 * slot)) & 3u;
                const uint8_t* gp = ring + slot * C::kSlot;
                if (i < plain && two == 3u) {
                    const int left[2] = {kCacheGroup, kCacheGroup}, lim[2][2] = {};
                    step<W, kCols, false>(st, gp, lane, qf, factor, left, lim, there);
                } else if (two) {
                    const int first = (g0 + every * i) * kStep;
                    int left[2], lim[2][2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool here = (two >> e) & 1u;
                        left[e] = here ? most - first - e * kCacheGroup : 0;
                        lim[e][0] = here ? mylim[0] - first - e * kCacheGroup : 0;
                        lim[e][1] = here ? mylim[1] - first - e * kCacheGroup : 0;
                    }
                    step<W, kCols, true>(st, gp, lane, qf, factor, left, lim, there);
                }
                // (the products that used the slot's last bytes have been issued, so these were read)
                __syncwarp();
                if (loaded < n) {
                    load(loaded, slot);
                    ++loaded;
                }
                slot = slot + 1 == C::kSlots ? 0 : slot + 1;
            }
        }
        __syncwarp();
        // blocks of V that are NaN, for the columns that see their tokens (looked for again in the pool: hardly ever)
        if (__any_sync(0xffffffffu, (there & kSawNan) != 0))
#pragma unroll 1
            for (int k = 0; k < 2 * n; ++k) {
                const int gi = 2 * (g0 + every * (k >> 1)) + (k & 1);
                const int pg = (uint32_t)gi * kCacheGroup < (uint32_t)most ? table[gi / per_page] : -1;
                if (pg < 0 || pg >= p.c.n_pages) continue;
                const int lim[2] = {mylim[0] - gi * kCacheGroup, mylim[1] - gi * kCacheGroup};
                nan_values<W, kCols>(st, p.c.pool + (((long long)pg * p.c.Hkv + h) * per_page + gi % per_page) * L::kGroupBytes,
                                     lane, lim);
            }

        // ------------------------------------------------------------ the warps' sums into warp 0
#pragma unroll
        for (int i = 0; i < 2; ++i) st.l[i] = over_lanes<kCols>(st.l[i], [](float a, float b) { return a + b; });
#pragma unroll
        for (int with = solo ? 0 : kWarps / 2; with >= 1; with >>= 1) {
            float* other = merge + (warp & (with - 1)) * (C::kMergeRegs * 32) + lane;
            __syncthreads();
            if (warp >= with && warp < 2 * with) {
                other[0] = st.m[0], other[32] = st.m[1], other[64] = st.l[0], other[96] = st.l[1];
#pragma unroll
                for (int j = 0; j < 4 * S::kO; ++j) other[32 * (4 + j)] = st.o[j >> 2][j & 3];
            }
            __syncthreads();
            if (warp < with) {
                float fa[2], fb[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float m;
                    join_scale(st.m[i], other[32 * i], m, fa[i], fb[i]);
                    st.m[i] = m;
                    st.l[i] = st.l[i] * fa[i] + other[32 * (2 + i)] * fb[i];
                }
#pragma unroll
                for (int j = 0; j < 4 * S::kO; ++j) {
                    const int col = column_of<kCols>(j & 3);
                    st.o[j >> 2][j & 3] = st.o[j >> 2][j & 3] * fa[col] + other[32 * (4 + j)] * fb[col];
                }
            }
        }
        if (warp == 0 || solo) {
            float* part = reinterpret_cast<float*>(p.ws + kPartOff) + (2ll * blockIdx.x + (begins ? 1 : 0)) * Part<W>::kFloats;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = mycol[i];
                const int id = ct * kCols + col;
                const long long r = q.first + id / p.group;
                const int hq = h * p.group + id % p.group;
                // the lane's elements of the column in runs of W/8
                constexpr int kRuns = kCols == 16 ? 2 : 1;
#pragma unroll
                for (int e = 0; e < kRuns; ++e) {
                    auto value = [&](int j) { return kCols == 16 ? st.o[j][2 * i + e] : st.o[j >> 1][2 * (j & 1) + i]; };
                    const int d = (kCols == 16 ? 2 * c + e : g) * (W / 8);
                    if (whole) {
                        if (col >= cols) continue;
                        const float f = norm(st.m[i], st.l[i], vg);
                        __nv_bfloat16* o = p.out + r * p.out_row + (long long)hq * p.out_head + d;
#pragma unroll
                        for (int j = 0; j < W / 8; j += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = cvt_bf16x2(f2(value(j + 2 * k) * f, value(j + 2 * k + 1) * f));
                            if (d + j < p.c.D) *reinterpret_cast<uint4*>(o + j) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        float* o = part + 2 * kPartCols + col * W + d;
#pragma unroll
                        for (int j = 0; j < W / 8; j += 4)
                            *reinterpret_cast<float4*>(o + j) = make_float4(value(j), value(j + 1), value(j + 2), value(j + 3));
                    }
                }
                if (kCols == 16 ? c == 0 : g == 0) {
                    if (!whole) {
                        part[2 * col] = st.m[i];
                        part[2 * col + 1] = st.l[i];
                    } else if (p.lse && col < cols) {
                        p.lse[r * p.Hq + hq] = log_sum(st.m[i], st.l[i]);
                    }
                }
            }
            if (begins && (p.by_unit || !whole)) {
                const long long i = p.by_unit ? units_before(s) + unit : blockIdx.x;
                const int count = whole ? 0 : shares.owner_of_last(ubegin, uend) - (int)blockIdx.x + 1;
                // (row offsets that overlap make more units than there can be)
                if (lane == 0 && i < kMaxCtas) cuts[i] = Cut{q.first, h, ct * kCols, cols, (int)blockIdx.x, count};
            }
        }
        if (!solo) at = ubegin + t1;
    }
}

// Columns of a unit that was cut: block (cut, columns).  Latency counts: the
// cut, then references, sums and O of the partials together.
constexpr int kJoinThreads = 512;

template <int W, int kSplit>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int kLanes = W / 4;                  // threads of a partial, four elements each; kSplit partials at a time
    constexpr int kJoinCols = kJoinThreads / (kLanes * kSplit);
    constexpr int kBatch = 4;                      // and of a thread in flight
    __shared__ float weight[kJoinCols][kMaxCtas];
    __shared__ float4 sum[kJoinThreads];
    __shared__ float red[2][kJoinThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    // (both loads in flight; a cut past the units' is not looked at)
    const int units = p.by_unit ? *reinterpret_cast<const volatile int*>(p.ws + kUnitsOff) : kMaxCtas;
    const Cut cut = reinterpret_cast<const Cut*>(p.ws + kCutOff)[blockIdx.x];
    if ((int)blockIdx.x >= units || cut.count == 0 || (int)blockIdx.y * kJoinCols >= cut.cols) return;
    const float vg = p.c.v_gscale ? __ldg(p.c.v_gscale + cut.head) : 1.0f;
    const int t = threadIdx.x, lane = t & 31, mine = t / (kLanes * kSplit), split = t / kLanes % kSplit;
    const int col = min((int)blockIdx.y * kJoinCols + mine, kPartCols - 1);   // (columns past the last are not written)
    // partial 0 is its CTA's second, the others are the first ones
    const float* parts = reinterpret_cast<const float*>(p.ws + kPartOff) + (2ll * cut.cta + 1) * Part<W>::kFloats;
    auto part = [&](int i) { return parts + (i == 0 ? 0 : 2 * i - 1) * Part<W>::kFloats; };
    const int at = 2 * kPartCols + col * W + 4 * (t % kLanes);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v[kBatch];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * kSplit;
            v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < cut.count) v[k] = *reinterpret_cast<const float4*>(part(i) + at);
        }
    };
    load(split);
    // references and sums: a partial per thread of the column, all in flight at once
    constexpr int kThreadsOfCol = kLanes * kSplit, kWarpsOfCol = kThreadsOfCol / 32;
    constexpr int kMine = (kMaxCtas + kThreadsOfCol - 1) / kThreadsOfCol;
    float2 ml[kMine];
    float m = kNone, l = 0.0f;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        const int i = t % kThreadsOfCol + k * kThreadsOfCol;
        ml[k] = make_float2(kNone, 0.0f);
        if (i < cut.count) ml[k] = *reinterpret_cast<const float2*>(part(i) + 2 * col);
    }
#pragma unroll
    for (int k = 0; k < kMine; ++k) m = fmaxf(m, ml[k].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int warp0 = mine * kWarpsOfCol;
    if (lane == 0) red[0][t >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarpsOfCol; ++w) m = fmaxf(m, red[0][warp0 + w]);
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        const int i = t % kThreadsOfCol + k * kThreadsOfCol;
        const float w = exp2f(ml[k].x - m);
        if (i < cut.count) weight[mine][i] = w;
        l += ml[k].y * w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) red[1][t >> 5] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarpsOfCol; ++w) l += red[1][warp0 + w];
    for (int i0 = split; i0 < cut.count; i0 += kBatch * kSplit) {
        if (i0 >= kBatch * kSplit) load(i0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * kSplit;
            const float f = i < cut.count ? weight[mine][i] : 0.0f;
            acc.x = fmaf(v[k].x, f, acc.x), acc.y = fmaf(v[k].y, f, acc.y);
            acc.z = fmaf(v[k].z, f, acc.z), acc.w = fmaf(v[k].w, f, acc.w);
        }
    }
    sum[t] = acc;
    __syncthreads();
    if (split > 0 || (int)blockIdx.y * kJoinCols + mine >= cut.cols) return;
#pragma unroll
    for (int i = 1; i < kSplit; ++i) {
        const float4 x = sum[t + i * kLanes];
        acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
    }
    const int id = cut.col + col, d = 4 * (t % kLanes);
    const long long r = (long long)cut.first + id / p.group;
    const int hq = cut.head * p.group + id % p.group;
    const float f = norm(m, l, vg);
    if (d < p.c.D)
        *reinterpret_cast<uint2*>(p.out + r * p.out_row + (long long)hq * p.out_head + d) =
            make_uint2(cvt_bf16x2(f2(acc.x * f, acc.y * f)), cvt_bf16x2(f2(acc.z * f, acc.w * f)));
    if (p.lse && d == 0) p.lse[r * p.Hq + hq] = log_sum(m, l);
}

template <int W, int kCols>
cudaError_t launch(AttnParams p, cudaStream_t s)
{
    // at most: a sequence's columns fill all but one of its units
    const long long units = p.c.Hkv * (p.c.nseq + p.M * p.group / kCols);
    p.by_unit = units <= kMaxCtas;
    using C = Config<W, kCols>;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(cache_attn_kernel<W, kCols>), (int)C::smem(kCacheMaxSeqs));
    if (e != cudaSuccess) return e;
    // as many as an SM holds beside a table of so many sequences (a second wave of CTAs would take as long again)
    const int held = std::max(1, std::min(C::kCtasPerSm, (int)(kSmemOfSm / (C::smem(p.c.nseq) + 1024))));
    int ctas = sm_count_current_device() * held;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::smem(p.c.nseq);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t first = cudaLaunchKernelEx(&cfg, cache_attn_kernel<W, kCols>, p);
    if (first != cudaSuccess) return first;
    // Few units, so that each was cut into many: their partials by many threads, a block per unit and column
    // (8 units of 76 partials: 3.5 us of the call against 7 with four partials at a time).
    constexpr int kMany = W == 64 ? 32 : W == 128 ? 16 : 8;
    constexpr int few_cols = kJoinThreads / (W / 4 * kMany), cols = kJoinThreads / W;
    static_assert(few_cols >= 1, "a column at least");
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    auto join = [&](const cudaLaunchConfig_t& cfg, void (*kernel)(AttnParams)) {
        const cudaError_t e = ensure_shared_carveout(reinterpret_cast<const void*>(kernel));
        return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kernel, p) : e;
    };
    if (p.by_unit && 16 * units <= ctas) {
        cfg.gridDim = dim3((unsigned)units, (kCols + few_cols - 1) / few_cols);
        return join(cfg, cache_join_kernel<W, kMany>);
    }
    cfg.gridDim = dim3((unsigned)(p.by_unit ? units : ctas), (kCols + cols - 1) / cols);
    return join(cfg, cache_join_kernel<W, 4>);
}

}  // namespace

size_t cache_attn_workspace_bytes(int D)
{
    const int w = cache_width(D);
    return kPartOff + 2 * kMaxCtas * sizeof(float) * (w == 64 ? Part<64>::kFloats : w == 128 ? Part<128>::kFloats : Part<256>::kFloats);
}

cudaError_t launch_cache_attn(const CacheAttnJob& job, cudaStream_t s)
{
    if (job.M == 0) return cudaSuccess;
    AttnParams p{};
    p.c = job.c;
    p.q = job.q;
    p.out = job.out;
    p.out_row = job.out_row;
    p.out_head = job.out_head;
    p.lse = job.lse;
    p.M = job.M;
    p.Hq = job.Hq;
    p.group = job.Hq / job.c.Hkv;
    p.causal = job.causal;
    p.stall = job.stall;
    p.scale_log2 = job.scale * kLog2E;
    p.ws = job.ws;
    p.wait_ns = job.wait_limit_ns;
    const int w = cache_width(job.c.D);
    // Eight columns a unit where a sequence has no more on average (its rows times the heads of a kv head):
    // half the products, scores and registers.  Either is right for any rows.
    const bool narrow = (p.M + p.c.nseq - 1) / p.c.nseq * p.group <= 8;
    if (w == 64) return narrow ? launch<64, 8>(p, s) : launch<64, 16>(p, s);
    if (w == 128) return narrow ? launch<128, 8>(p, s) : launch<128, 16>(p, s);
    return narrow ? launch<256, 8>(p, s) : launch<256, 16>(p, s);
}

}  // namespace h3fp4
