// The linear of a few rows over NVFP4 weights, activations as they are (bf16).
//
//     out[m][n] = bf16( R[m][n] + g[m][n] * (s_w * sum_k x[m][k] W[n][k] + b[n]) )
//
// or the SwiGLU of gate and up rows.  It has to read the weights, 9/16 byte an element: bound by
// HBM as long as nothing on the way needs an instruction per element.  So the weights go from
// memory to the FP4 matrix unit as they are (TMA, tcgen05.mma.kind::mxf4nvf4; W's rows are the
// 128 rows of A), and x comes to them: each row is written as the sum of kDigits = 8 rows of
// E2M1 digits in base 8,
//     x[k] = 2^(e_b) sum_t d_t[k] 8^-t,   |d_t| <= 4,  d_t = e2m1(what is left, in units of 8^-t),
// e_b the exponent of x's block of 16.  Up to 4, E2M1's steps are at most 1, so what is left
// shrinks by 8 each time: eight digits are exact for elements within 2^-16 of their block's
// largest and within 2^-23 of it otherwise.  All digits of a block share its scale
// 2^(e_b - e_row + 8), a power of two that E4M3 holds for 17 binades (blocks further below are
// held to 2^-40 of the row's largest); e_row is the row's.  The matrix unit multiplies 8 M <=
// 256 digit rows by each W tile in the time that the tile takes to arrive (M = 32: 128 of 199
// cycles); more than 32 rows take two passes over the tile, the second from L2.  The products
// and the sums of 16 are exact, the accumulators fp32.
//
// Two forms, by size (few_split).  One kernel, up to eight rows where a wave of CTAs has all
// tiles of W: rows_few_kernel, digits beside the products, a tile's CTAs joined in a cluster.
// Else three: digits_kernel writes the digits, their scales and the rows' factors;
// rows_gemm_kernel multiplies.  Its work is one row of (W tile, pass, 256-column K stage), cut
// evenly over one CTA per SM, and the sums of each (tile, CTA) piece go to the workspace;
// rows_join_kernel adds the pieces of a tile in order and finishes the outputs.  Each starts
// while the one before it drains; the first W tiles are on their way before the digits are
// there.  The same call gives the same bits.
//
// Measured, calls back to back over three sets of weights, of the measured 6793 GB/s:
//     rows  W               us     GB/s     bound by
//        1  9216 x 3072     6.3    2530     a launch, its start, one load's latency and the join (4.7 us of 2048 x 2048)
//        1  4096 x 14336    8.8    3760     the same, and the clusters' uneven stages
//        1  57344 x 8192    47.2   5600     HBM, and 3 kernels' ends (about 6 us)
//       16  4096 x 14336    12.5   2660     digits and joining, 7 us of them
//       16  57344 x 8192    50.9   5190     HBM
//       32  57344 x 8192    61.1   4330     a stage's way through the ring of four: 54 KB, of them 32 KB digits
//       64  57344 x 8192    108    2440     the same, two passes
// What was built and measured and is not here: whoever brings a tile's last piece joins it, in
// place of the third kernel (16 rows of 4096 x 14336 20 us against 13: few threads have all the
// pieces to read); the digits of one row beside the products of the three-kernel form (gains
// nothing once a row's loads were in flight together); pairs of CTAs that share the digits of
// more than 16 rows (64 rows of 57344 x 8192 101 us, but 61 rows of 6152 x 4160 13.8 against
// 13.4 and 4096 x 4096 12.2 against 11.2).
#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cuda_bf16.h>

#include "act_prologue.cuh"
#include "h3fp4_token.h"
#include "nvfp4_encode.cuh"
#include "ptx_sm103.cuh"
#include "tensor_map.h"

namespace h3fp4 {
namespace {

constexpr int kDigits = 8;
constexpr int kPassRows = 32;                          // rows of x per pass: 256 digit rows
constexpr int BM = 128;                                // rows of W per tile
constexpr int BK = 256;                                // columns per stage
constexpr int kMaxCtas = 160;
constexpr int kThreads = 384;                          // producer, MMA, 2 idle; 4 scale warps; 4 epilogue warps
constexpr uint32_t kWBytes = BM * BK / 2;
constexpr uint32_t kSfwBytes = BM * (BK / 16);
constexpr uint32_t kSfBox = 2048;                      // a stage's scale tiles of 128 rows
constexpr uint32_t kTmemCols = 512;

// Digit rows that a CTA takes at once, and what fits beside them: the ring's stages, the
// accumulators (two where they fit, so that one drains while the other fills), the scales.
template <int NB>
struct Plan {
    static constexpr int kHalves = (NB + 127) / 128;   // scale tiles of the digits
    static constexpr int kStages = NB <= 64 ? 7 : NB <= 128 ? 6 : 4;
    static constexpr int kAccs = NB <= 128 ? 2 : 1;
    static constexpr uint32_t kDBytes = NB * BK / 2;
    static constexpr uint32_t kStage = kWBytes + kDBytes + kSfwBytes + kHalves * kSfBox;
    static constexpr uint32_t kSfTmem = kAccs * NB;
    static constexpr uint32_t kSfCols = 16 + 16 * kHalves;
    static constexpr uint32_t kBarOff = kStages * kStage;
    static constexpr uint32_t kSmem = kBarOff + 8 * (3 * kStages + 2 * kAccs + 1) + 16;
    static_assert(kStage % 1024 == 0, "stages keep the swizzle's alignment");
    static_assert(kSfTmem + kStages * kSfCols <= kTmemCols, "TMEM budget");
    static_assert(kSmem <= 232448, "shared memory budget");
};

// Workspace: status, the rows' factors, digit codes, digit scales, pieces.
struct Layout {
    int passes, pass_rows;    // rows of x per pass, the last may have fewer
    int64_t digit_rows;       // rows of the code matrix: pass p's begin at 256 p
    int64_t tiles, kb4;
    size_t codes, scales, parts, bytes;
};

constexpr size_t kFactors = 256;

inline Layout layout(int64_t M, int64_t N, int64_t K)
{
    Layout l{};
    l.passes = (int)((M + kPassRows - 1) / kPassRows);
    l.pass_rows = (int)((M + l.passes - 1) / l.passes);
    l.digit_rows = 256 * (l.passes - 1) + kDigits * l.pass_rows;
    l.tiles = (N + BM - 1) / BM;
    l.kb4 = K / 64;
    auto round = [](size_t x) { return (x + 255) / 256 * 256; };
    l.codes = round(kFactors + kRowsMax * sizeof(float));
    l.scales = l.codes + round((size_t)l.digit_rows * (size_t)(K / 2));
    l.parts = l.scales + round((size_t)((l.digit_rows + 127) / 128) * (size_t)l.kb4 * 512);
    l.bytes = l.parts + (size_t)(l.tiles * l.passes + kMaxCtas) * l.pass_rows * BM * sizeof(float);
    return l;
}

// 2^x for x in the normal range.
__device__ __forceinline__ float pow2i(int x) { return __uint_as_float((uint32_t)(x + 127) << 23); }

// ------------------------------------------------------------------ digits

constexpr int kDigitThreads = 256;
constexpr int kDigitColumns = kDigitThreads * 8;   // of x per CTA

// The largest magnitude of bf16 pairs, as its bits (they order like the values).
__device__ __forceinline__ uint32_t top_bits(const uint4& v)
{
    auto two = [](uint32_t w) { return max(w & 0x7FFFu, (w >> 16) & 0x7FFFu); };
    return max(max(two(v.x), two(v.y)), max(two(v.z), two(v.w)));
}

// The exponent of the digits' unit where the largest magnitude is `top`: it lies in [2, 4) of them.
__device__ __forceinline__ int unit_of(uint32_t top) { return max(1, (int)(top >> 7)) - 127 - 1; }

// 2^(e_row - 8), what the sums of a row's digits are in (either factor may be subnormal together); NaN where the
// row holds an infinity or a NaN, which digits cannot say.
__device__ __forceinline__ float row_factor(uint32_t top)
{
    if (top >= 0x7F80u) return __int_as_float(0x7FFFFFFF);
    const int e_row = unit_of(top);
    return pow2i(e_row / 2) * pow2i(e_row - e_row / 2 - 8);
}

// y s f of a row's sum of digits y, the weight's global scale s and the row's factor f.  The two scales may lie at
// opposite ends of the range: y (below 2^40) meets first whichever keeps it inside, so that what fits fp32 comes out.
__device__ __forceinline__ float scaled(float y, float s, float f) { return f >= 1.0f ? y * s * f : y * f * s; }

// The digits of a lane's eight elements of x, eight codes a word; the scale of its block of 16, which it
// shares with the lane beside it: binades below the row's, as far as E4M3 goes (2^8 down to 2^-9).
struct Digits {
    uint32_t code[kDigits], scale;
};

__device__ __forceinline__ Digits digits_of(const uint4& v, int e_row)
{
    Digits o;
    uint32_t top = top_bits(v);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const int below = min(17, e_row - unit_of(top)), k = 8 - below;
    o.scale = k >= -6 ? (uint32_t)(k + 7) << 3 : 1u << (k + 9);
    const int e = below - e_row;   // what x is scaled with: two factors, as the sum may pass 127
    const float up0 = pow2i(e / 2), up1 = pow2i(e - e / 2);
    // What is left, in f16 pairs: below 4 with eight significant bits it is exact (elements below 2^-16 of the
    // block's largest to 2^-25 of the unit), and so is every difference.
    uint32_t r[4];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(bf16_hi(w[i]) * up0 * up1), "f"(bf16_lo(w[i]) * up0 * up1));
#pragma unroll
    for (int d = 0; d < kDigits; ++d) {
        uint32_t q[4];
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f16x2 a, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f16x2 b, %6;\n\t"
            "cvt.rn.satfinite.e2m1x2.f16x2 c, %7;\n\t"
            "cvt.rn.satfinite.e2m1x2.f16x2 d, %8;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, a;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, c;\n\t"
            "cvt.rn.f16x2.e2m1x2 %4, d;\n\t}"
            : "=r"(o.code[d]), "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3])
            : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            constexpr uint32_t k8 = 0x48004800u, kMinus8 = 0xC800C800u;   // 8 and -8, twice
            uint32_t r8;
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r8) : "r"(r[i]), "r"(k8));
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[i]) : "r"(q[i]), "r"(kMinus8), "r"(r8));
        }
    }
    return o;
}

// Eight lanes have the four scales of a 64-column group: their word, for each of them.
__device__ __forceinline__ uint32_t scale_word(uint32_t scale, int lane)
{
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, scale, (lane & ~7) + 2 * i) << (8 * i);
    return word;
}

// Block (columns, row): the digits of 2048 columns of a row, two threads a block of 16.
__global__ void __launch_bounds__(kDigitThreads)
    digits_kernel(const __nv_bfloat16* x, int K, int pass_rows, int kb4, uint8_t* codes, uint8_t* scales, float* factors)
{
    __shared__ uint32_t tops[kDigitThreads / 32];
    const int m = blockIdx.y, t = threadIdx.x, lane = t & 31;
    const __nv_bfloat16* row = x + (long long)m * K;
    griddep_wait();
    griddep_launch_dependents();   // the weights may be fetched: nothing before this call writes them any more
    uint32_t top = 0;
    for (int i = t; i < K / 8; i += 4 * kDigitThreads) {
        uint4 v[4];   // in flight together (one after another they took 4 us of 14336 columns)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = i + k * kDigitThreads;
            v[k] = at < K / 8 ? reinterpret_cast<const uint4*>(row)[at] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, top_bits(v[k]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) tops[t >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kDigitThreads / 32; ++i) top = max(top, tops[i]);
    const int e_row = unit_of(top);
    if (blockIdx.x == 0 && t == 0) factors[m] = row_factor(top);
    const int col = blockIdx.x * kDigitColumns + 8 * t;
    const bool real = col < K;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (real) v = *reinterpret_cast<const uint4*>(row + col);
    const Digits o = digits_of(v, e_row);
    const uint32_t word = scale_word(o.scale, lane);
    if (!real) return;
    const int pass = m / pass_rows, r0 = 256 * pass + kDigits * (m - pass * pass_rows);
#pragma unroll
    for (int d = 0; d < kDigits; ++d)
        *reinterpret_cast<uint32_t*>(codes + (long long)(r0 + d) * (K / 2) + col / 2) = o.code[d];
    const int rr = r0 + (lane & 7);   // each lane writes the word of one digit row
    *reinterpret_cast<uint32_t*>(scales + ((long long)(rr >> 7) * kb4 + (col >> 6)) * 512 + (rr & 31) * 16 +
                                 ((rr & 127) >> 5) * 4) = word;
}

// ------------------------------------------------------------------ products

struct GemmParams {
    long long units, chunk;   // (tile, pass) pairs; stages per CTA
    int passes, ks, kb4, nb;  // K stages of a unit, 64-column groups, digit rows of a pass
    int pass_rows, M;
    float* parts;
    unsigned int* status;
    unsigned long long wait_ns;
    int stall;
};

// A stage's scale tiles from shared memory into one lane quarter of TMEM (each quarter holds a copy).
template <int NB>
__device__ __forceinline__ void store_scales(uint32_t stage_smem, uint32_t tmem, uint32_t quarter, int lane)
{
    using P = Plan<NB>;
    const uint32_t sfa_s = stage_smem + kWBytes + P::kDBytes + 16u * (uint32_t)lane, sfb_s = sfa_s + kSfwBytes;
    const uint32_t t = tmem + ((32u * quarter) << 16) + P::kSfTmem;
    uint32_t va[16], vb[P::kHalves][16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 a = ld_shared_v4(sfa_s + 512u * j);
        va[4 * j] = a.x, va[4 * j + 1] = a.y, va[4 * j + 2] = a.z, va[4 * j + 3] = a.w;
#pragma unroll
        for (int h = 0; h < P::kHalves; ++h) {
            const uint4 b = ld_shared_v4(sfb_s + kSfBox * h + 512u * j);
            // columns: group j, then half h
            const int at = 4 * (P::kHalves * j + h);
            vb[at / 16][at % 16] = b.x, vb[at / 16][at % 16 + 1] = b.y;
            vb[at / 16][at % 16 + 2] = b.z, vb[at / 16][at % 16 + 3] = b.w;
        }
    }
    tc_st_32x32b_x16(t, va);
#pragma unroll
    for (int h = 0; h < P::kHalves; ++h) tc_st_32x32b_x16(t + 16 + 16 * h, vb[h]);
}

// The scale warps' role over n stages.  Stages that are there already go together: their stores are waited
// for once (one takes 0.3 us by itself).
template <int NB, int kStages>
__device__ __forceinline__ void scales_role(uint32_t smem, uint32_t tmem, uint64_t* sf_full, uint64_t* full, int n,
                                            uint32_t quarter, int lane, unsigned long long wait_ns, unsigned int* status,
                                            volatile int& s_abort)
{
    using P = Plan<NB>;
    constexpr int kTogether = 3;
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < n;) {
        const bool ok = mbar_wait(&sf_full[stage], phase, wait_ns, status, kStatusTimeoutMma);
        if (!__all_sync(0xffffffffu, ok && s_abort == 0)) {
            s_abort = 1;
            return;
        }
        const int first = stage;
        int together = 0;
        do {
            store_scales<NB>(smem + (uint32_t)stage * P::kStage, tmem + (uint32_t)stage * P::kSfCols, quarter, lane);
            ++together;
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        } while (together < kTogether && i + together < n && __all_sync(0xffffffffu, mbar_test(&sf_full[stage], phase)));
        i += together;
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane < together) mbar_arrive(&full[first + lane < kStages ? first + lane : first + lane - kStages]);
    }
}

// The MMAs of a stage and the release of its slot, by one lane.
template <int NB>
__device__ __forceinline__ void multiply(uint32_t stage_smem, uint32_t tmem, uint32_t d, uint32_t idesc, int nk, bool first,
                                         uint64_t* empty)
{
    using P = Plan<NB>;
    const uint64_t a = smem_desc(stage_smem, 16, 1024, 2), b = smem_desc(stage_smem + kWBytes, 16, 1024, 2);
    const uint32_t sfa = tmem + P::kSfTmem, sfb = sfa + 16;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < nk)
            mma_mxf4nvf4(d, a + 2u * j, b + 2u * j, idesc, sfa + 4u * j, sfb + 4u * P::kHalves * j, !first || j > 0 ? 1u : 0u);
    tc_commit(empty);
}

// E2M1 operands, K-major, N = nb, M = 128, UE4M3 scales.
__device__ __forceinline__ uint32_t mma_desc(int nb)
{
    return (1u << 7) | (1u << 10) | ((uint32_t)(nb >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

// Four rows' sums from their 32 columns of the accumulator: digit d weighs 8^-d.
__device__ __forceinline__ void four_rows(uint32_t tmem, float (&y)[4])
{
    uint32_t v[32];
    tc_ld_32x32b_x32(tmem, v);
    tc_wait_ld_x32(v);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        y[h] = __uint_as_float(v[8 * h + 7]);
#pragma unroll
        for (int t = kDigits - 2; t >= 0; --t) y[h] = fmaf(y[h], 0.125f, __uint_as_float(v[8 * h + t]));
    }
}

template <int NB>
__global__ void __launch_bounds__(kThreads, 1)
    rows_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmSfw,
                     const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmSfd, const GemmParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    using P = Plan<NB>;
    constexpr int kStages = P::kStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((smem_u32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadSmemAlign);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + P::kBarOff);   // codes landed and scales stored
    uint64_t* empty = full + kStages;                                  // the MMAs released the stage
    uint64_t* sf_full = empty + kStages;                               // scale tiles landed
    uint64_t* acc_full = sf_full + kStages;
    uint64_t* acc_empty = acc_full + P::kAccs;
    uint64_t* done_bar = acc_empty + P::kAccs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
    volatile int& s_abort = *reinterpret_cast<volatile int*>(tmem_slot + 1);
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1 + 4);   // the producer, four scale warps
            mbar_init(&empty[i], 1);
            mbar_init(&sf_full[i], 1);
        }
        for (int i = 0; i < P::kAccs; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 4);
        }
        mbar_init(done_bar, 1);
        fence_mbarrier_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmSfw);
        prefetch_tensormap(&tmD);
        prefetch_tensormap(&tmSfd);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();
    // this CTA's stages: `todo` from stage kb0 of unit u0 on (counted on by every role, as divisions take
    // a lone warp longer than a stage does)
    const long long begin = p.chunk * blockIdx.x;
    const int todo = (int)(min(p.units * p.ks, begin + p.chunk) - begin);
    const int u0 = (int)(begin / p.ks), kb0 = (int)(begin - (long long)u0 * p.ks);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        const uint32_t d_bytes = (uint32_t)p.nb * (BK / 2);
        const uint32_t d_halves = (uint32_t)(p.nb + 127) / 128;
        struct At {   // a stage's place
            int kb, pass, tile;
        };
        auto next = [&](At& a) {
            if (++a.kb < p.ks) return;
            a.kb = 0;
            if (++a.pass < p.passes) return;
            a.pass = 0;
            ++a.tile;
        };
        auto load_w = [&](const At& a, int stage) {
            uint8_t* st = smem + stage * P::kStage;
            mbar_arrive_expect_tx(&sf_full[stage], kSfwBytes + d_halves * kSfBox);
            tma_load_2d(st + kWBytes + P::kDBytes, &tmSfw, &sf_full[stage], 0, (a.tile * p.kb4 + a.kb * 4) * 2);
            mbar_arrive_expect_tx(&full[stage], kWBytes + d_bytes);
            tma_load_2d(st, &tmW, &full[stage], a.kb * (BK / 2), a.tile * BM);
        };
        auto load_d = [&](const At& a, int stage) {
            uint8_t* st = smem + stage * P::kStage;
            for (uint32_t h = 0; h < d_halves; ++h)
                tma_load_2d(st + kWBytes + P::kDBytes + kSfwBytes + h * kSfBox, &tmSfd, &sf_full[stage], 0,
                            ((2 * a.pass + (int)h) * p.kb4 + a.kb * 4) * 2);
            tma_load_2d(st + kWBytes, &tmD, &full[stage], a.kb * (BK / 2), 256 * a.pass);
        };
        const int ahead = min(kStages, todo);
        uint32_t fills[kStages] = {};
        if (!p.stall) {
            At w{kb0, u0 % p.passes, u0 / p.passes}, d = w;
            for (int i = 0; i < ahead; ++i, next(w))
                if (elect_one()) load_w(w, i);
            __syncwarp();
            griddep_wait();
            for (int i = 0; i < ahead; ++i, next(d))
                if (elect_one()) load_d(d, i);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kStages; ++i) fills[i] = i < ahead ? 1 : 0;
            int stage = 0;
            uint32_t phase = 0;
            for (int i = ahead; i < todo; ++i, next(w)) {
                const bool ok = mbar_wait(&empty[stage], phase, p.wait_ns, p.status, kStatusTimeoutProducer);
                if (!__all_sync(0xffffffffu, ok && s_abort == 0)) {
                    s_abort = 1;
                    break;
                }
                if (elect_one()) {
                    load_w(w, stage);
                    load_d(w, stage);
                }
                __syncwarp();
                ++fills[stage];
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // every copy lands before the CTA may end
        for (int i = 0; i < kStages; ++i)
            if (fills[i] > 0) {
                (void)mbar_wait(&sf_full[i], (fills[i] - 1u) & 1u, p.wait_ns, p.status, kStatusTimeoutProducer);
                (void)mbar_wait(&full[i], (fills[i] - 1u) & 1u, p.wait_ns, p.status, kStatusTimeoutProducer);
            }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        const uint32_t idesc = mma_desc(p.nb);
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int left = todo, kb = kb0; left > 0 && ok; kb = 0) {
            const int n = min(left, p.ks - kb);   // stages of this unit
            left -= n;
            ok = mbar_wait(&acc_empty[acc], acc_phase ^ 1u, p.wait_ns, p.status, kStatusTimeoutMma);
            ok = __all_sync(0xffffffffu, ok && s_abort == 0);
            tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(acc * NB);
            for (int i = 0; i < n; ++i) {
                ok = mbar_wait(&full[stage], phase, p.wait_ns, p.status, kStatusTimeoutMma);
                ok = __all_sync(0xffffffffu, ok && s_abort == 0);
                if (!ok) break;
                tc_fence_after();
                if (elect_one())
                    multiply<NB>(smem_u32(smem) + (uint32_t)stage * P::kStage, tmem + (uint32_t)stage * P::kSfCols, d, idesc,
                                 min(4, p.kb4 - (kb + i) * 4), i == 0, &empty[stage]);
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (ok && elect_one()) tc_commit(&acc_full[acc]);
            __syncwarp();
            if (++acc == P::kAccs) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (!ok) s_abort = 1;
        // every MMA ends before TMEM is released
        if (elect_one()) tc_commit(done_bar);
        __syncwarp();
        (void)mbar_wait(done_bar, 0u, p.wait_ns, p.status, kStatusTimeoutMma);
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------ scales into TMEM, a lane quarter per warp
        scales_role<NB, kStages>(smem_u32(smem), tmem, sf_full, full, todo, (uint32_t)(warp & 3), lane, p.wait_ns, p.status,
                                 s_abort);
    } else if (warp >= 8) {
        // ------------------------------------------------------------ a unit's sums: digits together, to the workspace
        const int quarter = warp & 3, n = 32 * quarter + lane;
        int acc = 0;
        uint32_t acc_phase = 0;
        griddep_wait();   // an earlier call's joining kernel may read the pieces
        int pass = u0 % p.passes;
        long long piece = (long long)u0 + blockIdx.x;
        for (int left = todo, kb = kb0; left > 0; kb = 0) {
            left -= min(left, p.ks - kb);
            const bool ok = mbar_wait(&acc_full[acc], acc_phase, p.wait_ns, p.status, kStatusTimeoutEpilogue);
            if (!__all_sync(0xffffffffu, ok && s_abort == 0)) {
                s_abort = 1;
                break;
            }
            tc_fence_after();
            const int rows = min(p.pass_rows, p.M - pass * p.pass_rows);
            float* part = p.parts + piece * p.pass_rows * BM + n;
            const uint32_t d = tmem + ((32u * (uint32_t)quarter) << 16) + (uint32_t)(acc * NB);
            for (int m = 0; m < rows; m += 4) {
                float y[4];
                four_rows(d + 8 * m, y);   // (rows past the last are not used)
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    if (m + h < rows) part[(m + h) * BM] = y[h];
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
            if (++acc == P::kAccs) {
                acc = 0;
                acc_phase ^= 1u;
            }
            ++piece;
            if (++pass == p.passes) pass = 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ outputs

struct JoinParams {
    const float* parts;
    const float* factors;
    const float* w_gscale;
    const float* gate;
    long long gate_stride;
    const __nv_bfloat16* bias;
    const __nv_bfloat16* resid;
    __nv_bfloat16* out;
    long long N, chunk;
    int passes, ks, pass_rows, swiglu, M;
};

// silu(g) = g * sigmoid(g) in a form that overflows nowhere (as the GEMM's epilogue has it).
__device__ __forceinline__ float silu_f32(float g)
{
    const float t = ex2_approx(-fabsf(g) * 1.4426950408889634f);
    const float r = rcp_approx(1.0f + t);
    return g * (g >= 0.0f ? r : t * r);
}

// Block (tile, rows): 128 outputs of kRows rows of a pass, the loads of all rows in flight.
template <int kRows>
__global__ void __launch_bounds__(BM) rows_join_kernel(const __grid_constant__ JoinParams p)
{
    const int i = threadIdx.x, groups = (p.pass_rows + kRows - 1) / kRows;   // of a pass
    const int pass = blockIdx.y / groups, mm = (blockIdx.y - pass * groups) * kRows, m0 = pass * p.pass_rows + mm;
    const int rows = min(kRows, min(p.pass_rows - mm, p.M - m0));
    if (rows <= 0) return;
    // What no kernel of this call writes is read ahead of the wait: what wrote it has ended (the digits kernel waited
    // for that, and this one starts behind its start).
    const float s = *p.w_gscale;
    const long long tile = p.swiglu ? 2ll * blockIdx.x : blockIdx.x;
    auto at = [&](long long t, int& pieces) {   // output i's sums of a tile
        const long long u = t * p.passes + pass, first = u * p.ks;
        // (below 2^32 stages for all sizes that are taken)
        const int c0 = (uint32_t)first / (uint32_t)p.chunk, c1 = (uint32_t)(first + p.ks - 1) / (uint32_t)p.chunk;
        pieces = c1 - c0 + 1;
        return p.parts + ((u + c0) * p.pass_rows + mm) * BM + i;
    };
    const long long n = tile * BM + i, step = (long long)p.pass_rows * BM;
    if (n >= p.N) return;
    float bias[2], g[kRows], r[kRows], f[kRows];
    bias[0] = p.bias ? __bfloat162float(p.bias[n]) : 0.0f;
    bias[1] = p.bias && p.swiglu ? __bfloat162float(p.bias[n + BM]) : 0.0f;
#pragma unroll
    for (int k = 0; k < kRows; ++k)
        if (p.gate && k < rows) {
            g[k] = p.gate[(m0 + k) * p.gate_stride + n];
            r[k] = __bfloat162float(p.resid[(m0 + k) * p.N + n]);
        }
    int left[2] = {0, 0};
    const float* from[2] = {at(tile, left[0]), nullptr};
    if (p.swiglu) from[1] = at(tile + 1, left[1]);
    const int most = max(left[0], left[1]);
    griddep_wait();
    griddep_launch_dependents();   // (behind the wait: a next call's first kernels took SMs from this one's products)
#pragma unroll
    for (int k = 0; k < kRows; ++k) f[k] = k < rows ? p.factors[m0 + k] : 0.0f;
    auto sums = [&](auto& y) {
        constexpr int kTiles = sizeof(y) / sizeof(y[0]);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int k = 0; k < kRows; ++k) y[t][k] = 0.0f;
#pragma unroll(kRows > 1 ? 2 : 4)
        for (int c = 0; c < most; ++c)
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int k = 0; k < kRows; ++k)
                    if (k < rows && c < left[t]) y[t][k] += from[t][c * step + k * BM];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int k = 0; k < kRows; ++k) y[t][k] = scaled(y[t][k], s, f[k]) + bias[t];
    };
    if (p.swiglu) {
        float y[2][kRows];
        sums(y);
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (k < rows)
                p.out[(m0 + k) * (p.N / 2) + (long long)blockIdx.x * BM + i] =
                    __float2bfloat16_rn(silu_f32(__bfloat162float(__float2bfloat16_rn(y[0][k]))) *
                                        __bfloat162float(__float2bfloat16_rn(y[1][k])));
        return;
    }
    float y[1][kRows];
    sums(y);
#pragma unroll
    for (int k = 0; k < kRows; ++k)
        if (k < rows) p.out[(m0 + k) * p.N + n] = __float2bfloat16_rn(p.gate ? fmaf(g[k], y[0][k], r[k]) : y[0][k]);
}

// ------------------------------------------------------------------ up to eight rows, in one kernel
//
// A launch, its start and the wait for the one before cost what a small weight's reading does.  So where a
// wave of CTAs has all tiles, a cluster of `split` CTAs (with SwiGLU twice as many: the gate and the up tile)
// takes one: each makes the digits of its own columns of x (under an exponent of its own) beside the other
// roles, multiplies, and adds its sums to those of the others in the first one's shared memory, which
// finishes the outputs.
constexpr int kFewThreads = 512;     // producer, MMA, 2 idle; 4 scale warps; 8 warps of digits, 4 of them of outputs
constexpr int kMaxCluster = 8;

constexpr int kFewRows = 8;

template <int kRows>   // four or eight
struct FewPlan : Plan<kDigits * kRows> {
    using P = Plan<kDigits * kRows>;
    static constexpr int kStages = kRows == 4 ? 8 : 6;
    static constexpr uint32_t kRedOff = kStages * P::kStage;
    static constexpr uint32_t kBarOff = kRedOff + kMaxCluster * kRows * BM * 4;
    static constexpr uint32_t kSmem = kBarOff + 8 * (3 * kStages + 1) + 8 + 4 * 8;
    static_assert(kSmem <= 232448, "shared memory budget");
    static_assert(P::kSfTmem + kStages * P::kSfCols <= kTmemCols, "TMEM budget");
};

struct FewParams {
    const __nv_bfloat16* x;
    JoinParams j;
    long long K;
    int split, ks, kb4;
    unsigned int* status;
    unsigned long long wait_ns;
    int stall;
};

template <int kRows>
__global__ void __launch_bounds__(kFewThreads, 1)
    rows_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmSfw, const FewParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    using P = FewPlan<kRows>;
    constexpr int kStages = P::kStages, kNB = kDigits * kRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((smem_u32(smem) & 1023u) != 0) {   // (the same in every CTA)
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadSmemAlign);
        return;
    }
    float* red = reinterpret_cast<float*>(smem + P::kRedOff);            // the first CTA's: [rank][row][output]
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + P::kBarOff);     // codes landed, digits and scales stored
    uint64_t* empty = full + kStages;
    uint64_t* sf_full = empty + kStages;                              // scale tiles landed and written
    uint64_t* acc_full = sf_full + kStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
    volatile int& s_abort = *reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint32_t* tops = tmem_slot + 2;   // per warp of digits: the largest that it read
    const int M = p.j.M, row_warps = kRows == 8 ? 8 : M > 2 ? 4 : M;   // warps of digits per stage
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1 + 4 + row_warps);   // W, the scale warps, those of digits
            mbar_init(&empty[i], 1);
            mbar_init(&sf_full[i], 1 + row_warps);
        }
        mbar_init(acc_full, 1);
        fence_mbarrier_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmSfw);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_arrive();   // (waited for before anything is written to the first CTA)
    const uint32_t tmem = *tmem_slot;
    const int rank = (int)cluster_ctarank(), size = p.j.swiglu ? 2 * p.split : p.split;
    const int group = blockIdx.x / size, part = rank % p.split;
    const int tile = p.j.swiglu ? 2 * group + rank / p.split : group;
    const int kb0 = p.ks * part / p.split, n = p.ks * (part + 1) / p.split - kb0;
    griddep_wait();
    griddep_launch_dependents();

    if (warp == 0) {
        // ------------------------------------------------------------ W and its scales
        uint32_t fills[kStages] = {};
        int stage = 0;
        uint32_t phase = 1;   // (the first fills wait for nothing)
        for (int i = 0; i < n && !p.stall; ++i) {
            const bool ok = mbar_wait(&empty[stage], phase, p.wait_ns, p.status, kStatusTimeoutProducer);
            if (!__all_sync(0xffffffffu, ok && s_abort == 0)) {
                s_abort = 1;
                break;
            }
            if (elect_one()) {
                uint8_t* st = smem + stage * P::kStage;
                mbar_arrive_expect_tx(&sf_full[stage], kSfwBytes);
                tma_load_2d(st + kWBytes + P::kDBytes, &tmSfw, &sf_full[stage], 0, (tile * p.kb4 + (kb0 + i) * 4) * 2);
                mbar_arrive_expect_tx(&full[stage], kWBytes);
                tma_load_2d(st, &tmW, &full[stage], (kb0 + i) * (BK / 2), tile * BM);
            }
            __syncwarp();
            ++fills[stage];
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // every copy lands before the CTA may end
        for (int i = 0; i < kStages; ++i)
            if (fills[i] > 0) {
                (void)mbar_wait(&sf_full[i], (fills[i] - 1u) & 1u, p.wait_ns, p.status, kStatusTimeoutProducer);
                (void)mbar_wait(&full[i], (fills[i] - 1u) & 1u, p.wait_ns, p.status, kStatusTimeoutProducer);
            }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        const uint32_t idesc = mma_desc(kDigits * M);
        int stage = 0;
        uint32_t phase = 0;
        for (int i = 0; i < n; ++i) {
            const bool ok = mbar_wait(&full[stage], phase, p.wait_ns, p.status, kStatusTimeoutMma);
            if (!__all_sync(0xffffffffu, ok && s_abort == 0)) {
                s_abort = 1;
                break;
            }
            tc_fence_after();
            if (elect_one())
                multiply<kNB>(smem_u32(smem) + (uint32_t)stage * P::kStage, tmem + (uint32_t)stage * P::kSfCols,
                                             tmem, idesc, min(4, p.kb4 - (kb0 + i) * 4), i == 0, &empty[stage]);
            __syncwarp();
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // every MMA ends before TMEM is released
        if (elect_one()) tc_commit(acc_full);
        __syncwarp();
        (void)mbar_wait(acc_full, 0u, p.wait_ns, p.status, kStatusTimeoutMma);
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------ scales into TMEM, a lane quarter per warp
        scales_role<kNB, kStages>(smem_u32(smem), tmem, sf_full, full, n, (uint32_t)(warp & 3), lane, p.wait_ns,
                                                 p.status, s_abort);
    } else if (warp >= 8) {
        // ------------------------------------------------------------ digits: warp w takes row w % row_warps of every
        // eighth, fourth or second stage.  A slot of the ring is always the same warp's: a parity tells a phase only
        // from its neighbours, so whoever waits for a slot has to have waited for its fill before (with six stages
        // warps took a slot whose last but one fill was still in use for free).  What it reads for the row's
        // largest it keeps.
        static_assert(kStages % 8 == 0 || kRows == 8, "a slot is one warp's");   // (eight rows: every slot is each one's)
        constexpr int kKept = 8;
        const int w = warp - 8, m = w % row_warps, every = 8 / row_warps, i0 = w / row_warps;
        const long long c0 = (long long)kb0 * BK + 8 * lane;
        auto read = [&](int i) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (m < M && i < n && c0 + (long long)i * BK < p.K)
                v = *reinterpret_cast<const uint4*>(p.x + m * p.K + c0 + i * BK);
            return v;
        };
        uint4 kept[kKept];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kKept; ++k) kept[k] = read(i0 + k * every);
#pragma unroll
        for (int k = 0; k < kKept; ++k) top = max(top, top_bits(kept[k]));
#pragma unroll 4
        for (int i = i0 + kKept * every; i < n; i += every) top = max(top, top_bits(read(i)));
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) tops[w] = top;
        named_bar_sync(2, 256);
        for (int k = m; k < 8; k += row_warps) top = max(top, tops[k]);
        const int e_row = unit_of(top);
        auto put = [&](int i, const uint4& v) {
            const int stage = i % kStages;
            const bool ok = mbar_wait(&empty[stage], (uint32_t)(i / kStages & 1) ^ 1u, p.wait_ns, p.status,
                                      kStatusTimeoutProducer);
            if (!__all_sync(0xffffffffu, ok && s_abort == 0)) {
                s_abort = 1;
                return false;
            }
            if (m < M) {
                uint8_t* codes = smem + stage * P::kStage + kWBytes;
                uint8_t* scales = codes + P::kDBytes + kSfwBytes;
                const Digits o = digits_of(v, e_row);
                // row 8 m + d of 128 bytes, its 16-byte chunks swizzled by the row in its eight
#pragma unroll
                for (int d = 0; d < kDigits; ++d)
                    *reinterpret_cast<uint32_t*>(codes + (kDigits * m + d) * 128 + (((lane >> 2) ^ d) << 4) + 4 * (lane & 3)) =
                        o.code[d];
                const int row = kDigits * m + (lane & 7);
                *reinterpret_cast<uint32_t*>(scales + (lane >> 3) * 512 + (row & 31) * 16 + (row >> 5) * 4) =
                    scale_word(o.scale, lane);
                fence_proxy_async_smem();   // the codes, for the MMAs
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sf_full[stage]);
                mbar_arrive(&full[stage]);
            }
            return true;
        };
        bool on = true;
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (on && i0 + k * every < n) on = put(i0 + k * every, kept[k]);
        int i = i0 + kKept * every;
        for (uint4 v = read(i); on && i < n; i += every) {
            const uint4 next = read(i + every);
            on = put(i, v);
            v = next;
        }
    }
    // what the last four warps need, most of it the first CTA's for the outputs
    const int o = (int)threadIdx.x - 12 * 32;
    const long long out0 = (p.j.swiglu ? 2ll * group : (long long)tile) * BM + o;   // the first tile's row of W
    float s = 0.0f, bias[2] = {0.0f, 0.0f}, gate[kRows], resid[kRows];
    if (warp >= 12) {
        // ------------------------------------------------------------ sums to the cluster's first CTA
        const int quarter = warp & 3;
        s = *p.j.w_gscale;
        if (rank == 0) {
            if (p.j.bias && out0 < p.j.N) bias[0] = __bfloat162float(p.j.bias[out0]);
            if (p.j.bias && p.j.swiglu) bias[1] = __bfloat162float(p.j.bias[out0 + BM]);
#pragma unroll
            for (int m = 0; m < kRows; ++m)
                if (p.j.gate && m < M && out0 < p.j.N) {
                    gate[m] = p.j.gate[m * p.j.gate_stride + out0];
                    resid[m] = __bfloat162float(p.j.resid[m * p.j.N + out0]);
                }
        }
        const bool ok = mbar_wait(acc_full, 0u, p.wait_ns, p.status, kStatusTimeoutEpilogue);
        if (!__all_sync(0xffffffffu, ok)) s_abort = 1;
        tc_fence_after();
        cluster_wait();   // the first CTA has begun
        auto factor = [&](int row) {   // (the barrier of the digits was behind what the warps read)
            uint32_t top = 0;
            for (int k = row; k < 8; k += row_warps) top = max(top, tops[k]);
            return row_factor(top);
        };
        const uint32_t to = mapa_shared(smem_u32(red), 0) + 4u * (uint32_t)(rank * kRows * BM + o);
#pragma unroll
        for (int m0 = 0; m0 < kRows; m0 += 4) {
            if (m0 >= M) continue;
            float y[4];
            four_rows(tmem + ((32u * (uint32_t)quarter) << 16) + 8 * m0, y);
#pragma unroll
            for (int h = 0; h < 4; ++h)
                if (m0 + h < M)
                    st_shared_cluster_u32(to + 4u * (uint32_t)((m0 + h) * BM), __float_as_uint(scaled(y[h], s, factor(m0 + h))));
        }
    }
    __syncwarp();
    if (warp < 12) cluster_wait();
    tc_fence_before();
    cluster_sync();   // all sums are there (and all warps of this CTA through)
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (rank != 0 || warp < 12 || out0 >= p.j.N) return;
    auto value = [&](int first, int m, float b) {
        float y = 0.0f;
        for (int r = first; r < first + p.split; ++r) y += red[(r * kRows + m) * BM + o];
        return y + b;
    };
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        if (m >= M) break;
        float v = value(0, m, bias[0]);
        if (p.j.swiglu) {
            const float g = __bfloat162float(__float2bfloat16_rn(v));
            const float u = __bfloat162float(__float2bfloat16_rn(value(p.split, m, bias[1])));
            p.j.out[m * (p.j.N / 2) + (long long)group * BM + o] = __float2bfloat16_rn(silu_f32(g) * u);
        } else {
            if (p.j.gate) v = fmaf(gate[m], v, resid[m]);
            p.j.out[m * p.j.N + out0] = __float2bfloat16_rn(v);
        }
    }
}

template <int kRows>
cudaLaunchConfig_t few_config(unsigned ctas, int cluster, cudaLaunchAttribute (&attr)[2], cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = FewPlan<kRows>::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

// Clusters of `size` CTAs that the current device holds at once (looked up once per device).
template <int kRows>
int few_clusters(int size)
{
    static std::mutex mu;
    static int known[64][kMaxCluster + 1] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int& n = known[dev][size];
    if (n == 0) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = few_config<kRows>((unsigned)size, size, attr, nullptr);
        if (ensure_dynamic_smem(reinterpret_cast<const void*>(rows_few_kernel<kRows>), (int)FewPlan<kRows>::kSmem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, rows_few_kernel<kRows>, &cfg) != cudaSuccess || n <= 0)
            n = -1;
    }
    return n > 0 ? n : 0;
}

// CTAs per tile of the one-kernel form; 0 where the others take less time.
template <int kRows>
int few_split(const LinearRowsJob& job, const Layout& l)
{
    const int ks = (int)((job.K + BK - 1) / BK), tiles_of = job.swiglu ? 2 : 1;
    const long long groups = l.tiles / tiles_of;
    int best = 0;
    for (int split = 1; split * tiles_of <= kMaxCluster && split <= ks; ++split)
        if (groups <= few_clusters<kRows>(split * tiles_of)) best = split;
    if (best == 0) return 0;
    // A stage takes an SM 0.4 us (0.75 with five to eight rows, whose digits every CTA makes for itself); the three
    // kernels share the stages evenly but take 3 us more.  (Measured, one row: 9216 x 3072 6.4 us against 8.4,
    // 4096 x 14336 8.8 against 12.2, 2048 x 2048 4.7 against 6.0; 512 x 65536, whose tiles would keep 64 SMs, 13.1 us
    // with three kernels.  Eight rows: 2048 x 2048 5.8 us against 5.7 and from Python 8.5
    // against 12.6, 9216 x 3072 8.3 against 7.9 and 9.0 against 12.9, 4096 x 14336 15.2 against 12.0.)
    const double stages = (double)l.tiles * ks / sm_count_current_device(), stage = kRows == 4 ? 0.4 : 0.75;
    return (ks + best - 1) / best * stage < stages * 0.4 + 3.0 ? best : 0;
}

// The maps of the weights' codes and scales.
bool weight_maps(const LinearRowsJob& job, const Layout& l, CUtensorMap* codes, CUtensorMap* scales)
{
    const uint64_t kbytes = (uint64_t)job.K / 2;
    return make_map_2d(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, job.w_codes, kbytes, (uint64_t)job.N, kbytes, BK / 2, BM,
                       CU_TENSOR_MAP_SWIZZLE_128B) &&
           make_map_2d(scales, CU_TENSOR_MAP_DATA_TYPE_UINT8, job.w_sf, 256, (uint64_t)(l.tiles * l.kb4 * 2), 256, 256,
                       kSfBox / 256, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int kRows>
cudaError_t launch_few(const LinearRowsJob& job, const Layout& l, const JoinParams& jp, int split, cudaStream_t s)
{
    CUtensorMap tmW, tmSfw;
    if (!weight_maps(job, l, &tmW, &tmSfw)) return cudaErrorInvalidValue;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(rows_few_kernel<kRows>), (int)FewPlan<kRows>::kSmem);
    if (e != cudaSuccess) return e;
    FewParams p{};
    p.x = job.x;
    p.j = jp;
    p.K = job.K;
    p.split = split;
    p.ks = (int)((job.K + BK - 1) / BK);
    p.kb4 = (int)l.kb4;
    p.status = reinterpret_cast<unsigned int*>(job.ws);
    p.wait_ns = job.wait_limit_ns;
    p.stall = job.stall;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = few_config<kRows>((unsigned)(l.tiles * split), job.swiglu ? 2 * split : split, attr, s);
    return cudaLaunchKernelEx(&cfg, rows_few_kernel<kRows>, tmW, tmSfw, p);
}

template <int NB>
cudaError_t launch_gemm_rows(const LinearRowsJob& job, const Layout& l, const GemmParams& p, unsigned ctas,
                             cudaLaunchConfig_t cfg)
{
    CUtensorMap tmW, tmSfw, tmD, tmSfd;
    const uint64_t kbytes = (uint64_t)job.K / 2;
    const uint64_t d_tiles = (uint64_t)((l.digit_rows + 127) / 128);
    if (!weight_maps(job, l, &tmW, &tmSfw) ||
        !make_map_2d(&tmD, CU_TENSOR_MAP_DATA_TYPE_UINT8, job.ws + l.codes, kbytes, (uint64_t)l.digit_rows, kbytes, BK / 2,
                     (uint32_t)p.nb, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_2d(&tmSfd, CU_TENSOR_MAP_DATA_TYPE_UINT8, job.ws + l.scales, 256, d_tiles * (uint64_t)l.kb4 * 2, 256,
                     256, kSfBox / 256, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(rows_gemm_kernel<NB>), (int)Plan<NB>::kSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Plan<NB>::kSmem;
    return cudaLaunchKernelEx(&cfg, rows_gemm_kernel<NB>, tmW, tmSfw, tmD, tmSfd, p);
}

}  // namespace

size_t linear_rows_workspace_bytes(int64_t M, int64_t N, int64_t K) { return layout(M, N, K).bytes; }

cudaError_t launch_linear_rows(const LinearRowsJob& job, cudaStream_t s)
{
    const Layout l = layout(job.M, job.N, job.K);
    JoinParams jp{};
    jp.w_gscale = job.w_gscale;
    jp.gate = job.gate;
    jp.gate_stride = job.gate_stride;
    jp.bias = job.bias;
    jp.resid = job.resid;
    jp.out = job.out;
    jp.N = job.N;
    jp.swiglu = job.swiglu;
    jp.M = (int)job.M;
    if (job.M <= 4) {
        if (const int split = few_split<4>(job, l)) return launch_few<4>(job, l, jp, split, s);
    } else if (job.M <= kFewRows) {
        if (const int split = few_split<8>(job, l)) return launch_few<8>(job, l, jp, split, s);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;

    cfg.gridDim = dim3((unsigned)((job.K + kDigitColumns - 1) / kDigitColumns), (unsigned)job.M);
    cfg.blockDim = dim3(kDigitThreads);
    float* factors = reinterpret_cast<float*>(job.ws + kFactors);
    cudaError_t e = ensure_shared_carveout(reinterpret_cast<const void*>(digits_kernel));
    if (e != cudaSuccess) return e;
    e = cudaLaunchKernelEx(&cfg, digits_kernel, job.x, (int)job.K, l.pass_rows, (int)l.kb4,
                                       job.ws + l.codes, job.ws + l.scales, factors);
    if (e != cudaSuccess) return e;

    GemmParams p{};
    p.units = l.tiles * l.passes;
    p.passes = l.passes;
    p.ks = (int)((job.K + BK - 1) / BK);
    p.kb4 = (int)l.kb4;
    p.nb = kDigits * l.pass_rows;
    p.pass_rows = l.pass_rows;
    p.M = (int)job.M;
    p.parts = reinterpret_cast<float*>(job.ws + l.parts);
    p.status = reinterpret_cast<unsigned int*>(job.ws);
    p.wait_ns = job.wait_limit_ns;
    p.stall = job.stall;
    const int sms = sm_count_current_device();
    const long long most = sms < kMaxCtas ? sms : kMaxCtas, stages = p.units * p.ks;
    p.chunk = (stages + most - 1) / most;
    const unsigned ctas = (unsigned)((stages + p.chunk - 1) / p.chunk);
    e = p.nb <= 64 ? launch_gemm_rows<64>(job, l, p, ctas, cfg)
        : p.nb <= 128 ? launch_gemm_rows<128>(job, l, p, ctas, cfg)
                      : launch_gemm_rows<256>(job, l, p, ctas, cfg);
    if (e != cudaSuccess) return e;

    jp.parts = p.parts;
    jp.factors = factors;
    jp.chunk = p.chunk;
    jp.passes = l.passes;
    jp.ks = p.ks;
    jp.pass_rows = l.pass_rows;
    auto join = [&](void (*kernel)(JoinParams)) {
        const cudaError_t e = ensure_shared_carveout(reinterpret_cast<const void*>(kernel));
        return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kernel, jp) : e;
    };
    // four rows a thread where there are many blocks (61 rows of 49 tiles 8 -> 5 us cold)
    const unsigned tiles = (unsigned)(job.swiglu ? l.tiles / 2 : l.tiles);
    cfg.blockDim = dim3(BM);
    if (tiles * job.M > 1216) {
        cfg.gridDim = dim3(tiles, (unsigned)(l.passes * ((l.pass_rows + 3) / 4)));
        return join(rows_join_kernel<4>);
    }
    cfg.gridDim = dim3(tiles, (unsigned)(l.passes * l.pass_rows));
    return join(rows_join_kernel<1>);
}

}  // namespace h3fp4
