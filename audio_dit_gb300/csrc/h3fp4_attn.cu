// Attention of packed query rows to an encoder's states and to a shared context.
//
//     out[r][h] = sum_j p_j v_j / l,  p_j = exp(scale q_r.k_j - m),  l = sum_j p_j
// over the context's keys and the keys of r's own segment, in one pass over the
// keys with a running maximum: scores S = Q K^T of 128 queries x 128 keys and
// the products P V run on the tensor cores (tcgen05, bf16 operands, fp32
// accumulators in TMEM); the softmax between them runs in registers, one thread
// per query row.
//
// The maximum in use, m, only follows the true one when that is more than 2^8
// above it (in exp's base 2): the p_j stay below 2^8, l and the sums lose
// nothing in fp32, and the accumulator is rescaled a few times per row instead
// of once per tile.  The p_j are rounded to bf16 for their product with V (the
// tensor cores' 16-bit input with fp32's range); l sums them unrounded.
//
// How units, steps and pieces are cut: attn_plan.h.
//
// Roles (512 threads, one CTA per SM):
//   warp 0       loads: Q tiles (three places, two with solo units) and a ring of K
//                and V tiles by TMA, 128-byte swizzled 64-column chunks; columns past
//                D are zero-filled
//   warps 1, 3   issue the MMAs of query tile A, of tile B.  Per key tile: S_X =
//                Q_X K^T, then, once the softmax stored P_X over S_X's first
//                columns (in two halves), O_X += P_X V.  One tile's MMAs run under
//                the other's softmax.  A warp of its own per tile, since the
//                waits and bookkeeping around a tile's sixteen MMAs take one warp
//                about as long as the MMAs themselves.
//   warp 2       allocates TMEM; walks the CTA's pieces for all roles; keys that
//                are left out (a mask, the end of a segment inside a tile): their
//                bits for the softmax, and zeros over their rows of the V tile,
//                since 0 * NaN is not 0
//   warps 4-11   softmax of tile A, of tile B (a warpgroup each)
//   warps 12-15  epilogue: divides by l, rounds, stores; or stores partial sums
// The epilogue of a unit overlaps the next unit's first MMAs and softmax.
//
// What bounds it: a step (two query tiles, 128 keys, heads of 128) is 2048 cycles
// of MMAs and takes about 2700, because a tile's softmax (about 1500) and its own
// MMAs follow one another and the other tile fills the tensor cores only in part.
// With heads of 64 the softmax warpgroups' latency is what is left (2490 a step,
// 1024 of them MMAs).  A unit's ends cost about one step more.  Kernel time with
// flushed caches: 2 x 8192 rows over 1024 shared and 8192 own keys, 24 heads of
// 128: 1068 us (1.74 PFLOP/s); 31744 rows over as many keys: 7.36 ms (1.68 PFLOP/s);
// 30720 rows over 512 keys: 152 us (1.27 PFLOP/s); 1024 rows over 30720 keys: 244 us
// (1.58 PFLOP/s); one row over 32768 keys, 32 heads over 8: 46 us (35 of them this
// kernel, 3.8 TB/s).
//
// Every wait is bounded; a role that gives up records it in the status word and
// leaves, and so do the roles that depend on it.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_bf16.h>

#include "attn_plan.h"
#include "h3fp4_heads.h"
#include "ptx_sm103.cuh"
#include "tensor_map.h"

namespace h3fp4 {
namespace {

constexpr int kThreads = 512;
// log2 of how far the true maximum may pass the one in use (2 x 8192 rows over 1024
// shared and 8192 own keys: 1066 us, following every new maximum 1325 us)
constexpr float kGrowth = 8.0f;
constexpr int kMaskSlots = 8;       // more than the ring's V tiles
constexpr int kPieceSlots = 4;
constexpr uint32_t kTmemCols = 512;
// The softmax holds 128 scores a thread; with 152 registers it spills. The others' split
// hardly matters (72/176/80 and 80/176/64: the same within 2 %; 96/168/80: 30720
// rows over 512 keys 164 us instead of 152, 112/160/80: 185).
constexpr uint32_t kRegsControl = 80, kRegsSoftmax = 176, kRegsEpilogue = 80;
static_assert(kRegsControl + 2 * kRegsSoftmax + kRegsEpilogue <= 512, "setmaxnreg shares exceed the launch budget");

constexpr unsigned int kStatusTimeoutAttnLoad = 64u, kStatusTimeoutAttnMma = 128u, kStatusTimeoutAttnSoftmax = 256u,
                       kStatusTimeoutAttnEpilogue = 512u, kStatusTimeoutAttnMask = 1024u;

template <int DP, bool kSolo>
struct Layout {
    static constexpr uint32_t kTile = 128 * DP * 2;   // bytes of a 128-row tile
    // Q tiles: one more than a unit has, so that the next unit's first tile is there
    // when this unit's last products are issued; the rest holds K and V tiles.
    static constexpr int kQ = kSolo ? 2 : 3;
    static constexpr int kStages = (7 - kQ) * (128 / DP);
    static constexpr uint32_t kKvOff = kQ * kTile;
    static constexpr uint32_t kBarOff = kKvOff + kStages * kTile;
    // barriers: q_full (two per Q tile), q_empty, kv_full (two per stage), kv_empty, s_full, p_half, p_full,
    // o_full, o_empty, stat_full, stat_empty, done, turn (2 each), gap_load, mask_full, zero_full (per slot),
    // piece_full, piece_empty (per slot)
    static constexpr int kBars = 3 * kQ + 3 * kStages + 18 + 3 * kMaskSlots + 2 * kPieceSlots;
    static_assert(kStages / 2 + 1 < kMaskSlots, "a mask slot's readers are through when its next V tile lands");
    static constexpr uint32_t kMaskOff = kBarOff + (kBars * 8 + 8 + 15) / 16 * 16;
    static constexpr uint32_t kPieceOff = kMaskOff + kMaskSlots * 16;
    static constexpr uint32_t kStatOff = kPieceOff + kPieceSlots * 48;
    static constexpr uint32_t kBytes = kStatOff + 2 * 128 * 8;
    static_assert(kBytes <= 232448, "shared memory budget");
};

struct AttnParams {
    AttnTable t;
    int Hq, group, D, T, C;
    const uint8_t* key_mask;
    const uint8_t* ctx_mask;
    float scale_log2, growth;      // growth: kGrowth in units of the raw scores
    __nv_bfloat16* out;
    long long out_row, out_head;
    int wide_out;                  // output rows 32-byte aligned, D % 16 == 0
    float* lse;
    float* part[2];                // partial sums: segments' units, the context entry's
    int slot_rows[2];
    uint32_t q_bytes;              // bytes a Q tile's copies deliver
    unsigned int* status;
    unsigned long long wait_ns;
    int stall;                     // self-test: the loads are left out, so every wait runs out
};

// Tiles of a piece for query tile X: how many, and which is the i-th (relative to t0).
template <bool kSolo>
__device__ __forceinline__ int tiles_for(const Piece& u, int X, int tok)
{
    if (kSolo) return X == 0 ? (u.nt + 1) >> 1 : u.nt >> 1;
    return X == 0 || u.ntok > tok ? u.nt : 0;
}
template <bool kSolo>
__device__ __forceinline__ int tile_at(int X, int i)
{
    return kSolo ? 2 * i + X : i;
}
// Places of K and V tile i of nt in the ring's order of loads.
template <bool kSolo>
__device__ __forceinline__ int k_place(int i)
{
    return kSolo ? (i == 0 ? 0 : 2 * i - 1) : 2 * i;
}
template <bool kSolo>
__device__ __forceinline__ int v_place(int i, int nt)
{
    return kSolo ? (i == nt - 1 ? 2 * nt - 1 : 2 * i + 2) : 2 * i + 1;
}

// One row's 32 sums v (columns c0...) as bf16, by the lanes whose `on` is set.
__device__ __forceinline__ void store_bf16(uint32_t on, __nv_bfloat16* o, const uint32_t (&v)[32], uint64_t f, int cols,
                                           bool wide)
{
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
        w[j] = cvt_bf16x2(mul2(f2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), f));
    if (wide) {
#pragma unroll
        for (int j = 0; j < 2; ++j) st_global_v8_if(on & (uint32_t)(16 * j < cols), o + 16 * j, w + 8 * j);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) st_global_v4_if(on & (uint32_t)(8 * j < cols), o + 8 * j, w + 4 * j);
    }
}

template <int DP, bool kSolo>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKc,
                const __grid_constant__ CUtensorMap tmVc, const __grid_constant__ AttnParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = Layout<DP, kSolo>;
    constexpr int kStages = L::kStages;
    constexpr int kChunks = DP / 64;
    constexpr uint32_t kTmS = 0, kTmO = 256;  // S_A, S_B at 0 and 128; O_A, O_B from 256, DP columns each
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // Swizzled TMA tiles need 1024-byte alignment; refuse to run otherwise.
    if ((smem_u32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadSmemAlign);
        griddep_wait();
        return;
    }
    // A wait tells a barrier's phase from the one before it by a parity, so it is
    // right only once the phase before has completed.  Copies may land out of
    // order, and a role that waits for some of the ring's places only can ask for
    // a fill before the previous one of its stage has landed (for another role).
    // So the "full" barriers alternate between two per stage: the fill before the
    // previous one is over when this one can be asked for, as the loads of what
    // the role used last have been issued since.
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);  // the Q tile landed, two per tile
    uint64_t* q_empty = q_full + 2 * L::kQ;         // its last S was computed
    uint64_t* kv_full = q_empty + L::kQ;            // the K or V tile landed, two per stage
    uint64_t* kv_empty = kv_full + 2 * kStages;     // its MMAs are done
    uint64_t* s_full = kv_empty + kStages;          // per query tile: S computed (and the MMAs before it done)
    uint64_t* p_half = s_full + 2;                  // P's first 64 keys stored, O rescaled where it had to be
    uint64_t* p_full = p_half + 2;                  // all of P stored
    uint64_t* o_full = p_full + 2;                  // O complete
    uint64_t* o_empty = o_full + 2;                 // O read by the epilogue
    uint64_t* stat_full = o_empty + 2;              // maximum and sum of each row stored
    uint64_t* stat_empty = stat_full + 2;           // and read
    uint64_t* gap_load = stat_empty + 2;            // per slot: the load of a V tile with gaps was issued
    uint64_t* mask_full = gap_load + kMaskSlots;    // per slot: bits stored
    uint64_t* zero_full = mask_full + kMaskSlots;   // per slot: V rows zeroed
    uint64_t* done = zero_full + kMaskSlots;        // a warp's MMAs are done
    uint64_t* turn = done + 2;                      // a warp may issue its next tile's MMAs
    uint64_t* piece_full = turn + 2;                // per slot: a piece is described
    uint64_t* piece_empty = piece_full + kPieceSlots;  // and read by all that work on it
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(piece_empty + kPieceSlots);
    uint32_t* mask_bits = reinterpret_cast<uint32_t*>(smem + L::kMaskOff);
    float2* stat = reinterpret_cast<float2*>(smem + L::kStatOff);  // [2][128]: (maximum, sum)

    if (threadIdx.x < L::kBars) {
        // one barrier per thread; the arrivals that complete a phase
        const uint64_t* b = q_full + threadIdx.x;
        auto in = [&](const uint64_t* first, int n) { return b >= first && b < first + n; };
        const uint32_t count = in(q_empty, L::kQ)                             ? (kSolo ? 2 : 1)
                               : in(kv_empty, kStages)                        ? (kSolo ? 1 : 2)
                               : in(p_half, 4) || in(o_empty, 6)              ? 4   // warps of a warpgroup
                               : in(piece_empty, kPieceSlots)                 ? 16  // loads, MMAs (2), gaps, softmax (8), epilogue (4)
                                                                              : 1;
        mbar_init(q_full + threadIdx.x, count);
        fence_mbarrier_init();
    }
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmQ);
        if (p.T > 0) {
            prefetch_tensormap(&tmK);
            prefetch_tensormap(&tmV);
        }
        if (p.C > 0) {
            prefetch_tensormap(&tmKc);
            prefetch_tensormap(&tmVc);
        }
    }
    Walk walk(p.t);  // warp 2's
    if (warp == 2) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
        walk.start(blockIdx.x);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Everything above overlaps the previous kernel's tail (programmatic
    // dependent launch); its outputs are read only after this.
    griddep_wait();
    const uint32_t tmem = *tmem_slot;
    const int tok = p.t.tok;
    // The pieces of this CTA, described by warp 2 a few ahead (a walk costs some hundred cycles of
    // constant loads; a slot is read in one).
    uint32_t piece_count = 0;
    auto next_piece = [&](Piece& u, bool& ok, unsigned int code) {
        const uint32_t slot = piece_count % kPieceSlots;
        ok &= mbar_wait(&piece_full[slot], (piece_count / kPieceSlots) & 1u, p.wait_ns, p.status, code);
        const int4* rec = reinterpret_cast<const int4*>(smem + L::kPieceOff + slot * 48);
        const int4 a = rec[0], b = rec[1], c = rec[2];
        ++piece_count;
        u.t0 = a.x, u.nt = a.y, u.ntok = a.z, u.tok0 = a.w;
        u.head0 = b.x, u.ctx_tiles = b.y, u.kv0 = b.z, u.kv_len = b.w;
        u.slot = c.x, u.e = c.y;
        u.whole = c.x < 0;
        u.find_gaps(p.t);
        __syncwarp();
        mbar_arrive_if(lane == 0, &piece_empty[slot]);
        return __all_sync(0xffffffffu, ok) && u.nt >= 0;  // -1: no piece is left
    };
    auto next_with_keys = [&](Piece& u, bool& ok, unsigned int code) {
        while (next_piece(u, ok, code))
            if (u.nt > 0) return true;
        return false;
    };
    // the "full" barrier of a place, and its parity
    auto q_bar = [&](uint32_t place) { return &q_full[place % (2 * L::kQ)]; };
    auto q_par = [&](uint32_t place) { return (place / (2 * L::kQ)) & 1u; };
    auto kv_bar = [&](uint32_t place) { return &kv_full[place % (2 * kStages)]; };
    auto kv_par = [&](uint32_t place) { return (place / (2 * kStages)) & 1u; };

    if (warp < 4) {
        setmaxnreg_dec<kRegsControl>();
        if (warp == 0) {
            // ------------------------------------------------------------ loads
            Piece u;
            uint32_t q_place = 0, place = 0, gaps = 0;
            bool ok = p.stall == 0;
            while (ok && next_with_keys(u, ok, kStatusTimeoutAttnLoad)) {
                const int tiles = !kSolo && u.ntok > tok ? 2 : 1;
                const int hk = u.head0 / p.group;
                // Q_A, K_0, Q_B, then the rest: Q_B's place is this unit's predecessor's Q_A, which is
                // given back last, and nothing else shall wait for it.
                for (int i = 0; i < 2 * u.nt; ++i, ++place) {
                    for (int X = i; X < tiles && i < 2; X += 2, ++q_place) {
                        const uint32_t st = q_place % L::kQ;
                        ok = mbar_wait(&q_empty[st], ((q_place / L::kQ) & 1u) ^ 1u, p.wait_ns, p.status,
                                       kStatusTimeoutAttnLoad);
                        if (!__all_sync(0xffffffffu, ok)) {
                            ok = false;
                            break;
                        }
                        if (elect_one()) {
                            mbar_arrive_expect_tx(q_bar(q_place), p.q_bytes);
                            for (int c = 0; c < kChunks; ++c)
                                tma_load_3d(smem + st * L::kTile + c * 16384, &tmQ, q_bar(q_place), 64 * c, u.head0,
                                            u.tok0 + X * tok);
                        }
                    }
                    if (!ok) break;
                    // which tile the ring's next place takes
                    bool is_v;
                    int t;
                    if (kSolo) {
                        is_v = i == 2 * u.nt - 1 || (i > 0 && (i & 1) == 0);
                        t = i == 0 ? 0 : i == 2 * u.nt - 1 ? u.nt - 1 : is_v ? i / 2 - 1 : (i + 1) / 2;
                    } else {
                        is_v = (i & 1) != 0;
                        t = i >> 1;
                    }
                    t += u.t0;
                    const uint32_t st = place % kStages;
                    ok = mbar_wait(&kv_empty[st], ((place / kStages) & 1u) ^ 1u, p.wait_ns, p.status,
                                   kStatusTimeoutAttnLoad);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const bool ctx = t < u.ctx_tiles;
                        const CUtensorMap* map = is_v ? (ctx ? &tmVc : &tmV) : (ctx ? &tmKc : &tmK);
                        const int row = ctx ? t * kKeyTile : u.kv0 + (t - u.ctx_tiles) * kKeyTile;
                        uint8_t* d = smem + L::kKvOff + st * L::kTile;
                        mbar_arrive_expect_tx(kv_bar(place), L::kTile);
                        for (int c = 0; c < kChunks; ++c)
                            tma_load_3d(d + c * 16384, map, kv_bar(place), 64 * c, hk, row);
                        if (is_v && u.has_gaps(t)) mbar_arrive(&gap_load[gaps % kMaskSlots]);
                    }
                    gaps += is_v && u.has_gaps(t);
                }
            }
            // No copy may be in flight when the CTA leaves (all have landed unless a role gave up).
            for (uint32_t b = 1; b <= L::kQ && b <= q_place; ++b)
                (void)mbar_wait(q_bar(q_place - b), q_par(q_place - b), p.wait_ns, p.status, kStatusTimeoutAttnLoad);
            for (uint32_t b = 1; b <= kStages && b <= place; ++b)
                (void)mbar_wait(kv_bar(place - b), kv_par(place - b), p.wait_ns, p.status, kStatusTimeoutAttnLoad);
        } else if (warp == 1 || warp == 3) {
            // ------------------------------------------------------------ MMAs of query tile X
            const uint32_t X = uniform((uint32_t)warp >> 1);
            constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
            constexpr uint32_t kIdescO =
                (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (((uint32_t)DP >> 3) << 17) | ((128u >> 4) << 24);
            // Descriptors: the low word holds the address and the leading offset in units of 16
            // bytes, the high word is the same for all (stride 1024, 128-byte swizzle).
            constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29), kDescK = 1u << 16, kDescV = 1024u << 16;
            auto desc = [](uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; };
            constexpr uint32_t kTile16 = L::kTile >> 4;
            const uint32_t sq = smem_u32(smem) >> 4, skv = sq + (L::kKvOff >> 4);
            const uint32_t tmS = uniform(tmem + kTmS + 128 * X), tmO = uniform(tmem + kTmO + DP * X);
            // Each branch costs a lone warp some 25 cycles, so what belongs to a tile has few:
            // instructions of the elected lane are predicated, a wait that ran out is looked
            // at once per tile.
            const uint32_t on = elect_one() ? 1u : 0u;
            Piece cur, nxt;
            uint32_t q_place = 0, place = 0, gaps = 0;  // of cur: first places of Q, of K and V; gap tiles before it
            uint32_t p_phase = 0, o_phase = 1, t_phase = X ^ 1u;
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok &= mbar_wait(bar, parity, p.wait_ns, p.status, kStatusTimeoutAttnMma);
            };
            // S = Q K_i^T of a unit whose places begin at qp and pl, in two steps: what it waits
            // for, and the products.  `last`: the unit's last for X.
            auto wait_s = [&](uint32_t qp, uint32_t pl, int i) {
                const uint32_t at = pl + (uint32_t)k_place<kSolo>(tile_at<kSolo>(X, i));
                if (i == 0) wait(q_bar(qp + (kSolo ? 0u : X)), q_par(qp + (kSolo ? 0u : X)));
                wait(kv_bar(at), kv_par(at));
            };
            auto issue_s = [&](uint32_t go, uint32_t qp, uint32_t pl, int i, bool last, uint32_t pass_turn) {
                const uint32_t st = (pl + (uint32_t)k_place<kSolo>(tile_at<kSolo>(X, i))) % kStages;
                const uint32_t qs = (qp + (kSolo ? 0u : X)) % L::kQ;
                const uint32_t q = uniform(kDescK + sq + qs * kTile16), k = uniform(kDescK + skv + st * kTile16);
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) {
                    // the other warp's products queue up behind the rest of these
                    if (c == DP / 32) mbar_arrive_if(pass_turn, &turn[X ^ 1u]);
                    const uint32_t o = (c >> 2) * 1024 + (c & 3) * 2;
                    mma_f16_ss(go, tmS, desc(q + o), desc(k + o), kIdescS, c > 0);
                }
                tc_commit_if(go, &s_full[X]);
                tc_commit_if(go, &kv_empty[st]);
                tc_commit_if(go & (uint32_t)last, &q_empty[qs]);
            };
            // A unit that has nothing for X: its places are given back as they fill.
            auto pass = [&](const Piece& u) {
                if (kSolo) {  // Q is the other warp's alone
                    const uint32_t qs = q_place % L::kQ;
                    wait(q_bar(q_place), q_par(q_place));
                    mbar_arrive_if(on, &q_empty[qs]);
                } else {
                    for (uint32_t at = place; __all_sync(0xffffffffu, ok) && at < place + 2 * (uint32_t)u.nt; ++at) {
                        const uint32_t st = at % kStages;
                        wait(kv_bar(at), kv_par(at));
                        mbar_arrive_if(on, &kv_empty[st]);
                    }
                }
            };
            // Only one piece is read ahead, with keys or not: warp 2 may be waiting for this unit's
            // tiles before it describes more than a few.
            bool have = next_piece(cur, ok, kStatusTimeoutAttnMma), begun = false;
            while (have && __all_sync(0xffffffffu, ok)) {
                const int n = tiles_for<kSolo>(cur, X, tok);
                // turns of a unit: none where B has no tile, else A's (B passes on what it has not)
                const int turns = tiles_for<kSolo>(cur, 1, tok) > 0 ? tiles_for<kSolo>(cur, 0, tok) : 0;
                if (n > 0 && !begun) {
                    wait_s(q_place, place, 0);
                    tc_fence_after();
                    issue_s(on, q_place, place, 0, n == 1, 0);
                }
                const uint32_t next_place = place + 2 * (uint32_t)cur.nt;
                const uint32_t next_q = q_place + (cur.nt == 0 ? 0u : !kSolo && cur.ntok > tok ? 2u : 1u);
                have = next_piece(nxt, ok, kStatusTimeoutAttnMma);
                const int n_next = have ? tiles_for<kSolo>(nxt, X, tok) : 0;
                begun = n > 0 && n_next > 0;
                if (n > 0) wait(&o_empty[X], o_phase);
                o_phase ^= (uint32_t)(n > 0);
                for (int i = 0; i < n && __all_sync(0xffffffffu, ok); ++i) {
                    // Everything but P is waited for while the softmax works on it.
                    const int t = tile_at<kSolo>(X, i);
                    const uint32_t at = place + (uint32_t)v_place<kSolo>(t, cur.nt), st = at % kStages;
                    const bool last = i == n - 1, more = !last || n_next > 0;
                    const uint32_t s_q = last ? next_q : q_place, s_place = last ? next_place : place;
                    const int s_i = last ? 0 : i + 1;
                    const uint32_t v = uniform(kDescV + skv + st * kTile16);
                    wait(kv_bar(at), kv_par(at));
                    if (cur.has_gaps(cur.t0 + t)) {
                        const uint32_t g = gaps + cur.gaps_before(cur.t0 + t);
                        wait(&zero_full[g % kMaskSlots], (g / kMaskSlots) & 1u);
                    }
                    if (more) wait_s(s_q, s_place, s_i);
                    wait(&p_half[X], p_phase);
                    // The two warps take turns: were their MMAs mixed, both tiles' would end at the
                    // same time and both softmaxes run while the tensor cores stand idle.
                    if (turns > 0) {
                        wait(&turn[X], t_phase);
                        t_phase ^= 1u;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        mma_f16_ts(on, tmO, tmS + 8 * c, desc(v + c * 128), kIdescO, c > 0 ? 1u : (uint32_t)(i > 0));
                    wait(&p_full[X], p_phase);
                    p_phase ^= 1u;
                    tc_fence_after();
#pragma unroll
                    for (int c = 4; c < 8; ++c) mma_f16_ts(on, tmO, tmS + 8 * c, desc(v + c * 128), kIdescO, 1u);
                    tc_commit_if(on, &kv_empty[st]);
                    tc_commit_if(on & (uint32_t)last, &o_full[X]);
                    issue_s(on & (uint32_t)more, s_q, s_place, s_i, last ? n_next == 1 : i + 2 == n,
                            on & (uint32_t)(turns > 0));
                }
                if (n == 0 && cur.nt > 0) pass(cur);
                for (int i = n; i < turns && __all_sync(0xffffffffu, ok); ++i) {
                    wait(&turn[X], t_phase);
                    t_phase ^= 1u;
                    mbar_arrive_if(on, &turn[X ^ 1u]);
                }
                gaps += cur.gaps_before(cur.t0 + cur.nt);
                q_place = next_q;
                place = next_place;
                cur = nxt;
            }
            // All MMAs are done before TMEM and shared memory go.
            tc_commit_if(on, &done[X]);
            (void)mbar_wait(&done[X], 0, p.wait_ns, p.status, kStatusTimeoutAttnMma);
        } else if (warp == 2) {
            // ------------------------------------------------------------ keys that are left out
            uint32_t described = 0;
            bool ok = true, left = true;
            int ctx_keep = -1, own_keep = 0, own_entry = -1;
            // Key tiles up to the last key that a mask of n bytes keeps. One tile after the other,
            // 0.3 us each, in every CTA: a long tail costs more than its tiles would, spread over
            // all CTAs (one row over 32768 keys: 32 us without a mask, 34 with all kept, 101 with
            // 1000 kept; 1024 rows over 4096: 58 with all kept, 51 with half).
            auto kept_tiles = [&](const uint8_t* mask, int n) {
                int tile = (n + kKeyTile - 1) / kKeyTile;
                for (bool some = false; tile > 0 && !some; tile -= some ? 0 : 1) {
                    bool on = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = (tile - 1) * kKeyTile + 32 * j + lane;
                        on |= k < n && mask[k] != 0;
                    }
                    some = __any_sync(0xffffffffu, on);
                }
                return tile;
            };
            auto describe = [&]() {  // the next piece, or that there is none
                if (!left) return;
                const uint32_t slot = described % kPieceSlots;
                ok &= mbar_wait(&piece_empty[slot], ((described / kPieceSlots) & 1u) ^ 1u, p.wait_ns, p.status,
                                kStatusTimeoutAttnMask);
                Piece n;
                left = __all_sync(0xffffffffu, ok) && walk.next(n);
                if (left && (p.ctx_mask != nullptr || p.key_mask != nullptr)) {
                    // Tiles behind the last key that a mask keeps are left out (padded prompts).
                    if (p.ctx_mask != nullptr && ctx_keep < 0) ctx_keep = kept_tiles(p.ctx_mask, p.C);
                    if (p.key_mask != nullptr && n.e < p.t.nseg && n.e != own_entry) {
                        own_entry = n.e;
                        own_keep = kept_tiles(p.key_mask + n.kv0, n.kv_len);
                    }
                    trim_piece(n, p.ctx_mask != nullptr ? min(n.ctx_tiles, ctx_keep) : n.ctx_tiles,
                               p.key_mask != nullptr && n.e < p.t.nseg ? own_keep : n.own_tiles);
                }
                if (lane == 0) {
                    int4* rec = reinterpret_cast<int4*>(smem + L::kPieceOff + slot * 48);
                    rec[0] = make_int4(n.t0, left ? n.nt : -1, n.ntok, n.tok0);
                    rec[1] = make_int4(n.head0, n.ctx_tiles, n.kv0, n.kv_len);
                    rec[2] = make_int4(n.whole ? -1 : n.slot, n.e, 0, 0);
                    mbar_arrive(&piece_full[slot]);
                }
                __syncwarp();
                ++described;
            };
#pragma unroll 1
            for (int i = 0; i < kPieceSlots - 1; ++i) describe();
            Piece u;
            uint32_t place = 0, gaps = 0;
            while (next_piece(u, ok, kStatusTimeoutAttnMask)) {
                describe();
                for (int i = 0; i < u.nt && ok; ++i) {
                    const int t = u.t0 + i;
                    if (!u.has_gaps(t)) continue;
                    const uint32_t at = place + (uint32_t)v_place<kSolo>(i, u.nt), st = at % kStages;
                    const uint32_t slot = gaps % kMaskSlots, par = (gaps / kMaskSlots) & 1u;
                    // Once the V tile's load is issued, its stage was free, so the mask slot's last
                    // readers are through too: the ring holds fewer V tiles than there are slots.
                    ok &= mbar_wait(&gap_load[slot], par, p.wait_ns, p.status, kStatusTimeoutAttnMask);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const bool ctx = t < u.ctx_tiles;
                    const uint8_t* mask = ctx ? p.ctx_mask : p.key_mask;
                    const long long first = ctx ? t * kKeyTile : u.kv0 + (long long)(t - u.ctx_tiles) * kKeyTile;
                    const int n = min(kKeyTile, ctx ? p.C - t * kKeyTile : u.kv_len - (t - u.ctx_tiles) * kKeyTile);
                    bool keep[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        keep[j] = 32 * j + lane < n && (mask == nullptr || mask[first + 32 * j + lane] != 0);
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = __ballot_sync(0xffffffffu, keep[j]);
                    if (lane == 0) {
                        *reinterpret_cast<uint4*>(mask_bits + 4 * slot) = make_uint4(w[0], w[1], w[2], w[3]);
                        mbar_arrive(&mask_full[slot]);
                    }
                    __syncwarp();
                    ok = mbar_wait(kv_bar(at), kv_par(at), p.wait_ns, p.status, kStatusTimeoutAttnMask);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    // zeros, eight lanes to a row of a chunk and four rows at a time
                    uint8_t* v = smem + L::kKvOff + st * L::kTile + lane * 16;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (w[j] == 0xffffffffu) continue;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (!((w[j] >> (4 * k + (lane >> 3))) & 1u))
#pragma unroll
                                for (int c = 0; c < kChunks; ++c)
                                    *reinterpret_cast<uint4*>(v + c * 16384 + (8 * j + k) * 512) =
                                        make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&zero_full[slot]);
                    ++gaps;
                }
                place += 2 * (uint32_t)u.nt;
            }
        }
    } else if (warp < 12) {
        // ---------------------------------------------------------------- softmax of tile X
        setmaxnreg_inc<kRegsSoftmax>();
        const int X = (warp - 4) >> 2, quarter = warp & 3;
        const int row = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t tS = tmem + kTmS + 128 * X + lanes, tO = tmem + kTmO + DP * X + lanes;
        const uint64_t sl2 = f2(p.scale_log2, p.scale_log2);
        Piece u;
        uint32_t s_phase = 0, stat_phase = 1, gaps = 0;
        bool ok = true;
        while (next_with_keys(u, ok, kStatusTimeoutAttnSoftmax)) {
            const int n = tiles_for<kSolo>(u, X, tok);
            const int rows = min(tok, u.ntok - (kSolo ? 0 : X * tok)) * p.t.pack;
            const bool work = 32 * quarter < rows;   // some row of this warp is a query
            float m = -INFINITY, l = 0.0f;
            for (int i = 0; i < n && __all_sync(0xffffffffu, ok); ++i) {
                ok &= mbar_wait(&s_full[X], s_phase, p.wait_ns, p.status, kStatusTimeoutAttnSoftmax);
                s_phase ^= 1u;
                tc_fence_after();
                if (work) {
                    const int t = u.t0 + tile_at<kSolo>(X, i);
                    if (u.has_gaps(t)) {
                        // -inf over the scores of the keys that are left out
                        const uint32_t g = gaps + u.gaps_before(t);
                        ok &= mbar_wait(&mask_full[g % kMaskSlots], (g / kMaskSlots) & 1u, p.wait_ns, p.status,
                                        kStatusTimeoutAttnSoftmax);
                        __syncwarp();
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t w = mask_bits[4 * (g % kMaskSlots) + c];
                            if (w == 0xffffffffu) continue;
                            uint32_t s[32];
                            tc_ld_32x32b_x32(tS + 32 * c, s);
                            tc_wait_ld_x32(s);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!((w >> j) & 1u)) s[j] = 0xFF800000u;
                            tc_st_32x32b_x32(tS + 32 * c, s);
                        }
                        tc_wait_st();
                    }
                    uint32_t s[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc_ld_32x32b_x32(tS + 32 * c, s[c]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc_wait_ld_x32(s[c]);
                    float top[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        top[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
                        for (int j = 2; j < 32; j += 2)
                            top[c] = max3(top[c], __uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1]));
                    }
                    const float m_new = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
                    if (__any_sync(0xffffffffu, row < rows && m_new > m + p.growth)) {
                        const float f = m_new == m ? 1.0f : ex2_approx_ftz((m - m_new) * p.scale_log2);
                        l *= f;
                        m = m_new;
                        if (i > 0) {  // S_X(i) is computed, so the MMAs into O_X before it are done
                            const uint64_t ff = f2(f, f);
#pragma unroll 1
                            for (int c = 0; c < DP / 16; ++c) {
                                uint32_t o[16];
                                tc_ld_32x32b_x16(tO + 16 * c, o);
                                tc_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; j += 2) {
                                    float a, b;
                                    unf2(mul2(f2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])), ff), a, b);
                                    o[j] = __float_as_uint(a);
                                    o[j + 1] = __float_as_uint(b);
                                }
                                tc_st_32x32b_x16(tO + 16 * c, o);
                            }
                        }
                    }
                    const float base = m == -INFINITY ? 0.0f : -m * p.scale_log2;
                    const uint64_t base2 = f2(base, base);
                    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float a, b;
                            unf2(fma2(f2(__uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1])), sl2, base2), a, b);
                            const uint64_t e = f2(ex2_approx_ftz(a), ex2_approx_ftz(b));
                            sum[(j >> 1) & 3] = add2(sum[(j >> 1) & 3], e);
                            w[j >> 1] = cvt_bf16x2(e);
                        }
                        tc_st_32x32b_x16(tS + 16 * c, w);
                        if (c == 1) {
                            tc_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            mbar_arrive_if(lane == 0, &p_half[X]);
                        }
                    }
                    float a, b;
                    unf2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
                    l += a + b;
                    tc_wait_st();
                } else {
                    mbar_arrive_if(lane == 0, &p_half[X]);
                }
                tc_fence_before();
                __syncwarp();
                mbar_arrive_if(lane == 0, &p_full[X]);
            }
            gaps += u.gaps_before(u.t0 + u.nt);
            if (n > 0) {
                ok &= mbar_wait(&stat_empty[X], stat_phase, p.wait_ns, p.status, kStatusTimeoutAttnSoftmax);
                stat_phase ^= 1u;
                stat[128 * X + row] = make_float2(m, l);
                __syncwarp();
                mbar_arrive_if(lane == 0, &stat_full[X]);
            }
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        setmaxnreg_dec<kRegsEpilogue>();
        const int quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const int row_tok = row / p.t.pack, row_head = row - row_tok * p.t.pack;
        Piece u;
        uint32_t phase = 0;  // bit X: parity of the next O_X
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok &= mbar_wait(bar, parity, p.wait_ns, p.status, kStatusTimeoutAttnEpilogue);
        };
        while (next_piece(u, ok, kStatusTimeoutAttnEpilogue)) {
            const int tiles = !kSolo && u.ntok > tok ? 2 : 1;
            for (int Y = 0; Y < tiles; ++Y) {  // a tile of queries
                const uint32_t on = row < min(tok, u.ntok - Y * tok) * p.t.pack;
                const long long r = u.tok0 + Y * tok + row_tok;
                const int h = u.head0 + row_head;
                // Sums and statistics: O_Y; solo: O_A and O_B, of the even and the odd key tiles.
                const int nA = u.nt, nB = kSolo ? u.nt >> 1 : 0;
                const int X = kSolo ? 0 : Y;
                float2 a = make_float2(-INFINITY, 0.0f), b = a;
                if (nA > 0) {
                    wait(&stat_full[X], (phase >> X) & 1u);
                    wait(&o_full[X], (phase >> X) & 1u);
                    phase ^= 1u << X;
                    a = stat[128 * X + row];
                }
                if (kSolo && nB > 0) {
                    wait(&stat_full[1], (phase >> 1) & 1u);
                    wait(&o_full[1], (phase >> 1) & 1u);
                    phase ^= 2u;
                    b = stat[128 + row];
                }
                __syncwarp();
                mbar_arrive_if(lane == 0 && nA > 0, &stat_empty[X]);
                if (kSolo) mbar_arrive_if(lane == 0 && nB > 0, &stat_empty[1]);
                tc_fence_after();
                const float top = fmaxf(a.x, b.x), top2 = top * p.scale_log2;
                // weights of the two parts against the common maximum
                float f0 = 1.0f, f1 = 0.0f, sum = a.y;
                if (kSolo && nB > 0) {
                    f0 = a.x == top ? 1.0f : ex2_approx_ftz((a.x - top) * p.scale_log2);
                    f1 = b.x == top ? 1.0f : ex2_approx_ftz((b.x - top) * p.scale_log2);
                    sum = a.y * f0 + b.y * f1;
                }
                // Where a part has no key (or only scores of -inf), its sums may be anything.
                const bool clear = __any_sync(0xffffffffu, on && (a.y == 0.0f || (kSolo && nB > 0 && b.y == 0.0f)));
                const uint32_t tA = tmem + kTmO + DP * X + lanes, tB = tmem + kTmO + DP + lanes;
                // the sums of columns 32 c...; solo: of both parts, weighted
                auto load = [&](int c, uint32_t (&v)[32]) {
                    if (nA > 0) {
                        tc_ld_32x32b_x32(tA + 32 * c, v);
                        tc_wait_ld_x32(v);
                        if (clear) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = a.y == 0.0f ? 0u : v[j];
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0u;
                    }
                    if (kSolo && nB > 0) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t w[16];
                            tc_ld_32x32b_x16(tB + 32 * c + 16 * k, w);
                            tc_wait_ld_x16(w);
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float x = clear && b.y == 0.0f ? 0.0f : __uint_as_float(w[j]);
                                v[16 * k + j] = __float_as_uint(fmaf(x, f1, __uint_as_float(v[16 * k + j]) * f0));
                            }
                        }
                    }
                };
                // a row without a key: zeros (scores past fp32's range leave no sum either: NaN)
                const bool none = sum == 0.0f && top == -INFINITY;
                const float inv = none ? 0.0f : rcp_approx(sum);
                const uint64_t f = f2(inv, inv);
                const int kind = u.e < p.t.nseg ? 0 : 1, rows = p.slot_rows[kind];
                float* base = p.part[kind] + (long long)u.slot * rows * (DP + 2);
                const int at = Y * tok * p.t.pack + row;
                float* part = base + 4 * at;
                __nv_bfloat16* o = p.out + r * p.out_row + (long long)h * p.out_head;
                if (on && !u.whole)
                    *reinterpret_cast<float2*>(base + (long long)rows * DP + 2 * at) =
                        make_float2(none ? -INFINITY : top2, sum);
                if (on && u.whole && p.lse)
                    p.lse[r * p.Hq + h] = none ? -INFINITY : (top2 + __log2f(sum)) * 0.69314718055994531f;
                auto release = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_if(lane == 0 && nA > 0, &o_empty[X]);
                    if (kSolo) mbar_arrive_if(lane == 0 && nB > 0, &o_empty[1]);
                };
                if (32 * quarter >= min(tok, u.ntok - Y * tok) * p.t.pack) {
                    release();  // none of this warp's rows is a query
                } else if (!kSolo && u.whole && p.wide_out && nA > 0 && !clear) {
                    // The usual case of the pair plan, whose next unit waits for these sums to be read.
#pragma unroll 1
                    for (int c = 0; c < DP / 32; ++c) {
                        uint32_t v[32];
                        tc_ld_32x32b_x32(tA + 32 * c, v);
                        tc_wait_ld_x32(v);
                        store_bf16(on, o + 32 * c, v, f, p.D - 32 * c, true);
                    }
                    release();
                } else {
                    // A loop and not straight code: it runs once per unit, when its instructions have
                    // left the caches; fetching them costs more than the branches.
#pragma unroll 1
                    for (int c = 0; c < DP / 32; ++c) {
                        uint32_t v[32];
                        load(c, v);
                        if (u.whole) {
                            store_bf16(on, o + 32 * c, v, f, p.D - 32 * c, p.wide_out != 0);
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) st_global_v4_if(on, part + (long long)(8 * c + j) * 4 * rows, v + 4 * j);
                        }
                    }
                    release();
                }
            }
        }
    }
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ joining partial sums
//
// With m_i (base 2) and l_i of a row's partials and m the largest m_i,
//     out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
// A partial holds its sums as [DP / 4][rows][4], so that both the attention's
// threads, a row each, and those here, a row and eight columns each, read and
// write whole lines; `shift` rows (log2) are side by side here, fewer than 32
// where a unit has fewer.  Bound by latency (8 units of 4 rows in 19 parts or so:
// 7 us by itself; 96 units of 256 rows in 2 or 3 parts: 10 us): kJoinAtOnce
// partials are read at once (8: 1 us slower on 512 to 2048 rows over 2048 keys).
// Ordinary loads: the attention kernel may still be writing when this one starts,
// and a read-only load could be moved above the wait for it.
constexpr int kJoinThreads = 256;
constexpr int kJoinAtOnce = 4;

struct JoinOut {
    __nv_bfloat16* out;
    long long out_row, out_head;
    float* lse;
    const float* part[2];
    int slot_rows[2];
    int D, Hq, pack;
    int shift;
};

// A row's sums from column col on, and its statistics, in one slot.
template <int DP>
struct JoinAt {
    const float4* o;
    const float2* ml;
    long long rows;
    __device__ __forceinline__ JoinAt(const JoinOut& p, int kind, int slot, int row, int col) : rows(p.slot_rows[kind])
    {
        const float* base = p.part[kind] + slot * rows * (DP + 2);
        o = reinterpret_cast<const float4*>(base) + (col >> 2) * rows + row;
        ml = reinterpret_cast<const float2*>(base + rows * DP) + row;
    }
};

// Columns col... of row r, head h: the partial `own`, and `others` more from
// `rest` on, `apart` slots from one to the next.
template <int DP>
__device__ __forceinline__ void join_row(const JoinOut& p, int r, int h, int col, const JoinAt<DP>& own,
                                         const JoinAt<DP>& rest, int others, int apart)
{
    const long long step = apart * rest.rows * (DP + 2);  // floats, a multiple of 4 (rows are even)
    const int all = 1 + others;
    float acc[8], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    for (int first = 0; first < all; first += kJoinAtOnce) {
        float2 ml[kJoinAtOnce];
        float4 lo[kJoinAtOnce], hi[kJoinAtOnce];
#pragma unroll
        for (int i = 0; i < kJoinAtOnce; ++i) {
            ml[i] = make_float2(-INFINITY, 0.0f);
            lo[i] = hi[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i == 0 && first == 0) {
                ml[i] = *own.ml;
                lo[i] = own.o[0];
                hi[i] = own.o[own.rows];
            } else if (first + i < all) {
                const long long off = (first + i - 1) * step;
                const float4* o = rest.o + (off >> 2);
                ml[i] = rest.ml[off >> 1];
                lo[i] = o[0];
                hi[i] = o[rest.rows];
            }
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kJoinAtOnce; ++i) top = fmaxf(top, ml[i].x);
        const float f = m == top ? 1.0f : ex2_approx_ftz(m - top);
        m = top;
        l *= f;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] *= f;
#pragma unroll
        for (int i = 0; i < kJoinAtOnce; ++i) {
            // a partial without a key counts nothing, whatever its sums are
            const bool some = ml[i].x != -INFINITY;
            const float w = !some ? 0.0f : ml[i].x == m ? 1.0f : ex2_approx_ftz(ml[i].x - m);
            const float v[8] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w, hi[i].x, hi[i].y, hi[i].z, hi[i].w};
            l = fmaf(ml[i].y, w, l);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = some ? fmaf(v[j], w, acc[j]) : acc[j];
        }
    }
    const bool none = l == 0.0f && m == -INFINITY;
    const float inv = none ? 0.0f : rcp_approx(l);
    if (col < p.D)  // D is a multiple of 8
        *reinterpret_cast<uint4*>(p.out + (long long)r * p.out_row + (long long)h * p.out_head + col) =
            make_uint4(cvt_bf16x2(f2(acc[0] * inv, acc[1] * inv)), cvt_bf16x2(f2(acc[2] * inv, acc[3] * inv)),
                       cvt_bf16x2(f2(acc[4] * inv, acc[5] * inv)), cvt_bf16x2(f2(acc[6] * inv, acc[7] * inv)));
    if (p.lse && col == 0)
        p.lse[(long long)r * p.Hq + h] = none ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}

// This thread's row of the block's unit, and its first column.
template <int DP>
__device__ __forceinline__ int join_place(int shift, int& col)
{
    const int i = blockIdx.y * kJoinThreads + threadIdx.x, group = i >> shift;
    col = group % (DP / 8) * 8;
    return (group / (DP / 8) << shift) + (i & ((1 << shift) - 1));
}

// The cut units of the pool: blocks (i, y) take the rows of cut i.
struct JoinCuts {
    JoinOut o;
    int lanes;
    Cut cuts[kAttnCtas];
};

template <int DP>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ JoinCuts p)
{
    const Cut c = p.cuts[blockIdx.x];
    int col;
    const int at = join_place<DP>(p.o.shift, col), tk = at / p.o.pack;
    griddep_wait();
    griddep_launch_dependents();
    if (at >= c.rows) return;
    // (slots: cut_slot() of the CTAs that hold the unit's pieces, of which the first begins it)
    join_row<DP>(p.o, c.tok0 + tk, c.head0 + at - tk * p.o.pack, col, JoinAt<DP>(p.o, 0, cut_slot(c.cta, true), at, col),
                 JoinAt<DP>(p.o, 0, cut_slot(c.cta + p.lanes, false), at, col), c.parts - 1, 2 * p.lanes);
}

// The separate plan: a row's own keys are one partial, the context's as many as its unit
// was cut into.  Blocks take the rows (pack heads of a token side by side) of a head block
// one after the other, whatever their segments: a block per segment's unit, each looking
// for its place in the plan, took 36 us for 2400 units of 400 rows and 12 us for 480.
template <int DP>
__global__ void __launch_bounds__(kJoinThreads)
    attn_join_separate_kernel(const __grid_constant__ JoinOut o, const __grid_constant__ AttnTable t, int groups)
{
    constexpr int kRows = kJoinThreads / (DP / 8);
    __shared__ int q_off[H3FP4_ATTN_MAX_SEGMENTS + 1];
    for (int i = threadIdx.x; i <= t.nseg; i += kJoinThreads) q_off[i] = t.q_off[i];
    __syncthreads();
    const int hb = blockIdx.x / groups;
    const int col = threadIdx.x / kRows * 8;
    const long long at = (long long)(blockIdx.x - hb * groups) * kRows + threadIdx.x % kRows;
    const int r = (int)(at / t.pack), head = (int)(at - (long long)r * t.pack);
    int own = 0, own_at = 0, first = 0, parts = 0, in = 0;
    if (r < t.M) {
        int e = 0, end = t.nseg;
        while (end - e > 1) {
            const int mid = (e + end) >> 1;
            if (q_off[mid] <= r) e = mid;
            else end = mid;
        }
        const int local = r - q_off[e], rb = local / t.unit_tok;
        own = t.pool_unit[e] + hb * t.row_blocks(e) + rb;
        own_at = (local - rb * t.unit_tok) * t.pack + head;
        const int ce = t.nseg, cn = t.steps(ce), block = r / t.unit_tok, cu = hb * t.row_blocks(ce) + block;
        const int begin = t.pool_step[ce] + cu * cn;
        first = t.stretch_of(begin);
        parts = t.stretch_of(begin + cn - 1) - first + 1;
        first += cu;
        in = (r - block * t.unit_tok) * t.pack + head;
    }
    griddep_wait();
    griddep_launch_dependents();
    if (r >= t.M) return;
    join_row<DP>(o, r, hb * t.pack + head, col, JoinAt<DP>(o, 0, own, own_at, col), JoinAt<DP>(o, 1, first, in, col),
                 parts, 1);
}

// ------------------------------------------------------------------ host side

// bf16 [rows][heads][D] as a tensor map with boxes of 64 columns x `heads_box` x `rows_box`.
bool make_heads_map(CUtensorMap* map, const HeadsIn& x, int64_t rows, int heads, int D, int heads_box, int rows_box)
{
    EncodeTiledFn fn = get_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)x.head * 2, (cuuint64_t)x.row * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)rows_box};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(x.p), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, bool kSolo>
cudaError_t run(const AttnPlan& pl, const CUtensorMap (&m)[5], const AttnParams& p, cudaStream_t s)
{
    auto kernel = attn_kernel<DP, kSolo>;
    constexpr uint32_t bytes = Layout<DP, kSolo>::kBytes;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), (int)bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)pl.t.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], m[2], m[3], m[4], p);
    if (e != cudaSuccess || !pl.join) return e;
    JoinOut o{p.out, p.out_row, p.out_head, p.lse, {p.part[0], p.part[1]}, {p.slot_rows[0], p.slot_rows[1]},
              p.D, p.Hq, pl.t.pack, 0};
    while (o.shift < 5 && (1 << o.shift) < pl.slot_rows[0]) ++o.shift;
    const int groups = (pl.slot_rows[0] + (1 << o.shift) - 1) >> o.shift;
    const unsigned blocks = (unsigned)(((groups << o.shift) * (DP / 8) + kJoinThreads - 1) / kJoinThreads);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    if (pl.t.separate) {
        const int rows = kJoinThreads / (DP / 8);
        const int per_head = (int)(((long long)pl.t.M * pl.t.pack + rows - 1) / rows);
        cfg.gridDim = dim3((unsigned)per_head * (unsigned)pl.t.head_blocks);
        return cudaLaunchKernelEx(&cfg, attn_join_separate_kernel<DP>, o, p.t, per_head);
    }
    JoinCuts cuts;
    cuts.o = o;
    cuts.lanes = pl.t.lanes;
    std::memcpy(cuts.cuts, pl.cuts, sizeof(cuts.cuts));
    cfg.gridDim = dim3((unsigned)pl.n_cuts, blocks);
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<DP>, cuts);
}

}  // namespace

cudaError_t launch_attn(const AttnJob& job, const AttnPlan& pl, cudaStream_t s)
{
    AttnParams p{};
    p.t = pl.t;
    p.t.own_masked = job.key_mask != nullptr;
    p.t.ctx_masked = job.ctx_mask != nullptr;
    p.Hq = job.Hq;
    p.group = job.Hq / job.Hkv;
    p.D = job.D;
    p.T = (int)job.T;
    p.C = (int)job.C;
    p.key_mask = job.key_mask;
    p.ctx_mask = job.ctx_mask;
    p.scale_log2 = job.scale * kLog2E;
    p.growth = fminf(kGrowth / p.scale_log2, 1e38f);  // finite: -inf plus it stays -inf
    p.out = job.out;
    p.out_row = job.out_row;
    p.out_head = job.out_head;
    p.wide_out = job.D % 16 == 0 && job.out_row % 16 == 0 && job.out_head % 16 == 0 &&
                 (reinterpret_cast<uintptr_t>(job.out) & 31u) == 0;
    p.lse = job.lse;
    for (int k = 0; k < 2; ++k) {
        p.part[k] = reinterpret_cast<float*>(job.ws + pl.slot_off[k]);
        p.slot_rows[k] = pl.slot_rows[k];
    }
    p.status = reinterpret_cast<unsigned int*>(job.ws + kWsStatus);
    p.wait_ns = attn_wait_ns(pl.t, job.wait_limit_ns);
    p.stall = job.stall;
    const int chunks = pl.dp / 64;
    p.q_bytes = (uint32_t)(chunks * 128 * pl.t.pack * pl.t.tok);
    CUtensorMap m[5] = {};
    if (!make_heads_map(&m[0], job.q, job.M, job.Hq, job.D, pl.t.pack, pl.t.tok)) return cudaErrorInvalidValue;
    if (job.T > 0 && (!make_heads_map(&m[1], job.k, job.T, job.Hkv, job.D, 1, kKeyTile) ||
                      !make_heads_map(&m[2], job.v, job.T, job.Hkv, job.D, 1, kKeyTile)))
        return cudaErrorInvalidValue;
    if (job.C > 0 && (!make_heads_map(&m[3], job.kc, job.C, job.Hkv, job.D, 1, kKeyTile) ||
                      !make_heads_map(&m[4], job.vc, job.C, job.Hkv, job.D, 1, kKeyTile)))
        return cudaErrorInvalidValue;
    if (pl.dp == 64) return pl.solo ? run<64, true>(pl, m, p, s) : run<64, false>(pl, m, p, s);
    return pl.solo ? run<128, true>(pl, m, p, s) : run<128, false>(pl, m, p, s);
}

}  // namespace h3fp4
