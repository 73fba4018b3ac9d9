// How an attention call's work is cut into units, steps and pieces; plain
// arithmetic shared by the host (planning, workspace size) and the kernels.
//
// A tile of queries is 128 rows: `pack` query heads of one kv head times
// tok = 128 / pack tokens, so that all of them use the same K and V.  A unit is
// what one CTA works on at a time: two tiles of queries against the same keys
// (pair plan), or one tile whose even and odd key tiles go to the CTA's two
// softmax warpgroups (solo plan, for few units).  Its steps are the 128-key tiles
// it walks: first the shared context's, then its own segment's.
//
// An entry is a segment; with the separate plan (many short segments over a long
// context) the segments walk their own keys only, and one more entry walks the
// context for the rows of all segments together.
//
// Units are dealt out in two parts.  Of each entry, whole waves of `ctas` units
// go to the CTAs one by one; consecutive CTAs then read the same keys at the
// same time.  What is left over (the pool) is laid out as one row of steps and
// cut into equal stretches, one per CTA: a unit that is cut leaves partial sums
// that a second kernel joins.  A cut within kSnap steps of a unit's edge moves
// there, since a partial costs about as much as that many steps.  Where units as
// they are come out sooner than cut ones and the second kernel, none is cut.
//
// Few units of a head over keys that do not fit in L2: were they cut one after
// the other, the units of a head would walk the same keys at different times and
// each read them from memory.  There the pool holds one row of steps per head,
// and a stretch goes to `lanes` CTAs side by side, one per unit of the head
// (1024 rows over 30720 keys, 24 heads, caches flushed: 247 us against 282 when it
// came in, 244 now).
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/h3fp4.h"

namespace h3fp4 {

constexpr int kKeyTile = 128;
constexpr int kAttnCtas = 152;   // one per SM of the GB300; on a device with fewer the last ones run alone
// 2 and 8 measured 0 and 1 % slower on 16384 rows over 9216 keys, where a CTA has 728 steps.
// At few steps a CTA it makes stretches uneven (4500 ragged rows, 19 steps on average: the
// fullest CTA has 24 with it, 22 with 2); that was not timed.
constexpr int kSnap = 4;
// What a unit costs beside its tiles, in steps: one of the pair plan's, three of the solo
// plan's, which are about half as long; a unit without keys one more.  9001 masked rows over
// six prompts, one without keys (pair; unit and empty unit): 0 and 1 69 us, 0 and 2 72, 1 and
// 2 62, 1 and 3 68, 2 and 4 64.
constexpr int kPairUnitSteps = 1, kSoloUnitSteps = 3;
static_assert(kSoloUnitSteps < kSnap && kSoloUnitSteps + 1 <= 2 * kSnap, "cuts lie behind a unit's overhead");
constexpr int kAttnEntries = H3FP4_ATTN_MAX_SEGMENTS + 1;

__host__ __device__ inline int lesser(int a, int b) { return a < b ? a : b; }

struct AttnTable {
    int nseg, entries;     // entries = nseg (+ 1: the context's, separate plan)
    int ctas;
    int pack, tok;         // heads and tokens of a tile
    int unit_tok;          // tokens of a unit: 2 tok (pair) or tok (solo)
    int head_blocks;       // Hq / pack
    int ctx_tiles;         // key tiles of the context
    int separate;
    int uncut;             // no unit of the pool is cut
    int unit_steps;        // steps a unit counts beside its tiles
    int any_full;          // some entry has whole waves
    int ctx_masked, own_masked, ctx_ragged;  // masks are given; the context's length is no multiple of a tile
    int pool_steps;
    int lanes, stretches;  // CTAs side by side on a stretch of the pool, and stretches
    int share, longer;     // steps of a stretch: share + 1 for the first `longer` of them
    int M;
    int q_off[H3FP4_ATTN_MAX_SEGMENTS + 1];
    int kv_off[H3FP4_ATTN_MAX_SEGMENTS + 1];
    int pool_step[kAttnEntries + 1];   // steps of the pool before each entry
    int pool_unit[kAttnEntries + 1];   // units of the pool before each entry

    __host__ __device__ int q_begin(int e) const { return e < nseg ? q_off[e] : 0; }
    __host__ __device__ int q_end(int e) const { return e < nseg ? q_off[e + 1] : M; }
    // Key tiles of an entry: the context's share and all of them.
    __host__ __device__ int tiles_ctx(int e) const { return separate && e < nseg ? 0 : ctx_tiles; }
    __host__ __device__ int tiles_own(int e) const
    {
        return e < nseg ? (kv_off[e + 1] - kv_off[e] + kKeyTile - 1) / kKeyTile : 0;
    }
    __host__ __device__ int tiles(int e) const { return tiles_ctx(e) + tiles_own(e); }
    // Steps of a unit: its tiles, and what beginning and ending it costs; a unit
    // without keys still writes zeros.
    __host__ __device__ int steps_of(int tiles) const { return (tiles > 0 ? tiles : 1) + unit_steps; }
    __host__ __device__ int steps(int e) const { return steps_of(tiles(e)); }
    __host__ __device__ int row_blocks(int e) const { return (q_end(e) - q_begin(e) + unit_tok - 1) / unit_tok; }
    __host__ __device__ int units(int e) const { return head_blocks * row_blocks(e); }
    __host__ __device__ int full(int e) const { return any_full ? units(e) / ctas * ctas : 0; }

    // Largest i in [0, entries) with start[i] <= x.
    __host__ __device__ int find(const int* start, int x) const
    {
        int lo = 0, hi = entries;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    // Where stretch c of the pool begins.
    __host__ __device__ int bound(int c) const
    {
        const int x = c * share + lesser(c, longer);
        if (c <= 0 || c >= stretches || x <= 0 || x >= pool_steps) return x;
        const int last = entries - 1, e = x >= pool_step[last] ? last : find(pool_step, x);
        const int n = steps(e), t = (x - pool_step[e]) % n;
        // (a segment's unit of the separate plan is never cut)
        const int snap = uncut || (separate && e < nseg) ? n : kSnap;
        if (t <= snap && t <= n - t) return x - t;
        if (n - t <= snap) return x + n - t;
        return x;
    }
    // The stretch that holds step x of the pool.
    __host__ __device__ int stretch_of(int x) const
    {
        const int head = longer * (share + 1);
        int c = x < head ? x / (share + 1) : share > 0 ? longer + (x - head) / share : stretches - 1;
        while (c > 0 && bound(c) > x) --c;
        while (c + 1 < stretches && bound(c + 1) <= x) ++c;
        return c;
    }
};

// A stretch of the pool has at most two cut units: its first, begun by another
// CTA, and its last, which it begins itself.
__host__ __device__ inline int cut_slot(int cta, bool begins_unit) { return 2 * cta + (begins_unit ? 1 : 0); }

// A piece of a unit: key tiles [t0, t0 + nt) of it, for tokens [tok0, tok0 + ntok).
struct Piece {
    int e, head0, tok0, ntok;   // e: entry
    int t0, nt;
    int ctx_tiles;          // tiles below this index are the context's
    int own_tiles, kv0, kv_len;
    // set by find_gaps():
    bool gaps_ctx, gaps_own;  // every tile of that source has keys that may be left out (a mask)
    int gap_ctx, gap_own;     // else the tile whose end lies past the source's last key, or -1
    bool whole;             // all steps of the unit
    int slot;               // of the partial sums, if not whole (or separate plan)

    // own_tiles and the gap fields, from the others (the kernel's roles read a piece without them).
    __host__ __device__ void find_gaps(const AttnTable& t)
    {
        own_tiles = (kv_len + kKeyTile - 1) / kKeyTile;
        gaps_ctx = t.ctx_masked != 0;
        gaps_own = t.own_masked != 0;
        gap_ctx = t.ctx_ragged ? ctx_tiles - 1 : -1;  // -1 too where no tile is the context's
        gap_own = (kv_len & (kKeyTile - 1)) ? ctx_tiles + own_tiles - 1 : -1;
    }

    // Whether tile t of the unit has keys that are left out.
    __host__ __device__ bool has_gaps(int t) const
    {
        return t < ctx_tiles ? gaps_ctx || t == gap_ctx : gaps_own || t == gap_own;
    }
    // How many such tiles there are among [t0, t).
    __host__ __device__ int gaps_before(int t) const
    {
        const int c = lesser(t, ctx_tiles) - lesser(t0, ctx_tiles), o = t - t0 - c;
        return (gaps_ctx ? c : (int)(t0 <= gap_ctx && gap_ctx < t)) + (gaps_own ? o : (int)(t0 <= gap_own && gap_own < t));
    }
};

// Leaves out of a piece the tiles behind the last keys that masks keep: of its
// unit's ctx_tiles + own_tiles tiles the first ctx_keep and own_keep are walked.
// Tiles are then counted over what is left.
__host__ __device__ inline void trim_piece(Piece& p, int ctx_keep, int own_keep)
{
    const int all = p.ctx_tiles, gone = all - ctx_keep;
    auto moved = [&](int t) { return t <= ctx_keep ? t : t - gone > ctx_keep ? t - gone : ctx_keep; };
    const int end = moved(lesser(p.t0 + p.nt, all + own_keep));
    p.t0 = moved(p.t0);
    p.nt = end > p.t0 ? end - p.t0 : 0;
    p.ctx_tiles = ctx_keep;
}

// The pieces of this CTA, in order; one warp walks them for all roles.  Divisions
// are done where an entry begins; from piece to piece the state is counted up.
struct Walk {
    const AttnTable& t;
    int cta;
    int e, hb, rb, blocks;     // entry, head block and row block of the next unit; row blocks of the entry
    int step_hb, step_rb;      // whole waves: what `ctas` units further is, and the units in them
    int wave_end;
    int tile, left;            // pool: first tile of the next piece, steps left of the stretch
    bool waves;

    __host__ __device__ explicit Walk(const AttnTable& table) : t(table) {}
    __host__ __device__ void start(int c)
    {
        cta = c;
        left = 0;
        tile = 0;
        step_hb = step_rb = wave_end = 0;
        waves = t.any_full != 0;
        if (waves) begin_waves(0);
        else begin_pool();
    }
    __host__ __device__ void begin_waves(int entry)
    {
        for (; entry < t.entries; ++entry) {
            wave_end = t.full(entry);
            if (wave_end == 0) continue;
            e = entry;
            blocks = t.row_blocks(e);
            step_hb = t.ctas / blocks;
            step_rb = t.ctas - step_hb * blocks;
            hb = cta / blocks;
            rb = cta - hb * blocks;
            return;
        }
        waves = false;
        begin_pool();
    }
    __host__ __device__ void begin_pool()
    {
        hb = rb = e = 0;
        blocks = 1;
        if (t.pool_steps == 0) return;
        const int stretch = cta / t.lanes;
        if (stretch >= t.stretches) return;
        const int pos = t.bound(stretch);
        left = t.bound(stretch + 1) - pos;
        if (left <= 0) return;
        e = t.find(t.pool_step, pos);
        const int n = t.steps(e), local = pos - t.pool_step[e], u = local / n;
        tile = local - u * n;
        blocks = t.row_blocks(e);
        if (t.lanes > 1) {
            hb = u;
            rb = cta - stretch * t.lanes;
            return;
        }
        hb = (t.full(e) + u) / blocks;
        rb = t.full(e) + u - hb * blocks;
    }
    __host__ __device__ void fill(Piece& p) const
    {
        p.e = e;
        p.head0 = hb * t.pack;
        p.tok0 = t.q_begin(e) + rb * t.unit_tok;
        p.ntok = lesser(t.unit_tok, t.q_end(e) - p.tok0);
        p.ctx_tiles = t.tiles_ctx(e);
        p.own_tiles = t.tiles_own(e);
        p.kv0 = e < t.nseg ? t.kv_off[e] : 0;
        p.kv_len = e < t.nseg ? t.kv_off[e + 1] - p.kv0 : 0;
    }
    __host__ __device__ bool next(Piece& p)
    {
        if (waves) {
            fill(p);
            p.t0 = 0;
            p.nt = p.ctx_tiles + p.own_tiles;
            p.whole = true;
            p.slot = 0;
            // the last whole wave of an entry ends where fewer than ctas units are left
            rb += step_rb;
            hb += step_hb;
            if (rb >= blocks) {
                rb -= blocks;
                ++hb;
            }
            if (hb * blocks + rb >= wave_end) begin_waves(e + 1);
            return true;
        }
        if (left <= 0) return false;
        fill(p);
        const int tiles = p.ctx_tiles + p.own_tiles, n = t.steps_of(tiles);
        const int take = lesser(n - tile, left);
        // a unit's first steps are its overhead; cuts lie behind them
        p.t0 = tile > t.unit_steps ? tile - t.unit_steps : 0;
        p.nt = tiles > 0 ? tile + take - t.unit_steps - p.t0 : 0;
        p.whole = take == n && !t.separate;
        // With the separate plan every piece leaves partials: one for a segment's unit, those of the
        // context's numbered along the pool.
        p.slot = !t.separate ? cut_slot(cta, tile == 0)
                 : e < t.nseg ? t.pool_unit[e] + hb * blocks + rb
                              : hb * blocks + rb + cta;
        left -= take;
        tile = 0;
        if (t.lanes > 1) {
            ++hb;
        } else if (++rb == blocks) {
            rb = 0;
            if (++hb == t.head_blocks && left > 0) {
                do ++e;
                while (t.pool_step[e + 1] == t.pool_step[e]);
                blocks = t.row_blocks(e);
                const int u = t.full(e);
                hb = u / blocks;
                rb = u - hb * blocks;
            }
        }
        return true;
    }
};

// A unit of the pool that is cut, the first CTA that holds a piece, and how many do
// (each `lanes` after the one before).
struct Cut {
    int tok0, head0, rows, cta, parts;
};

struct AttnPlan {
    AttnTable t;
    Cut cuts[kAttnCtas];
    int n_cuts;
    bool solo;
    bool join;           // partial sums exist: the second kernel runs
    int dp;              // D padded to 64 or 128
    int slot_rows[2];    // rows of a partial: segments' units, the context entry's
    long long slots[2];  // partials of each kind
    size_t slot_off[2];  // byte offsets in the workspace
    size_t bytes;        // workspace; 0: more steps than 32 bits count
};

// The limit of one device wait of a call with this table, from the limit that is
// set.  Some waits last as long as their unit does, not a step: the epilogue's for
// a unit's sums, those of a role that has nothing in it, and of all roles while a
// mask's end is looked for.  Four units may lie between (the pieces described
// ahead); a tile takes 1.6 us at most and 0.7 us to look for, so 20 us per tile of
// the longest unit are twice what they add up to.  A fixed limit ran out at units
// of 1.2 million tiles with the default of 2 s, and sooner with a lower one.
constexpr uint64_t kWaitNsPerTile = 20000;
inline uint64_t attn_wait_ns(const AttnTable& t, uint64_t limit_ns)
{
    uint64_t longest = 0;
    for (int e = 0; e < t.entries; ++e)
        if (t.row_blocks(e) > 0 && (uint64_t)t.tiles(e) > longest) longest = (uint64_t)t.tiles(e);
    const uint64_t more = longest * kWaitNsPerTile;
    return limit_ns > UINT64_MAX - more ? UINT64_MAX : limit_ns + more;
}

// Units, tiles of all of them and of the longest, for one choice of pack and of solo or
// pair units: with the segments' units walking the context too, and with it apart;
// the bytes of the context's keys that its units walk then.
struct Cost {
    double units, tiles, longest, units_apart, tiles_apart, ctx_bytes;
};

template <class Job>
inline Cost cost_of(const Job& job, const AttnTable& t, int pack, bool solo)
{
    const int tok = 128 / pack, unit_tok = solo ? tok : 2 * tok;
    const long long ctx = t.ctx_tiles;
    long long units = 0, tiles = 0, longest = 0, own = 0;
    for (int e = 0; e < t.nseg; ++e) {
        const long long rb = (t.q_off[e + 1] - t.q_off[e] + unit_tok - 1) / unit_tok, n = t.tiles_own(e);
        units += rb;
        tiles += rb * (ctx + n > 0 ? ctx + n : 1);
        own += rb * (n > 0 ? n : 1);
        if (rb > 0 && ctx + n > longest) longest = ctx + n;
    }
    const long long apart = (job.M + unit_tok - 1) / unit_tok, hb = job.Hq / pack;
    return Cost{(double)(hb * units), (double)hb * (double)tiles, (double)longest, (double)(hb * (units + apart)),
                (double)hb * (double)(own + apart * (ctx > 0 ? ctx : 1)),
                4.0 * job.D * (double)job.C * (double)(apart * hb)};
}

// The time of a plan in steps of a pair unit (1.35 us at heads of 128 in short calls, 1.6 in
// long ones): a tile of a solo unit takes 0.52, its ends 1.45 (a
// pair's 1); cutting costs a piece's end, the partials' way through memory and a second
// kernel, 13 us (pair) or 11 us (solo, half the rows).  Two things it leaves out: units of
// one to three tiles take longer than this counts (9001 rows over six prompts: 26 steps on
// the fullest CTA, 57 us), and whole units are dealt out by steps, so that where their
// lengths differ a CTA may hold two and another none (`dealt` counts one a wave): 5 and 4
// rows over 1647 and 2090 keys 26.5 us, over 2090 each 17.8.
// Measured, 24 heads of 128, bursts of calls back to back, us (the smallest is what is taken):
//     rows x keys      pair, cut   pair, whole   solo, cut   solo, whole
//     256 x 4096            26.9          50.4        22.6          29.9
//     512 x 2048            27.0          29.0        23.7          19.1
//     1024 x 2048           36.9          30.1        32.7          34.2
//     2048 x 2048           49.8          54.7        51.4          48.0
//     4096 x 512               -          28.7           -          36.7
//     4096 x 4096          137.5         144.7       147.8         158.7
//     1024 x 30720         237.5         336.8       247.5         361.6
// With the context apart (heads, rows a segment; cut):   pair, solo
//     32 over 8 of 128, 48 x 1 over 16384 keys           38.7, 36.2
//     24 of 128, 40 x 1 over 16384                       78.8, 63.7
//     24 of 64, 20 x 20 over 12000                       75.8, 78.9
//     24 of 128, 20 x 20 over 12000                      93.0, 120.9
// The last one's keys do not stay in L2 from one of a head's units to the next, and solo
// units are twice as many: hence the term with the bytes where all heads' keys exceed 96 MB
// (its two constants are fitted to that case alone).
struct PlanTime {
    double cut, whole, apart;
};

inline PlanTime time_of(const Cost& c, bool solo, double key_bytes)
{
    const double tile = solo ? 0.52 : 1.0, ends = solo ? 1.45 : 1.0, join = solo ? 8.0 : 10.0;
    const double all = tile * c.tiles + ends * c.units, unit = tile * c.longest + ends;
    double ctas = c.tiles / kSnap;
    if (ctas < c.units) ctas = c.units;
    if (ctas > kAttnCtas) ctas = kAttnCtas;
    const double waves = (double)(((long long)c.units + kAttnCtas - 1) / kAttnCtas);
    const double even = all / kAttnCtas + unit, dealt = waves * unit;
    double apart = tile * c.tiles_apart + (ends + 0.5) * c.units_apart;  // a partial of each unit
    if (key_bytes > 96.0 * 1024 * 1024) apart += kAttnCtas * c.ctx_bytes / 18e6;
    return PlanTime{ctas > 0 ? all / ctas + join : 0.0, dealt < even ? dealt : even,
                    apart / kAttnCtas + join};
}

template <class Job>
inline AttnPlan make_plan(const Job& job)
{
    AttnPlan pl;
    AttnTable& t = pl.t;
    pl.bytes = 0;
    pl.join = false;
    pl.n_cuts = 0;
    pl.slots[0] = pl.slots[1] = 0;
    pl.dp = job.D <= 64 ? 64 : 128;
    t.nseg = job.nseg;
    t.M = (int)job.M;
    t.ctx_tiles = (int)((job.C + kKeyTile - 1) / kKeyTile);
    t.ctx_ragged = job.C % kKeyTile != 0;
    t.ctx_masked = t.own_masked = 0;  // set at launch
    for (int i = 0; i <= job.nseg; ++i) {
        t.q_off[i] = (int)job.q_off[i];
        t.kv_off[i] = (int)job.kv_off[i];
    }
    // Heads of a kv group share a tile's keys; the largest pack with the fewest steps.
    const int group = job.Hq / job.Hkv;
    int pack = 1;
    double best = 0;
    for (int g = 1; g <= group && g <= 128; ++g) {
        if (group % g) continue;
        const double s = group == 1 ? 0 : cost_of(job, t, g, true).tiles;
        if (g == 1 || s <= best) {
            best = s;
            pack = g;
        }
    }
    const Cost pair = cost_of(job, t, pack, false), single = cost_of(job, t, pack, true);
    const double ctx_bytes = 4.0 * job.D * (double)job.C * job.Hkv;
    const PlanTime of_pair = time_of(pair, false, ctx_bytes), of_solo = time_of(single, true, ctx_bytes);
    const double best_pair = of_pair.cut < of_pair.whole ? of_pair.cut : of_pair.whole;
    const double best_solo = of_solo.cut < of_solo.whole ? of_solo.cut : of_solo.whole;
    const double apart = of_solo.apart < of_pair.apart ? of_solo.apart : of_pair.apart;
    // 48 tokens over 16384 shared keys: apart 41 us, each token for itself 146 us
    const bool sep = job.nseg > 1 && job.C > 0 && apart < best_pair && apart < best_solo;
    pl.solo = sep ? of_solo.apart <= of_pair.apart : best_solo <= best_pair;
    t.uncut = !sep && (pl.solo ? of_solo.whole <= of_solo.cut : of_pair.whole <= of_pair.cut);
    t.unit_steps = pl.solo ? kSoloUnitSteps : kPairUnitSteps;
    t.entries = job.nseg + (sep ? 1 : 0);
    t.pack = pack;
    t.tok = 128 / pack;
    t.unit_tok = pl.solo ? t.tok : 2 * t.tok;
    t.head_blocks = job.Hq / pack;
    t.separate = sep ? 1 : 0;

    // CTAs: one per SM where there is work for all of them.
    const Cost& cost = pl.solo ? single : pair;
    const double tiles = sep ? cost.tiles_apart : cost.tiles, units = sep ? cost.units_apart : cost.units;
    if (tiles + 2 * (kSoloUnitSteps + 1) * units >= 2147483648.0) return pl;  // steps are counted in 32 bits
    double ctas = t.uncut ? units : tiles / kSnap;
    if (ctas < units) ctas = units;
    t.ctas = ctas > kAttnCtas ? kAttnCtas : ctas < 1 ? 1 : (int)ctas;
    t.any_full = 0;
    if (!sep && t.ctas == kAttnCtas)
        for (int e = 0; e < t.entries; ++e)
            if (t.units(e) >= t.ctas) t.any_full = 1;
    // Units of a head side by side: one entry, all of it in the pool, keys of more
    // than 64 MB (half the L2), and at most a twentieth of the CTAs left idle.
    t.lanes = 1;
    t.stretches = t.ctas;
    if (t.entries == 1 && !t.uncut && !t.any_full && t.ctas == kAttnCtas) {
        const int rb = t.row_blocks(0), idle = kAttnCtas % rb;
        const double key_bytes = 4.0 * job.Hkv * job.D * ((double)job.T + (double)job.C);
        if (rb > 1 && rb <= kAttnCtas / 2 && idle * 20 <= kAttnCtas && key_bytes > 64.0 * 1024 * 1024) {
            t.lanes = rb;
            t.stretches = kAttnCtas / rb;
        }
    }
    int longest = 0;  // steps of a unit of the pool
    t.pool_unit[0] = t.pool_step[0] = 0;
    for (int e = 0; e < t.entries; ++e) {
        const int rest = t.units(e) - t.full(e);
        if (rest > 0 && t.steps(e) > longest) longest = t.steps(e);
        t.pool_unit[e + 1] = t.pool_unit[e] + rest;
        t.pool_step[e + 1] = t.pool_step[e] + rest / t.lanes * t.steps(e);
    }
    t.pool_steps = t.pool_step[t.entries];
    t.share = t.pool_steps / t.stretches;
    t.longer = t.pool_steps % t.stretches;

    // Partials: rows of the largest unit of each kind, an even number so that
    // every slot of rows * (dp + 2) floats begins on 16 bytes.
    int most = 0;
    for (int e = 0; e < t.nseg; ++e) {
        const int rows = t.q_end(e) - t.q_begin(e);
        if (rows > most) most = rows;
    }
    pl.slot_rows[0] = (most < t.unit_tok ? most : t.unit_tok) * pack;
    pl.slot_rows[1] = (t.M < t.unit_tok ? t.M : t.unit_tok) * pack;
    for (int& rows : pl.slot_rows) rows += rows & 1;
    if (sep) {
        pl.join = true;
        pl.slots[0] = t.pool_unit[t.nseg];
        pl.slots[1] = t.units(t.nseg) + t.ctas;
    } else {
        for (int c = 1, cut = -1; c < t.stretches && !t.uncut && longest > 2 * kSnap; ++c) {
            const int x = t.bound(c);
            if (x <= 0 || x >= t.pool_steps) continue;
            const int e = t.find(t.pool_step, x), n = t.steps(e), local = x - t.pool_step[e], u = local / n;
            if (local == u * n) continue;
            const int id = t.pool_unit[e] + u;
            if (id == cut) {  // cut once more
                for (int k = 1; k <= t.lanes; ++k) ++pl.cuts[pl.n_cuts - k].parts;
                continue;
            }
            cut = id;
            for (int k = 0; k < t.lanes; ++k) {
                const int rb = t.row_blocks(e), all = t.lanes > 1 ? u * rb + k : t.full(e) + u, hb = all / rb;
                const int tok0 = t.q_begin(e) + (all - hb * rb) * t.unit_tok;
                pl.cuts[pl.n_cuts++] = Cut{tok0, hb * pack, lesser(t.unit_tok, t.q_end(e) - tok0) * pack,
                                           (c - 1) * t.lanes + k, 2};
            }
        }
        pl.join = pl.n_cuts > 0;
        pl.slots[0] = pl.join ? 2 * t.ctas : 0;
    }
    size_t at = 256;
    for (int k = 0; k < 2; ++k) {
        pl.slot_off[k] = at;
        at += (size_t)pl.slots[k] * pl.slot_rows[k] * (pl.dp + 2) * 4;
        at = (at + 255) / 256 * 256;
    }
    pl.bytes = at;
    return pl;
}

}  // namespace h3fp4
