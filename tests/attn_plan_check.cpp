// Walks the pieces of an attention plan as the kernels do and checks that they
// cover every key tile of every unit exactly once, that partial sums never share
// a slot or leave the workspace, and that the joining kernel reads just the slots
// that were written.  Input lines: M T C Hq Hkv D nseg q_off... kv_off...
// Prints one line per problem: "ok solo separate join ctas lanes" or what is wrong.
#define __host__
#define __device__
#include <cstdio>
#include <map>
#include <set>
#include <vector>

#include "attn_plan.h"

using namespace h3fp4;

struct Job {
    int64_t M, T, C;
    int Hq, Hkv, D, nseg;
    std::vector<int64_t> q_off, kv_off;
};

static const char* check(const Job& job)
{
    const AttnPlan pl = make_plan(job);
    const AttnTable& t = pl.t;
    if (pl.bytes == 0) return "refused";
    if (t.pack * t.tok > 128 || (job.Hq / job.Hkv) % t.pack) return "pack";
    for (int k = 0; k < 2; ++k)  // 16-byte stores into every slot
        if (pl.slot_off[k] % 16 || (size_t)pl.slot_rows[k] * (pl.dp + 2) * 4 % 16) return "slot alignment";
    std::map<std::vector<int>, std::vector<int>> seen;  // (entry, head block, token) -> visits of each tile
    std::map<std::vector<int>, std::set<int>> slots[2];  // unit -> slots written
    std::set<int> used[2];
    for (int c = 0; c < t.ctas; ++c) {
        Walk w(t);
        w.start(c);
        Piece p;
        while (w.next(p)) {
            const int n = p.ctx_tiles + p.own_tiles;
            if (p.ntok < 1 || p.ntok > t.unit_tok || p.tok0 < t.q_begin(p.e) || p.tok0 + p.ntok > t.q_end(p.e))
                return "rows outside the segment";
            if (p.head0 < 0 || p.head0 + t.pack > job.Hq || p.head0 % t.pack) return "heads";
            const std::vector<int> key = {p.e, p.head0, p.tok0};
            auto& v = seen[key];
            if (v.empty()) v.resize(n + 1);
            if (p.nt == 0) {
                if (n != 0) return "empty piece of a unit with keys";
                ++v[0];
            }
            if (p.nt < 0 || p.t0 < 0 || p.t0 + p.nt > n) return "tiles outside the unit";
            for (int i = 0; i < p.nt; ++i) ++v[p.t0 + i];
            if (!p.whole) {
                const int kind = p.e < t.nseg ? 0 : 1;
                if (!pl.join) return "a partial without a joining kernel";
                if (p.slot < 0 || p.slot >= pl.slots[kind]) return "slot outside the workspace";
                if (!used[kind].insert(p.slot).second) return "slot written twice";
                if (p.ntok * t.pack > pl.slot_rows[kind]) return "rows of a slot";
                slots[kind][key].insert(p.slot);
            } else if (p.nt != n || p.t0 != 0) {
                return "whole piece that is not";
            }
        }
    }
    for (int e = 0; e < t.entries; ++e)
        for (int hb = 0; hb < t.head_blocks; ++hb)
            for (int k = t.q_begin(e); k < t.q_end(e); k += t.unit_tok) {
                const auto it = seen.find({e, hb * t.pack, k});
                if (it == seen.end()) return "unit left out";
                const int n = t.tiles(e);
                for (int i = 0; i < (n ? n : 1); ++i)
                    if (it->second[i] != 1) return "tile not visited once";
            }
    if ((int)seen.size() != [&] { int u = 0; for (int e = 0; e < t.entries; ++e) u += t.units(e); return u; }())
        return "units";
    if (!pl.join) return nullptr;
    // the joining kernels' view
    if (!t.separate) {
        std::map<std::vector<int>, std::set<int>> want;
        for (int i = 0; i < pl.n_cuts; ++i) {
            const Cut& c = pl.cuts[i];
            if (c.rows < 1 || c.rows > pl.slot_rows[0]) return "rows of a cut";
            int e = 0;
            while (c.tok0 >= t.q_end(e)) ++e;
            if (c.rows != lesser(t.unit_tok, t.q_end(e) - c.tok0) * t.pack) return "rows of a cut";
            for (int k = 0; k < c.parts; ++k) want[{e, c.head0, c.tok0}].insert(cut_slot(c.cta + k * t.lanes, k == 0));
        }
        return want == slots[0] ? nullptr : "slots joined are not those written";
    }
    for (int e = 0; e < t.entries; ++e)
        for (int u = 0; u < t.units(e); ++u) {
            const int n = t.steps(e), a = t.pool_step[e] + u * n, rb = t.row_blocks(e), hb = u / rb;
            std::set<int> want;
            if (e < t.nseg) want.insert(t.pool_unit[e] + u);
            else
                for (int c = t.stretch_of(a); c <= t.stretch_of(a + n - 1); ++c) want.insert(u + c);
            if (want != slots[e < t.nseg ? 0 : 1][{e, hb * t.pack, t.q_begin(e) + (u - hb * rb) * t.unit_tok}])
                return "slots joined are not those written";
        }
    return nullptr;
}

int main()
{
    long long M, T, C;
    int Hq, Hkv, D, n;
    while (std::scanf("%lld %lld %lld %d %d %d %d", &M, &T, &C, &Hq, &Hkv, &D, &n) == 7) {
        Job job{M, T, C, Hq, Hkv, D, n, std::vector<int64_t>(n + 1), std::vector<int64_t>(n + 1)};
        for (auto* v : {&job.q_off, &job.kv_off})
            for (int i = 0; i <= n; ++i) {
                long long x;
                if (std::scanf("%lld", &x) != 1) return 1;
                (*v)[i] = x;
            }
        const char* bad = check(job);
        const AttnPlan pl = make_plan(job);
        if (bad) std::printf("%s\n", bad);
        else std::printf("ok %d %d %d %d %d\n", (int)pl.solo, pl.t.separate, (int)pl.join, pl.t.ctas, pl.t.lanes);
    }
    return 0;
}
