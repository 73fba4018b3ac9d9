// Walks the pieces of an attention plan and trims them to the tiles that masks keep
// (trim_piece), as the kernel's describing warp does, and checks that each unit's
// kept tiles are walked exactly once, in the numbering that is left; and which tiles
// of an untrimmed piece have keys that are left out (find_gaps).  Input lines:
// M T C Hq Hkv D nseg q_off... kv_off... ctx_keep own_keep...; prints "ok" or what
// is wrong.
#define __host__
#define __device__
#include <cstdio>
#include <map>
#include <vector>

#include "attn_plan.h"

using namespace h3fp4;

struct Job {
    int64_t M, T, C;
    int Hq, Hkv, D, nseg;
    std::vector<int64_t> q_off, kv_off;
};

static const char* check(const Job& job, int ctx_keep, const std::vector<int>& own_keep)
{
    const AttnPlan pl = make_plan(job);
    const AttnTable& t = pl.t;
    if (pl.bytes == 0) return "refused";
    std::map<std::vector<int>, std::vector<int>> seen;  // (entry, head block, token) -> visits of each kept tile
    for (int c = 0; c < t.ctas; ++c) {
        Walk w(t);
        w.start(c);
        Piece p;
        while (w.next(p)) {
            const int ctx = lesser(p.ctx_tiles, ctx_keep), own = p.e < t.nseg ? own_keep[p.e] : p.own_tiles;
            if (own > p.own_tiles) return "more own tiles kept than there are";
            const int before = p.nt;
            trim_piece(p, ctx, own);
            auto& v = seen[{p.e, p.head0, p.tok0}];
            if (v.empty()) v.resize(ctx + own + 1);
            if (p.ctx_tiles != ctx) return "context tiles";
            if (p.nt < 0 || p.nt > before || p.t0 < 0 || (p.nt > 0 && p.t0 + p.nt > ctx + own)) return "tiles";
            for (int i = 0; i < p.nt; ++i) ++v[p.t0 + i];
        }
    }
    for (const auto& u : seen)
        for (size_t i = 0; i + 1 < u.second.size(); ++i)
            if (u.second[i] != 1) return "kept tile not walked once";
    return nullptr;
}

static const char* check_gaps(const Job& job)
{
    AttnPlan pl = make_plan(job);
    for (int masks = 0; masks < 4; ++masks) {
        pl.t.ctx_masked = masks & 1;
        pl.t.own_masked = masks >> 1;
        for (int c = 0; c < pl.t.ctas; ++c) {
            Walk w(pl.t);
            w.start(c);
            Piece p;
            while (w.next(p)) {
                p.own_tiles = -1;
                p.find_gaps(pl.t);
                const int all = p.ctx_tiles + p.own_tiles;
                if (p.own_tiles != (p.kv_len + 127) / 128 || p.t0 + p.nt > all) return "own tiles";
                int n = 0;
                for (int t = p.t0; t < p.t0 + p.nt; ++t) {
                    const bool ctx = t < p.ctx_tiles;
                    const long long end = ctx ? 128LL * (t + 1) : 128LL * (t - p.ctx_tiles + 1);
                    const bool want = ctx ? (masks & 1) || end > job.C : (masks >> 1) || end > p.kv_len;
                    if (p.gaps_before(t) != n) return "gaps before a tile";
                    if (p.has_gaps(t) != want) return "tiles with gaps";
                    n += want;
                }
                if (p.gaps_before(p.t0 + p.nt) != n) return "gaps of a piece";
            }
        }
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
        int ctx;
        std::vector<int> own(n);
        if (std::scanf("%d", &ctx) != 1) return 1;
        for (int& x : own)
            if (std::scanf("%d", &x) != 1) return 1;
        const char* bad = check(job, ctx, own);
        if (!bad) bad = check_gaps(job);
        std::printf("%s\n", bad ? bad : "ok");
    }
    return 0;
}
