// The limit of a device wait (attn_wait_ns) against the longest time that a plan's
// pieces may keep a role waiting.  Input lines: limit M T C Hq Hkv D nseg q_off...
// kv_off...; prints the call's limit and the tiles of four units of the longest
// pieces, as walked.
#define __host__
#define __device__
#include <cstdio>
#include <vector>

#include "attn_plan.h"

using namespace h3fp4;

struct Job {
    int64_t M, T, C;
    int Hq, Hkv, D, nseg;
    std::vector<int64_t> q_off, kv_off;
};

int main()
{
    unsigned long long limit;
    long long M, T, C;
    int Hq, Hkv, D, n;
    while (std::scanf("%llu %lld %lld %lld %d %d %d %d", &limit, &M, &T, &C, &Hq, &Hkv, &D, &n) == 8) {
        Job job{M, T, C, Hq, Hkv, D, n, std::vector<int64_t>(n + 1), std::vector<int64_t>(n + 1)};
        for (auto* v : {&job.q_off, &job.kv_off})
            for (int i = 0; i <= n; ++i) {
                long long x;
                if (std::scanf("%lld", &x) != 1) return 1;
                (*v)[i] = x;
            }
        const AttnPlan pl = make_plan(job);
        long long most = 0;
        for (int c = 0; c < pl.t.ctas; ++c) {
            Walk w(pl.t);
            w.start(c);
            Piece p;
            while (w.next(p))
                if (p.nt > most) most = p.nt;
        }
        std::printf("%llu %lld\n", (unsigned long long)attn_wait_ns(pl.t, limit), 4 * most);
    }
    return 0;
}
