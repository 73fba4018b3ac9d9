"""Which units an attention call is cut into: the choices whose times were measured, and
that every kind of plan covers its work (CPU)."""
import random

from test_attn_plan_cpu import check, cut, one  # noqa: F401  (check is a fixture)

PAIR_CUT, PAIR_WHOLE, SOLO_CUT, SOLO_WHOLE = ["0", "0", "1"], ["0", "0", "0"], ["1", "0", "1"], ["1", "0", "0"]


def test_measured_sizes(check):  # noqa: F811
    sizes = {(256, 4096): SOLO_CUT, (512, 2048): SOLO_WHOLE, (1024, 2048): PAIR_WHOLE, (2048, 2048): SOLO_WHOLE,
             (4096, 512): PAIR_WHOLE, (4096, 4096): PAIR_CUT, (1024, 30720): PAIR_CUT, (129, 4096): SOLO_CUT,
             (256, 1024): SOLO_WHOLE}
    got = check([one(M, T, 0, 24, 24) for M, T in sizes])
    assert {s: g.split()[1:4] for s, g in zip(sizes, got)} == sizes


def test_separate_contexts(check):  # noqa: F811
    def tokens(n, rows, ctx, Hq, Hkv, D):
        return (n * rows, 50 * n, ctx, Hq, Hkv, D, [i * rows for i in range(n + 1)], [50 * i for i in range(n + 1)])
    got = check([tokens(40, 1, 16384, 24, 24, 128), tokens(20, 20, 12000, 24, 24, 128),
                 tokens(200, 1, 8192, 16, 4, 128)])
    assert [g.split()[:4] for g in got] == [["ok", "1", "1", "1"], ["ok", "0", "1", "1"], ["ok", "1", "1", "1"]], got


def test_random_problems_of_medium_size(check):  # noqa: F811
    rng = random.Random(7)
    problems = []
    for _ in range(1200):
        n = rng.choice([1, 1, 2, 5, 30, 100])
        M, T = int(2 ** rng.uniform(6, 13)), int(2 ** rng.uniform(7, 14))
        C = rng.choice([0, 100, int(2 ** rng.uniform(9, 14))])
        Hkv = rng.choice([1, 4, 24])
        Hq = Hkv * rng.choice([1, 1, 3, 4])
        problems.append((M, T, C, Hq, Hkv, rng.choice([64, 128]), cut(rng, M, n), cut(rng, T, n)))
    got = check(problems)
    bad = [(g, p[:6], len(p[6]) - 1) for g, p in zip(got, problems) if not g.startswith("ok")]
    assert len(got) == len(problems) and not bad, bad[:5]
    kinds = {tuple(g.split()[1:4]) for g in got}
    want = {tuple(k) for k in (PAIR_CUT, PAIR_WHOLE, SOLO_CUT, SOLO_WHOLE)} | {("0", "1", "1"), ("1", "1", "1")}
    assert kinds == want, kinds
