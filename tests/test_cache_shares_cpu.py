"""How the cache attention cuts its tiles over CTAs (struct Shares in h3fp4_cache_attn.cu), modelled on the CPU: every cut
is in order, CTAs that share a unit have tiles of it each, and the CTA that is taken for a unit's last one is."""
import bisect
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def near():
    text = open(os.path.join(ROOT, "audio_dit_gb300", "csrc", "h3fp4_cache_attn.cu")).read()
    for line in ("return total < ctas ? min(total, (long long)b) : div(total * b, ctas);",
                 "if (total < ctas || down == 0) return x;", "if (next > last && up <= next - last) return last;",
                 "return before < first && down < first - before ? first : x;",
                 "const int c = (int)div(last * ctas + total - 1, total) - 1;",
                 "return x > first && moved(c, x, first, last) == last ? c - 1 : c;"):
        assert line in text, line                                     # what is modelled here
    return int(re.search(r"kNear = (\d+);", text).group(1))


class Shares:
    def __init__(self, units, ctas, near):
        self.edges = [0]
        for u in units:
            self.edges.append(self.edges[-1] + u)
        self.total, self.ctas, self.near = self.edges[-1], ctas, near

    def raw(self, b):
        return min(self.total, b) if self.total < self.ctas else self.total * b // self.ctas

    def moved(self, b, first, last):
        x = self.raw(b)
        up, down = last - x, x - first
        if self.total < self.ctas or down == 0:
            return x
        if up <= self.near and self.raw(b + 1) > last and up <= self.raw(b + 1) - last:
            return last
        if down > self.near:
            return x
        return first if self.raw(b - 1) < first and down < first - self.raw(b - 1) else x

    def start(self, b):
        x = self.raw(b)
        if x >= self.total:
            return x
        j = bisect.bisect_right(self.edges, x) - 1
        return self.moved(b, self.edges[j], self.edges[j + 1])

    def owner_of_last(self, first, last):
        if self.total < self.ctas:
            return last - 1
        c = -(-last * self.ctas // self.total) - 1
        return c - 1 if self.raw(c) > first and self.moved(c, first, last) == last else c


@pytest.mark.parametrize("equal", [True, False])
def test_cuts(equal):
    rng, n = random.Random(int(equal)), near()
    for _ in range(1500):
        most = rng.choice([1, 2, 5, 20, 100])
        units = [rng.randint(1, most) for _ in range(rng.randint(1, 60))]
        if equal:
            units = [units[0]] * len(units)
        s = Shares(units, rng.choice([1, 2, 7, 20, 64, 456, 608]), rng.choice([n, n, 0, 1000]))
        cuts = [s.start(b) for b in range(s.ctas + 1)]
        assert cuts[0] == 0 and cuts[-1] == s.total
        assert all(a < b or s.total < s.ctas and a == b for a, b in zip(cuts, cuts[1:]))
        for first, last in zip(s.edges, s.edges[1:]):
            a, b = (max(c for c in range(s.ctas) if cuts[c] <= x < cuts[c + 1]) for x in (first, last - 1))
            assert s.owner_of_last(first, last) == b
            assert all(max(cuts[c], first) < min(cuts[c + 1], last) for c in range(a, b + 1))
