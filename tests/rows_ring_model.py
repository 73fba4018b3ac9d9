"""A discrete-event model of the one-kernel linear of a few rows (rows_few_kernel in h3fp4_linear_rows.cu): its roles over
the ring of stages, with random delays.

As in attn_ring_model: a role is a generator that yields the waits of the kernel's role in its order, (barrier, parity) or
a delay; a wait sees nothing of a barrier but the parity. What each slot holds is tracked beside them, so that a role which
goes on too early is caught, and a run that stops short of its end is a deadlock.
"""
import random

from attn_ring_model import Bar, Broken, need

__all__ = ["failures"]


class Model:
    def __init__(self, rng, rows, n, stages, together):
        self.rng, self.n, self.stages, self.together = rng, n, stages, together
        self.row_warps = 8 if rows > 4 else 4 if rows > 2 else rows
        self.full = [Bar(1 + 4 + self.row_warps, f"full {i}") for i in range(stages)]
        self.sf_full = [Bar(1 + self.row_warps, f"sf_full {i}") for i in range(stages)]
        self.empty = [Bar(1, f"empty {i}") for i in range(stages)]
        self.w, self.sfw = [None] * stages, [None] * stages              # the stage whose tiles landed in a slot
        self.digits = [[None] * self.row_warps for _ in range(stages)]   # by the row warp
        self.tmem = [[None] * 4 for _ in range(stages)]                  # by the lane quarter
        self.done = 0                                                    # products issued
        self.busy = [None] * stages                                      # stage that the tensor cores read from a slot
        self.time, self.events = 0.0, []

    def owned(self, warp):
        return range(warp // self.row_warps, self.n, 8 // self.row_warps)

    def slow(self):
        return self.rng.choice([0.1, 1.0, 1.0, 5.0, 40.0]) * self.rng.random()

    def later(self, what):
        self.events.append((self.time + self.slow(), self.rng.random(), what))

    def producer(self):
        for i in range(self.n):
            s = i % self.stages
            yield self.empty[s], (i // self.stages & 1) ^ 1
            need(self.busy[s] is None, "a tile is loaded over one in use")
            self.sf_full[s].arrive(1)
            self.full[s].arrive(1)

            def land(s=s, i=i, codes=True):
                (self.w if codes else self.sfw)[s] = i
                (self.full if codes else self.sf_full)[s].land()
            self.later(land)
            self.later(lambda s=s, i=i: land(s, i, False))
            yield self.slow()

    def digit_warp(self, warp):
        row = warp % self.row_warps
        for i in self.owned(warp):
            s = i % self.stages
            yield self.empty[s], (i // self.stages & 1) ^ 1
            yield self.slow()
            need(self.busy[s] is None and (i < self.stages or self.done > i - self.stages), "digits over ones in use")
            self.digits[s][row] = i
            yield self.slow()
            self.sf_full[s].arrive()
            self.full[s].arrive()

    def scale_warp(self, quarter):
        i = 0
        while i < self.n:
            yield self.sf_full[i % self.stages], i // self.stages & 1
            go = 0
            while True:
                j = i + go
                s = j % self.stages
                need(self.sfw[s] == j and all(d == j for d in self.digits[s]), "scales of another stage")
                need(self.busy[s] is None, "scales over ones in use")
                self.tmem[s][quarter] = j
                go += 1
                yield self.slow()
                if go == self.together or i + go >= self.n:
                    break
                if not self.sf_full[(i + go) % self.stages].done((i + go) // self.stages & 1):
                    break
            for k in range(go):
                self.full[(i + k) % self.stages].arrive()
            i += go

    def mma(self):
        for i in range(self.n):
            s = i % self.stages
            yield self.full[s], i // self.stages & 1
            need(self.w[s] == i and all(d == i for d in self.digits[s]) and all(t == i for t in self.tmem[s]),
                 "products of another stage")
            self.busy[s] = i

            def release(s=s, i=i):
                if self.done != i:                                       # (they end in their order)
                    self.later(lambda: release(s, i))
                    return
                self.done, self.busy[s] = i + 1, None
                self.empty[s].arrive()
            self.later(release)
            yield self.slow()

    def run(self):
        roles = [self.producer(), self.mma(), *(self.scale_warp(q) for q in range(4)),
                 *(self.digit_warp(w) for w in range(8))]
        waiting = {k: None for k in range(len(roles))}                   # None: may go on
        asleep = {}
        while waiting or asleep or self.events:
            moved = False
            for k in self.rng.sample(sorted(waiting), len(waiting)):
                at = waiting[k]
                if at is not None and not at[0].done(at[1]):
                    continue
                moved = True
                try:
                    got = next(roles[k])
                except StopIteration:
                    del waiting[k]
                    continue
                if isinstance(got, tuple):
                    waiting[k] = got
                else:
                    del waiting[k]
                    asleep[k] = self.time + got
            if moved:
                continue
            times = list(asleep.values()) + [e[0] for e in self.events]
            need(times, "deadlock")
            self.time = min(times)
            for k in [k for k, t in asleep.items() if t <= self.time]:
                del asleep[k]
                waiting[k] = None
            due = [e for e in self.events if e[0] <= self.time]
            self.events = [e for e in self.events if e[0] > self.time]
            for _, _, what in sorted(due, key=lambda e: e[:2]):
                what()
        need(self.done == self.n, "stages left over")


def failures(runs, rows_of, stages, together, seed=1):
    """What went wrong in so many runs of some of these rows and random stages: {message: count}."""
    rng, found = random.Random(seed), {}
    for _ in range(runs):
        rows = rng.choice(rows_of)
        try:
            Model(rng, rows, rng.choice([1, 2, 5, 7, 13, 24, 40]), stages, together).run()
        except Broken as e:
            found[str(e.args[0])] = found.get(str(e.args[0]), 0) + 1
    return found
