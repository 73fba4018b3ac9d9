"""A discrete-event model of the attention kernel's roles and barriers (h3fp4_attn.cu) with random delays.

Every role is a generator that yields the waits of the kernel's role in its order: (barrier, parity) or a delay. Barriers
count arrivals and bytes as mbarriers do, and a wait sees nothing of them but the parity. What lies in the Q places, the
K/V ring, S, P, O and the mask slots is tracked beside them, so that a role which goes on too early is caught: it finds a
tile there that is not the one it wants, or overwrites one that is still needed. A run that stops short of its end is a
deadlock.

A unit is (tiles, has a second query tile); ``gaps[i]`` says which of unit i's tiles have keys that are left out.
"""
import heapq
import random


class Broken(AssertionError):
    """A role saw or did something that the kernel must not."""


def need(good, *what):
    if not good:
        raise Broken(*what)


class Bar:
    def __init__(self, count, name):
        self.count, self.pending, self.bytes, self.phase, self.name = count, count, 0, 0, name

    def arrive(self, copies=0):
        self.bytes += copies
        self.pending -= 1
        need(self.pending >= 0, "too many arrivals", self.name)
        self._turn()

    def land(self):
        self.bytes -= 1
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):
        """What a wait can see: whether the running phase has the other parity."""
        return (self.phase & 1) != parity


class Ring:
    """Places in the order of loads and the barriers that say they are full: ``fulls`` of them per stage, in turn."""

    def __init__(self, stages, fulls, count, name):
        self.stages, self.n = stages, stages * fulls
        self.full = [Bar(1, f"{name} full {i}") for i in range(self.n)]
        self.empty = [Bar(count, f"{name} empty {i}") for i in range(stages)]
        self.holds = [None] * stages

    def filled(self, place):
        return self.full[place % self.n], (place // self.n) & 1

    def free(self, place):
        return self.empty[place % self.stages], ((place // self.stages) & 1) ^ 1

    def give_back(self, place):
        self.empty[place % self.stages].arrive()

    def check(self, place, tile):
        need(self.holds[place % self.stages] == tile, "wrong tile", self.holds[place % self.stages], tile)


class Model:
    def __init__(self, solo, units, gaps, seed, stages, q_places, fulls=2, mask_slots=8, piece_slots=4):
        self.rng = random.Random(seed)
        self.solo, self.units, self.gaps = solo, units, gaps
        self.slots, self.pieces = mask_slots, piece_slots
        self.q = Ring(q_places, fulls, 2 if solo else 1, "Q")
        self.kv = Ring(stages, fulls, 1 if solo else 2, "K/V")
        two = lambda name: [Bar(1, f"{name} {x}") for x in "AB"]  # noqa: E731
        self.s_full, self.p_half, self.p_full = two("S full"), two("P half"), two("P full")
        self.o_full, self.o_empty = two("O full"), two("O empty")
        self.stat_full, self.stat_empty, self.turn = two("stat full"), two("stat empty"), two("turn")
        many = lambda n, count, name: [Bar(count, f"{name} {i}") for i in range(n)]  # noqa: E731
        self.gap_load, self.mask_full = many(mask_slots, 1, "gap load"), many(mask_slots, 1, "mask full")
        self.zero_full = many(mask_slots, 1, "zero full")
        self.piece_full, self.piece_empty = many(piece_slots, 1, "piece full"), many(piece_slots, 7, "piece empty")
        self.record, self.mask = [None] * piece_slots, [None] * mask_slots
        self.S, self.P, self.O = [None] * 2, [None] * 2, [None] * 2
        self.before = [0]
        for g in gaps:
            self.before.append(self.before[-1] + sum(g))
        self.time, self.events, self.count, self.pipe_free = 0, [], 0, 0
        self.slow = self.rng.choice([1, 1, 20])

    # ------------------------------------------------------------------ time

    def after(self, delay, what):
        self.count += 1
        heapq.heappush(self.events, (self.time + delay, self.count, what))

    def copy(self, ring, place, tile):
        """A TMA copy: the place is overwritten from now on, and lands at any time."""
        bar, stage = ring.full[place % ring.n], place % ring.stages
        bar.arrive(1)
        ring.holds[stage] = ("on its way", tile)

        def land():
            ring.holds[stage] = tile
            bar.land()
        self.after(self.rng.randint(1, 100) * self.slow, land)

    def issue(self, what):
        """Products: done one after the other in the order they were issued."""
        self.pipe_free = max(self.time, self.pipe_free) + 10
        self.after(self.pipe_free - self.time, what)

    # ------------------------------------------------------------------ arithmetic that the roles share

    def tiles_for(self, u, X):
        tiles, second = self.units[u]
        if self.solo:
            return (tiles + 1) // 2 if X == 0 else tiles // 2
        return tiles if X == 0 or second else 0

    def tile_at(self, X, i):
        return 2 * i + X if self.solo else i

    def k_place(self, i):
        return (0 if i == 0 else 2 * i - 1) if self.solo else 2 * i

    def v_place(self, i, n):
        return (2 * n - 1 if i == n - 1 else 2 * i + 2) if self.solo else 2 * i + 1

    def q_tiles(self, u):
        tiles, second = self.units[u]
        return 0 if tiles == 0 else 1 if self.solo or not second else 2

    def gap(self, u, t):
        return self.before[u] + sum(self.gaps[u][:t])

    def slot(self, bars, g):
        return bars[g % self.slots], (g // self.slots) & 1

    def take(self, c):
        """The c-th piece, or -1."""
        yield self.piece_full[c % self.pieces], (c // self.pieces) & 1
        number, u = self.record[c % self.pieces]
        need(number == c, "piece", number, c)
        self.piece_empty[c % self.pieces].arrive()
        return u

    # ------------------------------------------------------------------ roles

    def loads(self):
        q_place = place = c = 0
        while True:
            u = yield from self.take(c)
            c += 1
            if u < 0:
                return
            n = self.units[u][0]
            order = [None] * (2 * n)
            for i in range(n):
                order[self.k_place(i)], order[self.v_place(i, n)] = ("K", u, i), ("V", u, i)
            for i, tile in enumerate(order):
                if i < self.q_tiles(u):
                    yield self.q.free(q_place)
                    self.copy(self.q, q_place, ("Q", u, i))
                    q_place += 1
                yield self.kv.free(place)
                self.copy(self.kv, place, tile)
                place += 1
                if tile[0] == "V" and self.gaps[u][tile[2]]:
                    self.slot(self.gap_load, self.gap(u, tile[2]))[0].arrive()

    def products(self, X):
        q_place = place = c = 0
        p_phase, o_phase, t_phase = 0, 1, X ^ 1
        own_q = 0 if self.solo else X

        def wait_s(qp, pl, i):
            if i == 0:
                yield self.q.filled(qp + own_q)
            yield self.kv.filled(pl + self.k_place(self.tile_at(X, i)))

        def issue_s(u, qp, pl, i, last):
            t = self.tile_at(X, i)
            at, qat = pl + self.k_place(t), qp + own_q

            def look():
                self.kv.check(at, ("K", u, t))
                self.q.check(qat, ("Q", u, own_q))
            look()

            def done():
                look()
                need(self.S[X] is None, "S overwritten", self.S[X], u, t)
                self.S[X] = (u, t)
                self.s_full[X].arrive()
                self.kv.give_back(at)
                if last:
                    self.q.give_back(qat)
            self.issue(done)

        u, begun = (yield from self.take(c)), False
        c += 1
        while u >= 0:
            tiles, n = self.units[u][0], self.tiles_for(u, X)
            turns = self.tiles_for(u, 0) if self.tiles_for(u, 1) > 0 else 0
            if n > 0 and not begun:
                yield from wait_s(q_place, place, 0)
                issue_s(u, q_place, place, 0, n == 1)
            next_place, next_q = place + 2 * tiles, q_place + self.q_tiles(u)
            v = yield from self.take(c)
            c += 1
            n_next = self.tiles_for(v, X) if v >= 0 else 0
            begun = n > 0 and n_next > 0
            if n > 0:
                yield self.o_empty[X], o_phase
                o_phase ^= 1
            for i in range(n):
                t, last = self.tile_at(X, i), i == n - 1
                at = place + self.v_place(t, tiles)
                yield self.kv.filled(at)
                self.kv.check(at, ("V", u, t))
                if self.gaps[u][t]:
                    yield self.slot(self.zero_full, self.gap(u, t))
                if not last:
                    yield from wait_s(q_place, place, i + 1)
                elif n_next > 0:
                    yield from wait_s(next_q, next_place, 0)
                yield self.p_half[X], p_phase
                if turns > 0:
                    yield self.turn[X], t_phase
                    t_phase ^= 1
                yield self.p_full[X], p_phase
                p_phase ^= 1

                def done(at=at, t=t, last=last, u=u):
                    self.kv.check(at, ("V", u, t))
                    need(self.P[X] == (u, t), "P", self.P[X], u, t)
                    need(self.O[X] is None, "O not read yet", self.O[X], u)
                    self.P[X] = None
                    self.kv.give_back(at)
                    if last:
                        self.O[X] = u
                        self.o_full[X].arrive()
                self.issue(done)
                if not last:
                    issue_s(u, q_place, place, i + 1, i + 2 == n)
                elif n_next > 0:
                    issue_s(v, next_q, next_place, 0, n_next == 1)
                if turns > 0:
                    self.turn[X ^ 1].arrive()
            if n == 0 and tiles > 0:  # nothing for X: its places are given back as they fill
                if self.solo:
                    yield self.q.filled(q_place)
                    self.q.give_back(q_place)
                else:
                    for at in range(place, place + 2 * tiles):
                        yield self.kv.filled(at)
                        self.kv.give_back(at)
            for _ in range(n, turns):
                yield self.turn[X], t_phase
                t_phase ^= 1
                self.turn[X ^ 1].arrive()
            q_place, place, u = next_q, next_place, v

    def softmax(self, X):
        s_phase, stat_phase, c = 0, 1, 0
        while True:
            u = yield from self.take(c)
            c += 1
            if u < 0:
                return
            n = self.tiles_for(u, X)
            for i in range(n):
                yield self.s_full[X], s_phase
                s_phase ^= 1
                t = self.tile_at(X, i)
                if self.gaps[u][t]:
                    g = self.gap(u, t)
                    yield self.slot(self.mask_full, g)
                    need(self.mask[g % self.slots] == g, "mask", self.mask[g % self.slots], g)
                    yield self.rng.randint(1, 30)
                    need(self.mask[g % self.slots] == g, "mask", self.mask[g % self.slots], g)
                need(self.S[X] == (u, t), "S", self.S[X], u, t)
                yield self.rng.randint(1, 60)
                self.S[X], self.P[X] = None, (u, t)
                self.p_half[X].arrive()
                yield self.rng.randint(1, 60)
                self.p_full[X].arrive()
            if n > 0:
                yield self.stat_empty[X], stat_phase
                stat_phase ^= 1
                self.stat_full[X].arrive()

    def epilogue(self):
        phase, c = [0, 0], 0
        while True:
            u = yield from self.take(c)
            c += 1
            if u < 0:
                return
            for Y in range(1 if self.solo or not self.units[u][1] else 2):
                parts = [X for X in (0, 1) if self.tiles_for(u, X) > 0 and (self.solo or X == Y)]
                for X in parts:
                    yield self.stat_full[X], phase[X]
                    yield self.o_full[X], phase[X]
                    phase[X] ^= 1
                for X in parts:
                    self.stat_empty[X].arrive()
                yield self.rng.randint(1, 200)
                for X in parts:
                    need(self.O[X] == u, "O", self.O[X], u)
                    self.O[X] = None
                    self.o_empty[X].arrive()

    def left_out(self):
        """Describes the pieces a few ahead, and handles the keys that are left out."""
        described = place = c = 0

        def describe(d):
            yield self.piece_empty[d % self.pieces], ((d // self.pieces) & 1) ^ 1
            self.record[d % self.pieces] = (d, d if d < len(self.units) else -1)
            self.piece_full[d % self.pieces].arrive()
        while described < min(self.pieces - 1, len(self.units) + 1):
            yield from describe(described)
            described += 1
        while True:
            u = yield from self.take(c)
            c += 1
            if u < 0:
                return
            if described <= len(self.units):
                yield from describe(described)
                described += 1
            tiles = self.units[u][0]
            for i in range(tiles):
                if not self.gaps[u][i]:
                    continue
                at, g = place + self.v_place(i, tiles), self.gap(u, i)
                yield self.slot(self.gap_load, g)
                self.mask[g % self.slots] = g
                self.slot(self.mask_full, g)[0].arrive()
                yield self.kv.filled(at)
                self.kv.check(at, ("V", u, i))
                yield self.rng.randint(0, 50)
                self.kv.check(at, ("V", u, i))
                self.slot(self.zero_full, g)[0].arrive()
            place += 2 * tiles

    # ------------------------------------------------------------------ a run

    def run(self):
        roles = {"left out": self.left_out(), "loads": self.loads(), "products A": self.products(0),
                 "products B": self.products(1), "softmax A": self.softmax(0), "softmax B": self.softmax(1),
                 "epilogue": self.epilogue()}
        waits, asleep = dict.fromkeys(roles), set()
        while roles:
            moved = False
            for name in self.rng.sample(sorted(roles), len(roles)):
                if name in asleep or (waits[name] is not None and not waits[name][0].done(waits[name][1])):
                    continue
                moved = True
                try:
                    w = next(roles[name])
                except StopIteration:
                    del roles[name]
                    continue
                if isinstance(w, int):
                    asleep.add(name)
                    waits[name] = None
                    self.after(w, lambda name=name: asleep.discard(name))
                else:
                    waits[name] = w
            if not moved:
                need(self.events, "deadlock", {n: waits[n] and waits[n][0].name for n in roles})
                self.time, _, what = heapq.heappop(self.events)
                what()
        while self.events:
            self.time, _, what = heapq.heappop(self.events)
            what()
        need(not any(self.S) and not any(self.P) and not any(o is not None for o in self.O), "something left over")


def problem(seed, solo):
    """Random units: short and long ones, with and without a second query tile, keys or gaps."""
    rng = random.Random(seed)
    none = rng.choice([0, 0, 0.6])
    units = [(0 if rng.random() < none else rng.choice([1, 1, 2, 3, 4, rng.randint(1, 12)]), rng.random() < 0.7)
             for _ in range(rng.randint(1, 20))]
    gaps = [[rng.random() < share for _ in range(n)] for n, _ in units for share in [rng.choice([0, 0, 0.3, 1])]]
    return units, gaps


def failures(runs, solo, stages, q_places, **kw):
    """What broke in so many runs: {message: how often}."""
    broken = {}
    for seed in range(runs):
        units, gaps = problem(seed, solo)
        try:
            Model(solo, units, gaps, seed, stages, q_places, **kw).run()
        except Broken as e:
            broken[str(e.args[0])] = broken.get(str(e.args[0]), 0) + 1
    return broken
