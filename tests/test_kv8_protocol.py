"""The barriers of the attention kernel for many rows, restated on the CPU: every role in a random interleaving, waits
that know a phase only by its parity, as the hardware's do.  A run must end, no wait may pass early, and nobody may
write what another still reads."""
import random

import pytest

WARPS, BLOCKS = 6, 8  # converting warps; blocks of K (and of V) in a tile


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.pending, self.done = self.count, self.done + 1


class Model:
    """bufs: converted tiles of K and of V; row tiles; depth of a converting warp's ring; s_bufs: S of a row tile."""

    def __init__(self, n, bufs, tiles, depth, two_s, seed):
        self.n, self.bufs, self.tiles, self.depth, self.two_s = n, bufs, tiles, depth, two_s
        self.rng = random.Random(seed)
        self.slots = WARPS * depth
        mk = lambda k, c: [Bar(c) for _ in range(k)]  # noqa: E731
        self.k_full, self.k_empty, self.v_full, self.v_empty = mk(bufs, BLOCKS), mk(bufs, 1), mk(bufs, BLOCKS), mk(bufs, 1)
        self.s_full = mk(2, 1)
        self.p_ready = [mk(2, 4), mk(2, 4)]
        self.pv_done = [mk(2, 1), mk(2, 1)]
        self.o_done = mk(2, 1)
        self.sc_full, self.sc_empty = mk(4, 1), mk(4, 4 * tiles)
        self.raw_full, self.raw_empty = mk(self.slots, 1), mk(self.slots, 1)
        self.raw, self.k, self.v = [None] * self.slots, [[None] * BLOCKS for _ in range(bufs)], [[None] * BLOCKS for _ in range(bufs)]
        self.sc, self.s, self.copies, self.mmas = [None] * 4, [None] * 2, [], []
        self.p = [[[None] * 4, [None] * 4] for _ in range(2)]
        self.o = [0, 0]

    def wait(self, bar, phase):
        while (bar.done & 1) == (phase & 1):
            yield
        assert bar.done == phase + 1, "passed early, or two phases on"

    def loader_lane(self, u):
        turn = u // WARPS
        slot, rnd = u % WARPS * self.depth + turn % self.depth, turn // self.depth
        if rnd:
            yield from self.wait(self.raw_empty[slot], rnd - 1)
        self.copies.append([self.rng.randint(1, 300), slot, u])

    def loader(self):
        for j in range(self.n):
            for start in range(0, 16, self.slots):
                lanes = [self.loader_lane(16 * j + i) for i in range(start, min(16, start + self.slots))]
                while lanes:
                    for g in list(lanes):
                        if next(g, self) is self:
                            lanes.remove(g)
                    yield
            if j >= 4:
                yield from self.wait(self.sc_empty[j & 3], j // 4 - 1)
            self.sc[j & 3] = j
            self.sc_full[j & 3].arrive()

    def converter(self, first):
        for turn, u in enumerate(range(first, 16 * self.n, WARPS)):
            slot, rnd = first * self.depth + turn % self.depth, turn // self.depth
            yield from self.wait(self.raw_full[slot], rnd)
            assert self.raw[slot] == u
            self.raw_empty[slot].arrive()
            j, v, b = u >> 4, (u >> 3) & 1, u & 7
            buf = j % self.bufs
            if j >= self.bufs:
                yield from self.wait((self.v_empty if v else self.k_empty)[buf], j // self.bufs - 1)
            yield
            (self.v if v else self.k)[buf][b] = j
            (self.v_full if v else self.k_full)[buf].arrive()

    def issue(self, run, *bars):
        self.mmas.append([self.rng.randint(1, 60), run, bars])

    def qk(self, t, s, j):
        def run():
            assert all(x == j for x in self.k[j % self.bufs])
            self.s[s] = (t, j)
        self.issue(run, self.s_full[s])

    def pv(self, t, s, j, h, last):
        def run():
            assert all(x == j for x in self.v[j % self.bufs]) and self.p[s][h] == [j] * 4
            self.o[t] += 1
        bars = [self.v_empty[j % self.bufs]] if last else []
        bars.append(self.pv_done[t][h])
        if j == self.n - 1 and h == 1:
            bars.append(self.o_done[t])
        self.issue(run, *bars)

    def mma(self):
        n, bufs = self.n, self.bufs
        if not self.two_s:
            for j in range(n + 1):
                if j < n:
                    yield from self.wait(self.k_full[j % bufs], j // bufs)
                for t in range(self.tiles):
                    if j > 0:
                        if t == 0:
                            yield from self.wait(self.v_full[(j - 1) % bufs], (j - 1) // bufs)
                        for h in range(2):
                            yield from self.wait(self.p_ready[t][h], j - 1)
                            self.pv(t, t, j - 1, h, h == 1 and t == self.tiles - 1)
                    if j < n:
                        self.qk(t, t, j)
                if j < n:
                    self.issue(lambda: None, self.k_empty[j % bufs])
            return
        yield from self.wait(self.k_full[0], 0)
        self.qk(0, 0, 0)
        self.issue(lambda: None, self.k_empty[0])
        for j in range(n):
            if j + 1 < n:
                yield from self.wait(self.k_full[(j + 1) % bufs], (j + 1) // bufs)
                self.qk(0, (j + 1) & 1, j + 1)
                self.issue(lambda: None, self.k_empty[(j + 1) % bufs])
            yield from self.wait(self.v_full[j % bufs], j // bufs)
            for h in range(2):
                yield from self.wait(self.p_ready[j & 1][h], j >> 1)
                self.pv(0, j & 1, j, h, h == 1)

    def softmax(self, t, warp):
        for j in range(self.n):
            s, phase = (j & 1, j >> 1) if self.two_s else (t, j)
            yield from self.wait(self.s_full[s], phase)
            yield from self.wait(self.sc_full[j & 3], j >> 2)
            for h in range(2):
                assert self.s[s] == (t, j) and self.sc[j & 3] == j
                for _ in range(self.rng.randint(1, 8)):
                    yield
                if self.rng.random() < 0.3 and j + h > 0:  # rescale O: the product before this one is done
                    if j > 0:
                        yield from self.wait(self.pv_done[t][1], j - 1)
                    if h:
                        yield from self.wait(self.pv_done[t][0], j)
                    assert self.o[t] == 2 * j + h
                assert self.s[s] == (t, j) and self.sc[j & 3] == j
                self.p[s][h][warp] = j
                self.p_ready[s][h].arrive()
            self.sc_empty[j & 3].arrive()
        yield from self.wait(self.o_done[t], 0)
        assert self.o[t] == 2 * self.n

    def run(self):
        roles = [self.loader(), self.mma()] + [self.converter(w) for w in range(WARPS)]
        roles += [self.softmax(t, w) for t in range(self.tiles) for w in range(4)]
        idle = 0
        while roles:
            for g in list(roles):
                # each role now and then sleeps for long
                if self.rng.random() < 0.7 and next(g, self) is self:
                    roles.remove(g)
            for c in list(self.copies):
                c[0] -= self.rng.randint(0, 30)
                if c[0] <= 0:
                    self.copies.remove(c)
                    self.raw[c[1]] = c[2]
                    self.raw_full[c[1]].arrive()
            if self.mmas:
                self.mmas[0][0] -= self.rng.randint(0, 20)
                if self.mmas[0][0] <= 0:
                    _, work, bars = self.mmas.pop(0)
                    work()
                    for b in bars:
                        b.arrive()
            idle += 1
            assert idle < 200_000, "nobody gets on"
        assert not self.copies and not self.mmas


@pytest.mark.parametrize("bufs,tiles,depth,two_s", [(2, 2, 2, False), (2, 1, 2, False), (1, 1, 1, True)])
def test_every_interleaving_ends(bufs, tiles, depth, two_s):
    for n in (1, 2, 3, 5, 11):
        for seed in range(12):
            Model(n, bufs, tiles, depth, two_s, 1000 * n + seed).run()


def test_the_model_sees_a_wait_two_phases_behind():
    """A loader that waited for K's buffer instead of the scales' readers would find the parity turned twice."""
    class Old(Model):
        def loader(self):
            for j in range(self.n):
                for start in range(0, 16, self.slots):
                    lanes = [self.loader_lane(16 * j + i) for i in range(start, min(16, start + self.slots))]
                    while lanes:
                        for g in list(lanes):
                            if next(g, self) is self:
                                lanes.remove(g)
                        yield
                if j >= self.bufs:
                    yield from self.wait(self.k_empty[j % self.bufs], j // self.bufs - 1)
                self.sc[j & 3] = j
                self.sc_full[j & 3].arrive()

    failed = 0
    for seed in range(10):
        try:
            Old(11, 1, 1, 1, True, seed).run()
        except AssertionError:
            failed += 1
    assert failed
