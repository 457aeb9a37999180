"""Model check of the mbarrier protocols of the latent kernels (csrc/latent.cu, latent_dense.cu) and of the
weights kernel (csrc/weights.cu): every warp role under random latencies, with waits that poll by parity
as `mbarrier.try_wait.parity` does (the Barrier and the polling of the prefill kernel's model).

Checked under many random schedules:
  * a parity wait is never ambiguous: the barrier has completed k or k + 1 phases when a waiter polls
    for phase k;
  * no hazard: a buffer is refilled, overwritten, rescaled or read only when its last users are done;
  * every role finishes.
Planted mistakes are caught, so that the model can tell a broken protocol from a sound one."""
import heapq
import random

import pytest

from test_prefill_protocol import Barrier, Sim


class Model(Sim):
    def __init__(self, seed, plant=None):
        self.rng = random.Random(seed)
        self.plant, self.t, self.seq, self.q, self.finished = plant, 0, 0, [], 0
        self.last = {}      # issuing warp -> completion time of its latest MMA
        self.done_at = {}   # ("S", it) and the like -> completion time

    def bars(self, name, n, count=1):
        return [Barrier(f"{name}{i}", count) for i in range(n)]

    def mma(self, warp, what):
        self.done_at[what] = self.t + self.rng.randint(20, 400)
        self.last[warp] = max(self.last.get(warp, 0), self.done_at[what])

    def commit_of(self, warp, bar):  # arrives once every MMA of this warp has completed
        when = max(self.last.get(warp, 0), self.t) + self.rng.randint(0, 20)
        self.later(when - self.t, lambda: bar.arrive(self))

    def copy(self, bar, what):
        self.done_at[what] = float("inf")

        def land():
            self.done_at[what] = self.t
            bar.arrive(self)
        self.later(self.rng.randint(10, 2000), land)

    def need(self, *what):
        for w in what:
            assert self.done_at.get(w, float("inf")) <= self.t, f"{w} is not done"

    def mark(self, what):
        self.done_at[what] = self.t

    def delay(self, lo, hi):
        return ("delay", self.rng.randint(lo, hi))

    def finish(self, actors):
        for a in actors:
            self.run_actor(a)
        while self.q:
            self.t, _, fn = heapq.heappop(self.q)
            fn()
        assert self.finished == len(actors), f"deadlock: {self.finished} of {len(actors)} actors finished"


# ---------------------------------------------------------------- absorbed form

class Absorbed(Model):
    """One CTA's run: pieces of (tiles, softmax warps without a row); a tile may hold keys to zero, keys that
    some rows see and others do not (`partial`), and bad values among those (its PV goes by rows)."""

    def __init__(self, seed, plant=None, producers=1):
        super().__init__(seed, plant)
        r, self.producers = self.rng, producers
        self.pieces = [(r.randint(1, 6), r.choice([0, 0, 1, 3])) for _ in range(r.randint(1, 5))]
        n = sum(t for t, _ in self.pieces)
        self.zero = [r.random() < 0.3 for _ in range(n)]
        self.partial = [r.random() < 0.4 for _ in range(n)]
        self.bad = [p and r.random() < 0.5 for p in self.partial]
        self.full, self.empty, self.s_full = self.bars("full", 2, producers), self.bars("empty", 2), self.bars("s_full", 2)
        self.p_full, self.o_free = Barrier("p_full", 4), Barrier("o_free", 4)
        self.pv_done, self.q_full, self.q_empty, self.checked = (Barrier(x, 1) for x in ("pv_done", "q_full", "q_empty", "checked"))
        self.flag = None

    def tiles(self):
        it = 0
        for pc, (n, idle) in enumerate(self.pieces):
            for j in range(n):
                yield pc, j, n, idle, it
                it += 1

    def producer(self, w):
        for *_, it in self.tiles():
            if it >= 2:
                yield ("wait", (self.s_full if self.plant == "refill on S" else self.empty)[it & 1], (it >> 1) - 1)
                self.need(("S", it - 2), ("PV", it - 2))
            self.copy(self.full[it & 1], ("tile", it, w))
            yield self.delay(0, 50)

    def landed(self, it):
        self.need(*[("tile", it, w) for w in range(self.producers)])

    def queries(self):
        at = 0
        for pc, (n, _) in enumerate(self.pieces):
            if pc > 0:
                yield ("wait", self.q_empty, pc - 1)
                self.need(("S", at - 1))
            self.copy(self.q_full, ("Q", pc))
            at += n

    def scores(self):
        for pc, j, n, idle, it in self.tiles():
            if j == 0:
                yield ("wait", self.q_full, pc)
            yield ("wait", self.full[it & 1], it >> 1)
            self.landed(it)
            self.need(("Q", pc))
            if it >= 2:
                self.need(*[("read S", it - 2, w) for w in range(4)])
            self.mma("S", ("S", it))
            self.commit_of("S", self.s_full[it & 1])
            yield self.delay(1, 60)
            if j == n - 1:
                self.commit_of("S", self.q_empty)

    def values(self):
        for pc, j, n, idle, it in self.tiles():
            # (redundant for the hazard below: P of a piece's first tile needs all four warps, each past its O)
            if j == 0 and pc > 0:
                yield ("wait", self.o_free, pc - 1)
            if self.zero[it] or self.partial[it]:
                yield ("wait", self.full[it & 1], it >> 1)
                self.landed(it)
                yield self.delay(50, 500)
            if self.partial[it]:
                self.flag = (it, self.bad[it])
                self.checked.arrive(self)
            yield ("wait", self.p_full, it)
            self.need(*[("P", it, w) for w in range(4 - idle)])
            if j == 0 and pc > 0:
                self.need(*[("read O", pc - 1, w) for w in range(4)])
            if self.bad[it]:
                self.mark(("PV", it))
            else:
                self.mma("PV", ("PV", it))
            self.commit_of("PV", self.empty[it & 1])
            self.commit_of("PV", self.pv_done)
            yield self.delay(1, 60)

    def softmax(self, w):
        checks = 0
        for pc, j, n, idle, it in self.tiles():
            check, checks = checks, checks + self.partial[it]
            yield ("wait", self.s_full[it & 1], it >> 1)
            self.need(("S", it))
            if w >= 4 - idle:
                self.mark(("read S", it, w))
                if it > 0 and self.plant != "idle warps run ahead":
                    yield ("wait", self.pv_done, it - 1)
                self.p_full.arrive(self)
            else:
                yield self.delay(50, 900)
                self.mark(("read S", it, w))
                if it > 0 and self.plant != "P over a PV in flight":
                    yield ("wait", self.pv_done, it - 1)
                if it > 0:
                    self.need(("PV", it - 1))
                self.mark(("P", it, w))
                if self.partial[it]:
                    if self.plant != "no wait for the check":
                        yield ("wait", self.checked, check)
                    yield ("wait", self.full[it & 1], it >> 1)
                    assert self.flag == (it, self.bad[it]), "the flag of another tile"
                    if self.bad[it]:
                        yield self.delay(500, 3000)
                        assert ("PV", it) not in self.done_at and self.flag[0] == it
                self.p_full.arrive(self)
            if j == n - 1:
                yield ("wait", self.pv_done, it)
                self.need(("PV", it))
                yield self.delay(50, 2000)
                self.mark(("read O", pc, w))
                self.o_free.arrive(self)

    def run(self):
        self.finish([self.producer(w) for w in range(self.producers)] + [self.queries(), self.scores(), self.values()] +
                    [self.softmax(w) for w in range(4)])


# ---------------------------------------------------------------- expanded form

class Expanded(Model):
    """One work tile: query tiles 0 and 1 (if `two`) over nt tiles of keys, of which 0 sees the first nt0."""
    STAGES = 3

    def __init__(self, seed, plant=None):
        super().__init__(seed, plant)
        r = self.rng
        self.two, self.nt = r.random() < 0.7, r.randint(1, 12)
        self.nt0 = max(1, self.nt - r.choice([0, 1, 2])) if self.two else self.nt
        self.tail = r.random() < 0.6  # the last tile reaches past the segment
        self.partial = [[r.random() < 0.4 for _ in range(self.nt)] for _ in range(2)]
        self.bad = [[p and r.random() < 0.5 for p in row] for row in self.partial]
        self.xs = [0, 1] if self.two else [0]
        n = len(self.xs)
        self.q_full = self.bars("q_full", 2)
        self.checked = [self.bars(f"checked{i}_", 3) for i in range(2)]
        self.k_full, self.v_full = self.bars("k_full", 3), self.bars("v_full", 3)
        self.k_empty, self.v_empty = self.bars("k_empty", 3, n), self.bars("v_empty", 3, n if plant == "not counted" else 2 * n)
        self.s_full, self.pv_done = ([self.bars(f"{x}{i}_", 2) for i in range(2)] for x in ("s_full", "pv_done"))
        self.p_full = [self.bars(f"p_full{i}_", 2, 4) for i in range(2)]
        self.p_one = [Barrier(f"p_one{i}", 4) for i in range(2)]  # planted: one for both buffers
        self.v_tail, self.flag = Barrier("v_tail", 1), [[None] * 3 for _ in range(2)]

    def ntx(self, x):
        return self.nt0 if x == 0 else self.nt

    def copies(self):
        self.copy(self.q_full[0], ("Q", 0))
        for j in range(self.nt):
            s, use = j % 3, j // 3
            if use:
                yield ("wait", self.k_empty[s], use - 1)
                self.need(*[("S", x, j - 3) for x in self.xs if j - 3 < self.ntx(x)])
            self.copy(self.k_full[s], ("K", j))
            if j == 0 and self.two:
                self.copy(self.q_full[1], ("Q", 1))
            if use:
                yield ("wait", self.v_empty[s], use - 1)
                self.need(*[("PV", x, j - 3) for x in self.xs if j - 3 < self.ntx(x)], *[("look", x, j - 3) for x in self.xs])
            self.copy(self.v_full[s], ("V", j))
            yield self.delay(0, 50)

    def scores(self, x):
        yield ("wait", self.q_full[x], 0)
        for j in range(self.nt):
            s = j % 3
            yield ("wait", self.k_full[s], j // 3)
            if j < self.ntx(x):
                if j > 1 and self.plant != "S over P":
                    yield ("wait", self.pv_done[x][j & 1], (j >> 1) - 1)
                self.need(("K", j), ("Q", x))
                if j > 1:
                    self.need(("PV", x, j - 2))
                self.mma(f"S{x}", ("S", x, j))
                self.commit_of(f"S{x}", self.s_full[x][j & 1])
                self.commit_of(f"S{x}", self.k_empty[s])
            else:
                self.k_empty[s].arrive(self)
            yield self.delay(1, 60)

    def values(self, x):
        for j in range(self.nt):
            s = j % 3
            yield ("wait", self.v_full[s], j // 3)
            if j < self.ntx(x):
                if self.tail and j == self.nt - 1:
                    if x == self.xs[-1]:
                        yield self.delay(10, 900)
                        self.mark("tail is zero")
                        self.v_tail.arrive(self)
                    elif self.plant != "no wait for the tail":
                        yield ("wait", self.v_tail, 0)
                if self.plant == "one P barrier":
                    yield ("wait", self.p_one[x], j)
                else:
                    yield ("wait", self.p_full[x][j & 1], j >> 1)
                self.need(("V", j), *[("P", x, j, w) for w in range(4)])
                if self.tail and j == self.nt - 1:
                    self.need("tail is zero")
                if self.partial[x][j]:  # no wait of its own: the softmax warps had it before they wrote P
                    assert self.flag[x][s] == (j, self.bad[x][j]), "the flag of another tile"
                if self.bad[x][j]:
                    self.mark(("PV", x, j))
                else:
                    self.mma(f"PV{x}", ("PV", x, j))
                self.commit_of(f"PV{x}", self.pv_done[x][j & 1])
                self.commit_of(f"PV{x}", self.v_empty[s])
            else:
                self.v_empty[s].arrive(self)
            yield self.delay(1, 60)

    def look(self, x):
        for j in range(self.nt):
            s = j % 3
            yield ("wait", self.v_full[s], j // 3)
            self.need(("V", j))
            if j < self.ntx(x) and self.partial[x][j]:
                yield self.delay(50, 2500)
                self.flag[x][s] = (j, self.bad[x][j])
            self.mark(("look", x, j))
            self.checked[x][s].arrive(self)
            if self.plant != "not counted":
                self.v_empty[s].arrive(self)
            yield self.delay(1, 60) if self.rng.random() < 0.9 else self.delay(1000, 9000)

    def softmax(self, x, w):
        for j in range(self.ntx(x)):
            yield ("wait", self.s_full[x][j & 1], j >> 1)
            self.need(("S", x, j))
            yield self.delay(50, 900)
            rescale = self.rng.random() < 0.2 and j > 0
            if self.partial[x][j]:
                waits = [("wait", self.v_full[j % 3], j // 3), ("wait", self.checked[x][j % 3], j // 3)]
                if self.plant == "the look before the tile":
                    waits.reverse()
                if self.plant == "no wait for the look":
                    waits.pop()
                yield from waits
                assert self.flag[x][j % 3] == (j, self.bad[x][j]), "the flag of another tile"
                rescale = rescale or (self.bad[x][j] and j > 0)
            if rescale:
                yield ("wait", self.pv_done[x][(j - 1) & 1], (j - 1) >> 1)
                self.need(*[("PV", x, i) for i in range(j)])
                yield self.delay(10, 2000)
            self.mark(("P", x, j, w))
            (self.p_one[x] if self.plant == "one P barrier" else self.p_full[x][j & 1]).arrive(self)
        last = self.ntx(x) - 1
        yield ("wait", self.pv_done[x][last & 1], last >> 1)
        self.need(*[("PV", x, i) for i in range(last + 1)])

    def run(self):
        self.finish([self.copies()] + [f(x) for x in self.xs for f in (self.scores, self.values, self.look)] +
                    [self.softmax(x, w) for x in self.xs for w in range(4)])


# ---------------------------------------------------------------- weights

class Weights(Model):
    """One CTA's items of (heads, blocks); `teams` groups of four warps take the blocks in turn, each block in
    one of four score buffers."""

    def __init__(self, seed, plant=None, teams=3):
        super().__init__(seed, plant)
        r, self.teams = self.rng, teams
        self.items = [(r.randint(1, 4), r.randint(1, 6)) for _ in range(r.randint(1, 5))]
        self.ks = r.choice([1, 4])
        self.k_full, self.k_empty = self.bars("k_full", self.ks, 2), self.bars("k_empty", self.ks)
        self.q_full, self.q_empty = self.bars("q_full", 2), self.bars("q_empty", 2)
        self.s_full, self.s_empty = self.bars("s_full", 4), self.bars("s_empty", 4, 4)
        self.meet = {}  # a team's barriers: (team, number) -> warps there

    def heads(self):
        return range(sum(nh for nh, _ in self.items))

    def blocks(self):
        it = kc = 0
        for nh, nb in self.items:
            for _ in range(nh):
                for b in range(nb):
                    yield kc, b, nb, it
                    it += 1
                kc += 1

    def keys(self, w):
        for kc in self.heads():
            s, use = kc % self.ks, kc // self.ks
            if use:
                yield ("wait", self.k_empty[s], use - 1)
                self.need(("head", kc - self.ks))
            self.copy(self.k_full[s], ("K", kc, w))
            yield self.delay(0, 50)

    def queries(self):
        for *_, it in self.blocks():
            if it >= 2:
                yield ("wait", self.q_empty[it & 1], (it >> 1) - 1)
                self.need(("S", it - 2))
            self.copy(self.q_full[it & 1], ("Q", it))
            yield self.delay(0, 50)

    def scores(self):
        for kc, b, nb, it in self.blocks():
            if b == 0:
                yield ("wait", self.k_full[kc % self.ks], kc // self.ks)
            yield ("wait", self.q_full[it & 1], it >> 1)
            if it >= 4:
                if self.plant != "no wait for the score buffer":
                    yield ("wait", self.s_empty[it & 3], (it >> 2) - 1)
                self.need(*[("read", it - 4, w) for w in range(4)])
            self.need(("K", kc, 0), ("K", kc, 1), ("Q", it))
            self.mma("S", ("S", it))
            self.commit_of("S", self.q_empty[it & 1])
            self.commit_of("S", self.s_full[it & 3])
            if b == nb - 1:
                self.done_at[("head", kc)] = self.last["S"]
                self.commit_of("S", self.k_empty[kc % self.ks])
            yield self.delay(1, 60)

    def team(self, team, w):
        mine = [it for *_, it in self.blocks() if it % self.teams == team]
        for seq, it in enumerate(mine):
            # the column buffer seq & 1 may be written: its last readers, block seq - 2, are behind the
            # team's last barrier
            if seq >= 2:
                self.need(*[("columns", team, seq - 2, i) for i in range(4)])
            yield self.delay(1, 100)
            self.mark(("wrote columns", team, seq, w))
            self.meet[team, seq] = self.meet.get((team, seq), 0) + 1
            while self.plant != "no barrier of the team" and self.meet[team, seq] < 4:
                yield self.delay(5, 20)
            self.need(*[("wrote columns", team, seq, i) for i in range(4)])
            yield ("wait", self.s_full[it & 3], it >> 2)
            self.need(("S", it))
            yield self.delay(50, 900)
            self.mark(("read", it, w))
            self.mark(("columns", team, seq, w))
            self.s_empty[it & 3].arrive(self)

    def run(self):
        self.finish([self.keys(0), self.keys(1), self.queries(), self.scores()] +
                    [self.team(t, w) for t in range(self.teams) for w in range(4)])


def caught(make, seeds=300):
    n = 0
    for seed in range(seeds):
        try:
            make(seed).run()
        except AssertionError:
            n += 1
    return n


@pytest.mark.parametrize("producers", [1, 4])
def test_absorbed_protocol_is_sound(producers):
    for seed in range(600):
        Absorbed(seed, producers=producers).run()


@pytest.mark.parametrize("plant", ["refill on S", "idle warps run ahead", "P over a PV in flight", "no wait for the check"])
def test_absorbed_model_catches(plant):
    assert caught(lambda seed: Absorbed(seed, plant)) > 0


def test_expanded_protocol_is_sound():
    for seed in range(800):
        Expanded(seed).run()


@pytest.mark.parametrize("plant", ["one P barrier", "no wait for the tail", "S over P", "not counted", "no wait for the look",
                                   "the look before the tile"])
def test_expanded_model_catches(plant):
    assert caught(lambda seed: Expanded(seed, plant)) > 0


def test_weights_protocol_is_sound():
    for seed in range(600):
        Weights(seed).run()


@pytest.mark.parametrize("plant", ["no wait for the score buffer", "no barrier of the team"])
def test_weights_model_catches(plant):
    assert caught(lambda seed: Weights(seed, plant)) > 0


def test_more_teams_than_score_buffers_are_caught():
    """A team's next block must not share the buffer of one that another team may not have read yet."""
    assert caught(lambda seed: Weights(seed, teams=5)) > 0
