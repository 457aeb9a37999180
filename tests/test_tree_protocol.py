"""Model checks of the tree attention kernel (csrc/tree.cu, csrc/tree_plan.cu), no GPU.

Barriers: every warp role under random latencies, with waits that poll by parity (the Model of the latent kernels'
checks).  A parity wait is never ambiguous, no buffer is refilled, overwritten, rescaled or read before its last
users are done, every role finishes; planted mistakes are caught.

Shares: the plan's cuts give every tile of every unit to one CTA, their partials a slot each, and the join finds
exactly the pieces of each cut unit."""
import random

import pytest

from test_latent_protocol import Model, caught
from test_prefill_protocol import Barrier

SPLIT, PAIR, TURNS = "SPLIT", "PAIR", "TURNS"


class Tree(Model):
    """One CTA's run of pieces: (tiles, whether a pair has its second query tile, warps of a group without a row)."""

    def __init__(self, seed, form, plant=None, buffers=2):
        super().__init__(seed, plant)
        r = self.rng
        self.form, self.buffers, self.ns = form, buffers, r.choice([4, 6, 8])
        self.pieces = [(r.randint(1, 6), r.random() < 0.6, r.choice([0, 0, 1, 3])) for _ in range(r.randint(1, 6))]
        n = sum(p[0] for p in self.pieces)
        self.special = [r.random() < 0.4 for _ in range(n)]
        self.bad = [s and r.random() < 0.4 for s in self.special]
        self.rescale = [[r.random() < 0.3 for _ in range(n)] for _ in range(2)]
        two = lambda name, count=1: [self.bars(f"{name}{x}_", 2, count) for x in range(2)]
        self.q_full, self.q_empty = self.bars("q_full", 2), self.bars("q_empty", 2)
        self.s_full, self.p_full, self.pv_done = two("s_full"), two("p_full", 4), two("pv_done")
        self.o_final, self.checked = self.bars("o_final", 2), self.bars("checked", 2)
        self.o_free, self.joint = self.bars("o_free", 2, 8 if form == SPLIT else 4), Barrier("joint", 8)
        self.kv_full, self.kv_empty = self.bars("kv_full", self.ns), self.bars("kv_empty", self.ns)
        self.flag, self.seen = [None, None], {}

    def takes(self, p, x, j):
        if self.form == SPLIT:
            return j % 2 == x
        if self.form == TURNS:
            return p % 2 == x
        return x == 0 or self.pieces[p][1]

    def tiles(self):
        """(piece, tile of the piece, tiles, groups that take it, tile of the run)"""
        it = 0
        for p, (n, _, _) in enumerate(self.pieces):
            for j in range(n):
                yield p, j, n, [x for x in (0, 1) if self.takes(p, x, j)], it
                it += 1

    def users(self, what, it):
        xs = [t[3] for t in self.tiles()][it]
        return [(what, x, it) for x in xs]

    def copies(self, kv):
        for p, j, n, xs, it in self.tiles():
            if kv == 0 and j == 0:
                qs, ph = (p % 2, p // 2) if self.buffers == 2 else (0, p)
                if ph > 0:
                    yield ("wait", self.q_empty[qs], ph - 1)
                    old = p - self.buffers
                    self.need(*[u for q, _, _, _, k in self.tiles() if q == old for u in self.users("S", k)])
                self.copy(self.q_full[qs], ("Q", p))
            i = 2 * it + kv
            s, use = i % self.ns, i // self.ns
            if use:
                yield ("wait", self.kv_empty[s], use - 1)
                self.need(*self.users("PV" if kv else "S", (i - self.ns) // 2))
            self.copy(self.kv_full[s], ("V" if kv else "K", it))
            yield self.delay(0, 50)

    def scores(self):
        done = [0, 0]
        for p, j, n, xs, it in self.tiles():
            qs, ph = (p % 2, p // 2) if self.buffers == 2 else (0, p)
            if j == 0:
                yield ("wait", self.q_full[qs], ph)
            s = 2 * it % self.ns
            yield ("wait", self.kv_full[s], 2 * it // self.ns)
            for x in xs:
                k, b = done[x], done[x] & 1
                if k >= 2 and self.plant != "S over P":
                    yield ("wait", self.pv_done[x][b], (k >> 1) - 1)
                if k >= 2:
                    self.need(("PVn", x, k - 2), *[("read S", x, k - 2, w) for w in range(4)])
                self.need(("K", it), ("Q", p))
                self.mma("S", ("S", x, it))
                self.done_at["Sn", x, k] = self.done_at["S", x, it]
                self.commit_of("S", self.s_full[x][b])
                done[x] += 1
                yield self.delay(1, 60)
            self.commit_of("S", self.kv_empty[s])
            if j == n - 1:
                self.commit_of("S", self.q_empty[qs])

    def o_read(self, p, groups):
        return [("read O", p, x, w) for x in groups for w in range(4)]

    def old_o(self, p, x):
        """The reads that must be over before PV of piece p may write the accumulator of group x."""
        if self.form == SPLIT:
            return self.o_read(p - 1, (0, 1)) if p else []
        if self.form == TURNS:  # one accumulator
            return self.o_read(p - 1, (1 - x,)) if p else []
        last = [q for q in range(p) if self.takes(q, x, 0)]
        return self.o_read(last[-1], (x,)) if last else []

    def values(self):
        done, pieces = [0, 0], [0, 0]
        for p, j, n, xs, it in self.tiles():
            if j == 0 and self.plant != "O while it is read":
                if self.form == SPLIT:
                    if p:
                        yield ("wait", self.o_free[0], p - 1)
                else:
                    for x in xs:
                        y = 1 - x if self.form == TURNS else x
                        if pieces[y]:
                            yield ("wait", self.o_free[y], pieces[y] - 1)
            s = (2 * it + 1) % self.ns
            yield ("wait", self.kv_full[s], (2 * it + 1) // self.ns)
            self.need(("V", it))
            if self.special[it]:
                yield self.delay(50, 500)
                for x in xs:
                    self.flag[x] = (it, self.bad[it])
                    self.checked[x].arrive(self)
            for x in xs:
                k, b = done[x], done[x] & 1
                yield ("wait", self.p_full[x][b], k >> 1)
                self.need(*[("P", x, k, w) for w in range(4 - self.pieces[p][2])])
                if j < (2 if self.form == SPLIT else 1):
                    self.need(*self.old_o(p, x))
                if self.bad[it]:
                    self.mark(("PV", x, it))
                else:
                    self.mma("PV", ("PV", x, it))
                self.done_at["PVn", x, k] = self.done_at["PV", x, it]
                self.commit_of("PV", self.pv_done[x][b])
                if j == n - 1:
                    self.commit_of("PV", self.o_final[0 if self.form == SPLIT else x])
                    pieces[x] += 1
                done[x] += 1
                yield self.delay(1, 60)
            self.commit_of("PV", self.kv_empty[s])

    def softmax(self, x, w):
        k = checks = pieces = 0
        it0 = 0
        for p, (n, _, idle) in enumerate(self.pieces):
            first_it, it0 = it0, it0 + n
            if self.form != SPLIT and not self.takes(p, x, 0):
                continue
            mine = [j for j in range(n) if self.takes(p, x, j)]
            for j in mine:
                it, b = first_it + j, k & 1
                first = j < (2 if self.form == SPLIT else 1)
                if not (self.plant == "idle warps run ahead" and w >= 4 - idle):
                    yield ("wait", self.s_full[x][b], k >> 1)
                    self.need(("S", x, it))
                if w >= 4 - idle:
                    self.mark(("read S", x, k, w))
                    if self.special[it]:
                        yield ("wait", self.checked[x], checks)
                        checks += 1
                    self.p_full[x][b].arrive(self)
                    k += 1
                    continue
                yield self.delay(50, 900)
                self.mark(("read S", x, k, w))
                rows = False
                if self.special[it]:
                    if self.plant != "no wait for the look":
                        yield ("wait", self.checked[x], checks)
                    checks += 1
                    assert self.flag[x] == (it, self.bad[it]), "the flag of another tile"
                    rows = self.bad[it]
                if rows or (self.rescale[x][it] and not first):
                    if not first and self.plant != "O under a PV":
                        yield ("wait", self.pv_done[x][1 - b], (k - 1) >> 1)
                    if not first:
                        self.need(("PVn", x, k - 1))
                    else:
                        self.need(*self.old_o(p, x))
                    if rows:
                        self.need(("V", it))
                    yield self.delay(100, 2000)
                    if rows:
                        assert ("PV", x, it) not in self.done_at
                self.mark(("P", x, k, w))
                self.p_full[x][b].arrive(self)
                k += 1
            if self.form == SPLIT:
                self.seen[p, x, w] = self.t
                self.joint.arrive(self)
                yield ("wait", self.joint, pieces)
                assert all((p, y, v) in self.seen for y in (0, 1) for v in range(4))
            yield ("wait", self.o_final[0 if self.form == SPLIT else x], pieces)
            pieces += 1
            self.need(*[("PV", y, first_it + j) for y in ((0, 1) if self.form == SPLIT else (x,)) for j in range(n)
                        if self.takes(p, y, j)])
            yield self.delay(50, 2000)
            self.mark(("read O", p, x, w))
            self.o_free[0 if self.form == SPLIT else x].arrive(self)

    def run(self):
        self.finish([self.copies(0), self.copies(1), self.scores(), self.values()] +
                    [self.softmax(x, w) for x in range(2) for w in range(4)])


@pytest.mark.parametrize("form,buffers", [(SPLIT, 2), (PAIR, 2), (TURNS, 2), (TURNS, 1)])
def test_the_protocol_is_sound(form, buffers):
    for seed in range(250):
        Tree(seed, form, buffers=buffers).run()


@pytest.mark.parametrize("form", [SPLIT, PAIR, TURNS])
@pytest.mark.parametrize("plant", ["S over P", "O while it is read", "idle warps run ahead", "no wait for the look", "O under a PV"])
def test_mistakes_are_caught(form, plant):
    assert caught(lambda seed: Tree(seed, form, plant)) > 0


# ---------------------------------------------------------------- the plan's shares

TILE, HALF, PIECE, LEAST, LEAST_WHOLE = 3, 2, 6, 12, 8  # costs, in thirds of a tile


class Row:
    """nc tiles of cached keys, n drafted tokens in units of `unit` (a unit of up to half as many is a half)."""

    def __init__(self, nc, n, unit, pair):
        self.nc, self.n, self.unit, self.pair = nc, n, unit, pair
        self.units = -(-n // unit)

    def tiles(self, q):
        return self.nc + -(-min(self.n, (q + 1) * self.unit) // 64)

    def each(self, q):
        return HALF if self.pair and self.n - q * self.unit <= self.unit // 2 else TILE

    def cost(self, q):
        return self.tiles(q) * self.each(q) + PIECE

    def head(self):
        return sum(self.cost(q) for q in range(self.units))


def plan(rows, kv_heads, ctas, whole):
    lanes = next(h for h in range(min(kv_heads, ctas), 0, -1) if kv_heads % h == 0 and ctas % h * 32 <= ctas)
    heads, slices, before = kv_heads // lanes, ctas // lanes, [0]
    for r in rows:
        before.append(before[-1] + heads * r.head())
    total, starts = before.pop(), []
    share = max(-(-total // slices), LEAST_WHOLE if whole else LEAST)
    for c in range(ctas):
        piece = c // lanes

        def place(at):
            if at >= total:
                return (len(rows), 0, 0), 0, 0
            r = max(i for i, v in enumerate(before) if v <= at)
            row, off = rows[r], at - before[r]
            q, inside = 0, off % row.head()
            while inside >= row.cost(q):
                inside -= row.cost(q)
                q += 1
            each, begin, unit = row.each(q), at - inside, off // row.head() * row.units + q
            if whole:
                return (r, unit, 0), 0, 0
            return ((r, unit, max(0, inside - PIECE) // each), (begin + PIECE + each - 1) // share,
                    (begin + row.cost(q) - 1) // share)
        a, b = (place((piece + i) * share if piece < slices else total) for i in (0, 1))
        starts.append(dict(cta=c, lane=c % lanes, begin=a[0], end=b[0], tail=b[2] - b[1] + 1, lanes=lanes))
    return starts


def join_blocks(dim, warps, rows, count):
    """Blocks of the join of a unit: two pieces of a thread on their way at once."""
    groups, side = min(dim // 16, warps).bit_length() - 1, 4 if rows <= 8 else 2 if rows <= 16 else 1
    room, cut = (warps >> groups) * side * 2, 1  # cut: blocks that share rows
    while room < count and (groups or side < 4):
        groups, side, cut, room = (groups - 1, side, cut, 2 * room) if groups else (0, 2 * side, 2 * cut, 2 * room)
    return cut * ((dim // 16) >> groups)


def pieces(rows, kv_heads, s):
    (r, unit, tile), out = s["begin"], []
    while (r, unit, tile) < s["end"]:
        units = rows[r].units
        if unit >= kv_heads // s["lanes"] * units:
            r, unit = r + 1, 0
            continue
        cut = (r, unit) == s["end"][:2]
        head, q = unit // units * s["lanes"] + s["lane"], unit % units
        end = s["end"][2] if cut else rows[r].tiles(q)
        slot = 2 * s["cta"] if tile else 2 * s["cta"] + 1 if cut else None
        assert end > tile
        out.append(((r, head, q), tile, end, slot))
        unit, tile = unit + 1, 0
    return out


@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 152, 300])
def test_shares_and_joins(ctas):
    rng = random.Random(ctas)
    for _ in range(120):
        kv_heads, unit, pair, whole = rng.choice([1, 2, 3, 4, 8, 5, 16, 100]), rng.choice([8, 16, 42, 128]), rng.random() < 0.5, rng.random() < 0.2
        same, most = rng.random() < 0.5, rng.choice([1, 16, 60, 256])
        rows = [Row(0, 0, unit, pair) if rng.random() < 0.2 else
                Row(rng.choice([0, 1, 2, 9, 99, 999]), most if same else rng.randint(1, most), unit, pair) for _ in range(rng.randint(1, 30))]
        starts = plan(rows, kv_heads, ctas, whole)
        got, slots = {}, {}
        for s in starts:
            for what, begin, end, slot in pieces(rows, kv_heads, s):
                got.setdefault(what, []).append((begin, end, slot))
                if slot is not None:
                    assert slot not in slots and slot < 2 * ctas
                    slots[slot] = what
        assert set(got) == {(r, h, q) for r, row in enumerate(rows) for h in range(kv_heads) for q in range(row.units)}
        assert not (whole and slots)
        joined = {}
        for s in starts:
            (r, unit, tile), begin = s["end"], s["begin"]
            if r < len(rows) and tile and not (begin[:2] == (r, unit) and begin[2]):  # the unit that goes on begins here
                mine = [2 * s["cta"] + 1] + [2 * (s["cta"] + i * s["lanes"]) for i in range(1, s["tail"])]
                assert len({slots[x] for x in mine}) == 1
                joined[slots[mine[0]]] = mine
        for what, parts in got.items():
            parts.sort()
            assert parts[0][0] == 0 and parts[-1][1] == rows[what[0]].tiles(what[2])
            assert all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
            assert joined.get(what) == ([p[2] for p in parts] if len(parts) > 1 else None)
        for dim, warps in ((64, 4), (64, 8), (128, 8), (128, 16), (256, 8), (256, 16)):  # the joins' records fit their list
            blocks = sum(join_blocks(dim, warps, rng.choice([4, 8, 9, 128]), len(mine)) for mine in joined.values())
            assert blocks <= ctas * (2 if dim == 256 else 1)
        lanes = starts[0]["lanes"]
        if whole and kv_heads // lanes * sum(r.head() for r in rows) <= LEAST_WHOLE * (ctas // lanes):
            assert all(len(pieces(rows, kv_heads, s)) <= 1 for s in starts), "units that stay whole, one a CTA"
