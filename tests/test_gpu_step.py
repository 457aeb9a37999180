"""Page and slot maps, acceptance, and whole speculative steps on the GPU against their definitions (whole numbers
and copied values: equal bit by bit)."""
import numpy as np
import pytest
import torch

import tree_ref as R
from paged_kv_attention_gqa_gb300 import binding as B
from test_gpu_tree import compare, i32, randn

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def _build():
    from paged_kv_attention_gqa_gb300 import build
    build.build()


def full(n, value=-1):
    return torch.full((n,), value, dtype=torch.int32, device="cuda")


class Maps:
    """Rows of these lengths over shuffled pages; run() calls the kernel, want() the definition."""

    def __init__(self, seq, new, held, P, seed, *, free=None, width=None, tokens=None, indices=None, room=None):
        g = np.random.default_rng(seed)
        need = [-(-(a + b) // P) for a, b in zip(seq, new)]
        self.P, self.seq, self.new, self.held = P, list(seq), list(new), list(held)
        width = max(1, max(need, default=0), max(held, default=0)) + 2 if width is None else width
        free = sum(max(0, n - h) for n, h in zip(need, held)) + 3 if free is None else free
        ids = g.permutation(sum(max(0, h) for h in held) + free + 4).tolist()
        self.table = [[ids.pop() if b < h else -9 for b in range(width)] for h in held]
        self.count = free
        self.free = [ids.pop() for _ in range(free)] + [-8] * (sum(max(0, h) for h in held) if room is None else room)
        self.tokens = sum(new) + 5 if tokens is None else tokens
        self.kvi = [-7] * (sum(need) + 4 if indices is None else indices)
        self.h = B.Handle(num_qo_heads=1, num_kv_heads=1, head_dim=64, page_size=P, max_batch=max(1, len(seq)), max_num_pages=1,
                          num_cache_pages=1)

    def want(self):
        return R.maps(self.seq, self.new, self.table, self.held, self.free, self.count, self.P, self.kvi, self.tokens)

    def run(self, in_place=False, slots=True, positions=True, wide=0, stream=None):
        n = len(self.seq)
        table = np.asarray(self.table, np.int32).reshape(n, len(self.table[0]) if n else 1)
        whole = torch.full((n, table.shape[1] + wide), -6, dtype=torch.int32, device="cuda")
        whole[:, : table.shape[1]] = torch.from_numpy(table).cuda()
        d = dict(table=whole[:, : table.shape[1]], held=i32(self.held), free=i32(self.free), count=i32([self.count]), qo=full(n + 1),
                 kvp=full(n + 1), kvi=i32(self.kvi), last=full(n), status=full(1),
                 slots=full(self.tokens) if slots else None, positions=full(self.tokens) if positions else None)
        held_out, count_out = (d["held"], d["count"]) if in_place else (full(n), full(1))
        self.h.build_maps(i32(self.seq), i32(self.new), d["table"], d["held"], d["free"], d["count"], qo_indptr=d["qo"],
                          kv_indptr=d["kvp"], kv_indices=d["kvi"], last_page_len=d["last"], slots=d["slots"],
                          positions=d["positions"], status=d["status"], num_blocks_out=None if in_place else held_out,
                          free_count_out=None if in_place else count_out, stream=stream)
        torch.cuda.synchronize()
        if wide:
            assert (whole[:, table.shape[1]:] == -6).all(), "behind the table's columns"
        out = {k: v.tolist() for k, v in d.items() if v is not None}
        out["held"], out["count"] = held_out.tolist(), count_out.tolist()[0]
        return out

    def check(self, **kw):
        want, got = self.want(), self.run(**kw)
        n = len(self.seq)
        if not isinstance(want, dict):  # nothing changes and the step is empty
            assert got["status"] == [want]
            want = dict(qo=[0] * (n + 1), kvp=[0] * (n + 1), kvi=self.kvi, last=[0] * n, slots=[-1] * self.tokens,
                        positions=[0] * self.tokens, held=self.held, count=self.count, table=self.table, free=self.free)
        else:
            assert got["status"] == [0]
        for k, v in want.items():
            if k in got:
                assert got[k] == v, (k, got[k], v)


MAPS = {
    "one row": dict(seq=[517], new=[8], held=[33], P=16),
    "a first token": dict(seq=[0], new=[1], held=[0], P=16),
    "page edges": dict(seq=[15, 16, 17, 31, 32, 0], new=[1, 1, 1, 1, 1, 16], held=[1, 1, 2, 2, 2, 0], P=16),
    "no new tokens": dict(seq=[15, 16, 0, 40], new=[0, 0, 0, 0], held=[1, 1, 0, 3], P=16),
    "pages too many": dict(seq=[15, 16, 30, 40], new=[3, 1, 2, 0], held=[2, 9, 4, 5], P=16),
    "rows that ended": dict(seq=[0, 100, 0, 50, 0], new=[0, 30, 0, 17, 0], held=[7, 7, 1, 4, 0], P=16),
    "only given back": dict(seq=[0, 0], new=[0, 0], held=[5, 3], P=8),
    "taken from those given back": dict(seq=[0, 10, 5], new=[0, 200, 100], held=[30, 1, 1], P=8, free=2),
    "page size 1": dict(seq=[3, 0, 9], new=[2, 5, 0], held=[3, 0, 10], P=1),
    "page size 1024": dict(seq=[1023, 1024, 5000], new=[1, 1, 3000], held=[1, 1, 5], P=1024),
    "prompts": dict(seq=[0] * 5, new=[3000, 1, 777, 4096, 16], held=[0] * 5, P=16),
    "no rows": dict(seq=[], new=[], held=[], P=16),
    "exactly enough pages": dict(seq=[16, 16], new=[16, 1], held=[1, 1], P=16, free=2),
    "exact capacities": dict(seq=[16, 3], new=[5, 2], held=[1, 1], P=16, tokens=7, indices=3, width=2, free=1, room=0),
    "a page short": dict(seq=[16, 16], new=[16, 1], held=[1, 1], P=16, free=1),
    "many pages short": dict(seq=[16, 0], new=[1600, 0], held=[1, 3], P=16, free=0),
    "negative length": dict(seq=[16, -1], new=[1, 1], held=[1, 1], P=16, width=5),
    "negative new": dict(seq=[16, 4], new=[1, -1], held=[1, 1], P=16, width=5, tokens=9),
    "row past the table": dict(seq=[16, 40], new=[1, 9], held=[1, 3], P=16, width=3),
    "held past the table": dict(seq=[16, 4], new=[1, 9], held=[1, 4], P=16, width=3),
    "tokens past the slots": dict(seq=[16, 4], new=[7, 9], held=[2, 1], P=16, tokens=15),
    "pages past the list": dict(seq=[16, 4], new=[7, 9], held=[2, 1], P=16, indices=2),
    "stack too small": dict(seq=[0, 4], new=[0, 9], held=[5, 1], P=16, free=1, room=3),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", sorted(MAPS))
def test_maps(case, in_place):
    Maps(seed=3, **MAPS[case]).check(in_place=in_place)


def test_maps_with_some_outputs_and_a_strided_table():
    for slots in (False, True):
        for positions in (False, True):
            m = Maps([100, 0, 30], [9, 4, 0], [7, 0, 3], 16, 4)
            m.check(slots=slots, positions=positions, wide=3)


def test_maps_counts_outside_the_stack():
    for count in (-1, 99):
        m = Maps([16], [1], [1], 16, 5, room=0)
        m.count = count
        m.check()


@pytest.mark.parametrize("rows", [511, 512, 513, 1500, 8192])
def test_maps_of_many_rows(rows):
    g = np.random.default_rng(rows)
    seq = g.integers(0, 400, rows)
    new = np.where(g.random(rows) < 0.2, 0, g.integers(0, 40, rows))
    seq = np.where(g.random(rows) < 0.1, 0, seq)
    held = -(-seq // 8) + g.integers(0, 3, rows)
    for in_place in (False, True):
        Maps(seq.tolist(), new.tolist(), held.tolist(), 8, rows, width=64).check(in_place=in_place)


class Accept:
    """A planned step of trees with tokens; run() accepts, check() compares with the walk by the definition."""

    def __init__(self, ctx, trees, draft, target, *, Hkv=2, D=64, P=16, layers=3, seed=0, kind=torch.int64):
        self.ctx, self.trees, self.kind = ctx, trees, kind
        news = [len(t) for t in trees]
        self.qo = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        T, self.tail = int(self.qo[-1]), 2
        self.T = T
        self.kvp, self.kvi, self.last, pages = R.indices([c + n for c, n in zip(ctx, news)], P, seed)
        self.draft, self.target = draft, target
        self.cache = randn(seed, layers, pages, 2, P, Hkv, D)
        self.new = randn(seed + 1, layers, T + self.tail, 2, Hkv, D)
        self.h = B.Handle(num_qo_heads=Hkv, num_kv_heads=Hkv, head_dim=D, page_size=P, max_batch=max(1, len(ctx)),
                          max_total_tokens=T + self.tail, max_num_pages=max(1, len(self.kvi)), num_cache_pages=pages)
        self.ws = torch.empty(self.h.workspace_size(B.MODE_TREE), dtype=torch.uint8, device="cuda")
        self.dev = [i32(x) for x in (self.qo, self.kvp, self.kvi, self.last)]

    def plan(self):
        parents = i32([p for t in self.trees for p in t] + [0] * self.tail)
        self.h.plan_tree(*self.dev, parents, num_tokens=self.T + self.tail, max_new=max(1, max(len(t) for t in self.trees)),
                         workspace=self.ws)

    def run(self, new=None, cache=None, seq=True):
        n = len(self.ctx)
        self.got_cache = self.cache.cuda() if cache is None else cache
        new = self.new.cuda() if new is None else new
        tok = lambda x: torch.tensor(list(x) + [5] * self.tail, dtype=self.kind, device="cuda")
        self.accepted, self.count, self.seq = full(self.T + self.tail, -4), full(n), full(n, -3)
        self.next = torch.full((n,), -3, dtype=self.kind, device="cuda")
        self.h.run_accept(tok(self.draft), tok(self.target), new[:, :, 0], new[:, :, 1], self.got_cache, self.accepted,
                          self.count, self.next, self.seq if seq else None, workspace=self.ws)
        torch.cuda.synchronize()

    def check(self, seq=True):
        assert self.h.check_device_error(self.ws) == 0
        want, accepted, count, follow = self.cache.clone(), [], [], []
        P = self.cache.shape[3]
        for r, t in enumerate(self.trees):
            a, b = int(self.qo[r]), int(self.qo[r + 1])
            path, nxt = R.accept(t, list(self.draft[a:b]), list(self.target[a:b]))
            for i, j in enumerate(path):
                pos = self.ctx[r] + i
                want[:, int(self.kvi[self.kvp[r] + pos // P]), :, pos % P] = self.new[:, a + j]
            accepted += path + [-1] * (b - a - len(path))
            count.append(len(path))
            follow.append(nxt)
        assert self.accepted.tolist() == accepted + [-4] * self.tail
        assert self.count.tolist() == count and self.next.tolist() == follow
        assert self.seq.tolist() == [c + n if seq and n else -3 for c, n in zip(self.ctx, count)]
        assert torch.equal(self.got_cache.cpu().view(torch.int16), want.view(torch.int16)), "cache"


def walk(trees, seed, vocabulary=1000, share=0.8):
    """Tokens with which most nodes are confirmed by one of their children."""
    g = np.random.default_rng(seed)
    draft, target = [], []
    for t in trees:
        d, x = g.integers(0, vocabulary, len(t)), g.integers(0, vocabulary, len(t))
        for i in range(len(t)):
            kids = [j for j in range(len(t)) if t[j] == i]
            if kids and g.random() < share:
                x[i] = d[g.choice(kids)]
        draft += d.tolist()
        target += x.tolist()
    return draft, target


ACCEPT = {
    "one row": dict(ctx=[100], trees=[R.tree(8, 3)]),
    "roots alone": dict(ctx=[0, 15, 16], trees=[R.tree(1, 1)] * 3),
    "ragged": dict(ctx=[0, 7, 15, 16, 100, 5], trees=[R.tree(9, 3), R.tree(40, 2, 1), [], R.tree(64, 5), R.tree(33, 4, 2), []]),
    "chains": dict(ctx=[30, 0, 47], trees=[R.tree(70, 1), R.tree(256, 1), R.tree(5, 1)]),
    "several roots": dict(ctx=[12, 3], trees=[[-1, -1, 0, 1, 2, -1], [-1, 0, -1, 1]]),
    "nothing": dict(ctx=[4, 0], trees=[[], []]),
}


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("case", sorted(ACCEPT))
def test_accept(case, kind):
    for seed, (D, Hkv, P, layers) in enumerate([(64, 2, 16, 3), (128, 8, 8, 5), (256, 1, 64, 1), (64, 3, 16, 33), (256, 9, 8, 2), (64, 1, 32, 4)]):
        draft, target = walk(ACCEPT[case]["trees"], seed, share=[0.8, 1.0, 0.0, 0.95, 1.0, 0.9][seed])
        a = Accept(draft=draft, target=target, D=D, Hkv=Hkv, P=P, layers=layers, seed=seed, kind=kind, **ACCEPT[case])
        a.plan()
        a.run()
        a.check()


def test_accept_many_rows():
    trees = [R.tree(1 + r % 20, 1 + r % 4, r) for r in range(300)]
    draft, target = walk(trees, 1)
    a = Accept([r % 50 for r in range(300)], trees, draft, target, layers=7, seed=2)
    a.plan()
    a.run(seq=False)
    a.check(seq=False)


def test_accept_ties_and_wide_tokens():
    """Equal children: the first one; tokens that agree in their lower 32 bits alone do not agree; negative tokens."""
    t = [-1, 0, 0, 0, 1, 2, 2]
    a = Accept([20], [t], [9, 5, 5, 5, 6, 7, 7], [5, 0, 7, 0, 1, 1, 1])
    a.plan()
    a.run()
    a.check()
    assert a.accepted.tolist()[:2] == [0, 1]  # not 2, behind which there would be more
    big = 5 + (1 << 32)
    a = Accept([20], [t], [9, 5, big, 5, 6, 7, 7], [big, 0, -7, 0, 1, 1, 1])
    a.plan()
    a.run()
    a.check()
    assert a.accepted.tolist()[:3] == [0, 2, -1] and a.next.tolist() == [-7]


def test_accept_strided_layers():
    """Drafted keys and values as [tokens, layers, ...], and every other layer of a cache."""
    trees = [R.tree(9, 3), R.tree(12, 2)]
    draft, target = walk(trees, 3, share=1.0)
    a = Accept([40, 3], trees, draft, target, layers=4, seed=5)
    a.plan()
    new = a.new.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    assert not new.is_contiguous()
    twice = torch.full((8, *a.cache.shape[1:]), 3.0, dtype=torch.bfloat16, device="cuda")
    twice[::2] = a.cache.cuda()
    a.run(new=new, cache=twice[::2])
    a.check()
    assert (twice[1::2] == 3).all()


def test_accept_reports_pages_outside_the_cache():
    a = Accept([20, 30], [R.tree(9, 1), R.tree(5, 1)], [1] * 14, [1] * 14)
    a.dev[2][1] = a.h.cfg.num_cache_pages  # the page of row 0's slots 16 to 31, which takes all of its path
    a.plan()
    a.run()
    assert a.h.check_device_error(a.ws) == 6
    assert a.count.tolist() == [9, 5]
    changed = (a.got_cache.cpu().view(torch.int16) != a.cache.view(torch.int16)).flatten(4).any(-1).any(0)  # [pages, 2, P]
    rows = {int(p) for p in changed.any(-1).any(-1).nonzero()[:, 0]}
    assert rows == {int(x) for x in a.kvi[a.kvp[1] + 30 // 16:]}, "row 1's path alone"


def test_accept_of_rows_that_overlap():
    """Offsets that go back: the row after that, which would have tokens of an earlier one, counts as empty too, and its
    nodes do not mix with theirs."""
    a = Accept([20, 30, 40, 50], [R.tree(5, 1), R.tree(4, 2), R.tree(5, 1), R.tree(12, 1)], [7] * 26, [7] * 26)
    a.dev[0][2] = 2  # tokens [0, 5), [5, 2), [2, 14) and [14, 26)
    a.plan()
    assert a.h.check_device_error(a.ws) == 5
    a.run()
    assert a.count.tolist() == [5, 0, 0, 12] and a.next.tolist() == [7, -1, -1, 7] and a.seq.tolist() == [25, -3, -3, 62]
    assert a.accepted.tolist() == list(range(5)) + [-4] * 9 + list(range(12)) + [-4] * a.tail
    want, P = a.cache.clone(), a.cache.shape[3]
    for r, begin in ((0, 0), (3, 14)):
        for i in range(a.count[r].item()):
            pos = a.ctx[r] + i
            want[:, int(a.kvi[a.kvp[r] + pos // P]), :, pos % P] = a.new[:, begin + i]
    assert torch.equal(a.got_cache.cpu().view(torch.int16), want.view(torch.int16))


def test_accept_of_rows_that_overlap_far_apart():
    """Offsets that go back behind hundreds of rows."""
    n = 700
    a = Accept([3] * n, [R.tree(2, 1)] * n, [7] * (2 * n), [7] * (2 * n))
    a.dev[0][600], a.dev[0][601] = 4, 6  # row 599 ends before it begins, row 600 has row 2's tokens, row 601 too many
    a.plan()
    assert a.h.check_device_error(a.ws) == 5
    a.run()
    assert a.count.tolist() == [0 if r in (599, 600, 601) else 2 for r in range(n)]


class Loop:
    """Speculative steps one after another, all state on the device; mirror() replays them by the definitions."""

    def __init__(self, lens, H, Hkv, D, P, layers, width, seed, most):
        self.lens, self.P, self.layers, self.most = lens, P, layers, most
        R_, n = len(lens), len(lens) * most
        pages = 64 + sum(-(-(L + 60) // P) for L in lens)
        g = np.random.default_rng(seed)
        ids = g.permutation(pages).tolist()
        held = [-(-L // P) for L in lens]
        table = [[ids.pop() if b < h else -9 for b in range(width)] for h in held]
        self.state = dict(seq=list(lens), table=table, held=held, free=ids + [-8] * sum(held), count=len(ids))
        self.cache = randn(seed, layers, pages, 2, P, Hkv, D)
        self.h = B.Handle(num_qo_heads=H, num_kv_heads=Hkv, head_dim=D, page_size=P, max_batch=R_, max_total_tokens=n,
                          max_num_pages=R_ * width, num_cache_pages=pages)
        self.ws = torch.empty(self.h.workspace_size(B.MODE_TREE), dtype=torch.uint8, device="cuda")
        s, bf = self.state, torch.bfloat16
        self.d = dict(seq=i32(s["seq"]), new=full(R_, 0), table=i32(s["table"]), held=i32(s["held"]), free=i32(s["free"]),
                      count=i32([s["count"]]), qo=full(R_ + 1), kvp=full(R_ + 1), kvi=full(R_ * width), last=full(R_), slots=full(n),
                      pos=full(n), status=full(1), parents=full(n), draft=full(n, 0), target=full(n, 0), accepted=full(n),
                      num=full(R_), next=full(R_), cache=self.cache.cuda(), q=torch.zeros(layers, n, H, D, dtype=bf, device="cuda"),
                      kv=torch.zeros(layers, n, 2, Hkv, D, dtype=bf, device="cuda"), depth=full(n),
                      out=torch.zeros(layers, n, H, D, dtype=bf, device="cuda"), lse=torch.zeros(layers, n, H, device="cuda"))

    def step(self):
        """All calls of one step: nothing of it depends on the host."""
        d, h, ws = self.d, self.h, self.ws
        h.build_maps(d["seq"], d["new"], d["table"], d["held"], d["free"], d["count"], qo_indptr=d["qo"], kv_indptr=d["kvp"],
                     kv_indices=d["kvi"], last_page_len=d["last"], slots=d["slots"], positions=d["pos"], status=d["status"])
        h.plan_tree(d["qo"], d["kvp"], d["kvi"], d["last"], d["parents"], num_tokens=len(d["parents"]), max_new=self.most,
                    positions=d["depth"], workspace=ws)
        for l in range(self.layers):
            h.run_tree(d["q"][l], d["kv"][l, :, 0], d["kv"][l, :, 1], d["cache"][l], d["out"][l], d["lse"][l], workspace=ws)
        h.run_accept(d["draft"], d["target"], d["kv"][:, :, 0], d["kv"][:, :, 1], d["cache"], d["accepted"], d["num"], d["next"],
                     d["seq"], workspace=ws)

    def feed(self, trees, seed):
        """The step's inputs into the fixed tensors."""
        d, n = self.d, sum(len(t) for t in trees)
        self.trees, self.tokens = trees, walk(trees, seed)
        self.q, self.kv = randn(seed, *d["q"].shape), randn(seed + 1, *d["kv"].shape)
        d["q"].copy_(self.q)
        d["kv"].copy_(self.kv)
        d["new"].copy_(i32([len(t) for t in trees]))
        for name, x in (("parents", [p for t in trees for p in t]), ("draft", self.tokens[0]), ("target", self.tokens[1])):
            d[name][:n] = i32(x)

    def mirror(self):
        """The same step on the host, and what the device must hold now."""
        s, d, P = self.state, self.d, self.P
        new = [len(t) for t in self.trees]
        m = R.maps(s["seq"], new, s["table"], s["held"], s["free"], s["count"], P, [-1] * len(d["kvi"]), len(d["slots"]))
        assert isinstance(m, dict)
        nnz = m["kvp"][-1]
        assert d["status"].tolist() == [0] and d["qo"].tolist() == m["qo"] and d["kvp"].tolist() == m["kvp"]
        assert d["kvi"].tolist()[:nnz] == m["kvi"][:nnz] and d["last"].tolist() == m["last"] and d["slots"].tolist() == m["slots"]
        T = m["qo"][-1]
        for l in range(self.layers):
            ref = R.attention(self.q[l, :T], self.kv[l, :T, 0], self.kv[l, :T, 1], self.cache[l], m["qo"], np.array(m["kvp"]),
                              np.array(m["kvi"]), m["last"], self.trees, R.default_scale(self.q.shape[-1]))
            compare(d["out"][l, :T], d["lse"][l, :T], ref, f"layer {l}")
        num = []
        for r, t in enumerate(self.trees):
            a, b = m["qo"][r], m["qo"][r + 1]
            path, _ = R.accept(t, self.tokens[0][a:b], self.tokens[1][a:b])
            for i, j in enumerate(path):
                pos = s["seq"][r] + i
                self.cache[:, m["table"][r][pos // P], :, pos % P] = self.kv[:, a + j]
            num.append(len(path))
        assert d["num"].tolist() == num
        s.update(seq=[a + b for a, b in zip(s["seq"], num)], table=m["table"], held=m["held"], free=m["free"], count=m["count"])
        assert d["seq"].tolist() == s["seq"] and d["held"].tolist() == s["held"] and d["count"].tolist() == [s["count"]]
        assert torch.equal(d["cache"].cpu().view(torch.int16), self.cache.view(torch.int16))
        assert self.h.check_device_error(self.ws) == 0


def trees_of(step, rows, most):
    return [R.tree((step * 5 + r * 3) % (most + 1), 1 + (r + step) % 4, r) for r in range(rows)]


@pytest.mark.parametrize("captured", [False, True])
def test_steps_one_after_another(captured):
    """Five steps of rows with 0 to 12 drafted tokens; captured: one graph, replayed for every step."""
    loop = Loop([37, 0, 150, 16, 63], 8, 2, 64, 16, 2, 30, 11, 12)
    graph = None
    if captured:
        side = torch.cuda.Stream()
        saved = {k: v.clone() for k, v in loop.d.items()}
        loop.step()  # one call of each kind before the capture
        torch.cuda.synchronize()
        for k, v in saved.items():
            loop.d[k].copy_(v)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            loop.step()
    for i in range(5):
        loop.feed(trees_of(i, 5, 12), 100 + 7 * i)
        graph.replay() if graph else loop.step()
        torch.cuda.synchronize()
        loop.mirror()


def test_a_step_without_pages_does_nothing():
    """build_maps refuses: the calls behind it find an empty step."""
    loop = Loop([37, 20], 8, 2, 64, 16, 1, 30, 12, 12)
    loop.d["count"].fill_(0)
    loop.feed([R.tree(12, 2), R.tree(12, 3)], 5)
    before = loop.d["cache"].clone()
    loop.d["out"].fill_(7.0)
    loop.step()
    torch.cuda.synchronize()
    assert loop.d["seq"].tolist() == [37, 20], "the lengths stay"
    assert loop.d["status"].tolist() == [1] and loop.d["count"].tolist() == [0] and loop.d["held"].tolist() == [3, 2]
    assert torch.equal(loop.d["cache"], before) and (loop.d["out"] == 7).all() and loop.d["num"].tolist() == [0, 0]
    assert loop.h.check_device_error(loop.ws) == 0


def test_two_graphs_with_workspaces_of_their_own():
    """Two captured steps replayed at the same time."""
    loops = [Loop([37, 0, 1500], 8, 2, 64, 16, 2, 110, 13 + i, 12) for i in range(2)]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for loop, st in zip(loops, streams):
        saved = {k: v.clone() for k, v in loop.d.items()}
        loop.step()
        torch.cuda.synchronize()
        for k, v in saved.items():
            loop.d[k].copy_(v)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            loop.step()
        graphs.append(g)
    for i in range(3):
        for k, loop in enumerate(loops):
            loop.feed(trees_of(i + k, 3, 12), 50 + 9 * i + k)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for loop in loops:
            loop.mirror()
