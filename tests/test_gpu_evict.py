"""Accumulated attention weights and the eviction by them on the GPU, against their definitions in 64
bits (weights: per-slot error bounds from the scores' 32-bit arithmetic; selection and moves: exact)."""
import math

import numpy as np
import pytest
import torch

import evict_ref as E
from paged_kv_attention_gqa_gb300 import binding as B
from test_gpu_latent import bits, randn, table

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def _build():
    from paged_kv_attention_gqa_gb300 import build
    build.build()


class Step:
    def __init__(self, lens, news, Hq, Hkv, D, P, seed, *, mode, causal=True, window_left=-1, q_scale=1.5, sm_count=0):
        self.mode, self.D = mode, D
        self.qo = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.kvp, self.kvi, self.lpl, pages = table(lens, P, seed)
        T = int(self.qo[-1])
        self.kw = dict(causal=causal, window_left=window_left)
        self.scale = 1 / math.sqrt(D)
        self.q = randn(seed + 1, T, Hq, D, scale=q_scale)
        self.cache = randn(seed + 2, pages, 2, P, Hkv, D)
        used = torch.zeros(pages, P, dtype=torch.bool)
        for r, L in enumerate(lens):
            for i, p in enumerate(self.kvi[self.kvp[r]: self.kvp[r + 1]]):
                used[p, : max(0, min(P, L - i * P))] = True
        self.cache.transpose(1, 2)[~used] = float("nan")
        self.scores = torch.rand(pages, P, generator=torch.Generator().manual_seed(seed))
        self.used = used
        self.h = B.Handle(num_qo_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=P, max_batch=max(1, len(lens)),
                          max_total_tokens=max(T, 1), max_num_pages=max(1, len(self.kvi)), num_cache_pages=pages,
                          sm_count=sm_count)
        self.ws = torch.empty(self.h.workspace_size(mode), dtype=torch.uint8, device="cuda")
        self.plan()

    def idx(self):
        return self.qo, self.kvp, self.kvi, self.lpl

    def plan(self):
        self.h.plan(self.mode, None if self.mode == B.MODE_DECODE_WEIGHTS else self.qo, self.kvp, self.kvi, self.lpl,
                    workspace=self.ws, **self.kw)

    def check_scores(self, got, lse, decay, what):
        want, bound = E.add_weights(self.scores, self.q, lse, self.cache, *self.idx(), self.scale, decay, **self.kw)
        got = got.double().cpu()
        assert torch.equal(got[~self.used], self.scores.double()[~self.used]), f"{what}: slots without a token"
        off = ((got - want).abs() - bound)[self.used]
        assert torch.isfinite(got[self.used]).all() and (off.numel() == 0 or off.max() <= 0), f"{what}: {off.max()}"


DECODE = {
    "one token": dict(lens=[1], Hq=1, Hkv=1, D=64, P=16),
    "one row": dict(lens=[1001], Hq=32, Hkv=8, D=128, P=16),
    "page edges": dict(lens=[15, 16, 17, 127, 128, 129, 2], Hq=8, Hkv=2, D=128, P=16),
    "pages of 1": dict(lens=[33, 5, 70], Hq=4, Hkv=2, D=64, P=1),
    "pages of 2": dict(lens=[33, 130, 1], Hq=10, Hkv=2, D=64, P=2),
    "pages of 8": dict(lens=[200, 31], Hq=16, Hkv=1, D=128, P=8),
    "pages of 64, 256 wide": dict(lens=[300, 64, 65], Hq=7, Hkv=1, D=256, P=64),
    "window": dict(lens=[500, 40, 129], Hq=8, Hkv=4, D=128, P=16, window_left=100),
    "window, pages of 4": dict(lens=[200, 9], Hq=6, Hkv=2, D=64, P=4, window_left=37),
    "many pieces": dict(lens=[4000, 17, 3000], Hq=12, Hkv=4, D=128, P=32),
}


@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
@pytest.mark.parametrize("name", DECODE)
def test_decode_weights(name, decay):
    c = DECODE[name]
    s = Step(news=[1] * len(c["lens"]), seed=3 + len(name), mode=B.MODE_DECODE_WEIGHTS, **c)
    if decay == 0.0:
        s.scores[s.used] = float("nan")  # an old score is not read
    q, cache, scores = s.q.cuda(), s.cache.cuda(), s.scores.cuda()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    s.h.run_decode_weights(q, cache, out, lse, scores, decay=decay, workspace=s.ws)
    torch.cuda.synchronize()
    assert s.h.check_device_error(s.ws) == 0
    o, l, mag, err = E.attention(s.q, s.cache, *s.idx(), s.scale, **s.kw)
    bound = 1.01 * 2.0 ** -8 * (mag + o.abs()) + 2 * err[..., None] * mag
    assert ((out.double().cpu() - o).abs() <= bound).all()
    assert ((lse.double().cpu() - l).abs() <= err + 2.0 ** -20 * (1 + l.abs())).all()
    s.check_scores(scores, l, decay, name)
    # the same attention as an ordinary decode, bit for bit
    h2 = B.Handle(num_qo_heads=c["Hq"], num_kv_heads=c["Hkv"], head_dim=c["D"], page_size=c["P"], max_batch=len(c["lens"]),
                  max_num_pages=len(s.kvi), num_cache_pages=len(s.cache))
    ws = torch.empty(h2.workspace_size(B.MODE_DECODE), dtype=torch.uint8, device="cuda")
    h2.plan(B.MODE_DECODE, None, s.kvp, s.kvi, s.lpl, workspace=ws, **s.kw)
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    h2.run_decode(q, cache, out2, lse2, workspace=ws)
    assert torch.equal(bits(out), bits(out2)) and torch.equal(lse, lse2)


WEIGHTS = {
    "one token": dict(lens=[1], news=[1], Hq=1, Hkv=1, D=64, P=8),
    "decode-like": dict(lens=[300, 17, 129], news=[1, 1, 1], Hq=32, Hkv=8, D=128, P=16),
    "last tokens": dict(lens=[500, 40, 128], news=[32, 40, 7], Hq=8, Hkv=2, D=128, P=16),
    "whole prompts": dict(lens=[300, 129], news=[300, 129], Hq=8, Hkv=2, D=64, P=32),
    "groups of 5": dict(lens=[200, 60], news=[60, 3], Hq=10, Hkv=2, D=128, P=64),
    "groups of 16": dict(lens=[150], news=[20], Hq=16, Hkv=1, D=256, P=16),
    "groups of 7, large pages": dict(lens=[700, 5], news=[100, 5], Hq=7, Hkv=1, D=64, P=512),
    "rows without queries": dict(lens=[70, 0, 33], news=[0, 0, 5], Hq=4, Hkv=4, D=128, P=8),
    "window": dict(lens=[400, 90], news=[200, 3], Hq=4, Hkv=2, D=128, P=16, window_left=77),
    "not causal": dict(lens=[140, 66], news=[40, 2], Hq=4, Hkv=2, D=128, P=16, causal=False),
    "one SM": dict(lens=[300, 140], news=[140, 9], Hq=8, Hkv=4, D=128, P=16, sm_count=1),
}


@pytest.mark.parametrize("decay", [1.0, 0.25, 0.0])
@pytest.mark.parametrize("name", WEIGHTS)
def test_weights(name, decay):
    s = Step(seed=5 + len(name), mode=B.MODE_WEIGHTS, **WEIGHTS[name])
    _, l, _, _ = E.attention(s.q, s.cache, *s.idx(), s.scale, **s.kw)
    lse = l.float()
    if decay == 0.0:
        s.scores[s.used] = float("nan")
    scores = s.scores.cuda()
    s.h.run_weights(s.q.cuda(), lse.cuda(), s.cache.cuda(), scores, decay=decay, workspace=s.ws)
    torch.cuda.synchronize()
    assert s.h.check_device_error(s.ws) == 0
    s.check_scores(scores, lse, decay, name)


WEIGHTS_BLOCKS = {
    "one head, many blocks": dict(lens=[900], news=[900], Hq=1, Hkv=1, D=128, P=16),
    "one head, one block": dict(lens=[3000, 77], news=[5, 2], Hq=4, Hkv=1, D=128, P=32),
    "two SMs, heads of several tiles": dict(lens=[600, 333], news=[90, 333], Hq=12, Hkv=3, D=64, P=8, sm_count=2),
    "a window inside a block": dict(lens=[500], news=[300], Hq=5, Hkv=1, D=128, P=16, window_left=5),
    "window 0": dict(lens=[260, 3], news=[130, 3], Hq=4, Hkv=2, D=128, P=16, window_left=0),
    "the longest window": dict(lens=[260, 3], news=[130, 3], Hq=4, Hkv=2, D=128, P=16, window_left=2 ** 31 - 1),
    "not causal, a window": dict(lens=[300], news=[140], Hq=6, Hkv=2, D=128, P=16, causal=False, window_left=40),
    "columns that are no multiple of 32": dict(lens=[400], news=[43], Hq=6, Hkv=2, D=128, P=16),
}


@pytest.mark.parametrize("name", WEIGHTS_BLOCKS)
def test_weights_blocks(name):
    """Blocks and masks as the teams meet them: items without a block for some team, partial blocks, masks
    that cut through a block from either side."""
    s = Step(seed=61 + len(name), mode=B.MODE_WEIGHTS, **WEIGHTS_BLOCKS[name])
    _, l, _, _ = E.attention(s.q, s.cache, *s.idx(), s.scale, **s.kw)
    scores = s.scores.cuda()
    s.h.run_weights(s.q.cuda(), l.float().cuda(), s.cache.cuda(), scores, decay=0.5, workspace=s.ws)
    torch.cuda.synchronize()
    assert s.h.check_device_error(s.ws) == 0
    s.check_scores(scores, l.float(), 0.5, name)


def test_weights_without_any_query_decay_the_scores():
    s = Step([70, 33], [0, 0], 8, 2, 64, 16, 5, mode=B.MODE_WEIGHTS)
    scores = s.scores.cuda()
    s.h.run_weights(s.q.cuda(), torch.empty(0, 8, device="cuda"), s.cache.cuda(), scores, decay=0.25, workspace=s.ws)
    want = torch.where(s.used, s.scores * 0.25, s.scores)
    assert torch.equal(scores.cpu(), want)


def test_weights_sum_to_the_queries():
    """Without a window every query's weights sum to 1 per head."""
    s = Step([333, 64], [50, 64], 8, 2, 128, 16, 9, mode=B.MODE_WEIGHTS)
    _, l, _, _ = E.attention(s.q, s.cache, *s.idx(), s.scale)
    scores = torch.zeros_like(s.scores).cuda()
    s.h.run_weights(s.q.cuda(), l.float().cuda(), s.cache.cuda(), scores, decay=0.0, workspace=s.ws)
    assert abs(scores.double().sum().item() / (114 * 8) - 1) < 1e-5


def test_weights_of_another_sequence_do_not_leak():
    """Queries of the next row hold NaN: the first row's scores are the same bits."""
    s = Step([100, 100], [3, 3], 8, 2, 128, 16, 9, mode=B.MODE_WEIGHTS)
    _, l, _, _ = E.attention(s.q, s.cache, *s.idx(), s.scale)
    lse, cache = l.float().cuda(), s.cache.cuda()
    a, b = s.scores.cuda(), s.scores.cuda()
    s.h.run_weights(s.q.cuda(), lse, cache, a, workspace=s.ws)
    s.q[3:] = float("nan")
    s.h.run_weights(s.q.cuda(), lse, cache, b, workspace=s.ws)
    mine = torch.as_tensor(s.kvi[s.kvp[0]: s.kvp[1]]).long()
    assert torch.equal(a[mine], b[mine]) and torch.isfinite(a[mine]).all()


def test_graphs_of_two_handles_on_two_streams():
    """A decode step and a prompt's weights, each captured with its own handle and workspace, replayed at
    the same time on streams other than the capturing one: the bits of the eager calls."""
    d = Step([700, 40, 129], [1, 1, 1], 8, 2, 128, 16, 21, mode=B.MODE_DECODE_WEIGHTS)
    w = Step([400, 129], [90, 129], 8, 2, 128, 16, 22, mode=B.MODE_WEIGHTS)
    _, l, _, _ = E.attention(w.q, w.cache, *w.idx(), w.scale)
    wl, wq, wc = l.float().cuda(), w.q.cuda(), w.cache.cuda()
    dq, dc = d.q.cuda(), d.cache.cuda()
    out, dl = torch.empty_like(dq), torch.empty(3, 8, device="cuda")
    ds, wsc = d.scores.cuda(), w.scores.cuda()
    dec = lambda t: d.h.run_decode_weights(dq, dc, out, dl, t, decay=0.5, workspace=d.ws)
    wei = lambda t: w.h.run_weights(wq, wl, wc, t, decay=0.5, workspace=w.ws)
    want_d, want_w = d.scores.cuda(), w.scores.cuda()
    for _ in range(3):
        dec(want_d), wei(want_w)
    want_o, want_l = out.clone(), dl.clone()
    graphs = []
    for f, t in ((dec, ds), (wei, wsc)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f(t)
        graphs.append(g)
    out.zero_(), dl.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert d.h.check_device_error(d.ws) == 0 and w.h.check_device_error(w.ws) == 0
    assert torch.equal(bits(out), bits(want_o)) and torch.equal(dl, want_l)
    for got, want, s in ((ds, want_d, d), (wsc, want_w, w)):
        assert torch.equal(got[s.used.cuda()], want[s.used.cuda()])


# ---------------------------------------------------------------- eviction

class Cut:
    def __init__(self, lens, keep, sink, recent, Hkv, D, P, seed, scores="rand", share=False):
        g = np.random.default_rng(seed)
        self.lens, self.keep, self.sink, self.recent, self.P = lens, keep, sink, recent, P
        self.kvp, self.kvi, self.lpl, base = table(lens, P, seed, spare=0)
        if share and len(lens) > 1:  # the second row's first page is the first row's
            self.kvi = self.kvi.copy()
            self.kvi[self.kvp[1]] = self.kvi[0]
        need = [-(-k // P) if k < L else 0 for k, L in zip(keep, lens)]
        self.dst_indptr = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
        self.pages = base + sum(need) + 2
        self.dst = (base + g.permutation(sum(need) + 2)[: sum(need)]).astype(np.int32)
        self.kv = randn(seed, self.pages, 2, P, Hkv, D)
        gen = torch.Generator().manual_seed(seed)
        if scores == "rand":
            self.scores = torch.rand(self.pages, P, generator=gen) * 3 - 1
        elif scores == "ties":
            self.scores = torch.randint(0, 3, (self.pages, P), generator=gen).float() - 1
            self.scores[self.scores == 0] = torch.where(torch.rand(int((self.scores == 0).sum()), generator=gen) < 0.5, 0.0, -0.0)
        elif scores == "equal":
            self.scores = torch.full((self.pages, P), 0.25)
        else:
            self.scores = torch.rand(self.pages, P, generator=gen)
            pick = torch.rand(self.pages, P, generator=gen)
            self.scores[pick < 0.2] = float("nan")
            self.scores[(pick > 0.2) & (pick < 0.4)] = float("inf")
            self.scores[(pick > 0.4) & (pick < 0.6)] = float("-inf")
            self.scores[(pick > 0.6) & (pick < 0.7)] = 1e-42  # a denormal
        self.h = B.Handle(num_qo_heads=Hkv, num_kv_heads=Hkv, head_dim=D, page_size=P, max_batch=max(1, len(lens)),
                          max_num_pages=max(1, len(self.kvi), len(self.dst)), num_cache_pages=self.pages)
        self.ws = torch.empty(self.h.workspace_size(B.MODE_EVICT), dtype=torch.uint8, device="cuda")
        self.plan()

    def plan(self):
        self.h.plan_evict(self.kvp, self.kvi, self.lpl, self.keep, self.dst_indptr, self.dst, num_sink=self.sink,
                          num_recent=self.recent, workspace=self.ws)

    def want(self):
        kv, scores, kept = self.kv.clone(), self.scores.clone(), []
        for r, L in enumerate(self.lens):
            ids = torch.as_tensor(self.kvi[self.kvp[r]: self.kvp[r + 1]]).long()
            mine = E.select(self.scores[ids].reshape(-1)[:L].tolist(), L, self.keep[r], self.sink, self.recent)
            kept += mine
            if L > self.keep[r] and mine:
                j, i = torch.tensor(mine), torch.arange(len(mine))
                to = torch.as_tensor(self.dst[self.dst_indptr[r]: self.dst_indptr[r + 1]]).long()[i // self.P]
                kv[to, :, i % self.P] = self.kv[ids[j // self.P], :, j % self.P]
                scores[to, i % self.P] = self.scores[ids[j // self.P], j % self.P]
        return kv, scores, torch.tensor(kept, dtype=torch.int32)

    def run(self):
        kv, scores = self.kv.cuda(), self.scores.cuda()
        kept = torch.full((sum(min(k, L) for k, L in zip(self.keep, self.lens)),), -7, dtype=torch.int32, device="cuda")
        self.h.run_evict(kv, scores, kept, workspace=self.ws)
        torch.cuda.synchronize()
        return kv.cpu(), scores.cpu(), kept.cpu()

    def check(self, what):
        kv, scores, kept = self.run()
        want_kv, want_scores, want_kept = self.want()
        assert torch.equal(kept, want_kept), what
        assert torch.equal(scores.view(torch.int32), want_scores.view(torch.int32)), what
        assert torch.equal(bits(kv), bits(want_kv)), what


CUTS = {
    "one token stays": dict(lens=[2], keep=[1], sink=0, recent=0, Hkv=1, D=64, P=8),
    "one row": dict(lens=[2111], keep=[1024], sink=4, recent=64, Hkv=2, D=64, P=16),
    "nothing to choose": dict(lens=[50, 9], keep=[12, 12], sink=4, recent=8, Hkv=1, D=64, P=8),
    "nothing stays": dict(lens=[50, 0, 9], keep=[0, 0, 9], sink=0, recent=0, Hkv=1, D=64, P=8),
    "rows left alone": dict(lens=[40, 300, 0, 64], keep=[40, 128, 5, 65], sink=1, recent=3, Hkv=2, D=128, P=16),
    "pages of 1": dict(lens=[70, 33], keep=[20, 32], sink=2, recent=5, Hkv=1, D=64, P=1),
    "all but one": dict(lens=[513, 4097], keep=[512, 4096], sink=0, recent=0, Hkv=1, D=64, P=64),
    "edges of the cluster": dict(lens=[2048, 2049, 4096, 4097, 8193], keep=[1000, 7, 4095, 2049, 4000], sink=3, recent=2,
                                 Hkv=1, D=64, P=32),
    "long row": dict(lens=[50000], keep=[777], sink=4, recent=100, Hkv=1, D=64, P=256),
    "256 wide": dict(lens=[100, 200], keep=[33, 34], sink=0, recent=1, Hkv=5, D=256, P=2),
}


@pytest.mark.parametrize("scores", ["rand", "ties", "equal", "special"])
@pytest.mark.parametrize("name", CUTS)
def test_evict(name, scores):
    c = Cut(seed=len(name), scores=scores, **CUTS[name])
    c.check(name)


def test_evict_beyond_shared_memory():
    """A row whose slices do not fit the CTAs' shared memory (8 x 40K scores)."""
    c = Cut([400_000], [1000], 2, 3, 1, 64, 256, 5, scores="rand")
    c.check("400,000 tokens")


def test_evict_rows_share_pages_and_repeat():
    c = Cut([100, 90], [30, 20], 2, 4, 2, 64, 16, 3, share=True)
    c.check("shared")
    a, b = c.run(), c.run()
    assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))


def test_evict_graph_replay():
    c = Cut([700, 300], [100, 64], 2, 4, 2, 64, 16, 3)
    c.check("before the capture")
    kv, scores = c.kv.cuda(), c.scores.cuda()
    kept = torch.zeros(164, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.h.run_evict(kv, scores, kept, workspace=c.ws)
    c.scores = c.scores.flip(0).contiguous()
    scores.copy_(c.scores)
    g.replay()
    torch.cuda.synchronize()
    _, want_scores, want_kept = c.want()
    assert torch.equal(kept.cpu(), want_kept) and torch.equal(scores.cpu(), want_scores)


def test_decode_evict_decode():
    """A run of them as they are used: decode steps add up weights, the cache is cut down, and the next
    decode over the new pages equals attention over the kept tokens."""
    Hq, Hkv, D, P, L, keep = 8, 2, 64, 16, 200, 96
    s = Step([L], [1], Hq, Hkv, D, P, 77, mode=B.MODE_DECODE_WEIGHTS)
    n_dst = -(-keep // P)
    pool = torch.cat([s.cache, torch.zeros(n_dst + 1, 2, P, Hkv, D, dtype=torch.bfloat16)]).cuda()
    pages = pool.shape[0]
    dst = np.arange(pages - n_dst - 1, pages - 1, dtype=np.int32)
    h = B.Handle(num_qo_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=P, max_batch=1, max_total_tokens=1,
                 max_num_pages=pages, num_cache_pages=pages)
    ws = torch.empty(max(h.workspace_size(m) for m in (B.MODE_DECODE_WEIGHTS, B.MODE_EVICT)), dtype=torch.uint8, device="cuda")
    scores = torch.zeros(pages, P, device="cuda")
    q, out, lse = s.q.cuda(), torch.empty_like(s.q.cuda()), torch.empty(1, Hq, device="cuda")
    h.plan(B.MODE_DECODE_WEIGHTS, None, s.kvp, s.kvi, s.lpl, workspace=ws)
    for _ in range(3):
        h.run_decode_weights(q, pool, out, lse, scores, decay=1.0, workspace=ws)
    # three steps of weights that sum to 1 per head; the newest token's starts anew every time
    assert abs(scores.double().sum().item() - 3 * Hq + 2 * scores.view(-1)[int(s.kvi[-1]) * P + int(s.lpl[0]) - 1].item()) < 1e-3
    h.plan_evict(s.kvp, s.kvi, s.lpl, [keep], [0, n_dst], dst, num_sink=2, num_recent=20, workspace=ws)
    kept = torch.empty(keep, dtype=torch.int32, device="cuda")
    h.run_evict(pool, scores, kept, workspace=ws)
    h.plan(B.MODE_DECODE_WEIGHTS, None, [0, n_dst], dst, [(keep - 1) % P + 1], workspace=ws)
    h.run_decode_weights(q, pool, out, lse, scores, decay=1.0, workspace=ws)
    pos = kept.cpu().long()
    assert pos[:2].tolist() == [0, 1] and pos[-20:].tolist() == list(range(L - 20, L)) and (pos.diff() > 0).all()
    k = E.rows_of(s.cache, s.kvp, s.kvi, 0, L, 0)[pos].repeat_interleave(Hq // Hkv, 1)
    v = E.rows_of(s.cache, s.kvp, s.kvi, 0, L, 1)[pos].repeat_interleave(Hq // Hkv, 1)
    o, l, mag, = E.attend(s.q, k, v, torch.ones(1, keep, dtype=torch.bool), 1 / math.sqrt(D))
    assert ((out.double().cpu() - o).abs() <= 2.0 ** -7 * (mag + o.abs())).all()
    assert ((lse.double().cpu() - l).abs() <= 1e-4).all()


def test_refusals_of_the_run_calls():
    s = Step([64], [1], 8, 2, 64, 16, 3, mode=B.MODE_DECODE_WEIGHTS)
    q, cache, scores = s.q.cuda(), s.cache.cuda(), s.scores.cuda()
    out, lse = torch.empty_like(q), torch.empty(1, 8, device="cuda")
    with pytest.raises(B.PkvError) as e:  # a plan of the other kind
        s.h.run_decode(q, cache, out, lse, workspace=s.ws)
    assert e.value.status == B.ERR_NOT_PLANNED
    for decay in (-1.0, float("nan"), float("inf")):
        with pytest.raises(B.PkvError) as e:
            s.h.run_decode_weights(q, cache, out, lse, scores, decay=decay, workspace=s.ws)
        assert e.value.status == B.ERR_INVALID
    for bad in (dict(scores=scores.half()), dict(scores=scores[:-1]), dict(kv_layer=cache.float()), dict(lse=lse[:, :4])):
        args = dict(q=q, kv_layer=cache, out=out, lse=lse, scores=scores)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            s.h.run_decode_weights(**args, workspace=s.ws)
