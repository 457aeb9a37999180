"""Attention of trees of drafted tokens on the GPU against the definition in 64 bits.

Tolerances.  An output element is o = sum_j p_j v_j.  The kernel rounds each weight to bf16 (off by at
most half a step, 2^-8 of the value; their sum is taken unrounded) and the result to bf16 (2^-8 again):
|o - ref| <= 2^-8 (sum_j p_j |v_j| + |o|), plus the 32-bit arithmetic: a score of D products summed in
32 bits is off by at most D 2^-24 |q||k| scale, which shifts numerator and sum by that share each.  The
bound is computed per element in 64 bits and no element may exceed it (by the second-order terms' 1%).  lse: the
score's error, and 2^-20 of (1 + |lse|) for the sum and the logarithm.
"""
import numpy as np
import pytest
import torch

import tree_ref as R
from paged_kv_attention_gqa_gb300 import binding as B

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _build():
    from paged_kv_attention_gqa_gb300 import build
    build.build()


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


class Step:
    """A step of rows with ctx cached tokens and trees of drafted ones; every cache slot that no node may see holds NaN."""

    def __init__(self, ctx, trees, H, Hkv, D, P, seed, *, window=-1, scale=0.0, chain=False, sm_count=0, q_scale=1.0, tail=3,
                 max_new=None, rows_max=None):
        self.ctx, self.trees, self.window, self.chain, self.seed, self.tail = ctx, trees, window, chain, seed, tail
        news = [len(t) for t in trees]
        self.lens = [c + n for c, n in zip(ctx, news)]
        self.qo = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.T = int(self.qo[-1])
        self.kvp, self.kvi, self.last, pages = R.indices(self.lens, P, seed)
        self.scale = scale or R.default_scale(D)
        self.q = randn(seed + 1, self.T, H, D, scale=q_scale)
        self.k, self.v = randn(seed + 2, self.T, Hkv, D), randn(seed + 3, self.T, Hkv, D)
        cache = randn(seed + 4, pages, 2, P, Hkv, D)
        used = torch.zeros(pages, P, dtype=torch.bool)
        for r, c in enumerate(ctx):
            for i, p in enumerate(self.kvi[self.kvp[r]: self.kvp[r + 1]]):
                used[p, : max(0, min(P, c - i * P))] = True
        for x in (0, 1):
            cache[:, x][~used] = NAN
        self.cache = cache
        self.max_new = max_new or max(1, max(news, default=1))
        self.h = B.Handle(num_qo_heads=H, num_kv_heads=Hkv, head_dim=D, page_size=P, max_batch=max(1, len(ctx)),
                          max_total_tokens=self.T + tail, max_num_pages=max(1, len(self.kvi)), num_cache_pages=pages,
                          sm_count=sm_count)
        self.ws = torch.empty(self.h.workspace_size(B.MODE_TREE), dtype=torch.uint8, device="cuda")
        self.dev = dict(qo=i32(self.qo), kvp=i32(self.kvp), kvi=i32(self.kvi), last=i32(self.last))

    def parents(self):
        flat = [p for t in self.trees for p in t] + [-9] * self.tail  # what stands behind the last row is not read
        return None if self.chain else i32(flat)

    def plan(self, **kw):
        d = self.dev
        self.positions = torch.full((self.T + self.tail,), -5, dtype=torch.int32, device="cuda")
        args = dict(num_tokens=self.T + self.tail, max_new=self.max_new, workspace=self.ws, window_left=self.window,
                    sm_scale=self.scale, positions=self.positions)
        args.update(kw)
        self.h.plan_tree(d["qo"], d["kvp"], d["kvi"], d["last"], self.parents(), **args)

    def inputs(self):
        behind = lambda t: torch.cat([t, torch.full((self.tail, *t.shape[1:]), NAN, dtype=t.dtype)]).cuda()
        return behind(self.q), behind(self.k), behind(self.v), self.cache.cuda()

    def run(self, lse=True, given=None):
        q, k, v, kv = given or self.inputs()
        self.kv = kv
        T = self.T + self.tail
        self.out = torch.full((T, *self.q.shape[1:]), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, self.q.shape[1]), 7.0, device="cuda")
        self.h.run_tree(q, k, v, kv, self.out, self.lse if lse else None, workspace=self.ws)
        torch.cuda.synchronize()

    def reference(self):
        return R.attention(self.q, self.k, self.v, self.cache, self.qo, self.kvp, self.kvi, self.last, self.trees, self.scale,
                           self.window)

    def check(self, what="", lse=True):
        assert self.h.check_device_error(self.ws) == 0
        assert (self.out[self.T:] == 7).all() and (self.lse[self.T:] == 7).all(), f"{what}: behind the last row"
        assert torch.equal(self.kv.view(torch.int16).cpu(), self.cache.view(torch.int16)), f"{what}: the cache is only read"
        if self.T:
            compare(self.out[: self.T], self.lse[: self.T] if lse else None, self.reference(), what)
        if not lse:
            assert (self.lse == 7).all()


def compare(out, lse, ref, what):
    ro, rl, mag, err = ref
    o = out.double().cpu()
    assert torch.equal(torch.isnan(o), torch.isnan(ro)), f"{what}: NaN in other places"
    assert torch.equal(o[torch.isinf(ro)], ro[torch.isinf(ro)]), f"{what}: infinities"
    ok = torch.isfinite(ro)
    bound = 1.01 * 2.0 ** -8 * (mag + ro.abs()) + 2 * err[..., None] * mag + 1e-30
    worst = ((o - ro).abs()[ok] / bound[ok]).max().item() if ok.any() else 0.0
    assert worst <= 1, f"{what}: {worst:.2f} of the bound"
    if lse is None:
        return
    l, fine = lse.double().cpu(), torch.isfinite(rl)
    assert torch.equal(torch.isnan(l), torch.isnan(rl)) and torch.equal(l[torch.isinf(rl)], rl[torch.isinf(rl)]), f"{what}: lse"
    worst = ((l - rl).abs()[fine] / (err + 2.0 ** -20 * (1 + rl.abs()))[fine]).max().item() if fine.any() else 0.0
    assert worst <= 1, f"{what}: lse {worst:.2f} of the bound"


def step(*a, lse=True, **kw):
    s = Step(*a, **kw)
    s.plan()
    s.run(lse=lse)
    s.check(f"ctx {s.ctx}", lse=lse)
    for r, t in enumerate(s.trees):
        want = s.ctx[r] + R.ancestors(t)[1]
        assert torch.equal(s.positions[s.qo[r]: s.qo[r + 1]].cpu().long(), want), "positions"
    return s


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_numbers_of_drafted_tokens(D, n):
    step([70, 0, 1], [R.tree(n, 3), R.tree(max(1, n // 2), 4, 1), R.tree(n, 2, 2)], 4, 2, D, 16, n)


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 63, 64, 65, 127, 128, 129, 1000, 4096])
@pytest.mark.parametrize("P", [8, 16, 64, 256])
def test_lengths_and_pages(ctx, P):
    step([ctx, ctx // 2, ctx + 1], [R.tree(9, 3), R.tree(1, 1), R.tree(5, 2)], 8, 2, 128, P, ctx + P)


@pytest.mark.parametrize("P", [32, 128, 512, 1024])
def test_large_pages(P):
    step([3 * P + 5, P, 2 * P - 1], [R.tree(12, 3), R.tree(7, 2, 1), R.tree(3, 1)], 8, 8, 64, P, P)


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 6, 7, 8, 16])
@pytest.mark.parametrize("D,Hkv", [(64, 3), (128, 2), (256, 1)])
def test_groups(g, D, Hkv):
    step([300, 77], [R.tree(40, 4), R.tree(21, 5, 1)], g * Hkv, Hkv, D, 16, 10 * g + D)


@pytest.mark.parametrize("sm_count", [1, 2, 3, 7, 152, 300])
@pytest.mark.parametrize("D,H,n", [(64, 8, 6), (128, 16, 70), (256, 4, 9), (128, 8, 5)])
def test_cut_units(sm_count, D, H, n):
    """Units cut between few and many CTAs: whole, in two, in many pieces."""
    step([2500, 0, 700, 64, 5000], [R.tree(n, 3, r) for r in range(5)], H, 2, D, 16, sm_count + D, sm_count=sm_count)


@pytest.mark.parametrize("rows", [1, 2, 20])
@pytest.mark.parametrize("D,H,n", [(64, 3, 2), (64, 5, 3), (128, 8, 1), (128, 6, 2), (256, 4, 4), (256, 7, 2), (128, 8, 17)])
def test_long_rows_cut_into_many_pieces(D, H, n, rows):
    """One kv head, a row of 400 tiles and short ones: a unit of up to 150 pieces with 6 to 136 query rows, joined side by
    side in a warp, by several warps and in several rounds."""
    step([25600] + [70] * (rows - 1), [R.tree(n, 2, r) for r in range(rows)], H, 1, D, 64, 60 + D + H)


@pytest.mark.parametrize("window", [0, 1, 2, 5, 63, 64, 100, 1000])
@pytest.mark.parametrize("D,n", [(64, 30), (128, 90), (256, 20)])
def test_windows(window, D, n):
    step([400, 64, 3, 129], [R.tree(n, 3), R.tree(n, 1), R.tree(5, 2), R.tree(1, 1)], 4, 2, D, 16, window + D, window=window, sm_count=5)


def test_rows_without_drafted_tokens():
    """Rows in between that have no drafted token, or nothing at all, and a step without any."""
    step([50, 0, 33, 0, 200, 7], [R.tree(4, 2), [], [], R.tree(3, 1), R.tree(6, 3), []], 8, 2, 128, 16, 5)
    step([50, 0], [[], []], 8, 2, 128, 16, 6)
    s = Step([], [], 8, 2, 128, 16, 7)
    s.plan()
    s.run()
    s.check()


def test_chains_without_parents():
    a = step([300, 20, 0], [R.tree(9, 1), R.tree(1, 1), R.tree(33, 1)], 8, 2, 128, 16, 8, chain=True)
    b = step([300, 20, 0], [R.tree(9, 1), R.tree(1, 1), R.tree(33, 1)], 8, 2, 128, 16, 8)
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_several_roots():
    step([100, 0], [[-1, -1, 0, 1, -1, 4, 2], [-1, 0, -1, -1]], 8, 2, 64, 16, 9, window=3)


def test_without_lse_and_with_a_scale():
    step([100, 900], [R.tree(9, 3), R.tree(17, 3)], 8, 2, 128, 16, 11, lse=False, sm_count=4)
    step([100, 900], [R.tree(9, 3), R.tree(17, 3)], 8, 2, 128, 16, 12, scale=0.3)


def test_scores_far_apart():
    """Maxima that grow by more than the rescaling threshold from tile to tile."""
    s = Step([700, 300], [R.tree(20, 3), R.tree(8, 2)], 8, 2, 128, 16, 13, q_scale=6.0, sm_count=3)
    ramp = torch.linspace(0.1, 4, s.cache.shape[0] * 16).view(-1, 1, 16, 1, 1)
    s.cache = (s.cache.float() * ramp).to(torch.bfloat16)
    s.plan()
    s.run()
    s.check("ramp")


def test_long_row():
    step([40000], [R.tree(6, 2)], 4, 1, 64, 64, 14)


def test_thousands_of_rows():
    """More units than CTAs by far, rows without tokens among them, units of one query row."""
    step([r % 90 for r in range(2500)], [R.tree(r % 4, 2, r) for r in range(2500)], 2, 1, 64, 16, 51)


def test_a_larger_bound_of_drafted_tokens():
    """max_new says how many there may be at most, not how many there are."""
    for most in (9, 64, 65, 256):
        step([130, 20], [R.tree(9, 3), R.tree(4, 2)], 16, 2, 128, 16, 15, max_new=most)
        step([130, 20], [R.tree(9, 3), R.tree(4, 2)], 4, 2, 256, 16, 16, max_new=most)


def test_strided_inputs():
    """q, k and v as slices of one projection's output."""
    s = Step([130, 600], [R.tree(9, 3), R.tree(14, 4)], 8, 2, 64, 16, 17)
    s.plan()
    q, k, v, kv = s.inputs()
    qkv = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1), torch.full((len(q), 8), NAN, dtype=q.dtype, device="cuda")], 1)
    q2, k2, v2 = qkv[:, :512].view(-1, 8, 64), qkv[:, 512:640].view(-1, 2, 64), qkv[:, 640:768].view(-1, 2, 64)
    assert not q2.is_contiguous()
    s.run(given=(q2, k2, v2, kv))
    s.check("strided")


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("D,n", [(64, 7), (128, 70), (256, 66)])
def test_nodes_that_are_not_seen(value, D, n):
    """A node whose K, or V, or both are not finite reaches itself and those below it alone."""
    for where in ("k", "v", "kv"):
        s = Step([100, 65], [R.tree(n, 4), R.tree(5, 2)], 4, 2, D, 16, 18, sm_count=3)
        for x in where:
            t = getattr(s, x)
            t[n // 2, :, : D // 2 if x == "v" else D] = value
            t[n + 3] = value
        s.plan()
        s.run()
        seen = R.ancestors(s.trees[0])[0][:, n // 2]
        assert torch.isfinite(s.out[:n][~seen.cuda()]).all() and not torch.isfinite(s.out[n // 2]).all(), where
        s.check(where)


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_cached_tokens_that_are_not_seen(value, D):
    """Under a window, cached tokens that the deeper nodes no longer see."""
    s = Step([200, 90], [R.tree(12, 1), R.tree(9, 2)], 4, 2, D, 16, 19, window=20, sm_count=2)
    for r, c in enumerate(s.ctx):
        for at in (c - 19, c - 16, c - 30, 0):
            s.cache[int(s.kvi[s.kvp[r] + at // 16]), 1, at % 16] = value
    s.plan()
    s.run()
    s.check("window")


def test_scores_of_minus_infinity():
    """A query all of whose scores are -inf is 0 / 0; others are not touched by it."""
    s = Step([40], [[-1, 0, 0]], 2, 1, 64, 16, 20)
    s.q = torch.ones_like(s.q)
    s.cache[:, 0][~torch.isnan(s.cache[:, 0])] = -INF
    s.k[0], s.k[1] = -INF, 0.5
    s.k[2] = -INF
    s.plan()
    s.run()
    ro, rl, mag, err = s.reference()
    assert torch.isnan(s.out[0]).all() and torch.isnan(s.out[2]).all() and torch.isnan(ro[2]).all()
    assert (s.lse[0] == -INF).all() and (s.lse[2] == -INF).all()
    assert torch.allclose(s.out[1].double().cpu(), ro[1], atol=2e-2, rtol=1e-2)


def test_inconsistent_arrays_are_reported_and_skipped():
    def broken(change, parents=None):
        s = Step([100, 60, 30], [R.tree(5, 2), R.tree(4, 2), R.tree(6, 3)], 8, 2, 128, 16, 21)
        change(s)
        s.plan()
        s.run()
        return s

    def set_(name, at, value):
        def f(s):
            s.dev[name][at] = value
        return f

    for name, at, value in (("qo", 2, 99), ("qo", 2, -1), ("kvp", 2, 1000), ("kvp", 2, -7), ("last", 1, 0), ("last", 1, 17)):
        s = broken(set_(name, at, value))
        assert s.h.check_device_error(s.ws) == 5, (name, value)
        assert s.h.check_device_error(s.ws) == 0, "the word is cleared"
        compare(s.out[:5], s.lse[:5], tuple(y[:5] for y in s.reference()), "the first row is not touched by it")
        assert (s.out[5:9] == 7).all(), "the second row's result is left"
    s = broken(set_("kvi", 9, s.h.cfg.num_cache_pages))  # a page of row 1
    assert s.h.check_device_error(s.ws) == 6
    keep = torch.tensor([0, 1, 2, 3, 4, 9, 10, 11, 12, 13, 14])
    compare(s.out.cpu()[keep], s.lse.cpu()[keep], tuple(y[keep] for y in s.reference()), "rows with good pages")
    for value in (-2, 3, 4000):
        s = Step([100, 60], [R.tree(5, 2), R.tree(4, 2)], 8, 2, 128, 16, 22)
        good = s.trees
        s.trees = [good[0], [-1, 0, 1, value]]
        s.plan()
        assert s.h.check_device_error(s.ws) == 7
        s.trees = [good[0], [-1, 0, 1, -1]]  # taken as a root
        s.run()
        s.check("bad parent")


def test_rows_past_the_planned_sizes_are_reported():
    """More drafted tokens in a row than max_new, more in all than num_tokens: the rows count as empty."""
    s = Step([100, 60, 30], [R.tree(5, 2), R.tree(9, 2), R.tree(6, 3)], 8, 2, 128, 16, 40, max_new=8)
    s.plan()
    s.run()
    assert s.h.check_device_error(s.ws) == 5
    assert (s.out[5:14] == 7).all() and (s.lse[5:14] == 7).all()
    keep = torch.tensor([0, 1, 2, 3, 4, 14, 15, 16, 17, 18, 19])
    compare(s.out.cpu()[keep], s.lse.cpu()[keep], tuple(y[keep] for y in s.reference()), "the other rows")
    s = Step([100, 60], [R.tree(5, 2), R.tree(9, 2)], 8, 2, 128, 16, 41, tail=0)
    s.dev["qo"][2] = 15
    s.plan()
    s.run()
    assert s.h.check_device_error(s.ws) == 5 and (s.out[5:] == 7).all()


@pytest.mark.parametrize("D,H,Hkv", [(64, 16, 2), (128, 8, 2), (256, 4, 4)])
def test_plans_in_turn_on_one_workspace(D, H, Hkv):
    """Long and short steps, wide and narrow ones, under a window and not, on one handle; each layer is run twice."""
    steps = [Step([3000, 5], [R.tree(40, 3), R.tree(3, 1)], H, Hkv, D, 16, 50), Step([20], [R.tree(2, 1)], H, Hkv, D, 16, 51),
             Step([700, 64, 0, 900], [R.tree(100, 4), R.tree(64, 2), [], R.tree(9, 3)], H, Hkv, D, 16, 52, window=33),
             Step([], [], H, Hkv, D, 16, 53), Step([1, 2, 3], [R.tree(1, 1)] * 3, H, Hkv, D, 16, 54)]
    pages = max(s.cache.shape[0] for s in steps)
    h = B.Handle(num_qo_heads=H, num_kv_heads=Hkv, head_dim=D, page_size=16, max_batch=4, max_total_tokens=200, max_num_pages=pages,
                 num_cache_pages=pages)
    ws = torch.empty(h.workspace_size(B.MODE_TREE), dtype=torch.uint8, device="cuda")
    for s in steps + steps[::-1]:
        more = torch.full((pages - s.cache.shape[0], *s.cache.shape[1:]), NAN, dtype=s.cache.dtype)
        s.cache, s.h, s.ws = torch.cat([s.cache, more]), h, ws
        s.plan()
        s.run()
        s.check(f"{s.ctx}")
        s.run()
        s.check(f"{s.ctx} again")


def test_streams_and_workspaces():
    """Two steps with workspaces of their own on two streams, neither the default one."""
    steps = [Step([900, 40], [R.tree(9, 3), R.tree(20, 4)], 8, 2, 128, 16, 23 + i) for i in range(2)]
    given = [s.inputs() for s in steps]
    parents = [s.parents() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for s, (q, k, v, kv), par, st in zip(steps, given, parents, streams):
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        outs.append((out, lse, kv))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (q, k, v, kv), par, st, (out, lse, _) in zip(steps, given, parents, streams, outs):
            d = s.dev
            s.h.plan_tree(d["qo"], d["kvp"], d["kvi"], d["last"], par, num_tokens=len(q), max_new=s.max_new, workspace=s.ws,
                          stream=st)
            s.h.run_tree(q, k, v, kv, out, lse, workspace=s.ws, stream=st)
    torch.cuda.synchronize()
    for s, (out, lse, kv) in zip(steps, outs):
        s.out, s.lse, s.kv = out, lse, kv
        s.check("two streams")


def test_the_same_call_gives_the_same_bits():
    s = step([3000, 700], [R.tree(40, 4), R.tree(9, 2)], 16, 2, 128, 16, 30)
    first = s.out.clone(), s.lse.clone()
    for _ in range(3):
        s.run()
        assert torch.equal(first[0], s.out) and torch.equal(first[1], s.lse)


def test_refused_strides_and_alignment():
    s = Step([30], [R.tree(4, 2)], 8, 2, 64, 16, 31)
    s.plan()
    q, k, v, kv = s.inputs()
    out, T = torch.empty_like(q), len(q)
    wide = torch.zeros(T, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")  # rows 4 elements too long: not a multiple of 8
    odd = torch.zeros(T * 128 + 8, dtype=torch.bfloat16, device="cuda")[4:4 + T * 128].view(T, 2, 64)
    over = torch.zeros(128, dtype=torch.bfloat16, device="cuda").as_strided((T, 2, 64), (0, 64, 1))
    for bad in (wide[:, :128].view(T, 2, 64), odd, over):
        with pytest.raises(B.PkvError) as e:
            s.h.run_tree(q, bad, v, kv, out, workspace=s.ws)
        assert e.value.status == B.ERR_INVALID
        with pytest.raises(B.PkvError):
            s.h.run_tree(q, k, bad, kv, out, workspace=s.ws)
    with pytest.raises(B.PkvError) as e:
        s.h.run_decode(q, kv, out, workspace=s.ws)
    assert e.value.status == B.ERR_NOT_PLANNED
    other = torch.empty_like(s.ws)
    with pytest.raises(B.PkvError) as e:
        s.h.run_tree(q, k, v, kv, out, workspace=other)
    assert e.value.status == B.ERR_NOT_PLANNED
    s.run()
    s.check("after the refusals")
