"""Latent attention where keys that a query does not see hold NaN or infinities (later tokens of the
same step, tokens before the window): its result is as if they were not there, and the queries that see
them get what the definition gives.  Against the definition in 64 bits over each query's own keys; finite
results within the bounds of the latent tests (a weight and the result are rounded to bf16, 2^-8 each)."""
import math

import numpy as np
import pytest
import torch

import latent_ref as R
from paged_kv_attention_gqa_gb300 import binding as B

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

SCALE = 1 / math.sqrt(R.NOPE + R.ROPE)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _build():
    from paged_kv_attention_gqa_gb300 import build
    build.build()


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def by_query(q, k, v, n, L, causal, window_left):
    """out, lse, sum p|v| and the score error of each of n queries [n, H, W] over the keys it sees alone;
    k [L, H or 1, W], v [L, H or 1, D].  Infinite and NaN values follow the products of IEEE arithmetic."""
    H, parts = q.shape[1], []
    see = R.visible(L, n, causal, window_left)
    q, k, v = q.double(), k.double().expand(-1, H, -1), v.double().expand(-1, H, -1)
    for i in range(n):
        at = see[i].nonzero()[:, 0]
        x = torch.einsum("hw,lhw->hl", q[i], k[at]) * SCALE
        p = torch.softmax(x, -1)
        clean = v[at].nan_to_num(0, 0, 0)
        # one by one where a value is not finite: an einsum may sum in any order, and 0 * inf is NaN in each
        o = (p.transpose(0, 1)[..., None] * v[at]).sum(0)
        finite = k[at].nan_to_num(0, 0, 0)
        err = q.shape[-1] * 2.0 ** -24 * q[i].norm(dim=-1) * finite.norm(dim=-1).max() * SCALE
        parts.append((o, torch.logsumexp(x, -1), torch.einsum("hl,lhd->hd", p, clean.abs()), err))
    return tuple(torch.stack(y) for y in zip(*parts))


def check(out, lse, ref, what):
    o, l, (ro, rl, mag, err) = out.double().cpu(), lse.double().cpu(), ref
    ok = torch.isfinite(ro)
    assert torch.equal(torch.isnan(o), torch.isnan(ro)), f"{what}: NaN in other places"
    assert torch.equal(o[torch.isinf(ro)], ro[torch.isinf(ro)]), f"{what}: infinities"
    bound = 1.01 * 2.0 ** -8 * (mag + ro.abs()) + 2 * err[..., None] * mag + 1e-30
    assert ((o - ro).abs()[ok] <= bound[ok]).all(), f"{what}: {((o - ro).abs()[ok] / bound[ok]).max():.2f} of the bound"
    good = torch.isfinite(rl)
    assert torch.equal(torch.isfinite(l), good), f"{what}: lse"
    assert ((l - rl).abs()[good] <= (err + 2.0 ** -20 * (1 + rl.abs()))[good]).all(), f"{what}: lse"


# bad: positions (from the row's end) of the tokens that hold a value, which, and in how many columns
ABSORBED = {
    "the last of three tokens": dict(lens=[200], news=[3], H=16, P=64, bad={1: NAN}),
    "small pages": dict(lens=[200, 67], news=[3, 4], H=16, P=16, bad={1: NAN, 2: INF}),
    "the middle one": dict(lens=[130], news=[5], H=8, P=64, bad={3: INF}),
    "a few columns": dict(lens=[300], news=[4], H=16, P=64, bad={2: -INF}, columns=[0, 7, 64, 500, 511]),
    "one head, a prompt": dict(lens=[150], news=[150], H=1, P=16, bad={30: NAN, 31: INF, 100: -INF}, columns=[3, 200]),
    "a prompt of 16 heads": dict(lens=[90], news=[70], H=16, P=64, bad={5: NAN, 40: NAN}),
    "128 heads": dict(lens=[100, 300], news=[2, 3], H=128, P=16, bad={1: NAN}),
    "before the window, one token": dict(lens=[500, 90], news=[1, 1], H=16, P=64, window_left=70, bad={72: NAN, 73: INF, 89: NAN}),
    "before the window, small pages": dict(lens=[500, 90], news=[1, 1], H=128, P=8, window_left=33, bad={35: INF, 36: NAN}),
    "at the window's edge, three tokens": dict(lens=[500], news=[3], H=16, P=16, window_left=70, bad={72: NAN, 71: INF}),
    "a window shorter than the step": dict(lens=[200], news=[40], H=2, P=64, window_left=5, bad={10: NAN, 33: INF}, columns=[1, 90]),
    "not causal, a window": dict(lens=[200], news=[3], H=16, P=64, window_left=20, causal=False, bad={22: NAN, 21: NAN, 80: INF}),
    "many pieces": dict(lens=[4000], news=[3], H=16, P=64, bad={1: NAN, 2: INF}, columns=[17]),
    "one CTA": dict(lens=[200, 130, 64], news=[3, 2, 2], H=20, P=64, sm_count=1, bad={1: INF}),
    "two CTAs, both ends": dict(lens=[700, 260], news=[6, 70], H=16, P=32, sm_count=2, window_left=100, bad={1: NAN, 104: INF, 60: NAN},
                                columns=[2, 300]),
    # scores of -inf: rows that see nothing else, and pieces of a row that hold nothing else
    "an infinite key alone": dict(lens=[1, 70], news=[1, 1], H=64, P=16, window_left=0, bad={1: INF}, columns=[9]),
    "an infinite key alone in its piece": dict(lens=[65, 129], news=[1, 3], H=16, P=16, bad={1: INF}, columns=[9]),
}


@pytest.mark.parametrize("name", ABSORBED)
def test_absorbed(name):
    c = dict(causal=True, window_left=-1, columns=None, sm_count=0)
    c.update(ABSORBED[name])
    lens, news, H, P = c["lens"], c["news"], c["H"], c["P"]
    g = np.random.default_rng(3)
    pages = [-(-L // P) for L in lens]
    order = g.permutation(sum(pages) + 2).astype(np.int32)
    kvp = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    qo = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    T = int(qo[-1])
    q = randn(1, T, H, 576)
    flat = [randn(10 + r, L, 576) for r, L in enumerate(lens)]
    cache = torch.full((len(order), P, 576), NAN, dtype=torch.bfloat16)
    for r, L in enumerate(lens):
        for back, value in c["bad"].items():
            if back <= L:
                cols = c["columns"] or slice(0, 576)
                flat[r][L - back, cols] = value
        rows = torch.full((pages[r] * P, 576), NAN, dtype=torch.bfloat16)
        rows[:L] = flat[r]
        cache[torch.as_tensor(order[kvp[r]: kvp[r + 1]]).long()] = rows.view(-1, P, 576)
    h = B.LatentHandle(num_heads=H, page_size=P, max_batch=len(lens), max_total_tokens=T, max_num_pages=len(order),
                       num_cache_pages=len(order), sm_count=c["sm_count"])
    ws = torch.empty(h.workspace_size(B.MODE_PREFILL), dtype=torch.uint8, device="cuda")
    h.plan(qo, kvp, order, [(L - 1) % P + 1 for L in lens], workspace=ws, sm_scale=SCALE, causal=c["causal"],
           window_left=c["window_left"])
    out, lse = torch.zeros(T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, device="cuda")
    h.run(q.cuda(), cache.cuda(), out, lse, workspace=ws)
    assert h.check_device_error(ws) == 0
    for r, L in enumerate(lens):
        a, b = int(qo[r]), int(qo[r + 1])
        k = flat[r][:, None]
        ref = by_query(q[a:b], k, k[..., :512], b - a, L, c["causal"], c["window_left"])
        if any(x in (INF, -INF) for x in c["bad"].values()):  # an infinite score's lse is not compared
            seen = torch.isfinite(ref[1]).all(-1)
            l = lse[a:b].cpu()
            l[~seen] = ref[1][~seen].float()
            check(out[a:b], l, ref, name)
        else:
            check(out[a:b], lse[a:b], ref, name)


EXPANDED = {
    "a short prompt": dict(nq=[40], nk=[40], H=2, bad={10: NAN, 35: INF}),
    "every query alone": dict(nq=[128], nk=[128], H=1, bad={0: -INF, 64: NAN, 127: INF}),
    "both query tiles": dict(nq=[256, 200], nk=[256, 300], H=2, bad={63: INF, 64: NAN, 130: INF, 199: NAN, 255: -INF}),
    "odd lengths": dict(nq=[129, 190, 3], nk=[191, 193, 64], H=2, bad={63: NAN, 120: INF, 190: NAN}),
    "a window": dict(nq=[300, 20], nk=[300, 400], H=2, window_left=100, bad={5: NAN, 150: INF, 295: NAN}),
    "a window shorter than a tile": dict(nq=[300], nk=[700], H=1, window_left=3, bad={401: NAN, 500: INF, 640: -INF}),
    "not causal, a window": dict(nq=[300], nk=[450], H=2, causal=False, window_left=90, bad={70: NAN, 200: INF}),
    "many tiles": dict(nq=[257], nk=[2001], H=1, bad={1800: NAN, 1999: INF}),
    "growing maxima": dict(nq=[200], nk=[1001], H=2, q_scale=12.0, bad={900: NAN, 990: NAN}),
}


@pytest.mark.parametrize("columns", [[5], [0, 31, 32, 127], None])
@pytest.mark.parametrize("name", EXPANDED)
def test_expanded(name, columns):
    c = dict(causal=True, window_left=-1, q_scale=1.0)
    c.update(EXPANDED[name])
    nq, nk, H = c["nq"], c["nk"], c["H"]
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (nq, nk))
    T, K = int(cu_q[-1]), int(cu_k[-1])
    q = (randn(1, T, H, 192).float() * c["q_scale"]).to(torch.bfloat16)
    kn, kr, v = randn(2, K, H, 128), randn(3, K, 64), randn(4, K, H, 128)
    for s, L in enumerate(nk):
        for at, value in c["bad"].items():
            if at < L:
                v[cu_k[s] + at, H - 1, columns or slice(0, 128)] = value  # the first head of two stays clean
    h = B.LatentHandle(num_heads=H, page_size=64, max_batch=len(nq), max_total_tokens=T, max_num_pages=1, num_cache_pages=1)
    ws = torch.empty(h.workspace_size(B.MODE_DENSE), dtype=torch.uint8, device="cuda")
    h.plan_dense(cu_q, cu_k, workspace=ws, sm_scale=SCALE, causal=c["causal"], window_left=c["window_left"])
    out, lse = torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, device="cuda")
    h.run_dense(q.cuda(), kn.cuda(), kr.cuda(), v.cuda(), out, lse, workspace=ws)
    assert h.check_device_error(ws) == 0
    for s in range(len(nq)):
        a, b, x, y = int(cu_q[s]), int(cu_q[s + 1]), int(cu_k[s]), int(cu_k[s + 1])
        k = torch.cat([kn[x:y], kr[x:y, None].expand(-1, H, -1)], -1)
        check(out[a:b], lse[a:b], by_query(q[a:b], k, v[x:y], b - a, y - x, c["causal"], c["window_left"]), name)


def test_expanded_keys_that_are_not_seen():
    """NaN and infinite keys behind a query leave it alone; the queries that see them are NaN."""
    L, H = 200, 2
    q, kn, kr, v = randn(1, L, H, 192), randn(2, L, H, 128), randn(3, L, 64), randn(4, L, H, 128)
    kn[150, 1], kr[180] = NAN, NAN
    h = B.LatentHandle(num_heads=H, page_size=64, max_batch=1, max_total_tokens=L, max_num_pages=1, num_cache_pages=1)
    ws = torch.empty(h.workspace_size(B.MODE_DENSE), dtype=torch.uint8, device="cuda")
    h.plan_dense([0, L], [0, L], workspace=ws, sm_scale=SCALE)
    out, lse = torch.zeros(L, H, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(L, H, device="cuda")
    h.run_dense(q.cuda(), kn.cuda(), kr.cuda(), v.cuda(), out, lse, workspace=ws)
    k = torch.cat([kn, kr[:, None].expand(-1, H, -1)], -1)
    check(out, lse, by_query(q, k, v, L, L, True, -1), "keys")
    assert torch.isfinite(out[:180, 0]).all() and torch.isfinite(out[:150, 1]).all()


def test_expanded_scores_of_minus_infinity():
    """A query whose keys all score -inf is NaN, one that sees others is not."""
    L, H = 70, 1
    q, kn, kr, v = randn(1, L, H, 192), randn(2, L, H, 128), randn(3, L, 64), randn(4, L, H, 128)
    q[..., 5] = 1.0
    kn[0, :, 5], kn[20, :, 5] = -INF, -INF
    h = B.LatentHandle(num_heads=H, page_size=64, max_batch=1, max_total_tokens=L, max_num_pages=1, num_cache_pages=1)
    ws = torch.empty(h.workspace_size(B.MODE_DENSE), dtype=torch.uint8, device="cuda")
    for window in (-1, 0):
        h.plan_dense([0, L], [0, L], workspace=ws, sm_scale=SCALE, window_left=window)
        out, lse = torch.zeros(L, H, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(L, H, device="cuda")
        h.run_dense(q.cuda(), kn.cuda(), kr.cuda(), v.cuda(), out, lse, workspace=ws)
        k = torch.cat([kn, kr[:, None]], -1)
        check(out, lse, by_query(q, k, v, L, L, True, window), f"window {window}")
        assert torch.isnan(out[[0] if window else [0, 20]]).all() and lse[0, 0] == -INF


@pytest.mark.parametrize("value", [NAN, INF])
def test_absorbed_result_is_that_of_finite_keys(value):
    """The tokens that do not see the bad one: within rounding of the same step without it, and the same
    bits where no row of their 64 sees it."""
    H, L, n, P = 64, 130, 3, 64  # a unit a token
    q, x = randn(1, n, H, 576), randn(2, L, 576)
    outs = []
    for bad in (0.5, value):
        y = x.clone()
        y[L - 1] = bad
        cache = torch.zeros(3, P, 576, dtype=torch.bfloat16)
        cache.view(-1, 576)[:L] = y
        h = B.LatentHandle(num_heads=H, page_size=P, max_batch=1, max_total_tokens=n, max_num_pages=3, num_cache_pages=3)
        ws = torch.empty(h.workspace_size(B.MODE_PREFILL), dtype=torch.uint8, device="cuda")
        h.plan([0, n], [0, 3], [0, 1, 2], [L - 128], workspace=ws, sm_scale=SCALE)
        out = torch.zeros(n, H, 512, dtype=torch.bfloat16, device="cuda")
        h.run(q.cuda(), cache.cuda(), out, workspace=ws)
        outs.append(out.cpu())
    assert torch.equal(outs[0][:2].view(torch.int16), outs[1][:2].view(torch.int16))
    assert torch.isnan(outs[1][2]).all()
