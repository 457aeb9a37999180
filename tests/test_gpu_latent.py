"""Latent attention on the GPU (absorbed and expanded forms, the append) against the definition in 64
bits.

Tolerances.  An output element is o = sum_j p_j v_j.  The kernel rounds each weight to bf16 (off by at
most half a step, 2^-8 of the value; their sum is taken unrounded) and the result to bf16 (2^-8 again):
|o - ref| <= 2^-8 (sum_j p_j |v_j| + |o|), plus the 32-bit arithmetic: a score of W products summed in
32 bits is off by at most W 2^-24 |q||k| scale, which shifts numerator and sum by that share each.  The
bound is computed per element in 64 bits and no element may exceed it (by the second-order terms' 1%).
"""
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


@pytest.fixture(scope="module", autouse=True)
def _build():
    from paged_kv_attention_gqa_gb300 import build
    build.build()


def table(lens, P, seed, spare=3):
    g = np.random.default_rng(seed)
    pages = [-(-L // P) for L in lens]
    order = g.permutation(sum(pages) + spare).astype(np.int32)
    kvp = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    lpl = np.array([(L - 1) % P + 1 if L else 0 for L in lens], np.int32)
    return kvp, order[: kvp[-1]], lpl, sum(pages) + spare


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def bits(t):
    return t.contiguous().view(torch.int16)


def check(out, lse, ref, what):
    ref_o, ref_l, mag, err = ref
    o, l = out.double().cpu(), lse.double().cpu()
    assert o.shape == ref_o.shape and torch.isfinite(o).all(), what
    if not o.numel():
        return
    bound = 1.01 * 2.0 ** -8 * (mag + ref_o.abs()) + 2 * err[..., None] * mag + 1e-30
    worst = ((o - ref_o).abs() / bound).max().item()
    assert worst <= 1, f"{what}: {worst:.2f} of the bound"
    worst = ((l - ref_l).abs() / (err + 2.0 ** -20 * (1 + ref_l.abs()))).max().item()
    assert worst <= 1, f"{what}: lse {worst:.2f} of the bound"


class Step:
    def __init__(self, lens, news, H, P, seed, *, causal=True, window_left=-1, poison=True, q_scale=1.0, sm_count=0):
        self.qo = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.kvp, self.kvi, self.lpl, pages = table(lens, P, seed)
        T = int(self.qo[-1])
        self.kw = dict(causal=causal, window_left=window_left)
        self.q = randn(seed + 1, T, H, R.LATENT + R.ROPE, scale=q_scale)
        cache = randn(seed + 2, pages, P, R.LATENT + R.ROPE)
        if poison:  # every slot that holds no token
            used = torch.zeros(pages, P, dtype=torch.bool)
            for r, L in enumerate(lens):
                for i, p in enumerate(self.kvi[self.kvp[r]: self.kvp[r + 1]]):
                    used[p, : max(0, min(P, L - i * P))] = True
            cache[~used] = float("nan")
        self.cache = cache
        self.c_new, self.r_new = randn(seed + 3, T, R.LATENT), randn(seed + 4, T, R.ROPE)
        self.h = B.LatentHandle(num_heads=H, page_size=P, max_batch=max(1, len(lens)), max_total_tokens=max(1, T),
                                max_num_pages=max(1, len(self.kvi)), num_cache_pages=pages, sm_count=sm_count)
        self.ws = torch.empty(self.h.workspace_size(B.MODE_PREFILL), dtype=torch.uint8, device="cuda")
        self.plan()

    def plan(self):
        self.h.plan(self.qo, self.kvp, self.kvi, self.lpl, workspace=self.ws, sm_scale=SCALE, **self.kw)

    def after(self):
        """The cache after the append, by the definition of the write locations."""
        c = self.cache.clone()
        P = c.shape[1]
        for r in range(len(self.kvp) - 1):
            n = int(self.qo[r + 1] - self.qo[r])
            L = int((self.kvp[r + 1] - self.kvp[r] - 1) * P + self.lpl[r]) if n else 0
            for i in range(n):
                p, t = L - n + i, int(self.qo[r]) + i
                c[int(self.kvi[self.kvp[r] + p // P]), p % P] = torch.cat([self.c_new[t], self.r_new[t]])
        return c

    def reference(self, cache):
        return R.paged(self.q, cache, self.qo, self.kvp, self.kvi, self.lpl, SCALE, **self.kw)

    def run(self, append=True, lse=True):
        q, cache = self.q.cuda(), self.cache.cuda()
        T, H = q.shape[:2]
        self.out = torch.full((T + 1, H, R.LATENT), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T + 1, H), 7.0, device="cuda")
        if append:
            self.h.append_planned(self.c_new.cuda(), self.r_new.cuda(), cache, workspace=self.ws)
        self.h.run(q, cache, self.out[:T], self.lse[:T] if lse else None, workspace=self.ws)
        torch.cuda.synchronize()
        assert self.h.check_device_error(self.ws) == 0
        assert (self.out[T] == 7).all() and (self.lse[T] == 7).all(), "rows behind the last token are left alone"
        return self.out[:T], self.lse[:T], cache


CASES = {
    "one token": dict(lens=[1], news=[1], H=1, P=8),
    "one row": dict(lens=[517], news=[1], H=16, P=64),
    "tile edges": dict(lens=[63, 64, 65, 127, 128, 129, 1], news=[1] * 7, H=16, P=64),
    "small pages": dict(lens=[9, 8, 7, 300, 77], news=[1] * 5, H=5, P=8),
    "pages of 16": dict(lens=[100, 1000, 333], news=[1, 1, 1], H=32, P=16),
    "pages of 32": dict(lens=[95, 1025], news=[1, 2], H=64, P=32),
    "large pages": dict(lens=[1500, 3, 1024], news=[1, 3, 2], H=8, P=1024),
    "65 heads": dict(lens=[200, 70], news=[1, 1], H=65, P=64),
    "128 heads": dict(lens=[700, 333, 64], news=[1, 1, 1], H=128, P=16),
    "200 heads, 2 tokens": dict(lens=[130, 40], news=[2, 1], H=200, P=64),
    "ragged new tokens": dict(lens=[150, 9, 64, 40, 500], news=[17, 9, 0, 1, 3], H=20, P=16),
    "empty rows": dict(lens=[0, 33, 0, 5], news=[0, 1, 0, 5], H=16, P=8),
    "prompt": dict(lens=[257], news=[257], H=4, P=64),
    "window": dict(lens=[500, 90, 64], news=[1, 3, 2], H=16, P=16, window_left=70),
    "window 0": dict(lens=[130], news=[3], H=16, P=16, window_left=0),
    "not causal": dict(lens=[140, 66], news=[5, 1], H=16, P=32, causal=False),
    "peaked scores": dict(lens=[900, 222], news=[1, 2], H=16, P=64, q_scale=8.0),
    "many pieces": dict(lens=[9000, 64, 5000], news=[1, 1, 1], H=16, P=64),
    "few CTAs": dict(lens=[400, 900, 64, 1, 700], news=[1, 2, 1, 1, 4], H=40, P=16, sm_count=3),
    "one CTA": dict(lens=[400, 64, 130], news=[1, 1, 2], H=16, P=64, sm_count=1),
}


# several blocks of 64 rows over the same keys
BLOCKS = {
    "128 heads, one row": dict(lens=[1], news=[1], H=128, P=64),
    "128 heads, pages of 8": dict(lens=[200, 9, 1000], news=[1, 1, 1], H=128, P=8),
    "128 heads, pages of 32, a row longer than the others": dict(lens=[70, 9000, 65], news=[1, 1, 1], H=128, P=32),
    "100 heads": dict(lens=[300, 64, 65, 3000], news=[1, 1, 1, 1], H=100, P=64),
    "256 heads": dict(lens=[300, 700], news=[1, 1], H=256, P=16),
    "1024 heads": dict(lens=[130, 1], news=[1, 1], H=1024, P=64),
    "64 heads, two tokens, not causal": dict(lens=[500, 64], news=[2, 2], H=64, P=16, causal=False),
    "32 heads, four tokens": dict(lens=[500, 1000], news=[4, 4], H=32, P=64),
    "128 heads, a window": dict(lens=[500, 90], news=[1, 1], H=128, P=16, window_left=70),
    "128 heads, empty rows": dict(lens=[0, 33, 0, 5], news=[0, 1, 0, 1], H=128, P=8),
    "128 heads, three CTAs": dict(lens=[400, 900, 64, 1, 700], news=[1] * 5, H=128, P=16, sm_count=3),
    "128 heads, five CTAs": dict(lens=[400, 900, 64, 1, 700], news=[1] * 5, H=128, P=64, sm_count=5),
    "128 heads, peaked scores": dict(lens=[900, 222], news=[1, 1], H=128, P=64, q_scale=8.0),
    "some rows with one block": dict(lens=[400, 90], news=[2, 1], H=64, P=64),
}
CASES.update(BLOCKS)


@pytest.mark.parametrize("name", CASES)
def test_absorbed_step(name):
    c = CASES[name]
    s = Step(seed=11 + len(name), **c)
    out, lse, cache = s.run()
    want = s.after()
    assert torch.equal(bits(cache.cpu()), bits(want)), "append"
    check(out, lse, s.reference(want), name)


def test_absorbed_without_lse_and_twice():
    s = Step([700, 90], [1, 2], 24, 16, 5)
    a, l, _ = s.run()
    b, _, _ = s.run(lse=False)
    assert torch.equal(bits(a), bits(b))
    assert (s.lse == 7).all()
    c, l2, _ = s.run()
    assert torch.equal(bits(a), bits(c)) and torch.equal(l, l2)


def test_growing_scores_rescale():
    """Scores that grow along the row move the running maximum at nearly every tile."""
    s = Step([1000], [1], 16, 64, 21, poison=False, sm_count=2)
    ids = torch.as_tensor(s.kvi).long()
    flat = s.cache[ids].reshape(-1, 576)
    u = torch.nn.functional.normalize(s.q[0].double().mean(0), dim=0)
    ramp = torch.linspace(0, 6, 1000)[:, None].double()
    flat[:1000] = (flat[:1000].double() * 0.2 + ramp * u * 20).to(torch.bfloat16)
    s.cache[ids] = flat.reshape(-1, 64, 576)
    out, lse, cache = s.run(append=False)
    check(out, lse, s.reference(s.cache), "ramp")


def test_nan_query_stays_in_its_row():
    s = Step([300, 300], [1, 1], 16, 64, 3)
    clean, cl, _ = s.run()
    s.q[1, 3] = float("nan")
    out, lse, _ = s.run()
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
    keep = torch.ones(2, 16, dtype=torch.bool, device="cuda")
    keep[1, 3] = False
    assert torch.equal(bits(out[keep]), bits(clean[keep])) and torch.equal(lse[keep], cl[keep])


def test_result_does_not_depend_on_neighbours():
    """A row's result is the same bits beside rows with other values behind it in q."""
    s = Step([400, 400], [1, 1], 12, 64, 9, sm_count=14)
    a, al, _ = s.run()
    s.q[1] *= 50
    b, bl, _ = s.run()
    assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(al[0], bl[0])


def test_strided_append():
    s = Step([70, 20], [3, 2], 8, 16, 17)
    both = torch.cat([s.c_new, s.r_new, torch.zeros(5, 8, dtype=torch.bfloat16)], 1).cuda()
    cache = s.cache.cuda()
    s.h.append_planned(both[:, :512], both[:, 512:576], cache, workspace=s.ws)
    assert torch.equal(bits(cache.cpu()), bits(s.after()))


def test_graph_replay_and_streams():
    """A captured append + run, replayed on changed inputs; then the plan and the run on a side stream."""
    s = Step([333, 64, 700], [1, 2, 1], 16, 16, 23)
    first, _, _ = s.run()  # sets kernel attributes before the capture
    q, cache, cn, rn = s.q.cuda(), s.cache.cuda(), s.c_new.cuda(), s.r_new.cuda()
    out, lse = torch.zeros_like(first), torch.zeros(first.shape[:2], device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.h.append_planned(cn, rn, cache, workspace=s.ws)
        s.h.run(q, cache, out, lse, workspace=s.ws)
    q.mul_(-0.5)
    s.q = s.q * -0.5
    g.replay()
    torch.cuda.synchronize()
    check(out, lse, s.reference(s.after()), "replay")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = torch.zeros_like(out)
    with torch.cuda.stream(side):
        s.plan()
        s.h.run(q, cache, out2, None, workspace=s.ws)
    side.synchronize()
    assert torch.equal(bits(out), bits(out2))


def test_long_offsets():
    """A cache whose byte offsets pass 32 bits: the row's pages are the last ones of 4.7 GB."""
    P, pages, L = 1024, 4000, 2000
    cache = torch.zeros(pages, P, 576, dtype=torch.bfloat16, device="cuda")
    x = randn(4, L, 576)
    cache.view(-1, 576)[3999 * P: 3999 * P + 1024] = x[:1024].cuda()
    cache.view(-1, 576)[3998 * P: 3998 * P + L - 1024] = x[1024:].cuda()
    h = B.LatentHandle(num_heads=16, page_size=P, max_batch=1, max_total_tokens=1, max_num_pages=2, num_cache_pages=pages)
    ws = torch.empty(h.workspace_size(B.MODE_PREFILL), dtype=torch.uint8, device="cuda")
    h.plan(None, [0, 2], [3999, 3998], [L - 1024], workspace=ws, sm_scale=SCALE)
    q = randn(5, 1, 16, 576)
    out = torch.empty(1, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 16, device="cuda")
    c, r = randn(6, 1, 512), randn(7, 1, 64)
    h.append_planned(c.cuda(), r.cuda(), cache, workspace=ws)
    h.run(q.cuda(), cache, out, lse, workspace=ws)
    x[-1] = torch.cat([c, r], 1)
    x = x[:, None]
    check(out, lse, (*R.attend(q, x, x[..., :512], R.visible(L, 1), SCALE), R.score_error(q, x, SCALE)), "long offsets")


# ---------------------------------------------------------------- expanded form

DENSE = {
    "one token": dict(nq=[1], nk=[1], H=1),
    "one query": dict(nq=[1], nk=[300], H=3),
    "short": dict(nq=[137], nk=[137], H=16),
    "edges": dict(nq=[127, 128, 129, 256, 257], nk=[127, 128, 129, 256, 257], H=2),
    "ragged, empty segments": dict(nq=[5, 0, 300, 0, 1], nk=[40, 0, 513, 70, 129], H=4),
    "window": dict(nq=[300, 20], nk=[300, 400], H=2, window_left=100),
    "not causal": dict(nq=[200, 3], nk=[290, 130], H=2, causal=False),
    "peaked": dict(nq=[400], nk=[400], H=2, q_scale=6.0),
    "long": dict(nq=[1000], nk=[1500], H=2),
}


def dense_step(nq, nk, H, seed, *, causal=True, window_left=-1, q_scale=1.0, packed=True):
    cu_q = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum(nk)]).astype(np.int32)
    T, K = int(cu_q[-1]), int(cu_k[-1])
    q = randn(seed, T, H, 192, scale=q_scale)
    kv = randn(seed + 1, K, H, 256)
    kr = randn(seed + 2, K, 64)
    h = B.LatentHandle(num_heads=H, page_size=64, max_batch=len(nq), max_total_tokens=max(T, 1), max_num_pages=1,
                       num_cache_pages=1)
    ws = torch.empty(h.workspace_size(B.MODE_DENSE), dtype=torch.uint8, device="cuda")
    h.plan_dense(cu_q, cu_k, workspace=ws, sm_scale=SCALE, causal=causal, window_left=window_left)
    kvd = kv.cuda()
    kn, v = kvd[..., :128], kvd[..., 128:]
    if not packed:
        kn, v = kn.contiguous(), v.contiguous()
    out = torch.full((T + 1, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 1, H), 7.0, device="cuda")
    h.run_dense(q.cuda(), kn, kr.cuda(), v, out[:T], lse[:T], workspace=ws)
    torch.cuda.synchronize()
    assert h.check_device_error(ws) == 0
    assert (out[T] == 7).all() and (lse[T] == 7).all()
    return q, kv[..., :128], kr, kv[..., 128:], cu_q.tolist(), cu_k.tolist(), out[:T], lse[:T]


@pytest.mark.parametrize("name", DENSE)
@pytest.mark.parametrize("packed", [True, False])
def test_expanded(name, packed):
    c = dict(DENSE[name])
    mask = dict(causal=c.get("causal", True), window_left=c.get("window_left", -1))
    q, kn, kr, v, cu_q, cu_k, out, lse = dense_step(seed=31, packed=packed, **c)
    check(out, lse, R.dense(q, kn, kr, v, cu_q, cu_k, SCALE, **mask), name)


DENSE_TILES = {
    "64-key edges": dict(nq=[129, 190, 193, 1], nk=[191, 192, 193, 64], H=2),
    "a window across tiles": dict(nq=[260, 130, 64], nk=[260, 330, 65], H=2, window_left=65),
    "a window shorter than a tile": dict(nq=[300], nk=[700], H=1, window_left=3),
    "not causal, two query tiles": dict(nq=[129, 256], nk=[129, 1000], H=2, causal=False),
    "not causal, a window": dict(nq=[300], nk=[450], H=2, causal=False, window_left=90),
    "1024 heads": dict(nq=[2, 1], nk=[70, 1], H=1024),
    "many tiles": dict(nq=[257], nk=[6001], H=1),
    "many tiles, growing maxima": dict(nq=[200], nk=[3001], H=2, q_scale=12.0),
}


@pytest.mark.parametrize("name", DENSE_TILES)
def test_expanded_tiles(name):
    c = dict(DENSE_TILES[name])
    mask = dict(causal=c.get("causal", True), window_left=c.get("window_left", -1))
    q, kn, kr, v, cu_q, cu_k, out, lse = dense_step(seed=37, **c)
    check(out, lse, R.dense(q, kn, kr, v, cu_q, cu_k, SCALE, **mask), name)


def test_expanded_head_major_and_captured():
    """Keys and values stored head by head, and the call captured and replayed on another stream: the bits
    of the token-major call."""
    q, kn, kr, v, cu_q, cu_k, out, lse = dense_step([300, 70], [333, 70], 3, 43)
    h = B.LatentHandle(num_heads=3, page_size=64, max_batch=2, max_total_tokens=370, max_num_pages=1, num_cache_pages=1)
    ws = torch.empty(h.workspace_size(B.MODE_DENSE), dtype=torch.uint8, device="cuda")
    h.plan_dense(cu_q, cu_k, workspace=ws, sm_scale=SCALE)
    head_major = lambda t: t.permute(1, 0, 2).contiguous().cuda().permute(1, 0, 2)
    args = (q.cuda(), head_major(kn), kr.cuda(), head_major(v))
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        h.run_dense(*args, o2, l2, workspace=ws)
    with torch.cuda.stream(torch.cuda.Stream()):
        g.replay()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(o2), bits(out)) and torch.equal(l2, lse)


def test_expanded_refuses_strides_it_cannot_step():
    q, kn, kr, v, cu_q, cu_k, out, lse = dense_step([40], [40], 2, 47)
    h = B.LatentHandle(num_heads=2, page_size=64, max_batch=1, max_total_tokens=40, max_num_pages=1, num_cache_pages=1)
    ws = torch.empty(h.workspace_size(B.MODE_DENSE), dtype=torch.uint8, device="cuda")
    h.plan_dense(cu_q, cu_k, workspace=ws, sm_scale=SCALE)
    q, kn, kr, v = q.cuda(), kn.cuda(), kr.cuda(), v.cuda()
    wide = torch.zeros(40, 2, 132, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(k_nope=kn[:, :1].expand(-1, 2, -1)),    # every head the same row: a stride of nothing
                dict(v=wide[..., :128]),                      # rows 264 bytes apart
                dict(k_rope=kr[:1].expand(40, -1))):
        a = dict(q=q, k_nope=kn.contiguous(), k_rope=kr, v=v.contiguous(), out=out)
        a.update(bad)
        with pytest.raises(B.PkvError) as e:
            h.run_dense(**a, workspace=ws)
        assert e.value.status == B.ERR_INVALID


def test_expanded_next_segment_does_not_leak():
    """Keys and values of the next segment hold infinities and NaN: the first one's result is the same."""
    q, kn, kr, v, cu_q, cu_k, out, lse = dense_step([50, 30], [50, 30], 2, 41)
    h = B.LatentHandle(num_heads=2, page_size=64, max_batch=2, max_total_tokens=80, max_num_pages=1, num_cache_pages=1)
    ws = torch.empty(h.workspace_size(B.MODE_DENSE), dtype=torch.uint8, device="cuda")
    h.plan_dense(cu_q, cu_k, workspace=ws, sm_scale=SCALE)
    kn, kr, v, q = kn.clone(), kr.clone(), v.clone(), q.clone()
    kn[50:], kr[50:], v[50:70], v[70:], q[50:] = float("nan"), float("inf"), float("inf"), float("nan"), float("nan")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    h.run_dense(q.cuda(), kn.cuda(), kr.cuda(), v.cuda(), o2, l2, workspace=ws)
    assert torch.equal(bits(o2[:50]), bits(out[:50])) and torch.equal(l2[:50], lse[:50])


def test_both_forms_agree():
    """Absorbed and expanded attention of the same prompt, joined through the projections: q_nope W_uk^T
    on the latents equals q_nope on (c W_uk).  Each form's inputs carry two bf16 roundings of their own
    (2^-8 each, of scores of order 2 and of values), the outputs one more: within 2e-2 in norm."""
    g = torch.Generator().manual_seed(2)
    T, H = 150, 4
    c = torch.randn(T, 512, generator=g).to(torch.bfloat16)
    kr = torch.randn(T, 64, generator=g).to(torch.bfloat16)
    wk = (torch.randn(H, 512, 128, generator=g) / 512 ** 0.5).to(torch.bfloat16)
    wv = (torch.randn(H, 512, 128, generator=g) / 512 ** 0.5).to(torch.bfloat16)
    q = torch.randn(T, H, 192, generator=g).to(torch.bfloat16)
    kn = torch.einsum("tc,hcd->thd", c.float(), wk.float()).to(torch.bfloat16)
    v = torch.einsum("tc,hcd->thd", c.float(), wv.float()).to(torch.bfloat16)
    qa = torch.cat([torch.einsum("thd,hcd->thc", q[..., :128].float(), wk.float()).to(torch.bfloat16), q[..., 128:]], -1)
    P, pages = 16, -(-T // 16)
    h = B.LatentHandle(num_heads=H, page_size=P, max_batch=1, max_total_tokens=T, max_num_pages=pages, num_cache_pages=pages)
    ws = torch.empty(h.workspace_size(B.MODE_PREFILL), dtype=torch.uint8, device="cuda")
    h.plan([0, T], [0, pages], np.arange(pages), [(T - 1) % P + 1], workspace=ws, sm_scale=SCALE)
    cache = torch.zeros(pages, P, 576, dtype=torch.bfloat16, device="cuda")
    h.append_planned(c.cuda(), kr.cuda(), cache, workspace=ws)
    o = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda")
    h.run(qa.contiguous().cuda(), cache, o, workspace=ws)
    absorbed = torch.einsum("thc,hcd->thd", o.double().cpu(), wv.double())
    wd = torch.empty(h.workspace_size(B.MODE_DENSE), dtype=torch.uint8, device="cuda")
    h.plan_dense([0, T], [0, T], workspace=wd, sm_scale=SCALE)
    e = torch.empty(T, H, 128, dtype=torch.bfloat16, device="cuda")
    h.run_dense(q.cuda(), kn.cuda(), kr.cuda(), v.cuda(), e, workspace=wd)
    assert (absorbed - e.double().cpu()).norm() / absorbed.norm() < 2e-2


def test_stale_plans_and_wrong_tensors_are_refused():
    s = Step([64], [1], 16, 64, 3)
    q, cache = s.q.cuda(), s.cache.cuda()
    out = torch.empty(1, 16, 512, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.PkvError) as e:
        s.h.run(q, cache, out, workspace=torch.empty_like(s.ws))
    assert e.value.status == B.ERR_NOT_PLANNED
    for bad in (dict(q=q.float()), dict(q=s.q), dict(cache_layer=cache[:-1]), dict(out=out[..., :256]), dict(q=q.expand(2, -1, -1)),
                dict(lse=torch.empty(1, 15, device="cuda"))):
        args = dict(q=q, cache_layer=cache, out=out)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            s.h.run(**args, workspace=s.ws)
    wd = torch.empty(s.h.workspace_size(B.MODE_DENSE), dtype=torch.uint8, device="cuda")
    s.h.plan_dense([0, 1], [0, 1], workspace=wd, sm_scale=SCALE)
    with pytest.raises(B.PkvError) as e:
        s.h.run(q, cache, out, workspace=wd)
    assert e.value.status == B.ERR_NOT_PLANNED
    kv = torch.zeros(1, 16, 260, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.PkvError) as e:  # values that do not start on 16 bytes
        s.h.run_dense(torch.zeros(1, 16, 192, dtype=torch.bfloat16, device="cuda"), kv[..., :128],
                      torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda"), kv[..., 130:258],
                      torch.empty(1, 16, 128, dtype=torch.bfloat16, device="cuda"), workspace=wd)
    assert e.value.status == B.ERR_INVALID
