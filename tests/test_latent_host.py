"""Latent attention on the host (no GPU): configuration and plan refusals, workspace bounds, and the
64-bit reference of the GPU tests against closed forms."""
import ctypes
import math

import numpy as np
import pytest
import torch

import latent_ref as R
from paged_kv_attention_gqa_gb300 import binding as B
from paged_kv_attention_gqa_gb300 import build as pkv_build


@pytest.fixture(scope="module", autouse=True)
def _build():
    pkv_build.build()


def make(**kw):
    cfg = dict(num_heads=16, page_size=64, max_batch=4, max_total_tokens=100, max_num_pages=50, num_cache_pages=60, sm_count=152)
    cfg.update(kw)
    return B.LatentHandle(**cfg)


@pytest.mark.parametrize("kw,status", [
    (dict(latent_dim=256), B.ERR_UNSUPPORTED), (dict(rope_dim=32), B.ERR_UNSUPPORTED), (dict(v_dim=64), B.ERR_UNSUPPORTED),
    (dict(nope_dim=64), B.ERR_UNSUPPORTED), (dict(page_size=4), B.ERR_UNSUPPORTED), (dict(page_size=48), B.ERR_UNSUPPORTED),
    (dict(page_size=2048), B.ERR_UNSUPPORTED), (dict(num_heads=1025), B.ERR_UNSUPPORTED), (dict(num_heads=0), B.ERR_INVALID),
    (dict(max_batch=0), B.ERR_INVALID), (dict(max_total_tokens=0), B.ERR_INVALID), (dict(sm_count=-1), B.ERR_INVALID),
    (dict(num_cache_pages=1 << 26), B.ERR_UNSUPPORTED), (dict(max_total_tokens=1 << 28), B.ERR_UNSUPPORTED),
    (dict(max_num_pages=1 << 26), B.ERR_UNSUPPORTED), (dict(enable_nvtx=2), B.ERR_INVALID),
])
def test_create_rejects(kw, status):
    with pytest.raises(B.PkvError) as e:
        make(**kw)
    assert e.value.status == status


def plan(h, qo, kvp, kvi, lpl, causal=1, window=-1, scale=0.1, ws=256, ws_bytes=1 << 30):
    p = lambda a: None if a is None else np.ascontiguousarray(np.asarray(a, np.int32))
    arrs = [p(a) for a in (qo, kvp, kvi, lpl)]
    ptr = [None if a is None else a.ctypes.data_as(ctypes.c_void_p) for a in arrs]
    st = h.lib.pkv_latent_plan(h.h, *ptr, len(arrs[1]) - 1, causal, window, scale, ctypes.c_void_p(ws), ws_bytes, None)
    return st, h.lib.pkv_latent_last_error(h.h).decode()


@pytest.mark.parametrize("kw,word", [
    (dict(scale=0.0), "sm_scale"), (dict(scale=float("inf")), "sm_scale"), (dict(scale=float("nan")), "sm_scale"),
    (dict(scale=-1.0), "sm_scale"), (dict(causal=2), "causal"), (dict(window=-2), "window_left"),
    (dict(kvi=[1, 60]), "page id"), (dict(kvi=[-1, 2]), "page id"), (dict(lpl=[65]), "last_page_len"),
    (dict(lpl=[0]), "last_page_len"), (dict(qo=[0, 101]), "maximum"), (dict(kvp=[0, 1], kvi=[3], lpl=[2], qo=[0, 3]), "new tokens"),
    (dict(kvp=[1, 2]), "start at 0"), (dict(kvp=[0, 51], kvi=[1] * 51), "max_num_pages"), (dict(ws=0), "workspace"),
    (dict(ws=128), "aligned"), (dict(kvp=[0] * 6, lpl=[0] * 5, qo=[0] * 6), "max_batch"),
    (dict(kvp=[0] * 6, lpl=[0] * 5, qo=None), "max_batch"), (dict(ws_bytes=512), "too small"),
])
def test_plan_rejects(kw, word):
    args = dict(qo=[0, 1], kvp=[0, 2], kvi=[3, 4], lpl=[5])
    args.update(kw)
    st, msg = plan(make(), **args)
    assert st in (B.ERR_INVALID, B.ERR_WORKSPACE) and word in msg, (st, msg)


def test_dense_plan_rejects():
    h = make()
    for cu_q, cu_k, scale in (([0, 3], [0, 2], 0.1), ([0, 2, 1], [0, 2, 3], 0.1), ([1, 2], [0, 2], 0.1), ([0, 101], [0, 101], 0.1),
                              ([0, 2], [0, 2], 0.0)):
        a, b = np.asarray(cu_q, np.int32), np.asarray(cu_k, np.int32)
        st = h.lib.pkv_latent_plan_dense(h.h, a.ctypes.data_as(ctypes.c_void_p), b.ctypes.data_as(ctypes.c_void_p), len(a) - 1,
                                         1, -1, scale, ctypes.c_void_p(256), 1 << 30, None)
        assert st == B.ERR_INVALID, (cu_q, cu_k)


def test_run_without_a_plan_is_refused():
    h = make()
    p = ctypes.c_void_p(256)
    assert h.lib.pkv_latent_run(h.h, p, p, p, None, p, None) == B.ERR_NOT_PLANNED
    assert h.lib.pkv_latent_run(None, None, None, None, None, None, None) == B.ERR_INVALID
    with pytest.raises(B.PkvError):
        h.workspace_size(B.MODE_DECODE)


def test_workspace_grows_with_the_maxima():
    a, b = make().workspace_size(B.MODE_PREFILL), make(max_total_tokens=100000, max_batch=4000).workspace_size(B.MODE_PREFILL)
    # two 64-row partials per CTA, whatever the step's size
    assert 2 * 152 * 64 * 513 * 4 <= a < b < a + (8 << 20)


def test_reference_against_closed_forms():
    # equal keys: the output is the mean of the values seen
    n, L, H = 3, 10, 2
    q, k = torch.randn(n, H, 8), torch.ones(L, 1, 8)
    v = torch.randn(L, 1, 4)
    o, z, _ = R.attend(q, k, v, R.visible(L, n), 0.5)
    for i in range(n):
        seen = L - n + i + 1
        assert torch.allclose(o[i], v[:seen, 0].double().mean(0).expand(H, -1))
        assert torch.allclose(z[i], q[i].double().sum(-1) * 0.5 + math.log(seen))
    # a window of w sees w + 1 keys
    assert R.visible(L, n, window_left=2).sum(1).tolist() == [3, 3, 3]
    assert R.visible(L, n, causal=False).all()
