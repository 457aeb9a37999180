"""Eviction and weights plans on the host (no GPU): refusals and workspace bounds, and the 64-bit
references of the GPU tests."""
import ctypes
import math

import numpy as np
import pytest
import torch

import evict_ref as E
from paged_kv_attention_gqa_gb300 import binding as B
from paged_kv_attention_gqa_gb300 import build as pkv_build


@pytest.fixture(scope="module", autouse=True)
def _build():
    pkv_build.build()


def make(**kw):
    cfg = dict(num_qo_heads=8, num_kv_heads=2, head_dim=64, page_size=16, max_batch=4, max_total_tokens=100, max_num_pages=50,
               num_cache_pages=60, sm_count=152)
    cfg.update(kw)
    return B.Handle(**cfg)


def _ptrs(*arrays):
    keep = [None if a is None else np.ascontiguousarray(np.asarray(a, np.int32)) for a in arrays]
    return keep, [None if a is None else a.ctypes.data_as(ctypes.c_void_p) for a in keep]


def plan_evict(h, kvp, kvi, lpl, keep, dst_indptr, dst, sink=0, recent=0, ws=256, ws_bytes=1 << 30):
    a, p = _ptrs(kvp, kvi, lpl, keep, dst_indptr, dst)
    st = h.lib.pkv_plan_evict(h.h, p[0], p[1], p[2], len(a[0]) - 1, p[3], sink, recent, p[4], p[5], ctypes.c_void_p(ws),
                              ws_bytes, None)
    return st, h.lib.pkv_last_error(h.h).decode()


@pytest.mark.parametrize("kw,word", [
    (dict(keep=[-1]), "keep[0]"), (dict(sink=10, recent=11), "num_sink"), (dict(sink=-1), "num_sink"), (dict(recent=-1), "num_recent"),
    (dict(dst_indptr=[0, 1], dst=[50]), "needs 2 new pages"), (dict(dst_indptr=[1, 3]), "start at 0"),
    (dict(dst=[50, 50]), "listed twice"), (dict(dst=[50, 4]), "a page of a row"), (dict(dst=[50, 60]), "outside the cache"),
    (dict(dst=[50, -1]), "outside the cache"), (dict(keep=[36]), "needs 0 new pages"), (dict(keep=None), "required"),
    (dict(dst_indptr=None), "required"), (dict(dst=None), "dst_indices"), (dict(kvi=[3, 4, 60]), "page id"),
    (dict(lpl=[17]), "last_page_len"), (dict(ws=0), "workspace"), (dict(ws=64), "aligned"), (dict(ws_bytes=256), "too small"),
    (dict(kvp=[0] * 6, lpl=[0] * 5, keep=[0] * 5, dst_indptr=[0] * 6), "max_batch"),
])
def test_plan_evict_rejects(kw, word):
    args = dict(kvp=[0, 3], kvi=[3, 4, 5], lpl=[4], keep=[20], dst_indptr=[0, 2], dst=[50, 51])
    args.update(kw)
    st, msg = plan_evict(make(), **args)
    assert st in (B.ERR_INVALID, B.ERR_WORKSPACE) and word in msg, (st, msg)


def plan_weights(h, mode, qo=(0, 1), kvp=(0, 2), kvi=(3, 4), lpl=(4,), causal=1):
    a, p = _ptrs(None if mode == B.MODE_DECODE_WEIGHTS else qo, kvp, kvi, lpl)
    st = h.lib.pkv_plan(h.h, mode, *p, len(a[1]) - 1, causal, -1, 0.0, ctypes.c_void_p(256), 128, None)
    return st, h.lib.pkv_last_error(h.h).decode()


@pytest.mark.parametrize("mode", [B.MODE_DECODE_WEIGHTS, B.MODE_WEIGHTS])
def test_weights_plans_reject(mode):
    st, msg = plan_weights(make(), mode, kvi=(3, 3))
    assert st == B.ERR_INVALID and "listed twice" in msg
    st, msg = plan_weights(make(), mode, qo=(0, 1, 2), kvp=(0, 1, 2), kvi=(7, 7), lpl=(4, 4))
    assert st == B.ERR_INVALID and "listed twice" in msg
    st, msg = plan_weights(make(graph_static=1), mode)
    assert st == B.ERR_UNSUPPORTED
    st, msg = plan_weights(make(), mode, lpl=(17,))
    assert st == B.ERR_INVALID
    assert plan_weights(make(), mode)[0] == B.ERR_WORKSPACE  # nothing else was wrong


def test_weights_plan_needs_boxes_and_a_mask():
    st, msg = plan_weights(make(page_size=4), B.MODE_WEIGHTS)
    assert st == B.ERR_UNSUPPORTED and "8 slots" in msg
    assert plan_weights(make(), B.MODE_WEIGHTS, causal=2)[0] == B.ERR_INVALID
    # EVICT plans are made by their own call
    assert plan_weights(make(), B.MODE_EVICT)[0] == B.ERR_INVALID


def test_runs_without_a_plan_are_refused():
    h, p = make(), ctypes.c_void_p(256)
    assert h.lib.pkv_run_evict(h.h, p, p, p, p, None) == B.ERR_NOT_PLANNED
    assert h.lib.pkv_run_weights(h.h, p, p, p, p, 1.0, p, None) == B.ERR_NOT_PLANNED
    assert h.lib.pkv_run_decode_weights(h.h, p, p, p, p, p, 1.0, p, None) == B.ERR_NOT_PLANNED
    assert h.lib.pkv_run_evict(None, p, p, p, p, None) == B.ERR_INVALID


def test_workspace_sizes():
    h = make()
    logits = 8 * 4 * 50 * 16
    assert h.workspace_size(B.MODE_DECODE_WEIGHTS) >= h.workspace_size(B.MODE_DECODE) + logits
    assert h.workspace_size(B.MODE_EVICT) > 0 and h.workspace_size(B.MODE_WEIGHTS) > 0
    with pytest.raises(B.PkvError):
        h.workspace_size(7)


def test_reference_selection():
    nan = float("nan")
    assert E.select([5, 1, 3, 3, 0, 9], 6, 4, 1, 1) == [0, 2, 3, 5]
    assert E.select([1, 1, 1, 1], 4, 2, 0, 0) == [0, 1]
    assert E.select([nan, -math.inf, nan, 0.0], 4, 2, 0, 0) == [1, 3]
    assert E.select([0.0, -0.0, 0.0], 3, 2, 0, 0) == [0, 1]
    assert E.select([1, 2], 2, 5, 0, 0) == [0, 1]


def test_reference_weights():
    # one query over equal keys: every key gets 1 / L of each head; the newest from nothing
    cache = torch.ones(3, 2, 4, 1, 8)
    q = torch.randn(1, 2, 8)
    idx = ([0, 1], [0, 2], [2, 0], [3])
    _, lse, _, _ = E.attention(q, cache, *idx, 0.3)
    s, _ = E.add_weights(torch.full((3, 4), 10.0), q, lse, cache, *idx, 0.3, 0.5)
    want = torch.full((3, 4), 10.0).double()
    want[2, :] = 5 + 2 / 7
    want[0, :2] = 5 + 2 / 7
    want[0, 2] = 2 / 7
    assert torch.allclose(s, want)
