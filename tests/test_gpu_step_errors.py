"""Errors of a speculative step stay in the workspace until they are read: later plans, replayed ones among them, do not
wipe them, and none is reported that was not recorded."""
import pytest
import torch

import tree_ref as R
from paged_kv_attention_gqa_gb300 import binding as B
from test_gpu_step import Loop, trees_of
from test_gpu_tree import Step

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def _build():
    from paged_kv_attention_gqa_gb300 import build
    build.build()


@pytest.mark.parametrize("captured", [False, True])
def test_an_error_outlives_the_steps_behind_it(captured):
    """A page id outside the cache in one step, good steps behind it, and the host looks once, at the end."""
    loop = Loop([37, 20, 150], 8, 2, 64, 16, 2, 30, 21, 12)
    step = loop.step
    if captured:
        saved = {k: v.clone() for k, v in loop.d.items()}
        loop.step()
        torch.cuda.synchronize()
        for k, v in saved.items():
            loop.d[k].copy_(v)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            loop.step()
        step = graph.replay
    good = loop.d["table"][0, 0].clone()
    for i in range(4):
        loop.feed(trees_of(i + 1, 3, 12), 40 + i)
        loop.d["table"][0, 0] = loop.h.cfg.num_cache_pages if i == 1 else good  # row 0's first page: its keys read as zeros
        step()
        torch.cuda.synchronize()
    assert loop.h.check_device_error(loop.ws) == 6
    assert loop.h.check_device_error(loop.ws) == 0, "reading clears it"
    loop.feed(trees_of(5, 3, 12), 50)
    step()
    torch.cuda.synchronize()
    assert loop.h.check_device_error(loop.ws) == 0


def test_the_first_error_is_the_one_that_is_read():
    s = Step([100, 60], [R.tree(5, 2), R.tree(4, 2)], 8, 2, 128, 16, 60)
    good = s.trees
    s.trees = [good[0], [-1, 0, 1, 9]]  # a parent behind its child
    s.plan()
    s.trees = good
    s.dev["last"][1] = 0  # a row that does not agree
    s.plan()
    s.dev["last"][1] = int(s.last[1])
    s.plan()
    s.run()
    assert s.h.check_device_error(s.ws) == 7
    s.check("good rows behind it")


def test_what_a_workspace_held_before_is_no_error():
    """Memory of any content, a plan of another kind, and what another handle left unread."""
    s = Step([100, 60], [R.tree(5, 2), R.tree(4, 2)], 8, 2, 128, 16, 61)
    for value in (0, 1, 5, 255):
        s.ws.fill_(value)
        s.plan()
        s.run()
        s.check(f"bytes of {value}")
    s.dev["last"][1] = 0
    s.plan()  # left unread
    t = Step([70, 9], [R.tree(6, 2), R.tree(3, 2)], 8, 2, 128, 16, 62)
    t.ws = s.ws if s.ws.numel() >= t.ws.numel() else torch.cat([s.ws, t.ws])
    t.plan()
    t.run()
    t.check("another handle's steps")
    t.h.plan(B.MODE_DECODE, [0, 1, 2], t.kvp.tolist(), t.kvi.tolist(), t.last.tolist(), workspace=t.ws)  # an ordinary decode plan
    torch.cuda.synchronize()
    t.plan()
    t.run()
    t.check("behind a decode plan")
