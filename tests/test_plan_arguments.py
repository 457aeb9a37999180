"""What the plan calls refuse on the host (no GPU): new tokens a decode step cannot have."""
import ctypes

import numpy as np
import pytest

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


@pytest.mark.parametrize("qo,word", [([0, 1, 3], "one new token"), ([0, 0, 1], "one new token"), ([0, 2, 2], "one new token"),
                                     ([1, 2, 3], "start at 0"), ([0, 2, 1], "decreases")])
@pytest.mark.parametrize("mode", [B.MODE_DECODE, B.MODE_DECODE_WEIGHTS])
def test_a_decode_step_has_one_new_token_a_row(mode, qo, word):
    h = make()
    a = [np.array(x, np.int32) for x in (qo, [0, 2, 3], [3, 4, 5], [4, 7])]
    p = [x.ctypes.data_as(ctypes.c_void_p) for x in a]
    st = h.lib.pkv_plan(h.h, mode, *p, 2, 1, -1, 0.0, ctypes.c_void_p(256), 128, None)
    assert st == B.ERR_INVALID and word in h.lib.pkv_last_error(h.h).decode()
    a[0][:] = [0, 1, 2]
    st = h.lib.pkv_plan(h.h, mode, *p, 2, 1, -1, 0.0, ctypes.c_void_p(256), 128, None)
    assert st == B.ERR_WORKSPACE, "nothing else was wrong"
