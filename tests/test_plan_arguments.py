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


class Workspace:
    """What the plan calls read of a workspace tensor; nothing is copied to it."""

    def data_ptr(self):
        return 256

    def numel(self):
        return 128

    def element_size(self):
        return 1


# two rows of 2 and 1 pages, three entries, and one new token a row
ROWS = dict(kv_indptr=[0, 2, 3], kv_indices=[3, 4, 5], last_page_len=[4, 7])
SHORT = [(dict(kv_indices=[3, 4]), "kv_indices"), (dict(kv_indices=None), "kv_indices"), (dict(last_page_len=[4]), "last_page_len"),
         (dict(last_page_len=None), "last_page_len"), (dict(kv_indptr=[]), "kv_indptr"), (dict(kv_indptr=None), "kv_indptr")]


def refused(call, kw, word, **args):
    """The lists are checked before the library reads them: an entry that is missing is never read."""
    with pytest.raises(ValueError, match=word):
        call(**{**args, **kw}, workspace=Workspace(), stream=0)
    with pytest.raises(B.PkvError) as e:  # nothing else was wrong
        call(**args, workspace=Workspace(), stream=0)
    assert e.value.status == B.ERR_WORKSPACE


@pytest.mark.parametrize("kw,word", SHORT + [(dict(qo_indptr=[0, 1]), "qo_indptr")])
@pytest.mark.parametrize("mode", [B.MODE_DECODE, B.MODE_PREFILL, B.MODE_DECODE_WEIGHTS, B.MODE_WEIGHTS])
def test_plan_lists_are_long_enough(mode, kw, word):
    refused(make().plan, kw, word, mode=mode, qo_indptr=[0, 1, 2], **ROWS)


@pytest.mark.parametrize("kw,word", SHORT + [(dict(keep=[20]), "keep"), (dict(keep=None), "keep"), (dict(dst_indptr=[0, 2]), "dst_indptr"),
                                             (dict(dst_indptr=None), "dst_indptr"), (dict(dst_indices=[50]), "dst_indices"),
                                             (dict(dst_indices=None), "dst_indices")])
def test_evict_lists_are_long_enough(kw, word):
    args = dict(ROWS, kv_indptr=[0, 3, 4], kv_indices=[3, 4, 5, 6], last_page_len=[4, 7], keep=[20, 20], dst_indptr=[0, 2, 2],
                dst_indices=[50, 51])
    refused(make().plan_evict, kw, word, **args)


def latent():
    return B.LatentHandle(num_heads=16, page_size=16, max_batch=4, max_total_tokens=100, max_num_pages=50, num_cache_pages=60,
                          sm_count=152)


@pytest.mark.parametrize("kw,word", SHORT + [(dict(qo_indptr=[0, 1]), "qo_indptr")])
def test_latent_plan_lists_are_long_enough(kw, word):
    refused(latent().plan, kw, word, qo_indptr=[0, 1, 2], sm_scale=0.1, **ROWS)


@pytest.mark.parametrize("kw,word", [(dict(cu_k=[0, 5]), "cu_k"), (dict(cu_k=None), "cu_k"), (dict(cu_q=None), "cu_q"),
                                     (dict(cu_q=[]), "cu_q")])
def test_dense_plan_lists_are_long_enough(kw, word):
    dense = B.Handle(num_qo_heads=8, num_kv_heads=2, head_dim=64, page_size=16, max_batch=4, max_total_tokens=100,
                     max_num_pages=50, num_cache_pages=60, sm_count=152)
    refused(dense.plan_dense, kw, word, cu_q=[0, 3, 4], cu_k=[0, 5, 9])
    refused(latent().plan_dense, kw, word, cu_q=[0, 3, 4], cu_k=[0, 5, 9], sm_scale=0.1)


def test_lists_may_be_longer_than_the_batch():
    """Arrays kept at their maxima: the entries behind the batch are not looked at."""
    h = make()
    with pytest.raises(B.PkvError) as e:
        h.plan(B.MODE_WEIGHTS, [0, 1, 2, 99, 99], [0, 2, 3], [3, 4, 5, -1, -1], [4, 7, 99], workspace=Workspace(), stream=0)
    assert e.value.status == B.ERR_WORKSPACE
