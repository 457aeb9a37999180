"""Eviction at the lengths where the selection kernel changes its form: a CTA takes 8,192 tokens, a cluster
of 2, 4 or 8 the rows of a plan whose longest cut row is longer, and the scores past 40 a thread (327,680 a
row) are read again instead of kept; rows that are left alone stand beside the cut ones."""
import numpy as np
import pytest
import torch

import evict_ref as E
from paged_kv_attention_gqa_gb300 import binding as B

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def _build():
    from paged_kv_attention_gqa_gb300 import build
    build.build()


def cut(lens, keep, sink, recent, P, kind):
    """One kv head of 64; checks positions, scores and K and V bit for bit."""
    g = np.random.default_rng(len(lens) + lens[0])
    pages = [-(-L // P) for L in lens]
    need = [-(-k // P) if k < L else 0 for k, L in zip(keep, lens)]
    total = sum(pages) + sum(need)
    ids = g.permutation(total).astype(np.int32)
    kvp, dsp = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (pages, need))
    kvi, dst = ids[: kvp[-1]], ids[kvp[-1]:]
    gen = torch.Generator().manual_seed(lens[0])
    scores = torch.rand(total, P, generator=gen)
    if kind == "ties":
        scores = (scores * 4).floor()
    kv = torch.randint(-9, 9, (total, 2, P, 1, 64), generator=gen).to(torch.bfloat16)
    h = B.Handle(num_qo_heads=1, num_kv_heads=1, head_dim=64, page_size=P, max_batch=len(lens), max_num_pages=max(len(kvi), len(dst)),
                 num_cache_pages=total)
    ws = torch.empty(h.workspace_size(B.MODE_EVICT), dtype=torch.uint8, device="cuda")
    h.plan_evict(kvp, kvi, [(L - 1) % P + 1 if L else 0 for L in lens], keep, dsp, dst, num_sink=sink, num_recent=recent, workspace=ws)
    n = sum(min(k, L) for k, L in zip(keep, lens))
    kv_d, scores_d, kept = kv.cuda(), scores.cuda(), torch.full((n + 1,), -7, dtype=torch.int32, device="cuda")
    h.run_evict(kv_d, scores_d, kept[:n], workspace=ws)
    want_kv, want_scores, want = kv.clone(), scores.clone(), []
    for r, L in enumerate(lens):
        mine = torch.as_tensor(kvi[kvp[r]: kvp[r + 1]]).long()
        stay = E.select(scores[mine].reshape(-1)[:L].tolist(), L, keep[r], sink, recent)
        want += stay
        if L > keep[r] and stay:
            j, i = torch.tensor(stay), torch.arange(len(stay))
            to = torch.as_tensor(dst[dsp[r]: dsp[r + 1]]).long()[i // P]
            want_kv[to, :, i % P] = kv[mine[j // P], :, j % P]
            want_scores[to, i % P] = scores[mine[j // P], j % P]
    assert kept[:n].tolist() == want and kept[n] == -7
    assert torch.equal(scores_d.cpu(), want_scores)
    assert torch.equal(kv_d.cpu().view(torch.int16), want_kv.view(torch.int16))


LONGEST = [8192, 8193, 16384, 16385, 32768, 32769, 327680, 327681]


@pytest.mark.parametrize("kind", ["rand", "ties"])
@pytest.mark.parametrize("L", LONGEST)
def test_longest_cut_row(L, kind):
    cut([L], [L // 3], 4, 100, 64, kind)


@pytest.mark.parametrize("L", [8192, 8193, 16385, 32769])
def test_rows_left_alone_beside_the_cut_one(L):
    """Shorter, as long, longer and empty rows that keep all they have."""
    cut([100, L, L, 2 * L + 3, 0, 1], [100, L - 1, L, 2 * L + 3, 5, 7], 1, 3, 32, "rand")


def test_short_rows_share_the_cluster_of_a_long_one():
    cut([3, 20000, 1025, 64, 9000], [2, 100, 1024, 9, 8999], 1, 1, 16, "ties")
