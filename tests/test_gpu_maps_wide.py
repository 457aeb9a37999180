"""Maps whose sums are taken in 64 bits: tables of 2^30 tokens and more, against the definition, and the border
between the two forms."""
import numpy as np
import pytest
import torch

from paged_kv_attention_gqa_gb300 import binding as B
from test_gpu_step import Maps, full
from test_gpu_tree import i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def _build():
    from paged_kv_attention_gqa_gb300 import build
    build.build()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows", [1023, 1024, 1100])
def test_short_rows_of_a_wide_table(rows, in_place):
    """1,024 blocks of 1,024 tokens a row: 1,023 rows are summed in 32 bits, 1,024 in 64."""
    g = np.random.default_rng(rows)
    seq = g.integers(0, 2500, rows)
    seq = np.where(g.random(rows) < 0.1, 0, seq)
    new = np.where(g.random(rows) < 0.2, 0, g.integers(0, 1500, rows))
    held = -(-seq // 1024) + g.integers(0, 3, rows)
    Maps(seq.tolist(), new.tolist(), held.tolist(), 1024, rows, width=1024).check(in_place=in_place)


def refused(new, free, P=1024, blocks=1024, tokens=None):
    """The status of rows without pages that get these new tokens, and whether the step is empty and nothing has changed."""
    n, pages = len(new), int(sum(-(-x // P) for x in new))
    h = B.Handle(num_qo_heads=1, num_kv_heads=1, head_dim=64, page_size=P, max_batch=n, max_num_pages=1, num_cache_pages=1)
    table, held, stack, count = full(n * blocks).view(n, blocks), full(n, 0), i32(np.arange(free + 1)), full(1, free)
    qo, kvp, kvi, last, status = full(n + 1), full(n + 1), full(pages), full(n), full(1, -9)
    slots = None if tokens is None else full(tokens, -4)
    h.build_maps(full(n, 0), i32(new), table, held, stack, count, qo_indptr=qo, kv_indptr=kvp, kv_indices=kvi, last_page_len=last,
                 slots=slots, status=status)
    torch.cuda.synchronize()
    assert not qo.any() and not kvp.any() and not last.any() and not held.any() and count.item() == free
    assert (table == -1).all() and (kvi == -1).all() and stack.tolist() == list(range(free + 1))
    assert slots is None or (slots == -1).all()
    return status.item()


def test_sums_past_32_bits_are_refused():
    """Pages are short in all of these; sums that 32-bit entries cannot hold are refused before that.  (The kernel steps
    up to 4,096 entries past the last one in 32 bits, so the border lies that much lower.)"""
    row, most = 1 << 20, (1 << 31) - 1 - 4096
    fits = [row] * 2047 + [most - 2047 * row]
    assert refused(fits, 5) == 2047 * 1024 + -(-fits[-1] // 1024) - 5
    assert refused(fits[:-1] + [fits[-1] + 1], 5) == -2
    assert refused([row] * 2048, 5) == -2  # 2^31
    assert refused([row] * 4096, 5) == -2  # 2^32: 0 in 32 bits
    assert refused([row] * 4096 + [1], 5) == -2
    assert refused([row] * 4096 + [3], 5, tokens=7) == -2
    assert refused([row] * 1024, 5) == 1024 * 1024 - 5
    assert refused([row] * 1023, 5) == 1023 * 1024 - 5  # in 32 bits
