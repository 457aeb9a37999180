"""A captured speculative step needs one uncaptured step before it, of any size: which kernels a size chooses is the
library's affair.  In processes of their own, since a kernel's limits are raised once a process."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = r"""
import sys
sys.path[:0] = [".", "tests"]
import torch
import tree_ref as R
from test_gpu_step import Loop

D, H, small, large, rows = (int(x) for x in sys.argv[1:])


big = Loop([130, 40] + [0] * (rows - 2), H, 2, D, 16, 1, 60, 7, large)
# the uncaptured step: the handle of the captured one, few drafted tokens, two rows and a short page list
few = Loop([130, 40], H, 2, D, 16, 1, 15, 8, small)
few.h, few.ws = big.h, big.ws
few.cache = torch.zeros_like(big.cache)
few.d["cache"] = few.cache.cuda()
few.feed([R.tree(small, 2), R.tree(1, 1)], 3)
few.step()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    big.step()
for i in range(2):
    big.feed([R.tree(large - 5 * i, 3), R.tree(large // 2, 2, 1)] + [[]] * (rows - 2), 60 + i)
    graph.replay()
    torch.cuda.synchronize()
    big.mirror()
print("captured")
"""


MAPS = r"""
import sys
sys.path[:0] = [".", "tests"]
import torch
from paged_kv_attention_gqa_gb300 import binding as B
from test_gpu_step import full

h = B.Handle(num_qo_heads=1, num_kv_heads=1, head_dim=64, page_size=1024, max_batch=2500, max_num_pages=1, num_cache_pages=1)


class Rows:
    def __init__(self, rows, blocks):
        self.d = dict(seq=full(rows, 5), new=torch.arange(rows, dtype=torch.int32, device="cuda") % 9, table=full(rows * blocks).view(rows, blocks),
                      held=full(rows, 0), free=torch.arange(rows + 3, dtype=torch.int32, device="cuda"), count=full(1, rows + 2),
                      qo=full(rows + 1), kvp=full(rows + 1), kvi=full(rows), last=full(rows), slots=full(9 * rows), status=full(1, -9))

    def step(self):
        d = self.d
        h.build_maps(d["seq"], d["new"], d["table"], d["held"], d["free"], d["count"], qo_indptr=d["qo"], kv_indptr=d["kvp"],
                     kv_indices=d["kvi"], last_page_len=d["last"], slots=d["slots"], status=d["status"])


few, many = Rows(2, 4), Rows(2500, 1024)
few.step()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    many.step()
graph.replay()
once = Rows(2500, 1024)
once.step()
torch.cuda.synchronize()
assert once.d["status"].item() == 0 and once.d["held"].eq(1).all()
for k in once.d:
    assert torch.equal(many.d[k], once.d[k]), k
print("captured")
"""


def run(code, *args):
    from paged_kv_attention_gqa_gb300 import build
    build.build()
    out = subprocess.run([sys.executable, "-c", code, *map(str, args)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip().endswith("captured"), out.stderr[-3000:]


# two query tiles behind one (group 8), cut units behind whole ones, maps of 2,500 rows behind those of two
@pytest.mark.parametrize("D,H,small,large,rows", [(128, 16, 3, 40, 2), (64, 16, 3, 40, 2), (256, 8, 2, 30, 2), (64, 4, 2, 9, 2500)])
def test_the_uncaptured_step_may_be_of_another_size(D, H, small, large, rows):
    run(CODE, D, H, small, large, rows)


def test_the_uncaptured_maps_may_be_of_another_size():
    """2,500 rows of 2^20 tokens, whose sums are taken in 64 bits and whose offsets need more than 48 KB of shared memory,
    behind two short ones."""
    run(MAPS)


CUT = r"""
import sys
sys.path[:0] = [".", "tests"]
import torch
from test_gpu_step import Loop, trees_of

D, H, most = (int(x) for x in sys.argv[1:])
loop = Loop([3000, 700, 1500], H, 2, D, 16, 1, 230, 17, most)
saved = {k: v.clone() for k, v in loop.d.items()}
loop.step()
torch.cuda.synchronize()
for k, v in saved.items():
    loop.d[k].copy_(v)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    loop.step()
for i in range(4):
    loop.feed(trees_of(i + 1, 3, most), 80 + 5 * i)
    graph.replay()
    torch.cuda.synchronize()
    loop.mirror()
print("captured")
"""


@pytest.mark.parametrize("D,H,most", [(64, 4, 9), (128, 8, 70), (256, 4, 20)])
def test_replayed_steps_cut_their_units_elsewhere(D, H, most):
    """Long rows whose trees change from replay to replay, and with them the join's records."""
    run(CUT, D, H, most)
