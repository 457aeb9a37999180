"""What the compiler and the caches may do with the loads of the step's kernels, which start beside the kernel before them
(no GPU: the sources are read)."""
import os
import re

import pytest

from paged_kv_attention_gqa_gb300 import build as B


def source(name):
    with open(os.path.join(B.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["maps.cu", "tree_plan.cu", "tree.cu"])
def test_nothing_is_read_by_the_read_only_path(name):
    """Its loads may be moved before the wait for the earlier kernel, and ask for memory that nobody writes meanwhile; every
    array of the step is written by some kernel of it."""
    text = source(name)
    assert "griddep_wait" in text and "__ldg" not in text and "ld.global.nc" not in text and "__restrict__" not in text


def test_what_the_join_reads_before_its_wait_comes_past_l1():
    """Its record is the plan's, two kernels before; nothing else is read before the wait."""
    body = source("tree.cu").split("tree_join_kernel(const TreeArgs a, int part_rows) {")[1].split("griddep_wait()")[0]
    reads = re.findall(r"[^;{}]*\ba\.(?:joins|rows|starts|nodes|masks|pages|part_o|part_lse)\b[^;]*;", body)
    assert len(reads) == 1 and "__ldcg(" in reads[0], reads
