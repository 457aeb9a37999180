"""A plan whose host buffers cannot be had says so (no GPU): run in a process of its own, whose memory is
limited before the call."""
import os
import subprocess
import sys

from paged_kv_attention_gqa_gb300 import build as pkv_build

CODE = r"""
import ctypes, resource
import numpy as np
from paged_kv_attention_gqa_gb300 import binding as B

rows = 100_000_000
h = B.LatentHandle(num_heads=16, page_size=16, max_batch=rows, max_total_tokens=100, max_num_pages=50, num_cache_pages=60,
                   sm_count=152)
one = np.zeros(2, np.int32).ctypes.data_as(ctypes.c_void_p)
plan = lambda batch, scale: h.lib.pkv_latent_plan(h.h, None, one, one, one, batch, 1, -1, scale, ctypes.c_void_p(256), 1 << 30, None)
assert plan(1, -1.0) == B.ERR_INVALID  # an earlier failure, whose text must not stay
assert b"sm_scale" in h.lib.pkv_latent_last_error(h.h)
with open("/proc/self/statm") as f:
    used = int(f.read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (64 << 20), resource.RLIM_INFINITY))
st = plan(rows, 0.1)  # its list of rows is 400 MB, built before the caller's arrays are read
print(st, h.lib.pkv_latent_last_error(h.h).decode())
"""


def test_a_plan_that_runs_out_of_memory_says_so():
    pkv_build.build()
    out = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=120,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert out.returncode == 0, out.stderr
    status, text = out.stdout.strip().split(" ", 1)
    assert int(status) == 1 and "bad_alloc" in text, out.stdout
