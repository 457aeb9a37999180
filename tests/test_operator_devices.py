"""Calls with a workspace on another device than the current one are refused (no GPU: tensors are stand-ins that
say where they are, the library one that counts its calls)."""
import types

import pytest

from paged_kv_attention_gqa_gb300 import binding as B
from paged_kv_attention_gqa_gb300 import build as pkv_build


class Tensor:
    def __init__(self, dtype, *shape, device=1):
        self.dtype, self.shape, self.device = dtype, shape, device

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def stride(self, dim):
        n = 1
        for x in self.shape[dim + 1:]:
            n *= x
        return n


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or B.OK


@pytest.fixture
def calls(monkeypatch):
    pkv_build.build()
    torch = types.SimpleNamespace(bfloat16="bf16", float32="fp32", int32="i32", uint8="u8",
                                  cuda=types.SimpleNamespace(current_device=lambda: 1))
    monkeypatch.setattr(B, "_torch", torch)
    monkeypatch.setattr(B, "_raw_stream", lambda device: 0)
    bf, f32 = "bf16", "fp32"
    h = B.Handle(num_qo_heads=4, num_kv_heads=2, head_dim=64, page_size=16, max_batch=4, max_total_tokens=8, max_num_pages=5,
                 num_cache_pages=6, sm_count=152)
    m = B.LatentHandle(num_heads=4, page_size=16, max_batch=4, max_total_tokens=8, max_num_pages=5, num_cache_pages=6, sm_count=152)
    h._planned_tokens, h._kept, m._tokens, m._keys = 3, 7, 3, 5
    kv, scores = Tensor(bf, 6, 2, 16, 2, 64), Tensor(f32, 6, 16)
    q, lse = Tensor(bf, 3, 4, 64), Tensor(f32, 3, 4)
    cache = Tensor(bf, 6, 16, 576)
    made = {
        "run_decode_weights": lambda ws: h.run_decode_weights(q, kv, q, lse, scores, workspace=ws),
        "run_weights": lambda ws: h.run_weights(q, lse, kv, scores, workspace=ws),
        "run_evict": lambda ws: h.run_evict(kv, scores, Tensor("i32", 7), workspace=ws),
        "append_planned": lambda ws: m.append_planned(Tensor(bf, 3, 512), Tensor(bf, 3, 64), cache, workspace=ws),
        "run": lambda ws: m.run(Tensor(bf, 3, 4, 576), cache, Tensor(bf, 3, 4, 512), workspace=ws),
        "run_dense": lambda ws: m.run_dense(Tensor(bf, 3, 4, 192), Tensor(bf, 5, 4, 128), Tensor(bf, 5, 64), Tensor(bf, 5, 4, 128),
                                            Tensor(bf, 3, 4, 128), workspace=ws),
    }
    lib = Library()
    close = (h.lib, m.lib)
    h.lib = m.lib = lib
    yield made, lib
    h.lib, m.lib = close


NAMES = ["run_decode_weights", "run_weights", "run_evict", "append_planned", "run", "run_dense"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("device", [0, 2, -1])
def test_a_workspace_elsewhere_is_refused(calls, name, device):
    made, lib = calls
    with pytest.raises(ValueError, match="workspace must be on the current CUDA device"):
        made[name](Tensor("u8", 4096, device=device))
    assert not lib.calls
    made[name](Tensor("u8", 4096, device=1))
    assert len(lib.calls) == 1
