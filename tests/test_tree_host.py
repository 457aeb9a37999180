"""The speculative step on the host (no GPU): refusals of the C ABI and of the binding, workspace bounds, and the
references of the GPU tests against worked cases.  No call here reaches a launch."""
import ctypes
import types

import pytest
import torch

import tree_ref as R
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


OK = 256  # an aligned address that no refused call reads


def plan(h, **kw):
    a = dict(qo=OK, kvp=OK, kvi=OK, n_idx=10, last=OK, batch=2, parents=OK, tokens=20, most=8, window=-1, scale=0.0, pos=None, ws=OK,
             size=1 << 40)
    a.update(kw)
    st = h.lib.pkv_plan_tree(h.h, a["qo"], a["kvp"], a["kvi"], a["n_idx"], a["last"], a["batch"], a["parents"], a["tokens"], a["most"],
                             a["window"], a["scale"], a["pos"], a["ws"], a["size"], None)
    return st, h.lib.pkv_last_error(h.h).decode()


@pytest.mark.parametrize("kw,status,word", [
    (dict(ws=None), B.ERR_INVALID, "workspace"), (dict(ws=128), B.ERR_INVALID, "aligned"), (dict(batch=-1), B.ERR_INVALID, "batch"),
    (dict(batch=5), B.ERR_INVALID, "max_batch"), (dict(tokens=-1), B.ERR_INVALID, "num_tokens"),
    (dict(tokens=101), B.ERR_INVALID, "max_total_tokens"), (dict(most=0), B.ERR_INVALID, "max_new"),
    (dict(most=257), B.ERR_UNSUPPORTED, "max_new"), (dict(window=-2), B.ERR_INVALID, "window_left"),
    (dict(scale=float("nan")), B.ERR_INVALID, "sm_scale"), (dict(scale=-1.0), B.ERR_INVALID, "sm_scale"),
    (dict(scale=float("inf")), B.ERR_INVALID, "sm_scale"), (dict(n_idx=51), B.ERR_INVALID, "max_num_pages"),
    (dict(n_idx=-1), B.ERR_INVALID, "num_indices"), (dict(qo=None), B.ERR_INVALID, "null"), (dict(kvp=None), B.ERR_INVALID, "null"),
    (dict(kvi=None), B.ERR_INVALID, "null"), (dict(last=None), B.ERR_INVALID, "null"), (dict(qo=258), B.ERR_INVALID, "aligned"),
    (dict(parents=257), B.ERR_INVALID, "aligned"), (dict(pos=2), B.ERR_INVALID, "aligned"), (dict(size=1000), B.ERR_WORKSPACE, "too small"),
])
def test_plan_rejects(kw, status, word):
    st, msg = plan(make(), **kw)
    assert st == status and word in msg, (st, msg)


def test_small_pages_are_refused():
    for P in (1, 2, 4):
        st, msg = plan(make(page_size=P))
        assert st == B.ERR_UNSUPPORTED and "page_size" in msg


def test_runs_without_a_plan_are_refused():
    h = make()
    assert h.lib.pkv_run_tree(h.h, OK, 512, OK, 128, OK, 128, OK, OK, None, OK, None) == B.ERR_NOT_PLANNED
    assert h.lib.pkv_run_accept(h.h, OK, OK, 8, OK, 128, 128, OK, 128, 128, OK, 1 << 20, 1, OK, OK, OK, None, OK, None) == B.ERR_NOT_PLANNED
    assert h.lib.pkv_run_tree(None, *[None] * 1, 0, None, 0, None, 0, None, None, None, None, None) == B.ERR_INVALID
    assert plan(types.SimpleNamespace(lib=types.SimpleNamespace(pkv_plan_tree=h.lib.pkv_plan_tree, pkv_last_error=h.lib.pkv_last_error),
                                      h=None))[0] == B.ERR_INVALID


def maps(h, **kw):
    a = dict(seq=OK, new=OK, batch=2, table=OK, stride=9, blocks=9, held=OK, held_out=4096, free=OK, room=5, count=OK, count_out=OK, qo=OK,
             kvp=OK, kvi=OK, n_idx=9, last=OK, slots=OK, pos=OK, tokens=9, status=OK)
    a.update(kw)
    st = h.lib.pkv_build_maps(h.h, *(a[k] for k in (
        "seq", "new", "batch", "table", "stride", "blocks", "held", "held_out", "free", "room", "count", "count_out", "qo", "kvp", "kvi",
        "n_idx", "last", "slots", "pos", "tokens", "status")), None)
    return st, h.lib.pkv_last_error(h.h).decode()


@pytest.mark.parametrize("kw,word", [
    (dict(batch=5), "max_batch"), (dict(batch=-1), "batch"), (dict(blocks=-1), "capacities"), (dict(room=-1), "capacities"),
    (dict(n_idx=-1), "capacities"), (dict(tokens=-1), "capacities"), (dict(stride=8), "table_stride"), (dict(qo=None), "null"),
    (dict(kvp=None), "null"), (dict(status=None), "null"), (dict(count=None), "null"), (dict(count_out=None), "null"),
    (dict(seq=None), "null"), (dict(new=None), "null"), (dict(held=None), "null"), (dict(held_out=None), "null"), (dict(last=None), "null"),
    (dict(table=None), "null"), (dict(free=None), "null"), (dict(kvi=None), "null"), (dict(seq=257), "aligned"), (dict(slots=258), "aligned"),
    (dict(held_out=OK + 4), "overlap"), (dict(held=OK + 4, held_out=OK), "overlap"),
])
def test_maps_rejects(kw, word):
    st, msg = maps(make(), **kw)
    assert st == B.ERR_INVALID and word in msg, (st, msg)


def test_maps_of_too_many_rows():
    st, msg = maps(make(max_batch=9000), batch=8193, held_out=1 << 20)
    assert st == B.ERR_UNSUPPORTED and "8192" in msg


def test_workspace_sizes():
    a, b = make().workspace_size(B.MODE_TREE), make(max_total_tokens=10000, max_batch=1000).workspace_size(B.MODE_TREE)
    # two partials of 256 rows per CTA, whatever the step's size; a few words per token and row
    assert 2 * 152 * 256 * 65 * 4 <= a < b < a + (1 << 20)


I32, I64, BF, F32, U8 = torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.uint8


def Tensor(dtype, *shape, strides=None):
    """A tensor on the host, whose device index is -1: the fixture makes that the current one."""
    return torch.empty(1 << 20, dtype=dtype).as_strided(shape, strides) if strides else torch.empty(shape, dtype=dtype)


@pytest.fixture
def called(monkeypatch):
    """A handle whose library only counts the calls."""
    calls, back = [], ctypes.CFUNCTYPE(ctypes.c_int)
    h = make()
    h._planned_tokens, h._planned_rows = 5, 2
    B._load_marshal()
    fake = [back(lambda i=i: calls.append(i) or B.OK) for i in range(4)]
    B._marshal.connect(*(ctypes.cast(f, ctypes.c_void_p).value for f in fake))
    h.device = -1
    monkeypatch.setattr(B, "_torch", types.SimpleNamespace(cuda=types.SimpleNamespace(current_device=lambda: h.device)))
    monkeypatch.setattr(B, "_raw_stream", lambda device: 0)
    h.calls = calls
    yield h
    monkeypatch.undo()
    B._load_marshal()


def ints(**kw):
    d = dict(seq=Tensor(I32, 2), new=Tensor(I32, 2), table=Tensor(I32, 2, 9), held=Tensor(I32, 2), free=Tensor(I32, 7),
             count=Tensor(I32, 1), qo=Tensor(I32, 3), kvp=Tensor(I32, 3), kvi=Tensor(I32, 9), last=Tensor(I32, 2),
             slots=Tensor(I32, 5), pos=Tensor(I32, 5), status=Tensor(I32, 1), parents=Tensor(I32, 5), ws=Tensor(U8, 4096))
    d.update(kw)
    return d


def do_maps(h, d):
    h.build_maps(d["seq"], d["new"], d["table"], d["held"], d["free"], d["count"], qo_indptr=d["qo"], kv_indptr=d["kvp"],
                 kv_indices=d["kvi"], last_page_len=d["last"], slots=d["slots"], positions=d["pos"], status=d["status"])


def do_plan(h, d):
    h.plan_tree(d["qo"], d["kvp"], d["kvi"], d["last"], d["parents"], num_tokens=5, max_new=3, positions=d["pos"], workspace=d["ws"])


def do_tree(h, d):
    d = {**dict(q=Tensor(BF, 5, 8, 64), k=Tensor(BF, 5, 2, 64), v=Tensor(BF, 5, 2, 64), kv=Tensor(BF, 60, 2, 16, 2, 64),
                out=Tensor(BF, 5, 8, 64), lse=Tensor(F32, 5, 8)), **d}
    h.run_tree(d["q"], d["k"], d["v"], d["kv"], d["out"], d["lse"], workspace=d["ws"])


def do_accept(h, d):
    d = {**dict(draft=Tensor(I64, 5), target=Tensor(I64, 5), k=Tensor(BF, 3, 5, 2, 64), v=Tensor(BF, 3, 5, 2, 64),
                cache=Tensor(BF, 3, 60, 2, 16, 2, 64), accepted=Tensor(I32, 5), num=Tensor(I32, 2), next=Tensor(I64, 2)), **d}
    h.run_accept(d["draft"], d["target"], d["k"], d["v"], d["cache"], d["accepted"], d["num"], d["next"], d["seq"], workspace=d["ws"])


CALLS = {"maps": do_maps, "plan": do_plan, "tree": do_tree, "accept": do_accept}


@pytest.mark.parametrize("call", sorted(CALLS))
def test_the_binding_passes_good_arguments(called, call):
    CALLS[call](called, ints())
    assert called.calls == [list(CALLS).index(call)]


@pytest.mark.parametrize("call", sorted(CALLS))
def test_tensors_on_another_device_are_refused(called, call):
    called.device = 0
    with pytest.raises(ValueError, match="on the current CUDA device"):
        CALLS[call](called, ints())
    assert not called.calls


def test_a_closed_handle_is_refused(called):
    """Address 0 reaches the library, which refuses it (test_runs_without_a_plan_are_refused)."""
    called.close()
    assert called._address() == 0


WRONG = [
    ("maps", dict(seq=Tensor(I64, 2)), TypeError, "seq_lens"), ("maps", dict(new=Tensor(I32, 3)), ValueError, "new_lens"),
    ("maps", dict(seq=Tensor(I32, 2, 1)), ValueError, "seq_lens"), ("maps", dict(seq=[1, 2]), TypeError, "seq_lens"),
    ("maps", dict(table=Tensor(I32, 18)), ValueError, "block_table"),
    ("maps", dict(table=Tensor(I32, 2, 9, strides=(1, 2))), ValueError, "block_table"),
    ("maps", dict(table=Tensor(I32, 3, 9)), ValueError, "block_table"), ("maps", dict(table=Tensor(I64, 2, 9)), TypeError, "block_table"),
    ("maps", dict(held=Tensor(I32, 3)), ValueError, "num_blocks"), ("maps", dict(free=Tensor(I32, 7, 1)), ValueError, "free_pages"),
    ("maps", dict(count=Tensor(I32, 2)), ValueError, "free_count"), ("maps", dict(qo=Tensor(I32, 2)), ValueError, "qo_indptr"),
    ("maps", dict(kvp=Tensor(I32, 4)), ValueError, "kv_indptr"), ("maps", dict(last=None), TypeError, "last_page_len"),
    ("maps", dict(kvi=Tensor(I32, 9, strides=(2,))), ValueError, "kv_indices"), ("maps", dict(pos=Tensor(I32, 6)), ValueError, "positions"),
    ("maps", dict(slots=Tensor(F32, 5)), TypeError, "slots"), ("maps", dict(status=Tensor(I32, 2)), ValueError, "status"),
    ("plan", dict(parents=Tensor(I32, 4)), ValueError, "parents"), ("plan", dict(parents=Tensor(I64, 5)), TypeError, "parents"),
    ("plan", dict(qo=Tensor(I32, 4)), ValueError, "qo_indptr"), ("plan", dict(last=Tensor(I32, 3)), ValueError, "last_page_len"),
    ("plan", dict(kvp=Tensor(I32, 0), qo=Tensor(I32, 0)), ValueError, "kv_indptr"), ("plan", dict(pos=Tensor(I32, 4)), ValueError, "positions"),
    ("plan", dict(ws=None), TypeError, "workspace"), ("plan", dict(ws=Tensor(U8, 64, strides=(2,))), ValueError, "workspace"),
    ("tree", dict(q=Tensor(F32, 5, 8, 64)), TypeError, "q must"), ("tree", dict(q=Tensor(BF, 4, 8, 64)), ValueError, "q must"),
    ("tree", dict(q=Tensor(BF, 5, 8, 64, strides=(1024, 128, 1))), ValueError, "side by side"),
    ("tree", dict(k=Tensor(BF, 5, 2, 64, strides=(256, 128, 1))), ValueError, "side by side"),
    ("tree", dict(v=Tensor(BF, 5, 2, 64, strides=(256, 64, 2))), ValueError, "side by side"),
    ("tree", dict(out=Tensor(BF, 5, 8, 64, strides=(1024, 64, 1))), ValueError, "out"), ("tree", dict(lse=Tensor(BF, 5, 8)), TypeError, "lse"),
    ("tree", dict(kv=Tensor(BF, 61, 2, 16, 2, 64)), ValueError, "kv_layer"), ("tree", dict(k=None), TypeError, "k_new"),
    ("accept", dict(draft=Tensor(F32, 5)), TypeError, "draft_tokens"), ("accept", dict(target=Tensor(I32, 5)), TypeError, "target_tokens"),
    ("accept", dict(next=Tensor(I32, 2)), TypeError, "next_tokens"), ("accept", dict(num=Tensor(I32, 3)), ValueError, "num_accepted"),
    ("accept", dict(seq=Tensor(I32, 3)), ValueError, "seq_lens"), ("accept", dict(k=Tensor(BF, 2, 5, 2, 64)), ValueError, "k_new"),
    ("accept", dict(cache=Tensor(BF, 3, 60, 2, 8, 2, 64)), ValueError, "kv_cache"), ("accept", dict(cache=Tensor(BF, 60, 2, 16, 2, 64)), ValueError, "kv_cache"),
    ("accept", dict(cache=Tensor(BF, 1, 60, 2, 16, 2, 64, strides=(0, 4096, 2048, 64, 1024, 1)), k=Tensor(BF, 1, 5, 2, 64), v=Tensor(BF, 1, 5, 2, 64)), ValueError, "contiguous layers"),
    ("accept", dict(accepted=Tensor(I64, 5)), TypeError, "accepted"), ("accept", dict(ws=7), TypeError, "workspace"),
]


@pytest.mark.parametrize("call,kw,error,word", WRONG, ids=[f"{i}-{w[0]}-{w[3].split()[0]}" for i, w in enumerate(WRONG)])
def test_the_binding_refuses(called, call, kw, error, word):
    with pytest.raises(error, match=word):
        CALLS[call](called, ints(**kw))
    assert not called.calls


def test_reference_trees():
    up, depth = R.ancestors([-1, 0, 0, 2, -1, 4])
    assert depth.tolist() == [0, 1, 1, 2, 0, 1]
    assert up.long().tolist() == [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 0, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0], [0, 0, 0, 0, 1, 0],
                                  [0, 0, 0, 0, 1, 1]]
    assert R.visible(2, [-1, 0], 1).long().tolist() == [[0, 1, 1, 0], [0, 0, 1, 1]]
    o, z, _, _ = R.attend(torch.zeros(1, 2, 4), torch.ones(3, 1, 4), torch.tensor([1.0, 2, 6]).view(3, 1, 1).expand(-1, -1, 4),
                          torch.tensor([[True, False, True]]), 1.0)
    assert torch.allclose(o, torch.full_like(o, 3.5)) and torch.allclose(z, torch.full_like(z, 2.0).log())


def test_reference_accept():
    assert R.accept([-1, 0, 0, 1, 2], [0, 7, 7, 8, 9], [7, 8, 9, 5, 5]) == ([0, 1, 3], 5)
    assert R.accept([-1, -1], [3, 4], [4, 3]) == ([0], 4)
    assert R.accept([], [], []) == ([], -1)


def test_reference_maps():
    m = R.maps([0, 10, 5], [0, 20, 10], [[1, 2, 3, -9, -9], [4, -9, -9, -9, -9], [5, -9, -9, -9, -9]], [3, 1, 1], [7, 8, 0, 0, 0, 0], 2, 8,
               [-1] * 9, 31)
    assert m["free"][:5] == [7, 8, 1, 2, 3] and m["count"] == 1
    assert m["table"][1] == [4, 3, 2, 1, -9] and m["table"][2] == [5, 8, -9, -9, -9]
    assert m["kvi"] == [4, 3, 2, 1, 5, 8, -1, -1, -1] and m["kvp"] == [0, 0, 4, 6] and m["qo"] == [0, 0, 20, 30]
    assert m["slots"][:7] == [3 * 8 + 2 + i for i in range(6)] + [2 * 8]
    assert m["positions"][:2] == [10, 11] and m["last"] == [0, 6, 7] and m["slots"][-1] == -1
