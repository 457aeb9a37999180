"""ctypes binding of libpkv (include/pkv.h).  Argument marshalling only: every step of
the attention path runs in the library's CUDA kernels.  torch tensors are passed as
device pointers; the stream is torch's current CUDA stream unless one is given.

``load()`` raises if libpkv.so has not been built; nothing here falls back to another
implementation.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpkv.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_TOO_MANY_PREFILL_ROWS, ERR_NOT_PLANNED, ERR_CUDA, ERR_DEVICE = range(8)
MODE_DECODE, MODE_PREFILL, MODE_MIXED, MODE_DENSE = 0, 1, 2, 3
MODE_EVICT, MODE_DECODE_WEIGHTS, MODE_WEIGHTS = 4, 5, 6
NON_CAUSAL, CAUSAL, CONTEXT_ONLY = 0, 1, 2
STATUS_NAMES = ["OK", "INVALID", "UNSUPPORTED", "WORKSPACE", "TOO_MANY_PREFILL_ROWS", "NOT_PLANNED", "CUDA", "DEVICE"]

# every symbol include/pkv.h declares
EXPORTS = ["pkv_create", "pkv_destroy", "pkv_last_error", "pkv_workspace_size", "pkv_plan", "pkv_kv_append", "pkv_kv_append_planned",
           "pkv_run_decode", "pkv_run_prefill", "pkv_run_mixed", "pkv_check_device_error", "pkv_append_slots",
           "pkv_mixed_layout", "pkv_decode_split", "pkv_decode_head_rows", "pkv_run_decode_static", "pkv_context_only_views",
           "pkv_plan_dense", "pkv_run_dense", "pkv_gather_kv", "pkv_run_decode_append", "pkv_selftest_wait_timeout",
           "pkv_run_decode_weights", "pkv_run_weights", "pkv_plan_evict", "pkv_run_evict", "pkv_latent_create", "pkv_latent_destroy", "pkv_latent_last_error", "pkv_latent_workspace_size",
           "pkv_latent_plan", "pkv_latent_append_planned", "pkv_latent_run", "pkv_latent_plan_dense",
           "pkv_latent_run_dense", "pkv_latent_check_device_error"]


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"pkv status {name}: {message}")


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_qo_heads", "num_kv_heads", "head_dim", "page_size", "max_batch", "max_total_tokens",
        "max_num_pages", "num_cache_pages", "max_prefill_rows", "sm_count", "sink_page", "graph_static",
        "enable_nvtx")]


class LatentConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_heads", "latent_dim", "rope_dim", "nope_dim", "v_dim", "page_size", "max_batch", "max_total_tokens",
        "max_num_pages", "num_cache_pages", "sm_count", "enable_nvtx")]


_lib = None


def load(path: str = LIB_PATH):
    """Open libpkv.so (built by paged_kv_attention_gqa_gb300.build); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with `python -m paged_kv_attention_gqa_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i, i32p, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64
    sig = {
        "pkv_create": ([ctypes.POINTER(Config), ctypes.POINTER(vp)], i),
        "pkv_destroy": ([vp], None),
        "pkv_last_error": ([vp], ctypes.c_char_p),
        "pkv_workspace_size": ([vp, i, ctypes.POINTER(ctypes.c_size_t)], i),
        "pkv_plan": ([vp, i, i32p, i32p, i32p, i32p, i, i, i, ctypes.c_float, vp, ctypes.c_size_t, vp], i),
        "pkv_kv_append": ([vp, vp, vp, i, vp, vp, vp, vp, vp, i, vp], i),
        "pkv_kv_append_planned": ([vp, vp, vp, vp, vp, vp], i),
        "pkv_run_decode": ([vp, vp, vp, vp, vp, vp, vp], i),
        "pkv_run_decode_append": ([vp, vp, vp, vp, vp, vp, vp, vp, vp], i),
        "pkv_selftest_wait_timeout": ([vp, vp, i, vp], i),
        "pkv_run_prefill": ([vp, vp, vp, vp, vp, vp, vp], i),
        "pkv_run_mixed": ([vp, vp, vp, vp, vp, vp, vp], i),
        "pkv_check_device_error": ([vp, vp, vp, ctypes.POINTER(i)], i),
        "pkv_append_slots": ([i, i32p, i32p, i32p, i32p, i, i32p, i32p], i),
        "pkv_mixed_layout": ([i32p, i32p, i32p, i32p, i, i, i] + [i32p] * 9 + [ctypes.POINTER(i)], i),
        "pkv_decode_split": ([vp, i32p, i32p, i, i, i32p, ctypes.POINTER(i), ctypes.POINTER(i)], i),
        "pkv_decode_head_rows": ([vp, i32p, i32p, i32p, i, i, i32p, ctypes.POINTER(i)], i),
        "pkv_run_decode_static": ([vp, vp, vp, vp, vp, i32p, i32p, i32p, i, i, ctypes.c_float, vp], i),
        "pkv_context_only_views": ([i, i32p, i32p, i32p, i32p, i, i32p, i32p, i32p, ctypes.POINTER(i)], i),
        "pkv_plan_dense": ([vp, i32p, i32p, i, i, i, ctypes.c_float, vp, ctypes.c_size_t, vp], i),
        "pkv_run_dense": ([vp, vp, vp, vp, vp, vp, vp, vp], i),
        "pkv_gather_kv": ([vp, vp, vp, i, vp, vp, vp], i),
        "pkv_run_decode_weights": ([vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp], i),
        "pkv_run_weights": ([vp, vp, vp, vp, vp, ctypes.c_float, vp, vp], i),
        "pkv_plan_evict": ([vp, i32p, i32p, i32p, i, i32p, i, i, i32p, i32p, vp, ctypes.c_size_t, vp], i),
        "pkv_run_evict": ([vp, vp, vp, vp, vp, vp], i),
        "pkv_latent_create": ([ctypes.POINTER(LatentConfig), ctypes.POINTER(vp)], i),
        "pkv_latent_destroy": ([vp], None),
        "pkv_latent_last_error": ([vp], ctypes.c_char_p),
        "pkv_latent_workspace_size": ([vp, i, ctypes.POINTER(ctypes.c_size_t)], i),
        "pkv_latent_plan": ([vp, i32p, i32p, i32p, i32p, i, i, i, ctypes.c_float, vp, ctypes.c_size_t, vp], i),
        "pkv_latent_append_planned": ([vp, vp, i64, vp, i64, vp, vp, vp], i),
        "pkv_latent_run": ([vp, vp, vp, vp, vp, vp, vp], i),
        "pkv_latent_plan_dense": ([vp, i32p, i32p, i, i, i, ctypes.c_float, vp, ctypes.c_size_t, vp], i),
        "pkv_latent_run_dense": ([vp, vp, vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, vp], i),
        "pkv_latent_check_device_error": ([vp, vp, vp, ctypes.POINTER(i)], i),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _i32(a):
    if a is None:
        return None
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _need(name, a, entries):
    """The library takes the lengths of its host lists on trust: they are checked here (longer is fine)."""
    if entries > 0 and (a is None or a.size < entries):
        raise ValueError(f"{name} needs {entries} entries, has {0 if a is None else a.size}")


def _paged_lists(qo_indptr, kv_indptr, kv_indices, last_page_len):
    """The index arrays of a paged plan as int32 and its number of rows."""
    qo, kvp, kvi, lpl = _i32(qo_indptr), _i32(kv_indptr), _i32(kv_indices), _i32(last_page_len)
    _need("kv_indptr", kvp, 1)
    batch = len(kvp) - 1
    if kvi is None or lpl is None or len(kvi) < kvp[-1] or len(lpl) < batch:
        _need("kv_indices", kvi, kvp[-1])
        _need("last_page_len", lpl, batch)
    if qo is not None:
        _need("qo_indptr", qo, batch + 1)
    return [qo, kvp, kvi, lpl], batch


def _dense_lists(cu_q, cu_k):
    cq, ck = _i32(cu_q), _i32(cu_k)
    _need("cu_q", cq, 1)
    _need("cu_k", ck, cq.size)
    return cq, ck, cq.size - 1


def _p(a):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def _dptr(t):
    """Device pointer of a torch tensor (or None), as the integer that ctypes takes for a void *."""
    return None if t is None else t.data_ptr()


_torch = None       # torch, imported by the first call that needs it
_raw_stream = None  # the current stream of a device as an integer


def _load_torch():
    global _torch, _raw_stream
    import torch
    _torch = torch
    # torch.cuda.current_stream() builds a Stream object (3 us); the integer alone takes 0.2 us
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    return torch


def _stream(stream):
    if stream is None:
        torch = _torch or _load_torch()
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_tensor(name, t, dtype, shape, device, contiguous=True):
    """The operators that take tensors' shapes on trust in C check them here: type, shape, device (the
    current one, by its index) and layout."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and (not contiguous or t.is_contiguous()):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current CUDA device, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _workspace(ws, device):
    """Pointer of the workspace of a call whose kernels run on `device`."""
    if ws.get_device() != device:
        raise ValueError(f"workspace must be on the current CUDA device, is on {ws.device}")
    return ws.data_ptr()


def _stride(t, dim, least):
    """Stride of one dimension in elements; of a dimension of one entry, which is never stepped, the least."""
    return t.stride(dim) if t.shape[dim] > 1 else least


class Handle:
    """One pkv handle: static shape and the last plan (see include/pkv.h)."""

    def __init__(self, *, num_qo_heads, num_kv_heads, head_dim, page_size, max_batch, max_total_tokens=0,
                 max_num_pages, num_cache_pages, max_prefill_rows=0, sm_count=0, sink_page=-1, graph_static=0,
                 enable_nvtx=False):
        self.lib = load()
        self.cfg = Config(num_qo_heads, num_kv_heads, head_dim, page_size, max_batch, max_total_tokens,
                          max_num_pages, num_cache_pages, max_prefill_rows, sm_count, sink_page, int(graph_static),
                          int(enable_nvtx))
        h = ctypes.c_void_p()
        st = self.lib.pkv_create(ctypes.byref(self.cfg), ctypes.byref(h))
        if st != OK:
            raise PkvError(st, self.lib.pkv_last_error(None).decode())
        self.h = h
        self._keep = []
        self._planned_tokens = self._kept = 0

    def close(self):
        if getattr(self, "h", None):
            self.lib.pkv_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, st):
        if st != OK:
            raise PkvError(st, self.lib.pkv_last_error(self.h).decode())

    def workspace_size(self, mode: int) -> int:
        n = ctypes.c_size_t()
        self._check(self.lib.pkv_workspace_size(self.h, mode, ctypes.byref(n)))
        return n.value

    def plan(self, mode, qo_indptr, kv_indptr, kv_indices, last_page_len, *, workspace, causal=True,
             window_left=-1, sm_scale=0.0, stream=None):
        arrs, batch = _paged_lists(qo_indptr, kv_indptr, kv_indices, last_page_len)
        self._keep = arrs  # host arrays are read synchronously; kept only for symmetry
        st = self.lib.pkv_plan(self.h, mode, *(_p(a) for a in arrs), batch,
                               int(causal) if causal == CONTEXT_ONLY else int(bool(causal)), int(window_left),
                               float(sm_scale), _dptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream))
        self._check(st)
        self._planned_tokens = batch if arrs[0] is None else arrs[0].item(batch)

    def kv_append(self, k, v, num_new_tokens, kv_layer, qo_indptr, kv_indptr, kv_indices, last_page_len, batch,
                  stream=None):
        """pkv_kv_append: k / v, the layer slice and the four index arrays are device
        tensors (qo_indptr may be None: one new token per row)."""
        self._check(self.lib.pkv_kv_append(self.h, _dptr(k), _dptr(v), int(num_new_tokens), _dptr(kv_layer),
                                           _dptr(qo_indptr), _dptr(kv_indptr), _dptr(kv_indices),
                                           _dptr(last_page_len), int(batch), _stream(stream)))

    def kv_append_planned(self, k, v, kv_layer, *, workspace, stream=None):
        """pkv_kv_append_planned: at the write locations of the last plan on `workspace`."""
        self._check(self.lib.pkv_kv_append_planned(self.h, _dptr(k), _dptr(v), _dptr(kv_layer), _dptr(workspace),
                                                   _stream(stream)))

    def _run(self, fn, q, kv_layer, out, lse, workspace, stream):
        self._check(fn(self.h, _dptr(q), _dptr(kv_layer), _dptr(out), _dptr(lse), _dptr(workspace), _stream(stream)))

    def run_decode(self, q, kv_layer, out, lse=None, *, workspace, stream=None):
        self._run(self.lib.pkv_run_decode, q, kv_layer, out, lse, workspace, stream)

    def run_decode_append(self, q, k, v, kv_layer, out, lse=None, *, workspace, stream=None):
        """kv_append + run_decode in one launch (decode plans)."""
        self._check(self.lib.pkv_run_decode_append(self.h, _dptr(q), _dptr(k), _dptr(v), _dptr(kv_layer), _dptr(out),
                                                    _dptr(lse), _dptr(workspace), _stream(stream)))

    def run_prefill(self, q, kv_layer, out, lse=None, *, workspace, stream=None):
        self._run(self.lib.pkv_run_prefill, q, kv_layer, out, lse, workspace, stream)

    def run_mixed(self, q, kv_layer, out, lse=None, *, workspace, stream=None):
        self._run(self.lib.pkv_run_mixed, q, kv_layer, out, lse, workspace, stream)

    def plan_dense(self, cu_q, cu_k, *, workspace, causal=True, window_left=-1, sm_scale=0.0, stream=None):
        cq, ck, batch = _dense_lists(cu_q, cu_k)
        self._check(self.lib.pkv_plan_dense(self.h, _p(cq), _p(ck), batch, int(bool(causal)), int(window_left),
                                            float(sm_scale), _dptr(workspace),
                                            workspace.numel() * workspace.element_size(), _stream(stream)))

    def run_dense(self, q, k, v, out, lse=None, *, workspace, stream=None):
        self._check(self.lib.pkv_run_dense(self.h, _dptr(q), _dptr(k), _dptr(v), _dptr(out), _dptr(lse),
                                           _dptr(workspace), _stream(stream)))

    def _check_layer(self, kv_layer, scores):
        """Checks the slices; returns torch and the current device."""
        torch, c = _torch or _load_torch(), self.cfg
        device = torch.cuda.current_device()
        _check_tensor("kv_layer", kv_layer, torch.bfloat16,
                      (c.num_cache_pages, 2, c.page_size, c.num_kv_heads, c.head_dim), device)
        _check_tensor("scores", scores, torch.float32, (c.num_cache_pages, c.page_size), device)
        return torch, device

    def _check_q(self, q, lse, torch, device):
        tokens, heads = self._planned_tokens, self.cfg.num_qo_heads
        _check_tensor("q", q, torch.bfloat16, (tokens, heads, self.cfg.head_dim), device)
        _check_tensor("lse", lse, torch.float32, (tokens, heads), device)

    def run_decode_weights(self, q, kv_layer, out, lse, scores, *, decay=1.0, workspace, stream=None):
        """run_decode of a MODE_DECODE_WEIGHTS plan that also adds every key's softmax weight, summed over
        the query heads, into scores [pages, page_size] (fp32): decay * old + new, the row's newest
        token from nothing."""
        torch, device = self._check_layer(kv_layer, scores)
        self._check_q(q, lse, torch, device)
        _check_tensor("out", out, torch.bfloat16, q.shape, device)
        self._check(self.lib.pkv_run_decode_weights(
            self.h, q.data_ptr(), kv_layer.data_ptr(), out.data_ptr(), lse.data_ptr(), scores.data_ptr(), decay,
            _workspace(workspace, device), _raw_stream(device) if stream is None else _stream(stream)))

    def run_weights(self, q, lse, kv_layer, scores, *, decay=1.0, workspace, stream=None):
        """The same scores from the queries and the lse of a prefill (MODE_WEIGHTS plans)."""
        torch, device = self._check_layer(kv_layer, scores)
        self._check_q(q, lse, torch, device)
        self._check(self.lib.pkv_run_weights(
            self.h, q.data_ptr(), lse.data_ptr(), kv_layer.data_ptr(), scores.data_ptr(), decay, _workspace(workspace, device),
            _raw_stream(device) if stream is None else _stream(stream)))

    def plan_evict(self, kv_indptr, kv_indices, last_page_len, keep, dst_indptr, dst_indices, *, num_sink=0,
                   num_recent=0, workspace, stream=None):
        """Row r keeps keep[r] tokens if it has more: the first num_sink, the last num_recent and the
        best-scored between; they move to the new pages dst_indices[dst_indptr[r]:dst_indptr[r + 1]]."""
        lists, batch = _paged_lists(None, kv_indptr, kv_indices, last_page_len)
        a = lists[1:] + [_i32(x) for x in (keep, dst_indptr, dst_indices)]
        _need("keep", a[3], batch)
        _need("dst_indptr", a[4], batch + 1)
        _need("dst_indices", a[5], a[4].item(batch))
        if len(a[3]) != batch or len(a[4]) != batch + 1:
            raise ValueError("keep has one entry per row, dst_indptr one more")
        self._check(self.lib.pkv_plan_evict(self.h, _p(a[0]), _p(a[1]), _p(a[2]), batch, _p(a[3]), int(num_sink),
                                            int(num_recent), _p(a[4]), _p(a[5]), _dptr(workspace),
                                            workspace.numel() * workspace.element_size(), _stream(stream)))
        pages = np.diff(a[0])
        lens = np.where(pages > 0, (pages - 1) * self.cfg.page_size + a[2][:batch], 0)
        self._kept = int(np.minimum(lens, a[3]).sum())

    def run_evict(self, kv_layer, scores, kept, *, workspace, stream=None):
        """Move the kept tokens of one layer; kept (int32) receives their positions, row after row."""
        torch, device = self._check_layer(kv_layer, scores)
        _check_tensor("kept", kept, torch.int32, (self._kept,), device)
        self._check(self.lib.pkv_run_evict(
            self.h, kv_layer.data_ptr(), scores.data_ptr(), kept.data_ptr(), _workspace(workspace, device),
            _raw_stream(device) if stream is None else _stream(stream)))

    def gather_kv(self, kv_layer, pages, num_tokens, k_out, v_out, stream=None):
        """pages: a device int32 tensor of page ids."""
        self._check(self.lib.pkv_gather_kv(self.h, _dptr(kv_layer), _dptr(pages), int(num_tokens), _dptr(k_out),
                                           _dptr(v_out), _stream(stream)))

    def selftest_wait_timeout(self, workspace, polls=1000, stream=None):
        """Make one device wait give up (see pkv.h); check_device_error then reports code 4."""
        self._check(self.lib.pkv_selftest_wait_timeout(self.h, _dptr(workspace), int(polls), _stream(stream)))

    def check_device_error(self, workspace, stream=None) -> int:
        code = ctypes.c_int()
        st = self.lib.pkv_check_device_error(self.h, _dptr(workspace), _stream(stream), ctypes.byref(code))
        if st not in (OK, ERR_DEVICE):
            self._check(st)
        return code.value

    def decode_split(self, kv_indptr, last_page_len, window_left=-1):
        kvp, lpl = _i32(kv_indptr), _i32(last_page_len)
        batch = len(kvp) - 1
        cap = batch + 16 * max(1, self.cfg.sm_count or 256) + 8  # up to 8 decode CTAs per SM
        tiles = np.zeros(5 * cap, np.int32)
        nt, nc = ctypes.c_int(cap), ctypes.c_int()
        self._check(self.lib.pkv_decode_split(self.h, _p(kvp), _p(lpl), batch, int(window_left), _p(tiles),
                                              ctypes.byref(nt), ctypes.byref(nc)))
        return tiles[: 5 * nt.value].reshape(-1, 5), nc.value

    def decode_head_rows(self, kv_indptr, kv_indices, last_page_len, window_left=-1):
        """Cache rows of each decode CTA's first 4 chunks ([CTAs, 4], -1 past its end)."""
        kvp, kvi, lpl = _i32(kv_indptr), _i32(kv_indices), _i32(last_page_len)
        batch = len(kvp) - 1
        cap = batch + 16 * max(1, self.cfg.sm_count or 256) + 8  # up to 8 decode CTAs per SM
        rows = np.zeros(4 * cap, np.int32)
        nc = ctypes.c_int(cap)
        self._check(self.lib.pkv_decode_head_rows(self.h, _p(kvp), _p(kvi), _p(lpl), batch, int(window_left),
                                                  _p(rows), ctypes.byref(nc)))
        return rows[: 4 * nc.value].reshape(-1, 4)


class LatentHandle:
    """Latent attention (pkv_latent_*): keys and values from one vector [latent | rope] per token.  The
    absorbed form runs over a paged cache [pages, page_size, 576]; the expanded form over contiguous
    per-head keys and values (see include/pkv.h)."""

    LATENT, ROPE, NOPE, V = 512, 64, 128, 128

    def __init__(self, *, num_heads, page_size, max_batch, max_total_tokens, max_num_pages, num_cache_pages,
                 latent_dim=512, rope_dim=64, nope_dim=128, v_dim=128, sm_count=0, enable_nvtx=False):
        self.lib = load()
        self.cfg = LatentConfig(num_heads, latent_dim, rope_dim, nope_dim, v_dim, page_size, max_batch,
                                max_total_tokens, max_num_pages, num_cache_pages, sm_count, int(enable_nvtx))
        h = ctypes.c_void_p()
        st = self.lib.pkv_latent_create(ctypes.byref(self.cfg), ctypes.byref(h))
        if st != OK:
            raise PkvError(st, self.lib.pkv_latent_last_error(None).decode())
        self.h = h
        self._tokens = self._keys = 0
        self._cache_shape = (num_cache_pages, page_size, self.LATENT + self.ROPE)

    def close(self):
        if getattr(self, "h", None):
            self.lib.pkv_latent_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, st):
        if st != OK:
            raise PkvError(st, self.lib.pkv_latent_last_error(self.h).decode())

    def workspace_size(self, mode: int) -> int:
        """mode: MODE_PREFILL for plan(), MODE_DENSE for plan_dense()."""
        n = ctypes.c_size_t()
        self._check(self.lib.pkv_latent_workspace_size(self.h, mode, ctypes.byref(n)))
        return n.value

    def plan(self, qo_indptr, kv_indptr, kv_indices, last_page_len, *, workspace, sm_scale, causal=True,
             window_left=-1, stream=None):
        """qo_indptr None: one new token per row."""
        arrs, batch = _paged_lists(qo_indptr, kv_indptr, kv_indices, last_page_len)
        self._check(self.lib.pkv_latent_plan(self.h, *(_p(a) for a in arrs), batch, int(bool(causal)), int(window_left),
                                             float(sm_scale), _dptr(workspace),
                                             workspace.numel() * workspace.element_size(), _stream(stream)))
        self._tokens = batch if arrs[0] is None else arrs[0].item(batch)

    def _rows(self, name, t, width, torch, device):
        """Pointer and row stride of a [tokens, width] tensor whose rows may be strided."""
        _check_tensor(name, t, torch.bfloat16, (self._tokens, width), device, contiguous=False)
        if t.stride(1) != 1:
            raise ValueError(f"{name} must have unit stride in its last dimension")
        return t.data_ptr(), _stride(t, 0, width)

    def append_planned(self, c_new, rope_new, cache_layer, *, workspace, stream=None):
        """The step's new vectors into their slots: c_new [T, 512] and rope_new [T, 64], rows may be strided."""
        torch = _torch or _load_torch()
        device = torch.cuda.current_device()
        c, cs = self._rows("c_new", c_new, self.LATENT, torch, device)
        r, rs = self._rows("rope_new", rope_new, self.ROPE, torch, device)
        _check_tensor("cache_layer", cache_layer, torch.bfloat16, self._cache_shape, device)
        self._check(self.lib.pkv_latent_append_planned(
            self.h, c, cs, r, rs, cache_layer.data_ptr(), _workspace(workspace, device),
            _raw_stream(device) if stream is None else _stream(stream)))

    def _check_out(self, out, lse, width, torch, device):
        tokens, heads = self._tokens, self.cfg.num_heads
        _check_tensor("out", out, torch.bfloat16, (tokens, heads, width), device)
        if lse is not None:
            _check_tensor("lse", lse, torch.float32, (tokens, heads), device)

    def run(self, q, cache_layer, out, lse=None, *, workspace, stream=None):
        """Absorbed form: q [T, heads, 576], out [T, heads, 512], lse [T, heads]."""
        torch = _torch or _load_torch()
        device = torch.cuda.current_device()
        _check_tensor("q", q, torch.bfloat16, (self._tokens, self.cfg.num_heads, self.LATENT + self.ROPE), device)
        _check_tensor("cache_layer", cache_layer, torch.bfloat16, self._cache_shape, device)
        self._check_out(out, lse, self.LATENT, torch, device)
        self._check(self.lib.pkv_latent_run(
            self.h, q.data_ptr(), cache_layer.data_ptr(), out.data_ptr(), _dptr(lse), _workspace(workspace, device),
            _raw_stream(device) if stream is None else _stream(stream)))

    def plan_dense(self, cu_q, cu_k, *, workspace, sm_scale, causal=True, window_left=-1, stream=None):
        cq, ck, batch = _dense_lists(cu_q, cu_k)
        self._check(self.lib.pkv_latent_plan_dense(self.h, _p(cq), _p(ck), batch, int(bool(causal)),
                                                   int(window_left), float(sm_scale), _dptr(workspace),
                                                   workspace.numel() * workspace.element_size(), _stream(stream)))
        self._tokens, self._keys = cq.item(batch), ck.item(batch)

    def run_dense(self, q, k_nope, k_rope, v, out, lse=None, *, workspace, stream=None):
        """Expanded form: q [T, heads, 192], k_nope and v [keys, heads, 128], k_rope [keys, 64] (these three
        with any token and head strides), out [T, heads, 128], lse [T, heads]."""
        torch = _torch or _load_torch()
        device, bf, H = torch.cuda.current_device(), torch.bfloat16, self.cfg.num_heads
        _check_tensor("q", q, bf, (self._tokens, H, self.NOPE + self.ROPE), device)
        _check_tensor("k_nope", k_nope, bf, (self._keys, H, self.NOPE), device, contiguous=False)
        _check_tensor("k_rope", k_rope, bf, (self._keys, self.ROPE), device, contiguous=False)
        _check_tensor("v", v, bf, (self._keys, H, self.V), device, contiguous=False)
        if k_nope.stride(2) != 1 or k_rope.stride(1) != 1 or v.stride(2) != 1:
            raise ValueError("k_nope, k_rope and v must have unit stride in their last dimension")
        self._check_out(out, lse, self.V, torch, device)
        self._check(self.lib.pkv_latent_run_dense(
            self.h, q.data_ptr(), k_nope.data_ptr(), _stride(k_nope, 0, self.NOPE), _stride(k_nope, 1, self.NOPE),
            k_rope.data_ptr(), _stride(k_rope, 0, self.ROPE), v.data_ptr(), _stride(v, 0, self.V), _stride(v, 1, self.V),
            out.data_ptr(), _dptr(lse), _workspace(workspace, device),
            _raw_stream(device) if stream is None else _stream(stream)))

    def check_device_error(self, workspace, stream=None) -> int:
        code = ctypes.c_int()
        st = self.lib.pkv_latent_check_device_error(self.h, _dptr(workspace), _stream(stream), ctypes.byref(code))
        if st not in (OK, ERR_DEVICE):
            self._check(st)
        return code.value


def append_slots(page_size, qo_indptr, kv_indptr, kv_indices, last_page_len):
    lib = load()
    qo, kvp, kvi, lpl = _i32(qo_indptr), _i32(kv_indptr), _i32(kv_indices), _i32(last_page_len)
    T = int(qo[-1])
    pages, slots = np.zeros(T, np.int32), np.zeros(T, np.int32)
    st = lib.pkv_append_slots(page_size, _p(qo), _p(kvp), _p(kvi), _p(lpl), len(kvp) - 1, _p(pages), _p(slots))
    if st != OK:
        raise PkvError(st, "append_slots")
    return pages, slots


def context_only_views(page_size, qo_indptr, kv_indptr, kv_indices, last_page_len):
    lib = load()
    qo, kvp, kvi, lpl = _i32(qo_indptr), _i32(kv_indptr), _i32(kv_indices), _i32(last_page_len)
    B = len(kvp) - 1
    okvp, okvi, olpl = np.zeros(B + 1, np.int32), np.zeros(max(len(kvi), 1), np.int32), np.zeros(B, np.int32)
    nnz = ctypes.c_int()
    st = lib.pkv_context_only_views(page_size, _p(qo), _p(kvp), _p(kvi), _p(lpl), B, _p(okvp), _p(okvi), _p(olpl),
                                    ctypes.byref(nnz))
    if st != OK:
        raise PkvError(st, "context_only_views")
    return okvp, okvi[: nnz.value], olpl


def mixed_layout(qo_indptr, kv_indptr, kv_indices, last_page_len, *, max_prefill_rows, sink_page):
    lib = load()
    qo, kvp, kvi, lpl = _i32(qo_indptr), _i32(kv_indptr), _i32(kv_indices), _i32(last_page_len)
    B, T = len(kvp) - 1, int(qo[-1])
    out = dict(is_decode=np.zeros(B, np.int32), prompt_rows=np.zeros(max_prefill_rows, np.int32),
               perm=np.zeros(T, np.int32), pf_qo_indptr=np.zeros(max_prefill_rows + 1, np.int32),
               dec_kv_indptr=np.zeros(B + 1, np.int32), dec_kv_indices=np.zeros(len(kvi) + B, np.int32),
               dec_last_page_len=np.zeros(B, np.int32), dec_q_token=np.zeros(B, np.int32),
               dec_out_token=np.zeros(B, np.int32))
    nnz = ctypes.c_int()
    keys = ["is_decode", "prompt_rows", "perm", "pf_qo_indptr", "dec_kv_indptr", "dec_kv_indices",
            "dec_last_page_len", "dec_q_token", "dec_out_token"]
    st = lib.pkv_mixed_layout(_p(qo), _p(kvp), _p(kvi), _p(lpl), B, max_prefill_rows, sink_page,
                              *(_p(out[k]) for k in keys), ctypes.byref(nnz))
    if st != OK:
        raise PkvError(st, "mixed_layout")
    out["dec_kv_indices"] = out["dec_kv_indices"][: nnz.value]
    return out
