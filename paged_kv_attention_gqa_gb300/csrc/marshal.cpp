// Argument marshalling of the speculative step's calls (the Python module _marshal): each checks its tensors
// (type, shape, device, layout) and hands their pointers to the C ABI.  The same checks written in Python
// cost 0.5 us a tensor (Grace), 13 to 19 us a call; here a call's are below 1 us.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <string>

#include "../../include/pkv.h"

namespace {

struct Entries {
    decltype(&pkv_build_maps) build_maps = nullptr;
    decltype(&pkv_plan_tree) plan_tree = nullptr;
    decltype(&pkv_run_tree) run_tree = nullptr;
    decltype(&pkv_run_accept) run_accept = nullptr;
} g_entries;

// Thrown with a Python exception set.
struct Raised {};

[[noreturn]] void raise(PyObject *kind, const char *format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(kind, format, args);
    va_end(args);
    throw Raised();
}

std::string text(PyObject *o, const char *attribute) {
    PyObject *a = PyObject_GetAttrString(o, attribute), *s = a ? PyObject_Str(a) : nullptr;
    const char *c = s ? PyUnicode_AsUTF8(s) : nullptr;
    std::string out = c ? c : "?";
    PyErr_Clear();
    Py_XDECREF(s);
    Py_XDECREF(a);
    return out;
}

const char *type_name(at::ScalarType t) {
    switch (t) {
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kFloat: return "torch.float32";
        default: return "torch.bfloat16";
    }
}

const at::Tensor &tensor(const char *name, PyObject *o) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

// A tensor of this type and shape on `device`, contiguous unless said otherwise.
const at::Tensor &checked(const char *name, PyObject *o, at::ScalarType type, at::IntArrayRef shape, int64_t device,
                          bool contiguous = true) {
    const at::Tensor &t = tensor(name, o);
    if (t.scalar_type() != type)
        raise(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), text(o, "dtype").c_str());
    if (t.sizes() != shape) {
        std::string want;
        for (int64_t d : shape) want += (want.empty() ? "" : ", ") + std::to_string(d);
        raise(PyExc_ValueError, "%s must have shape (%s), got %s", name, want.c_str(), text(o, "shape").c_str());
    }
    if (t.layout() != at::kStrided) raise(PyExc_ValueError, "%s must be a dense tensor", name);
    if (t.get_device() != device)
        raise(PyExc_ValueError, "%s must be on the current CUDA device, got %s", name, t.device().str().c_str());
    if (contiguous && !t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    return t;
}

int32_t *ints(const char *name, PyObject *o, int64_t entries, int64_t device) {
    return static_cast<int32_t *>(checked(name, o, at::kInt, {entries}, device).data_ptr());
}
int32_t *ints_or_none(const char *name, PyObject *o, int64_t entries, int64_t device) {
    return o == Py_None ? nullptr : ints(name, o, entries, device);
}
// One dimension of any length that fits 32 bits.
int length(const char *name, PyObject *o) {
    const at::Tensor &t = tensor(name, o);
    if (t.dim() != 1) raise(PyExc_ValueError, "%s must have one dimension, has %d", name, (int)t.dim());
    if (t.numel() > INT32_MAX) raise(PyExc_ValueError, "%s has too many entries", name);
    return (int)t.numel();
}

// Stride of one dimension in elements; of a dimension of one entry, which is never stepped, the least.
int64_t stride(const at::Tensor &t, int64_t dim, int64_t least) { return t.size(dim) > 1 ? t.stride(dim) : least; }

void heads_side_by_side(const char *name, const at::Tensor &t) {
    if (t.stride(-1) != 1 || (t.size(-2) > 1 && t.stride(-2) != t.size(-1)))
        raise(PyExc_ValueError, "%s must have its heads side by side", name);
}

long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}
int integer32(const char *name, PyObject *o) {
    const long long v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_ValueError, "%s does not fit 32 bits", name);
    return (int)v;
}
void *pointer(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised();
    return p;
}

struct Workspace {
    void *data;
    size_t bytes;
};
Workspace workspace(PyObject *o, int64_t device) {
    const at::Tensor &t = tensor("workspace", o);
    if (t.get_device() != device)
        raise(PyExc_ValueError, "workspace must be on the current CUDA device, is on %s", t.device().str().c_str());
    if (!t.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
    return Workspace{t.data_ptr(), (size_t)t.numel() * t.element_size()};
}

// What every call begins with: the handle, the current device and the stream.
struct Call {
    pkv_handle_t h;
    int64_t device;
    pkv_stream_t stream;
    explicit Call(PyObject *const *a)
        : h(static_cast<pkv_handle_t>(pointer(a[0]))), device(integer(a[1])), stream(pointer(a[2])) {}
};

// The handle's shape: (num_cache_pages, page_size, num_qo_heads, num_kv_heads, head_dim).
struct Dims {
    int64_t pages, page, hq, hkv, d;
    explicit Dims(PyObject *o)
        : pages(integer(PyTuple_GetItem(o, 0))), page(integer(PyTuple_GetItem(o, 1))), hq(integer(PyTuple_GetItem(o, 2))),
          hkv(integer(PyTuple_GetItem(o, 3))), d(integer(PyTuple_GetItem(o, 4))) {}
};

template <typename F>
PyObject *released(F &&f) {  // the call itself without the interpreter's lock: it may wait for the driver
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

template <int N, typename F>
PyObject *guarded(Py_ssize_t n, F &&f) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", N, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// handle, device, stream, seq_lens, new_lens, block_table, num_blocks, num_blocks_out, free_pages, free_count,
// free_count_out, qo_indptr, kv_indptr, kv_indices, last_page_len, slots, positions, status
PyObject *build_maps(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<18>(n, [&] {
        const Call c(a);
        const int batch = length("seq_lens", a[3]);
        const at::Tensor &table = tensor("block_table", a[5]);
        if (table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
            raise(PyExc_ValueError, "block_table must be [batch, blocks] with unit stride in its last dimension");
        const int64_t blocks = table.size(1);
        checked("block_table", a[5], at::kInt, {batch, blocks}, c.device, false);
        if (blocks > INT32_MAX) raise(PyExc_ValueError, "block_table has too many columns");
        // without slots and positions nothing is listed by token
        const int tokens = a[15] != Py_None ? length("slots", a[15]) : a[16] != Py_None ? length("positions", a[16]) : INT32_MAX;
        const int free_pages = length("free_pages", a[8]), indices = length("kv_indices", a[13]);
        int32_t *const seq = ints("seq_lens", a[3], batch, c.device), *const fresh = ints("new_lens", a[4], batch, c.device);
        int32_t *const held = ints("num_blocks", a[6], batch, c.device);
        int32_t *const held_out = ints("num_blocks_out", a[7], batch, c.device);
        int32_t *const free = ints("free_pages", a[8], free_pages, c.device);
        int32_t *const count = ints("free_count", a[9], 1, c.device), *const count_out = ints("free_count_out", a[10], 1, c.device);
        int32_t *const qo = ints("qo_indptr", a[11], batch + 1, c.device), *const kvp = ints("kv_indptr", a[12], batch + 1, c.device);
        int32_t *const kvi = ints("kv_indices", a[13], indices, c.device), *const last = ints("last_page_len", a[14], batch, c.device);
        int32_t *const slots = ints_or_none("slots", a[15], tokens, c.device);
        int32_t *const positions = ints_or_none("positions", a[16], tokens, c.device);
        int32_t *const status = ints("status", a[17], 1, c.device);
        int32_t *const blocks_at = static_cast<int32_t *>(table.data_ptr());
        const int64_t step = stride(table, 0, blocks);
        return released([&] {
            return g_entries.build_maps(c.h, seq, fresh, batch, blocks_at, step, (int)blocks, held, held_out, free, free_pages, count,
                                        count_out, qo, kvp, kvi, indices, last, slots, positions, tokens, status, c.stream);
        });
    });
}

// handle, device, stream, qo_indptr, kv_indptr, kv_indices, last_page_len, parents, num_tokens, max_new, positions,
// workspace, window_left, sm_scale
PyObject *plan_tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<14>(n, [&] {
        const Call c(a);
        const int rows = length("kv_indptr", a[4]);
        if (rows < 1) raise(PyExc_ValueError, "kv_indptr needs 1 entries, has 0");
        const int indices = length("kv_indices", a[5]), tokens = integer32("num_tokens", a[8]), most = integer32("max_new", a[9]);
        int32_t *const qo = ints("qo_indptr", a[3], rows, c.device), *const kvp = ints("kv_indptr", a[4], rows, c.device);
        int32_t *const kvi = ints("kv_indices", a[5], indices, c.device);
        int32_t *const last = ints("last_page_len", a[6], rows - 1, c.device);
        int32_t *const parents = ints_or_none("parents", a[7], tokens, c.device);
        int32_t *const positions = ints_or_none("positions", a[10], tokens, c.device);
        const Workspace ws = workspace(a[11], c.device);
        const int window = integer32("window_left", a[12]);
        const double scale = PyFloat_AsDouble(a[13]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised();
        return released([&] {
            return g_entries.plan_tree(c.h, qo, kvp, kvi, indices, last, rows - 1, parents, tokens, most, window, (float)scale,
                                       positions, ws.data, ws.bytes, c.stream);
        });
    });
}

// handle, device, stream, shape, tokens, q, k_new, v_new, kv_layer, out, lse, workspace
PyObject *run_tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<12>(n, [&] {
        const Call c(a);
        const Dims s(a[3]);
        const int64_t tokens = integer(a[4]);
        const at::Tensor &k = checked("k_new", a[6], at::kBFloat16, {tokens, s.hkv, s.d}, c.device, false);
        const at::Tensor &v = checked("v_new", a[7], at::kBFloat16, {tokens, s.hkv, s.d}, c.device, false);
        const at::Tensor &q = checked("q", a[5], at::kBFloat16, {tokens, s.hq, s.d}, c.device, false);
        heads_side_by_side("q", q);
        heads_side_by_side("k_new", k);
        heads_side_by_side("v_new", v);
        const at::Tensor &kv = checked("kv_layer", a[8], at::kBFloat16, {s.pages, 2, s.page, s.hkv, s.d}, c.device);
        void *const out = checked("out", a[9], at::kBFloat16, {tokens, s.hq, s.d}, c.device).data_ptr();
        void *const lse = a[10] == Py_None ? nullptr : checked("lse", a[10], at::kFloat, {tokens, s.hq}, c.device).data_ptr();
        const Workspace ws = workspace(a[11], c.device);
        const int64_t qs = stride(q, 0, s.hq * s.d), ks = stride(k, 0, s.hkv * s.d), vs = stride(v, 0, s.hkv * s.d);
        const void *const qp = q.data_ptr(), *const kp = k.data_ptr(), *const vp = v.data_ptr(), *const cache = kv.data_ptr();
        return released([&] {
            return g_entries.run_tree(c.h, qp, qs, kp, ks, vp, vs, cache, out, static_cast<float *>(lse), ws.data, c.stream);
        });
    });
}

// handle, device, stream, shape, tokens, batch, draft_tokens, target_tokens, k_new, v_new, kv_cache, accepted,
// num_accepted, next_tokens, seq_lens, workspace
PyObject *run_accept(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<16>(n, [&] {
        const Call c(a);
        const Dims s(a[3]);
        const int64_t tokens = integer(a[4]), batch = integer(a[5]);
        const at::Tensor &draft = tensor("draft_tokens", a[6]), &cache = tensor("kv_cache", a[10]);
        const at::ScalarType kind = draft.scalar_type();
        if (kind != at::kInt && kind != at::kLong)
            raise(PyExc_TypeError, "draft_tokens must be int32 or int64, got %s", text(a[6], "dtype").c_str());
        checked("draft_tokens", a[6], kind, {tokens}, c.device);
        const at::Tensor &target = checked("target_tokens", a[7], kind, {tokens}, c.device);
        int32_t *const accepted = ints("accepted", a[11], tokens, c.device);
        int32_t *const count = ints("num_accepted", a[12], batch, c.device);
        const at::Tensor &next = checked("next_tokens", a[13], kind, {batch}, c.device);
        int32_t *const seq = ints_or_none("seq_lens", a[14], batch, c.device);
        if (cache.dim() != 6) raise(PyExc_ValueError, "kv_cache must be [layers, pages, 2, page_size, kv heads, head_dim]");
        const int64_t layers = cache.size(0);
        checked("kv_cache", a[10], at::kBFloat16, {layers, s.pages, 2, s.page, s.hkv, s.d}, c.device, false);
        int64_t width = s.d;
        bool dense = cache.stride(5) == 1;
        for (int d = 4; d >= 1; --d) {
            dense = dense && (cache.size(d) == 1 || cache.stride(d) == width);
            width *= cache.size(d);
        }
        if (!dense) raise(PyExc_ValueError, "kv_cache must have contiguous layers");
        const at::Tensor &k = checked("k_new", a[8], at::kBFloat16, {layers, tokens, s.hkv, s.d}, c.device, false);
        const at::Tensor &v = checked("v_new", a[9], at::kBFloat16, {layers, tokens, s.hkv, s.d}, c.device, false);
        heads_side_by_side("k_new", k);
        heads_side_by_side("v_new", v);
        if (layers > INT32_MAX) raise(PyExc_ValueError, "kv_cache has too many layers");
        const Workspace ws = workspace(a[15], c.device);
        const int64_t least = s.hkv * s.d;
        const int64_t kl = stride(k, 0, least), kt = stride(k, 1, least), vl = stride(v, 0, least), vt = stride(v, 1, least);
        const int64_t cl = stride(cache, 0, width);
        const void *const dp = draft.data_ptr(), *const tp = target.data_ptr(), *const kp = k.data_ptr(), *const vp = v.data_ptr();
        void *const cp = cache.data_ptr(), *const np = next.data_ptr();
        const int bytes = kind == at::kLong ? 8 : 4;
        return released([&] {
            return g_entries.run_accept(c.h, dp, tp, bytes, kp, kl, kt, vp, vl, vt, cp, cl, (int)layers, accepted, count, np, seq,
                                        ws.data, c.stream);
        });
    });
}

// Addresses of the library's build_maps, plan_tree, run_tree and run_accept.
PyObject *connect(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<4>(n, [&]() -> PyObject * {
        g_entries.build_maps = reinterpret_cast<decltype(&pkv_build_maps)>(pointer(a[0]));
        g_entries.plan_tree = reinterpret_cast<decltype(&pkv_plan_tree)>(pointer(a[1]));
        g_entries.run_tree = reinterpret_cast<decltype(&pkv_run_tree)>(pointer(a[2]));
        g_entries.run_accept = reinterpret_cast<decltype(&pkv_run_accept)>(pointer(a[3]));
        Py_RETURN_NONE;
    });
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
    static PyMethodDef methods[] = {{"connect", fast(connect), METH_FASTCALL, nullptr},
                                    {"build_maps", fast(build_maps), METH_FASTCALL, nullptr},
                                    {"plan_tree", fast(plan_tree), METH_FASTCALL, nullptr},
                                    {"run_tree", fast(run_tree), METH_FASTCALL, nullptr},
                                    {"run_accept", fast(run_accept), METH_FASTCALL, nullptr},
                                    {nullptr, nullptr, 0, nullptr}};
    static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
    return PyModule_Create(&module);
}
