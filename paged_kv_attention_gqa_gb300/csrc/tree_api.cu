// The C ABI of the speculative step (pkv_build_maps, pkv_plan_tree, pkv_run_tree, pkv_run_accept in
// include/pkv.h): checks, tensor maps, launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <exception>

#include "handle.h"
#include "launch.h"
#include "tree.h"

using pkv::Shape;
using pkv::TreePlan;

static pkv_status fail(pkv_handle_t h, pkv_status st, const std::string &msg) {
    h->err = msg;
    return st;
}
static pkv_status cuda_fail(pkv_handle_t h, cudaError_t e, const char *what) {
    return fail(h, PKV_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

// No C++ exception crosses the C boundary (the text of an error may find no memory).
template <typename F>
static pkv_status guarded(pkv_handle_t h, F &&f) {
    if (!h) return PKV_ERR_INVALID;
    try {
        return f();
    } catch (const std::exception &) {
        h->err.clear();
        return PKV_ERR_INVALID;
    }
}

// The handle's mark in a workspace.  A negative number as an integer, since other plans' words there are counts.
static uint32_t tag(pkv_handle_t h) {
    static std::atomic<uint32_t> handles{0};
    if (!h->tree_tag) h->tree_tag = 0x80000000u | handles.fetch_add(1) * 0x9e3779b1u;
    return h->tree_tag;
}

// Kernel attributes are set outside captures alone.  So a handle's first uncaptured call on a device sets those of all
// kernels that its calls of any size may choose: a captured one may be of another size than those before it.
template <typename F>
static cudaError_t prepare(int &ready, cudaStream_t st, F &&raise) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess || device == ready) return e;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cs) == cudaSuccess && cs != cudaStreamCaptureStatusNone) return cudaSuccess;
    e = raise();
    if (e == cudaSuccess) ready = device;
    return e;
}

static uintptr_t bits(const void *p) { return reinterpret_cast<uintptr_t>(p); }

extern "C" pkv_status pkv_build_maps(pkv_handle_t h, const int32_t *seq_lens, const int32_t *new_lens, int batch,
                                     int32_t *block_table, int64_t table_stride, int max_blocks, const int32_t *num_blocks,
                                     int32_t *num_blocks_out, int32_t *free_pages, int free_capacity,
                                     const int32_t *free_count, int32_t *free_count_out, int32_t *qo_indptr,
                                     int32_t *kv_indptr, int32_t *kv_indices, int indices_capacity,
                                     int32_t *last_page_len, int32_t *slots, int32_t *positions, int token_capacity,
                                     int32_t *status, pkv_stream_t stream) {
    return guarded(h, [&]() -> pkv_status {
        NvtxCall range(h, "pkv_build_maps");
        if (batch < 0 || batch > h->shape.max_batch) return fail(h, PKV_ERR_INVALID, "batch is negative or above max_batch");
        if (batch > pkv::kMapsMaxRows)
            return fail(h, PKV_ERR_UNSUPPORTED, "more than " + std::to_string(pkv::kMapsMaxRows) + " rows are not mapped at once");
        if (max_blocks < 0 || free_capacity < 0 || indices_capacity < 0 || token_capacity < 0)
            return fail(h, PKV_ERR_INVALID, "capacities must be >= 0");
        if (table_stride < max_blocks) return fail(h, PKV_ERR_INVALID, "table_stride is below max_blocks");
        if (!qo_indptr || !kv_indptr || !status || !free_count || !free_count_out)
            return fail(h, PKV_ERR_INVALID, "null qo_indptr, kv_indptr, status or free_count");
        if (batch && (!seq_lens || !new_lens || !num_blocks || !num_blocks_out || !last_page_len))
            return fail(h, PKV_ERR_INVALID, "null seq_lens, new_lens, num_blocks or last_page_len");
        if ((batch && max_blocks && !block_table) || (free_capacity && !free_pages) || (indices_capacity && !kv_indices))
            return fail(h, PKV_ERR_INVALID, "null block_table, free_pages or kv_indices");
        if ((bits(seq_lens) | bits(new_lens) | bits(block_table) | bits(num_blocks) | bits(num_blocks_out) | bits(free_pages) |
             bits(free_count) | bits(free_count_out) | bits(qo_indptr) | bits(kv_indptr) | bits(kv_indices) |
             bits(last_page_len) | bits(slots) | bits(positions) | bits(status)) % 4)
            return fail(h, PKV_ERR_INVALID, "arrays must be 4-byte aligned");
        if (num_blocks != num_blocks_out && num_blocks_out < num_blocks + batch && num_blocks < num_blocks_out + batch)
            return fail(h, PKV_ERR_INVALID, "num_blocks_out is num_blocks itself or does not overlap it");
        pkv::MapsArgs a;
        a.seq = seq_lens;
        a.fresh = new_lens;
        a.held = num_blocks;
        a.free_count = free_count;
        a.table = block_table;
        a.free_pages = free_pages;
        a.table_stride = table_stride;
        a.rows = batch;
        a.max_blocks = max_blocks;
        a.free_capacity = free_capacity;
        a.indices_capacity = indices_capacity;
        a.token_capacity = token_capacity;
        a.page_shift = h->shape.page_shift();
        a.held_out = num_blocks_out;
        a.free_count_out = free_count_out;
        a.qo = qo_indptr;
        a.kvp = kv_indptr;
        a.kvi = kv_indices;
        a.last = last_page_len;
        a.slots = slots;
        a.positions = positions;
        a.status = status;
        const cudaStream_t st = static_cast<cudaStream_t>(stream);
        cudaError_t e = prepare(h->maps_ready, st, [&] { return pkv::prepare_maps(st); });
        if (e == cudaSuccess) e = pkv::launch_maps(a, st);
        return e == cudaSuccess ? PKV_OK : cuda_fail(h, e, "maps launch");
    });
}

extern "C" pkv_status pkv_plan_tree(pkv_handle_t h, const int32_t *qo_indptr, const int32_t *kv_indptr,
                                    const int32_t *kv_indices, int num_indices, const int32_t *last_page_len, int batch,
                                    const int32_t *parents, int num_tokens, int max_new, int window_left, float sm_scale,
                                    int32_t *positions, void *workspace, size_t workspace_bytes, pkv_stream_t stream) {
    return guarded(h, [&]() -> pkv_status {
        NvtxCall range(h, "pkv_plan_tree");
        const Shape &s = h->shape;
        if (!workspace) return fail(h, PKV_ERR_INVALID, "null workspace");
        if (bits(workspace) % pkv::kAlign) return fail(h, PKV_ERR_INVALID, "workspace must be 256-byte aligned");
        if (s.page_size < pkv::kTreeMinPage)
            return fail(h, PKV_ERR_UNSUPPORTED, "page_size below 8 is not computed for trees of drafted tokens");
        if (batch < 0 || batch > s.max_batch) return fail(h, PKV_ERR_INVALID, "batch is negative or above max_batch");
        if (num_tokens < 0 || num_tokens > s.max_total_tokens)
            return fail(h, PKV_ERR_INVALID, "num_tokens is negative or above max_total_tokens");
        if (max_new < 1) return fail(h, PKV_ERR_INVALID, "max_new must be >= 1");
        if (max_new > pkv::kTreeMaxNew)
            return fail(h, PKV_ERR_UNSUPPORTED,
                        "max_new " + std::to_string(max_new) + " is not computed (at most " + std::to_string(pkv::kTreeMaxNew) + ")");
        if (window_left < -1) return fail(h, PKV_ERR_INVALID, "window_left must be >= -1");
        if (!(sm_scale >= 0.f) || std::isinf(sm_scale)) return fail(h, PKV_ERR_INVALID, "sm_scale must be finite and >= 0");
        if (num_indices < 0 || num_indices > s.max_num_pages)
            return fail(h, PKV_ERR_INVALID, "num_indices is negative or above max_num_pages");
        if (batch && (!qo_indptr || !kv_indptr || !last_page_len || (num_indices && !kv_indices)))
            return fail(h, PKV_ERR_INVALID, "null index array");
        if ((bits(qo_indptr) | bits(kv_indptr) | bits(kv_indices) | bits(last_page_len) | bits(parents) | bits(positions)) % 4)
            return fail(h, PKV_ERR_INVALID, "index arrays must be 4-byte aligned");
        TreePlan p;
        pkv::tree_layout(s, batch, num_tokens, max_new, num_indices, window_left, p);
        h->planned_ws = nullptr;
        if (p.total > workspace_bytes)
            return fail(h, PKV_ERR_WORKSPACE,
                        "workspace of " + std::to_string(workspace_bytes) + " bytes is too small: this plan needs " +
                            std::to_string(p.total) + " bytes (pkv_workspace_size gives the bound at the maxima)");
        p.scale_log2 = (sm_scale > 0.f ? sm_scale : 1.f / std::sqrt((float)s.head_dim)) * 1.4426950408889634f;
        p.pages = kv_indices;
        const pkv::TreeIndex x{qo_indptr, kv_indptr, kv_indices, last_page_len, parents, num_indices, positions};
        const cudaStream_t st = static_cast<cudaStream_t>(stream);
        cudaError_t e = prepare(h->tree_ready, st, [&] { return pkv::prepare_tree(s, st); });
        if (e == cudaSuccess) e = pkv::launch_tree_plan(s, p, x, tag(h), workspace, st);
        if (e != cudaSuccess) return cuda_fail(h, e, "tree plan launch");
        pkv::Plan plan;
        plan.mode = PKV_MODE_TREE;
        plan.batch = batch;
        plan.num_tokens = num_tokens;
        plan.lay.total = p.total;
        h->spare_image.swap(h->plan.image);
        h->plan = std::move(plan);
        h->tree = p;
        h->planned_ws = workspace;
        return PKV_OK;
    });
}

static pkv_status check_planned(pkv_handle_t h, const void *ws) {
    if (!h->planned_ws || h->planned_ws != ws)
        return fail(h, PKV_ERR_NOT_PLANNED, "no plan was made on this workspace by this handle");
    if (h->plan.mode != PKV_MODE_TREE) return fail(h, PKV_ERR_NOT_PLANNED, "the workspace holds a plan of another mode");
    return PKV_OK;
}

// Tensor map over a bf16 tensor [outer][rows][head_dim], boxes of 64 columns x box_rows x box_outer, 128-byte swizzle.
static pkv_status encode(pkv_handle_t h, const void *base, long long rows, long long row_stride, long long outer,
                         long long outer_stride, int box_rows, int box_outer, CUtensorMap *tm) {
    auto fn = pkv::encode_fn();
    if (!fn) return fail(h, PKV_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    const cuuint64_t dims[3] = {(cuuint64_t)h->shape.head_dim, (cuuint64_t)rows, (cuuint64_t)outer};
    const cuuint64_t strides[2] = {(cuuint64_t)row_stride * 2, (cuuint64_t)outer_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_outer}, es[3] = {1, 1, 1};
    const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(h, PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")");
    return PKV_OK;
}

static bool bad_stride(int64_t stride, int64_t least) { return stride < least || stride % 8 || stride >= (1ll << 38); }

extern "C" pkv_status pkv_run_tree(pkv_handle_t h, const void *q, int64_t q_stride, const void *k_new, int64_t k_stride,
                                   const void *v_new, int64_t v_stride, const void *kv_layer, void *out, float *lse,
                                   void *workspace, pkv_stream_t stream) {
    return guarded(h, [&]() -> pkv_status {
        NvtxCall range(h, "pkv_run_tree");
        pkv_status st = check_planned(h, workspace);
        if (st != PKV_OK) return st;
        const Shape &s = h->shape;
        const TreePlan &p = h->tree;
        if (p.num_tokens == 0 || p.batch == 0) return PKV_OK;
        if (!q || !k_new || !v_new || !kv_layer || !out) return fail(h, PKV_ERR_INVALID, "null q, k_new, v_new, kv_layer or out");
        if ((bits(q) | bits(k_new) | bits(v_new) | bits(kv_layer) | bits(out)) % 16 || bits(lse) % 4)
            return fail(h, PKV_ERR_INVALID, "q, k_new, v_new, kv_layer and out must be 16-byte aligned (lse 4-byte)");
        const long long D = s.head_dim, Hq = s.num_qo_heads, Hkv = s.num_kv_heads;
        if (bad_stride(q_stride, Hq * D) || bad_stride(k_stride, Hkv * D) || bad_stride(v_stride, Hkv * D))
            return fail(h, PKV_ERR_INVALID, "token strides are multiples of 8 elements and at least a token's width");
        const int box_new = std::min(pkv::kTreeKeys, (p.max_new + 7) / 8 * 8);
        const int box_q = std::min(pkv::tree_tile_tokens(s), p.max_new);
        CUtensorMap tkv, tk, tv, tq;
        if ((st = encode(h, kv_layer, (long long)s.num_cache_pages * 2 * s.page_size, Hkv * D, Hkv, D,
                         std::min(s.page_size, pkv::kTreeKeys), 1, &tkv)) != PKV_OK ||
            (st = encode(h, k_new, p.num_tokens, k_stride, Hkv, D, box_new, 1, &tk)) != PKV_OK ||
            (st = encode(h, v_new, p.num_tokens, v_stride, Hkv, D, box_new, 1, &tv)) != PKV_OK ||
            (st = encode(h, q, Hq, D, p.num_tokens, q_stride, s.group(), box_q, &tq)) != PKV_OK)
            return st;
        const cudaError_t e = pkv::launch_tree(s, p, tkv, tk, tv, tq, box_new, box_q, workspace, out, lse,
                                               static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? PKV_OK : cuda_fail(h, e, "tree launch");
    });
}

extern "C" pkv_status pkv_run_accept(pkv_handle_t h, const void *draft_tokens, const void *target_tokens, int token_bytes,
                                     const void *k_new, int64_t k_layer_stride, int64_t k_token_stride, const void *v_new,
                                     int64_t v_layer_stride, int64_t v_token_stride, void *kv_cache,
                                     int64_t cache_layer_stride, int num_layers, int32_t *accepted, int32_t *num_accepted,
                                     void *next_tokens, int32_t *seq_lens, void *workspace, pkv_stream_t stream) {
    return guarded(h, [&]() -> pkv_status {
        NvtxCall range(h, "pkv_run_accept");
        pkv_status st = check_planned(h, workspace);
        if (st != PKV_OK) return st;
        const Shape &s = h->shape;
        const TreePlan &p = h->tree;
        if (p.batch == 0) return PKV_OK;
        if (token_bytes != 4 && token_bytes != 8) return fail(h, PKV_ERR_INVALID, "token_bytes is 4 or 8");
        if (num_layers < 0 || num_layers > 65535) return fail(h, PKV_ERR_INVALID, "num_layers is between 0 and 65535");
        if (!num_accepted || !next_tokens) return fail(h, PKV_ERR_INVALID, "null num_accepted or next_tokens");
        if (p.num_tokens && (!draft_tokens || !target_tokens || !accepted))
            return fail(h, PKV_ERR_INVALID, "null draft_tokens, target_tokens or accepted");
        if (p.num_tokens && num_layers && (!k_new || !v_new || !kv_cache))
            return fail(h, PKV_ERR_INVALID, "null k_new, v_new or kv_cache");
        if ((bits(draft_tokens) | bits(target_tokens) | bits(next_tokens)) % token_bytes ||
            (bits(accepted) | bits(num_accepted) | bits(seq_lens)) % 4)
            return fail(h, PKV_ERR_INVALID, "token and index arrays must be aligned to their entries");
        if ((bits(k_new) | bits(v_new) | bits(kv_cache)) % 16)
            return fail(h, PKV_ERR_INVALID, "k_new, v_new and kv_cache must be 16-byte aligned");
        const long long width = (long long)s.num_kv_heads * s.head_dim;
        if (bad_stride(k_layer_stride, width) || bad_stride(k_token_stride, width) || bad_stride(v_layer_stride, width) ||
            bad_stride(v_token_stride, width) || bad_stride(cache_layer_stride, width * 2 * s.page_size * s.num_cache_pages))
            return fail(h, PKV_ERR_INVALID, "strides are multiples of 8 elements and at least the width stepped over");
        const pkv::TreeAccept x{draft_tokens,   target_tokens,  token_bytes == 8,  k_new,        v_new,       k_layer_stride,
                                k_token_stride, v_layer_stride, v_token_stride,    kv_cache,     cache_layer_stride,
                                num_layers,     accepted,       num_accepted,      next_tokens,  seq_lens};
        const cudaError_t e = pkv::launch_tree_accept(s, p, x, workspace, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? PKV_OK : cuda_fail(h, e, "accept launch");
    });
}
