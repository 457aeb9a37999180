// The C ABI of latent attention (pkv_latent_* in include/pkv.h): handle, checks, plan staging, launches.
#include <cmath>
#include <new>

#include "handle.h"
#include "latent.h"
#include "launch.h"

using pkv::LatentPlan;
using pkv::LatentShape;

struct pkv_latent_s {
    LatentShape shape{};
    std::string err;
    LatentPlan plan;
    std::vector<uint8_t> spare_image;
    void *planned_ws = nullptr;
    PkvStaging staging;
    bool nvtx = false;
};

static thread_local std::string g_latent_create_err;

static pkv_status fail(pkv_latent_t h, pkv_status st, const std::string &msg) {
    if (h)
        h->err = msg;
    else
        g_latent_create_err = msg;
    return st;
}
static pkv_status cuda_fail(pkv_latent_t h, cudaError_t e, const char *what) {
    return fail(h, PKV_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

// No C++ exception crosses the C boundary: the planners' host buffers may fail to grow.  The text of the
// exception becomes the handle's; if there is no memory for that either, the last one is cleared.
template <typename F>
static pkv_status guarded(pkv_latent_t h, F &&f) {
    try {
        return f();
    } catch (const std::exception &ex) {
        if (h) h->planned_ws = nullptr;
        std::string &err = h ? h->err : g_latent_create_err;
        err.clear();
        try {
            err = ex.what();
        } catch (const std::exception &) {
        }
        return PKV_ERR_INVALID;
    }
}

static uintptr_t bits(const void *p) { return reinterpret_cast<uintptr_t>(p); }

extern "C" pkv_status pkv_latent_create(const pkv_latent_config *cfg, pkv_latent_t *out) {
    return guarded(nullptr, [&]() -> pkv_status {
        if (!cfg || !out) return fail(nullptr, PKV_ERR_INVALID, "null argument");
        const pkv_latent_config &c = *cfg;
        if (c.num_heads <= 0 || c.page_size <= 0 || c.max_batch <= 0 || c.max_total_tokens <= 0 || c.max_num_pages <= 0 ||
            c.num_cache_pages <= 0 || c.sm_count < 0 || c.latent_dim < 0 || c.rope_dim < 0 || c.nope_dim < 0 || c.v_dim < 0)
            return fail(nullptr, PKV_ERR_INVALID, "configuration sizes must be positive");
        auto is = [](int v, int want) { return v == 0 || v == want; };
        if (!is(c.latent_dim, pkv::kLatentDim) || !is(c.rope_dim, pkv::kLatentRope) || !is(c.nope_dim, pkv::kLatentNope) ||
            !is(c.v_dim, pkv::kLatentV))
            return fail(nullptr, PKV_ERR_UNSUPPORTED, "these widths are not computed (latent 512, rope 64, nope 128, v 128)");
        if ((c.page_size & (c.page_size - 1)) != 0 || c.page_size < pkv::kLatentMinPage || c.page_size > 1024)
            return fail(nullptr, PKV_ERR_UNSUPPORTED,
                        "page_size " + std::to_string(c.page_size) + " is not computed (a power of two from 8 to 1024)");
        if (c.num_heads > 1024) return fail(nullptr, PKV_ERR_UNSUPPORTED, "num_heads above 1024 is not computed");
        if (c.enable_nvtx != 0 && c.enable_nvtx != 1) return fail(nullptr, PKV_ERR_INVALID, "enable_nvtx is 0 or 1");
        if ((long long)c.num_cache_pages * c.page_size >= (1ll << 31) - 64 ||
            (long long)c.max_num_pages * c.page_size >= (1ll << 31) - 64 ||
            (long long)c.max_total_tokens * c.num_heads >= (1ll << 31) - 64)
            return fail(nullptr, PKV_ERR_UNSUPPORTED, "cache slots or query rows exceed 32-bit indices");
        int sms = c.sm_count;
        if (sms == 0) {
            int dev = 0;
            cudaError_t e = cudaGetDevice(&dev);
            if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            if (e != cudaSuccess)
                return fail(nullptr, PKV_ERR_CUDA, std::string("SM count query: ") + cudaGetErrorString(e));
        }
        pkv_latent_t h = new pkv_latent_s();
        h->shape.num_heads = c.num_heads;
        h->shape.page_size = c.page_size;
        h->shape.max_batch = c.max_batch;
        h->shape.max_total_tokens = c.max_total_tokens;
        h->shape.max_num_pages = c.max_num_pages;
        h->shape.num_cache_pages = c.num_cache_pages;
        h->shape.sm_count = sms;
        h->nvtx = c.enable_nvtx != 0;
        *out = h;
        return PKV_OK;
    });
}

extern "C" void pkv_latent_destroy(pkv_latent_t h) {
    if (!h) return;
    h->staging.release();
    delete h;
}

extern "C" const char *pkv_latent_last_error(pkv_latent_t h) { return h ? h->err.c_str() : g_latent_create_err.c_str(); }

extern "C" pkv_status pkv_latent_workspace_size(pkv_latent_t h, int mode, size_t *bytes) {
    if (!h || !bytes) return fail(h, PKV_ERR_INVALID, "null argument");
    if (mode != PKV_MODE_PREFILL && mode != PKV_MODE_DENSE)
        return fail(h, PKV_ERR_INVALID, "mode is PKV_MODE_PREFILL (paged) or PKV_MODE_DENSE");
    *bytes = pkv::latent_workspace_bound(h->shape, mode == PKV_MODE_DENSE);
    return PKV_OK;
}

static pkv_status check_ws(pkv_latent_t h, const void *workspace) {
    if (!workspace) return fail(h, PKV_ERR_INVALID, "null workspace");
    if (bits(workspace) % pkv::kAlign) return fail(h, PKV_ERR_INVALID, "workspace must be 256-byte aligned");
    return PKV_OK;
}

static pkv_status stage(pkv_latent_t h, LatentPlan &plan, int rc, const std::string &err, void *workspace, size_t bytes,
                        pkv_stream_t stream) {
    h->planned_ws = nullptr;
    if (rc) {
        h->spare_image.swap(plan.image);
        return fail(h, (pkv_status)rc, err);
    }
    if (plan.total > bytes)
        return fail(h, PKV_ERR_WORKSPACE,
                    "workspace of " + std::to_string(bytes) + " bytes is too small: this plan needs " +
                        std::to_string(plan.total) + " bytes (pkv_latent_workspace_size gives the bound at the maxima)");
    const char *what = "";
    const cudaError_t e =
        h->staging.copy(plan.image.data(), plan.image.size(), workspace, static_cast<cudaStream_t>(stream), &what);
    if (e != cudaSuccess) return cuda_fail(h, e, what);
    h->spare_image.swap(plan.image);
    h->plan = std::move(plan);
    h->planned_ws = workspace;
    return PKV_OK;
}

extern "C" pkv_status pkv_latent_plan(pkv_latent_t h, const int32_t *qo_indptr, const int32_t *kv_indptr,
                                      const int32_t *kv_indices, const int32_t *last_page_len, int batch, int causal,
                                      int window_left, float sm_scale, void *workspace, size_t workspace_bytes,
                                      pkv_stream_t stream) {
    if (!h) return PKV_ERR_INVALID;
    NvtxCall range(h->nvtx, "pkv_latent_plan");
    return guarded(h, [&]() -> pkv_status {
        pkv_status st = check_ws(h, workspace);
        if (st != PKV_OK) return st;
        std::string err;
        LatentPlan plan;
        plan.image.swap(h->spare_image);
        const int rc = pkv::make_latent_plan(h->shape, qo_indptr, kv_indptr, kv_indices, last_page_len, batch, causal,
                                             window_left, sm_scale, plan, err);
        return stage(h, plan, rc, err, workspace, workspace_bytes, stream);
    });
}

static pkv_status check_planned(pkv_latent_t h, const void *ws, bool dense) {
    if (!h) return PKV_ERR_INVALID;
    if (!h->planned_ws || h->planned_ws != ws)
        return fail(h, PKV_ERR_NOT_PLANNED, "no plan was made on this workspace by this handle");
    if (h->plan.dense != dense) return fail(h, PKV_ERR_NOT_PLANNED, "the workspace holds a plan of the other form");
    return PKV_OK;
}

extern "C" pkv_status pkv_latent_append_planned(pkv_latent_t h, const void *c_new, int64_t c_stride,
                                                const void *rope_new, int64_t rope_stride, void *cache_layer,
                                                void *workspace, pkv_stream_t stream) {
    return guarded(h, [&]() -> pkv_status {
        pkv_status st = check_planned(h, workspace, false);
        if (st != PKV_OK) return st;
        NvtxCall range(h->nvtx, "pkv_latent_append_planned");
        if (h->plan.num_append == 0) return PKV_OK;
        if (!c_new || !rope_new || !cache_layer) return fail(h, PKV_ERR_INVALID, "null c_new, rope_new or cache_layer");
        if ((bits(c_new) | bits(rope_new) | bits(cache_layer)) % 16)
            return fail(h, PKV_ERR_INVALID, "c_new, rope_new and cache_layer must be 16-byte aligned");
        if (c_stride % 8 || rope_stride % 8 || c_stride < pkv::kLatentDim || rope_stride < pkv::kLatentRope)
            return fail(h, PKV_ERR_INVALID, "row strides are multiples of 8 elements and at least the width");
        const cudaError_t e = pkv::launch_latent_append(h->shape, h->plan, workspace, c_new, c_stride, rope_new,
                                                        rope_stride, cache_layer, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? PKV_OK : cuda_fail(h, e, "latent append launch");
    });
}

// Tensor map over a bf16 tensor of `rank` dims (innermost first; strides in elements of dims 1..) with
// boxes of 64 columns x box_rows of dim 1 x box_outer of dim 2, 128-byte swizzle.
static pkv_status encode(pkv_latent_t h, const void *base, int rank, const long long *dims, const long long *strides,
                         int box_rows, CUtensorMap *tm, int box_outer = 1) {
    auto fn = pkv::encode_fn();
    if (!fn) return fail(h, PKV_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    cuuint64_t d[3], st[2];
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_outer}, es[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) d[i] = (cuuint64_t)dims[i];
    for (int i = 0; i + 1 < rank; ++i) st[i] = (cuuint64_t)strides[i] * 2;
    const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), d, st, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(h, PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")");
    return PKV_OK;
}

extern "C" pkv_status pkv_latent_run(pkv_latent_t h, const void *q, const void *cache_layer, void *out, float *lse,
                                     void *workspace, pkv_stream_t stream) {
    return guarded(h, [&]() -> pkv_status {
        pkv_status st = check_planned(h, workspace, false);
        if (st != PKV_OK) return st;
        NvtxCall range(h->nvtx, "pkv_latent_run");
        if (h->plan.num_tokens == 0) return PKV_OK;
        if (!q || !cache_layer || !out) return fail(h, PKV_ERR_INVALID, "null q, cache_layer or out");
        if ((bits(q) | bits(cache_layer) | bits(out)) % 16 || bits(lse) % 4)
            return fail(h, PKV_ERR_INVALID, "q, cache_layer and out must be 16-byte aligned (lse 4-byte)");
        const LatentShape &s = h->shape;
        CUtensorMap tc, tq;
        const long long cd[3] = {64, (long long)s.num_cache_pages * s.page_size, pkv::kLatentWidth / 64};
        const long long cs[2] = {pkv::kLatentWidth, 64};
        const long long qd[2] = {pkv::kLatentWidth, (long long)h->plan.num_tokens * s.num_heads};
        const long long stride[1] = {pkv::kLatentWidth};
        if ((st = encode(h, cache_layer, 3, cd, cs, s.box_rows(), &tc, s.box_chunks())) != PKV_OK) return st;
        if ((st = encode(h, q, 2, qd, stride, h->plan.box_q, &tq)) != PKV_OK) return st;
        const cudaError_t e =
            pkv::launch_latent(s, h->plan, tc, tq, workspace, out, lse, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? PKV_OK : cuda_fail(h, e, "latent launch");
    });
}

extern "C" pkv_status pkv_latent_plan_dense(pkv_latent_t h, const int32_t *cu_q, const int32_t *cu_k, int batch,
                                            int causal, int window_left, float sm_scale, void *workspace,
                                            size_t workspace_bytes, pkv_stream_t stream) {
    if (!h) return PKV_ERR_INVALID;
    NvtxCall range(h->nvtx, "pkv_latent_plan_dense");
    return guarded(h, [&]() -> pkv_status {
        pkv_status st = check_ws(h, workspace);
        if (st != PKV_OK) return st;
        std::string err;
        LatentPlan plan;
        plan.image.swap(h->spare_image);
        const int rc =
            pkv::make_latent_dense_plan(h->shape, cu_q, cu_k, batch, causal, window_left, sm_scale, plan, err);
        return stage(h, plan, rc, err, workspace, workspace_bytes, stream);
    });
}

extern "C" pkv_status pkv_latent_run_dense(pkv_latent_t h, const void *q, const void *k_nope, int64_t kn_token_stride,
                                           int64_t kn_head_stride, const void *k_rope, int64_t kr_token_stride,
                                           const void *v, int64_t v_token_stride, int64_t v_head_stride, void *out,
                                           float *lse, void *workspace, pkv_stream_t stream) {
    return guarded(h, [&]() -> pkv_status {
        pkv_status st = check_planned(h, workspace, true);
        if (st != PKV_OK) return st;
        NvtxCall range(h->nvtx, "pkv_latent_run_dense");
        if (h->plan.num_tokens == 0) return PKV_OK;
        if (!q || !k_nope || !k_rope || !v || !out) return fail(h, PKV_ERR_INVALID, "null q, k_nope, k_rope, v or out");
        if ((bits(q) | bits(k_nope) | bits(k_rope) | bits(v) | bits(out)) % 16 || bits(lse) % 4)
            return fail(h, PKV_ERR_INVALID, "q, k_nope, k_rope, v and out must be 16-byte aligned (lse 4-byte)");
        const int64_t strides[] = {kn_token_stride, kn_head_stride, kr_token_stride, v_token_stride, v_head_stride};
        const int64_t least[] = {pkv::kLatentNope, pkv::kLatentNope, pkv::kLatentRope, pkv::kLatentV, pkv::kLatentV};
        for (int i = 0; i < 5; ++i)
            if (strides[i] < least[i] || strides[i] % 8 || strides[i] >= (1ll << 38))
                return fail(h, PKV_ERR_INVALID, "strides are multiples of 8 elements and at least the width stepped over");
        const long long H = h->shape.num_heads, T = h->plan.num_tokens, K = h->plan.num_keys;
        constexpr long long QW = pkv::kLatentNope + pkv::kLatentRope;
        CUtensorMap tq, tk, tr, tv;
        const long long qd[3] = {QW, T, H}, qs[2] = {H * QW, QW};
        const long long kd[3] = {pkv::kLatentNope, K, H}, ks[2] = {kn_token_stride, kn_head_stride};
        const long long rd[2] = {pkv::kLatentRope, K}, rs[1] = {kr_token_stride};
        const long long vd[3] = {pkv::kLatentV, K, H}, vs[2] = {v_token_stride, v_head_stride};
        if ((st = encode(h, q, 3, qd, qs, 128, &tq)) != PKV_OK) return st;
        if ((st = encode(h, k_nope, 3, kd, ks, 64, &tk)) != PKV_OK) return st;
        if ((st = encode(h, k_rope, 2, rd, rs, 64, &tr)) != PKV_OK) return st;
        if ((st = encode(h, v, 3, vd, vs, 64, &tv)) != PKV_OK) return st;
        const cudaError_t e = pkv::launch_latent_dense(h->shape, h->plan, tq, tk, tr, tv, workspace, out, lse,
                                                       static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? PKV_OK : cuda_fail(h, e, "expanded latent launch");
    });
}

extern "C" pkv_status pkv_latent_check_device_error(pkv_latent_t h, void *workspace, pkv_stream_t stream, int *code) {
    return guarded(h, [&]() -> pkv_status {
        if (!h || !workspace || !code) return fail(h, PKV_ERR_INVALID, "null argument");
        if (h->planned_ws != workspace) return fail(h, PKV_ERR_NOT_PLANNED, "no plan on this workspace");
        NvtxCall range(h->nvtx, "pkv_latent_check_device_error");
        int v = 0;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        cudaError_t e = cudaMemcpyAsync(&v, workspace, sizeof(int), cudaMemcpyDeviceToHost, s);  // the header's first word
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        if (e != cudaSuccess) return cuda_fail(h, e, "error word read");
        *code = v;
        if (!v) return PKV_OK;
        const int zero = 0;
        e = cudaMemcpyAsync(workspace, &zero, sizeof(int), cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        if (e != cudaSuccess) return cuda_fail(h, e, "error word reset");
        return fail(h, PKV_ERR_DEVICE, "a kernel gave up waiting (device error " + std::to_string(v) + ")");
    });
}
