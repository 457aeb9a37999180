// The decode pass's launchers (the kernel is in decode_kernel.cuh), the split-KV merge, and the
// last-page append.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "decode_kernel.cuh"

namespace pkv {
namespace dev {

// Merge the split-KV partials of each cut row after the decode kernel: with
// w_j = exp(lse_j - max lse), o = sum_j w_j o_j / sum_j w_j and
// lse = max lse + ln sum_j w_j.  One warp per (cut row, q head), eight to a CTA: lane j
// holds piece j's lse, and every lane requests its D/32 columns of the row's first B pieces
// together with the lse values, before the weights are known, so that a row of up to B pieces
// costs one round trip to L2 after its MergeRow; longer rows take one more per B pieces (each
// batch's loads issued together).  B pieces hold B * D/32 registers: the small instance
// (64) keeps enough warps resident for the many rows of a batch, the large one (128) takes
// the rows of many pieces of long contexts in one batch.
constexpr int kMergeWarps = 8;
constexpr int merge_batch(int D, bool large) {
    return (large ? 128 : 64) / (D / 32) < 32 ? (large ? 128 : 64) / (D / 32) : 32;
}

template <int D, int B>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const PlanHeader *hdr, const MergeRow *rows,
                                                                 const float *part_o, const float *part_lse,
                                                                 __nv_bfloat16 *out, float *lse, int Hq) {
    constexpr int C = D / 32;  // columns per lane: 2, 4 or 8
    static_assert(B >= 1 && B <= 32, "a batch's weights come from one lane each");
    const int lane = threadIdx.x & 31;
    const long long u = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    const int m = (int)(u / Hq), h = (int)(u % Hq);
    // the plan's own values (copied before the decode launch) are read before waiting for the
    // decode kernel; the partials it writes only after
    const bool active = m < hdr->num_merge;
    MergeRow mr{};
    if (active) mr = rows[m];
    griddep_wait();
    griddep_launch();
    if (!active || mr.out_token < 0) return;
    const int count = mr.count;
    const float *lse_of = part_lse + (size_t)mr.first * Hq + h;              // piece j at lse_of[j * Hq]
    const float *o_of = part_o + ((size_t)mr.first * Hq + h) * D + lane * C;  // piece j at o_of[j * Hq * D]
    auto load = [&](float (&dst)[C], int j) { load_cols<C>(dst, o_of + (size_t)j * Hq * D); };
    const float lj = lane < count ? __ldcg(lse_of + (size_t)lane * Hq) : -INFINITY;
    float x[B][C];
#pragma unroll
    for (int j = 0; j < B; ++j)
        if (j < count) load(x[j], j);
    // M = max_j lse_j and sum_j w_j over the warp (pieces past 32: one more lse each per lane)
    float M = lj;
    for (int j = lane + 32; j < count; j += 32) M = fmaxf(M, __ldcg(lse_of + (size_t)j * Hq));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float wl = lane < count ? __expf(lj - M) : 0.f;
    float sum = wl;
    for (int j = lane + 32; j < count; j += 32) sum += __expf(__ldcg(lse_of + (size_t)j * Hq) - M);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    for (int j0 = 0;;) {
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const float w0 = __shfl_sync(0xffffffffu, wl, (j0 + j) & 31);
            if (j0 + j < count) {
                const float w = j0 + j < 32 ? w0 : __expf(__ldcg(lse_of + (size_t)(j0 + j) * Hq) - M);
#pragma unroll
                for (int c = 0; c < C; ++c) acc[c] += w * x[j][c];
            }
        }
        j0 += B;
        if (j0 >= count) break;
#pragma unroll
        for (int j = 0; j < B; ++j)  // the next batch (rows of many pieces)
            if (j0 + j < count) load(x[j], j0 + j);
    }
    const float inv = 1.f / sum;
    uint32_t packed[C / 2];
#pragma unroll
    for (int c = 0; c < C; c += 2) packed[c / 2] = pack_bf16(acc[c] * inv, acc[c + 1] * inv);
    __nv_bfloat16 *dst = out + ((size_t)mr.out_token * Hq + h) * D + lane * C;
    if constexpr (C == 2) {
        *reinterpret_cast<uint32_t *>(dst) = packed[0];
    } else if constexpr (C == 4) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(packed[0], packed[1]);
    } else {
        *reinterpret_cast<uint4 *>(dst) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
    }
    if (lse && lane == 0) lse[(size_t)mr.out_token * Hq + h] = M + __logf(sum);
}


// Last-page append: one thread per 16-byte chunk of a new token's K and V rows (num_kv_heads
// x D bf16 each), all chunks in flight at once, written to slot rows[t] of the layer slice
// viewed as [pages * 2 * page_size] rows (V rows page_size further).
__global__ void __launch_bounds__(256) append_kernel(const PlanHeader *hdr, const uint4 *k, const uint4 *v, uint4 *cache,
                                                     const int32_t *rows, int vec_per_token, int page_size) {
    griddep_wait();
    griddep_launch();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int t = (int)(i / vec_per_token), c = (int)(i % vec_per_token);
    if (t >= hdr->num_append) return;
    const size_t row = (size_t)rows[t];
    const uint4 kk = k[(size_t)t * vec_per_token + c];
    const uint4 vv = v[(size_t)t * vec_per_token + c];
    cache[row * vec_per_token + c] = kk;
    cache[(row + page_size) * vec_per_token + c] = vv;
}

// Last-page append straight from the DEVICE index arrays (no plan): one thread per 16-byte
// chunk of a new token's K and V rows.  Token t belongs to the row r with qo_indptr[r] <=
// t < qo_indptr[r+1] (row t when qo_indptr is null: one token per row), sits at position
// p = L_r - n_r + (t - qo_indptr[r]) of that row and lands in page
// kv_indices[kv_indptr[r] + p / page_size] at slot p % page_size.  The arrays were not seen
// by the host, so every index is checked before it is used: a token whose row arrays are
// inconsistent (non-monotone offsets, a fill outside 1..page_size, a position outside the
// row, a page id outside the cache) is not written, and nothing is read or written out of
// bounds.
__global__ void __launch_bounds__(256)
    append_indexed_kernel(const uint4 *k, const uint4 *v, uint4 *cache, const int32_t *qo_indptr,
                          const int32_t *kv_indptr, const int32_t *kv_indices, const int32_t *last_page_len, int batch,
                          int num_tokens, int vec_per_token, int page_size, int page_shift, int num_cache_pages) {
    griddep_wait();
    griddep_launch();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int t = (int)(i / vec_per_token), c = (int)(i % vec_per_token);
    if (t >= num_tokens) return;
    int r, n, first;
    if (qo_indptr) {
        if (t >= __ldg(qo_indptr + batch)) return;
        int lo = 0, hi = batch - 1;  // the last row whose offset is <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(qo_indptr + mid) <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        r = lo;
        first = __ldg(qo_indptr + r);
        n = __ldg(qo_indptr + r + 1) - first;
        if (first > t || t >= first + n) return;
    } else {
        if (t >= batch) return;
        r = t;
        first = t;
        n = 1;
    }
    const int kb = __ldg(kv_indptr + r), ke = __ldg(kv_indptr + r + 1), nnz = __ldg(kv_indptr + batch);
    const int fill = __ldg(last_page_len + r);
    if (kb < 0 || ke <= kb || ke > nnz || fill < 1 || fill > page_size) return;
    const long long L = (long long)(ke - kb - 1) * page_size + fill;
    const long long p = L - n + (t - first);
    if (p < 0 || p >= L) return;
    const int page = __ldg(kv_indices + kb + (int)(p >> page_shift));
    if (page < 0 || page >= num_cache_pages) return;
    const size_t row = (size_t)page * 2 * page_size + (size_t)(p & (page_size - 1));
    const uint4 kk = k[(size_t)t * vec_per_token + c];
    const uint4 vv = v[(size_t)t * vec_per_token + c];
    cache[row * vec_per_token + c] = kk;
    cache[(row + page_size) * vec_per_token + c] = vv;
}

// Gather of a frozen prefix (DenseAttentionManager): one warp per position t copies
// K and V of slot t % page_size of page pages[t / page_size] to row t of k_out / v_out.
__global__ void __launch_bounds__(256) gather_kernel(const uint4 *cache, const int32_t *pages, int num_tokens,
                                                     int vec_per_token, int page_size, uint4 *k_out, uint4 *v_out) {
    griddep_wait();
    griddep_launch();
    const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= num_tokens) return;
    const size_t row = (size_t)pages[t / page_size] * 2 * page_size + t % page_size;
    const int lane = threadIdx.x & 31;
    const uint4 *ks = cache + row * vec_per_token;
    const uint4 *vs = cache + (row + page_size) * vec_per_token;
    uint4 *kd = k_out + (size_t)t * vec_per_token;
    uint4 *vd = v_out + (size_t)t * vec_per_token;
    for (int i = lane; i < vec_per_token; i += 32) {
        kd[i] = ks[i];
        vd[i] = vs[i];
    }
}

// Self-test of the device error path: one thread waits, with `polls` polls, on an mbarrier
// nothing ever arrives on; the wait gives up, records kErrWaitSelfTest in the plan's error
// word and the kernel returns (no fault, no hang, the context stays usable).
__global__ void __launch_bounds__(32) selftest_wait_kernel(PlanHeader *hdr, uint32_t polls) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
        mbar_wait(&bar, 0, &hdr->err, kErrWaitSelfTest, polls);
    }
}

}  // namespace dev

cudaError_t launch_selftest_wait(const Plan &p, void *ws, uint32_t polls, cudaStream_t st) {
    dev::selftest_wait_kernel<<<1, 32, 0, st>>>(
        reinterpret_cast<PlanHeader *>(static_cast<uint8_t *>(ws) + p.lay.err), polls);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------------
// launchers

cudaError_t launch_gather(const Shape &s, const void *kv_layer, const int32_t *pages, int num_tokens, void *k_out,
                          void *v_out, cudaStream_t st) {
    if (num_tokens <= 0) return cudaSuccess;
    const int vec = s.num_kv_heads * s.head_dim * 2 / 16;
    const int wpb = 8;
    return launch_pdl(dev::gather_kernel, dim3((num_tokens + wpb - 1) / wpb), dim3(wpb * 32), 0, st,
                      static_cast<const uint4 *>(kv_layer), pages, num_tokens, vec, s.page_size,
                      static_cast<uint4 *>(k_out), static_cast<uint4 *>(v_out));
}

static uint32_t decode_stage_bytes(const Shape &s) { return s.dec_stage_bytes(); }

int decode_stages(const Shape &s) {
    const uint32_t sb = decode_stage_bytes(s);
    int st = (int)(kDecodeRingBytes / (uint32_t)s.dec_ctas_per_sm() / sb);
    return st < 2 ? 0 : (st > dev::kDecodeMaxStages ? dev::kDecodeMaxStages : st);
}

size_t decode_smem_bytes(const Shape &s) {
    return 1024 + (size_t)decode_stages(s) * decode_stage_bytes(s) + 2 * 8 * dev::kDecodeMaxStages + 16;
}

// Raise a kernel's dynamic shared-memory limit; skipped while `st` is being captured
// into a CUDA graph (a launch before the capture has set it already).
cudaError_t set_smem_limit(const void *fn, size_t smem, cudaStream_t st) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cs) == cudaSuccess && cs != cudaStreamCaptureStatusNone) return cudaSuccess;
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

bool decode_args(const Shape &s, const Plan &p, void *ws, const void *q, void *kv_layer, void *out, float *lse,
                 const void *k_new, const void *v_new, dev::DecodeArgs &a) {
    uint8_t *w = static_cast<uint8_t *>(ws);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.tiles = reinterpret_cast<const DecodeTile *>(w + p.lay.dec_tiles);
    a.cta_ptr = reinterpret_cast<const int32_t *>(w + p.lay.dec_cta_ptr);
    a.cta_rows = reinterpret_cast<const int32_t *>(w + p.lay.dec_cta_rows);
    a.pages = reinterpret_cast<const int32_t *>(w + p.lay.dec_pages);
    a.part_o = reinterpret_cast<float *>(w + p.lay.part_o);
    a.part_lse = reinterpret_cast<float *>(w + p.lay.part_lse);
    a.hdr = reinterpret_cast<PlanHeader *>(w + p.lay.err);
    a.k_new = static_cast<const uint4 *>(k_new);
    a.v_new = static_cast<const uint4 *>(v_new);
    a.kv_layer = static_cast<uint4 *>(kv_layer);
    a.append_rows = reinterpret_cast<const int32_t *>(w + p.lay.append_rows);
    a.num_qo_heads = s.num_qo_heads;
    a.num_kv_heads = s.num_kv_heads;
    a.heads = s.dec_heads();
    a.page_size = s.page_size;
    a.page_shift = s.page_shift();
    a.box_rows = s.dec_box_rows();
    a.kpb_shift = __builtin_ctz((unsigned)s.dec_keys_per_box());
    a.gather = s.dec_gather() ? 1 : 0;
    a.kv_in_box = s.dec_kv_in_box() ? 1 : 0;
    a.producers = s.dec_producer_warps();
    a.box_stride = s.dec_box_stride();
    a.stages = decode_stages(s);
    a.stage_bytes = decode_stage_bytes(s);
    a.logits = nullptr;
    a.logit_stride = 0;
    return a.stages != 0;
}

cudaError_t launch_decode(const Shape &s, const Plan &p, const CUtensorMap &tm, void *ws, const void *q,
                          void *kv_layer, void *out, float *lse, cudaStream_t st, const void *k_new,
                          const void *v_new) {
    const int grid = s.graph_static ? static_counts(s, p.mode).dec_ctas : p.dec_ctas;
    if (grid == 0) return cudaSuccess;
    dev::DecodeArgs a;
    if (!decode_args(s, p, ws, q, kv_layer, out, lse, k_new, v_new, a)) return cudaErrorInvalidValue;
    const int warps = a.heads + a.producers;
    const size_t smem = decode_smem_bytes(s);
    cudaError_t e = cudaErrorInvalidValue;
    const int g = s.group();
#define PKV_DEC(DD, GG)                                                                                  \
    if (s.head_dim == DD && g == GG)                                                                      \
        e = s.page_size < 16                                                                               \
                ? launch_decode_t<DD, GG, true, false>(tm, a, dim3(grid, s.dec_head_groups()), warps, smem, st)          \
                : launch_decode_t<DD, GG, false, false>(tm, a, dim3(grid, s.dec_head_groups()), warps, smem, st);
    PKV_FOR_EACH_HEAD_DIM_AND_GROUP(PKV_DEC)
#undef PKV_DEC
    return e == cudaSuccess ? launch_decode_merge(s, p, ws, a, st) : e;
}

cudaError_t launch_decode_merge(const Shape &s, const Plan &p, void *ws, const dev::DecodeArgs &a, cudaStream_t st) {
    uint8_t *w = static_cast<uint8_t *>(ws);
    cudaError_t e = cudaSuccess;
    // the merge of the rows cut into several pieces (graph mode always launches it at the
    // maxima; its warps past the plan's cut rows return at once)
    const int merges = s.graph_static ? static_counts(s, p.mode).num_merge : p.num_merge;
    if (merges) {
        const long long warps = (long long)merges * s.num_qo_heads;
        const dim3 mgrid((unsigned)((warps + dev::kMergeWarps - 1) / dev::kMergeWarps));
        // the large batch for rows of more pieces than the small one holds (graph mode, whose
        // launch serves every later plan, keeps the small one)
        const bool large = !s.graph_static && p.max_pieces > dev::merge_batch(s.head_dim, false);
        using dev::merge_batch;
        auto mk = s.head_dim == 64    ? dev::merge_kernel<64, merge_batch(64, false)>
                  : s.head_dim == 128 ? (large ? dev::merge_kernel<128, merge_batch(128, true)>
                                               : dev::merge_kernel<128, merge_batch(128, false)>)
                                      : (large ? dev::merge_kernel<256, merge_batch(256, true)>
                                               : dev::merge_kernel<256, merge_batch(256, false)>);
        e = launch_pdl(mk, mgrid, dim3(dev::kMergeWarps * 32), 0, st, static_cast<const PlanHeader *>(a.hdr),
                       reinterpret_cast<const MergeRow *>(w + p.lay.merge_rows), static_cast<const float *>(a.part_o),
                       static_cast<const float *>(a.part_lse), a.out, a.lse, s.num_qo_heads);
    }
    return e;
}

cudaError_t launch_append(const Shape &s, const Plan &p, void *ws, const void *k, const void *v, void *kv_layer,
                          cudaStream_t st) {
    const int tokens = s.graph_static ? static_counts(s, p.mode).tokens : p.num_append;
    if (tokens == 0) return cudaSuccess;
    uint8_t *w = static_cast<uint8_t *>(ws);
    const int vec = s.num_kv_heads * s.head_dim * 2 / 16;
    const long long chunks = (long long)tokens * vec;
    const int grid = (int)((chunks + 255) / 256);
    return launch_pdl(dev::append_kernel, dim3(grid), dim3(256), 0, st,
                      reinterpret_cast<const PlanHeader *>(w + p.lay.err), static_cast<const uint4 *>(k),
                      static_cast<const uint4 *>(v), static_cast<uint4 *>(kv_layer),
                      reinterpret_cast<const int32_t *>(w + p.lay.append_rows), vec, s.page_size);
}

cudaError_t launch_append_indexed(const Shape &s, const void *k, const void *v, int num_tokens, void *kv_layer,
                                  const int32_t *qo_indptr, const int32_t *kv_indptr, const int32_t *kv_indices,
                                  const int32_t *last_page_len, int batch, cudaStream_t st) {
    if (num_tokens == 0 || batch == 0) return cudaSuccess;
    const int vec = s.num_kv_heads * s.head_dim * 2 / 16;
    const long long chunks = (long long)num_tokens * vec;
    const int grid = (int)((chunks + 255) / 256);
    return launch_pdl(dev::append_indexed_kernel, dim3(grid), dim3(256), 0, st, static_cast<const uint4 *>(k),
                      static_cast<const uint4 *>(v), static_cast<uint4 *>(kv_layer), qo_indptr, kv_indptr, kv_indices,
                      last_page_len, batch, num_tokens, vec, s.page_size, s.page_shift(), s.num_cache_pages);
}

}  // namespace pkv

// ------------------------------------------------------------------------------------
// Scratch for callers that cannot allocate device memory (pkv_run_decode_static).
//
// The plan image and the split-KV partials of such a call live in this file-scope
// array instead of a caller workspace.  Every GPU that loads the library holds it until
// the process exits.  Host code must not use the array's name as an address: its
// device address is fetched once per device with cudaGetSymbolAddress.
namespace pkv {

constexpr size_t kStaticScratchBytes = size_t(16) << 20;  // 16 MiB

static __device__ __align__(256) uint8_t g_decode_scratch[kStaticScratchBytes];

size_t static_scratch_bytes() { return kStaticScratchBytes; }

// Device address of g_decode_scratch in the current device's context.  The first call in
// a context resolves it (with that device current) and caches it under the context's
// unique id; a later call in another context -- another device, or the same device after
// cudaDeviceReset made a new primary context -- resolves it again, so a cached address
// never outlives the context it belongs to.
namespace {
using CtxGetCurrent = CUresult (*)(CUcontext *);
using CtxGetId = CUresult (*)(CUcontext, unsigned long long *);
template <typename F>
cudaError_t driver_fn(const char *name, F *out) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    cudaError_t e = cudaGetDriverEntryPointByVersion(name, &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorSymbolNotFound;
    *out = reinterpret_cast<F>(fn);
    return cudaSuccess;
}
}  // namespace

cudaError_t static_scratch(void **ptr) {
    static CtxGetCurrent ctx_get = nullptr;
    static CtxGetId ctx_id = nullptr;
    static std::mutex mu;
    static struct {
        unsigned long long id;
        void *addr;
    } cached[128] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!ctx_get && (e = driver_fn("cuCtxGetCurrent", &ctx_get)) != cudaSuccess) return e;
    if (!ctx_id && (e = driver_fn("cuCtxGetId", &ctx_id)) != cudaSuccess) return e;
    auto current_id = [&](unsigned long long *id) {
        CUcontext ctx = nullptr;
        return ctx_get(&ctx) == CUDA_SUCCESS && ctx && ctx_id(ctx, id) == CUDA_SUCCESS;
    };
    unsigned long long id = 0;
    if (current_id(&id) && cached[dev].addr && cached[dev].id == id) {
        *ptr = cached[dev].addr;
        return cudaSuccess;
    }
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_decode_scratch);  // makes the primary context current if needed
    if (e != cudaSuccess) return e;
    if (!current_id(&id)) return cudaErrorDeviceUninitialized;
    cached[dev].id = id;
    cached[dev].addr = p;
    *ptr = p;
    return cudaSuccess;
}

}  // namespace pkv
