// Softmax weights added up per key (pkv_run_weights, pkv_run_decode_weights):
//     w_j = sum over a row's queries i and heads h of exp(sm_scale q_ih k_j - lse_ih),
// summed in a fixed order, then scores[slot of j] = decay * old (or 0) + w_j.
//
// WEIGHTS plans: a CTA takes 128 keys of one row and goes through the kv heads and blocks of up to
// 128 query rows (tokens x the group's heads).  The product is taken transposed, S^T = K Q^T: keys are
// the 128 rows of the MMA and tensor-memory lanes, so a thread owns one key and adds up its weights
// over the queries in registers, with no reduction across lanes.  K is read once (one 64-column box
// per page run and head), Q blocks come from L2.  Few query rows: bounded by K's bytes; many: by the
// exponentials (16 per cycle and SM, 1,024 cycles a block, against 512 of its MMAs at head_dim 128).
// With fewer tiles than SMs the kv heads are shared out over several CTAs (hsplit), whose sums the
// finishing kernel adds in order.
//
// DECODE_WEIGHTS plans: the decode kernel has left its logits; a thread per key adds the weights.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "evict.h"
#include "launch.h"
#include "tcgen05.cuh"

namespace pkv {
namespace dev {

constexpr int kWtThreads = 192;  // warps 0-3: a key a thread; 4: copies; 5: MMAs
constexpr float kWtLog2e = 1.4426950408889634f;

template <int D>
struct WtSmem {
    static constexpr int CHUNKS = D / 64;
    static constexpr uint32_t CHUNK = 128 * 128;  // 128 rows x 64 columns
    static constexpr uint32_t TILE = CHUNKS * CHUNK;
    static constexpr int KS = D == 256 ? 1 : 2, QS = 2;
    static constexpr uint32_t K_OFF = 0;
    static constexpr uint32_t Q_OFF = KS * TILE;
    static constexpr uint32_t BAR_OFF = Q_OFF + QS * TILE;
    static constexpr uint32_t COL_OFF = BAR_OFF + 256;      // per block column: lse (base 2), first and last key
    static constexpr uint32_t BYTES = COL_OFF + 2 * 3 * 128 * 4;
};
static_assert(1024 + WtSmem<256>::BYTES <= 227 * 1024, "the weights kernel fits shared memory");

struct WeightsArgs {
    const WeightsTile *tiles;
    const int32_t *pages;
    PlanHeader *hdr;
    const float *lse;
    float *part;  // [hsplit][tiles][128]
    int num_qo_heads, group, heads_per_cta, num_tiles;
    int page_size, page_shift, box_rows, box_tokens, oob_row;
};

template <int D>
__global__ void __launch_bounds__(kWtThreads)
    weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                   const WeightsArgs a) {
    using L = WtSmem<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR_OFF);
    uint64_t *k_full = bars + 0, *k_empty = bars + 2, *q_full = bars + 4, *q_empty = bars + 6;  // [2] each
    uint64_t *s_full = bars + 8, *s_empty = bars + 10;                                          // [2] each
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 12);
    float *cols = reinterpret_cast<float *>(sm + L::COL_OFF);

    const WeightsTile t = a.tiles[blockIdx.x];
    int *const err = &a.hdr->err;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = a.page_size, G = a.group;
    const int causal = a.hdr->causal, window = a.hdr->window_left;
    // the row's tokens any of which may see a key of this tile, as blocks of box_tokens
    const int bt = a.box_tokens, pos0 = t.new_begin;  // token i sits at position pos0 + i
    const int i0 = causal ? max(0, t.key0 - pos0) : 0;
    const int i1 = window >= 0 ? (int)min((long long)t.n_q, (long long)t.key0 + kWeightKeys + window - pos0) : t.n_q;
    const int blocks = i1 > i0 ? (i1 - i0 + bt - 1) / bt : 0;
    const int h0 = blockIdx.y * a.heads_per_cta, nh = blocks ? a.heads_per_cta : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
            mbar_init(&s_full[s], 1);
            mbar_init(&s_empty[s], 4);
        }
        fence_barrier_init();
    }
    if (warp == 5) {
        tmem_alloc(tmem_holder, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch();
    const uint32_t tmem = *tmem_holder;

    if (warp == 4) {
        // ------------------------------------------------ copies
        const int R = a.box_rows, jobs = kWeightKeys / R * L::CHUNKS;  // a box is one page run of one chunk
        const int npages = (t.length + P - 1) >> a.page_shift;
        const uint32_t q_bytes = (uint32_t)(bt * G) * 128u * L::CHUNKS;
        if (lane == 0 && nh) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_q);
        }
        uint32_t it = 0;
        int hs = 0;  // heads whose K has been requested
        bool ok = true;
        for (int h = 0; h < nh && ok; ++h) {
            const int ks = h % L::KS;
            ok = h < L::KS || mbar_wait(&k_empty[ks], (h / L::KS - 1) & 1, err, kErrWaitEmpty);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            ++hs;
            if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], L::TILE);
            __syncwarp();
            for (int j = lane; j < jobs; j += 32) {
                const int b = j / L::CHUNKS, c = j % L::CHUNKS;
                const int kb = t.key0 + b * R, pg = kb >> a.page_shift;
                const int row = pg < npages ? a.pages[t.kv_base + pg] * 2 * P + (kb & (P - 1)) : a.oob_row;
                tma_load_3d(sm + L::K_OFF + ks * L::TILE + c * L::CHUNK + b * R * 128, &tm_k, &k_full[ks], c * 64, row,
                            h0 + h);
            }
            for (int b = 0; b < blocks; ++b, ++it) {
                const int s = it & 1;
                ok = it < 2 || mbar_wait(&q_empty[s], ((it >> 1) - 1) & 1, err, kErrWaitEmpty);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&q_full[s], q_bytes);
                    for (int c = 0; c < L::CHUNKS; ++c)
                        tma_load_3d(sm + L::Q_OFF + s * L::TILE + c * L::CHUNK, &tm_q, &q_full[s], c * 64, (h0 + h) * G,
                                    t.q_begin + i0 + b * bt);
                }
                __syncwarp();
            }
        }
        // copies in flight land before the CTA may end (they have, unless a wait gave up)
        for (int d = hs > L::KS ? hs - L::KS : 0; d < hs; ++d)
            mbar_wait(&k_full[d % L::KS], (d / L::KS) & 1, err, kErrWaitDrain);
        for (uint32_t d = it > 2 ? it - 2 : 0; d < it; ++d)
            mbar_wait(&q_full[d & 1], (d >> 1) & 1, err, kErrWaitDrain);
    } else if (warp == 5) {
        // ------------------------------------------------ S^T = K Q^T
        const int ncol = (bt * G + 15) & ~15;
        const uint32_t id = idesc_bf16_f32(128, 16, 0, 0) - (16u >> 3 << 17) + ((uint32_t)(ncol >> 3) << 17);
        const uint64_t dK = smem_desc(smem_u32(sm + L::K_OFF), 16, 1024, kSwizzle128B);
        const uint64_t dQ = smem_desc(smem_u32(sm + L::Q_OFF), 16, 1024, kSwizzle128B);
        auto add = [](uint64_t d, uint32_t off) { return d + (off >> 4); };
        uint32_t it = 0;
        bool ok = true;
        for (int h = 0; h < nh && ok; ++h) {
            const int ks = h % L::KS;
            ok = mbar_wait(&k_full[ks], (h / L::KS) & 1, err, kErrWaitFull);
            for (int b = 0; b < blocks && ok; ++b, ++it) {
                const int s = it & 1;
                ok = mbar_wait(&q_full[s], (it >> 1) & 1, err, kErrWaitFull) &&
                     (it < 2 || mbar_wait(&s_empty[s], ((it >> 1) - 1) & 1, err, kErrWaitEmpty));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk / 4) * L::CHUNK + (kk % 4) * 32;
                    mma_ss_elect(tmem + 128u * s, add(dK, ks * L::TILE + off), add(dQ, s * L::TILE + off), id, kk > 0);
                }
                mma_commit_elect(&q_empty[s]);
                mma_commit_elect(&s_full[s]);
            }
            if (ok) mma_commit_elect(&k_empty[ks]);
        }
        if (!ok)  // a wait gave up: let the MMAs in flight finish before the tensor memory is released
            for (uint32_t i = 0; i < 1024; ++i) __nanosleep(1000);
    } else {
        // ------------------------------------------------ a key a thread
        const int m = threadIdx.x;  // 0..127: key, and the block column whose lse this thread fetches
        const int key = t.key0 + m;
        const float sl = a.hdr->scale_log2;
        float total = 0.f;
        uint32_t it = 0;
        bool ok = true;
        auto fetch = [&](int h, int b, float &ls, int &lo, int &hi) {
            const int i = i0 + b * bt + m / G;
            const bool valid = m < bt * G && i < i1;
            const int pos = pos0 + i;
            ls = valid ? a.lse[(size_t)(t.q_begin + i) * a.num_qo_heads + (h0 + h) * G + m % G] * kWtLog2e : 0.f;
            lo = window >= 0 ? max(0, pos - window) : 0;
            hi = valid ? (causal ? pos : t.length - 1) : -1;
        };
        float ls;
        int lo, hi;
        if (nh) fetch(0, 0, ls, lo, hi);
        // a wait that gives up clears ok; the warps still walk their blocks, without further waits, so
        // that they keep meeting at their barrier (which has no time limit)
        for (int h = 0; h < nh; ++h) {
            for (int b = 0; b < blocks; ++b, ++it) {
                const int s = it & 1;
                float *c_ls = cols + s * 384;
                int *c_lo = reinterpret_cast<int *>(c_ls) + 128, *c_hi = c_lo + 128;
                c_ls[m] = ls;
                c_lo[m] = lo;
                c_hi[m] = hi;
                // every column of the block sees every key of the tile: no masks
                const int ncols = min(bt, i1 - i0 - b * bt) * G;
                const bool mine = m >= ncols || (lo <= t.key0 && hi >= t.key0 + kWeightKeys - 1);
                unsigned all;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\t"
                             "selp.u32 %0, 1, 0, q;\n\t}"
                             : "=r"(all)
                             : "r"((unsigned)mine)
                             : "memory");
                if (b + 1 < blocks)
                    fetch(h, b + 1, ls, lo, hi);
                else if (h + 1 < nh)
                    fetch(h + 1, 0, ls, lo, hi);
                ok = ok && mbar_wait(&s_full[s], (it >> 1) & 1, err, kErrWaitFull);
                __syncwarp();
                tc_fence_after();
                float a4[4] = {0.f, 0.f, 0.f, 0.f};
                for (int c0 = 0; c0 < ncols; c0 += 32) {
                    uint32_t r[32];
                    tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16) + 128u * s + c0, r);
                    tmem_wait_ld();
                    if (all && c0 + 32 <= ncols) {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            a4[c & 3] += ex2_ftz(fmaf(__uint_as_float(r[c]), sl, -c_ls[c0 + c]));
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const bool sees = c0 + c < ncols && key >= c_lo[c0 + c] && key <= c_hi[c0 + c];
                            a4[c & 3] += sees ? ex2_ftz(fmaf(__uint_as_float(r[c]), sl, -c_ls[c0 + c])) : 0.f;
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[s]);
                total += (a4[0] + a4[1]) + (a4[2] + a4[3]);
            }
        }
        a.part[((size_t)blockIdx.y * a.num_tiles + blockIdx.x) * kWeightKeys + m] = total;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, 256);
}

__device__ __forceinline__ void put_score(const WeightsTile &t, const int32_t *pages, int page_size, int page_shift, int key,
                                          float w, float *scores, float decay) {
    const size_t slot = (size_t)pages[t.kv_base + (key >> page_shift)] * page_size + (key & (page_size - 1));
    scores[slot] = (decay != 0.f && key < t.new_begin ? decay * scores[slot] : 0.f) + w;
}

__global__ void __launch_bounds__(kWeightKeys) weights_finish_kernel(const WeightsTile *tiles, const int32_t *pages,
                                                                     const float *part, int hsplit, int page_size,
                                                                     int page_shift, float *scores, float decay) {
    const WeightsTile t = tiles[blockIdx.x];
    const int key = t.key0 + threadIdx.x;
    griddep_wait();
    griddep_launch();
    if (key >= t.length) return;
    float w = 0.f;
    for (int h = 0; h < hsplit; ++h) w += __ldcg(part + ((size_t)h * gridDim.x + blockIdx.x) * kWeightKeys + threadIdx.x);
    put_score(t, pages, page_size, page_shift, key, w, scores, decay);
}

// A thread per key: the logits of one head lie key by key, so a warp reads 128 consecutive bytes a
// head.  Four chains of sums, joined in a fixed order.
__global__ void __launch_bounds__(kWeightKeys) decode_scores_kernel(const WeightsTile *tiles, const int32_t *pages,
                                                                    const float *logits, long long logit_stride,
                                                                    const float *lse, int heads, int page_size,
                                                                    int page_shift, float *scores, float decay) {
    extern __shared__ float ls[];
    const WeightsTile t = tiles[blockIdx.x];
    const int key = t.key0 + threadIdx.x;
    griddep_wait();
    griddep_launch();
    for (int h = threadIdx.x; h < heads; h += kWeightKeys) ls[h] = lse[(size_t)t.q_begin * heads + h] * kWtLog2e;
    __syncthreads();
    if (key >= t.length) return;
    float a4[4] = {0.f, 0.f, 0.f, 0.f};
    if (key >= t.lo) {
        const float *lg = logits + (size_t)t.logit_base * 16 + key;
        int h = 0;
        for (; h + 8 <= heads; h += 8) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __ldcg(lg + (h + i) * logit_stride);
#pragma unroll
            for (int i = 0; i < 8; ++i) a4[i & 3] += ex2_ftz(x[i] - ls[h + i]);
        }
        for (; h < heads; ++h) a4[h & 3] += ex2_ftz(__ldcg(lg + h * logit_stride) - ls[h]);
    }
    put_score(t, pages, page_size, page_shift, key, (a4[0] + a4[1]) + (a4[2] + a4[3]), scores, decay);
}

}  // namespace dev

template <int D>
static cudaError_t launch_weights_t(const CUtensorMap &tk, const CUtensorMap &tq, const dev::WeightsArgs &a, dim3 grid,
                                    cudaStream_t st) {
    auto fn = dev::weights_kernel<D>;
    // at least 80 KB, so that no more than two CTAs (2 x 256 tensor-memory columns) share an SM
    const size_t need = 1024 + dev::WtSmem<D>::BYTES, smem = need < 80 * 1024 ? 80 * 1024 : need;
    cudaError_t e = set_smem_limit((const void *)fn, smem, st);
    return e == cudaSuccess ? launch_pdl(fn, grid, dim3(dev::kWtThreads), smem, st, tk, tq, a) : e;
}

cudaError_t launch_weights(const Shape &s, const Plan &p, const WeightsPlan &wp, const CUtensorMap &tm_k,
                           const CUtensorMap &tm_q, void *ws, const float *lse, float *scores, float decay,
                           cudaStream_t st) {
    (void)p;
    uint8_t *w = static_cast<uint8_t *>(ws);
    dev::WeightsArgs a;
    a.tiles = reinterpret_cast<const WeightsTile *>(w + wp.off_tiles);
    a.pages = reinterpret_cast<const int32_t *>(w + wp.off_pages);
    a.hdr = reinterpret_cast<PlanHeader *>(w);
    a.lse = lse;
    a.part = reinterpret_cast<float *>(w + wp.off_part);
    a.num_qo_heads = s.num_qo_heads;
    a.group = s.group();
    a.heads_per_cta = s.num_kv_heads / wp.hsplit;
    a.num_tiles = wp.tiles;
    a.page_size = s.page_size;
    a.page_shift = s.page_shift();
    a.box_rows = s.page_size < kWeightKeys ? s.page_size : kWeightKeys;
    a.box_tokens = wp.box_tokens;
    a.oob_row = s.num_cache_pages * 2 * s.page_size;
    const dim3 grid(wp.tiles, wp.hsplit);
    cudaError_t e = s.head_dim == 64    ? launch_weights_t<64>(tm_k, tm_q, a, grid, st)
                    : s.head_dim == 128 ? launch_weights_t<128>(tm_k, tm_q, a, grid, st)
                                        : launch_weights_t<256>(tm_k, tm_q, a, grid, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(dev::weights_finish_kernel, dim3(wp.tiles), dim3(kWeightKeys), 0, st, a.tiles, a.pages,
                      static_cast<const float *>(a.part), wp.hsplit, s.page_size, s.page_shift(), scores, decay);
}

cudaError_t launch_decode_scores(const Shape &s, const Plan &p, const WeightsPlan &wp, void *ws, const float *lse,
                                 float *scores, float decay, cudaStream_t st) {
    (void)p;
    if (wp.tiles == 0) return cudaSuccess;
    uint8_t *w = static_cast<uint8_t *>(ws);
    return launch_pdl(dev::decode_scores_kernel, dim3(wp.tiles), dim3(kWeightKeys), s.num_qo_heads * sizeof(float), st,
                      reinterpret_cast<const WeightsTile *>(w + wp.off_tiles),
                      reinterpret_cast<const int32_t *>(w + wp.off_pages),
                      reinterpret_cast<const float *>(w + wp.off_logits), wp.logit_stride, lse, s.num_qo_heads, s.page_size,
                      s.page_shift(), scores, decay);
}

}  // namespace pkv
