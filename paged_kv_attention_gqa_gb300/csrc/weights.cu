// Softmax weights added up per key (pkv_run_weights, pkv_run_decode_weights):
//     w_j = sum over a row's queries i and heads h of exp(sm_scale q_ih k_j - lse_ih),
// summed in a fixed order, then scores[slot of j] = decay * old (or 0) + w_j.
//
// WEIGHTS plans: the product is taken transposed, S^T = K Q^T: 128 keys are the rows of the MMA and
// tensor-memory lanes, so a thread owns a key and adds up its weights over a block's query rows (up to
// 128: tokens x the group's heads) in registers, with no reduction across lanes.  Three teams of four
// warps take the blocks in turn; four S buffers (all of tensor memory) let the MMAs run ahead of them.
// One CTA per SM walks items (kv heads or query blocks of one tile, planned to an eighth of an SM's
// share) with its rings running on across them; a team's sums of an item go to a part of their own, and
// the finishing kernel adds a tile's parts in order.  K is read once from HBM (two warps issue its
// copies: a page and 64 columns each, some 50 cycles an instruction), Q blocks come from L2.
//
// Measured (32 query heads on 8, head_dim 128): last 32 tokens of 8 rows of 1,999 to 16,381, 34 us, 23 of
// them K's bytes at the copy rate; two whole prompts of 2,003 tokens 49 us, 17 of operations.  The bound
// is the teams' work: some 900 cycles a block of 128 x 128 with all warps busy (512 of them the
// exponentials at 32 a cycle and SM), half as much again between two blocks of a team (its columns' lse,
// the barrier, the next fetch), which the other teams cover in part.  Before: two teams 35 / 52; with a
// block's head and number found by division and first and last key read per column 36 / 62; steps of 64
// columns (spilling registers) 40 / 67; an MMA warp a team 48 / 81; the lse as a k-step of the MMA 44 / 70.
//
// DECODE_WEIGHTS plans: the decode kernel has left its logits; a thread per key adds the weights.  64 rows
// of 517 to 8,190 tokens, 32 heads: 11 us for 36 MB of logits, most of them in L2 still, after 185 us of
// decode and join.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "evict.h"
#include "launch.h"
#include "tcgen05.cuh"

namespace pkv {
namespace dev {

// warps 0-11: the three teams, a key a thread; 12, 13: copies of K; 14: copies of Q; 15: MMAs
constexpr int kWtThreads = 128 * kWeightTeams + 128, kWtK = 4 * kWeightTeams, kWtQ = kWtK + 2, kWtMma = kWtK + 3;
constexpr int kWtProducers = 2;
constexpr float kWtLog2e = 1.4426950408889634f;

template <int D>
struct WtSmem {
    static constexpr int CHUNKS = D / 64;
    static constexpr uint32_t CHUNK = 128 * 128;  // 128 rows x 64 columns
    static constexpr uint32_t TILE = CHUNKS * CHUNK;
    static constexpr int KS = D == 256 ? 1 : 4, QS = 2;  // ring stages of K tiles and of Q blocks
    static constexpr uint32_t K_OFF = 0;
    static constexpr uint32_t Q_OFF = KS * TILE;
    static constexpr uint32_t BAR_OFF = Q_OFF + QS * TILE;
    static constexpr uint32_t COL_OFF = BAR_OFF + 256;  // -lse (base 2) of a block's columns: [team][buffer][128]
    static constexpr uint32_t BYTES = COL_OFF + kWeightTeams * 2 * 128 * 4;
};
static_assert(1024 + WtSmem<256>::BYTES <= 227 * 1024, "the weights kernel fits shared memory");
// A team's wait for its next block tells the two phases of that block's buffer apart because its last block
// used another of the four buffers, less than a turn before.
static_assert(kWeightTeams < 4, "a team's step is shorter than the ring of score buffers");

struct WeightsArgs {
    const WeightsItem *items;
    const int32_t *pages;
    PlanHeader *hdr;
    const float *lse;
    float *part;  // [item][team][128]
    int num_items, num_qo_heads, group;
    int page_size, page_shift, box_rows, box_tokens, oob_row;
};

// Add the weights of the block's `ncols` columns of this thread's key to acc: 2^(s sl - lse), with MASKED
// only of the columns [c_begin, c_end).  (Columns come 32 at a time; without MASKED ncols is a multiple.)
template <bool MASKED>
__device__ __forceinline__ void add_columns(uint64_t (&acc)[4], uint32_t s_lane, int ncols, uint64_t sl2, const float *c_ls,
                                            int c_begin, int c_end) {
#pragma unroll 1
    for (int c0 = 0; c0 < ncols; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(s_lane + c0, r);
        tmem_wait_ld();
        const ulonglong2 *ls2 = reinterpret_cast<const ulonglong2 *>(c_ls + c0);
        const int begin = c_begin - c0, end = c_end - c0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const ulonglong2 l = ls2[c];
            float x[4];
            f2_split(ffma2(f2_make(__uint_as_float(r[4 * c]), __uint_as_float(r[4 * c + 1])), sl2, l.x), x[0], x[1]);
            f2_split(ffma2(f2_make(__uint_as_float(r[4 * c + 2]), __uint_as_float(r[4 * c + 3])), sl2, l.y), x[2], x[3]);
            if constexpr (MASKED) {  // selects, not products: a masked score may be NaN
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = (4 * c + i >= begin) & (4 * c + i < end) ? x[i] : -INFINITY;
            }
            acc[(2 * c) & 3] = fadd2(acc[(2 * c) & 3], f2_make(ex2_ftz(x[0]), ex2_ftz(x[1])));
            acc[(2 * c + 1) & 3] = fadd2(acc[(2 * c + 1) & 3], f2_make(ex2_ftz(x[2]), ex2_ftz(x[3])));
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kWtThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                   const WeightsArgs a) {
    using L = WtSmem<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR_OFF);
    // K tiles are counted over the CTA's items (kc: one per item and head), blocks too (it)
    uint64_t *k_full = bars + 0, *k_empty = bars + 4;                                              // [KS] each
    uint64_t *q_full = bars + 8, *q_empty = bars + 10;  // [2] each
    uint64_t *s_full = bars + 12, *s_empty = bars + 16;  // [4] each: block it in S buffer it % 4
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 20);

    int *const err = &a.hdr->err;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = a.page_size, G = a.group, bt = a.box_tokens;
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::KS; ++s) {
            mbar_init(&k_full[s], kWtProducers);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_empty[s], 4);
        }
        fence_barrier_init();
    }
    if (warp == kWtMma) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch();
    const uint32_t tmem = *tmem_holder;

    if (warp == kWtK || warp == kWtK + 1) {
        // ------------------------------------------------ copies of K: a box is one page run of one chunk
        const int R = a.box_rows, jobs = kWeightKeys / R * L::CHUNKS;      // 1 to 64
        const int per = (jobs + kWtProducers - 1) / kWtProducers;           // at most 32 a warp, one a lane
        const int job = (warp - kWtK) * per + lane;
        const bool copies = lane < per && job < jobs;
        const uint32_t bytes = (uint32_t)max(0, min(per, jobs - (warp - kWtK) * per)) * R * 128u;
        if (warp == kWtK && lane == 0) prefetch_tmap(&tm_k);
        uint32_t kc = 0;
        bool ok = true;
        WeightsItem w = a.items[blockIdx.x];
        for (int n = blockIdx.x; n < a.num_items && ok; n += gridDim.x) {
            const int kb = w.key0 + job / L::CHUNKS * R, pg = kb >> a.page_shift;
            const int row = copies && pg < ((w.length + P - 1) >> a.page_shift)
                                ? a.pages[w.kv_base + pg] * 2 * P + (kb & (P - 1))
                                : a.oob_row;
            const WeightsItem next = a.items[min(n + (int)gridDim.x, a.num_items - 1)];  // lands meanwhile
            for (int h = 0; h < w.nh; ++h, ++kc) {
                const int ks = kc % L::KS;
                const uint32_t use = kc / L::KS;
                ok = use == 0 || mbar_wait(&k_empty[ks], (use - 1) & 1, err, kErrWaitEmpty);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], bytes);
                __syncwarp();
                if (copies)
                    tma_load_3d(sm + L::K_OFF + ks * L::TILE + job % L::CHUNKS * L::CHUNK + job / L::CHUNKS * R * 128, &tm_k,
                                &k_full[ks], job % L::CHUNKS * 64, row, w.h0 + h);
            }
            w = next;
        }
        // copies in flight land before the CTA may end (they have, unless a wait gave up)
        if (!ok)
            for (int s = 0; s < L::KS; ++s)
                for (int p = 0; p < 2; ++p) mbar_wait(&k_full[s], p, nullptr, 0, 1u << 16);
    } else if (warp == kWtQ) {
        // ------------------------------------------------ copies of Q blocks
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            const uint32_t bytes = (uint32_t)(bt * G) * 128u * L::CHUNKS;
            uint32_t it = 0;
            bool ok = true;
            WeightsItem w = a.items[blockIdx.x];
            for (int n = blockIdx.x; n < a.num_items && ok; n += gridDim.x) {
                const WeightsItem next = a.items[min(n + (int)gridDim.x, a.num_items - 1)];
                const int q_begin = w.q_begin + w.i0;
                for (int h = 0; h < w.nh && ok; ++h)
                    for (int b = 0; b < w.blocks; ++b, ++it) {
                        const int s = it & 1;
                        ok = it < 2 || mbar_wait(&q_empty[s], ((it >> 1) - 1) & 1, err, kErrWaitEmpty);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&q_full[s], bytes);
                        for (int c = 0; c < L::CHUNKS; ++c)
                            tma_load_3d(sm + L::Q_OFF + s * L::TILE + c * L::CHUNK, &tm_q, &q_full[s], c * 64,
                                        (w.h0 + h) * G, q_begin + b * bt);
                    }
                w = next;
            }
            if (!ok)
                for (int s = 0; s < 2; ++s)
                    for (int p = 0; p < 2; ++p) mbar_wait(&q_full[s], p, nullptr, 0, 1u << 16);
        }
    } else if (warp == kWtMma) {
        // ------------------------------------------------ S^T = K Q^T
        const uint32_t ncol = (uint32_t)(bt * G + 15) & ~15u;
        const uint32_t id = idesc_bf16_f32(128, 0, 0, 0) | ((ncol >> 3) << 17);
        const uint64_t dK = smem_desc(smem_u32(sm + L::K_OFF), 16, 1024, kSwizzle128B);
        const uint64_t dQ = smem_desc(smem_u32(sm + L::Q_OFF), 16, 1024, kSwizzle128B);
        auto add = [](uint64_t d, uint32_t off) { return d + (off >> 4); };
        uint32_t it = 0, kc = 0;
        bool ok = true;
        int nh = a.items[blockIdx.x].nh, blocks = a.items[blockIdx.x].blocks;
        for (int n = blockIdx.x; n < a.num_items && ok; n += gridDim.x) {
            const WeightsItem &next = a.items[min(n + (int)gridDim.x, a.num_items - 1)];
            const int next_nh = next.nh, next_blocks = next.blocks;
            for (int h = 0; h < nh && ok; ++h, ++kc) {
                const int ks = kc % L::KS;
                ok = mbar_wait(&k_full[ks], (kc / L::KS) & 1, err, kErrWaitFull);
                for (int b = 0; b < blocks && ok; ++b, ++it) {
                    const int s = it & 1, sb = it & 3;
                    ok = mbar_wait(&q_full[s], (it >> 1) & 1, err, kErrWaitFull) &&
                         (it < 4 || mbar_wait(&s_empty[sb], ((it >> 2) - 1) & 1, err, kErrWaitEmpty));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk / 4) * L::CHUNK + (kk % 4) * 32;
                        mma_ss_elect(tmem + 128u * sb, add(dK, ks * L::TILE + off), add(dQ, s * L::TILE + off), id, kk > 0);
                    }
                    mma_commit_elect(&q_empty[s]);
                    mma_commit_elect(&s_full[sb]);
                }
                if (ok) mma_commit_elect(&k_empty[ks]);
            }
            nh = next_nh;
            blocks = next_blocks;
        }
        if (!ok)  // a wait gave up: let the MMAs in flight finish before the tensor memory is released
            for (uint32_t i = 0; i < 1024; ++i) __nanosleep(1000);
    } else {
        // ------------------------------------------------ the teams: a key a thread
        const int team = warp >> 2, m = threadIdx.x & 127;  // the key, and the block column whose lse it fetches
        const uint32_t s_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float sl = a.hdr->scale_log2;
        const uint64_t sl2 = f2_make(sl, sl);
        const int causal = a.hdr->causal, window = a.hdr->window_left;
        const int m_tok = m / G, m_head = m % G;
        // a wait that gives up clears ok; the warps still walk their blocks, without further waits, so
        // that they keep meeting at their barriers (which have no time limit)
        bool ok = true;
        // The lse of column m of a block, fetched one block ahead and not touched before it is stored, so
        // that the fetch does not wait for it.
        float ls = 0.f;
        auto fetch = [&](const WeightsItem &w, int h, int b) {
            const int i = w.i0 + b * bt + m_tok;
            ls = 0.f;
            if (m < bt * G && i < w.i1) ls = a.lse[(size_t)(w.q_begin + i) * a.num_qo_heads + (w.h0 + h) * G + m_head];
        };
        // This team's blocks are every third one: (h, b) steps by three, past the item's end into the next
        // one.  (Counted, not divided: the divisions cost 500 cycles a block.)
        auto settle = [](const WeightsItem &w, int &h, int &b) {
            while (b >= w.blocks) {
                b -= w.blocks;
                ++h;
            }
        };
        WeightsItem w = a.items[blockIdx.x];
        uint32_t seq = 0, it = team;  // block of the CTA's whole run
        int h = 0, b = team;
        settle(w, h, b);
        if (h < w.nh) fetch(w, h, b);
        for (int n = blockIdx.x; n < a.num_items; n += gridDim.x) {
            const int key = w.key0 + m;
            const bool last = n + (int)gridDim.x >= a.num_items;
            const WeightsItem next = a.items[last ? n : n + (int)gridDim.x];  // lands meanwhile
            bool fetched = false;
            float total = 0.f;
            while (h < w.nh) {
                const int i_first = w.i0 + b * bt, i_count = min(bt, w.i1 - i_first);
                const int ncols = i_count * G, pos0 = w.new_begin + i_first;
                // every column of the block sees every key of the tile: no masks then
                const bool all = w.key0 + kWeightKeys <= w.length && (!causal || pos0 >= w.key0 + kWeightKeys - 1) &&
                                 (window < 0 || pos0 + i_count - 1 - window <= w.key0) && !(ncols & 31);
                // two buffers of columns, so one barrier a block: behind it the block before last has been read
                float *const c_ls = reinterpret_cast<float *>(sm + L::COL_OFF) + (team * 2 + (seq & 1)) * 128;
                c_ls[m] = ls * -kWtLog2e;
                named_barrier_sync(1 + team, 128);
                int h2 = h, b2 = b + kWeightTeams;
                settle(w, h2, b2);
                if (h2 < w.nh) {
                    fetch(w, h2, b2);
                } else if (!last) {
                    int hn = 0, bn = (h2 - w.nh) * w.blocks + b2;
                    settle(next, hn, bn);
                    if (hn < next.nh) {
                        fetch(next, hn, bn);
                        fetched = true;
                    }
                }
                ok = ok && mbar_wait(&s_full[it & 3], (it >> 2) & 1, err, kErrWaitFull);
                __syncwarp();
                tc_fence_after();
                uint64_t acc[4] = {0, 0, 0, 0};
                if (all) {
                    add_columns<false>(acc, s_lane + 128u * (it & 3), ncols, sl2, c_ls, 0, 0);
                } else {
                    // token t of the block, at pos0 + t, sees the key from t = key - pos0 (causal) to
                    // key - pos0 + window; a key past the row is seen by none
                    const int t_begin = causal ? max(0, key - pos0) : 0;
                    const int t_end = key >= w.length ? 0
                                      : window < 0 ? i_count
                                                   : (int)max(0ll, min((long long)i_count, (long long)key - pos0 + window + 1));
                    add_columns<true>(acc, s_lane + 128u * (it & 3), ncols, sl2, c_ls, min(t_begin, bt) * G, t_end * G);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[it & 3]);
                float u0, u1;
                f2_split(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), u0, u1);
                total += u0 + u1;
                h = h2;
                b = b2;
                it += kWeightTeams;
                ++seq;
            }
            a.part[((size_t)w.part * kWeightTeams + team) * kWeightKeys + m] = total;
            b += (h - w.nh) * w.blocks;
            h = 0;
            w = next;
            settle(w, h, b);
            if (!fetched && !last && h < w.nh) fetch(w, h, b);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWtMma) tmem_dealloc(tmem, 512);
}

__device__ __forceinline__ void put_score(const WeightsTile &t, const int32_t *pages, int page_size, int page_shift, int key,
                                          float w, float *scores, float decay) {
    const size_t slot = (size_t)pages[t.kv_base + (key >> page_shift)] * page_size + (key & (page_size - 1));
    scores[slot] = (decay != 0.f && key < t.new_begin ? decay * scores[slot] : 0.f) + w;
}

// A tile's parts: a CTA of 128 keys x 8 slices, a thread adding every eighth part of its key, eight in
// flight, the slices joined in order.
constexpr int kWtSlices = 8;
__global__ void __launch_bounds__(kWeightKeys * kWtSlices) weights_finish_kernel(const WeightsTile *tiles,
                                                                                 const int32_t *pages, const float *part,
                                                                                 int page_size, int page_shift,
                                                                                 float *scores, float decay) {
    __shared__ float sums[kWtSlices][kWeightKeys];
    const WeightsTile t = tiles[blockIdx.x];
    const int m = threadIdx.x % kWeightKeys, slice = threadIdx.x / kWeightKeys, key = t.key0 + m;
    griddep_wait();
    griddep_launch();
    const float *p = part + (size_t)t.first * kWeightTeams * kWeightKeys + m;
    const int n = kWeightTeams * t.base;
    float w = 0.f;
    for (int i0 = slice; i0 < n; i0 += 8 * kWtSlices) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i0 + i * kWtSlices < n ? __ldcg(p + (size_t)(i0 + i * kWtSlices) * kWeightKeys) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) w += x[i];
    }
    sums[slice][m] = w;
    __syncthreads();
    if (slice || key >= t.length) return;
#pragma unroll
    for (int i = 1; i < kWtSlices; ++i) w += sums[i][m];
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
    if (key >= t.first) {
        const float *lg = logits + (size_t)t.base * 16 + key;
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
    // more than half an SM's shared memory: one CTA per SM
    const size_t need = 1024 + dev::WtSmem<D>::BYTES, smem = need < 116 * 1024 ? 116 * 1024 : need;
    cudaError_t e = set_smem_limit((const void *)fn, smem, st);
    return e == cudaSuccess ? launch_pdl(fn, grid, dim3(dev::kWtThreads), smem, st, tk, tq, a) : e;
}

cudaError_t launch_weights(const Shape &s, const Plan &p, const WeightsPlan &wp, const CUtensorMap &tm_k,
                           const CUtensorMap &tm_q, void *ws, const float *lse, float *scores, float decay,
                           cudaStream_t st) {
    (void)p;
    uint8_t *w = static_cast<uint8_t *>(ws);
    dev::WeightsArgs a;
    const WeightsTile *tiles = reinterpret_cast<const WeightsTile *>(w + wp.off_tiles);
    a.pages = reinterpret_cast<const int32_t *>(w + wp.off_pages);
    a.hdr = reinterpret_cast<PlanHeader *>(w);
    a.lse = lse;
    a.part = reinterpret_cast<float *>(w + wp.off_part);
    a.items = reinterpret_cast<const WeightsItem *>(w + wp.off_items);
    a.num_items = wp.items;
    a.num_qo_heads = s.num_qo_heads;
    a.group = s.group();
    a.page_size = s.page_size;
    a.page_shift = s.page_shift();
    a.box_rows = s.page_size < kWeightKeys ? s.page_size : kWeightKeys;
    a.box_tokens = wp.box_tokens;
    a.oob_row = s.num_cache_pages * 2 * s.page_size;
    const dim3 grid(wp.items < s.sm_count ? wp.items : s.sm_count);
    cudaError_t e = wp.items == 0       ? cudaSuccess
                    : s.head_dim == 64  ? launch_weights_t<64>(tm_k, tm_q, a, grid, st)
                    : s.head_dim == 128 ? launch_weights_t<128>(tm_k, tm_q, a, grid, st)
                                        : launch_weights_t<256>(tm_k, tm_q, a, grid, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(dev::weights_finish_kernel, dim3(wp.tiles), dim3(kWeightKeys * dev::kWtSlices), 0, st, tiles, a.pages,
                      static_cast<const float *>(a.part), s.page_size, s.page_shift(), scores, decay);
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
