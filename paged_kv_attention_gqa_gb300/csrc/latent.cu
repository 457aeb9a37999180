// Latent attention, absorbed form, over a paged cache of one vector per token (pkv_latent_run), the
// join of its split units and the append of new vectors.
//
// Every token keeps x_j = [c_j | r_j] (512 latent + 64 rope values).  Query row f = token * H + head
// holds [q W_uk^T | q_rope], so that
//     s_fj = sm_scale * <q_f, x_j>,  p_f = softmax_j(s_f),  o_f = sum_j p_fj c_j,
// with one key and value vector for all heads: 2 * (576 + 512) operations per row and key on 1,152
// bytes per key.  One token of 16 heads does 30 operations per byte read (HBM-bound), one of 128
// heads 242, near the balance of this GPU (1,917 TFLOP/s over 6,674 GB/s: 287).
//
// Work: a unit is up to 64 query rows of one sequence (tokens x heads, flattened) over the 64-key
// tiles that they see; the planner gives every CTA (one per SM) an equal run of tiles.
//  * S = Q X^T: M = 64 rows, N = 64 keys, 36 k-steps, both operands from shared memory; O += P C:
//    N = 512 as two of 256, 4 k-steps, P from shared memory.  M = 64 because O takes all 512
//    tensor-memory columns: an M = 64 accumulator fills 16 of the 32 lanes of each warp's quarter, O
//    the lower ones, and S (two buffers of 64 columns) the upper ones.  An M = 64 MMA takes as long as
//    M = 128, and 32 cycles at least (measured at N = 64 and at N = 32: a tile of 32 keys costs as much
//    S time as one of 64): 2,183 cycles a tile, below the 3,190 in which an SM's share of HBM delivers it.
//  * Shared memory: Q 72 KB (64 rows, whatever the unit has), two tiles of 72 KB (a tile serves as keys
//    and, its first 512 columns, as values), P 8 KB.  A step is bounded by the time a tile's buffer waits for its copy, S, the softmax
//    and PV (two of them: half that time a tile; bringing later tiles into L2 ahead shortened the copies
//    and lengthened the start by as much).  Pages of 64 slots and more are copied with one TMA
//    instruction a tile; smaller ones with one per page and 64 columns, spread over four warps, because
//    a warp takes some 50 cycles for each.  Copies are whole cache rows on purpose: split by columns
//    they lost HBM more than they freed early (5,400 cycles a tile), and tiles of 32 keys pay twice
//    for S (3,940 cycles per 64 keys).
//  * Warps 0-3 softmax (16 rows each, a quad per row pair), 4 and 7-9 copy tiles, 5 issues S, 10 issues
//    PV (a warp each, so that neither's wait holds up the other), 6 copies Q.
//  * A key that a row does not see has weight 0, but 0 * NaN would reach O.  Those that no row of the unit
//    sees are zeroed in shared memory; a tile with keys that some rows see and others do not (several
//    tokens of a step, causal or windowed) is looked over by warp 10 before its PV, and one that holds NaN or
//    infinities there is left to the softmax warps, each row adding the keys it sees.
//  * A row's running maximum moves (and O is rescaled in tensor memory) only when it grows by more
//    than 2^8.  Sums and maxima are 32-bit; P is rounded to bf16 for the MMA (relative 2^-8 a weight at
//    most, as the output's own rounding), the sum adds the unrounded weights.
// Measured, append and join included: 32 rows of 203 to 8,190 tokens, 16 heads, 156 MB: 41 us (23 at the
// copy rate); 48 rows of 611 to 6,151, 128 heads: 79 us (2,580 cycles a tile, the rest pieces and their
// join); one row of 517: 10 us.  Two CTAs sharing a sequence's tiles by multicast changed nothing at 128
// heads: the copies are not what bounds it.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "latent.h"
#include "launch.h"
#include "tcgen05.cuh"

namespace pkv {
namespace dev {

constexpr int kLtThreads = 352;
constexpr int kLtProducers = 4;                // warps that copy pages of fewer than 64 slots
constexpr int kLtChunks = kLatentWidth / 64;   // 64-column chunks of a key
constexpr int kLtValueChunks = kLatentDim / 64;
constexpr float kLtRescale = 8.f;              // log2
constexpr float kLtLn2 = 0.6931471805599453f;

struct LtSmem {
    static constexpr uint32_t CHUNK = kLatentKeys * 128;      // 64 keys x 64 columns
    static constexpr uint32_t TILE = kLtChunks * CHUNK;       // 73,728
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t K_OFF = TILE;
    static constexpr uint32_t P_OFF = K_OFF + 2 * TILE;
    static constexpr uint32_t BAR_OFF = P_OFF + CHUNK;
    static constexpr uint32_t BYTES = BAR_OFF + 256;
};
static_assert(1024 + LtSmem::BYTES <= 227 * 1024, "the latent kernel fits shared memory");

struct LatentArgs {
    __nv_bfloat16 *out;
    float *lse;
    const LatentTile *tiles;
    const int32_t *cta_ptr;
    const int32_t *pages;
    float *part_o;    // [slot][64][512], normalised
    float *part_lse;  // [slot][64], base 2
    LatentHeader *hdr;
    int num_heads, page_size, page_shift, box_rows, box_q;
    int oob_row;      // a row past the cache: TMA fills zeros
};

// The positions that the rows of a unit see.  Their keys range over [lo_min, hi_max]; all rows see
// [lo_max, hi_min] of them, and of the rest some rows see one and others do not (causal or windowed units
// of several tokens).
struct LatentSeen {
    int lo_min, lo_max, hi_min, hi_max;
};
__device__ __forceinline__ LatentSeen latent_seen(const LatentTile &t, int heads, int causal, int window_left) {
    const int first = t.pos0 + t.q_row / heads, last = t.pos0 + (t.q_row + t.n_rows - 1) / heads;
    LatentSeen u;
    u.lo_min = window_left >= 0 ? max(0, first - window_left) : 0;
    u.lo_max = window_left >= 0 ? max(0, last - window_left) : 0;
    u.hi_min = causal ? first : t.length - 1;
    u.hi_max = causal ? last : t.length - 1;
    return u;
}
// The piece's tiles that hold keys which some rows see and others do not: those below `low` and from `high`.
struct LatentMixed {
    int low, high;
    __device__ __forceinline__ bool operator()(int j) const { return j < low || j >= high; }
};
__device__ __forceinline__ LatentMixed latent_mixed(const LatentSeen &u, int tile0) {
    LatentMixed m;
    m.low = u.lo_min < u.lo_max ? (u.lo_max + kLatentKeys - 1) / kLatentKeys - tile0 : 0;
    m.high = u.hi_min < u.hi_max ? (u.hi_min + 1) / kLatentKeys - tile0 : INT_MAX;
    return m;
}

// O += P C of one tile without the tensor cores, for tiles that hold NaN or infinities in a key that
// some rows see and others do not: each row adds the keys it sees alone.  A thread holds the two rows and
// the columns of tmem_ld16x64; P is read back from shared memory.
__device__ __noinline__ void latent_pv_rows(uint32_t o_addr, const uint8_t *tile, const uint8_t *p_sm, int row_a,
                                            int quad, int key0, int lo_a, int hi_a, int lo_b, int hi_b, float al_a, float al_b,
                                            bool first) {
    const int row_b = row_a + 8;
#pragma unroll 1
    for (int n = 0; n < kLatentDim / 64; ++n) {
        uint32_t r[32];
        float o[32];
        __syncwarp();
        tmem_ld16x64(o_addr + 64 * n, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = first ? 0.f : __uint_as_float(r[i]) * ((i & 2) ? al_b : al_a);
        const uint8_t *chunk = tile + n * LtSmem::CHUNK + quad * 4;
#pragma unroll 1
        for (int k = 0; k < kLatentKeys; ++k) {
            const bool sees_a = key0 + k >= lo_a && key0 + k <= hi_a, sees_b = key0 + k >= lo_b && key0 + k <= hi_b;
            if (!sees_a && !sees_b) continue;
            auto weight = [&](int row) {
                return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p_sm + swz128(row, k >> 3) + (k & 7) * 2));
            };
            const float p_a = weight(row_a), p_b = weight(row_b);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(chunk + swz128(k, c)));
                if (sees_a) {
                    o[4 * c] = fmaf(p_a, v.x, o[4 * c]);
                    o[4 * c + 1] = fmaf(p_a, v.y, o[4 * c + 1]);
                }
                if (sees_b) {
                    o[4 * c + 2] = fmaf(p_b, v.x, o[4 * c + 2]);
                    o[4 * c + 3] = fmaf(p_b, v.y, o[4 * c + 3]);
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(o[i]);
        tmem_st16x64(o_addr + 64 * n, r);
    }
    tmem_wait_st();
}

__global__ void __launch_bounds__(kLtThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tm_cache, const __grid_constant__ CUtensorMap tm_q,
                  const LatentArgs a) {
    using L = LtSmem;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *const k_sm = sm + L::K_OFF, *const p_sm = sm + L::P_OFF;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR_OFF);
    // Tiles are counted over the CTA's whole run (it), pieces too (pc).  No waiter is ever two
    // phases behind: each next phase needs something the waiter has yet to provide.
    uint64_t *full = bars + 0;     // [2] tile it in stage it % 2
    uint64_t *empty = bars + 2;    // [2] PV(it) completed: the stage may be refilled
    uint64_t *s_full = bars + 4;   // [2] S(it) in buffer it % 2
    uint64_t *p_full = bars + 6;   // P(it) in shared memory (and O rescaled if it had to be)
    uint64_t *pv_done = bars + 7;  // PV(it) completed
    uint64_t *q_full = bars + 8;   // the piece's Q landed
    uint64_t *q_empty = bars + 9;  // the piece's last S completed
    uint64_t *o_free = bars + 10;  // the piece's O has been read
    uint64_t *checked = bars + 11;  // a tile with keys that not all rows see has been looked over
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 12);
    uint32_t *by_rows = tmem_holder + 1;  // it holds NaN or infinities there: its PV goes by rows

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // the plan's arrays come from the host's copy, never from a kernel: they are read before waiting
    // for the previous kernel
    const int t_begin = a.cta_ptr[blockIdx.x], t_end = a.cta_ptr[blockIdx.x + 1];
    const LatentTile first_tile = a.tiles[t_begin];
    int *const err = &a.hdr->err;
    const int P = a.page_size;
    // copies.  Pages of 64 slots and more: one box of the tile's rows and all nine 64-column chunks.
    // Smaller ones: a box per page and chunk; producer warp w takes `per` of them, one a lane, from w * per
    const bool whole = a.box_rows == kLatentKeys;
    const int R = a.box_rows, jobs = whole ? 1 : kLatentKeys / R * kLtChunks;  // 1, 18, 36 or 72
    const int per = whole ? 1 : (jobs + kLtProducers - 1) / kLtProducers;
    const int producer = warp == 4 ? 0 : warp - 6;  // of warps 4, 7, 8 and 9
    const int job = producer * per + lane;
    const bool copies = lane < per && job < jobs;
    auto row_of = [&](const LatentTile &t, int j) {  // the cache row of this lane's box
        const int kb = (t.tile0 + j) * kLatentKeys + (whole ? 0 : job / kLtChunks * R), pg = kb >> a.page_shift;
        return copies && pg < ((t.length + P - 1) >> a.page_shift) ? a.pages[t.kv_base + pg] * P + (kb & (P - 1))
                                                                   : a.oob_row;
    };
    int row = 0;
    const bool producing = warp == 4 || (warp > 6 && warp < 10);
    if (producing) row = row_of(first_tile, 0);
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&full[s], whole ? 1 : kLtProducers);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(p_full, 4);
        mbar_init(pv_done, 1);
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(o_free, 4);
        mbar_init(checked, 1);
        fence_barrier_init();
        prefetch_tmap(&tm_cache);
        prefetch_tmap(&tm_q);
    }
    if (warp == 5) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();  // q and the cache may come from the previous kernel (an append)
    griddep_launch();
    const uint32_t tmem = *tmem_holder;
    const uint32_t s_base = tmem + (16u << 16);  // S buffers: upper 16 lanes, columns 0 and 64

    if (producing) {
        // ------------------------------------------------ tiles
        if (warp == 4 || !whole) {
            const uint32_t bytes = whole ? L::TILE : (uint32_t)max(0, min(per, jobs - producer * per)) * R * 128u;
            uint32_t it = 0;
            bool ok = true;
            for (int ti = t_begin; ti < t_end && ok; ++ti) {
                const LatentTile t = ti == t_begin ? first_tile : a.tiles[ti];
                if (ti > t_begin) row = row_of(t, 0);
                for (int j = 0; j < t.ntiles; ++j, ++it) {
                    const int s = it & 1;
                    ok = it < 2 || mbar_wait(&empty[s], ((it >> 1) - 1) & 1, err, kErrWaitEmpty);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
                    __syncwarp();
                    uint8_t *st = k_sm + s * L::TILE;
                    if (copies) {
                        if (whole)
                            tma_load_3d(st, &tm_cache, &full[s], 0, row, 0);
                        else
                            tma_load_3d(st + job % kLtChunks * L::CHUNK + job / kLtChunks * R * 128, &tm_cache, &full[s], 0,
                                        row, job % kLtChunks);
                    }
                    if (j + 1 < t.ntiles) row = row_of(t, j + 1);  // lands while the next stage is awaited
                }
            }
            // copies in flight land before the CTA may end (they have, unless a wait gave up)
            for (uint32_t d = it > 2 ? it - 2 : 0; d < it; ++d) mbar_wait(&full[d & 1], (d >> 1) & 1, err, kErrWaitDrain);
        }
    } else if (warp == 6) {
        // ------------------------------------------------ Q of each piece
        if (lane == 0) {
            uint32_t pc = 0;
            for (int ti = t_begin; ti < t_end; ++ti, ++pc) {
                const int q_row = ti == t_begin ? first_tile.q_row : a.tiles[ti].q_row;
                if (pc > 0 && !mbar_wait(q_empty, (pc - 1) & 1, err, kErrWaitEmpty)) break;
                mbar_arrive_expect_tx(q_full, (uint32_t)(kLtChunks * a.box_q) * 128u);
                for (int c = 0; c < kLtChunks; ++c)
                    tma_load_2d(sm + L::Q_OFF + c * L::CHUNK, &tm_q, q_full, c * 64, q_row);
            }
            if (pc > 0) mbar_wait(q_full, (pc - 1) & 1, err, kErrWaitDrain);
        }
    } else if (warp == 5) {
        // ------------------------------------------------ S = Q X^T
        constexpr uint32_t ID_S = idesc_bf16_f32(64, kLatentKeys, 0, 0);
        const uint64_t dQ = smem_desc(smem_u32(sm + L::Q_OFF), 16, 1024, kSwizzle128B);
        const uint64_t dK = smem_desc(smem_u32(k_sm), 16, 1024, kSwizzle128B);
        auto add = [](uint64_t d, uint32_t off) { return d + (off >> 4); };
        uint32_t it = 0, pc = 0;
        bool ok = true;
        for (int ti = t_begin; ti < t_end && ok; ++ti, ++pc) {
            const int n = ti == t_begin ? first_tile.ntiles : a.tiles[ti].ntiles;
            ok = mbar_wait(q_full, pc & 1, err, kErrWaitFull);
            for (int j = 0; j < n && ok; ++j, ++it) {
                // the stage was refilled after PV(it - 2), so the softmax has read that tile's S out of this
                // buffer
                const uint32_t b = it & 1;
                ok = mbar_wait(&full[b], (it >> 1) & 1, err, kErrWaitFull);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kLatentWidth / 16; ++kk) {
                    const uint32_t off = (kk / 4) * L::CHUNK + (kk % 4) * 32;
                    mma_ss_elect(s_base + 64u * b, add(dQ, off), add(dK, b * L::TILE + off), ID_S, kk > 0 ? 1u : 0u);
                }
                mma_commit_elect(&s_full[b]);
            }
            if (ok) mma_commit_elect(q_empty);  // the piece's last reader of Q
        }
        if (!ok)  // a wait gave up: let the MMAs in flight finish before the tensor memory is released
            for (uint32_t i = 0; i < 1024; ++i) __nanosleep(1000);
    } else if (warp == 10) {
        // ------------------------------------------------ O += P C
        constexpr uint32_t ID_O = idesc_bf16_f32(64, 256, 0, 1);
        const uint64_t dP = smem_desc(smem_u32(p_sm), 16, 1024, kSwizzle128B);
        // values: N-major, 64-column chunks CHUNK apart, 8-key groups 1024 bytes apart
        const uint64_t dV = smem_desc(smem_u32(k_sm), L::CHUNK, 1024, kSwizzle128B);
        auto add = [](uint64_t d, uint32_t off) { return d + (off >> 4); };
        uint32_t it = 0, pc = 0;
        bool ok = true;
        for (int ti = t_begin; ti < t_end && ok; ++ti, ++pc) {
            const LatentTile t = ti == t_begin ? first_tile : a.tiles[ti];
            const LatentSeen u = latent_seen(t, a.num_heads, a.hdr->causal, a.hdr->window_left);
            const LatentMixed mixed = latent_mixed(u, t.tile0);
            // the piece's tiles below edge_low and from edge_high hold keys that not all rows see
            const int page_end = (t.length + P - 1) & ~(P - 1);
            const int edge_low = (u.lo_max + kLatentKeys - 1) / kLatentKeys - t.tile0;
            const int edge_high = u.hi_min + 1 < page_end ? (u.hi_min + 1) / kLatentKeys - t.tile0 : INT_MAX;
            // O may be overwritten once the last piece's has been read
            if (pc > 0) ok = mbar_wait(o_free, (pc - 1) & 1, err, kErrWaitEmpty);
            for (int j = 0; j < t.ntiles && ok; ++j, ++it) {
                const uint32_t b = it & 1;
                bool rows = false;
                if (j < edge_low || j >= edge_high) {
                    ok = mbar_wait(&full[b], (it >> 1) & 1, err, kErrWaitFull);
                    if (!ok) break;
                    uint8_t *const tile = k_sm + b * L::TILE;
                    // Keys that no row of the unit sees hold anything (past the sequence's end to the end of its
                    // last page, behind the last row's position, before the window); their P is 0, but 0 * NaN
                    // would reach O: zero them (S of these columns is masked whatever it reads)
                    const int key0 = (t.tile0 + j) * kLatentKeys, ze = min(page_end, key0 + kLatentKeys);
                    const int n_low = max(0, min(u.lo_min, ze) - key0), high = max(u.hi_max + 1, key0);
                    const int n_zero = n_low + max(0, ze - high);
                    for (int e = lane; e < n_zero * kLtValueChunks * 8; e += 32) {
                        const int i = e / (kLtValueChunks * 8), c = e % (kLtValueChunks * 8);
                        const int k = i < n_low ? i : high - key0 + i - n_low;
                        *reinterpret_cast<uint4 *>(tile + (c >> 3) * L::CHUNK + swz128(k, c & 7)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    // Keys that some rows see and others do not stay; a NaN or an infinity among them goes to
                    // the rows that see it, one by one
                    if (mixed(j)) {
                        const int begin = max(key0, u.lo_min), end = min(key0 + kLatentKeys, u.hi_max + 1);
                        const int first = (begin < u.lo_max ? begin : max(begin, u.hi_min + 1)) - key0;
                        const int n = ((u.hi_min + 1 < end ? end : min(end, u.lo_max)) - key0 - first) * kLtValueChunks * 8;
                        uint32_t f0 = 0, f1 = 0;
                        for (int e0 = lane; e0 < n; e0 += 4 * 32) {  // four vectors in flight
                            uint4 x[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int e = min(e0 + 32 * i, n - 1), c = e % (kLtValueChunks * 8);
                                x[i] = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * L::CHUNK +
                                                                        swz128(first + e / (kLtValueChunks * 8), c & 7));
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                f0 = keep_nonfinite(x[i].x, keep_nonfinite(x[i].y, f0));
                                f1 = keep_nonfinite(x[i].z, keep_nonfinite(x[i].w, f1));
                            }
                        }
                        rows = __any_sync(0xffffffffu, has_nan(f0) || has_nan(f1));
                        if (lane == 0) {
                            *by_rows = rows;
                            mbar_arrive(checked);
                        }
                    }
                    __syncwarp();
                }
                ok = mbar_wait(p_full, it & 1, err, kErrWaitFull);
                if (!ok) break;
                tc_fence_after();
                if (!rows) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int kk = 0; kk < kLatentKeys / 16; ++kk)
                            mma_ss_elect(tmem + 256u * h, add(dP, kk * 32),
                                         add(dV, b * L::TILE + h * 4 * L::CHUNK + kk * 2048), ID_O,
                                         (j > 0 || kk > 0) ? 1u : 0u);
                }
                mma_commit_elect(&empty[b]);
                mma_commit_elect(pv_done);
            }
        }
        if (!ok)  // a wait gave up: let the MMAs in flight finish before the tensor memory is released
            for (uint32_t i = 0; i < 1024; ++i) __nanosleep(1000);
    } else {
        // ------------------------------------------------ softmax and epilogue: warps 0-3
        const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
        const int quad = lane & 3, row_a = warp * 16 + (lane >> 2), row_b = row_a + 8;
        const float sl = a.hdr->scale_log2;
        const int causal = a.hdr->causal, window_left = a.hdr->window_left;
        uint8_t *const pa = p_sm + quad * 4;
        uint32_t it = 0, pc = 0, checks = 0;  // tiles of `checked` so far
        bool ok = true;
        for (int ti = t_begin; ti < t_end && ok; ++ti, ++pc) {
            const LatentTile t = ti == t_begin ? first_tile : a.tiles[ti];
            // keys [lo, hi] of each of the thread's two rows.  Rows past the unit's hold whatever Q's
            // shared memory held: they are never stored and never move a maximum
            const bool live_a = row_a < t.n_rows, live_b = row_b < t.n_rows;
            const bool idle = warp * 16 >= t.n_rows;  // the warp has no row of this unit
            int lo_a = 0, hi_a = INT_MAX, lo_b = 0, hi_b = INT_MAX;
            auto range = [&](int m, int &lo, int &hi) {
                if (m >= t.n_rows) return;
                const int pos = t.pos0 + (t.q_row + m) / a.num_heads;
                hi = causal ? pos : t.length - 1;
                lo = window_left >= 0 ? max(0, pos - window_left) : 0;
            };
            range(row_a, lo_a, hi_a);
            range(row_b, lo_b, hi_b);
            const int lo_max = max(lo_a, lo_b), hi_min = min(hi_a, hi_b);
            const LatentMixed mixed = latent_mixed(latent_seen(t, a.num_heads, causal, window_left), t.tile0);
            float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;
            for (int j = 0; j < t.ntiles; ++j, ++it) {
                const uint32_t b = it & 1;
                if (!mbar_wait(&s_full[b], (it >> 1) & 1, err, kErrWaitFull)) {
                    ok = false;
                    break;
                }
                if (idle) {  // P's rows of this warp stay as they are: O's are never read
                    checks += mixed(j);
                    if (it > 0 && !mbar_wait(pv_done, (it - 1) & 1, err, kErrWaitFull)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive(p_full);
                    continue;
                }
                tc_fence_after();
                uint32_t r[32];
                tmem_ld16x64(s_base + lane_off + 64u * b, r);
                tmem_wait_ld();
                const int key0 = (t.tile0 + j) * kLatentKeys;
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
                if (key0 < lo_max || key0 + kLatentKeys - 1 > hi_min) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int k = key0 + 8 * (i >> 2) + 2 * quad + (i & 1);
                        const bool sees = (i & 2) ? ((k >= lo_b) & (k <= hi_b)) : ((k >= lo_a) & (k <= hi_a));
                        x[i] = sees ? x[i] : -INFINITY;
                    }
                }
                float m2[4] = {fmaxf(x[0], x[1]), fmaxf(x[2], x[3]), fmaxf(x[4], x[5]), fmaxf(x[6], x[7])};
#pragma unroll
                for (int c = 2; c < 8; ++c) {
                    m2[2 * (c & 1)] = max3f(m2[2 * (c & 1)], x[4 * c], x[4 * c + 1]);
                    m2[2 * (c & 1) + 1] = max3f(m2[2 * (c & 1) + 1], x[4 * c + 2], x[4 * c + 3]);
                }
                float mx_a = fmaxf(m2[0], m2[2]), mx_b = fmaxf(m2[1], m2[3]);
                mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 1));
                mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 1));
                mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 2)) * sl;
                mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 2)) * sl;
                mx_a = live_a ? mx_a : -INFINITY;
                mx_b = live_b ? mx_b : -INFINITY;
                // move a row's maximum only when it grows by more than the threshold
                const bool grow_a = mx_a > m_a + kLtRescale, grow_b = mx_b > m_b + kLtRescale;
                const bool any = __any_sync(0xffffffffu, grow_a || grow_b);
                float al_a = 1.f, al_b = 1.f;
                if (grow_a) {
                    al_a = ex2_ftz(m_a - mx_a);
                    m_a = mx_a;
                }
                if (grow_b) {
                    al_b = ex2_ftz(m_b - mx_b);
                    m_b = mx_b;
                }
                const float r_a = m_a == -INFINITY ? 0.f : m_a, r_b = m_b == -INFINITY ? 0.f : m_b;
                float sa[2] = {0.f, 0.f}, sb[2] = {0.f, 0.f};
                uint32_t pk[16];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float p0 = ex2_ftz(fmaf(x[4 * c], sl, -r_a)), p1 = ex2_ftz(fmaf(x[4 * c + 1], sl, -r_a));
                    const float p2 = ex2_ftz(fmaf(x[4 * c + 2], sl, -r_b)), p3 = ex2_ftz(fmaf(x[4 * c + 3], sl, -r_b));
                    sa[c & 1] += p0 + p1;
                    sb[c & 1] += p2 + p3;
                    pk[2 * c] = pack_bf16(p0, p1);
                    pk[2 * c + 1] = pack_bf16(p2, p3);
                }
                l_a = l_a * al_a + (sa[0] + sa[1]);
                l_b = l_b * al_b + (sb[0] + sb[1]);
                // P has one buffer, and O may be touched, once PV(it - 1) has completed
                if (it > 0 && !mbar_wait(pv_done, (it - 1) & 1, err, kErrWaitFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    *reinterpret_cast<uint32_t *>(pa + swz128(row_a, c)) = pk[2 * c];
                    *reinterpret_cast<uint32_t *>(pa + swz128(row_b, c)) = pk[2 * c + 1];
                }
                fence_proxy_async_smem();
                if ((any && j > 0) || mixed(j)) {
                    bool rows = false;
                    if (mixed(j)) {
                        if (!mbar_wait(checked, checks++ & 1, err, kErrWaitFull) ||
                            !mbar_wait(&full[b], (it >> 1) & 1, err, kErrWaitFull)) {  // (has: S(it) has read the tile)
                            ok = false;
                            break;
                        }
                        rows = *by_rows != 0;
                    }
                    if (rows) {
                        latent_pv_rows(tmem + lane_off, k_sm + b * L::TILE, p_sm, row_a, quad, key0, lo_a, hi_a, lo_b, hi_b,
                                       al_a, al_b, j == 0);
                    } else if (any && j > 0) {
#pragma unroll 1
                        for (int c0 = 0; c0 < kLatentDim; c0 += 64) {
                            uint32_t o[32];
                            tmem_ld16x64(tmem + lane_off + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * ((i & 2) ? al_b : al_a));
                            tmem_st16x64(tmem + lane_off + c0, o);
                        }
                        tmem_wait_st();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            if (!ok) break;
            // the piece's O
            l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
            l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
            l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
            l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
            if (!mbar_wait(pv_done, (it - 1) & 1, err, kErrWaitFull)) break;
            tc_fence_after();
            // a piece may hold no visible key of a row (causal, several tokens): weight 0, lse -inf.  Keys whose
            // scores are all -inf weigh nothing against other pieces, but 0 * inf of their values stays; a
            // row that has no others is NaN (0 / 0).
            const int first_key = t.tile0 * kLatentKeys, last_key = first_key + t.ntiles * kLatentKeys - 1;
            auto inverse = [&](float l, int lo, int hi) {
                return max(lo, first_key) > min(hi, last_key) ? 0.f : l == 0.f && t.partial >= 0 ? 1.f : 1.f / l;
            };
            const float inv_a = inverse(l_a, lo_a, hi_a), inv_b = inverse(l_b, lo_b, hi_b);
            const float lse_a = l_a == 0.f ? -INFINITY : m_a + log2f(l_a);
            const float lse_b = l_b == 0.f ? -INFINITY : m_b + log2f(l_b);
            const size_t g_a = (size_t)t.q_row + row_a, g_b = (size_t)t.q_row + row_b;
            float *po = a.part_o + (size_t)max(t.partial, 0) * kLatentRows * kLatentDim;
            if (!idle) {
                uint32_t o[2][32];  // the next 64 columns load while these are stored
                tmem_ld16x64(tmem + lane_off, o[0]);
#pragma unroll
                for (int n = 0; n < kLatentDim / 64; ++n) {
                    tmem_wait_ld();
                    if (n + 1 < kLatentDim / 64) tmem_ld16x64(tmem + lane_off + 64 * (n + 1), o[(n + 1) & 1]);
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {  // select, not multiply: 0 * NaN of a key the row does not see
                        const float inv = (i & 2) ? inv_b : inv_a;
                        f[i] = inv == 0.f ? 0.f : __uint_as_float(o[n & 1][i]) * inv;
                    }
                    // lane pairs exchange so that each holds four columns in a row: of group c the even lane
                    // (columns 8 c + 4 (quad / 2) ..), of group c + 1 the odd one; a store then covers
                    // 64 bytes (32 of bf16) of each of its eight rows, and half as many lines pass the SM
                    const bool odd = quad & 1;
#pragma unroll
                    for (int c = 0; c < 8; c += 2) {
                        float4 va, vb;
#pragma unroll
                        for (int w = 0; w < 2; ++w) {  // the thread's two rows
                            const float k0 = f[4 * (c + 0) + 2 * w], k1 = f[4 * (c + 0) + 2 * w + 1];
                            const float n0 = f[4 * (c + 1) + 2 * w], n1 = f[4 * (c + 1) + 2 * w + 1];
                            const float g0 = __shfl_xor_sync(0xffffffffu, odd ? k0 : n0, 1);
                            const float g1 = __shfl_xor_sync(0xffffffffu, odd ? k1 : n1, 1);
                            const float4 v = odd ? make_float4(g0, g1, n0, n1) : make_float4(k0, k1, g0, g1);
                            if (w == 0)
                                va = v;
                            else
                                vb = v;
                        }
                        const int col = 64 * n + 8 * (c + odd) + 4 * (quad >> 1);
                        if (t.partial < 0) {
                            if (live_a)
                                *reinterpret_cast<uint2 *>(a.out + g_a * kLatentDim + col) =
                                    make_uint2(pack_bf16(va.x, va.y), pack_bf16(va.z, va.w));
                            if (live_b)
                                *reinterpret_cast<uint2 *>(a.out + g_b * kLatentDim + col) =
                                    make_uint2(pack_bf16(vb.x, vb.y), pack_bf16(vb.z, vb.w));
                        } else {
                            if (live_a) *reinterpret_cast<float4 *>(po + (size_t)row_a * kLatentDim + col) = va;
                            if (live_b) *reinterpret_cast<float4 *>(po + (size_t)row_b * kLatentDim + col) = vb;
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            if (quad == 0) {
                if (t.partial >= 0) {
                    float *pl = a.part_lse + (size_t)t.partial * kLatentRows;
                    if (live_a) pl[row_a] = lse_a;
                    if (live_b) pl[row_b] = lse_b;
                } else if (a.lse) {
                    if (live_a) a.lse[g_a] = lse_a * kLtLn2;
                    if (live_b) a.lse[g_b] = lse_b * kLtLn2;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, 512);
}

// Join of the pieces of a cut unit: with w_i = 2^(lse_i - max lse), o = sum w_i o_i / sum w_i.  A CTA per
// query row, four columns a thread; plans with units of more than eight pieces launch 256 threads, whose
// halves take batches of eight pieces in turn, others 128.  A thread's first batch is requested before
// the weights are known.  Bounded by the trips to L2: one for 16 (8) pieces, one more per 16.
constexpr int kLtMergeBatch = 8, kLtMergeCols = kLatentDim / 4;
__global__ void __launch_bounds__(2 * kLtMergeCols) latent_merge_kernel(const LatentMerge *merges, const float *part_o,
                                                                        const float *part_lse, __nv_bfloat16 *out,
                                                                        float *lse) {
    __shared__ float4 other[kLtMergeCols];
    const LatentMerge m = merges[blockIdx.y];
    const int row = blockIdx.x, lane = threadIdx.x & 31, col = threadIdx.x & (kLtMergeCols - 1);
    const int half = threadIdx.x / kLtMergeCols, halves = blockDim.x / kLtMergeCols;
    griddep_wait();
    griddep_launch();
    if (row >= m.n_rows) return;
    const float *pl = part_lse + (size_t)m.first * kLatentRows + row;
    const float *po = part_o + ((size_t)m.first * kLatentRows + row) * kLatentDim + col * 4;
    constexpr size_t STEP = (size_t)kLatentRows * kLatentDim;
    float4 v[kLtMergeBatch];
    const int first = half * kLtMergeBatch;
#pragma unroll
    for (int i = 0; i < kLtMergeBatch; ++i)
        if (first + i < m.count) v[i] = __ldcg(reinterpret_cast<const float4 *>(po + (first + i) * STEP));
    float mx = -INFINITY;
    const float l0 = lane < m.count ? __ldcg(pl + (size_t)lane * kLatentRows) : -INFINITY;
    for (int i = lane + 32; i < m.count; i += 32) mx = fmaxf(mx, __ldcg(pl + (size_t)i * kLatentRows));
    mx = fmaxf(mx, l0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float w0 = exp2f(l0 - mx);  // the first 32 pieces' weights, one a lane
    float sum = w0;
    for (int i = lane + 32; i < m.count; i += 32) sum += exp2f(__ldcg(pl + (size_t)i * kLatentRows) - mx);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = first; i0 < m.count; i0 += halves * kLtMergeBatch) {
        if (i0 > first) {
#pragma unroll
            for (int i = 0; i < kLtMergeBatch; ++i)
                if (i0 + i < m.count) v[i] = __ldcg(reinterpret_cast<const float4 *>(po + (i0 + i) * STEP));
        }
#pragma unroll
        for (int i = 0; i < kLtMergeBatch; ++i) {
            const float s = __shfl_sync(0xffffffffu, w0, (i0 + i) & 31);
            if (i0 + i < m.count) {
                const float w = i0 + i < 32 ? s : exp2f(__ldcg(pl + (size_t)(i0 + i) * kLatentRows) - mx);
                acc.x += w * v[i].x;
                acc.y += w * v[i].y;
                acc.z += w * v[i].z;
                acc.w += w * v[i].w;
            }
        }
    }
    if (halves > 1 && m.count > kLtMergeBatch) {  // the second half has pieces
        if (half) other[col] = acc;
        __syncthreads();
        if (!half) {
            const float4 o = other[col];
            acc.x += o.x;
            acc.y += o.y;
            acc.z += o.z;
            acc.w += o.w;
        }
    }
    if (half) return;
    const float inv = 1.f / sum;  // every row sees a key in some piece, so the largest weight is 1
    *reinterpret_cast<uint2 *>(out + ((size_t)m.q_row + row) * kLatentDim + col * 4) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (lse && threadIdx.x == 0) lse[(size_t)m.q_row + row] = (mx + log2f(sum)) * kLtLn2;
}

// Append: one thread per 16-byte chunk of a new token's vector (64 of the latent part, 8 of the rope).
__global__ void __launch_bounds__(288) latent_append_kernel(const int32_t *rows, int num, const uint4 *c_new,
                                                            long long c_stride, const uint4 *rope_new,
                                                            long long rope_stride, uint4 *cache) {
    constexpr int V = kLatentWidth / 8, VC = kLatentDim / 8;
    griddep_wait();
    griddep_launch();
    const int t = blockIdx.x * 4 + threadIdx.x / V, c = threadIdx.x % V;
    if (t >= num) return;
    cache[(size_t)rows[t] * V + c] = c < VC ? c_new[t * c_stride + c] : rope_new[t * rope_stride + c - VC];
}

}  // namespace dev

cudaError_t launch_latent(const LatentShape &s, const LatentPlan &p, const CUtensorMap &tm_cache,
                          const CUtensorMap &tm_q, void *ws, void *out, float *lse, cudaStream_t st) {
    if (p.ctas == 0) return cudaSuccess;
    uint8_t *w = static_cast<uint8_t *>(ws);
    dev::LatentArgs a;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.tiles = reinterpret_cast<const LatentTile *>(w + p.off_tiles);
    a.cta_ptr = reinterpret_cast<const int32_t *>(w + p.off_cta);
    a.pages = reinterpret_cast<const int32_t *>(w + p.off_pages);
    a.part_o = reinterpret_cast<float *>(w + p.off_part_o);
    a.part_lse = reinterpret_cast<float *>(w + p.off_part_lse);
    a.hdr = reinterpret_cast<LatentHeader *>(w);
    a.num_heads = s.num_heads;
    a.page_size = s.page_size;
    a.page_shift = s.page_shift();
    a.box_rows = s.box_rows();
    a.box_q = p.box_q;
    a.oob_row = s.num_cache_pages * s.page_size;
    const size_t smem = 1024 + dev::LtSmem::BYTES;
    cudaError_t e = set_smem_limit((const void *)dev::latent_kernel, smem, st);
    if (e == cudaSuccess)
        e = launch_pdl(dev::latent_kernel, dim3(p.ctas), dim3(dev::kLtThreads), smem, st, tm_cache, tm_q, a);
    if (e == cudaSuccess && p.num_merge)
        e = launch_pdl(dev::latent_merge_kernel, dim3(p.box_q, p.num_merge),
                       dim3((p.max_pieces > dev::kLtMergeBatch ? 2 : 1) * dev::kLtMergeCols), 0, st,
                       reinterpret_cast<const LatentMerge *>(w + p.off_merge), static_cast<const float *>(a.part_o),
                       static_cast<const float *>(a.part_lse), a.out, lse);
    return e;
}

cudaError_t launch_latent_append(const LatentShape &s, const LatentPlan &p, void *ws, const void *c_new,
                                 long long c_stride, const void *rope_new, long long rope_stride, void *cache,
                                 cudaStream_t st) {
    (void)s;
    if (p.num_append == 0) return cudaSuccess;
    return launch_pdl(dev::latent_append_kernel, dim3((p.num_append + 3) / 4), dim3(288), 0, st,
                      reinterpret_cast<const int32_t *>(static_cast<uint8_t *>(ws) + p.off_append), p.num_append,
                      static_cast<const uint4 *>(c_new), c_stride / 8, static_cast<const uint4 *>(rope_new),
                      rope_stride / 8, static_cast<uint4 *>(cache));
}

}  // namespace pkv
