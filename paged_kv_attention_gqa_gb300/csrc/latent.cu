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
// Work: a unit is up to 64 query rows of one sequence (tokens x heads, flattened) over the 32-key
// tiles that they see; the planner gives every CTA (one per SM) an equal run of tiles.
//  * S = Q X^T: M = 64 rows, N = 32 keys, 36 k-steps, both operands from shared memory; O += P C:
//    N = 512 as two of 256, 2 k-steps, P from shared memory.  M = 64 because O takes all 512
//    tensor-memory columns: an M = 64 accumulator fills 16 of the 32 lanes of each warp's quarter, O
//    the lower ones, and S (four buffers of 32 columns) the upper ones.  An M = 64 MMA takes as long as
//    M = 128 (measured 128 cycles at N = 256).
//  * Shared memory: Q (1,152 bytes a row), four tiles of 36 KB or five where Q has 32 rows or fewer (a
//    tile serves as keys and, its first 512 columns, as values), P 8 KB (two tiles side by side).
//    What bounds a bandwidth-bound step is the time a tile's buffer waits for its copy, its S, its
//    softmax and its PV: with two 64-key tiles in the same space an SM had 3,554 cycles a 64 keys in
//    steady state, against the 3,190 in which its share of HBM delivers them.
//  * Warps 0-3 softmax (16 rows each, a quad per row pair), 4 copies tiles, 5 issues MMAs (of a tile's
//    PV and a later tile's S whichever has its operands), 6 copies Q.
//  * A row's running maximum moves (and O is rescaled in tensor memory) only when it grows by more
//    than 2^8.  Sums and maxima are 32-bit; P is rounded to bf16 for the MMA (relative 2^-8 a weight at
//    most, as the output's own rounding), the sum adds the unrounded weights.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "latent.h"
#include "launch.h"
#include "tcgen05.cuh"

namespace pkv {
namespace dev {

constexpr int kLtThreads = 224;
constexpr int kLtChunks = kLatentWidth / 64;   // 64-column chunks of a key
constexpr int kLtValueChunks = kLatentDim / 64;
constexpr float kLtRescale = 8.f;              // log2
constexpr float kLtLn2 = 0.6931471805599453f;
constexpr uint32_t kLtPolls = 1u << 25;        // a poll is some tens of cycles: about a second

struct LtSmem {
    static constexpr uint32_t CHUNK = kLatentKeys * 128;      // 32 keys x 64 columns
    static constexpr uint32_t TILE = kLtChunks * CHUNK;       // 36,864
    static constexpr uint32_t P_BYTES = kLatentRows * 128;
    static constexpr int MAX_STAGES = 5;
    // order: Q (9 chunks of q_rows x 128 bytes), tiles, P, barriers.  An M = 64 read of a Q of fewer rows
    // runs on into the tiles: rows of S that nobody uses
    static constexpr uint32_t bytes(int stages, int q_rows) {
        return kLtChunks * q_rows * 128u + stages * TILE + P_BYTES + 256u;
    }
    // stages of a plan whose units have up to q_rows query rows
    static constexpr int stages(int q_rows) { return q_rows <= 32 ? 5 : 4; }
};
static_assert(1024 + LtSmem::bytes(4, 64) <= 227 * 1024 && 1024 + LtSmem::bytes(5, 32) <= 227 * 1024,
              "the latent kernel fits shared memory");

struct LatentArgs {
    __nv_bfloat16 *out;
    float *lse;
    const LatentTile *tiles;
    const int32_t *cta_ptr;
    const int32_t *pages;
    float *part_o;    // [slot][64][512], normalised
    float *part_lse;  // [slot][64], base 2
    LatentHeader *hdr;
    int num_heads, page_size, page_shift, box_rows, box_q, stages;
    int oob_row;      // a row past the cache: TMA fills zeros
};

__global__ void __launch_bounds__(kLtThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tm_cache, const __grid_constant__ CUtensorMap tm_q,
                  const LatentArgs a) {
    using L = LtSmem;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t NS = (uint32_t)a.stages;
    const uint32_t q_chunk = (uint32_t)a.box_q * 128;
    uint8_t *const q_sm = sm, *const k_sm = sm + kLtChunks * q_chunk, *const p_sm = k_sm + NS * L::TILE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(p_sm + L::P_BYTES);
    // Tiles are counted over the CTA's whole run (it), pieces too (pc).  No waiter is ever two
    // phases behind: each next phase needs something the waiter has yet to provide.
    uint64_t *full = bars + 0;      // [NS] tile it in stage it % NS
    uint64_t *empty = bars + 5;     // [NS] PV(it) completed: the stage may be refilled
    uint64_t *s_full = bars + 10;   // [4] S(it) in buffer it % 4
    uint64_t *p_full = bars + 14;   // [2] P(it) in half it % 2 (and O rescaled if it had to be)
    uint64_t *pv_done = bars + 16;  // [2] PV(it) completed, counted on it % 2
    uint64_t *q_full = bars + 18;   // the piece's Q landed
    uint64_t *q_empty = bars + 19;  // the piece's last S completed
    uint64_t *o_free = bars + 20;   // the piece's O has been read
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 21);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // the plan's arrays come from the host's copy, never from a kernel: they are read before waiting
    // for the previous kernel
    const int t_begin = a.cta_ptr[blockIdx.x], t_end = a.cta_ptr[blockIdx.x + 1];
    const LatentTile first_tile = a.tiles[t_begin];
    int *const err = &a.hdr->err;
    const int P = a.page_size;
    // copies: one lane per (box, chunk) of a tile; the cache rows of a tile's boxes
    const int R = a.box_rows, jobs = kLatentKeys / R * kLtChunks;  // 9, 18 or 36
    auto rows_of = [&](const LatentTile &t, int j, int (&row)[2]) {
        const int key0 = (t.tile0 + j) * kLatentKeys, npages = (t.length + P - 1) >> a.page_shift;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int job = lane + 32 * i, kb = key0 + (job / kLtChunks) * R, pg = kb >> a.page_shift;
            row[i] = job < jobs && pg < npages ? a.pages[t.kv_base + pg] * P + (kb & (P - 1)) : a.oob_row;
        }
    };
    int row[2] = {0, 0};
    if (warp == 4) rows_of(first_tile, 0, row);
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 4; ++s) mbar_init(&s_full[s], 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&p_full[s], 4);
            mbar_init(&pv_done[s], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(o_free, 4);
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
    const uint32_t s_base = tmem + (16u << 16);  // S buffers: upper 16 lanes, columns 0, 32, 64, 96

    if (warp == 4) {
        // ------------------------------------------------ tiles
        uint32_t it = 0, s = 0, round = 0;  // stage it % NS, it / NS
        bool ok = true;
        for (int ti = t_begin; ti < t_end && ok; ++ti) {
            const LatentTile t = ti == t_begin ? first_tile : a.tiles[ti];
            if (ti > t_begin) rows_of(t, 0, row);
            for (int j = 0; j < t.ntiles; ++j, ++it) {
                ok = round == 0 || mbar_wait(&empty[s], (round - 1) & 1, err, kErrWaitEmpty);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                uint8_t *st = k_sm + s * L::TILE;
                if (lane == 0) mbar_arrive_expect_tx(&full[s], L::TILE);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int job = lane + 32 * i;
                    if (job < jobs) {
                        const int b = job / kLtChunks, c = job % kLtChunks;
                        tma_load_2d(st + c * L::CHUNK + b * R * 128, &tm_cache, &full[s], c * 64, row[i]);
                    }
                }
                if (j + 1 < t.ntiles) rows_of(t, j + 1, row);  // lands while the next stage is awaited
                if (++s == NS) {
                    s = 0;
                    ++round;
                }
            }
        }
        // copies in flight land before the CTA may end (they have, unless a wait gave up)
        for (uint32_t d = it > NS ? it - NS : 0; d < it; ++d) mbar_wait(&full[d % NS], (d / NS) & 1, err, kErrWaitDrain);
    } else if (warp == 6) {
        // ------------------------------------------------ Q of each piece
        if (lane == 0) {
            uint32_t pc = 0;
            for (int ti = t_begin; ti < t_end; ++ti, ++pc) {
                const int q_row = a.tiles[ti].q_row;
                if (pc > 0 && !mbar_wait(q_empty, (pc - 1) & 1, err, kErrWaitEmpty)) break;
                mbar_arrive_expect_tx(q_full, kLtChunks * q_chunk);
                for (int c = 0; c < kLtChunks; ++c) tma_load_2d(q_sm + c * q_chunk, &tm_q, q_full, c * 64, q_row);
            }
            if (pc > 0) mbar_wait(q_full, (pc - 1) & 1, err, kErrWaitDrain);
        }
    } else if (warp == 5) {
        // ------------------------------------------------ MMAs
        constexpr uint32_t ID_S = idesc_bf16_f32(64, kLatentKeys, 0, 0);
        constexpr uint32_t ID_O = idesc_bf16_f32(64, 256, 0, 1);
        const uint64_t dQ = smem_desc(smem_u32(q_sm), 16, 1024, kSwizzle128B);
        const uint64_t dK = smem_desc(smem_u32(k_sm), 16, 1024, kSwizzle128B);
        const uint64_t dP = smem_desc(smem_u32(p_sm), 16, 1024, kSwizzle128B);
        // values: N-major, 64-column chunks CHUNK apart, 8-key groups 1024 bytes apart
        const uint64_t dV = smem_desc(smem_u32(k_sm), L::CHUNK, 1024, kSwizzle128B);
        auto add = [](uint64_t d, uint32_t off) { return d + (off >> 4); };
        uint32_t it0 = 0, pc = 0;             // tiles before this piece
        uint32_t ss = 0, sr = 0, ps = 0;      // stage and round of the next S, stage of the next PV
        bool ok = true;
        for (int ti = t_begin; ti < t_end && ok; ++ti, ++pc) {
            const LatentTile t = ti == t_begin ? first_tile : a.tiles[ti];
            ok = mbar_wait(q_full, pc & 1, err, kErrWaitFull);
            // S runs at most three tiles ahead of PV: S(it)'s buffer was last read by the softmax of tile
            // it - 4, whose P has been awaited.  PV goes first when both have their operands.
            int js = 0, jp = 0;
            uint32_t polls = 0;
            while (jp < t.ntiles && ok) {
                const uint32_t ip = it0 + jp;
                if (js > jp && __all_sync(0xffffffffu, mbar_test_wait(&p_full[ip & 1], (ip >> 1) & 1))) {
                    if (jp == 0 && pc > 0) ok = mbar_wait(o_free, (pc - 1) & 1, err, kErrWaitEmpty);
                    if (!ok) break;
                    // Cache rows of the sequence's last page past its end hold anything; their P is 0, but
                    // 0 * NaN would reach O: zero them
                    const int key0 = (t.tile0 + jp) * kLatentKeys;
                    const int zb = max(t.length, key0), ze = min((t.length + P - 1) & ~(P - 1), key0 + kLatentKeys);
                    if (zb < ze) {
                        uint8_t *vs = k_sm + ps * L::TILE;
                        for (int e = lane; e < (ze - zb) * kLtValueChunks * 8; e += 32) {
                            const int k = zb - key0 + e / (kLtValueChunks * 8), c = e % (kLtValueChunks * 8);
                            *reinterpret_cast<uint4 *>(vs + (c >> 3) * L::CHUNK + swz128(k, c & 7)) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    tc_fence_after();
                    const uint64_t p = add(dP, (ip & 1) * 64), v = add(dV, ps * L::TILE);
#pragma unroll
                    for (int kk = 0; kk < kLatentKeys / 16; ++kk)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            mma_ss_elect(tmem + 256u * h, add(p, kk * 32), add(v, h * 4 * L::CHUNK + kk * 2048), ID_O,
                                         (jp > 0 || kk > 0) ? 1u : 0u);
                    mma_commit_elect(&empty[ps]);
                    mma_commit_elect(&pv_done[ip & 1]);
                    if (++ps == NS) ps = 0;
                    ++jp;
                    polls = 0;
                } else if (js < t.ntiles && js < jp + 4 &&
                           __all_sync(0xffffffffu, mbar_test_wait(&full[ss], sr & 1))) {
                    const uint32_t is = it0 + js;
                    tc_fence_after();
                    const uint64_t k = add(dK, ss * L::TILE);
#pragma unroll
                    for (int kk = 0; kk < kLatentWidth / 16; ++kk)
                        mma_ss_elect(s_base + 32u * (is & 3), add(dQ, (kk / 4) * q_chunk + (kk % 4) * 32),
                                     add(k, (kk / 4) * L::CHUNK + (kk % 4) * 32), ID_S, kk > 0 ? 1u : 0u);
                    mma_commit_elect(&s_full[is & 3]);
                    if (++ss == NS) {
                        ss = 0;
                        ++sr;
                    }
                    if (++js == t.ntiles) mma_commit_elect(q_empty);  // the piece's last reader of Q
                    polls = 0;
                } else if (++polls == kLtPolls) {
                    if (lane == 0) atomicCAS(err, 0, (int)kErrWaitFull);
                    ok = false;
                }
            }
            it0 += t.ntiles;
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
        uint32_t it = 0, pc = 0;
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
            float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;
            for (int j = 0; j < t.ntiles; ++j, ++it) {
                if (!mbar_wait(&s_full[it & 3], (it >> 2) & 1, err, kErrWaitFull)) {
                    ok = false;
                    break;
                }
                if (idle) {  // P's rows of this warp stay as they are: O's are never read
                    if (it >= 2 && !mbar_wait(&pv_done[it & 1], ((it >> 1) - 1) & 1, err, kErrWaitFull)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive(&p_full[it & 1]);
                    continue;
                }
                tc_fence_after();
                uint32_t r[16];
                tmem_ld16x32(s_base + lane_off + 32u * (it & 3), r);
                tmem_wait_ld();
                const int key0 = (t.tile0 + j) * kLatentKeys;
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
                if (key0 < lo_max || key0 + kLatentKeys - 1 > hi_min) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int k = key0 + 8 * (i >> 2) + 2 * quad + (i & 1);
                        const bool sees = (i & 2) ? ((k >= lo_b) & (k <= hi_b)) : ((k >= lo_a) & (k <= hi_a));
                        x[i] = sees ? x[i] : -INFINITY;
                    }
                }
                float mx_a = fmaxf(max3f(x[0], x[1], x[4]), max3f(x[5], x[8], x[9]));
                float mx_b = fmaxf(max3f(x[2], x[3], x[6]), max3f(x[7], x[10], x[11]));
                mx_a = max3f(mx_a, x[12], x[13]);
                mx_b = max3f(mx_b, x[14], x[15]);
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
                float sum_a = 0.f, sum_b = 0.f;
                uint32_t pk[8];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float p0 = ex2_ftz(fmaf(x[4 * c], sl, -r_a)), p1 = ex2_ftz(fmaf(x[4 * c + 1], sl, -r_a));
                    const float p2 = ex2_ftz(fmaf(x[4 * c + 2], sl, -r_b)), p3 = ex2_ftz(fmaf(x[4 * c + 3], sl, -r_b));
                    sum_a += p0 + p1;
                    sum_b += p2 + p3;
                    pk[2 * c] = pack_bf16(p0, p1);
                    pk[2 * c + 1] = pack_bf16(p2, p3);
                }
                l_a = l_a * al_a + sum_a;
                l_b = l_b * al_b + sum_b;
                // P's half was last read by PV(it - 2)
                if (it >= 2 && !mbar_wait(&pv_done[it & 1], ((it >> 1) - 1) & 1, err, kErrWaitFull)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    *reinterpret_cast<uint32_t *>(pa + swz128(row_a, c + 4 * (it & 1))) = pk[2 * c];
                    *reinterpret_cast<uint32_t *>(pa + swz128(row_b, c + 4 * (it & 1))) = pk[2 * c + 1];
                }
                if (any && j > 0) {
                    // O may be touched once PV(it - 1) has completed
                    if (!mbar_wait(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, err, kErrWaitFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
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
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[it & 1]);
            }
            if (!ok) break;
            // the piece's O
            l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
            l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
            l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
            l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
            if (!mbar_wait(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, err, kErrWaitFull)) break;
            tc_fence_after();
            // a piece may hold no visible key of a row (causal, several tokens): weight 0, lse -inf
            const float inv_a = l_a == 0.f ? 0.f : 1.f / l_a, inv_b = l_b == 0.f ? 0.f : 1.f / l_b;
            const float lse_a = l_a == 0.f ? -INFINITY : m_a + log2f(l_a);
            const float lse_b = l_b == 0.f ? -INFINITY : m_b + log2f(l_b);
            const size_t g_a = (size_t)t.q_row + row_a, g_b = (size_t)t.q_row + row_b;
            float *po = a.part_o + (size_t)max(t.partial, 0) * kLatentRows * kLatentDim;
#pragma unroll 1
            for (int c0 = 0; c0 < (idle ? 0 : kLatentDim); c0 += 64) {
                uint32_t o[32];
                tmem_ld16x64(tmem + lane_off + c0, o);
                tmem_wait_ld();
                float f[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {  // select, not multiply: 0 * NaN of a key the row does not see
                    const float inv = (i & 2) ? inv_b : inv_a;
                    f[i] = inv == 0.f ? 0.f : __uint_as_float(o[i]) * inv;
                }
                if (t.partial < 0) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int col = c0 + 8 * c + 2 * quad;
                        if (live_a)
                            *reinterpret_cast<uint32_t *>(a.out + g_a * kLatentDim + col) = pack_bf16(f[4 * c], f[4 * c + 1]);
                        if (live_b)
                            *reinterpret_cast<uint32_t *>(a.out + g_b * kLatentDim + col) =
                                pack_bf16(f[4 * c + 2], f[4 * c + 3]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int col = c0 + 8 * c + 2 * quad;
                        if (live_a)
                            *reinterpret_cast<float2 *>(po + (size_t)row_a * kLatentDim + col) =
                                make_float2(f[4 * c], f[4 * c + 1]);
                        if (live_b)
                            *reinterpret_cast<float2 *>(po + (size_t)row_b * kLatentDim + col) =
                                make_float2(f[4 * c + 2], f[4 * c + 3]);
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

// Join of the pieces of a cut unit: with w_i = 2^(lse_i - max lse), o = sum w_i o_i / sum w_i.  A CTA of
// 128 threads per query row, four columns a thread, eight pieces in flight; the first eight are
// requested before the weights are known.  Bounded by the trips to L2: one for the lse values and the
// first eight pieces, one more per eight.
constexpr int kLtMergeBatch = 8;
__global__ void __launch_bounds__(kLatentDim / 4) latent_merge_kernel(const LatentMerge *merges, const float *part_o,
                                                                      const float *part_lse, __nv_bfloat16 *out,
                                                                      float *lse) {
    const LatentMerge m = merges[blockIdx.y];
    const int row = blockIdx.x, lane = threadIdx.x & 31;
    griddep_wait();
    griddep_launch();
    if (row >= m.n_rows) return;
    const float *pl = part_lse + (size_t)m.first * kLatentRows + row;
    const float *po = part_o + ((size_t)m.first * kLatentRows + row) * kLatentDim + threadIdx.x * 4;
    constexpr size_t STEP = (size_t)kLatentRows * kLatentDim;
    float4 v[kLtMergeBatch];
#pragma unroll
    for (int i = 0; i < kLtMergeBatch; ++i)
        if (i < m.count) v[i] = __ldcg(reinterpret_cast<const float4 *>(po + i * STEP));
    float mx = -INFINITY;
    const float l0 = lane < m.count ? __ldcg(pl + (size_t)lane * kLatentRows) : -INFINITY;
    for (int i = lane + 32; i < m.count; i += 32) mx = fmaxf(mx, __ldcg(pl + (size_t)i * kLatentRows));
    mx = fmaxf(mx, l0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float w0 = exp2f(l0 - mx);  // the first 32 pieces' weights, one a lane
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int i0 = 0; i0 < m.count; i0 += kLtMergeBatch) {
        if (i0 > 0) {
#pragma unroll
            for (int i = 0; i < kLtMergeBatch; ++i)
                if (i0 + i < m.count) v[i] = __ldcg(reinterpret_cast<const float4 *>(po + (i0 + i) * STEP));
        }
#pragma unroll
        for (int i = 0; i < kLtMergeBatch; ++i) {
            const float s = __shfl_sync(0xffffffffu, w0, (i0 + i) & 31);
            if (i0 + i < m.count) {
                const float w = i0 + i < 32 ? s : exp2f(__ldcg(pl + (size_t)(i0 + i) * kLatentRows) - mx);
                sum += w;
                acc.x += w * v[i].x;
                acc.y += w * v[i].y;
                acc.z += w * v[i].z;
                acc.w += w * v[i].w;
            }
        }
    }
    const float inv = 1.f / sum;  // every row sees a key in some piece, so the largest weight is 1
    *reinterpret_cast<uint2 *>(out + ((size_t)m.q_row + row) * kLatentDim + threadIdx.x * 4) =
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
    a.stages = dev::LtSmem::stages(p.box_q);
    const size_t smem = 1024 + dev::LtSmem::bytes(a.stages, p.box_q);  // one CTA per SM
    cudaError_t e = set_smem_limit((const void *)dev::latent_kernel, 227 * 1024, st);
    if (e == cudaSuccess)
        e = launch_pdl(dev::latent_kernel, dim3(p.ctas), dim3(dev::kLtThreads), smem, st, tm_cache, tm_q, a);
    if (e == cudaSuccess && p.num_merge)
        e = launch_pdl(dev::latent_merge_kernel, dim3(p.box_q, p.num_merge), dim3(kLatentDim / 4), 0, st,
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
