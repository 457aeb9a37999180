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
//    tensor-memory columns: an M = 64 accumulator fills 16 of the 32 lanes of each warp's quarter,
//    O the lower ones, and S (two buffers of 64 columns) the upper ones.  An M = 64 MMA takes as
//    long as M = 128 (measured 128 cycles at N = 256, 32 at N = 64): 2,183 cycles a tile, below the
//    3,190 cycles in which an SM's share of HBM delivers it, so up to 64 rows stay bandwidth-bound.
//  * Shared memory: Q 72 KB, two stages of 72 KB (a tile serves as keys and, its first 512 columns,
//    as values), P 8 KB.
//  * Warps 0-3 softmax (16 rows each, a quad per row pair), 4 copies tiles, 5 issues MMAs, 6 copies Q.
//  * The running maximum moves (and O is rescaled in tensor memory) only when it grows by more than
//    2^8.  Sums and maxima are 32-bit; P is rounded to bf16 for the MMA (relative 2^-8 a weight at
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
    static constexpr uint32_t CHUNK = 64 * 128;               // 64 rows x 64 columns
    static constexpr uint32_t TILE = kLtChunks * CHUNK;       // 73,728
    static constexpr int STAGES = 2;
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t K_OFF = TILE;
    static constexpr uint32_t P_OFF = K_OFF + STAGES * TILE;
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

__global__ void __launch_bounds__(kLtThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tm_cache, const __grid_constant__ CUtensorMap tm_q,
                  const LatentArgs a) {
    using L = LtSmem;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 11);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int t_begin = a.cta_ptr[blockIdx.x], t_end = a.cta_ptr[blockIdx.x + 1];
    int *const err = &a.hdr->err;
    const int P = a.page_size;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&s_full[s], 1);
        }
        mbar_init(p_full, 4);
        mbar_init(pv_done, 1);
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(o_free, 4);
        fence_barrier_init();
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

    if (warp == 4) {
        // ------------------------------------------------ tiles: one lane per (box, chunk)
        const int R = a.box_rows;
        const int nb = kLatentKeys / R, jobs = nb * kLtChunks;  // 9, 18, 36 or 72
        if (lane == 0) prefetch_tmap(&tm_cache);
        uint32_t it = 0;
        bool ok = true;
        for (int ti = t_begin; ti < t_end && ok; ++ti) {
            const LatentTile t = a.tiles[ti];
            const int npages = (t.length + P - 1) >> a.page_shift;
            for (int j = 0; j < t.ntiles; ++j, ++it) {
                const int key0 = (t.tile0 + j) * kLatentKeys;
                int row[3];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int job = lane + 32 * i;
                    const int kb = key0 + (job / kLtChunks) * R, pg = kb >> a.page_shift;
                    row[i] = job < jobs && pg < npages ? a.pages[t.kv_base + pg] * P + (kb & (P - 1)) : a.oob_row;
                }
                const int s = it & 1;
                if (it >= 2 && !mbar_wait(&empty[s], ((it >> 1) - 1) & 1, err, kErrWaitEmpty)) {
                    ok = false;
                    break;
                }
                uint8_t *st = sm + L::K_OFF + s * L::TILE;
                if (lane == 0) mbar_arrive_expect_tx(&full[s], L::TILE);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int job = lane + 32 * i;
                    if (job < jobs) {
                        const int b = job / kLtChunks, c = job % kLtChunks;
                        tma_load_2d(st + c * L::CHUNK + b * R * 128, &tm_cache, &full[s], c * 64, row[i]);
                    }
                }
            }
        }
        // copies in flight land before the CTA may end (they have, unless a wait gave up)
        for (uint32_t d = it > 2 ? it - 2 : 0; d < it; ++d) mbar_wait(&full[d & 1], (d >> 1) & 1, err, kErrWaitDrain);
    } else if (warp == 6) {
        // ------------------------------------------------ Q of each piece
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            uint32_t pc = 0;
            for (int ti = t_begin; ti < t_end; ++ti, ++pc) {
                const int q_row = a.tiles[ti].q_row;
                if (pc > 0 && !mbar_wait(q_empty, (pc - 1) & 1, err, kErrWaitEmpty)) break;
                mbar_arrive_expect_tx(q_full, (uint32_t)(kLtChunks * a.box_q) * 128u);
                for (int c = 0; c < kLtChunks; ++c)
                    tma_load_2d(sm + L::Q_OFF + c * L::CHUNK, &tm_q, q_full, c * 64, q_row);
            }
            if (pc > 0) mbar_wait(q_full, (pc - 1) & 1, err, kErrWaitDrain);
        }
    } else if (warp == 5) {
        // ------------------------------------------------ MMAs
        constexpr uint32_t ID_S = idesc_bf16_f32(64, kLatentKeys, 0, 0);
        constexpr uint32_t ID_O = idesc_bf16_f32(64, 256, 0, 1);
        const uint64_t dQ = smem_desc(smem_u32(sm + L::Q_OFF), 16, 1024, kSwizzle128B);
        const uint64_t dK = smem_desc(smem_u32(sm + L::K_OFF), 16, 1024, kSwizzle128B);
        const uint64_t dP = smem_desc(smem_u32(sm + L::P_OFF), 16, 1024, kSwizzle128B);
        // values: N-major, 64-column chunks CHUNK apart, 8-key groups 1024 bytes apart
        const uint64_t dV = smem_desc(smem_u32(sm + L::K_OFF), L::CHUNK, 1024, kSwizzle128B);
        auto add = [](uint64_t d, uint32_t off) { return d + (off >> 4); };
        bool ok = true;
        auto issue_s = [&](uint32_t it, bool last) {
            const uint32_t b = it & 1;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kLatentWidth / 16; ++kk) {
                const uint32_t off = (kk / 4) * L::CHUNK + (kk % 4) * 32;
                mma_ss_elect(s_base + 64u * b, add(dQ, off), add(dK, b * L::TILE + off), ID_S, kk > 0 ? 1u : 0u);
            }
            mma_commit_elect(&s_full[b]);
            if (last) mma_commit_elect(q_empty);  // the piece's last reader of Q
        };
        uint32_t it = 0, pc = 0;
        for (int ti = t_begin; ti < t_end && ok; ++ti, ++pc) {
            const LatentTile t = a.tiles[ti];
            ok = mbar_wait(q_full, pc & 1, err, kErrWaitFull) && mbar_wait(&full[it & 1], (it >> 1) & 1, err, kErrWaitFull);
            if (!ok) break;
            issue_s(it, t.ntiles == 1);
            for (int j = 0; j < t.ntiles; ++j, ++it) {
                const uint32_t b = it & 1, nx = it + 1;
                // Cache rows of the sequence's last page past its end hold anything; their P is 0, but
                // 0 * NaN would reach O: zero them (S of these columns is masked whatever it reads)
                const int key0 = (t.tile0 + j) * kLatentKeys;
                const int zb = max(t.length, key0), ze = min((t.length + P - 1) & ~(P - 1), key0 + kLatentKeys);
                if (zb < ze) {
                    uint8_t *vs = sm + L::K_OFF + b * L::TILE;
                    for (int e = lane; e < (ze - zb) * kLtValueChunks * 8; e += 32) {
                        const int k = zb - key0 + e / (kLtValueChunks * 8), c = e % (kLtValueChunks * 8);
                        *reinterpret_cast<uint4 *>(vs + (c >> 3) * L::CHUNK + swz128(k, c & 7)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (j == 0 && pc > 0) ok = mbar_wait(o_free, (pc - 1) & 1, err, kErrWaitEmpty);
                // S(it + 1) and PV(it) in the order in which their operands arrive: with the next tile
                // there, S runs under this tile's softmax; else PV goes first and frees its stage.  (S's
                // buffer was last read by the softmax of tile it - 1, whose P has been awaited.)
                bool need_s = j + 1 < t.ntiles, have_p = false;
                for (uint32_t i = 0; i < kLtPolls && ok && !have_p; ++i) {
                    if (need_s && __all_sync(0xffffffffu, mbar_test_wait(&full[nx & 1], (nx >> 1) & 1))) {
                        issue_s(nx, j + 2 == t.ntiles);
                        need_s = false;
                    }
                    have_p = __all_sync(0xffffffffu, mbar_test_wait(p_full, it & 1));
                }
                if (!have_p) {
                    if (ok && lane == 0) atomicCAS(err, 0, (int)kErrWaitFull);
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int kk = 0; kk < kLatentKeys / 16; ++kk)
                        mma_ss_elect(tmem + 256u * h, add(dP, kk * 32),
                                     add(dV, b * L::TILE + h * 4 * L::CHUNK + kk * 2048), ID_O,
                                     (j > 0 || kk > 0) ? 1u : 0u);
                mma_commit_elect(pv_done);
                mma_commit_elect(&empty[b]);
                if (need_s) {
                    ok = mbar_wait(&full[nx & 1], (nx >> 1) & 1, err, kErrWaitFull);
                    if (!ok) break;
                    issue_s(nx, j + 2 == t.ntiles);
                }
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
        uint8_t *const pa = sm + L::P_OFF + quad * 4;
        uint32_t it = 0, pc = 0;
        bool ok = true;
        for (int ti = t_begin; ti < t_end && ok; ++ti, ++pc) {
            const LatentTile t = a.tiles[ti];
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
            float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;
            for (int j = 0; j < t.ntiles; ++j, ++it) {
                const uint32_t b = it & 1;
                if (!mbar_wait(&s_full[b], (it >> 1) & 1, err, kErrWaitFull)) {
                    ok = false;
                    break;
                }
                if (idle) {
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
                if (key0 < max(lo_a, lo_b) || key0 + kLatentKeys - 1 > min(hi_a, hi_b)) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int k = key0 + 8 * (i >> 2) + 2 * quad + (i & 1);
                        const bool sees = (i & 2) ? (k >= lo_b && k <= hi_b) : (k >= lo_a && k <= hi_a);
                        x[i] = sees ? x[i] : -INFINITY;
                    }
                }
                float mx_a = fmaxf(x[0], x[1]), mx_b = fmaxf(x[2], x[3]);
#pragma unroll
                for (int c = 1; c < 8; ++c) {
                    mx_a = max3f(mx_a, x[4 * c], x[4 * c + 1]);
                    mx_b = max3f(mx_b, x[4 * c + 2], x[4 * c + 3]);
                }
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
                uint32_t pk[16];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float p0 = ex2_ftz(fmaf(x[4 * c], sl, -r_a)), p1 = ex2_ftz(fmaf(x[4 * c + 1], sl, -r_a));
                    const float p2 = ex2_ftz(fmaf(x[4 * c + 2], sl, -r_b)), p3 = ex2_ftz(fmaf(x[4 * c + 3], sl, -r_b));
                    sum_a += p0 + p1;
                    sum_b += p2 + p3;
                    pk[2 * c] = pack_bf16(p0, p1);
                    pk[2 * c + 1] = pack_bf16(p2, p3);
                }
                l_a = l_a * al_a + sum_a;
                l_b = l_b * al_b + sum_b;
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
                if (any && j > 0) {
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

// Join of the pieces of a cut unit: with w_i = 2^(lse_i - max lse), o = sum w_i o_i / sum w_i.  One
// warp per query row, four to a CTA; a lane holds 16 columns as four float4 of 128 columns apart, so
// every load of a warp is 512 consecutive bytes.  Bounded by the partials' trip through L2.
constexpr int kLtMergeWarps = 4;
__global__ void __launch_bounds__(kLtMergeWarps * 32) latent_merge_kernel(const LatentMerge *merges, const float *part_o,
                                                                          const float *part_lse, __nv_bfloat16 *out,
                                                                          float *lse) {
    const LatentMerge m = merges[blockIdx.x];
    const int row = blockIdx.y * kLtMergeWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    griddep_wait();
    griddep_launch();
    if (row >= m.n_rows) return;
    const float *pl = part_lse + (size_t)m.first * kLatentRows + row;
    float mx = -INFINITY;
    for (int i = lane; i < m.count; i += 32) mx = fmaxf(mx, __ldcg(pl + (size_t)i * kLatentRows));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float4 acc[4] = {};
    float sum = 0.f;
    const float *po = part_o + ((size_t)m.first * kLatentRows + row) * kLatentDim + lane * 4;
#pragma unroll 4
    for (int i = 0; i < m.count; ++i) {
        const float w = exp2f(__ldcg(pl + (size_t)i * kLatentRows) - mx);
        sum += w;
        const float *p = po + (size_t)i * kLatentRows * kLatentDim;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + c * 128));
            acc[c].x += w * v.x;
            acc[c].y += w * v.y;
            acc[c].z += w * v.z;
            acc[c].w += w * v.w;
        }
    }
    const float inv = 1.f / sum;  // every row sees a key in some piece, so the largest weight is 1
    __nv_bfloat16 *dst = out + ((size_t)m.q_row + row) * kLatentDim + lane * 4;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint2 *>(dst + c * 128) =
            make_uint2(pack_bf16(acc[c].x * inv, acc[c].y * inv), pack_bf16(acc[c].z * inv, acc[c].w * inv));
    if (lse && lane == 0) lse[(size_t)m.q_row + row] = (mx + log2f(sum)) * kLtLn2;
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
        e = launch_pdl(dev::latent_merge_kernel, dim3(p.num_merge, (p.box_q + dev::kLtMergeWarps - 1) / dev::kLtMergeWarps),
                       dim3(dev::kLtMergeWarps * 32), 0, st, reinterpret_cast<const LatentMerge *>(w + p.off_merge),
                       static_cast<const float *>(a.part_o), static_cast<const float *>(a.part_lse), a.out, lse);
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
