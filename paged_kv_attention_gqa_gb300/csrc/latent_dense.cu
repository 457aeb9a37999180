// Latent attention, expanded form (pkv_latent_run_dense): prompts over contiguous per-head keys
// [k_nope | k_rope] (128 + 64 columns, the rope part shared by all heads) and values (128), made from
// the latent vectors by the caller.  s_ij = sm_scale * (<qn_i, kn_j> + <qr_i, kr_j>); softmax over the
// keys a query sees; o_i = sum_j p_ij v_j.
//
// Bounded by the tensor cores: 640 operations per query, key and head, on operands that fit L2.  A
// work tile is two query tiles of 128 tokens of one head that share every 64-key tile, one CTA per SM:
//  * warp 8 copies Q0 and Q1 once, then streams the K tiles ([k_nope | k_rope], 24 KB) and the V tiles
//    (16 KB) through three stages each; a stage is refilled as soon as the MMAs of both query tiles
//    that read it are done;
//  * warps 9 and 10 issue S = Q K^T of Q0 and Q1 (12 k-steps, N = 64), up to two tiles ahead of the
//    softmax, warps 11 and 12 O += P V (4 k-steps, N = 128, P from tensor memory over its S);
//  * warps 0-3 and 4-7 run the softmax of Q0 and Q1, a thread a query.  The running maximum moves, and
//    O is rescaled, only when it grows by more than 2^8;
//  * warps 13 and 14 look over the value tiles that some queries of Q0 or Q1 see and others do not
//    (causal diagonal, window edges) as they land: the weight of a value that a query does not see is 0,
//    but 0 * NaN would reach it.  A tile that holds NaN or infinities there is left to the softmax
//    warps, each query adding the values it sees.  (In the PV warps, between two tiles, the look cost 14 us; in
//    warps of its own 6.)
// Tensor memory: two S buffers of 64 columns and an O of 128 for each query tile, all 512 columns.
// Tiles of 128 keys leave room for one S each; then a query tile's S, softmax and PV wait for one
// another, two chains of 4,600 cycles per 128 keys against 2,560 of MMAs: 305 us (32 heads, prompts of
// 801 to 4,093 tokens, 9,788 in all, causal) when this kernel had one issuing warp a query tile and waits that
// looped from the start; that form has not been timed with what came later.  N = 64 costs 48 cycles a k-step of S (the A operand's
// reads) in place of 32, 3,328 cycles per 128 keys.  A warp's MMA takes it 33 cycles to issue, a commit
// or a wait, even for a completed phase, 100 to 200; so S and PV of both query tiles have a warp each:
// 241 us in short runs of calls and 251 in long ones (234 and 245 without the look at the values), the
// operations at the measured rate being 160.  (One warp for S and PV of a query tile: 265 us, one for both
// query tiles: 412 us; PV as two N = 64 halves: + 10 us; all in short runs, without the look.)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "latent.h"
#include "launch.h"
#include "tcgen05.cuh"

namespace pkv {
namespace dev {

constexpr int kLdKeys = 64, kLdQueries = 128;
constexpr int kLdThreads = 512;
// Registers: 512 x 128 at launch = 65,536; the softmax groups take most of the other warps' share
// (256 x 64 + 256 x 184 = 63,488).
constexpr int kLdLaunchRegs = 128, kLdSoftmaxRegs = 184, kLdOtherRegs = 64;
static_assert(256 * kLdOtherRegs + 256 * kLdSoftmaxRegs <= kLdThreads * kLdLaunchRegs, "setmaxnreg split fits the launch");
constexpr float kLdRescale = 8.f;  // log2
constexpr float kLdLn2 = 0.6931471805599453f;

struct LdSmem {
    static constexpr uint32_t QCHUNK = 128 * 128;        // 128 queries x 64 columns
    static constexpr uint32_t CHUNK = kLdKeys * 128;     // 64 keys x 64 columns
    static constexpr int QC = 3, KC = 3, VC = 2, STAGES = 3;
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t K_OFF = 2 * QC * QCHUNK;
    static constexpr uint32_t V_OFF = K_OFF + STAGES * KC * CHUNK;
    static constexpr uint32_t BAR_OFF = V_OFF + STAGES * VC * CHUNK;
    static constexpr uint32_t BYTES = BAR_OFF + 320;
};
static_assert(1024 + LdSmem::BYTES <= 227 * 1024, "the expanded latent kernel fits shared memory");

struct LatentDenseArgs {
    __nv_bfloat16 *out;
    float *lse;
    const PrefillTile *tiles;
    PlanHeader *hdr;
    int num_heads;
};

// The tiles (counted from kt0) with keys that some queries of a query tile see and others do not: those below
// `low`, whose keys start before `lo_max`, and those from `high`, that hold key `hi_min` + 1 or later ones.
struct LdMixed {
    int lo_max, hi_min, low, high;
    __device__ __forceinline__ bool operator()(int j) const { return j < low || j >= high; }
};
__device__ __forceinline__ LdMixed ld_mixed(const PrefillTile &t, int x, int kt0, int causal, int window_left) {
    const int first = t.pos0 + x * kLdQueries, last = t.pos0 + min(t.n_q, (x + 1) * kLdQueries) - 1;
    LdMixed m;
    m.lo_max = window_left >= 0 ? max(0, last - window_left) : 0;
    m.hi_min = causal == 1 ? first : t.length - 1;
    m.low = (m.lo_max + kLdKeys - 1) / kLdKeys - kt0;
    m.high = m.hi_min + 1 < t.length ? (m.hi_min + 1) / kLdKeys - kt0 : INT_MAX;
    return m;
}

// O += P V of one tile without the tensor cores, for tiles that hold NaN or infinities in a key that
// some queries see and others do not: each query adds the keys [lo, hi] that it sees alone.  P is read back
// from tensor memory.
__device__ __noinline__ void ld_pv_rows(uint32_t o_addr, uint32_t p_addr, const uint8_t *v, int key0, int lo, int hi,
                                        float alpha, bool first) {
#pragma unroll 1
    for (int c0 = 0; c0 < kLatentV; c0 += 32) {
        uint32_t r[32];
        float o[32];
        tmem_ld32(o_addr + c0, r);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = first ? 0.f : __uint_as_float(r[c]) * alpha;
        const uint8_t *chunk = v + (c0 >> 6) * LdSmem::CHUNK;
#pragma unroll 1
        for (int k = 0; k < kLdKeys; ++k) {
            __syncwarp();
            const uint32_t pair = tmem_ld1(p_addr + (k >> 1));
            tmem_wait_ld();
            const float p = __uint_as_float((k & 1) ? pair & 0xffff0000u : pair << 16);
            if (key0 + k >= lo && key0 + k <= hi) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(chunk + swz128(k, ((c0 & 63) >> 3) + i));
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        o[8 * i + 2 * c] = fmaf(p, __uint_as_float(w[c] << 16), o[8 * i + 2 * c]);
                        o[8 * i + 2 * c + 1] = fmaf(p, __uint_as_float(w[c] & 0xffff0000u), o[8 * i + 2 * c + 1]);
                    }
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(o[c]);
        tmem_st32(o_addr + c0, r);
    }
    tmem_wait_st();
}

__global__ void __launch_bounds__(kLdThreads, 1)
    latent_dense_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v,
                        const LatentDenseArgs a) {
    using L = LdSmem;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR_OFF);
    uint64_t *q_full = bars + 0;     // [2] Q_X landed
    uint64_t *k_full = bars + 2;     // [3] K stage landed
    uint64_t *k_empty = bars + 5;    // [3] the S MMAs that read it completed (one arrival per query tile)
    uint64_t *v_full = bars + 8;     // [3] V stage landed
    uint64_t *v_empty = bars + 11;   // [3] the PV MMAs that read it completed, and it has been looked over
    uint64_t *s_full = bars + 14;    // [2][2] S_X(j) in buffer j & 1
    uint64_t *p_full = bars + 18;    // [2][2] P_X(j) written over S_X(j) (and O_X rescaled if it had to be)
    uint64_t *pv_done = bars + 22;   // [2][2] PV_X(j) completed, of buffer j & 1
    uint64_t *v_tail = bars + 26;    // the value rows past the segment are zero (at most one tile)
    uint64_t *checked = bars + 27;   // [2][3] the V stage has been looked over for X
    uint32_t *by_rows = reinterpret_cast<uint32_t *>(bars + 33);  // [2][3] its PV goes by rows
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 36);

    const PrefillTile t = a.tiles[blockIdx.x];
    int *const err = &a.hdr->err;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const bool two = t.n_q > kLdQueries;  // the tile's tokens reach into Q1
    const int kt0 = t.key_begin / kLdKeys;
    const int nt = (t.key_end + kLdKeys - 1) / kLdKeys - kt0;  // >= 1: every query sees itself
    const int causal = a.hdr->causal;
    // Q0's own tiles: of a causal pair it does not see the last ones
    const int q0_end = causal == 1 ? min(t.length, t.pos0 + min(t.n_q, kLdQueries)) : t.length;
    const int nt0 = two ? min(nt, (q0_end + kLdKeys - 1) / kLdKeys - kt0) : nt;

    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 1);
            mbar_init(&s_full[2 * x], 1);
            mbar_init(&s_full[2 * x + 1], 1);
            mbar_init(&p_full[2 * x], 4);
            mbar_init(&p_full[2 * x + 1], 4);
            mbar_init(&pv_done[2 * x], 1);
            mbar_init(&pv_done[2 * x + 1], 1);
        }
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&v_full[s], 1);
            mbar_init(&k_empty[s], two ? 2 : 1);
            mbar_init(&v_empty[s], two ? 4 : 2);
            mbar_init(&checked[s], 1);
            mbar_init(&checked[3 + s], 1);
        }
        mbar_init(v_tail, 1);
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch();
    const uint32_t tmem = *tmem_holder;
    auto S_col = [tmem](int x) { return tmem + 128u * (uint32_t)x; };  // the second buffer 64 columns on
    auto O_col = [tmem](int x) { return tmem + 256u + 128u * (uint32_t)x; };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLdOtherRegs));
        if (warp == 8) {
            // ------------------------------------------------ copies: one thread, a box of 64 columns each
            if (lane == 0) {
                prefetch_tmap(&tm_q);
                prefetch_tmap(&tm_k);
                prefetch_tmap(&tm_r);
                prefetch_tmap(&tm_v);
                auto load_q = [&](int x) {
                    mbar_arrive_expect_tx(&q_full[x], L::QC * L::QCHUNK);
                    for (int c = 0; c < L::QC; ++c)
                        tma_load_3d(sm + L::Q_OFF + (x * L::QC + c) * L::QCHUNK, &tm_q, &q_full[x], c * 64,
                                    t.q_begin + x * kLdQueries, t.kv_head);
                };
                load_q(0);
                int j = 0;
                for (; j < nt; ++j) {
                    const int row = t.kv_base + (kt0 + j) * kLdKeys;  // first key row of the tile
                    const int s = j % L::STAGES, use = j / L::STAGES;
                    uint8_t *kd = sm + L::K_OFF + s * L::KC * L::CHUNK, *vd = sm + L::V_OFF + s * L::VC * L::CHUNK;
                    if (use > 0 && !mbar_wait(&k_empty[s], (use - 1) & 1, err, kErrWaitEmpty)) break;
                    mbar_arrive_expect_tx(&k_full[s], L::KC * L::CHUNK);
                    tma_load_3d(kd, &tm_k, &k_full[s], 0, row, t.kv_head);
                    tma_load_3d(kd + L::CHUNK, &tm_k, &k_full[s], 64, row, t.kv_head);
                    tma_load_2d(kd + 2 * L::CHUNK, &tm_r, &k_full[s], 0, row);
                    if (j == 0 && two) load_q(1);  // needed after S0(0)
                    if (use > 0 && !mbar_wait(&v_empty[s], (use - 1) & 1, err, kErrWaitEmpty)) {
                        mbar_wait(&k_full[s], use & 1, err, kErrWaitDrain);
                        break;
                    }
                    mbar_arrive_expect_tx(&v_full[s], L::VC * L::CHUNK);
                    tma_load_3d(vd, &tm_v, &v_full[s], 0, row, t.kv_head);
                    tma_load_3d(vd + L::CHUNK, &tm_v, &v_full[s], 64, row, t.kv_head);
                }
                // copies in flight land before the CTA may end (they have, unless a wait gave up)
                for (int d = max(0, j - L::STAGES); d < j; ++d) {
                    mbar_wait(&k_full[d % L::STAGES], (d / L::STAGES) & 1, err, kErrWaitDrain);
                    mbar_wait(&v_full[d % L::STAGES], (d / L::STAGES) & 1, err, kErrWaitDrain);
                }
            }
        } else if (warp == 9 || (warp == 10 && two)) {
            // ------------------------------------------------ S = Q K^T: warp 9 for Q0, warp 10 for Q1
            const int x = warp - 9, ntx = x == 0 ? nt0 : nt;
            constexpr uint32_t ID_S = idesc_bf16_f32(128, kLdKeys, 0, 0);
            const uint64_t dQ = smem_desc(smem_u32(sm + L::Q_OFF + x * L::QC * L::QCHUNK), 16, 1024, kSwizzle128B);
            const uint64_t dK = smem_desc(smem_u32(sm + L::K_OFF), 16, 1024, kSwizzle128B);
            const uint32_t hi = (uint32_t)(dQ >> 32);  // dK's too
            auto desc = [hi](uint32_t lo, uint32_t off) { return ((uint64_t)hi << 32) | (lo + (off >> 4)); };
            const uint32_t Sx = S_col(x);
            bool ok = mbar_wait(&q_full[x], 0, err, kErrWaitFull);
            int s = 0, ph = 0;  // stage and its phase
            for (int j = 0; j < nt && ok; ++j) {
                ok = mbar_wait(&k_full[s], ph, err, kErrWaitFull);
                if (j < ntx) {
                    // S_X(j) into buffer j & 1, which held P_X(j-2): PV_X(j-2) has completed
                    if (ok && j > 1) ok = mbar_wait(&pv_done[2 * x + (j & 1)], ((j >> 1) - 1) & 1, err, kErrWaitFull);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t lK = (uint32_t)dK + ((s * L::KC * L::CHUNK) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4 * L::KC; ++kk)
                        mma_ss_elect(Sx + 64u * (j & 1), desc((uint32_t)dQ, (kk >> 2) * L::QCHUNK + (kk & 3) * 32),
                                     desc(lK, (kk >> 2) * L::CHUNK + (kk & 3) * 32), ID_S, kk > 0 ? 1u : 0u);
                    mma_commit_elect(&s_full[2 * x + (j & 1)]);
                    mma_commit_elect(&k_empty[s]);
                } else if (ok && lane == 0) {
                    mbar_arrive(&k_empty[s]);  // a tile of the pair's that Q0 does not see
                }
                if (++s == L::STAGES) s = 0, ph ^= 1;
            }
            if (!ok)  // a wait gave up: let the MMAs in flight finish before the tensor memory is released
                for (uint32_t k = 0; k < 1024; ++k) __nanosleep(1000);
        } else if (warp == 11 || (warp == 12 && two)) {
            // ------------------------------------------------ O += P V: warp 11 for Q0, warp 12 for Q1
            const int x = warp - 11, ntx = x == 0 ? nt0 : nt;
            constexpr uint32_t ID_O = idesc_bf16_f32(128, kLatentV, 0, 1);
            // the leading offset steps from the first 64 value columns to the second
            const uint64_t dV = smem_desc(smem_u32(sm + L::V_OFF), L::CHUNK, 1024, kSwizzle128B);
            const uint32_t hi = (uint32_t)(dV >> 32);
            const uint32_t Sx = S_col(x), Ox = O_col(x);
            const LdMixed mixed = ld_mixed(t, x, kt0, causal, a.hdr->window_left);
            bool ok = true;
            int s = 0, ph = 0;
            for (int j = 0; j < nt && ok; ++j) {
                ok = mbar_wait(&v_full[s], ph, err, kErrWaitFull);
                if (!ok) break;
                if (j < ntx) {
                    // Value rows past the segment's end belong to the next segment (or are zero past the
                    // tensor): their P is 0, but 0 * NaN would reach O.  The last query tile's warp zeroes
                    // them; the other waits for that on the one tile that has them.
                    const int zb = t.length - (kt0 + j) * kLdKeys;  // >= 1: the tile holds a visible key
                    if (zb < kLdKeys) {
                        if (x == (two ? 1 : 0)) {
                            for (int e = lane; e < (kLdKeys - zb) * 16; e += 32) {
                                const int k = zb + (e >> 4), ch = e & 15;
                                *reinterpret_cast<uint4 *>(sm + L::V_OFF + (s * L::VC + (ch >> 3)) * L::CHUNK +
                                                           swz128(k, ch & 7)) = make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(v_tail);
                        } else {
                            ok = mbar_wait(v_tail, 0, err, kErrWaitFull);
                        }
                    }
                    if (ok) ok = mbar_wait(&p_full[2 * x + (j & 1)], (j >> 1) & 1, err, kErrWaitFull);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t lV = (uint32_t)dV + ((s * L::VC * L::CHUNK) >> 4);
                    if (!(mixed(j) && by_rows[3 * x + s])) {  // (written before the softmax warps arrived)
#pragma unroll
                        for (int kk = 0; kk < kLdKeys / 16; ++kk)
                            mma_ts_elect(Ox, Sx + 64u * (j & 1) + kk * 8, ((uint64_t)hi << 32) | (lV + kk * (2048 >> 4)),
                                         ID_O, (j > 0 || kk > 0) ? 1u : 0u);
                    }
                    mma_commit_elect(&pv_done[2 * x + (j & 1)]);
                    mma_commit_elect(&v_empty[s]);
                } else if (lane == 0) {
                    mbar_arrive(&v_empty[s]);
                }
                if (++s == L::STAGES) s = 0, ph ^= 1;
            }
            if (!ok)
                for (uint32_t k = 0; k < 1024; ++k) __nanosleep(1000);
        } else if (warp == 13 || (warp == 14 && two)) {
            // ------------------------------------------------ values that not all queries see
            // A NaN or an infinity among the values that some queries of X see and others do not would reach
            // all of them, as 0 * NaN: such tiles are left to the softmax warps, which add to each query the
            // keys it sees.  The stages are looked over as they land, ahead of their use; those that every
            // query sees are passed on at once.
            const int x = warp - 13, ntx = x == 0 ? nt0 : nt;
            const LdMixed mixed = ld_mixed(t, x, kt0, causal, a.hdr->window_left);
            int s = 0, ph = 0;
            for (int j = 0; j < nt; ++j) {
                if (!mbar_wait(&v_full[s], ph, err, kErrWaitFull)) break;
                if (j < ntx && mixed(j)) {
                    const int key0 = (kt0 + j) * kLdKeys, end = min(key0 + kLdKeys, t.length);
                    const int k_begin = (j < mixed.low ? key0 : max(key0, mixed.hi_min + 1)) - key0;
                    const int k_end = (j >= mixed.high ? end : min(end, mixed.lo_max)) - key0;
                    // a lane reads 16 bytes of every second key, four of them in flight
                    const uint8_t *const v = sm + L::V_OFF + (s * L::VC + ((lane >> 3) & 1)) * L::CHUNK;
                    uint32_t f0 = 0, f1 = 0;
                    for (int k0 = k_begin + (lane >> 4); k0 < k_end; k0 += 8) {
                        uint4 w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = *reinterpret_cast<const uint4 *>(v + swz128(min(k0 + 2 * i, k_end - 1), lane & 7));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f0 = keep_nonfinite(w[i].x, keep_nonfinite(w[i].y, f0));
                            f1 = keep_nonfinite(w[i].z, keep_nonfinite(w[i].w, f1));
                        }
                    }
                    const bool rows = __any_sync(0xffffffffu, has_nan(f0) || has_nan(f1));
                    if (lane == 0) by_rows[3 * x + s] = rows;
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&checked[3 * x + s]);
                    mbar_arrive(&v_empty[s]);
                }
                if (++s == L::STAGES) s = 0, ph ^= 1;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLdSoftmaxRegs));
        // ------------------------------------------------ softmax + epilogue (warps 0-7)
        const int x = warp >> 2;               // query tile of this warp group
        const int m = (warp & 3) * 32 + lane;  // query = TMEM lane
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        if (x == 0 || two) {
            const int tok = x * kLdQueries + m;  // token within the work tile
            const bool live = tok < t.n_q;
            const int pos = t.pos0 + tok;
            const int window_left = a.hdr->window_left, ntx = x == 0 ? nt0 : nt;
            const int hi = min(causal == 1 ? pos : t.length - 1, t.length - 1);
            const int lo = window_left >= 0 ? max(0, pos - window_left) : 0;
            const float sl = a.hdr->scale_log2;
            const uint32_t Sx = S_col(x) + lane_off, Ox = O_col(x) + lane_off;
            const LdMixed mixed = ld_mixed(t, x, kt0, causal, window_left);
            float m_run = -INFINITY, l_run = 0.f;
            bool ok = true;
            for (int j = 0; j < ntx; ++j) {
                const uint32_t Sj = Sx + 64u * (j & 1);
                const int key0 = (kt0 + j) * kLdKeys;
                if (!mbar_wait(&s_full[2 * x + (j & 1)], (j >> 1) & 1, err, kErrWaitFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t r0[32], r1[32];
                tmem_ld32(Sj, r0);
                tmem_ld32(Sj + 32, r1);
                tmem_wait_ld();
                float sv[kLdKeys];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    sv[c] = __uint_as_float(r0[c]);
                    sv[32 + c] = __uint_as_float(r1[c]);
                }
                if (key0 < lo || key0 + kLdKeys - 1 > hi) {
#pragma unroll
                    for (int c = 0; c < kLdKeys; ++c) {
                        const int k = key0 + c;
                        sv[c] = (k >= lo && k <= hi) ? sv[c] : -INFINITY;
                    }
                }
                float m8[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) m8[c] = fmaxf(sv[2 * c], sv[2 * c + 1]);
#pragma unroll
                for (int c = 16; c < kLdKeys; c += 16)
#pragma unroll
                    for (int q = 0; q < 8; ++q) m8[q] = max3f(m8[q], sv[c + 2 * q], sv[c + 2 * q + 1]);
                // rows past the tile's tokens hold another segment's queries: they move no maximum
                const float m_tile =
                    live ? max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])) * sl
                         : -INFINITY;
                // each row moves its maximum by its own growth alone, so that a row's bits do not
                // depend on its neighbours
                const bool grow = m_tile > m_run + kLdRescale;
                const bool warp_grow = __any_sync(0xffffffffu, grow) && j > 0;
                float alpha = 1.f;
                if (grow) {
                    alpha = ex2_ftz(m_run - m_tile);  // 0 when m_run = -inf
                    m_run = m_tile;
                }
                // p = 2^(s * sl - m), two columns per packed FMA; P goes back over S as packed bf16
                const float mref = m_run == -INFINITY ? 0.f : m_run;
                const uint64_t sl2 = f2_make(sl, sl), nm2 = f2_make(-mref, -mref);
                uint64_t acc[4] = {0, 0, 0, 0};
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float x0, x1;
                    f2_split(ffma2(f2_make(sv[2 * c], sv[2 * c + 1]), sl2, nm2), x0, x1);
                    const float p0 = ex2_ftz(x0), p1 = ex2_ftz(x1);
                    acc[c & 3] = fadd2(acc[c & 3], f2_make(p0, p1));
                    pk[c] = pack_bf16(p0, p1);
                }
                tmem_st32(Sj, pk);
                float u0, u1;
                f2_split(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), u0, u1);
                l_run = l_run * alpha + (u0 + u1);
                tmem_wait_st();
                if (warp_grow || mixed(j)) {
                    bool rows = false;
                    if (mixed(j)) {
                        const int s = j % L::STAGES;
                        // the tile first: it lands once the stage's last one has been looked over, so that
                        // the wait for the look is never two phases early
                        if (!mbar_wait(&v_full[s], (j / L::STAGES) & 1, err, kErrWaitFull) ||
                            !mbar_wait(&checked[3 * x + s], (j / L::STAGES) & 1, err, kErrWaitFull)) {
                            ok = false;
                            break;
                        }
                        rows = by_rows[3 * x + s] != 0;
                        if (rows) {
                            if (j > 0 && !mbar_wait(&pv_done[2 * x + ((j - 1) & 1)], ((j - 1) >> 1) & 1, err, kErrWaitFull)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            ld_pv_rows(Ox, Sj, sm + L::V_OFF + s * L::VC * L::CHUNK, key0, lo, hi, alpha, j == 0);
                        }
                    }
                    if (warp_grow && !rows) {
                        // O holds P_0..P_{j-1} V: wait for the last of those MMAs, then scale O's rows
                        if (!mbar_wait(&pv_done[2 * x + ((j - 1) & 1)], ((j - 1) >> 1) & 1, err, kErrWaitFull)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < kLatentV; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(Ox + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                            tmem_st32(Ox + c0, o);
                        }
                        tmem_wait_st();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * x + (j & 1)]);
            }
            if (ok && mbar_wait(&pv_done[2 * x + ((ntx - 1) & 1)], ((ntx - 1) >> 1) & 1, err, kErrWaitFull)) {
                tc_fence_after();
                const float inv = 1.f / l_run;  // every query sees a key; one whose scores are all -inf is NaN (0 / 0)
                const size_t row = (size_t)(t.q_begin + tok) * a.num_heads + t.kv_head;
                __nv_bfloat16 *orow = a.out + row * kLatentV;
#pragma unroll 1
                for (int c0 = 0; c0 < kLatentV; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(Ox + c0, o);
                    tmem_wait_ld();
                    uint32_t pkd[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        pkd[c] = pack_bf16(__uint_as_float(o[2 * c]) * inv, __uint_as_float(o[2 * c + 1]) * inv);
                    if (live) {
                        uint4 *dst = reinterpret_cast<uint4 *>(orow + c0);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            dst[c] = make_uint4(pkd[4 * c], pkd[4 * c + 1], pkd[4 * c + 2], pkd[4 * c + 3]);
                    }
                }
                if (live && a.lse) a.lse[row] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * kLdLn2;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

}  // namespace dev

cudaError_t launch_latent_dense(const LatentShape &s, const LatentPlan &p, const CUtensorMap &tm_q,
                                const CUtensorMap &tm_k, const CUtensorMap &tm_r, const CUtensorMap &tm_v, void *ws,
                                void *out, float *lse, cudaStream_t st) {
    if (p.pf_tiles == 0) return cudaSuccess;
    uint8_t *w = static_cast<uint8_t *>(ws);
    dev::LatentDenseArgs a;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.tiles = reinterpret_cast<const PrefillTile *>(w + p.dense_lay.pf_tiles);
    a.hdr = reinterpret_cast<PlanHeader *>(w + p.dense_lay.err);
    a.num_heads = s.num_heads;
    const size_t smem = 1024 + dev::LdSmem::BYTES;
    cudaError_t e = set_smem_limit((const void *)dev::latent_dense_kernel, smem, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(dev::latent_dense_kernel, dim3(p.pf_tiles), dim3(dev::kLdThreads), smem, st, tm_q, tm_k, tm_r,
                      tm_v, a);
}

}  // namespace pkv
