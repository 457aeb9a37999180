// Latent attention, expanded form (pkv_latent_run_dense): prompts over contiguous per-head keys
// [k_nope | k_rope] (128 + 64 columns, the rope part shared by all heads) and values (128), made from
// the latent vectors by the caller.  s_ij = sm_scale * (<qn_i, kn_j> + <qr_i, kr_j>); softmax over the
// keys a query sees; o_i = sum_j p_ij v_j.
//
// Bounded by the tensor cores: 640 operations per query, key and head, on operands that fit L2.  A
// work tile is two query tiles of 128 tokens of one head that share every 128-key tile, one CTA per
// SM, in the division of the two-query-tile prefill kernel:
//  * warp 16 copies Q0 and Q1 once, then streams the K/V tiles as 64-column chunks of 128 keys (16 KB:
//    two of k_nope, one of k_rope, two of v) through one ring of eight; a chunk is refilled as soon as
//    the MMAs of both query tiles that read it are done;
//  * warps 17 and 18 issue the MMAs of Q0 and Q1: S = Q K^T (12 k-steps, N = 128), then O += P V (P from
//    tensor memory; N = 64 per chunk, which runs at the full rate: measured 32 cycles a k-step), with
//    S0, S1, O0, O1 in 128 tensor-memory columns each;
//  * warps 0-7 and 8-15 run the softmax of Q0 and Q1 by turns, so that each runs under the other tile's
//    MMAs.  A query's 128 scores are shared by two threads, two warps per SM sub-partition, which halves
//    the phases of a turn that leave the exponential unit idle (one thread a query: 305 us on four
//    prompts of 801 to 4,093 tokens and 32 heads).  The two agree on the maximum through shared memory
//    only when it has to move: it moves, and O is rescaled, when it grows by more than 2^8.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "latent.h"
#include "launch.h"
#include "tcgen05.cuh"

namespace pkv {
namespace dev {

constexpr int kLdKeys = 128, kLdQueries = 128;
constexpr int kLdThreads = 640;
// Registers: 640 x 96 at launch = 61,440; the softmax groups take most of warp group 4's share
// (128 x 56 + 512 x 104 = 60,416).
constexpr int kLdLaunchRegs = 96, kLdSoftmaxRegs = 104, kLdOtherRegs = 56;
static_assert(128 * kLdOtherRegs + 512 * kLdSoftmaxRegs <= kLdThreads * kLdLaunchRegs, "setmaxnreg split fits the launch");
constexpr float kLdRescale = 8.f;  // log2
constexpr float kLdLn2 = 0.6931471805599453f;

struct LdSmem {
    static constexpr uint32_t CHUNK = 128 * 128;  // 128 rows x 64 columns
    static constexpr int QC = 3, KC = 3, VC = 2, SLOTS = 8;
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t RING_OFF = 2 * QC * CHUNK;
    static constexpr uint32_t BAR_OFF = RING_OFF + SLOTS * CHUNK;
    static constexpr uint32_t EXCH_OFF = BAR_OFF + 256;  // per query tile and query: a maximum
    static constexpr uint32_t BYTES = EXCH_OFF + 2 * 128 * 4;
};
static_assert(1024 + LdSmem::BYTES <= 227 * 1024, "the expanded latent kernel fits shared memory");

struct LatentDenseArgs {
    __nv_bfloat16 *out;
    float *lse;
    const PrefillTile *tiles;
    PlanHeader *hdr;
    int num_heads;
};

__global__ void __launch_bounds__(kLdThreads, 1)
    latent_dense_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v,
                        const LatentDenseArgs a) {
    using L = LdSmem;
    constexpr int PER = L::KC + L::VC;  // ring chunks of one K/V tile
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR_OFF);
    uint64_t *q_full = bars + 0;     // [2] Q_X landed
    uint64_t *kv_full = bars + 2;    // [8] ring slot landed
    uint64_t *kv_empty = bars + 10;  // [8] the MMAs that read the slot completed (one commit per query tile)
    uint64_t *s_full = bars + 18;    // [2] S_X(j) in tensor memory
    uint64_t *p_full = bars + 20;    // [2] P_X(j) written (and O_X rescaled if it had to be)
    uint64_t *pv_done = bars + 22;   // [2] PV_X(j) completed
    uint64_t *v_tail = bars + 24;    // warp 17 zeroed the value rows past the segment (at most once)
    uint64_t *turn = bars + 25;      // [2] the softmax group of Q_X may start its next tile
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 27);

    const PrefillTile t = a.tiles[blockIdx.x];
    int *const err = &a.hdr->err;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const bool two = t.n_q > kLdQueries;  // the tile's tokens reach into Q1
    const int kt0 = t.key_begin / kLdKeys;
    const int nt = (t.key_end + kLdKeys - 1) / kLdKeys - kt0;  // >= 1: every query sees itself

    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 1);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 8);
            mbar_init(&pv_done[x], 1);
            mbar_init(&turn[x], 8);
        }
        for (int s = 0; s < L::SLOTS; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], two ? 2 : 1);
        }
        mbar_init(v_tail, 1);
        fence_barrier_init();
    }
    if (warp == 17) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch();
    const uint32_t tmem = *tmem_holder;
    auto S_col = [tmem](int x) { return tmem + 128u * (uint32_t)x; };
    auto O_col = [tmem](int x) { return tmem + 256u + 128u * (uint32_t)x; };

    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLdOtherRegs));
        if (warp == 16) {
            // ------------------------------------------------ copies: one thread, one box per chunk
            if (lane == 0) {
                prefetch_tmap(&tm_q);
                prefetch_tmap(&tm_k);
                prefetch_tmap(&tm_r);
                prefetch_tmap(&tm_v);
                auto load_q = [&](int x) {
                    mbar_arrive_expect_tx(&q_full[x], L::QC * L::CHUNK);
                    for (int c = 0; c < L::QC; ++c)
                        tma_load_3d(sm + L::Q_OFF + (x * L::QC + c) * L::CHUNK, &tm_q, &q_full[x], c * 64,
                                    t.q_begin + x * kLdQueries, t.kv_head);
                };
                load_q(0);
                bool ok = true;
                uint32_t i = 0;
                for (int j = 0; j < nt && ok; ++j) {
                    const int row = t.kv_base + (kt0 + j) * kLdKeys;  // first key row of the tile
#pragma unroll
                    for (int c = 0; c < PER; ++c, ++i) {
                        const uint32_t s = i % L::SLOTS, use = i / L::SLOTS;
                        if (use > 0 && !mbar_wait(&kv_empty[s], (use - 1) & 1, err, kErrWaitEmpty)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&kv_full[s], L::CHUNK);
                        uint8_t *dst = sm + L::RING_OFF + s * L::CHUNK;
                        if (c < 2)
                            tma_load_3d(dst, &tm_k, &kv_full[s], c * 64, row, t.kv_head);
                        else if (c == 2)
                            tma_load_2d(dst, &tm_r, &kv_full[s], 0, row);
                        else
                            tma_load_3d(dst, &tm_v, &kv_full[s], (c - 3) * 64, row, t.kv_head);
                        if (j == 0 && c == 2 && two) load_q(1);  // needed after S0(0)
                    }
                }
                // copies in flight land before the CTA may end (they have, unless a wait gave up)
                for (uint32_t d = i > L::SLOTS ? i - L::SLOTS : 0; d < i; ++d)
                    mbar_wait(&kv_full[d % L::SLOTS], (d / L::SLOTS) & 1, err, kErrWaitDrain);
            }
        } else if (warp == 17 || (warp == 18 && two)) {
            // ------------------------------------------------ MMAs: warp 17 for Q0, warp 18 for Q1
            const int x = warp - 17;
            constexpr uint32_t ID_S = idesc_bf16_f32(128, kLdKeys, 0, 0);
            constexpr uint32_t ID_O = idesc_bf16_f32(128, 64, 0, 1);
            const uint64_t dQ = smem_desc(smem_u32(sm + L::Q_OFF + x * L::QC * L::CHUNK), 16, 1024, kSwizzle128B);
            const uint64_t dR = smem_desc(smem_u32(sm + L::RING_OFF), 16, 1024, kSwizzle128B);
            // one 64-column chunk is all of N: the leading offset is never stepped
            const uint64_t dV = smem_desc(smem_u32(sm + L::RING_OFF), L::CHUNK, 1024, kSwizzle128B);
            auto add = [](uint64_t d, uint32_t off) { return d + (off >> 4); };
            const uint32_t Sx = S_col(x), Ox = O_col(x);
            bool ok = mbar_wait(&q_full[x], 0, err, kErrWaitFull);
            uint32_t i = 0;  // ring chunks, as the producer counts them
            for (int j = 0; j < nt && ok; ++j) {
                // S_X(j) overwrites P_X(j-1), which PV_X(j-1) reads
                if (j > 0) ok = mbar_wait(&pv_done[x], (j - 1) & 1, err, kErrWaitFull);
#pragma unroll 1
                for (int c = 0; c < L::KC && ok; ++c, ++i) {
                    const uint32_t s = i % L::SLOTS;
                    ok = mbar_wait(&kv_full[s], (i / L::SLOTS) & 1, err, kErrWaitFull);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss_elect(Sx, add(dQ, c * L::CHUNK + kk * 32), add(dR, s * L::CHUNK + kk * 32), ID_S,
                                     (c > 0 || kk > 0) ? 1u : 0u);
                    mma_commit_elect(&kv_empty[s]);
                }
                if (!ok) break;
                mma_commit_elect(&s_full[x]);
                // Value rows past the segment's end belong to the next segment (or are zero past the
                // tensor): their P is 0, but 0 * NaN would reach O.  Warp 17 zeroes them; warp 18 waits
                // for that on the one tile that has them.
                const int key0 = (kt0 + j) * kLdKeys;
                const bool tail = key0 + kLdKeys > t.length;
                for (int c = 0; c < L::VC && ok; ++c)
                    ok = mbar_wait(&kv_full[(i + c) % L::SLOTS], ((i + c) / L::SLOTS) & 1, err, kErrWaitFull);
                if (ok && tail) {
                    if (x == 0) {
                        const int zb = t.length - key0;  // >= 1: the tile holds a visible key
                        for (int e = lane; e < (kLdKeys - zb) * 16; e += 32) {
                            const int k = zb + (e >> 4), ch = e & 15;
                            *reinterpret_cast<uint4 *>(sm + L::RING_OFF + ((i + (ch >> 3)) % L::SLOTS) * L::CHUNK +
                                                       swz128(k, ch & 7)) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && two) mbar_arrive(v_tail);
                    } else {
                        ok = mbar_wait(v_tail, 0, err, kErrWaitFull);
                    }
                }
                if (ok) ok = mbar_wait(&p_full[x], j & 1, err, kErrWaitFull);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < L::VC; ++c, ++i) {
                    const uint32_t s = i % L::SLOTS;
#pragma unroll
                    for (int kk = 0; kk < kLdKeys / 16; ++kk)
                        mma_ts_elect(Ox + 64u * c, Sx + kk * 8, add(dV, s * L::CHUNK + kk * 2048), ID_O,
                                     (j > 0 || kk > 0) ? 1u : 0u);
                    if (c == 1) mma_commit_elect(&pv_done[x]);
                    mma_commit_elect(&kv_empty[s]);
                }
            }
            if (!ok)  // a wait gave up: let the MMAs in flight finish before the tensor memory is released
                for (uint32_t k = 0; k < 1024; ++k) __nanosleep(1000);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLdSoftmaxRegs));
        // ------------------------------------------------ softmax + epilogue (warps 0-15)
        const int x = warp >> 3;               // query tile of this warp's group
        const int hf = (warp >> 2) & 1;        // which 64 of a tile's keys, of P's columns and of O's
        const int m = (warp & 3) * 32 + lane;  // query = TMEM lane
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        if (x == 0 || two) {
            float *const exch = reinterpret_cast<float *>(sm + L::EXCH_OFF) + x * 128;
            const int tok = x * kLdQueries + m;  // token within the work tile
            const bool live = tok < t.n_q;
            const int pos = t.pos0 + tok;
            const int causal = a.hdr->causal, window_left = a.hdr->window_left;
            const int hi = min(causal == 1 ? pos : t.length - 1, t.length - 1);
            const int lo = window_left >= 0 ? max(0, pos - window_left) : 0;
            const float sl = a.hdr->scale_log2;
            const uint32_t Sx = S_col(x) + lane_off, Ox = O_col(x) + lane_off + 64u * hf;
            float m_run = -INFINITY, l_run = 0.f;  // l_run: this half's keys
            // a wait that gives up clears ok; the warps still walk their tiles, without further waits, so that
            // they keep meeting at their barriers (which have no time limit)
            bool ok = true;
            for (int j = 0; j < nt; ++j) {
                const int key0 = (kt0 + j) * kLdKeys + 64 * hf;
                // group 1 starts tile j after group 0 finished it, group 0 tile j + 1 after group 1 tile j
                if (two && (x == 1 || j > 0)) ok = ok && mbar_wait(&turn[x], (x ? j : j - 1) & 1, err, kErrWaitFull);
                ok = ok && mbar_wait(&s_full[x], j & 1, err, kErrWaitFull);
                __syncwarp();
                tc_fence_after();
                uint32_t r0[32], r1[32];
                tmem_ld32(Sx + 64u * hf, r0);
                tmem_ld32(Sx + 64u * hf + 32, r1);
                tmem_wait_ld();
                float sv[64];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    sv[c] = __uint_as_float(r0[c]);
                    sv[32 + c] = __uint_as_float(r1[c]);
                }
                if (key0 < lo || key0 + 63 > hi) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        const int k = key0 + c;
                        sv[c] = ((k >= lo) & (k <= hi)) ? sv[c] : -INFINITY;
                    }
                }
                float m4[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) m4[c] = fmaxf(sv[2 * c], sv[2 * c + 1]);
#pragma unroll
                for (int c = 8; c < 64; c += 8)
#pragma unroll
                    for (int q = 0; q < 4; ++q) m4[q] = max3f(m4[q], sv[c + 2 * q], sv[c + 2 * q + 1]);
                // rows past the tile's tokens hold another segment's queries: they move no maximum
                const float m_half = live ? max3f(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * sl : -INFINITY;
                // whether any query of the group moves its maximum.  The barrier also says that every
                // thread holds its scores: the second half's P goes over columns of the first half's S
                unsigned any;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 256, p;\n\t"
                             "selp.u32 %0, 1, 0, q;\n\t}"
                             : "=r"(any)
                             : "r"((unsigned)(m_half > m_run + kLdRescale)), "r"(1 + x)
                             : "memory");
                float alpha = 1.f;
                bool grow = false;
                if (any) {
                    // the first half's maximum to the second, the joint one back.  Each query moves its
                    // maximum by its own growth alone, so that its bits do not depend on its neighbours
                    if (hf == 0) exch[m] = m_half;
                    named_barrier_sync(1 + x, 256);
                    float m_tile = hf ? fmaxf(m_half, exch[m]) : 0.f;
                    if (hf) exch[m] = m_tile;
                    named_barrier_sync(1 + x, 256);
                    if (!hf) m_tile = exch[m];
                    grow = m_tile > m_run + kLdRescale;
                    if (grow) {
                        alpha = ex2_ftz(m_run - m_tile);  // 0 when m_run = -inf
                        m_run = m_tile;
                    }
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
                tmem_st32(Sx + 32u * hf, pk);
                float u0, u1;
                f2_split(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), u0, u1);
                l_run = l_run * alpha + (u0 + u1);
                __syncwarp();
                if (two && lane == 0) mbar_arrive(&turn[1 - x]);  // the other group's turn
                tmem_wait_st();
                if (__any_sync(0xffffffffu, grow) && j > 0) {
                    // O holds P_0..P_{j-1} V: wait for the last of those MMAs, then scale O's rows
                    ok = ok && mbar_wait(&pv_done[x], (j - 1) & 1, err, kErrWaitFull);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < 64; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld32(Ox + c0, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                        tmem_st32(Ox + c0, o);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
            }
            // the two halves' sums, through the query tile's shared memory: nothing reads Q_X any more
            ok = ok && mbar_wait(&pv_done[x], (nt - 1) & 1, err, kErrWaitFull);
            __syncwarp();
            float *const sums = reinterpret_cast<float *>(sm + L::Q_OFF + x * L::QC * L::CHUNK);
            if (ok) sums[hf * 128 + m] = l_run;
            named_barrier_sync(1 + x, 256);
            const float l = l_run + sums[(1 - hf) * 128 + m];
            if (__all_sync(0xffffffffu, ok)) {
                tc_fence_after();
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const size_t row = (size_t)(t.q_begin + tok) * a.num_heads + t.kv_head;
                __nv_bfloat16 *orow = a.out + row * kLatentV + 64 * hf;
#pragma unroll 1
                for (int c0 = 0; c0 < 64; c0 += 32) {
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
                if (hf == 0 && live && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m_run + log2f(l)) * kLdLn2;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 17) tmem_dealloc(tmem, 512);
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
