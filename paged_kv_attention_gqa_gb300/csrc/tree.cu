// Attention of a tree of drafted tokens over a paged cache (pkv_run_tree).
//
// Row r has C cached tokens and n drafted ones; node i's parent stands before it.  Node i sees the cached
// keys and those of its ancestors and itself (under a window, those at most window_left positions above
// its own, C + depth):
//     s_ij = sm_scale <q_i, k_j>,  p_i = softmax_j(s_i),  o_i = sum_j p_ij v_j.
// The drafted tokens' K and V come from the step's own tensors; the cache is only read.  n * g rows (g query
// heads a kv head) share a head's keys: 4 D n g operations on 4 D bytes a key.  The tensor cores and HBM
// balance near n g = 280; below it the cached K and V, read once, are the floor.
//
// Work: a unit is one query tile of up to 128 rows (row m = token * g + head), or two that share every
// K and V tile, over the 64-key tiles of its row: those of the cached keys, then those of the drafted
// ones, which so begin at a tile's first key.  A persistent CTA per SM takes an equal run of tiles, cut
// by the plan; a unit that several CTAs share leaves normalised partials, joined by a second kernel.
//  * warps 0-3 and 4-7 are two softmax groups (thread = query row = tensor-memory lane), each with two S
//    buffers of 64 columns, so that S of its next tile runs under its softmax, and an accumulator.
//    SPLIT: a unit's tiles in turn, each group with a running maximum, sum and O of its own, joined in the
//    epilogue, where a group reads half of the columns of both (one group alone takes 950 cycles a tile: more
//    than the 700 in which HBM delivers one of head_dim 64).
//    PAIR: group x has query tile x of two.
//    TURNS (head_dim 256, where tensor memory has room for one O): the pieces in turn, so that one group's
//    epilogue runs under the other's tiles.
//  * warp 8 copies Q of each piece (two buffers where they fit) and the K tiles, warp 11 the V tiles, into
//    one ring of 16 KB stages (8 at head_dim 64, 32 at 256): one lane a box of a page and 64 columns.
//  * warp 9 issues S = Q K^T, warp 10 O += P V (P from tensor memory, over its S).
//  * A key that a row does not see has weight 0, but 0 * NaN would reach O.  Those that no row sees are
//    left out by 16s or zeroed in shared memory by warp 10; a tile with keys that some rows see and others do not is
//    looked over by it, and if it holds NaN or infinities each row adds the keys it sees alone.
//  * The running maximum moves (and O is rescaled) only when it grows by more than 2^8.  Maxima and
//    sums are 32-bit; P is rounded to bf16 for the MMA (relative 2^-8 a weight at most), the sum adds it unrounded.
// Measured, one state replayed in a graph (32 or 64 query heads on 8 kv heads of 128 unless said): one row of 517 tokens, 8
// drafted: 9.5 us; 32 rows of 203 to 8,190, 16 drafted: 94 to 95 us, 557 MB, at the copy rate between start and end; 16 rows
// of 611 to 12,001, 61 drafted, 64 query heads: 149 us, 995 TFLOP/s (161 us, 920 TFLOP/s, with states that change and the
// card under its power cap); 3 chains of 5 behind 30,011 to 65,521 tokens, 20 heads on 4 of 64: 38 us; 24 rows of head_dim
// 256 under a window of 2,047: 71 us.  Of the wide case's 1,950 cycles a tile of two query tiles the MMAs take 1,280: S over 64
// keys reads both operands from shared memory, 48 cycles a k-step for 32 of arithmetic (over 128 keys: 64 for 64).  Query
// rows are padded to 128: 16 rows of 49 drafted tokens, 392 query rows a head, take 170 us, of 48, 384, 149.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "launch.h"
#include "tcgen05.cuh"
#include "tree.h"

namespace pkv {
namespace dev {

constexpr int kTrThreads = 384;
// Registers: launched with 168 a thread (384 x 168 = 64,512 of the SM's 65,536); warps 8-11 give most of their share
// to the softmax groups: 128 x 96 + 256 x 200 = 63,488.
constexpr int kTrLaunchRegs = 168, kTrSoftmaxRegs = 200, kTrOtherRegs = 96;
static_assert(128 * kTrOtherRegs + 256 * kTrSoftmaxRegs <= kTrThreads * kTrLaunchRegs, "the split fits the launch");
enum TreeForm { SPLIT, PAIR, TURNS };
constexpr float kTrRescale = 8.f;  // log2
constexpr float kTrLn2 = 0.6931471805599453f;

template <int D, TreeForm FORM>
struct TrSmem {
    static constexpr int HALVES = D / 64;
    static constexpr uint32_t Q_TILE = 128u * D * 2;  // one query tile
    // two pieces' queries (at head_dim 256 one of 128 rows or two of 64)
    static constexpr uint32_t Q_BYTES = Q_TILE * (FORM == PAIR ? 4 : FORM == TURNS ? 1 : 2);
    static constexpr uint32_t STAGE = kTreeKeys * D * 2u;
    // even: a stage holds K tiles or V tiles
    static constexpr int NS = FORM == TURNS ? 4 : FORM == PAIR ? (D == 64 ? 16 : 6) : (D == 64 ? 18 : 8);
    static_assert(NS % 2 == 0, "each stage has one producer and one reader");
    static constexpr uint32_t HALF = STAGE / HALVES;
    static constexpr uint32_t RING_OFF = Q_BYTES;
    static constexpr uint32_t BAR_OFF = RING_OFF + NS * STAGE;
    static constexpr uint32_t ML_OFF = BAR_OFF + 1024;  // [2][group][128 rows] maximum and sum (SPLIT)
    static constexpr uint32_t BYTES = ML_OFF + (FORM == SPLIT ? 2 * 2 * 128 * 8 : 0);
    static_assert(1024 + BYTES <= 227 * 1024, "the tree kernel fits shared memory");
    static_assert(1024 + BYTES > 228 * 1024 / 2, "one CTA an SM: each takes all tensor-memory columns");
};

struct TreeArgs {
    __nv_bfloat16 *out;
    float *lse;
    const TreeRow *rows;
    const TreeStart *starts;
    const TreeJoin *joins;
    const TreeNode *nodes;
    const unsigned long long *masks;
    const int32_t *pages;
    float4 *part_o;   // [slot][D / 4][part_rows], normalised: a warp's rows lie side by side
    float *part_lse;  // [slot][part_rows], base 2
    TreeHeader *hdr;
    float scale_log2;
    int batch, window_left, words, num_qo_heads, num_kv_heads, group, page_size, page_shift, num_cache_pages;
    int tile_tokens;  // query tokens of a 128-row tile
    int box_rows, box_new, box_q;
    int q_rows;       // rows of a Q buffer: 128, or 64 at head_dim 256 where two then fit
    int oob_row;      // a row past the cache: TMA fills zeros
};

// A piece: tiles [tile, tile + cnt) of a unit.
struct TreePiece {
    TreeRow row;
    int kvh, qt, tile, cnt;
    int slot;   // of its partial, -1 = the whole unit
    int index;  // of the CTA
};

template <typename F>
__device__ __forceinline__ void tree_pieces(const TreeArgs &a, const TreeStart &s, int unit_tokens, F &&piece) {
    TreePiece p;
    p.row = s.row;
    p.index = 0;
    int r = s.r, unit = s.unit, tile = s.tile;
    while (r < s.r_end || (r == s.r_end && (unit < s.unit_end || (unit == s.unit_end && tile < s.tile_end)))) {
        if (unit >= a.num_kv_heads / s.hi * p.row.nq) {
            ++r;
            unit = 0;
            if (r < a.batch) p.row = a.rows[r];
            continue;
        }
        const bool cut = r == s.r_end && unit == s.unit_end;  // the next CTA goes on with it
        p.kvh = unit / p.row.nq * s.hi + s.h0;
        p.qt = unit % p.row.nq;
        p.tile = tile;
        p.cnt = (cut ? s.tile_end : tree_unit_tiles(p.row, p.qt, unit_tokens)) - tile;
        // a unit that began in another CTA, or goes on in the next one
        p.slot = tile > 0 ? 2 * (int)blockIdx.x : cut ? 2 * (int)blockIdx.x + 1 : -1;
        if (!piece(p)) return;
        tile = 0;
        ++unit;
        ++p.index;
    }
}

// The tile of keys `t` of a row: how many there are, and which the row's nodes do not all see.
struct TreeTile {
    bool drafted;
    int key0;       // cached: position of the first key; drafted: its node
    int keys;       // 1..64 (0: a window that begins behind the cached keys)
    int first;      // keys below it are seen by no node
    int mixed0, mixed1;  // keys in [mixed0, mixed1) are seen by some and may be not by others
    bool special;   // keys to zero or to look at
};
__device__ __forceinline__ TreeTile tree_tile(const TreeRow &row, int t, int window_left) {
    TreeTile k;
    k.drafted = t >= row.nc;
    k.key0 = (k.drafted ? t - row.nc : row.kt0 + t) * kTreeKeys;
    k.keys = min(kTreeKeys, (k.drafted ? row.n : row.ctx) - k.key0);
    k.first = k.mixed0 = k.mixed1 = 0;
    if (k.drafted) {
        k.mixed1 = row.n > 1 ? k.keys : 0;
        k.special = true;
        return k;
    }
    if (window_left >= 0) {
        // a root's first key, and that of a node below n - 1 others
        const int lo = max(0, row.ctx - window_left) - k.key0, hi = max(0, row.ctx + row.n - 1 - window_left) - k.key0;
        k.first = max(0, min(lo, k.keys));
        k.mixed0 = k.first;
        k.mixed1 = max(k.first, min(hi, k.keys));
    }
    k.special = k.keys < kTreeKeys || k.first > 0 || k.mixed1 > k.mixed0;
    return k;
}

// O += P V of one tile without the tensor cores: the row of this thread adds the keys in `vis` alone.
template <int D, uint32_t HALF>  // HALF: bytes of 64 columns of the tile
__device__ __noinline__ void tree_pv_rows(uint32_t o_addr, uint32_t p_addr, const uint8_t *tile, unsigned long long vis,
                                          float alpha, bool first) {
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t r[32];
        float o[32];
        __syncwarp();
        tmem_ld32(o_addr + c0, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = first ? 0.f : __uint_as_float(r[i]) * alpha;
        const uint8_t *half = tile + (c0 >> 6) * HALF;
#pragma unroll 1
        for (int k = 0; k < kTreeKeys; ++k) {
            const uint32_t w = tmem_ld1(p_addr + (k >> 1));
            tmem_wait_ld();
            if ((vis >> k) & 1) {
                const float p = __uint_as_float((k & 1) ? w & 0xffff0000u : w << 16);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(half + swz128(k, ((c0 & 32) >> 3) + c));
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[8 * c + 2 * i] = fmaf(p, __uint_as_float(u[i] << 16), o[8 * c + 2 * i]);
                        o[8 * c + 2 * i + 1] = fmaf(p, __uint_as_float(u[i] & 0xffff0000u), o[8 * c + 2 * i + 1]);
                    }
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(o[i]);
        tmem_st32(o_addr + c0, r);
    }
    tmem_wait_st();
}

template <int D, TreeForm FORM>
__global__ void __launch_bounds__(kTrThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q,
                const __grid_constant__ TreeArgs a) {
    using L = TrSmem<D, FORM>;
    constexpr int HALVES = L::HALVES, NS = L::NS;
    constexpr int PART_ROWS = FORM == PAIR ? 256 : 128;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR_OFF);
    // Every waiter waits for the consecutive phases of a barrier, or for one that cannot be passed before the
    // waiter has provided something; so none is ever two phases behind or ahead.
    uint64_t *q_full = bars + 0;    // [2] Q buffer of a piece landed
    uint64_t *q_empty = bars + 2;   // [2] its last S completed
    uint64_t *s_full = bars + 4;    // [group][buffer]
    uint64_t *p_full = bars + 8;    // [group][buffer] P written (and O rescaled if it had to be)
    uint64_t *pv_done = bars + 12;  // [group][buffer] PV completed: the buffer may be overwritten
    uint64_t *o_final = bars + 16;  // [group] the piece's last PV completed (SPLIT: of both groups, the first)
    uint64_t *o_free = bars + 18;   // [group] the piece's O has been read (SPLIT: by both groups, the first)
    uint64_t *checked = bars + 20;  // [group] a special tile's V has been looked over
    uint64_t *joint = bars + 22;    // SPLIT: both groups' maxima and sums of a piece are in shared memory
    uint64_t *kv_full = bars + 23;           // [NS]
    uint64_t *kv_empty = bars + 23 + NS;     // [NS]
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 23 + 2 * NS);
    uint32_t *by_rows = tmem_holder + 1;     // [group] that tile's PV goes by rows

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *const err = &a.hdr->err;
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 1);
            mbar_init(&q_empty[x], 1);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&s_full[2 * x + b], 1);
                mbar_init(&p_full[2 * x + b], 4);
                mbar_init(&pv_done[2 * x + b], 1);
            }
            mbar_init(&o_final[x], 1);
            mbar_init(&o_free[x], FORM == SPLIT ? 8 : 4);
            mbar_init(&checked[x], 1);
        }
        mbar_init(joint, 8);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        fence_barrier_init();
        prefetch_tmap(&tm_kv);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        prefetch_tmap(&tm_q);
    }
    if (warp == 9) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();  // the plan, q, k, v and the cache may come from the previous kernels
    griddep_launch();
    const uint32_t tmem = *tmem_holder;
    const TreeStart start = a.starts[blockIdx.x];
    auto S_col = [tmem](int x, int b) { return tmem + 128u * (uint32_t)x + 64u * (uint32_t)b; };
    auto O_col = [tmem](int x) { return tmem + 256u + (FORM == TURNS ? 0u : (uint32_t)(D * x)); };
    const int unit_tokens = a.tile_tokens * (FORM == PAIR ? 2 : 1);
    const bool two_q = a.q_rows == 64 || D <= 128;  // Q buffers: one at head_dim 256 with 128 rows
    const uint32_t q_half = (uint32_t)a.q_rows * 128u, q_buf = q_half * HALVES;
    // PAIR: the unit's tokens reach into the second query tile
    auto second = [&](const TreePiece &p) { return FORM == PAIR && p.row.n - p.qt * unit_tokens > a.tile_tokens; };
    // whether group x has a part in tile j of a piece
    auto takes = [&](const TreePiece &p, int x, int j) {
        return FORM == SPLIT ? (j & 1) == x : FORM == TURNS ? (p.index & 1) == x : x == 0 || second(p);
    };
    auto q_slot = [&](const TreePiece &p) { return two_q ? p.index & 1 : 0; };
    auto q_phase = [&](const TreePiece &p) { return (uint32_t)(two_q ? p.index >> 1 : p.index); };
    // query tile of group x in buffer qs
    auto q_tile = [&](int qs, int x) { return (uint32_t)(FORM == PAIR ? 2 * qs + x : qs) * q_buf; };

    // each group of four warps changes its register share at the top of its own branch
    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTrOtherRegs));
    if (warp == 8 || warp == 11) {
        // ------------------------------------------------ copies: warp 8 Q and K, warp 11 V
        const int kv = warp == 11;
        const int P = a.page_size, R = a.box_rows, half = lane % HALVES, box = lane / HALVES;
        const bool mine = box < kTreeKeys / R;
        uint32_t i = kv;  // ring position: K of tile it at 2 it, V at 2 it + 1
        bool ok = true;
        tree_pieces(a, start, unit_tokens, [&](const TreePiece &p) {
            if (!kv) {
                const int qs = q_slot(p);
                const uint32_t ph = q_phase(p);
                if (ph > 0) ok = mbar_wait(&q_empty[qs], (ph - 1) & 1, err, kErrWaitEmpty);
                if (!__all_sync(0xffffffffu, ok)) return ok = false;
                const int tiles = second(p) ? 2 : 1;
                if (lane == 0) mbar_arrive_expect_tx(&q_full[qs], (uint32_t)(tiles * HALVES * a.box_q * a.group) * 128u);
                __syncwarp();
                if (lane < tiles * HALVES)
                    tma_load_3d(sm + q_tile(qs, lane / HALVES) + lane % HALVES * q_half, &tm_q, &q_full[qs],
                                lane % HALVES * 64, p.kvh * a.group,
                                p.row.q_begin + p.qt * unit_tokens + lane / HALVES * a.tile_tokens);
            }
            // the cache row of this lane's box of cached tile t
            auto box_row = [&](int t) {
                const int kb = (p.row.kt0 + t) * kTreeKeys + box * R;
                if (!mine || t >= p.row.nc || kb >= p.row.ctx) return a.oob_row;
                const int page = a.pages[p.row.kv_base + (kb >> a.page_shift)];
                if ((unsigned)page >= (unsigned)a.num_cache_pages) {
                    atomicCAS(err, 0, kErrTreePage);
                    return a.oob_row;
                }
                return page * 2 * P + (kb & (P - 1)) + kv * P;
            };
            int row = box_row(p.tile);
            for (int j = 0; j < p.cnt; ++j, i += 2) {
                const int s = i % NS, t = p.tile + j;
                const uint32_t use = i / NS;
                if (use > 0) ok = mbar_wait(&kv_empty[s], (use - 1) & 1, err, kErrWaitEmpty);
                if (!__all_sync(0xffffffffu, ok)) return ok = false;
                const bool drafted = t >= p.row.nc;
                if (lane == 0) mbar_arrive_expect_tx(&kv_full[s], drafted ? (uint32_t)(a.box_new * D * 2) : L::STAGE);
                __syncwarp();
                uint8_t *dst = sm + L::RING_OFF + s * L::STAGE + half * L::HALF;
                if (drafted) {
                    if (box == 0)
                        tma_load_3d(dst, kv ? &tm_v : &tm_k, &kv_full[s], half * 64, p.row.q_begin + (t - p.row.nc) * kTreeKeys,
                                    p.kvh);
                } else if (mine) {
                    tma_load_3d(dst + box * R * 128, &tm_kv, &kv_full[s], half * 64, row, p.kvh);
                }
                if (j + 1 < p.cnt) row = box_row(t + 1);  // lands while the next stage is awaited
            }
            return true;
        });
        // copies in flight land before the CTA may end (they have, unless a wait gave up)
        if (!ok) {
            for (uint32_t b = 0; b < 2 && !kv; ++b) mbar_wait(&q_full[b], 0, nullptr, 0, 1u << 12);
            const uint32_t end = (i - kv) / 2;
            for (uint32_t d = end > NS ? end - NS : 0; d < end; ++d) {
                const uint32_t k = 2 * d + kv;
                mbar_wait(&kv_full[k % NS], (k / NS) & 1, nullptr, 0, 1u << 12);
            }
            for (uint32_t d = 0; d < 1024; ++d) __nanosleep(1000);
        }
    } else if (warp == 9) {
        // ------------------------------------------------ S = Q K^T
        constexpr uint32_t ID_S = idesc_bf16_f32(128, kTreeKeys, 0, 0);
        auto add = [](uint64_t d, uint32_t off) { return d + (off >> 4); };
        const uint64_t dQ = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B);
        const uint64_t dK = smem_desc(smem_u32(sm + L::RING_OFF), 16, 1024, kSwizzle128B);
        uint32_t i = 0, done[2] = {0, 0};  // tiles of each group
        bool ok = true;
        tree_pieces(a, start, unit_tokens, [&](const TreePiece &p) {
            const int qs = q_slot(p);
            ok = mbar_wait(&q_full[qs], q_phase(p) & 1, err, kErrWaitFull);
            for (int j = 0; j < p.cnt && ok; ++j, i += 2) {
                const int s = i % NS;
                ok = mbar_wait(&kv_full[s], (i / NS) & 1, err, kErrWaitFull);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!takes(p, x, j) || !ok) continue;
                    const uint32_t it = done[x], b = it & 1;
                    // S overwrites P of two tiles before, which that tile's PV reads
                    if (it >= 2) ok = mbar_wait(&pv_done[2 * x + b], ((it >> 1) - 1) & 1, err, kErrWaitFull);
                    if (!ok) continue;
                    tc_fence_after();
                    const uint64_t q = add(dQ, q_tile(qs, x)), k = add(dK, s * L::STAGE);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss_elect(S_col(x, b), add(q, (kk / 4) * q_half + (kk % 4) * 32),
                                     add(k, (kk / 4) * L::HALF + (kk % 4) * 32), ID_S, kk > 0 ? 1u : 0u);
                    mma_commit_elect(&s_full[2 * x + b]);
                    ++done[x];
                }
                if (ok) mma_commit_elect(&kv_empty[s]);
            }
            if (ok) mma_commit_elect(&q_empty[qs]);
            return ok;
        });
        if (!ok)  // a wait gave up: let the MMAs in flight finish before the tensor memory is released
            for (uint32_t d = 0; d < 1024; ++d) __nanosleep(1000);
    } else {
        // ------------------------------------------------ warp 10: O += P V
        constexpr uint32_t ID_O = idesc_bf16_f32(128, D, 0, 1);
        auto add = [](uint64_t d, uint32_t off) { return d + (off >> 4); };
        const uint64_t dV = smem_desc(smem_u32(sm + L::RING_OFF), L::HALF, 1024, kSwizzle128B);
        uint32_t i = 1, done[2] = {0, 0}, pieces[2] = {0, 0};
        bool ok = true;
        tree_pieces(a, start, unit_tokens, [&](const TreePiece &p) {
            // O may be overwritten once what it held has been read
            if (FORM == SPLIT) {
                if (p.index > 0) ok = mbar_wait(&o_free[0], (p.index - 1) & 1, err, kErrWaitEmpty);
            } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!takes(p, x, 0) || !ok) continue;
                    const int y = FORM == TURNS ? 1 - x : x;
                    if (pieces[y] > 0) ok = mbar_wait(&o_free[y], (pieces[y] - 1) & 1, err, kErrWaitEmpty);
                }
            }
            for (int j = 0; j < p.cnt && ok; ++j, i += 2) {
                const int s = i % NS;
                const TreeTile k = tree_tile(p.row, p.tile + j, a.window_left);
                ok = mbar_wait(&kv_full[s], (i / NS) & 1, err, kErrWaitFull);
                if (!ok) break;
                uint8_t *const tile = sm + L::RING_OFF + s * L::STAGE;
                // k-steps of 16 keys, without those that no row sees (one at least: it may be the one that begins O)
                const int steps = (k.keys + 15) / 16, step0 = min(k.first / 16, steps - 1);
                bool rows = false;
                if (k.special) {
                    // the other keys that no row sees: their P is 0, but 0 * NaN would reach O
                    const int before = k.first - step0 * 16, n_zero = before + steps * 16 - k.keys;
                    for (int e = lane; e < n_zero * (D / 8); e += 32) {
                        const int n = e / (D / 8), c = e % (D / 8), key = n < before ? step0 * 16 + n : k.keys + n - before;
                        *reinterpret_cast<uint4 *>(tile + (c >> 3) * L::HALF + swz128(key, c & 7)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    // Keys from a multiple of eight on (those before were zeroed): a lane has every eighth of them and every fourth
                    // 16-byte chunk, so that its addresses differ by constants (one row of 119 drafted tokens of head_dim 256 14.4
                    // -> 13.4 us, the mean of 48 steps 14.7 -> 14.5; looked over by the tile's softmax group 12.5, but
                    // that slowed the loop of ordinary tiles by 3 % at head_dim 64; eight sums for two: 14.9)
                    uint32_t f0 = 0, f1 = 0;
                    const uint8_t *const even = tile + swz128(lane >> 2, lane & 3), *const odd = tile + swz128(lane >> 2, 4 + (lane & 3));
#pragma unroll (4 / HALVES)
                    for (int key = k.mixed0 & ~7; key < k.mixed1; key += 8) {
#pragma unroll
                        for (int h = 0; h < HALVES; ++h) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(even + key * 128 + h * L::HALF);
                            const uint4 w = *reinterpret_cast<const uint4 *>(odd + key * 128 + h * L::HALF);
                            f0 = keep_nonfinite(v.x, keep_nonfinite(v.y, keep_nonfinite(v.z, keep_nonfinite(v.w, f0))));
                            f1 = keep_nonfinite(w.x, keep_nonfinite(w.y, keep_nonfinite(w.z, keep_nonfinite(w.w, f1))));
                        }
                    }
                    rows = __any_sync(0xffffffffu, has_nan(f0) || has_nan(f1));
                    if (lane == 0)
                        for (int x = 0; x < 2; ++x) {
                            if (!takes(p, x, j)) continue;
                            by_rows[x] = rows;
                            mbar_arrive(&checked[x]);
                        }
                    __syncwarp();
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!takes(p, x, j) || !ok) continue;
                    const uint32_t it = done[x], b = it & 1;
                    ok = mbar_wait(&p_full[2 * x + b], (it >> 1) & 1, err, kErrWaitFull);
                    if (!ok) continue;
                    tc_fence_after();
                    if (!rows) {
                        const uint64_t v = add(dV, s * L::STAGE);
                        const uint32_t more = j >= (FORM == SPLIT ? 2 : 1) ? 1u : 0u;  // not the group's first tile
                        if (steps == kTreeKeys / 16 && step0 == 0) {
#pragma unroll
                            for (int kk = 0; kk < kTreeKeys / 16; ++kk)
                                mma_ts_elect(O_col(x), S_col(x, b) + kk * 8, add(v, kk * 2048), ID_O, kk > 0 ? 1u : more);
                        } else {
                            for (int kk = step0; kk < steps; ++kk)
                                mma_ts_elect(O_col(x), S_col(x, b) + kk * 8, add(v, kk * 2048), ID_O, kk > step0 ? 1u : more);
                        }
                    }
                    mma_commit_elect(&pv_done[2 * x + b]);
                    if (j == p.cnt - 1) {
                        mma_commit_elect(&o_final[FORM == SPLIT ? 0 : x]);
                        ++pieces[x];
                    }
                    ++done[x];
                }
                if (ok) mma_commit_elect(&kv_empty[s]);
            }
            return ok;
        });
        if (!ok)
            for (uint32_t d = 0; d < 1024; ++d) __nanosleep(1000);
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTrSoftmaxRegs));
        // ------------------------------------------------ softmax and epilogue: warps 0-7
        const int x = warp >> 2, m = (warp & 3) * 32 + lane;  // group; query row = lane of tensor memory
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const float sl = a.scale_log2;
        const uint32_t O = O_col(x) + lane_off;
        const int tok_in_tile = m / a.group, head = m % a.group;
        uint32_t it = 0, pieces = 0, checks = 0, before = 0;  // before: tiles of the CTA's earlier pieces, both groups'
        bool ok = true;
        tree_pieces(a, start, unit_tokens, [&](const TreePiece &p) {
            const uint32_t tiles0 = before;
            before += p.cnt;
            if (FORM != SPLIT && !takes(p, x, 0)) return true;
            const int tok = p.qt * unit_tokens + (FORM == PAIR ? x * a.tile_tokens : 0) + tok_in_tile;
            const bool live = tok_in_tile < a.tile_tokens && tok < p.row.n;
            const bool idle = !__any_sync(0xffffffffu, live);  // the warp has no row of this unit
            const size_t node = (size_t)p.row.q_begin + tok;
            int lo = 0;  // first cached key that the row sees
            if (live && a.window_left >= 0) lo = max(0, p.row.ctx + a.nodes[node].depth - a.window_left);
            float m_run = -INFINITY, l_run = 0.f;
            bool seen = false;
            // Tiles [ordinary0, ordinary1) are whole, cached and seen by every row.  In pairs, which the softmax bounds, they go
            // through a body without anything of the others (1,000 rows a head of 64 82.2 -> 77.2 us, 16 rows of 352
            // 23.9 -> 22.7, wide trees 151 -> 150); the other forms lost by it (27 rows of 43 drafted tokens at head_dim 256
            // 16.5 -> 17.3, 62 rows of 16 at 64 22.6 -> 23.0).
            const int last = p.row.ctx + p.row.n - 1 - a.window_left;  // all rows see the cached keys from here on
            const int ordinary0 = a.window_left >= 0 && last > 0 ? (last + kTreeKeys - 1) / kTreeKeys - p.row.kt0 : 0;
            const int ordinary1 = p.row.ctx / kTreeKeys - p.row.kt0;
            auto tile = [&](auto ordinary, int j) {
                constexpr bool ORDINARY = decltype(ordinary)::value;
                const bool first = j < (FORM == SPLIT ? 2 : 1);  // the group's first tile of the piece
                const uint32_t b = it & 1, S = S_col(x, b) + lane_off;
                TreeTile k = {};
                unsigned long long vis = ~0ull;
                if constexpr (!ORDINARY) {
                    k = tree_tile(p.row, p.tile + j, a.window_left);
                    if (k.drafted) {
                        if (live) vis = a.masks[node * a.words + (k.key0 >> 6)];
                    } else if (k.special) {
                        const int begin = min(max(lo - k.key0, 0), 64);
                        vis = begin < 64 ? ~0ull << begin : 0ull;
                        if (k.keys < 64) vis &= (1ull << max(k.keys, 0)) - 1;
                    }
                }
                if (!mbar_wait(&s_full[2 * x + b], (it >> 1) & 1, err, kErrWaitFull)) return false;
                if (idle) {  // P's rows of this warp stay as they are: O's are never read
                    if (!ORDINARY && k.special && !mbar_wait(&checked[x], checks++ & 1, err, kErrWaitFull)) return false;
                    if (lane == 0) mbar_arrive(&p_full[2 * x + b]);
                    return true;
                }
                tc_fence_after();
                uint32_t r0[32], r1[32];
                tmem_ld32(S, r0);
                tmem_ld32(S + 32, r1);
                tmem_wait_ld();
                float sv[kTreeKeys];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    sv[c] = __uint_as_float(r0[c]);
                    sv[32 + c] = __uint_as_float(r1[c]);
                }
                if (!ORDINARY && k.special) {
                    const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        sv[c] = (v0 >> c) & 1u ? sv[c] : -INFINITY;
                        sv[32 + c] = (v1 >> c) & 1u ? sv[32 + c] : -INFINITY;
                    }
                }
                seen |= vis != 0;
                float mx;
                {
                    float a0 = sv[0], a1 = sv[1], a2 = sv[2], a3 = sv[3];
#pragma unroll
                    for (int c = 4; c < 60; c += 8) {
                        a0 = max3f(a0, sv[c], sv[c + 1]);
                        a1 = max3f(a1, sv[c + 2], sv[c + 3]);
                        a2 = max3f(a2, sv[c + 4], sv[c + 5]);
                        a3 = max3f(a3, sv[c + 6], sv[c + 7]);
                    }
                    a0 = max3f(a0, sv[60], sv[61]);
                    a1 = max3f(a1, sv[62], sv[63]);
                    mx = max3f(fmaxf(a0, a1), a2, a3);
                }
                const float m_tile = live ? mx * sl : -INFINITY;
                const bool grow = m_tile > m_run + kTrRescale;
                const bool warp_grow = __any_sync(0xffffffffu, grow);
                float alpha = 1.f;
                if (grow) {
                    alpha = ex2_ftz(m_run - m_tile);  // 0 when m_run = -inf
                    m_run = m_tile;
                }
                const float mref = m_run == -INFINITY ? 0.f : m_run;
                // p = 2^(s * sl - mref), two columns per packed FMA; sums in four packed chains
                const uint64_t sl2 = f2_make(sl, sl), nm2 = f2_make(-mref, -mref);
                uint64_t acc[4] = {0, 0, 0, 0};
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float y0, y1;
                    f2_split(ffma2(f2_make(sv[2 * c], sv[2 * c + 1]), sl2, nm2), y0, y1);
                    const float p0 = ex2_ftz(y0), p1 = ex2_ftz(y1);
                    acc[c & 3] = fadd2(acc[c & 3], f2_make(p0, p1));
                    pk[c] = pack_bf16(p0, p1);
                }
                float u0, u1;
                f2_split(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), u0, u1);
                l_run = l_run * alpha + (u0 + u1);
                tmem_st32(S, pk);
                tmem_wait_st();
                bool rows = false;
                if (!ORDINARY && k.special) {
                    if (!mbar_wait(&checked[x], checks++ & 1, err, kErrWaitFull)) return false;
                    rows = by_rows[x] != 0;
                }
                if (rows || (warp_grow && !first)) {
                    // O holds the group's earlier tiles: wait for the last of those MMAs
                    if (!first && !mbar_wait(&pv_done[2 * x + (1 - b)], ((it - 1) >> 1) & 1, err, kErrWaitFull)) return false;
                    tc_fence_after();
                    if (rows) {
                        const uint32_t at = 2 * (tiles0 + j) + 1, s = at % NS;  // V's stage (it has landed: `checked`)
                        if (!mbar_wait(&kv_full[s], (at / NS) & 1, err, kErrWaitFull)) return false;
                        tree_pv_rows<D, L::HALF>(O, S, sm + L::RING_OFF + s * L::STAGE, vis, alpha, first);
                    } else {
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(O + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                            tmem_st32(O + c0, o);
                        }
                        tmem_wait_st();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * x + b]);
                return true;
            };
            for (int j = FORM == SPLIT ? x : 0; j < p.cnt; j += FORM == SPLIT ? 2 : 1, ++it) {
                const int t = p.tile + j;
                const bool ordinary = FORM == PAIR && t >= ordinary0 && t < ordinary1;
                if (!(ordinary ? tile(std::bool_constant<FORM == PAIR>(), j) : tile(std::false_type(), j))) return ok = false;
            }
            // the piece's O = w0 O of group 0 + w1 O of group 1 (SPLIT), or this group's alone, normalised.
            // A piece may hold no key that a row sees: weight 0, lse -inf.  Keys whose scores are all -inf weigh
            // nothing against other pieces, but 0 * inf of their values stays; a row that has no others is NaN (0 / 0).
            float w0 = 1.f, w1 = 0.f;
            bool seen0 = seen, seen1 = false;
            if constexpr (FORM == SPLIT) {
                float2 *const ml = reinterpret_cast<float2 *>(sm + L::ML_OFF) + (pieces & 1) * 256;
                ml[x * 128 + m] = make_float2(m_run, seen ? l_run : -1.f);
                __syncwarp();
                if (lane == 0) mbar_arrive(joint);
                if (!mbar_wait(joint, pieces & 1, err, kErrWaitFull)) return ok = false;
                const float2 e0 = ml[m], e1 = ml[128 + m];
                seen0 = !(e0.y < 0.f);
                seen1 = !(e1.y < 0.f);
                m_run = fmaxf(e0.x, e1.x);
                const float ref = m_run == -INFINITY ? 0.f : m_run;
                w0 = !seen0 ? 0.f : m_run == -INFINITY ? 1.f : ex2_ftz(e0.x - ref);
                w1 = !seen1 ? 0.f : m_run == -INFINITY ? 1.f : ex2_ftz(e1.x - ref);
                l_run = (seen0 ? w0 * e0.y : 0.f) + (seen1 ? w1 * e1.y : 0.f);
                seen = seen0 || seen1;
            }
            if (!mbar_wait(&o_final[FORM == SPLIT ? 0 : x], pieces & 1, err, kErrWaitFull)) return ok = false;
            ++pieces;
            tc_fence_after();
            if (!idle) {
                const float inv = !seen ? 0.f : l_run == 0.f && p.slot >= 0 ? 1.f : 1.f / l_run;
                const float lse2 = l_run == 0.f ? -INFINITY : m_run + log2f(l_run);
                const size_t orow = node * a.num_qo_heads + p.kvh * a.group + head;
                const int prow = (FORM == PAIR ? x * 128 : 0) + m;
                w0 *= inv;
                w1 *= inv;
                const uint32_t O0 = O_col(FORM == SPLIT ? 0 : x) + lane_off, O1 = O_col(1) + lane_off;
                const int c_begin = FORM == SPLIT ? x * (D / 2) : 0, c_end = FORM == SPLIT ? c_begin + D / 2 : D;
#pragma unroll 1
                for (int c0 = c_begin; c0 < c_end; c0 += 32) {
                    uint32_t o[32], o1[32];
                    __syncwarp();
                    tmem_ld32(O0 + c0, o);
                    if (FORM == SPLIT) tmem_ld32(O1 + c0, o1);
                    tmem_wait_ld();
                    float f[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {  // select, not multiply: O may hold anything if the row saw no key
                        f[c] = seen0 ? __uint_as_float(o[c]) * w0 : 0.f;
                        if (FORM == SPLIT) f[c] = seen1 ? fmaf(__uint_as_float(o1[c]), w1, f[c]) : f[c];
                    }
                    if (!live) continue;
                    if (p.slot < 0) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + orow * D + c0);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            dst[c] = make_uint4(pack_bf16(f[8 * c], f[8 * c + 1]), pack_bf16(f[8 * c + 2], f[8 * c + 3]),
                                                pack_bf16(f[8 * c + 4], f[8 * c + 5]), pack_bf16(f[8 * c + 6], f[8 * c + 7]));
                    } else {
                        float4 *dst = a.part_o + ((size_t)p.slot * (D / 4) + c0 / 4) * PART_ROWS + prow;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            dst[c * PART_ROWS] = make_float4(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3]);
                    }
                }
                if (live && (FORM != SPLIT || x == 0)) {
                    if (p.slot >= 0)
                        a.part_lse[(size_t)p.slot * PART_ROWS + prow] = lse2;
                    else if (a.lse)
                        a.lse[orow] = lse2 * kTrLn2;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[FORM == SPLIT ? 0 : x]);
            return true;
        });
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

// Join of a unit's pieces: with w_i = 2^(lse_i - max lse), o = sum w_i o_i / sum w_i.  A block takes up to 32 rows of a
// cut unit and the columns that its record says; a thread has a row and four vectors of four columns, warps (and
// parts of a warp, where the unit has few rows) beside that take the pieces in turn.  Bounded by trips to L2
// (the plan's record, the partials), so all pieces are on their way at once as far as they fit.  Records of the cut
// units alone, with as many blocks as their pieces ask for, against a column of blocks for every CTA and one rule for all
// units: 4 rows of one drafted token at head_dim 256 16.4 -> 12.0 us, 16 rows of 352 query rows a head 28.9 -> 23.8,
// the mean of 48 steps 15.2 -> 14.7 (a third of that by kTreeLeastWhole).
// Joining in the CTA that finishes last took longer (wide trees 167 -> 185 us, long chains 42 -> 45): its few warps
// make those trips one after another.
struct JoinSum {
    float top, sum;
    float4 acc[4];
};
__device__ __forceinline__ float4 scaled(const float4 &x, float w) { return make_float4(x.x * w, x.y * w, x.z * w, x.w * w); }
__device__ __forceinline__ float4 fma4(float w, const float4 &x, const float4 &y) {
    return make_float4(fmaf(w, x.x, y.x), fmaf(w, x.y, y.y), fmaf(w, x.z, y.z), fmaf(w, x.w, y.w));
}
// j: the sums to the maximum `top`
__device__ __forceinline__ void raise_top(JoinSum &j, float top) {
    const float w = j.top == -INFINITY ? 0.f : exp2f(j.top - top);
    j.top = top;
    j.sum *= w;
#pragma unroll
    for (int c = 0; c < 4; ++c) j.acc[c] = scaled(j.acc[c], w);
}
template <int D, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) tree_join_kernel(const TreeArgs a, int part_rows) {
    constexpr int COLS = 4, C = D / 4;
    __shared__ float4 others[WARPS * COLS * 32];
    __shared__ float2 sums[WARPS * 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // The plan was complete before the attention kernel let this one start.  But nothing has been waited for here, so the
    // record is read past L1, which may still hold an earlier step's
    union {
        int4 part[2];
        TreeJoin u;
    } record;
    for (int i = 0; i < 2; ++i) record.part[i] = __ldcg(reinterpret_cast<const int4 *>(a.joins + blockIdx.x) + i);
    const TreeJoin u = record.u;
    const int rows = u.tokens * a.group, tile_rows = a.tile_tokens * a.group;
    const int R = u.rows, place0 = blockIdx.y * tree_join_rows(rows) + u.row0, place = place0 + (lane & (R - 1));
    // rows of the unit (token * group + head) at these places of its one or two tiles
    const int f = (place >> 7) * tile_rows + (place & 127), f0 = (place0 >> 7) * tile_rows + (place0 & 127);
    if (u.count == 0 || (place0 & 127) >= tile_rows || f0 >= rows) {
        griddep_wait();
        griddep_launch();
        return;
    }
    const bool live = (place & 127) < tile_rows && f < rows;
    const int set = warp >> u.groups, sets = WARPS >> u.groups, side = 32 / R, stride = sets * side;
    const int c0 = (u.group0 + (warp & ((1 << u.groups) - 1))) * COLS;
    const size_t out_row = ((size_t)u.token + f / a.group) * a.num_qo_heads + u.kvh * a.group + f % a.group;
    griddep_wait();
    griddep_launch();
    JoinSum j = {-INFINITY, 0.f, {}};
    for (int i0 = set * side + lane / R; live && i0 < u.count; i0 += kJoinBatch * stride) {
        float l[kJoinBatch];
        float4 v[kJoinBatch][COLS];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            const int at = i0 + i * stride;
            l[i] = -INFINITY;
            if (at >= u.count) continue;
            const size_t slot = at == 0 ? 2 * u.cta + 1 : 2 * (u.cta + at * u.step);
            l[i] = __ldcg(a.part_lse + slot * part_rows + place);
#pragma unroll
            for (int c = 0; c < COLS; ++c) v[i][c] = __ldcg(a.part_o + (slot * C + c0 + c) * part_rows + place);
        }
        float top = j.top;
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) top = fmaxf(top, l[i]);
        raise_top(j, top);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            if (i0 + i * stride >= u.count) continue;
            const float w = exp2f(l[i] - ref);
            j.sum += w;
#pragma unroll
            for (int c = 0; c < COLS; ++c) j.acc[c] = fma4(w, v[i][c], j.acc[c]);
        }
    }
    // parts of a warp with the same rows
    for (int o = R; o < 32; o <<= 1) {
        const float top = fmaxf(j.top, __shfl_xor_sync(0xffffffffu, j.top, o));
        raise_top(j, top);
        j.sum += __shfl_xor_sync(0xffffffffu, j.sum, o);
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            j.acc[c].x += __shfl_xor_sync(0xffffffffu, j.acc[c].x, o);
            j.acc[c].y += __shfl_xor_sync(0xffffffffu, j.acc[c].y, o);
            j.acc[c].z += __shfl_xor_sync(0xffffffffu, j.acc[c].z, o);
            j.acc[c].w += __shfl_xor_sync(0xffffffffu, j.acc[c].w, o);
        }
    }
    if (sets > 1) {
        if (set > 0) {
            sums[threadIdx.x] = make_float2(j.top, j.sum);
#pragma unroll
            for (int c = 0; c < COLS; ++c) others[(warp * COLS + c) * 32 + lane] = j.acc[c];
        }
        __syncthreads();
        if (set > 0) return;
        float top = j.top;
        for (int i = 1; i < sets; ++i) top = fmaxf(top, sums[(i << u.groups) * 32 + threadIdx.x].x);
        raise_top(j, top);
        const float ref = top == -INFINITY ? 0.f : top;
        for (int i = 1; i < sets; ++i) {
            const int from = (i << u.groups) + warp;
            const float2 e = sums[from * 32 + lane];
            const float w = exp2f(e.x - ref);
            j.sum = fmaf(w, e.y, j.sum);
#pragma unroll
            for (int c = 0; c < COLS; ++c) j.acc[c] = fma4(w, others[(from * COLS + c) * 32 + lane], j.acc[c]);
        }
    }
    if (!live || lane >= R) return;
    const float inv = 1.f / j.sum;  // (0 / 0 if every key of the row scores -inf)
    uint4 *dst = reinterpret_cast<uint4 *>(a.out + out_row * D + 4 * c0);
#pragma unroll
    for (int c = 0; c < COLS; c += 2) {
        const float4 x = scaled(j.acc[c], inv), y = scaled(j.acc[c + 1], inv);
        dst[c / 2] = make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
    }
    if (a.lse && c0 == 0) a.lse[out_row] = (j.sum == 0.f ? -INFINITY : j.top + log2f(j.sum)) * kTrLn2;
}

template <int D, TreeForm FORM>
static cudaError_t raise_limit(cudaStream_t st) {
    return set_smem_limit((const void *)tree_kernel<D, FORM>, 1024 + TrSmem<D, FORM>::BYTES, st);
}

template <int D, TreeForm FORM>
static cudaError_t launch(const TreeArgs &a, const TreePlan &p, int ctas, const CUtensorMap &tm_kv, const CUtensorMap &tm_k,
                          const CUtensorMap &tm_v, const CUtensorMap &tm_q, cudaStream_t st) {
    const size_t smem = 1024 + TrSmem<D, FORM>::BYTES;
    cudaError_t e = raise_limit<D, FORM>(st);
    if (e == cudaSuccess) e = launch_pdl(tree_kernel<D, FORM>, dim3(ctas), dim3(kTrThreads), smem, st, tm_kv, tm_k, tm_v, tm_q, a);
    if (e != cudaSuccess || ctas == 1 || p.whole) return e;
    constexpr int WARPS = D == 64 ? 4 : 8;
    const dim3 grid(p.join_blocks, p.join_rows), block(32 * p.join_warps);
    return launch_pdl(p.join_warps == WARPS ? tree_join_kernel<D, WARPS> : tree_join_kernel<D, 2 * WARPS>, grid, block, 0, st, a,
                      p.part_rows);
}

}  // namespace dev

cudaError_t prepare_tree(const Shape &s, cudaStream_t st) {
    if (s.head_dim == 256) return dev::raise_limit<256, dev::TURNS>(st);
    const cudaError_t e = s.head_dim == 64 ? dev::raise_limit<64, dev::SPLIT>(st) : dev::raise_limit<128, dev::SPLIT>(st);
    if (e != cudaSuccess) return e;
    return s.head_dim == 64 ? dev::raise_limit<64, dev::PAIR>(st) : dev::raise_limit<128, dev::PAIR>(st);
}

cudaError_t launch_tree(const Shape &s, const TreePlan &p, const CUtensorMap &tm_kv, const CUtensorMap &tm_k,
                        const CUtensorMap &tm_v, const CUtensorMap &tm_q, int box_new, int box_q, void *ws, void *out,
                        float *lse, cudaStream_t st) {
    uint8_t *w = static_cast<uint8_t *>(ws);
    dev::TreeArgs a;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.rows = reinterpret_cast<const TreeRow *>(w + p.off_rows);
    a.starts = reinterpret_cast<const TreeStart *>(w + p.off_starts);
    a.joins = reinterpret_cast<const TreeJoin *>(w + p.off_joins);
    a.nodes = reinterpret_cast<const TreeNode *>(w + p.off_nodes);
    a.masks = reinterpret_cast<const unsigned long long *>(w + p.off_masks);
    a.pages = p.pages;
    a.part_o = reinterpret_cast<float4 *>(w + p.off_part_o);
    a.part_lse = reinterpret_cast<float *>(w + p.off_part_lse);
    a.hdr = reinterpret_cast<TreeHeader *>(w);
    a.scale_log2 = p.scale_log2;
    a.batch = p.batch;
    a.window_left = p.window_left;
    a.words = p.words;
    a.num_qo_heads = s.num_qo_heads;
    a.num_kv_heads = s.num_kv_heads;
    a.group = s.group();
    a.page_size = s.page_size;
    a.page_shift = s.page_shift();
    a.num_cache_pages = s.num_cache_pages;
    a.tile_tokens = tree_tile_tokens(s);
    a.box_rows = s.page_size < kTreeKeys ? s.page_size : kTreeKeys;
    a.box_new = box_new;
    a.box_q = box_q;
    a.q_rows = s.head_dim == 256 && box_q * a.group <= 64 ? 64 : 128;
    a.oob_row = s.num_cache_pages * 2 * s.page_size;
    if (s.head_dim == 64)
        return p.pair ? dev::launch<64, dev::PAIR>(a, p, s.sm_count, tm_kv, tm_k, tm_v, tm_q, st)
                      : dev::launch<64, dev::SPLIT>(a, p, s.sm_count, tm_kv, tm_k, tm_v, tm_q, st);
    if (s.head_dim == 128)
        return p.pair ? dev::launch<128, dev::PAIR>(a, p, s.sm_count, tm_kv, tm_k, tm_v, tm_q, st)
                      : dev::launch<128, dev::SPLIT>(a, p, s.sm_count, tm_kv, tm_k, tm_v, tm_q, st);
    return dev::launch<256, dev::TURNS>(a, p, s.sm_count, tm_kv, tm_k, tm_v, tm_q, st);
}

}  // namespace pkv
