// Eviction (pkv_run_evict): which tokens of each row stay, and their move to new pages.
//
// Selection.  Of the m = keep - sink - recent best among a row's n = L - sink - recent middle tokens,
// the m-th largest score is found by radix selection on the scores as ordered 32-bit integers (11, 11
// and 10 bits from the top: up to three histograms, fewer once a bin is taken whole), then the tokens
// above it and, from the lowest position up, as many equal to it as are still wanted are written out in
// position order.  Each thread owns a run of consecutive tokens, so that one scan over the threads
// orders the output.  Every row of a plan gets the CTAs that its longest cut row needs at 8,192 tokens
// each, one or a cluster of up to eight (histograms and counts joined through distributed shared memory); the scores are read once,
// through the page list, into shared memory.  Counters are integers, so the result does not depend on
// the order of the atomics.  Latency-bound: a row of 16,000 tokens is 64 KB.
//
// Move.  One CTA per 32 kept tokens copies K, V and the score of each; the new pages are nobody's
// source, so all of it runs at once.  HBM-bound: each kept token is read and written once.
//
// Measured (8 kv heads of 128): 16 rows of 4,321 to 16,345 tokens cut to 4,096, 538 MB: 17 us the
// selection, 79 the move (6.8 TB/s, the copy rate); one row of 2,111 to 1,024: 12 us both.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "evict.h"
#include "launch.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace dev {

constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelRun = 40;  // scores of a thread kept in shared memory; the rest of its run is re-read
constexpr int kSelSlice = 8192;  // tokens of one CTA before a cluster shares the row
constexpr int kSelWarps = kSelThreads / 32;

struct SelShared {
    uint32_t hist[2][kSelBins];
    uint32_t count[2];             // the slice's tokens that stay for sure, and equal to the threshold
    uint32_t warp[2][kSelWarps];
    uint32_t pick[3];              // of the current pass: bin, tokens above it, tokens in it
};

// A score as an integer that orders as the number does (-0 as 0), NaN below every number.
__device__ __forceinline__ uint32_t score_key(float f) {
    if (f != f) return 0u;
    const uint32_t u = __float_as_uint(f + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sums over the CTA of two counts a thread; the CTA's totals in a, b's place.
__device__ __forceinline__ void scan2(uint32_t &a, uint32_t &b, uint32_t &a_before, uint32_t &b_before,
                                      uint32_t (&warps)[2][kSelWarps]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    if (lane == 31) {
        warps[0][warp] = x;
        warps[1][warp] = y;
    }
    __syncthreads();
    uint32_t p = warps[0][lane], q = warps[1][lane];  // 32 warps: every warp scans their sums
    const uint32_t p0 = p, q0 = q;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, p, o), v = __shfl_up_sync(0xffffffffu, q, o);
        if (lane >= o) {
            p += u;
            q += v;
        }
    }
    a_before = x - a + __shfl_sync(0xffffffffu, p - p0, warp);
    b_before = y - b + __shfl_sync(0xffffffffu, q - q0, warp);
    a = __shfl_sync(0xffffffffu, p, 31);
    b = __shfl_sync(0xffffffffu, q, 31);
    __syncthreads();
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictRow *rows, const int32_t *pages,
                                                                   const float *scores, int32_t *kept, int num_sink,
                                                                   int num_recent, int cluster, int page_size, int page_shift,
                                                                   int run_cap) {
    extern __shared__ __align__(16) uint8_t sel_raw[];
    SelShared &sh = *reinterpret_cast<SelShared *>(sel_raw);
    uint32_t *keys = reinterpret_cast<uint32_t *>(sel_raw + sizeof(SelShared));  // [run_cap][threads]
    cg::cluster_group cl = cg::this_cluster();
    const int rank = blockIdx.x % cluster;
    const EvictRow row = rows[blockIdx.x / cluster];
    const int tid = threadIdx.x;
    const int L = row.length;
    auto join = [&]() {
        if (cluster > 1)
            cl.sync();
        else
            __syncthreads();
    };
    // this thread's tokens: [i0, i0 + n)
    const int run = (L + cluster * kSelThreads - 1) / (cluster * kSelThreads);
    const int i0 = min(L, (rank * kSelThreads + tid) * run), n = min(L - i0, run);
    griddep_wait();  // the scores may come from the previous kernel
    griddep_launch();
    if (row.keep >= L) {  // left alone (the whole cluster alike)
        for (int j = 0; j < n; ++j) kept[row.kept_base + i0 + j] = i0 + j;
        return;
    }
    const int mid0 = num_sink, mid1 = L - num_recent;
    auto slot = [&](int i) { return (size_t)pages[row.kv_base + (i >> page_shift)] * page_size + (i & (page_size - 1)); };
    auto key_at = [&](int j) { return j < run_cap ? keys[j * kSelThreads + tid] : score_key(scores[slot(i0 + j)]); };
    // eight page ids, then eight scores, in flight
    for (int j0 = 0; j0 < min(n, run_cap); j0 += 8) {
        size_t at[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) at[j] = j0 + j < n ? slot(i0 + j0 + j) : 0;
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = j0 + j < n ? scores[at[j]] : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < min(n, run_cap)) keys[(j0 + j) * kSelThreads + tid] = score_key(f[j]);
    }
    for (int i = tid; i < kSelBins; i += kSelThreads) sh.hist[0][i] = 0;
    __syncthreads();

    uint32_t prefix = 0, mask = 0;                // the threshold's bits found so far
    int want = row.keep - num_sink - num_recent;  // tokens still to take among those that match them
    bool whole = want == 0;                       // every token that matches is taken (or none is wanted)
    const bool none = want == 0;
    for (int pass = 0; pass < 3 && !whole; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t bits = pass == 2 ? 1023u : 2047u;
        uint32_t *h = sh.hist[pass & 1];
        for (int j = 0; j < run; ++j) {
            const int i = i0 + j;
            const uint32_t k = j < n ? key_at(j) : 0u;
            const bool in = j < n && i >= mid0 && i < mid1 && (k & mask) == prefix;
            const uint32_t bin = (k >> shift) & bits;
            // the lanes that share the first one's bin (equal scores are common: tokens that nobody
            // looks at) add once
            const unsigned act = __ballot_sync(0xffffffffu, in);
            if (in) {
                const int first = __ffs(act) - 1;
                const uint32_t b0 = __shfl_sync(act, bin, first);
                const unsigned same = __ballot_sync(act, bin == b0);
                if (bin != b0)
                    atomicAdd(&h[bin], 1u);
                else if ((tid & 31) == first)
                    atomicAdd(&h[bin], (uint32_t)__popc(same));
            }
        }
        join();
        // the cluster's histogram from the top, two bins a thread; every CTA finds the same bin
        uint32_t hi = 0, lo = 0;
        const int top = kSelBins - 1 - 2 * tid;  // this thread's bins: top, top - 1
        if (cluster == 1) {
            hi = h[top];
            lo = h[top - 1];
        } else {
            uint2 v[kEvictMaxCluster];
#pragma unroll
            for (int r = 0; r < kEvictMaxCluster; ++r)
                if (r < cluster) v[r] = *reinterpret_cast<const uint2 *>(cl.map_shared_rank(h, r) + top - 1);
#pragma unroll
            for (int r = 0; r < kEvictMaxCluster; ++r)
                if (r < cluster) {
                    lo += v[r].x;
                    hi += v[r].y;
                }
        }
        uint32_t all = hi + lo, zero = 0, above, unused;
        // the other histogram was last read in the pass before, which the barrier above has ended
        uint32_t *next = sh.hist[(pass + 1) & 1];
        for (int i = tid; i < kSelBins; i += kSelThreads) next[i] = 0;
        const uint32_t mine = all;
        scan2(all, zero, above, unused, sh.warp);
        if (above < (uint32_t)want && above + mine >= (uint32_t)want) {
            const bool second = above + hi < (uint32_t)want;
            sh.pick[0] = second ? top - 1 : top;
            sh.pick[1] = second ? above + hi : above;
            sh.pick[2] = second ? lo : hi;
        }
        __syncthreads();
        prefix |= sh.pick[0] << shift;
        mask |= bits << shift;
        want -= (int)sh.pick[1];
        whole = want == (int)sh.pick[2];
        __syncthreads();
    }
    // tokens whose leading bits are above `prefix` stay; of those that match it all (whole), or the
    // first `want`
    auto kind = [&](int j, bool &sure, bool &equal) {
        const int i = i0 + j;
        sure = i < mid0 || i >= mid1;
        equal = false;
        if (!sure && !none) {
            const uint32_t k = key_at(j) & mask;
            sure = k > prefix || (whole && k == prefix);
            equal = !whole && k == prefix;
        }
    };
    uint32_t n_sure = 0, n_equal = 0, s_before, e_before;
    for (int j = 0; j < n; ++j) {
        bool s, e;
        kind(j, s, e);
        n_sure += s;
        n_equal += e;
    }
    scan2(n_sure, n_equal, s_before, e_before, sh.warp);
    int out = row.kept_base, left = want;  // where this CTA writes; equal tokens still wanted
    if (cluster > 1) {
        if (tid == 0) {
            sh.count[0] = n_sure;
            sh.count[1] = n_equal;
        }
        cl.sync();
        for (int r = 0; r < rank; ++r) {
            const uint32_t *o = cl.map_shared_rank(sh.count, r);
            const int take = min(left, (int)o[1]);
            out += (int)o[0] + take;
            left -= take;
        }
    }
    // this thread's first output: the sure tokens before it and the equal ones that were taken
    int e_seen = (int)e_before;
    out += (int)s_before + min(e_seen, left);
    for (int j = 0; j < n; ++j) {
        bool s, e;
        kind(j, s, e);
        if (s || (e && e_seen < left)) kept[out++] = i0 + j;
        e_seen += e;
    }
    if (cluster > 1) cl.sync();  // nobody leaves while another CTA may still read its shared memory
}

// `vec` 16-byte vectors of one token's K (and V, page_size slots further).  `group` lanes (a power of
// two) copy a token, four vectors of K and four of V in flight each.
constexpr int kMoveThreads = 256;
__global__ void __launch_bounds__(kMoveThreads, 4)
    evict_move_kernel(const EvictRow *rows, const EvictTask *tasks, const int32_t *pages, const int32_t *dst,
                      const int32_t *kept, uint4 *kv, float *scores, int vec, int group, int page_size, int page_shift) {
    __shared__ long long src_slot[kEvictTaskTokens], dst_slot[kEvictTaskTokens];
    const EvictTask task = tasks[blockIdx.x];
    const EvictRow row = rows[task.row];
    const int n = min(kEvictTaskTokens, row.keep - task.first);
    griddep_wait();
    griddep_launch();
    if ((int)threadIdx.x < n) {
        const int i = task.first + threadIdx.x, from = kept[row.kept_base + i];
        const long long sp = pages[row.kv_base + (from >> page_shift)], dp = dst[row.dst_base + (i >> page_shift)];
        const int so = from & (page_size - 1), dn = i & (page_size - 1);
        src_slot[threadIdx.x] = (sp * 2 * page_size + so) * vec;
        dst_slot[threadIdx.x] = (dp * 2 * page_size + dn) * vec;
        scores[dp * page_size + dn] = scores[sp * page_size + so];
    }
    __syncthreads();
    const long long to_v = (long long)page_size * vec;
    const int lane = threadIdx.x & (group - 1);
    for (int k = threadIdx.x / group; k < n; k += kMoveThreads / group) {
        const uint4 *from = kv + src_slot[k];
        uint4 *to = kv + dst_slot[k];
        for (int c0 = lane; c0 < vec; c0 += 4 * group) {
            uint4 x[4], y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + j * group < vec) {
                    x[j] = __ldcs(from + c0 + j * group);
                    y[j] = __ldcs(from + to_v + c0 + j * group);
                }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + j * group < vec) {
                    __stcs(to + c0 + j * group, x[j]);
                    __stcs(to + to_v + c0 + j * group, y[j]);
                }
        }
    }
}

}  // namespace dev

cudaError_t launch_evict(const Shape &s, const EvictPlan &p, void *ws, void *kv_layer, float *scores, int32_t *kept,
                         cudaStream_t st) {
    uint8_t *w = static_cast<uint8_t *>(ws);
    const EvictRow *rows = reinterpret_cast<const EvictRow *>(w + p.off_rows);
    const int32_t *pages = reinterpret_cast<const int32_t *>(w + p.off_pages);
    const int32_t *dst = reinterpret_cast<const int32_t *>(w + p.off_dst);
    int cluster = 1;
    while (cluster < kEvictMaxCluster && p.longest > dev::kSelSlice * cluster) cluster *= 2;
    const int run = (p.longest + cluster * dev::kSelThreads - 1) / (cluster * dev::kSelThreads);
    const int cap = run < dev::kSelRun ? run : dev::kSelRun;
    const size_t smem = sizeof(dev::SelShared) + (size_t)cap * dev::kSelThreads * 4;
    cudaError_t e = set_smem_limit((const void *)dev::evict_select_kernel,
                                   sizeof(dev::SelShared) + (size_t)dev::kSelRun * dev::kSelThreads * 4, st);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.rows * cluster);
    cfg.blockDim = dim3(dev::kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, dev::evict_select_kernel, rows, pages, static_cast<const float *>(scores), kept, p.num_sink,
                           p.num_recent, cluster, s.page_size, s.page_shift(), cap);
    if (e != cudaSuccess || p.tasks == 0) return e;
    const int vec = s.num_kv_heads * s.head_dim / 8;
    int group = 1;
    while (group < 32 && group < vec) group *= 2;
    return launch_pdl(dev::evict_move_kernel, dim3(p.tasks), dim3(dev::kMoveThreads), 0, st, rows,
                      reinterpret_cast<const EvictTask *>(w + p.off_tasks), pages, dst, static_cast<const int32_t *>(kept),
                      static_cast<uint4 *>(kv_layer), scores, vec, group, s.page_size, s.page_shift());
}

}  // namespace pkv
