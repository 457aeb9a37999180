// Eviction (pkv_run_evict): which tokens of each row stay, and their move to new pages.
//
// Selection.  Of the m = keep - sink - recent best among a row's n = L - sink - recent middle tokens,
// the m-th largest score is found by radix selection on the scores as ordered 32-bit integers (11, 11
// and 10 bits from the top: three histograms), then the tokens above it and, from the lowest position
// up, as many equal to it as are still wanted are written out in position order.  A cluster of up to
// eight CTAs shares a row: each reads its slice of the scores once, through the page list, into
// shared memory; histograms and counts are joined through distributed shared memory.  Counters are
// integers, so the result does not depend on the order of the atomics.  Latency-bound: a row of 2,000
// tokens is 8 KB.
//
// Move.  One CTA per 32 kept tokens copies K, V and the score of each; the new pages are nobody's
// source, so all of it runs at once.  HBM-bound: each kept token is read and written once.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "evict.h"
#include "launch.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace dev {

constexpr int kSelThreads = 512;
constexpr int kSelBins = 2048;
constexpr int kSelKeysMax = 40 * 1024;  // scores of one CTA's slice kept in shared memory; later ones are re-read
constexpr int kSelWarps = kSelThreads / 32;

struct SelShared {
    uint32_t hist[2][kSelBins];
    uint32_t count[2];             // the slice's middle tokens above, and equal to, the threshold
    uint32_t warp[2][kSelWarps];
    uint32_t pick[3];              // of the current pass: bin, tokens above it, tokens in it
};

// A score as an integer that orders as the number does (-0 as 0), NaN below every number.
__device__ __forceinline__ uint32_t score_key(float f) {
    if (f != f) return 0u;
    const uint32_t u = __float_as_uint(f + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictRow *rows, const int32_t *pages,
                                                                   const float *scores, int32_t *kept, int num_sink,
                                                                   int num_recent, int cluster, int page_size, int page_shift,
                                                                   int keys_cap) {
    extern __shared__ __align__(16) uint8_t sel_raw[];
    SelShared &sh = *reinterpret_cast<SelShared *>(sel_raw);
    uint32_t *keys = reinterpret_cast<uint32_t *>(sel_raw + sizeof(SelShared));
    cg::cluster_group cl = cg::this_cluster();
    const int rank = blockIdx.x % cluster;
    const EvictRow row = rows[blockIdx.x / cluster];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = row.length;
    const int slice = ((L + cluster - 1) / cluster + 31) & ~31;
    const int begin = min(L, rank * slice), end = min(L, begin + slice);
    griddep_wait();  // the scores may come from the previous kernel
    griddep_launch();
    if (row.keep >= L) {  // left alone (the whole cluster alike)
        for (int i = begin + tid; i < end; i += kSelThreads) kept[row.kept_base + i] = i;
        return;
    }
    const int mid0 = num_sink, mid1 = L - num_recent;
    auto load = [&](int i) {
        return score_key(scores[(size_t)pages[row.kv_base + (i >> page_shift)] * page_size + (i & (page_size - 1))]);
    };
    auto key_at = [&](int i) { return i - begin < keys_cap ? keys[i - begin] : load(i); };
    for (int i = begin + tid; i < min(end, begin + keys_cap); i += kSelThreads) keys[i - begin] = load(i);
    for (int i = tid; i < kSelBins; i += kSelThreads) sh.hist[0][i] = 0;
    __syncthreads();

    uint32_t prefix = 0, mask = 0;               // the threshold's bits found so far
    int want = row.keep - num_sink - num_recent;  // tokens still to take among those that match them
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t bits = pass == 2 ? 1023u : 2047u;
        uint32_t *h = sh.hist[pass & 1];
        for (int i0 = begin; i0 < end; i0 += kSelThreads) {
            const int i = i0 + tid;
            const uint32_t k = i < end ? key_at(i) : 0u;
            const bool in = i < end && i >= mid0 && i < mid1 && (k & mask) == prefix;
            const uint32_t bin = (k >> shift) & bits;
            // lanes of one bin (equal scores are common: tokens never looked at) add once
            const unsigned act = __ballot_sync(0xffffffffu, in);
            if (in) {
                const int first = __ffs(act) - 1;
                const uint32_t b0 = __shfl_sync(act, bin, first);
                const unsigned same = __ballot_sync(act, bin == b0);
                if (bin != b0)
                    atomicAdd(&h[bin], 1u);
                else if (lane == first)
                    atomicAdd(&h[bin], (uint32_t)__popc(same));
            }
        }
        cl.sync();
        // the cluster's histogram from the top, four bins a thread; every CTA finds the same bin
        uint32_t n[4] = {0, 0, 0, 0};
        const int top = kSelBins - 1 - 4 * tid;  // this thread's bins: top, top - 1, top - 2, top - 3
        for (int r = 0; r < cluster; ++r) {
            const uint32_t *o = cl.map_shared_rank(h, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) n[j] += o[top - j];
        }
        const uint32_t mine = n[0] + n[1] + n[2] + n[3];
        uint32_t run = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += v;
        }
        if (lane == 31) sh.warp[0][warp] = run;
        uint32_t *next = sh.hist[(pass + 1) & 1];
        for (int i = tid; i < kSelBins; i += kSelThreads) next[i] = 0;
        __syncthreads();
        uint32_t above = run - mine;
        for (int w = 0; w < warp; ++w) above += sh.warp[0][w];
        if (want > 0 && above < (uint32_t)want && above + mine >= (uint32_t)want) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (above < (uint32_t)want && above + n[j] >= (uint32_t)want) {
                    sh.pick[0] = top - j;
                    sh.pick[1] = above;
                }
                above += n[j];
            }
        }
        __syncthreads();
        if (want > 0) {
            prefix |= sh.pick[0] << shift;
            mask |= bits << shift;
            want -= (int)sh.pick[1];
        }
        __syncthreads();
    }
    // the threshold is `prefix`; of the tokens equal to it the first `want` stay (none at all if the
    // middle gives none)
    const bool none = row.keep == num_sink + num_recent;
    auto kind = [&](int i, bool &sure, bool &equal) {
        sure = equal = false;
        if (i >= end) return;
        if (i < mid0 || i >= mid1) {
            sure = true;
        } else if (!none) {
            const uint32_t k = key_at(i);
            sure = k > prefix;
            equal = k == prefix;
        }
    };
    uint32_t n_sure = 0, n_equal = 0;
    for (int i = begin + tid; i < end; i += kSelThreads) {
        bool s, e;
        kind(i, s, e);
        n_sure += s;
        n_equal += e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        n_sure += __shfl_xor_sync(0xffffffffu, n_sure, o);
        n_equal += __shfl_xor_sync(0xffffffffu, n_equal, o);
    }
    if (lane == 0) {
        sh.warp[0][warp] = n_sure;
        sh.warp[1][warp] = n_equal;
    }
    __syncthreads();
    if (tid < 2) {
        uint32_t v = 0;
        for (int w = 0; w < kSelWarps; ++w) v += sh.warp[tid][w];
        sh.count[tid] = v;
    }
    cl.sync();
    int out = row.kept_base, left = none ? 0 : want;  // where this slice writes; equals still wanted
    for (int r = 0; r < rank; ++r) {
        const uint32_t *o = cl.map_shared_rank(sh.count, r);
        const int take = min(left, (int)o[1]);
        out += (int)o[0] + take;
        left -= take;
    }
    for (int i0 = begin; i0 < end; i0 += kSelThreads) {
        const int i = i0 + tid;
        bool s, e;
        kind(i, s, e);
        const unsigned bs = __ballot_sync(0xffffffffu, s), be = __ballot_sync(0xffffffffu, e);
        __syncthreads();  // the counts of the block before have been read
        if (lane == 0) {
            sh.warp[0][warp] = __popc(bs);
            sh.warp[1][warp] = __popc(be);
        }
        __syncthreads();
        int s_before = 0, e_before = 0, s_all = 0, e_all = 0;
        for (int w = 0; w < kSelWarps; ++w) {
            const int a = sh.warp[0][w], b = sh.warp[1][w];
            if (w < warp) {
                s_before += a;
                e_before += b;
            }
            s_all += a;
            e_all += b;
        }
        const unsigned below = (1u << lane) - 1u;
        s_before += __popc(bs & below);
        e_before += __popc(be & below);
        if (s || (e && e_before < left)) kept[out + s_before + min(e_before, left)] = i;
        const int take = min(left, e_all);
        out += s_all + take;
        left -= take;
    }
    cl.sync();  // nobody leaves while another CTA may still read its shared memory
}

// `vec` 16-byte vectors of one token's K (and V), page_size slots apart.
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictRow *rows, const EvictTask *tasks, const int32_t *pages,
                                                         const int32_t *dst, const int32_t *kept, uint4 *kv, float *scores,
                                                         int vec, int page_size, int page_shift) {
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
        src_slot[threadIdx.x] = sp * 2 * page_size + so;
        dst_slot[threadIdx.x] = dp * 2 * page_size + dn;
        scores[dp * page_size + dn] = scores[sp * page_size + so];
    }
    __syncthreads();
    // vectors of K then of V, token after token; eight loads in flight a thread
    const int per = 2 * vec, all = n * per;
    for (int v0 = threadIdx.x; v0 < all; v0 += 8 * blockDim.x) {
        uint4 x[8];
        long long to[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int v = v0 + j * blockDim.x;
            if (v < all) {
                const int k = v / per, w = v % per, c = w < vec ? w : w - vec;
                const long long off = w < vec ? 0 : page_size;
                x[j] = __ldcs(kv + (src_slot[k] + off) * vec + c);
                to[j] = (dst_slot[k] + off) * vec + c;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (v0 + j * (int)blockDim.x < all) kv[to[j]] = x[j];
    }
}

}  // namespace dev

cudaError_t launch_evict(const Shape &s, const EvictPlan &p, void *ws, void *kv_layer, float *scores, int32_t *kept,
                         cudaStream_t st) {
    uint8_t *w = static_cast<uint8_t *>(ws);
    const EvictRow *rows = reinterpret_cast<const EvictRow *>(w + p.off_rows);
    const int32_t *pages = reinterpret_cast<const int32_t *>(w + p.off_pages);
    const int32_t *dst = reinterpret_cast<const int32_t *>(w + p.off_dst);
    // a CTA per 2,048 tokens of the longest cut row, up to eight
    int cluster = 1;
    while (cluster < kEvictMaxCluster && p.longest > 2048 * cluster) cluster *= 2;
    const int slice = ((p.longest + cluster - 1) / cluster + 31) & ~31;
    const int keys = slice < dev::kSelKeysMax ? slice : dev::kSelKeysMax;
    const size_t smem = sizeof(dev::SelShared) + (size_t)keys * 4;
    cudaError_t e = set_smem_limit((const void *)dev::evict_select_kernel,
                                   sizeof(dev::SelShared) + (size_t)dev::kSelKeysMax * 4, st);
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
                           p.num_recent, cluster, s.page_size, s.page_shift(), keys);
    if (e != cudaSuccess || p.tasks == 0) return e;
    return launch_pdl(dev::evict_move_kernel, dim3(p.tasks), dim3(256), 0, st, rows,
                      reinterpret_cast<const EvictTask *>(w + p.off_tasks), pages, dst, static_cast<const int32_t *>(kept),
                      static_cast<uint4 *>(kv_layer), scores, s.num_kv_heads * s.head_dim / 8, s.page_size, s.page_shift());
}

}  // namespace pkv
