// Page and slot maps of a step, built on the device from the rows' lengths (pkv_build_maps).
//
// Row r holds len_r tokens in held_r pages and gets new_r more: need_r = ceil((len_r + new_r) / P) pages.  Pages
// past need_r go on the stack of free pages, rows and blocks ascending; then rows in order take their missing
// ones from its top.  So with B and T the sums of the pages given back and taken by earlier rows, block b of
// row r is, of the stack F_0 .. F_n-1 followed by the pages given back, number
//     n + sum(back) - 1 - (T_r + b - held_r),
// and everything follows from prefix sums over the rows.  Every CTA makes these sums for itself in shared
// memory, which costs less than a second launch or a barrier over the grid; the outputs (page list, slots,
// positions) are then cut evenly over the CTAs, and a warp finds its first row by bisection.
// The pages held and the free count may be updated in place: a CTA could then overwrite what another has yet to
// read, so in that case a second kernel writes them.
// Latency-bound: a chain of loads (lengths, offsets, table) and the stores.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "ptx.cuh"
#include "tree.h"

namespace pkv {
namespace dev {

constexpr int kMapThreads = 512, kMapWarps = kMapThreads / 32;
constexpr int kMapBadRow = -1, kMapBadSize = -2, kMapBadStack = -3;

struct MapSums {
    long long fresh, need, back, taken;
};
__device__ __forceinline__ MapSums operator+(const MapSums &a, const MapSums &b) {
    return MapSums{a.fresh + b.fresh, a.need + b.need, a.back + b.back, a.taken + b.taken};
}

// In shared memory: for row r, offsets of its new tokens, pages, pages given back and pages taken, and its length.
struct MapRows {
    int32_t *qo, *kvp, *back, *taken, *seq, *held;
};

// The last row whose offset is at or below `at` (offsets ascend; rows without an entry share one).
__device__ __forceinline__ int map_row(const int32_t *off, int rows, int at) {
    int lo = 0, hi = rows - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= at)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kMapThreads) maps_kernel(const MapsArgs a, int own_counts) {
    extern __shared__ __align__(16) int32_t map_raw[];
    __shared__ MapSums warp_sums[kMapWarps];
    __shared__ int bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = a.rows;
    const MapRows m{map_raw, map_raw + R + 1, map_raw + 2 * (R + 1), map_raw + 3 * (R + 1), map_raw + 4 * (R + 1),
                    map_raw + 5 * (R + 1)};
    if (tid == 0) bad = 0;
    griddep_wait();
    griddep_launch();
    __syncthreads();
    const int P = 1 << a.page_shift, F = *a.free_count;
    MapSums before = {0, 0, 0, 0};
    for (int r0 = 0; r0 < R; r0 += kMapThreads) {
        const int r = r0 + tid;
        MapSums v = {0, 0, 0, 0};
        if (r < R) {
            const int seq = a.seq[r], fresh = a.fresh[r], held = a.held[r];
            const long long need = ((long long)seq + fresh + P - 1) >> a.page_shift;
            if (seq < 0 || fresh < 0 || held < 0 || held > a.max_blocks || need > a.max_blocks || (long long)seq + fresh > INT32_MAX)
                bad = kMapBadRow;
            else
                v = MapSums{fresh, need, need < held ? held - need : 0, need > held ? need - held : 0};
            m.seq[r] = seq;
            m.held[r] = held;
        }
        MapSums s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const MapSums u{__shfl_up_sync(0xffffffffu, s.fresh, o), __shfl_up_sync(0xffffffffu, s.need, o),
                            __shfl_up_sync(0xffffffffu, s.back, o), __shfl_up_sync(0xffffffffu, s.taken, o)};
            if (lane >= o) s = s + u;
        }
        if (lane == 31) warp_sums[warp] = s;
        __syncthreads();
        MapSums mine = before, all = before;
        for (int w = 0; w < kMapWarps; ++w) {
            if (w < warp) mine = mine + warp_sums[w];
            all = all + warp_sums[w];
        }
        if (r < R) {
            m.qo[r] = (int)(mine.fresh + s.fresh - v.fresh);
            m.kvp[r] = (int)(mine.need + s.need - v.need);
            m.back[r] = (int)(mine.back + s.back - v.back);
            m.taken[r] = (int)(mine.taken + s.taken - v.taken);
        }
        before = all;
        __syncthreads();
    }
    int status = bad;
    constexpr long long MOST = INT32_MAX - 4096;  // 32-bit steps past the last entry
    if (!status && (before.fresh > min((long long)a.token_capacity, MOST) || before.need > min((long long)a.indices_capacity, MOST)))
        status = kMapBadSize;
    if (!status && (F < 0 || F > a.free_capacity || F + before.back > a.free_capacity)) status = kMapBadStack;
    if (!status && before.taken > F + before.back) status = (int)min(before.taken - F - before.back, (long long)INT32_MAX);
    const int T = status ? 0 : (int)before.fresh, pages = status ? 0 : (int)before.need;
    const int back = status ? 0 : (int)before.back, taken = status ? 0 : (int)before.taken;
    if (tid == 0) {
        m.qo[R] = T;
        m.kvp[R] = pages;
        m.back[R] = back;
        m.taken[R] = taken;
    }
    __syncthreads();

    auto given_back_at = [&](int q) -> const int32_t * {  // where page number q of those given back stands
        const int r = map_row(m.back, R, q);
        return a.table + r * a.table_stride + (m.kvp[r + 1] - m.kvp[r]) + (q - m.back[r]);
    };
    // where the id of block b of row r stands
    auto page_at = [&](int r, int b) -> const int32_t * {
        if (b < m.held[r]) return a.table + r * a.table_stride + b;
        const int at = F + back - 1 - (m.taken[r] + b - m.held[r]);
        return at < F ? a.free_pages + at : given_back_at(at - F);
    };
    const int id = blockIdx.x * kMapThreads + tid, step = gridDim.x * kMapThreads;
    // A warp takes a run of entries, a thread every 32nd of it: their rows follow from the first one's.  Four page
    // ids are in flight a thread.  The warps are shared out between pages and tokens, so that neither waits
    // for the other
    constexpr int BATCH = 4;
    const int warps = gridDim.x * kMapWarps, my_warp = warp * gridDim.x + blockIdx.x, tokens = a.slots || a.positions ? T : 0;
    const int page_warps = tokens ? max(1, min(warps - 1, (int)((long long)warps * pages / ((long long)pages + tokens)))) : warps;
    auto entries = [&](int total, int w, int of, const int32_t *off, auto &&source, auto &&store) {
        if (w < 0 || w >= of) return;
        const int per = (int)(((long long)total + of - 1) / of + 31) & ~31;
        const long long begin = (long long)w * per;
        if (begin >= total) return;
        const int end = (int)min((long long)total, begin + per);
        int r = map_row(off, R, (int)begin);
        for (int e0 = (int)begin + lane; e0 < end; e0 += 32 * BATCH) {
            const int32_t *from[BATCH];
            int row[BATCH], page[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int e = e0 + 32 * i;
                from[i] = nullptr;
                if (e >= end) continue;
                while (off[r + 1] <= e) ++r;
                row[i] = r;
                from[i] = source(r, e);
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) page[i] = from[i] ? *from[i] : -1;
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (e0 + 32 * i < end) store(row[i], e0 + 32 * i, page[i]);
        }
    };
    entries(
        pages, my_warp, page_warps, m.kvp, [&](int r, int e) { return page_at(r, e - m.kvp[r]); },
        [&](int r, int e, int page) {
            a.kvi[e] = page;
            const int b = e - m.kvp[r];
            if (b >= m.held[r]) a.table[r * a.table_stride + b] = page;
        });
    for (int q = id; q < back; q += step) a.free_pages[F + q] = *given_back_at(q);
    if (a.slots || a.positions) {
        auto position = [&](int r, int t) { return m.seq[r] + t - m.qo[r]; };
        entries(
            T, my_warp - page_warps, warps - page_warps, m.qo, [&](int r, int t) { return a.slots ? page_at(r, position(r, t) >> a.page_shift) : nullptr; },
            [&](int r, int t, int page) {
                const int pos = position(r, t);
                if (a.slots) a.slots[t] = (page << a.page_shift) + (pos & (P - 1));
                if (a.positions) a.positions[t] = pos;
            });
        for (int t = T + id; t < a.token_capacity; t += step) {
            if (a.slots) a.slots[t] = -1;
            if (a.positions) a.positions[t] = 0;
        }
    }
    for (int r = id; r <= R; r += step) {
        a.qo[r] = status ? 0 : m.qo[r];
        a.kvp[r] = status ? 0 : m.kvp[r];
        if (r < R) {
            const int fresh = m.qo[r + 1] - m.qo[r], need = m.kvp[r + 1] - m.kvp[r];
            a.last[r] = !status && need ? ((m.seq[r] + fresh - 1) & (P - 1)) + 1 : 0;
            if (own_counts) a.held_out[r] = status ? m.held[r] : need;
        }
    }
    if (id == 0) {
        *a.status = status;
        if (own_counts) *a.free_count_out = F + back - taken;
    }
}

// The pages held and the free count in place, from what maps_kernel wrote.
__global__ void __launch_bounds__(kMapThreads) maps_counts_kernel(const MapsArgs a) {
    __shared__ long long sums[kMapWarps];
    griddep_wait();
    griddep_launch();
    if (*a.status != 0) {
        // nothing changes; a target that is not the source still gets the value
        if (a.held_out != a.held)
            for (int r = threadIdx.x; r < a.rows; r += kMapThreads) a.held_out[r] = a.held[r];
        if (threadIdx.x == 0) *a.free_count_out = *a.free_count;
        return;
    }
    long long more = 0;  // pages given back less pages taken
    for (int r = threadIdx.x; r < a.rows; r += kMapThreads) {
        const int need = a.kvp[r + 1] - a.kvp[r];
        more += a.held[r] - need;
        a.held_out[r] = need;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = more;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kMapWarps; ++w) more += sums[w];
        *a.free_count_out = (int)(*a.free_count + more);
    }
}

}  // namespace dev

cudaError_t launch_maps(const MapsArgs &a, cudaStream_t st) {
    const size_t smem = (size_t)6 * (a.rows + 1) * 4;
    cudaError_t e = set_smem_limit((const void *)dev::maps_kernel, (size_t)6 * (kMapsMaxRows + 1) * 4, st);
    if (e != cudaSuccess) return e;
    // an entry a thread, or as many CTAs as fit the GPU
    const long long work = (long long)a.indices_capacity + (a.slots || a.positions ? a.token_capacity : 0);
    const int ctas = (int)std::min<long long>(304, 1 + work / dev::kMapThreads);
    const bool in_place = a.held_out == a.held || a.free_count_out == a.free_count;
    e = launch_pdl(dev::maps_kernel, dim3(ctas), dim3(dev::kMapThreads), smem, st, a, in_place ? 0 : 1);
    if (e == cudaSuccess && in_place) e = launch_pdl(dev::maps_counts_kernel, dim3(1), dim3(dev::kMapThreads), 0, st, a);
    return e;
}

}  // namespace pkv
