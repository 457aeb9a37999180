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
// Latency-bound: a chain of loads (lengths, offsets, table) and the stores.  Measured with the counts written elsewhere, one
// state replayed in a graph (called with states that change from call to call): one row 3.1 us (4.2), 200 rows of up to
// 8,190 tokens in pages of 16 4.5 us (4.8), 500 rows of up to 30,011 in pages of 8 (971,000 page ids) 7.2 us (7.4), 48
// prompts of 8,111 tokens without pages 4.5 us (4.6).  Counts in place: 1.4 to 1.8 us more.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "ptx.cuh"
#include "tree.h"

namespace pkv {
namespace dev {

constexpr int kMapThreads = 512, kMapWarps = kMapThreads / 32;
constexpr int kMapBadRow = -1, kMapBadSize = -2, kMapBadStack = -3;

// Sums over rows: 64-bit where the largest table could overflow 32 (see launch_maps).
template <typename Int>
struct MapSums {
    Int fresh, need, back, taken;
};
template <typename Int>
__device__ __forceinline__ MapSums<Int> operator+(const MapSums<Int> &a, const MapSums<Int> &b) {
    return MapSums<Int>{a.fresh + b.fresh, a.need + b.need, a.back + b.back, a.taken + b.taken};
}
// The sums of this lane and those before it.
template <typename Int>
__device__ __forceinline__ MapSums<Int> scan(MapSums<Int> s, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const MapSums<Int> u{__shfl_up_sync(0xffffffffu, s.fresh, o), __shfl_up_sync(0xffffffffu, s.need, o),
                             __shfl_up_sync(0xffffffffu, s.back, o), __shfl_up_sync(0xffffffffu, s.taken, o)};
        if (lane >= o) s = s + u;
    }
    return s;
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

template <typename Int>
__global__ void __launch_bounds__(kMapThreads) maps_kernel(const MapsArgs a, int own_counts) {
    using Sums = MapSums<Int>;
    extern __shared__ __align__(16) int32_t map_raw[];
    __shared__ Sums warp_sums[kMapWarps + 1];  // of the warps before each, and of all
    __shared__ int bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = a.rows;
    const MapRows m{map_raw, map_raw + R + 1, map_raw + 2 * (R + 1), map_raw + 3 * (R + 1), map_raw + 4 * (R + 1),
                    map_raw + 5 * (R + 1)};
    if (tid == 0) bad = 0;
    griddep_wait();
    griddep_launch();
    __syncthreads();
    const int P = 1 << a.page_shift, F = *a.free_count;
    Sums before = {0, 0, 0, 0};
    for (int r0 = 0; r0 < R; r0 += kMapThreads) {
        const int r = r0 + tid;
        Sums v = {0, 0, 0, 0};
        if (r < R) {
            const int seq = a.seq[r], fresh = a.fresh[r], held = a.held[r];
            const long long need = ((long long)seq + fresh + P - 1) >> a.page_shift;
            if (seq < 0 || fresh < 0 || held < 0 || held > a.max_blocks || need > a.max_blocks || (long long)seq + fresh > INT32_MAX)
                bad = kMapBadRow;
            else
                v = Sums{fresh, (Int)need, (Int)(need < held ? held - need : 0), (Int)(need > held ? need - held : 0)};
            m.seq[r] = seq;
            m.held[r] = held;
        }
        const Sums s = scan(v, lane);
        if (lane == 31) warp_sums[warp] = s;
        __syncthreads();
        if (warp == 0) {
            const Sums w = lane < kMapWarps ? warp_sums[lane] : Sums{0, 0, 0, 0}, t = scan(w, lane);
            __syncwarp();
            if (lane < kMapWarps) warp_sums[lane] = Sums{t.fresh - w.fresh, t.need - w.need, t.back - w.back, t.taken - w.taken};
            if (lane == 31) warp_sums[kMapWarps] = t;
        }
        __syncthreads();
        const Sums mine = before + warp_sums[warp];
        if (r < R) {
            m.qo[r] = (int)(mine.fresh + s.fresh - v.fresh);
            m.kvp[r] = (int)(mine.need + s.need - v.need);
            m.back[r] = (int)(mine.back + s.back - v.back);
            m.taken[r] = (int)(mine.taken + s.taken - v.taken);
        }
        before = before + warp_sums[kMapWarps];
        __syncthreads();
    }
    int status = bad;
    constexpr long long MOST = INT32_MAX - 4096;  // 32-bit steps past the last entry
    if (!status && (before.fresh > min((long long)a.token_capacity, MOST) || before.need > min((long long)a.indices_capacity, MOST)))
        status = kMapBadSize;
    if (!status && (F < 0 || F > a.free_capacity || (long long)F + before.back > a.free_capacity)) status = kMapBadStack;
    if (!status && before.taken > (long long)F + before.back) status = (int)min((long long)before.taken - F - before.back, (long long)INT32_MAX);
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
    const int id = blockIdx.x * kMapThreads + tid, step = gridDim.x * kMapThreads;
    // A warp takes a run of entries, a thread every 32nd of it: their rows follow from the first one's.  Four page
    // ids are in flight a thread.  The warps are shared out between pages and tokens, so that neither waits
    // for the other
    constexpr int BATCH = 4;
    const int warps = gridDim.x * kMapWarps, my_warp = warp * gridDim.x + blockIdx.x, tokens = a.slots || a.positions ? T : 0;
    // a token counts for as many as 32 of them have rows: a warp goes from row to row
    const long long weight = tokens ? min(8, 1 + (int)(32ll * R / tokens)) : 0;
    const int page_warps = tokens ? max(1, min(warps - 1, (int)(warps * (long long)pages / (pages + weight * tokens)))) : warps;
    struct Row {  // the row of the current entry
        int r, begin, end, held, above;  // above: number on the stack of its first missing block
        const int32_t *table;
    };
    auto entries = [&](int total, int w, int of, const int32_t *off, auto &&block, auto &&store) {
        if (w < 0 || w >= of) return;
        const int per = (int)(((long long)total + of - 1) / of + 31) & ~31;
        const long long first = (long long)w * per;
        if (first >= total) return;
        const int end = (int)min((long long)total, first + per);
        Row row;
        auto enter = [&](int r) {
            row.r = r;
            row.begin = off[r];
            row.end = off[r + 1];
            row.held = m.held[r];
            row.above = F + back - 1 - m.taken[r];
            row.table = a.table + r * a.table_stride;
        };
        enter(map_row(off, R, (int)first));
        for (int e0 = (int)first + lane; e0 < end; e0 += 32 * BATCH) {
            int page[BATCH];
            Row at[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int e = e0 + 32 * i;
                if (e >= end) continue;
                while (row.end <= e) enter(row.r + 1);
                at[i] = row;
                const int b = block(row, e);
                const int up = row.above - (b - row.held);  // its number on the stack if it is missing
                page[i] = b < 0 ? -1 : b < row.held ? row.table[b] : up < F ? a.free_pages[up] : *given_back_at(up - F);
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (e0 + 32 * i < end) store(at[i], e0 + 32 * i, page[i]);
        }
    };
    entries(
        pages, my_warp, page_warps, m.kvp, [&](const Row &row, int e) { return e - row.begin; },
        [&](const Row &row, int e, int page) {
            a.kvi[e] = page;
            const int b = e - row.begin;
            if (b >= row.held) a.table[row.r * a.table_stride + b] = page;
        });
    for (long long q = id; q < back; q += step) a.free_pages[F + q] = *given_back_at((int)q);
    if (a.slots || a.positions) {
        auto position = [&](const Row &row, int t) { return m.seq[row.r] + t - row.begin; };
        entries(
            T, my_warp - page_warps, warps - page_warps, m.qo,
            [&](const Row &row, int t) { return a.slots ? position(row, t) >> a.page_shift : -1; },
            [&](const Row &row, int t, int page) {
                const int pos = position(row, t);
                if (a.slots) a.slots[t] = (page << a.page_shift) + (pos & (P - 1));
                if (a.positions) a.positions[t] = pos;
            });
        for (long long t = (long long)T + id; t < a.token_capacity; t += step) {
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

static cudaError_t raise_limit(const void *kernel, cudaStream_t st) {
    return set_smem_limit(kernel, (size_t)6 * (kMapsMaxRows + 1) * 4, st);
}

cudaError_t prepare_maps(cudaStream_t st) {
    const cudaError_t e = raise_limit((const void *)dev::maps_kernel<int>, st);
    return e != cudaSuccess ? e : raise_limit((const void *)dev::maps_kernel<long long>, st);
}

cudaError_t launch_maps(const MapsArgs &a, cudaStream_t st) {
    const size_t smem = (size_t)6 * (a.rows + 1) * 4;
    // an entry a thread, or as many CTAs as fit the GPU
    const long long work = (long long)a.indices_capacity + (a.slots || a.positions ? a.token_capacity : 0);
    const int ctas = (int)std::min<long long>(304, 1 + work / dev::kMapThreads);
    const bool in_place = a.held_out == a.held || a.free_count_out == a.free_count;
    auto launch = [&](auto kernel) {
        const cudaError_t e = raise_limit((const void *)kernel, st);
        return e != cudaSuccess ? e : launch_pdl(kernel, dim3(ctas), dim3(dev::kMapThreads), smem, st, a, in_place ? 0 : 1);
    };
    // no sum is above the tokens that full tables hold
    const bool wide = ((long long)a.rows * a.max_blocks >> (30 - a.page_shift)) > 0;
    cudaError_t e = wide ? launch(dev::maps_kernel<long long>) : launch(dev::maps_kernel<int>);
    if (e == cudaSuccess && in_place) e = launch_pdl(dev::maps_counts_kernel, dim3(1), dim3(dev::kMapThreads), 0, st, a);
    return e;
}

}  // namespace pkv
