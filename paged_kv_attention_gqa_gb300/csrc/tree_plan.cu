// The plan of a speculative step, made on the device (pkv_plan_tree), and the acceptance of a path
// (pkv_run_accept).
//
// Plan.  Block 0 reads the rows' index arrays and gives every attention CTA of a lane (see TreeStart) an equal
// share of the lane's key tiles (a piece of a unit costs two tiles beside its own): prefix sums over the
// rows, then the place of each CTA's first tile by bisection.  The other blocks take a row per warp and walk each node's parents
// to its root: depth, and a bit for every ancestor.
//
// Accept.  A CTA per row and a few layers, a thread per node.  A node goes on from its parent if it is the first
// child whose token is the model's choice there; it is on the path if all nodes above it go on, up to
// the root, which doubling the parents' pointers tells in log2(depth) rounds; its place is its depth.
// Every CTA of the row does this for itself, which costs less than a launch that would pass it on.  Then bulk copies
// take the path's keys and values to the row's next slots (copies by all threads, 16 bytes each, were bound by the
// instructions of their addresses: 12.4 us where bulk copies take 9.0).  HBM-bound for batches (each accepted vector
// read and written once), a chain of loads for one row.
// Measured with states that change from call to call (one state replayed in a graph, whose bytes then come from L2): 64 rows
// of up to 16 nodes, 32 layers of 8 heads of 128, 43 MB: 10.3 us (7.5); 40 rows with paths of 20, 24 layers of 4 heads of 64,
// 16.5 MB: 6.6 us (6.5); one row, 32 layers: 3.8 us (2.7).
// The plan, replayed: one row of 8 nodes 4.3 us, 32 rows of 16 5.1, 64 rows of 61 5.4, 40 rows of 61 up to 32
// deep 7.1.  A lane walks each of its nodes to the root, a load after the other, so deep trees take long: a row's chain of 200
// 100 us, of 256 136, 64 bushy trees of 200 18.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "ptx.cuh"
#include "tree.h"

namespace pkv {

static size_t put(size_t &at, size_t bytes) {
    const size_t here = at;
    at = align_up(at + bytes);
    return here;
}

void tree_layout(const Shape &s, int batch, int tokens, int max_new, int num_indices, int window_left, TreePlan &p) {
    p.window_left = window_left;
    p.batch = batch;
    p.num_tokens = tokens;
    p.max_new = max_new;
    p.words = (max_new + 63) / 64;
    // head_dim 256 has no tensor memory for two query tiles' accumulators
    p.pair = s.head_dim <= 128 && max_new * s.group() > 128;
    p.part_rows = p.pair ? 256 : 128;
    const int tile = tree_tile_tokens(s), unit = tile * (p.pair ? 2 : 1);  // tokens
    const long long units = (long long)batch * s.num_kv_heads * ((max_new + unit - 1) / unit);
    const int whole_tiles = kTreeWholeTiles / (s.head_dim == 256 ? 2 : 1);
    p.whole = (long long)num_indices * s.page_size <= kTreeKeys * whole_tiles * std::min(batch, kTreeWholeRows);
    if (window_left >= 0 && units <= kTreeWholeUnits * s.sm_count) {
        const long long cached = ((long long)window_left + kTreeKeys - 1) / kTreeKeys + 1;  // tiles at most
        p.whole = p.whole || cached + (max_new + kTreeKeys - 1) / kTreeKeys <= whole_tiles;
    }
    const long long most = (long long)s.sm_count * (s.head_dim == 256 ? 2 : 1);
    p.join_blocks = (int)std::min(units * (s.head_dim / 16) * 4, most);
    p.join_rows = max_new > tile ? 8 : (max_new * s.group() + 31) / 32;
    // Blocks of twice the warps where two a unit find room side by side: they take more pieces at once (one row of 517
    // tokens 9.64 us with the small ones, 9.41 with these; one of 64 heads on 4 8.65 and 8.29), but many of them
    // run in turns (two rows of 52 drafted tokens, head_dim 256, 14.2 and 18.0; wide trees 152 and 159).
    p.join_warps = (s.head_dim == 64 ? 4 : 8) * (2 * units * p.join_rows <= s.sm_count ? 2 : 1);
    size_t at = kAlign;
    p.off_rows = put(at, (size_t)batch * sizeof(TreeRow));
    p.off_starts = put(at, (size_t)s.sm_count * sizeof(TreeStart));
    p.off_joins = put(at, (size_t)most * sizeof(TreeJoin));
    p.off_nodes = put(at, (size_t)tokens * sizeof(TreeNode));
    p.off_masks = put(at, (size_t)tokens * p.words * 8);
    p.off_cost = put(at, (size_t)batch * 8);
    p.off_part_o = put(at, (size_t)2 * s.sm_count * p.part_rows * s.head_dim * 4);
    p.off_part_lse = put(at, (size_t)2 * s.sm_count * p.part_rows * 4);
    p.total = at;
}

namespace dev {

struct TreePlanArgs {
    TreeIndex x;
    int batch, tokens, max_new, words, window_left, page_size, page_shift, kv_heads, unit_tokens, tile_tokens, ctas;
    int whole;     // no unit is cut
    int group, head_dim, join_warps, join_blocks;
    int hi;        // kv heads side by side
    TreeHeader *hdr;
    uint32_t tag;  // the handle's
    TreeRow *rows;
    TreeStart *starts;
    TreeJoin *joins;
    TreeNode *nodes;
    unsigned long long *masks;
    long long *cost;  // before row r, of one kv head
};

// Records an error (0: begins the error word).  The plan's blocks do so in any order, so each leaves a word with the
// handle's tag behind; what a word with another tag says is no error of this handle's.
__device__ __forceinline__ void plan_error(const TreePlanArgs &a, int code) {
    unsigned long long *const word = reinterpret_cast<unsigned long long *>(a.hdr);
    const unsigned long long mine = (unsigned long long)a.tag << 32;
    unsigned long long old = *reinterpret_cast<volatile unsigned long long *>(word);
    // three tries do: other blocks of a plan change the word once from a foreign one, and once from no error to one
    for (int i = 0; i < 4 && ((old >> 32) != a.tag || (code != 0 && (uint32_t)old == 0)); ++i) {
        const unsigned long long seen = atomicCAS(word, old, mine | (uint32_t)code);
        if (seen == old) break;
        old = seen;
    }
}

// The index arrays are read by ordinary loads: the kernel before this one, beside which it may already run, writes them,
// and the read-only path (__ldg) asks for memory that nobody writes while the kernel lives.
// A row's first token, 0 if that is no token of the step; and the highest of the rows [from, to), for the whole warp.
__device__ __forceinline__ int first_token(const TreePlanArgs &a, int r) {
    const int q = a.x.qo[r];
    return q <= a.tokens ? q : 0;
}
__device__ __forceinline__ int highest_token(const TreePlanArgs &a, int from, int to) {
    int top = 0;
#pragma unroll 4
    for (int r = from + (threadIdx.x & 31); r < to; r += 32) top = max(top, first_token(a, r));
    return __reduce_max_sync(0xffffffffu, top);
}

// The row's numbers if its index arrays agree (n = 0 and ctx = -1 if not).  `highest`: of the earlier rows' first
// tokens.  A row that begins below it could have tokens of another one, whose nodes would be written twice.
__device__ __forceinline__ TreeRow tree_row(const TreePlanArgs &a, int r, int highest, bool &ok) {
    TreeRow t = {};
    const int q0 = a.x.qo[r], q1 = a.x.qo[r + 1], k0 = a.x.kvp[r], k1 = a.x.kvp[r + 1];
    const int fill = a.x.last[r];
    ok = q0 >= highest && q1 >= q0 && q1 <= a.tokens && q1 - q0 <= a.max_new && k0 >= 0 && k1 >= k0 && k1 <= a.x.num_indices;
    if (r == 0) ok = ok && q0 == 0 && k0 == 0;
    long long length = 0;
    if (ok && k1 > k0) {
        ok = fill >= 1 && fill <= a.page_size;
        length = ((long long)(k1 - k0 - 1) << a.page_shift) + fill;
    }
    ok = ok && length >= q1 - q0 && length < (1ll << 31) - 2 * kTreeKeys;
    t.ctx = -1;
    if (!ok) return t;
    t.q_begin = q0;
    t.n = q1 - q0;
    t.ctx = (int)length - t.n;
    t.kv_base = k0;
    if (t.n == 0) return t;
    const int lo = a.window_left >= 0 ? max(0, t.ctx - a.window_left) : 0;  // the root's first key
    t.kt0 = lo / kTreeKeys;
    t.nc = (t.ctx + kTreeKeys - 1) / kTreeKeys - t.kt0;
    t.nq = (t.n + a.unit_tokens - 1) / a.unit_tokens;
    return t;
}

// The cost of a tile of query unit q of a row, of the unit, and of the row's units of one kv head.
__device__ __forceinline__ int tile_cost(const TreePlanArgs &a, const TreeRow &t, int q) {
    return t.n - q * a.unit_tokens <= a.tile_tokens && a.unit_tokens > a.tile_tokens ? kTreeHalfCost : kTreeTileCost;
}
__device__ __forceinline__ long long unit_cost(const TreePlanArgs &a, const TreeRow &t, int q) {
    return (long long)tree_unit_tiles(t, q, a.unit_tokens) * tile_cost(a, t, q) + kTreePieceCost;
}
__device__ __forceinline__ long long head_cost(const TreePlanArgs &a, const TreeRow &t) {
    long long sum = 0;
    for (int q = 0; q < t.nq; ++q) sum += unit_cost(a, t, q);
    return sum;
}

constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32;

__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const TreePlanArgs a) {
    __shared__ int32_t parent[kPlanWarps][kTreeMaxNew];
    __shared__ long long sums[kPlanWarps];
    __shared__ int joins;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();
    griddep_launch();
    if (blockIdx.x > 0) {
        // ------------------------------------------------ the nodes of a row
        const int r = (blockIdx.x - 1) * kPlanWarps + warp;
        if (r >= a.batch) return;
        bool ok;
        const TreeRow t = tree_row(a, r, highest_token(a, 0, r), ok);
        int32_t *const p = parent[warp];
        for (int i = lane; i < t.n; i += 32) {
            int32_t up = a.x.parents ? a.x.parents[t.q_begin + i] : i - 1;
            if (up < -1 || up >= i) {
                plan_error(a, kErrTreeParent);
                up = -1;
            }
            p[i] = up;
        }
        __syncwarp();
        for (int i = lane; i < t.n; i += 32) {
            unsigned long long m[kTreeMaxNew / 64] = {};
            int depth = -1;
            for (int j = i; j >= 0; j = p[j]) {
                ++depth;
                if (a.window_left < 0 || depth <= a.window_left) {
#pragma unroll
                    for (int w = 0; w < kTreeMaxNew / 64; ++w)
                        if (j >> 6 == w) m[w] |= 1ull << (j & 63);
                }
            }
            a.nodes[t.q_begin + i] = TreeNode{p[i], depth};
            for (int w = 0; w < a.words; ++w) {
                unsigned long long v = m[0];
#pragma unroll
                for (int u = 1; u < kTreeMaxNew / 64; ++u)
                    if (w == u) v = m[u];
                a.masks[(size_t)(t.q_begin + i) * a.words + w] = v;
            }
            if (a.x.positions) a.x.positions[t.q_begin + i] = t.ctx + depth;
        }
        return;
    }
    // ------------------------------------------------ the rows, and each CTA's share
    if (threadIdx.x == kPlanThreads - 1) plan_error(a, 0);  // (of the warp that most often has no row)
    long long before = 0;
    int highest = 0, known = 0;  // of the rows before `known`
    for (int r0 = 0; r0 < a.batch; r0 += kPlanThreads) {
        const int r = r0 + threadIdx.x, first = min(r0 + warp * 32, a.batch);  // (the warp's first row)
        highest = max(highest, highest_token(a, known, first));
        known = first;
        int top = r < a.batch ? first_token(a, r) : 0;  // of the warp's rows up to this one, which is at or above itself
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, top, o);
            if (lane >= o) top = max(top, x);
        }
        long long v = 0;
        if (r < a.batch) {
            bool ok;
            const TreeRow t = tree_row(a, r, max(highest, top), ok);
            if (!ok) plan_error(a, kErrTreeRow);
            a.rows[r] = t;
            v = head_cost(a, t);
        }
        long long c = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, c, o);
            if (lane >= o) c += x;
        }
        if (lane == 31) sums[warp] = c;
        __syncthreads();
        long long mine = before;
        for (int w = 0; w < kPlanWarps; ++w) {
            if (w < warp) mine += sums[w];
            before += sums[w];
        }
        __syncthreads();
        if (r < a.batch) a.cost[r] = mine + c - v;
    }
    if (threadIdx.x == 0) joins = 0;
    __syncthreads();
    const int lanes = a.hi, slices = a.ctas / lanes, heads = a.kv_heads / lanes;
    const long long total = heads * before, share = max((total + slices - 1) / slices, (long long)(a.whole ? kTreeLeastWhole : kTreeLeastCost));
    for (int c = threadIdx.x; c < a.ctas; c += kPlanThreads) {
        TreeStart s = {};
        const int slice = c / lanes;
        s.h0 = c % lanes;
        s.hi = lanes;
        struct Place {
            int r, unit, tile;
            long long first, last;  // the slices with the unit's first and last piece
        };
        auto place = [&](long long at) {
            Place p = {a.batch, 0, 0, 0, 0};
            if (at >= total) return p;
            int lo = 0, hi = a.batch - 1;  // the last row that begins at or before `at`
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (heads * a.cost[mid] <= at)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            p.r = lo;
            const TreeRow t = a.rows[lo];
            const long long off = at - heads * a.cost[lo], head = head_cost(a, t);
            int q = 0;
            long long inside = off % head, cost = unit_cost(a, t, 0);
            while (inside >= cost) {
                inside -= cost;
                cost = unit_cost(a, t, ++q);
            }
            const int each = tile_cost(a, t, q);
            const long long begin = at - inside;
            p.unit = (int)(off / head) * t.nq + q;
            if (a.whole) return p;  // every CTA from the beginning of the unit that it would have begun in
            p.tile = (int)(max(0ll, inside - kTreePieceCost) / each);  // (one of them: inside is below the unit's cost)
            // a CTA begins inside the unit if it is past the unit's own cost and first tile
            p.first = (begin + kTreePieceCost + each - 1) / share;
            p.last = (begin + cost - 1) / share;
            return p;
        };
        const bool used = slice < slices;
        const Place from = place(used ? slice * share : total), to = place(used ? (slice + 1) * share : total);
        s.r = from.r;
        s.unit = from.unit;
        s.tile = from.tile;
        if (from.r < a.batch) s.row = a.rows[from.r];
        s.r_end = to.r;
        s.unit_end = to.unit;
        s.tile_end = to.tile;
        a.starts[c] = s;
        // the unit that goes on in the next CTA, if it begins here
        if (to.r < a.batch && to.tile > 0 && (from.r != to.r || from.unit != to.unit || from.tile == 0)) {
            const TreeRow t = a.rows[to.r];
            const int q = to.unit % t.nq;
            TreeJoin j;
            j.token = t.q_begin + q * a.unit_tokens;
            j.tokens = min(a.unit_tokens, t.n - q * a.unit_tokens);
            j.kvh = to.unit / t.nq * lanes + s.h0;
            j.cta = c;
            j.step = lanes;
            j.count = (int)(to.last - to.first) + 1;
            const TreeJoinPart part = tree_join_part(a.head_dim, a.join_warps, j.tokens * a.group, j.count);
            j.groups = (int16_t)part.groups;
            j.rows = (int16_t)part.rows;
            const int columns = a.head_dim / 16 >> part.groups, blocks = columns * (tree_join_rows(j.tokens * a.group) / part.rows);
            const int at = atomicAdd(&joins, blocks);
            for (int i = 0; i < blocks; ++i) {
                j.group0 = (int16_t)(i % columns << part.groups);
                j.row0 = (int16_t)(i / columns * part.rows);
                if (at + i < a.join_blocks) a.joins[at + i] = j;
            }
        }
    }
    __syncthreads();
    for (int i = joins + threadIdx.x; i < a.join_blocks; i += kPlanThreads) a.joins[i].count = 0;
}

struct AcceptArgs {
    TreeAccept x;
    const TreeRow *rows;
    const TreeNode *nodes;
    const int32_t *pages;
    TreeHeader *hdr;
    int lanes;  // with a buffer, of each warp
    int layers_per_cta, page_size, page_shift, vecs, num_cache_pages;  // vecs: 16-byte vectors of a token's K (or V)
};

constexpr int kAcceptThreads = 256, kAcceptWarps = kAcceptThreads / 32, kAcceptBuffer = 2048;
constexpr int kAcceptBytes = 32768;  // of buffers
constexpr int kAcceptCtas = 5;       // an SM (64 rows, 32 layers: 10.2 us; three with twice the buffers 11.3)

static_assert(kAcceptThreads == kTreeMaxNew, "a thread a node");
constexpr int kAcceptRounds = 8;
static_assert(1 << kAcceptRounds >= kTreeMaxNew, "as many rounds reach past the root of the longest path");

template <typename Token>
__global__ void __launch_bounds__(kAcceptThreads, kAcceptCtas) tree_accept_kernel(const AcceptArgs a) {
    extern __shared__ __align__(128) uint8_t buffers[];
    __shared__ uint64_t bars[kAcceptThreads];
    __shared__ Token draft[kTreeMaxNew], target[kTreeMaxNew];
    __shared__ int32_t first[kTreeMaxNew], path[kTreeMaxNew];
    __shared__ int2 above[kTreeMaxNew];      // a node above it (-1: none) and whether all below that go on
    __shared__ long long slot[kTreeMaxNew];  // the cache row of K of the row's token ctx + i, -1 = its page is not one
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (lane < a.lanes) mbar_init(&bars[warp * a.lanes + lane], 1);
    fence_barrier_init();
    griddep_wait();
    griddep_launch();
    const TreeRow t = a.rows[r];
    const bool node = tid < t.n;
    TreeNode self = {-1, 0};
    if (node) {
        const int pos = t.ctx + tid, page = a.pages[t.kv_base + (pos >> a.page_shift)];
        self = a.nodes[t.q_begin + tid];
        draft[tid] = static_cast<const Token *>(a.x.draft)[t.q_begin + tid];
        target[tid] = static_cast<const Token *>(a.x.target)[t.q_begin + tid];
        first[tid] = kTreeMaxNew;
        slot[tid] = (unsigned)page < (unsigned)a.num_cache_pages ? (long long)page * 2 * a.page_size + (pos & (a.page_size - 1)) : -1;
    }
    __syncthreads();
    const bool agrees = node && self.parent >= 0 && draft[tid] == target[self.parent];
    if (agrees) atomicMin(&first[self.parent], tid);
    __syncthreads();
    int up = node ? self.parent : -1;
    bool on = tid == 0 || (agrees && first[self.parent] == tid);
    for (int round = 0; round < kAcceptRounds && __syncthreads_or(up >= 0); ++round) {
        above[tid] = make_int2(up, on);
        __syncthreads();
        if (up >= 0) {
            const int2 e = above[up];
            up = e.x;
            on = on && e.y;
        }
    }
    on = on && node;
    if (on) path[self.depth] = tid;
    const int len = __syncthreads_count(on);
    if (blockIdx.y == 0) {
        if (node) a.x.accepted[t.q_begin + tid] = tid < len ? path[tid] : -1;
        if (tid < len && slot[tid] < 0) atomicCAS(&a.hdr->err, 0, kErrTreePage);
        if (tid == 0) {
            a.x.count[r] = len;
            static_cast<Token *>(a.x.next)[r] = len ? target[path[len - 1]] : Token(-1);
            if (a.x.seq && len) a.x.seq[r] = t.ctx + len;
        }
    }
    // A copy is up to 2 KB of K or V of a path node in a layer, through a buffer in shared memory of its lane: two lanes of
    // each warp have one, more where they are smaller
    if (lane >= a.lanes) return;
    const int l0 = blockIdx.y * a.layers_per_cta, layers = min(a.x.layers - l0, a.layers_per_cta);
    const int bytes = a.vecs * 16, parts = (bytes + kAcceptBuffer - 1) / kAcceptBuffer, each = 2 * parts;
    const int mine = warp * a.lanes + lane;
    uint8_t *const buffer = buffers + mine * (kAcceptBytes / (kAcceptWarps * a.lanes));
    uint64_t *const bar = bars + mine;
    uint32_t phase = 0;
    for (int q = mine; q < layers * len * each; q += kAcceptWarps * a.lanes) {
        const int part = q % parts, v = q / parts & 1, item = q / each, i = item % len;
        const long long l = l0 + item / len, token = t.q_begin + path[i], at = slot[i];
        if (at < 0) continue;
        const int begin = part * kAcceptBuffer, size = min(kAcceptBuffer, bytes - begin);
        const long long from = v ? l * a.x.v_layer + token * a.x.v_token : l * a.x.k_layer + token * a.x.k_token;  // elements
        const long long to = l * a.x.cache_layer + (at + (v ? a.page_size : 0)) * a.vecs * 8;
        if (phase) bulk_store_wait_read();  // the buffer's last store
        mbar_arrive_expect_tx(bar, size);
        bulk_load(buffer, static_cast<const uint8_t *>(v ? a.x.v : a.x.k) + from * 2 + begin, size, bar);
        if (!mbar_wait(bar, phase++ & 1, &a.hdr->err, kErrWaitFull)) {
            for (uint32_t d = 0; d < 1024; ++d) __nanosleep(1000);  // the copy in flight lands before the CTA may end
            break;
        }
        bulk_store(static_cast<uint8_t *>(a.x.cache) + to * 2 + begin, buffer, size);
    }
    bulk_store_wait();
}

}  // namespace dev

cudaError_t launch_tree_plan(const Shape &s, const TreePlan &p, const TreeIndex &x, uint32_t tag, void *ws, cudaStream_t st) {
    uint8_t *w = static_cast<uint8_t *>(ws);
    dev::TreePlanArgs a;
    a.x = x;
    a.batch = p.batch;
    a.tokens = p.num_tokens;
    a.max_new = p.max_new;
    a.words = p.words;
    a.window_left = p.window_left;
    a.page_size = s.page_size;
    a.page_shift = s.page_shift();
    a.kv_heads = s.num_kv_heads;
    a.tile_tokens = tree_tile_tokens(s);
    a.unit_tokens = a.tile_tokens * (p.pair ? 2 : 1);
    a.ctas = s.sm_count;
    a.whole = p.whole;
    a.hdr = reinterpret_cast<TreeHeader *>(w);
    a.tag = tag;
    a.rows = reinterpret_cast<TreeRow *>(w + p.off_rows);
    a.starts = reinterpret_cast<TreeStart *>(w + p.off_starts);
    a.joins = reinterpret_cast<TreeJoin *>(w + p.off_joins);
    a.group = s.group();
    a.head_dim = s.head_dim;
    a.join_warps = p.join_warps;
    a.join_blocks = p.join_blocks;
    a.nodes = reinterpret_cast<TreeNode *>(w + p.off_nodes);
    a.masks = reinterpret_cast<unsigned long long *>(w + p.off_masks);
    a.cost = reinterpret_cast<long long *>(w + p.off_cost);
    // as many heads side by side as leave no more than a 32nd of the CTAs without work (one always does)
    a.hi = s.num_kv_heads;
    while (s.num_kv_heads % a.hi || a.hi > s.sm_count || s.sm_count % a.hi * 32 > s.sm_count) --a.hi;
    return launch_pdl(dev::tree_plan_kernel, dim3(1 + (p.batch + dev::kPlanWarps - 1) / dev::kPlanWarps),
                      dim3(dev::kPlanThreads), 0, st, a);
}

cudaError_t launch_tree_accept(const Shape &s, const TreePlan &p, const TreeAccept &x, void *ws, cudaStream_t st) {
    if (p.batch == 0) return cudaSuccess;
    uint8_t *w = static_cast<uint8_t *>(ws);
    dev::AcceptArgs a;
    a.x = x;
    a.rows = reinterpret_cast<const TreeRow *>(w + p.off_rows);
    a.nodes = reinterpret_cast<const TreeNode *>(w + p.off_nodes);
    a.pages = p.pages;
    a.hdr = reinterpret_cast<TreeHeader *>(w);
    a.page_size = s.page_size;
    a.page_shift = s.page_shift();
    a.vecs = s.num_kv_heads * s.head_dim / 8;
    a.num_cache_pages = s.num_cache_pages;
    // a layer a CTA, more where the rows' CTAs would not all run at once
    const int most = std::max(1, dev::kAcceptCtas * s.sm_count / p.batch), chunks = std::max(1, std::min(x.layers, most));
    a.layers_per_cta = std::max(1, (x.layers + chunks - 1) / chunks);
    a.lanes = 2;
    while (a.lanes < 32 && a.vecs * 16 * 2 * a.lanes <= dev::kAcceptBytes / dev::kAcceptWarps) a.lanes *= 2;
    // the copies of a CTA are counted in 32 bits
    const int parts = (a.vecs * 16 + dev::kAcceptBuffer - 1) / dev::kAcceptBuffer;
    a.layers_per_cta = std::min(a.layers_per_cta, std::max(1, (1 << 30) / (kTreeMaxNew * 2 * parts)));
    const dim3 grid(p.batch, std::max(1, (x.layers + a.layers_per_cta - 1) / a.layers_per_cta));
    const size_t smem = dev::kAcceptBytes;
    auto launch = [&](auto kernel) {
        const cudaError_t e = set_smem_limit((const void *)kernel, smem, st);
        return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(dev::kAcceptThreads), smem, st, a);
    };
    return x.wide ? launch(dev::tree_accept_kernel<long long>) : launch(dev::tree_accept_kernel<int>);
}

}  // namespace pkv
