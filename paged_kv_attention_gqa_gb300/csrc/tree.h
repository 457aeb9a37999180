// Plan structures and launchers of the speculative step: page and slot maps built on the GPU, attention of
// a tree of drafted tokens, acceptance of a path.  Its index arrays live on the device, so the plan is
// made there too.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "plan.h"

namespace pkv {

constexpr int kTreeKeys = 64;        // keys of one tile
constexpr int kTreeMaxNew = 256;     // most drafted tokens of a row
constexpr int kTreeMinPage = 8;      // a TMA box fills whole 8-row swizzle atoms
// What the plan shares out, in thirds of a tile: a tile with two query tiles, or the only one, 3; a pair's unit
// that reaches into one of its query tiles alone 2 a tile (it is bound by its copies, the others by the MMAs too);
// a piece as much as two tiles beside its own; and a CTA takes no less than four tiles' worth.  Where units stay whole
// it takes no less than the smallest unit, so that none has two while others have none (11 rows of 35 drafted
// tokens 12.6 us with the other bound, 9.1 with this one).
constexpr int kTreeTileCost = 3, kTreeHalfCost = 2, kTreePieceCost = 6, kTreeLeastCost = 12;
constexpr int kTreeLeastWhole = kTreePieceCost + kTreeHalfCost;
static_assert(kTreeLeastCost > kTreePieceCost + kTreeTileCost, "the CTAs' first tiles are all different");
// Steps leave units whole if their page list holds no more than eight tiles a row (four at head_dim 256, whose tiles take
// twice as long), of at most four rows, since one row may have all of them: the join of cut units is a kernel
// more, 2 us, in which a CTA goes through eight tiles.  (Steps of one to 63 short rows 6.8 to 16.2 us cut,
// 5.6 to 13.2 whole; one row of 517 tokens 9.5 cut, 10.5 whole.)
// So do steps of up to two units a CTA whose window leaves each so few tiles, whatever the page list holds (40 windowed
// steps 10.8 us in the mean cut, 10.4 with one unit a CTA at most, 10.3 with two; 33 rows of 4 heads under a window of
// 127 tokens 12.3 and 8.2, but one row of 198 drafted tokens 10.4 and 12.0).
constexpr int kTreeWholeTiles = 8, kTreeWholeRows = 4, kTreeWholeUnits = 2;
constexpr int kMapsMaxRows = 8192;   // rows whose offsets fit the shared memory of the maps kernel

// Device error words of the speculative step (beside those of the bounded waits in ptx.cuh).
enum TreeError : int { kErrTreeRow = 5, kErrTreePage = 6, kErrTreeParent = 7 };

// Errors outlive the plans behind them: a step that is replayed without the host would otherwise lose all but the
// last one's.  `tag` tells a word that this handle's plans have begun from whatever else the memory held.
struct alignas(8) TreeHeader {
    int32_t err;  // the device error word: the first error since it was read
    uint32_t tag;
};
static_assert(sizeof(TreeHeader) == 8, "changed as one 64-bit word");

// One row as the plan read it.  A row without drafted tokens, or an inconsistent one, has n = nq = 0.
struct alignas(16) TreeRow {
    int32_t q_begin;  // its first token
    int32_t n;        // drafted tokens
    int32_t ctx;      // cached tokens (-1: inconsistent row)
    int32_t kv_base;  // offset of its first page in the page list
    int32_t kt0;      // first key tile (keys 64 * kt0 ..; after 0 under a window)
    int32_t nc;       // tiles of cached keys
    int32_t nq;       // units per kv head: query tiles (or pairs of them)
    int32_t pad;
};
static_assert(sizeof(TreeRow) == 32, "TreeRow is 8 ints");

// What a CTA does: the tiles from (r, unit, tile) up to (r_end, unit_end, tile_end).  CTA b is in lane b % hi of the
// grid, whose units of a row are the kv heads h0, h0 + hi, .. with their query units (inner).  The lanes go through
// the rows side by side, so that CTAs which read other heads of the same pages do so at the same time (a batch of 32
// rows 105.5 -> 100.5 us, wide trees 199.8 -> 185.6, when that was the only difference).
struct alignas(16) TreeStart {
    TreeRow row;  // row r
    int32_t r, unit, tile;
    int32_t r_end, unit_end, tile_end;
    int32_t h0, hi;
    int32_t pad[4];
};
static_assert(sizeof(TreeStart) == 80, "TreeStart is 80 bytes");

// A block's part of the join of a cut unit: 2^groups groups of 16 columns from group0 on, and of every 32 rows (or 16 or
// 8, if the unit has no more) `rows` from row0 on.  Its warps and what places they have beside that take the
// pieces in turn.
struct alignas(16) TreeJoin {
    int32_t token, tokens, kvh;  // the unit's first token in q, their number, its kv head
    int32_t cta, step, count;    // its pieces: of CTAs cta, cta + step, .. (count 0: nothing to do)
    int16_t group0, groups, row0, rows;
};
static_assert(sizeof(TreeJoin) == 32, "two vectors");
constexpr int kJoinBatch = 2;  // pieces of a thread on their way at once
PKV_HOST_DEVICE int tree_join_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }
// The part of a block for a unit of `count` pieces: as much as leaves all pieces on their way at once, columns before
// rows (one row of 130,000 tokens among 99 of 500, 8 heads on one of 128: 50 us where every unit of a step has the same
// number of warps, 24 so; 60,000 among 39, 64 query rows a head of 64: 23.8 by columns alone, 16.3).  A unit so has no more blocks (a multiple of 32 rows each) than cuts, twice as many at head_dim 256, which bounds
// them by the CTAs.
struct TreeJoinPart {
    int groups, rows;
};
PKV_HOST_DEVICE TreeJoinPart tree_join_part(int head_dim, int warps, int rows, int count) {
    TreeJoinPart p{2, tree_join_rows(rows)};
    while (16 << (p.groups + 1) <= head_dim && 2 << p.groups <= warps) ++p.groups;
    int room = (warps >> p.groups) * (32 / p.rows) * kJoinBatch;
    for (; room < count && (p.groups > 0 || p.rows > 8); room *= 2) {
        if (p.groups > 0)
            --p.groups;
        else
            p.rows /= 2;
    }
    return p;
}

struct TreeNode {
    int32_t parent, depth;
};

// Tiles of unit q of a row: of the cached keys, and behind them of the drafted ones up to its last token's.
PKV_HOST_DEVICE int tree_unit_tiles(const TreeRow &t, int q, int unit_tokens) {
    const int end = (q + 1) * unit_tokens;
    return t.nc + ((end < t.n ? end : t.n) + kTreeKeys - 1) / kTreeKeys;
}

struct TreePlan {
    int batch = 0, num_tokens = 0, max_new = 0, words = 0;  // words: 64-bit words of a node's mask
    int window_left = -1;
    float scale_log2 = 0.f;
    bool pair = false;                     // two query tiles of 128 rows per unit
    bool whole = false;                    // no unit is cut
    int part_rows = 0;                     // rows of a partial
    int join_warps = 0, join_blocks = 0, join_rows = 0;  // of the join: a block's warps, most records, blocks of a record
    const int32_t *pages = nullptr;        // the caller's page list (device)
    size_t off_rows = 0, off_starts = 0, off_joins = 0, off_nodes = 0, off_masks = 0, off_cost = 0, off_part_o = 0,
           off_part_lse = 0, total = 0;
};

// Query tokens of one 128-row tile.
inline int tree_tile_tokens(const Shape &s) { return 128 / s.group(); }
// The workspace of a step of `batch` rows, `tokens` tokens and up to `max_new` a row.
void tree_layout(const Shape &s, int batch, int tokens, int max_new, int num_indices, int window_left, TreePlan &p);

struct TreeIndex {  // device arrays
    const int32_t *qo, *kvp, *kvi, *last, *parents;
    int num_indices;
    int32_t *positions;
};
cudaError_t launch_tree_plan(const Shape &s, const TreePlan &p, const TreeIndex &x, uint32_t tag, void *ws, cudaStream_t st);
// `tm_kv`: boxes of 64 columns x min(page_size, 64) slots of the layer slice; `tm_k`, `tm_v`: of 64 columns x
// box_new rows of the new keys and values; `tm_q`: of 64 columns x the group's heads x box_q tokens.
cudaError_t launch_tree(const Shape &s, const TreePlan &p, const CUtensorMap &tm_kv, const CUtensorMap &tm_k,
                        const CUtensorMap &tm_v, const CUtensorMap &tm_q, int box_new, int box_q, void *ws, void *out,
                        float *lse, cudaStream_t st);

// Raise the shared-memory limits of every kernel that a tree step of this head_dim may choose.
cudaError_t prepare_tree(const Shape &s, cudaStream_t st);

struct TreeAccept {
    const void *draft, *target;
    int wide;  // the tokens are 64-bit
    const void *k, *v;
    long long k_layer, k_token, v_layer, v_token;  // strides in elements
    void *cache;
    long long cache_layer;
    int layers;
    int32_t *accepted, *count;
    void *next;
    int32_t *seq;
};
cudaError_t launch_tree_accept(const Shape &s, const TreePlan &p, const TreeAccept &x, void *ws, cudaStream_t st);

struct MapsArgs {
    const int32_t *seq, *fresh, *held, *free_count;
    int32_t *table, *free_pages;
    long long table_stride;
    int rows, max_blocks, free_capacity, indices_capacity, token_capacity, page_shift;
    int32_t *held_out, *free_count_out, *qo, *kvp, *kvi, *last, *slots, *positions, *status;
};
cudaError_t launch_maps(const MapsArgs &a, cudaStream_t st);
cudaError_t prepare_maps(cudaStream_t st);  // as prepare_tree

}  // namespace pkv
