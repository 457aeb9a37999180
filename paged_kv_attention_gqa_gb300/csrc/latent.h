// Plan structures and launchers of latent attention (pkv_latent_*): the absorbed form over a paged
// cache of one shared vector per token, and the expanded form over contiguous per-head keys and
// values with one rope key per token.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>
#include <vector>

#include "plan.h"

namespace pkv {

// The widths the kernels are compiled for.
constexpr int kLatentDim = 512;                      // the latent part: keys' first columns, and the values
constexpr int kLatentRope = 64;                      // the rope part of the keys
constexpr int kLatentWidth = kLatentDim + kLatentRope;
constexpr int kLatentNope = 128, kLatentV = 128;     // the expanded heads: key without rope, value
constexpr int kLatentRows = 64;                      // query rows (token, head) of one work unit
constexpr int kLatentKeys = 64;                      // keys of one tile
constexpr int kLatentMinPage = 8;                    // a TMA box fills whole 8-row swizzle atoms

struct LatentShape {
    int num_heads = 0, page_size = 0;
    int max_batch = 0, max_total_tokens = 0, max_num_pages = 0, num_cache_pages = 0;
    int sm_count = 0;
    int page_shift() const { return __builtin_ctz((unsigned)page_size); }
    // rows of one TMA box of the cache: a whole page up to one key tile; a box of a whole tile takes all
    // columns, a smaller one 64
    int box_rows() const { return page_size < kLatentKeys ? page_size : kLatentKeys; }
    int box_chunks() const { return page_size < kLatentKeys ? 1 : kLatentWidth / 64; }
};

// First bytes of a latent plan in the workspace.
struct LatentHeader {
    int32_t err;        // device error word (bounded waits that gave up)
    int32_t causal;
    int32_t window_left;
    float scale_log2;   // sm_scale * log2(e)
};

// One piece of a work unit handled by one CTA: `ntiles` key tiles of up to 64 consecutive query
// rows of one sequence.  Query rows are numbered over the whole step, row f = token * H + head.
struct LatentTile {
    int32_t q_row;    // first query row
    int32_t n_rows;   // 1..64
    int32_t pos0;     // row f sits at position pos0 + f / H
    int32_t length;   // L of the sequence
    int32_t kv_base;  // offset of the sequence's first page in the plan's page list
    int32_t tile0;    // first key tile (keys tile0 * kLatentKeys ..)
    int32_t ntiles;   // >= 1
    int32_t partial;  // split-KV partial slot, -1 = this piece is the whole unit
};
static_assert(sizeof(LatentTile) == 32, "LatentTile is 8 ints");

// A unit cut into several pieces: partials [first, first + count).
struct LatentMerge {
    int32_t q_row, n_rows, first, count;
};

struct LatentPlan {
    bool dense = false;
    int num_tokens = 0, num_keys = 0, num_append = 0;
    int causal = 1, window_left = -1;
    int box_q = 64;         // rows of one TMA box of q
    int ctas = 0, num_partials = 0, num_merge = 0, pf_tiles = 0;
    int max_pieces = 0;     // of the unit that is cut most
    size_t off_append = 0, off_pages = 0, off_tiles = 0, off_cta = 0, off_merge = 0, off_part_o = 0, off_part_lse = 0;
    size_t total = 0;
    PlanLayout dense_lay;   // dense plans: PlanHeader and PrefillTiles, as the other dense plans
    std::vector<uint8_t> image;
};

// Host planners (plain C++): 0 on success, else a pkv_status with `err` explaining it.
int make_latent_plan(const LatentShape &s, const int32_t *qo, const int32_t *kvp, const int32_t *kvi,
                     const int32_t *lpl, int batch, int causal, int window_left, float sm_scale, LatentPlan &plan,
                     std::string &err);
int make_latent_dense_plan(const LatentShape &s, const int32_t *cu_q, const int32_t *cu_k, int batch, int causal,
                           int window_left, float sm_scale, LatentPlan &plan, std::string &err);
size_t latent_workspace_bound(const LatentShape &s, bool dense);

// Launchers.  `tm_cache`: boxes of (64 columns, box_rows() rows, box_chunks() chunks) of the layer slice
// viewed as [9 chunks][pages * page_size][64] (chunks outermost, so that one chunk's rows land together);
// `tm_q`: boxes of (64 columns, box_q rows) of q viewed as [T * H][576].
cudaError_t launch_latent(const LatentShape &s, const LatentPlan &p, const CUtensorMap &tm_cache,
                          const CUtensorMap &tm_q, void *ws, void *out, float *lse, cudaStream_t st);
// Expanded form: boxes of 64 columns x 128 rows of q [H][T][192], and of 64 columns x 64 rows of
// k_nope [H][keys][128], k_rope [keys][64] and v [H][keys][128].
cudaError_t launch_latent_dense(const LatentShape &s, const LatentPlan &p, const CUtensorMap &tm_q,
                                const CUtensorMap &tm_k, const CUtensorMap &tm_r, const CUtensorMap &tm_v, void *ws,
                                void *out, float *lse, cudaStream_t st);
// Rows c_new[t] (512 values) and rope_new[t] (64 values), `*_stride` elements apart, into the slot of
// new token t.
cudaError_t launch_latent_append(const LatentShape &s, const LatentPlan &p, void *ws, const void *c_new,
                                 long long c_stride, const void *rope_new, long long rope_stride, void *cache,
                                 cudaStream_t st);

}  // namespace pkv
