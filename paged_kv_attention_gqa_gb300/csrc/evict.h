// Plan structures and launchers of eviction by accumulated attention weight: the scores that decode
// steps and prompts add up per cache slot, and the selection and gather of the kept tokens.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>
#include <vector>

#include "plan.h"

namespace pkv {

constexpr int kWeightKeys = 128;       // keys of one work tile of the score kernels
constexpr int kWeightTeams = 3;        // thread groups of the weights kernel that take query blocks in turn
constexpr int kWeightsMinPage = 8;     // the K boxes of a WEIGHTS plan fill whole 8-row swizzle atoms
constexpr int kEvictTaskTokens = 32;   // kept tokens copied by one CTA of the gather
constexpr int kEvictMaxCluster = 8;    // CTAs that select one row's tokens

// 128 keys of one row whose scores are updated.
struct WeightsTile {
    int32_t kv_base;     // offset of the row's first page in the plan's page list
    int32_t length;      // L
    int32_t key0;        // first key
    int32_t new_begin;   // L - n: the row's new tokens, whose scores start from nothing
    int32_t q_begin;     // first query token
    int32_t n_q;         // n
    int32_t first;       // DECODE_WEIGHTS: first visible position; WEIGHTS: the tile's first part
    int32_t base;        // DECODE_WEIGHTS: the row's first logit, in units of 16 keys; WEIGHTS: its parts
};
static_assert(sizeof(WeightsTile) == 32, "WeightsTile is 8 ints");

// Work of one CTA at a time (WEIGHTS): kv heads [h0, h0 + nh) of a tile with the query tokens
// [i0, i1) of its row, in `blocks` blocks; with the tile's own numbers, so that one load tells all.
struct alignas(16) WeightsItem {
    int32_t kv_base, length, key0, new_begin;
    int32_t q_begin, h0, nh, blocks;
    int32_t i0, i1, part, pad;
};
static_assert(sizeof(WeightsItem) == 48, "WeightsItem is 12 ints");

struct WeightsPlan {
    size_t off_pages = 0, off_tiles = 0, off_items = 0, off_part = 0;  // in the workspace
    size_t off_logits = 0;      // decode: float[num_qo_heads][logit_stride]
    long long logit_stride = 0;
    int tiles = 0, items = 0;
    int box_tokens = 1;         // WEIGHTS: query tokens of one block
};

// One row of an eviction plan.
struct EvictRow {
    int32_t kv_base, length, keep;  // keep >= length: the row is left alone
    int32_t kept_base;              // offset of the row's kept positions in the output
    int32_t dst_base;               // offset of the row's first new page in the plan's list
    int32_t pad[3];
};
struct EvictTask {  // kept tokens [first, first + 32) of row `row`
    int32_t row, first;
};

struct EvictPlan {
    size_t off_pages = 0, off_dst = 0, off_rows = 0, off_tasks = 0, total = 0;
    int rows = 0, tasks = 0, kept = 0, num_sink = 0, num_recent = 0, longest = 0;
    std::vector<uint8_t> image;
};

// DECODE_WEIGHTS: a DECODE plan with the score tiles; WEIGHTS: the score tiles of a prefill-like step.
int make_weights_plan(const Shape &s, int mode, const int32_t *qo, const int32_t *kvp, const int32_t *kvi,
                      const int32_t *lpl, int batch, int causal, int window_left, float sm_scale, Plan &plan,
                      WeightsPlan &w, std::string &err);
int make_evict_plan(const Shape &s, const int32_t *kvp, const int32_t *kvi, const int32_t *lpl, int batch,
                    const int32_t *keep, int num_sink, int num_recent, const int32_t *dst_indptr,
                    const int32_t *dst_indices, EvictPlan &plan, std::string &err);
size_t evict_workspace_bound(const Shape &s, int mode);  // EVICT, DECODE_WEIGHTS, WEIGHTS

// scores[slot] = decay * scores[slot] (older tokens) or 0 (new ones) + the weights of the step.
cudaError_t launch_weights(const Shape &s, const Plan &p, const WeightsPlan &w, const CUtensorMap &tm_k,
                           const CUtensorMap &tm_q, void *ws, const float *lse, float *scores, float decay,
                           cudaStream_t st);
// The same from the logits that a decode of this plan left in the workspace.
cudaError_t launch_decode_scores(const Shape &s, const Plan &p, const WeightsPlan &w, void *ws, const float *lse,
                                 float *scores, float decay, cudaStream_t st);
// Decode pass of a DECODE_WEIGHTS plan: launch_decode that also stores its logits.
cudaError_t launch_decode_weights(const Shape &s, const Plan &p, const WeightsPlan &w, const CUtensorMap &tm, void *ws,
                                  const void *q, void *kv_layer, void *out, float *lse, cudaStream_t st);
cudaError_t launch_evict(const Shape &s, const EvictPlan &p, void *ws, void *kv_layer, float *scores, int32_t *kept,
                         cudaStream_t st);

}  // namespace pkv
