// Host planner of latent attention: validation (shared with the other paged plans), KV write
// locations, the split of the key tiles over CTAs, and the workspace image.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/pkv.h"
#include "latent.h"

namespace pkv {

static Shape as_shape(const LatentShape &s) {
    Shape b{};
    b.num_qo_heads = b.num_kv_heads = s.num_heads;
    b.head_dim = 128;
    b.page_size = s.page_size;
    b.max_batch = s.max_batch;
    b.max_total_tokens = s.max_total_tokens;
    b.max_num_pages = s.max_num_pages;
    b.num_cache_pages = s.num_cache_pages;
    b.sm_count = s.sm_count;
    b.sink_page = -1;
    return b;
}

// What a piece of a unit costs beside its tiles, in tiles: its Q, the first S, and writing O, which the
// next piece's first PV waits for.  (48 rows of 128 heads: 82.8 us with 0, 78.7 with 2, 85.4 with 4, where
// CTAs that take no further piece leave too much to the others; a batch of 32 rows 41.2, 40.7, 41.0.)
static constexpr long long kPieceCost = 2;

namespace {
struct Unit {
    int q_row, n_rows, pos0, length, kv_base, tile0, ntiles;
};
}  // namespace

// A sequence's query rows f = token * H + head are cut into blocks of 64; (sequence, block) is a
// unit over the key tiles any of its rows sees.  The blocks of one index over all sequences form a
// lane; each lane gets CTAs in proportion to its tiles and is cut into equal runs of tiles and pieces.  With
// equal blocks per sequence (a step of one token each) the lanes are cut alike, so the CTAs that
// read the same keys for different heads do it at the same time and share them in L2.
static void split_units(const LatentShape &s, const std::vector<std::vector<Unit>> &lanes, std::vector<LatentTile> &tiles,
                        std::vector<int32_t> &cta_ptr, std::vector<LatentMerge> &merges, int &num_partials) {
    tiles.clear();
    cta_ptr.assign(1, 0);
    merges.clear();
    num_partials = 0;
    long long all = 0;
    std::vector<long long> w(lanes.size(), 0);
    for (size_t b = 0; b < lanes.size(); ++b) {
        for (const Unit &u : lanes[b]) w[b] += u.ntiles;
        all += w[b];
    }
    if (!all) return;
    const long long cmax = std::max(1, s.sm_count);
    const bool flat = (long long)lanes.size() * 2 > cmax;  // more blocks than CTAs to give them: one lane
    auto cut = [&](const std::vector<const Unit *> &us, long long total, long long ctas) {
        // a budget per CTA with which the run takes no more than `ctas` of them, found by growing the even
        // share step by step (by a quarter of what is missing: near the least one, not always at it).  A CTA
        // that has a piece takes no other one that its budget leaves no tile for
        auto count = [&](long long per) {
            long long n = 1, budget = per;
            for (const Unit *u : us)
                for (int used = 0; used < u->ntiles;) {
                    if (budget <= kPieceCost) {
                        ++n;
                        budget = per;
                    }
                    const int take = (int)std::min<long long>(budget - kPieceCost, u->ntiles - used);
                    used += take;
                    budget -= take + kPieceCost;
                }
            return n;
        };
        long long per = kPieceCost + std::max<long long>((total + ctas - 1) / ctas, 1);
        for (long long n; (n = count(per)) > ctas;) per += std::max<long long>(1, per * (n - ctas) / (4 * n));
        long long budget = per;
        for (const Unit *u : us) {
            int used = 0;
            const int first_tile = (int)tiles.size();
            while (used < u->ntiles) {
                if (budget <= kPieceCost) {
                    cta_ptr.push_back((int32_t)tiles.size());
                    budget = per;
                }
                const int take = (int)std::min<long long>(budget - kPieceCost, u->ntiles - used);
                tiles.push_back(LatentTile{u->q_row, u->n_rows, u->pos0, u->length, u->kv_base, u->tile0 + used, take, -1});
                used += take;
                budget -= take + kPieceCost;
            }
            const int pieces = (int)tiles.size() - first_tile;
            if (pieces > 1) {
                merges.push_back(LatentMerge{u->q_row, u->n_rows, num_partials, pieces});
                for (int i = 0; i < pieces; ++i) tiles[first_tile + i].partial = num_partials++;
            }
        }
        if ((int32_t)tiles.size() > cta_ptr.back()) cta_ptr.push_back((int32_t)tiles.size());
    };
    std::vector<const Unit *> us;
    if (flat) {
        size_t most = 0;
        for (const auto &l : lanes) most = std::max(most, l.size());
        // sequence by sequence, so that neighbouring CTAs read the same keys
        for (size_t i = 0; i < most; ++i)
            for (const auto &l : lanes)
                if (i < l.size()) us.push_back(&l[i]);
        cut(us, all, cmax);
        return;
    }
    long long left = cmax, rest = all;
    for (size_t b = 0; b < lanes.size(); ++b) {
        if (!w[b]) continue;
        us.clear();
        for (const Unit &u : lanes[b]) us.push_back(&u);
        // at least one CTA for this lane and one for each lane after it
        long long after = 0;
        for (size_t c = b + 1; c < lanes.size(); ++c) after += w[c] > 0;
        long long mine = rest > 0 ? left * w[b] / rest : 1;
        mine = std::max<long long>(1, std::min(mine, left - after));
        const size_t before = cta_ptr.size();
        cut(us, w[b], mine);
        left -= (long long)(cta_ptr.size() - before);
        left = std::max(left, after);
        rest -= w[b];
    }
}

static size_t put(size_t &at, size_t bytes) {
    const size_t here = at;
    at = align_up(at + bytes);
    return here;
}

static int check_scale(float sm_scale, std::string &err) {
    if (!(sm_scale > 0.f) || std::isinf(sm_scale)) {
        err = "sm_scale must be finite and > 0 (the width it comes from is not the cached one)";
        return PKV_ERR_INVALID;
    }
    return PKV_OK;
}

static constexpr double kLog2e = 1.4426950408889634;

int make_latent_plan(const LatentShape &s, const int32_t *qo, const int32_t *kvp, const int32_t *kvi,
                     const int32_t *lpl, int batch, int causal, int window_left, float sm_scale, LatentPlan &plan,
                     std::string &err) {
    const Shape b = as_shape(s);
    std::vector<int32_t> iota;
    if (!qo && batch >= 0 && batch <= s.max_batch) {
        iota.resize((size_t)batch + 1);
        for (int r = 0; r <= batch; ++r) iota[r] = r;
        qo = iota.data();
    }
    int rc = check_scale(sm_scale, err);
    if (rc) return rc;
    if (causal != 0 && causal != 1) {
        err = "causal is 0 or 1";
        return PKV_ERR_INVALID;
    }
    rc = validate_rows(b, PKV_MODE_PREFILL, qo, kvp, kvi, lpl, batch, window_left, err, causal);
    if (rc) return rc;
    const int H = s.num_heads, P = s.page_size, T = qo[batch], nnz = kvp[batch];
    std::vector<std::vector<Unit>> lanes;
    std::vector<int32_t> rows(T);
    int most_rows = 0;
    for (int r = 0; r < batch; ++r) {
        const int np = kvp[r + 1] - kvp[r];
        const int n = qo[r + 1] - qo[r];
        if (np == 0 || n == 0) continue;
        const int L = (np - 1) * P + lpl[r];
        for (int i = 0; i < n; ++i) {
            const int p = L - n + i;
            rows[qo[r] + i] = kvi[kvp[r] + p / P] * P + p % P;
        }
        const int total_rows = n * H;
        for (int f0 = 0, blk = 0; f0 < total_rows; f0 += kLatentRows, ++blk) {
            const int nr = std::min(kLatentRows, total_rows - f0);
            const int p_first = L - n + f0 / H, p_last = L - n + (f0 + nr - 1) / H;
            const int lo = window_left >= 0 ? std::max(0, p_first - window_left) : 0;
            const int hi = causal ? p_last : L - 1;  // last key any row of the block sees
            const int t0 = lo / kLatentKeys;
            if ((int)lanes.size() <= blk) lanes.resize(blk + 1);
            lanes[blk].push_back(Unit{qo[r] * H + f0, nr, L - n - qo[r], L, kvp[r], t0, hi / kLatentKeys - t0 + 1});
            most_rows = std::max(most_rows, nr);
        }
    }
    std::vector<LatentTile> tiles;
    std::vector<int32_t> cta;
    std::vector<LatentMerge> merges;
    int parts = 0;
    split_units(s, lanes, tiles, cta, merges, parts);
    plan.dense = false;
    plan.num_tokens = T;
    plan.num_append = T;
    plan.num_keys = 0;
    plan.causal = causal;
    plan.window_left = window_left;
    plan.box_q = std::max(8, (most_rows + 7) / 8 * 8);
    plan.ctas = tiles.empty() ? 0 : (int)cta.size() - 1;
    plan.num_partials = parts;
    plan.num_merge = (int)merges.size();
    plan.max_pieces = 0;
    for (const LatentMerge &m : merges) plan.max_pieces = std::max(plan.max_pieces, (int)m.count);
    plan.pf_tiles = 0;
    size_t at = kAlign;
    plan.off_append = put(at, rows.size() * 4);
    plan.off_pages = put(at, (size_t)nnz * 4);
    plan.off_tiles = put(at, tiles.size() * sizeof(LatentTile));
    plan.off_cta = put(at, cta.size() * 4);
    plan.off_merge = put(at, merges.size() * sizeof(LatentMerge));
    const size_t int_bytes = at;
    plan.off_part_o = put(at, (size_t)parts * kLatentRows * kLatentDim * 4);
    plan.off_part_lse = put(at, (size_t)parts * kLatentRows * 4);
    plan.total = at;
    plan.image.assign(int_bytes, 0);
    LatentHeader hd{0, causal, window_left, (float)((double)sm_scale * kLog2e)};
    std::memcpy(plan.image.data(), &hd, sizeof hd);
    auto cp = [&](size_t off, const void *src, size_t n) {
        if (n) std::memcpy(plan.image.data() + off, src, n);
    };
    cp(plan.off_append, rows.data(), rows.size() * 4);
    cp(plan.off_pages, kvi, (size_t)nnz * 4);
    cp(plan.off_tiles, tiles.data(), tiles.size() * sizeof(LatentTile));
    cp(plan.off_cta, cta.data(), cta.size() * 4);
    cp(plan.off_merge, merges.data(), merges.size() * sizeof(LatentMerge));
    return PKV_OK;
}

// Expanded form: the dense plan of a one-query-head-per-key-head shape (work tiles of two query
// tiles of 128 tokens of one head).
int make_latent_dense_plan(const LatentShape &s, const int32_t *cu_q, const int32_t *cu_k, int batch, int causal,
                           int window_left, float sm_scale, LatentPlan &plan, std::string &err) {
    int rc = check_scale(sm_scale, err);
    if (rc) return rc;
    Plan p;
    p.image.swap(plan.image);
    rc = make_dense_plan(as_shape(s), cu_q, cu_k, batch, causal, window_left, sm_scale, p, err);
    plan.image.swap(p.image);
    if (rc) return rc;
    plan.dense = true;
    plan.num_tokens = p.num_tokens;
    plan.num_keys = p.num_keys;
    plan.num_append = 0;
    plan.causal = causal;
    plan.window_left = window_left;
    plan.ctas = plan.num_partials = plan.num_merge = 0;
    plan.pf_tiles = p.pf_tiles;
    plan.dense_lay = p.lay;
    plan.total = p.lay.total;
    return PKV_OK;
}

size_t latent_workspace_bound(const LatentShape &s, bool dense) {
    if (dense) return workspace_bound(as_shape(s), PKV_MODE_DENSE);
    // a row block starts at most every 64 rows of a sequence, plus one ragged block per sequence
    const size_t H = s.num_heads, T = s.max_total_tokens, B = s.max_batch;
    const size_t units = std::min(T * ((H + kLatentRows - 1) / kLatentRows), (T * H) / kLatentRows + std::min(B, T));
    const size_t ctas = (size_t)std::max(1, s.sm_count);
    // each CTA's run cuts a unit at most at its two ends
    const size_t parts = 2 * ctas, pieces = units + ctas;
    size_t at = kAlign;
    put(at, T * 4);
    put(at, (size_t)s.max_num_pages * 4);
    put(at, pieces * sizeof(LatentTile));
    put(at, (ctas + 1) * 4);
    put(at, std::min(units, ctas) * sizeof(LatentMerge));
    put(at, parts * kLatentRows * kLatentDim * 4);
    put(at, parts * kLatentRows * 4);
    return at;
}

}  // namespace pkv
