// Host planner of eviction by accumulated attention weight.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/pkv.h"
#include "evict.h"

namespace pkv {

static size_t put(size_t &at, size_t bytes) {
    const size_t here = at;
    at = align_up(at + bytes);
    return here;
}

// Every page of the plan once: a page's slots have one score each, so two rows that share a page
// would both update them.
static int distinct_pages(const Shape &s, const int32_t *kvi, int nnz, std::vector<uint8_t> &seen, std::string &err) {
    seen.assign(s.num_cache_pages, 0);
    for (int i = 0; i < nnz; ++i) {
        if (seen[kvi[i]]) {
            err = "page " + std::to_string(kvi[i]) + " is listed twice (at paged_kv_indices[" + std::to_string(i) +
                  "]): a slot has one score";
            return PKV_ERR_INVALID;
        }
        seen[kvi[i]] = 1;
    }
    return PKV_OK;
}

static int keys16(int L) { return (L + 15) / 16; }

// The (kv head, query block) pairs of the WEIGHTS tiles cut into items of about an eighth of an SM's
// share, longest first: a CTA per SM takes items round robin.  An item is a run of whole heads of one
// tile, or a run of blocks of one head where a head alone has more.
static void weight_items(const Shape &s, int causal, int window, int bt, std::vector<WeightsTile> &tiles,
                         std::vector<WeightsItem> &items) {
    struct Range {
        int i0, i1, nb;
    };
    std::vector<Range> ranges(tiles.size());
    long long total = 0;
    for (size_t t = 0; t < tiles.size(); ++t) {
        const WeightsTile &w = tiles[t];
        // the tokens that may see a key of the tile (token i sits at position new_begin + i)
        const int i0 = causal ? std::max(0, w.key0 - w.new_begin) : 0;
        const int i1 = window >= 0 ? (int)std::min<long long>(w.n_q, (long long)w.key0 + kWeightKeys + window - w.new_begin)
                                   : w.n_q;
        ranges[t] = Range{i0, std::max(i0, i1), i1 > i0 ? (i1 - i0 + bt - 1) / bt : 0};
        total += (long long)ranges[t].nb * s.num_kv_heads;
    }
    const int cap = (int)std::max<long long>(1, total / (8ll * std::max(1, s.sm_count)));
    items.clear();
    for (size_t t = 0; t < tiles.size(); ++t) {
        const Range &r = ranges[t];
        tiles[t].first = (int)items.size();
        auto add = [&](int h0, int nh, int a, int b) {
            const WeightsTile &w = tiles[t];
            items.push_back(WeightsItem{w.kv_base, w.length, w.key0, w.new_begin, w.q_begin, h0, nh, (b - a + bt - 1) / bt,
                                        a, b, (int)items.size(), 0});
        };
        if (r.nb > 0 && r.nb <= cap) {
            const int nh = std::min(s.num_kv_heads, cap / r.nb);
            for (int h = 0; h < s.num_kv_heads; h += nh) add(h, std::min(nh, s.num_kv_heads - h), r.i0, r.i1);
        } else if (r.nb > 0) {
            const int chunks = (r.nb + cap - 1) / cap, step = (r.nb + chunks - 1) / chunks * bt;
            for (int h = 0; h < s.num_kv_heads; ++h)
                for (int a = r.i0; a < r.i1; a += step) add(h, 1, a, std::min(r.i1, a + step));
        }
        tiles[t].base = (int)items.size() - tiles[t].first;
    }
    std::stable_sort(items.begin(), items.end(),
                     [](const WeightsItem &a, const WeightsItem &b) { return a.nh * a.blocks > b.nh * b.blocks; });
}

int make_weights_plan(const Shape &s, int mode, const int32_t *qo, const int32_t *kvp, const int32_t *kvi,
                      const int32_t *lpl, int batch, int causal, int window_left, float sm_scale, Plan &plan,
                      WeightsPlan &w, std::string &err) {
    const bool decode = mode == PKV_MODE_DECODE_WEIGHTS;
    if (s.graph_static) {
        err = "weights plans are not made on a graph_static handle";
        return PKV_ERR_UNSUPPORTED;
    }
    if (!decode && s.page_size < kWeightsMinPage) {
        err = "weights plans need pages of 8 slots or more";
        return PKV_ERR_UNSUPPORTED;
    }
    if (!decode && causal != 0 && causal != 1) {
        err = "weights plans are causal (1) or non-causal (0)";
        return PKV_ERR_INVALID;
    }
    int rc = decode ? make_plan(s, PKV_MODE_DECODE, qo, kvp, kvi, lpl, batch, 1, window_left, sm_scale, plan, err)
                    : validate_rows(s, PKV_MODE_PREFILL, qo, kvp, kvi, lpl, batch, window_left, err, causal);
    if (rc) return rc;
    std::vector<uint8_t> seen;
    if ((rc = distinct_pages(s, kvi, kvp[batch], seen, err))) return rc;
    const int P = s.page_size, nnz = kvp[batch];
    std::vector<WeightsTile> tiles;
    std::vector<int32_t> base(batch, 0);
    int at16 = 0, most = 1;
    for (int r = 0; r < batch; ++r) {
        const int np = kvp[r + 1] - kvp[r];
        const int L = np ? (np - 1) * P + lpl[r] : 0;
        const int n = decode ? 1 : qo[r + 1] - qo[r];
        base[r] = at16;
        at16 += keys16(L);
        most = std::max(most, n);
        const int lo = decode && window_left >= 0 ? std::max(0, L - 1 - window_left) : 0;
        for (int k = 0; k < L; k += kWeightKeys)
            tiles.push_back(WeightsTile{kvp[r], L, k, L - n, decode ? r : qo[r], n, lo, base[r]});
    }
    w = WeightsPlan();
    w.tiles = (int)tiles.size();
    if (decode) {
        // the score tiles join the image behind the decode plan's arrays; its partials move up
        DecodeTile *dt = reinterpret_cast<DecodeTile *>(plan.image.data() + plan.lay.dec_tiles);
        for (int i = 0; i < plan.dec_tiles; ++i) dt[i].logit_base = base[dt[i].q_token];
        w.off_pages = plan.lay.dec_pages;
        w.off_tiles = plan.lay.int_bytes;
        const size_t grow = align_up(tiles.size() * sizeof(WeightsTile));
        plan.image.resize(plan.lay.int_bytes + grow, 0);
        if (!tiles.empty()) std::memcpy(plan.image.data() + w.off_tiles, tiles.data(), tiles.size() * sizeof(WeightsTile));
        plan.lay.int_bytes += grow;
        plan.lay.part_o += grow;
        plan.lay.part_lse += grow;
        plan.lay.total += grow;
        w.logit_stride = 16ll * at16;
        w.off_logits = put(plan.lay.total, (size_t)w.logit_stride * s.num_qo_heads * 4);
        plan.mode = PKV_MODE_DECODE_WEIGHTS;
        return PKV_OK;
    }
    std::vector<uint8_t> image;
    image.swap(plan.image);
    plan = Plan();
    plan.mode = PKV_MODE_WEIGHTS;
    plan.batch = batch;
    plan.num_tokens = qo[batch];
    plan.causal = causal;
    plan.window_left = window_left;
    plan.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt((float)s.head_dim);
    w.box_tokens = std::min(kPrefillRowsPerTile / s.group(), most);
    std::vector<WeightsItem> items;
    weight_items(s, causal, window_left, w.box_tokens, tiles, items);
    w.items = (int)items.size();
    size_t at = kAlign;
    w.off_pages = put(at, (size_t)nnz * 4);
    w.off_tiles = put(at, tiles.size() * sizeof(WeightsTile));
    w.off_items = put(at, items.size() * sizeof(WeightsItem));
    plan.lay.int_bytes = at;
    w.off_part = put(at, items.size() * kWeightTeams * kWeightKeys * 4);  // one per item and team
    plan.lay.total = at;
    image.assign(plan.lay.int_bytes, 0);
    PlanHeader hdr{};
    hdr.causal = causal;
    hdr.window_left = window_left;
    hdr.scale_log2 = plan.sm_scale * 1.4426950408889634f;
    std::memcpy(image.data(), &hdr, sizeof hdr);
    if (nnz) std::memcpy(image.data() + w.off_pages, kvi, (size_t)nnz * 4);
    if (!tiles.empty()) std::memcpy(image.data() + w.off_tiles, tiles.data(), tiles.size() * sizeof(WeightsTile));
    if (!items.empty()) std::memcpy(image.data() + w.off_items, items.data(), items.size() * sizeof(WeightsItem));
    plan.image.swap(image);
    return PKV_OK;
}

int make_evict_plan(const Shape &s, const int32_t *kvp, const int32_t *kvi, const int32_t *lpl, int batch,
                    const int32_t *keep, int num_sink, int num_recent, const int32_t *dst_indptr,
                    const int32_t *dst_indices, EvictPlan &plan, std::string &err) {
    if (batch < 0 || batch > s.max_batch) {
        err = "batch " + std::to_string(batch) + " outside [0, max_batch=" + std::to_string(s.max_batch) + "]";
        return PKV_ERR_INVALID;
    }
    if (!keep || !dst_indptr) {
        err = "keep and dst_indptr are required";
        return PKV_ERR_INVALID;
    }
    if (num_sink < 0 || num_recent < 0) {
        err = "num_sink and num_recent must be >= 0";
        return PKV_ERR_INVALID;
    }
    const std::vector<int32_t> none((size_t)batch + 1, 0);  // no new tokens
    int rc = validate_rows(s, PKV_MODE_PREFILL, none.data(), kvp, kvi, lpl, batch, -1, err, 1);
    if (rc) return rc;
    const int P = s.page_size, nnz = kvp[batch];
    if ((long long)nnz * P >= (1ll << 31) - 64) {
        err = "the rows' pages hold more slots than 32-bit positions count";
        return PKV_ERR_INVALID;
    }
    if (dst_indptr[0] != 0) {
        err = "dst_indptr must start at 0";
        return PKV_ERR_INVALID;
    }
    std::vector<EvictRow> rows(batch);
    std::vector<EvictTask> tasks;
    int kept = 0, longest = 0;
    for (int r = 0; r < batch; ++r) {
        const int np = kvp[r + 1] - kvp[r], L = np ? (np - 1) * P + lpl[r] : 0;
        const bool cut = keep[r] < L;
        if (keep[r] < 0 || (cut && (long long)num_sink + num_recent > keep[r])) {
            err = "keep[" + std::to_string(r) + "]=" + std::to_string(keep[r]) +
                  " is below num_sink + num_recent (the tokens that stay whatever their score)";
            return PKV_ERR_INVALID;
        }
        const int want = cut ? (keep[r] + P - 1) / P : 0, got = dst_indptr[r + 1] - dst_indptr[r];
        if (got != want) {
            err = "row " + std::to_string(r) + " needs " + std::to_string(want) + " new pages, dst_indptr gives " +
                  std::to_string(got);
            return PKV_ERR_INVALID;
        }
        rows[r] = EvictRow{kvp[r], L, keep[r], kept, dst_indptr[r], {0, 0, 0}};
        kept += std::min(keep[r], L);
        longest = std::max(longest, cut ? L : 0);
        if (cut)
            for (int i = 0; i < keep[r]; i += kEvictTaskTokens) tasks.push_back(EvictTask{r, i});
    }
    const int nd = dst_indptr[batch];
    if (nd > 0 && !dst_indices) {
        err = "dst_indices is required";
        return PKV_ERR_INVALID;
    }
    if (nd > s.max_num_pages) {
        err = "dst_indices has " + std::to_string(nd) + " entries, above max_num_pages=" + std::to_string(s.max_num_pages);
        return PKV_ERR_INVALID;
    }
    // a new page is written while every row is still being read: it may be nobody's page, and nobody
    // else's new page
    std::vector<uint8_t> used(s.num_cache_pages, 0);
    for (int i = 0; i < nnz; ++i) used[kvi[i]] = 1;
    for (int i = 0; i < nd; ++i) {
        if (dst_indices[i] < 0 || dst_indices[i] >= s.num_cache_pages || used[dst_indices[i]]) {
            err = "dst_indices[" + std::to_string(i) + "]=" + std::to_string(dst_indices[i]) +
                  " is outside the cache, a page of a row, or listed twice";
            return PKV_ERR_INVALID;
        }
        used[dst_indices[i]] = 1;
    }
    plan.rows = batch;
    plan.tasks = (int)tasks.size();
    plan.kept = kept;
    plan.num_sink = num_sink;
    plan.num_recent = num_recent;
    plan.longest = longest;
    size_t at = kAlign;
    plan.off_pages = put(at, (size_t)nnz * 4);
    plan.off_dst = put(at, (size_t)nd * 4);
    plan.off_rows = put(at, rows.size() * sizeof(EvictRow));
    plan.off_tasks = put(at, tasks.size() * sizeof(EvictTask));
    plan.total = at;
    plan.image.assign(at, 0);
    auto cp = [&](size_t off, const void *src, size_t n) {
        if (n) std::memcpy(plan.image.data() + off, src, n);
    };
    cp(plan.off_pages, kvi, (size_t)nnz * 4);
    cp(plan.off_dst, dst_indices, (size_t)nd * 4);
    cp(plan.off_rows, rows.data(), rows.size() * sizeof(EvictRow));
    cp(plan.off_tasks, tasks.data(), tasks.size() * sizeof(EvictTask));
    return PKV_OK;
}

size_t evict_workspace_bound(const Shape &s, int mode) {
    const size_t P = s.page_size, nnz = s.max_num_pages, B = s.max_batch;
    if (mode == PKV_MODE_EVICT) {
        size_t at = kAlign;
        put(at, nnz * 4);
        put(at, nnz * 4);
        put(at, B * sizeof(EvictRow));
        put(at, (nnz * P / kEvictTaskTokens + B) * sizeof(EvictTask));
        return at;
    }
    const size_t tiles = nnz * P / kWeightKeys + B;
    if (mode == PKV_MODE_DECODE_WEIGHTS) {
        size_t at = workspace_bound(s, PKV_MODE_DECODE);
        put(at, tiles * sizeof(WeightsTile));
        put(at, (nnz * P + 16 * B) * s.num_qo_heads * 4);
        return at;
    }
    size_t at = kAlign;
    put(at, nnz * 4);
    put(at, tiles * sizeof(WeightsTile));
    // an item is at least half an eighth of an SM's share, but for the last one of each tile (and one
    // block of one head where the share is less)
    const size_t items = 16 * (size_t)std::max(1, s.sm_count) + 2 * tiles;
    put(at, items * sizeof(WeightsItem));
    put(at, items * kWeightTeams * kWeightKeys * 4);
    return at;
}

}  // namespace pkv
