"""Measured cases of the operators that keep a paged KV cache small.

Two families, both over the paged cache of this package:

* latent attention: every token keeps one shared vector [latent | rope] instead of K and V rows per
  head.  "latent" is the absorbed form of a serving step (the step's new vectors are appended to
  their pages, then every head's query attends to the vectors themselves); "expanded" is the form
  for prompts (per-head keys and values made from the latent vectors, one rope key for all heads).
* eviction by accumulated attention weight: "decode_weights" is a decode step that also adds every
  key's softmax weight, summed over the query heads, into a score per cache slot; "weights" does
  that for several query tokens per row (a prompt, or its last tokens) from their lse; "evict"
  keeps the best-scored tokens of each row and gathers them into fresh pages.

Plain forms are elementary torch operations in 32 bits on padded batches; exact() computes the same
per row in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128  # widths of the latent cache and of the expanded heads
SCALE_LATENT = 1.0 / math.sqrt(NOPE + ROPE)


def listed():
    return [
        # one sequence answering alone, its heads split over 8 GPUs: latency
        dict(name="latent, one row", op="latent", rows=1, heads=16, new=1, shortest=517, longest=517, page=64),
        # an ordinary serving batch of the same share of heads
        dict(name="latent, batch of 32", op="latent", rows=32, heads=16, new=1, shortest=203, longest=8190, page=64),
        # all 128 heads on one GPU, small pages
        dict(name="latent, 128 heads", op="latent", rows=48, heads=128, new=1, shortest=611, longest=6151, page=16),
        # few long documents, three draft tokens each, an odd head count
        dict(name="latent, long, 3 tokens", op="latent", rows=4, heads=20, new=3, shortest=30011, longest=65521, page=64),
        # a short prompt alone
        dict(name="expanded, short", op="expanded", rows=1, heads=16, new=137, shortest=137, longest=137),
        # a prefill step of ragged prompts
        dict(name="expanded, ragged", op="expanded", rows=4, heads=32, new=0, shortest=801, longest=4093),
        # one conversation whose cache is under a budget
        dict(name="decode+weights, one row", op="decode_weights", rows=1, heads=32, kv_heads=8, dim=128, shortest=1001,
             longest=1001, page=16, decay=1.0),
        # a serving batch of such conversations
        dict(name="decode+weights, batch", op="decode_weights", rows=64, heads=32, kv_heads=8, dim=128, shortest=517,
             longest=8170, page=16, decay=0.97),
        # the last 32 tokens of long prompts judge the prompts before they are cut down
        dict(name="weights, last 32 tokens", op="weights", rows=8, heads=32, kv_heads=8, dim=128, new=32, shortest=1999,
             longest=16381, page=16, decay=0.0),
        # two whole prompts
        dict(name="weights, whole prompts", op="weights", rows=2, heads=32, kv_heads=8, dim=128, new=2003, shortest=2003,
             longest=2003, page=16, decay=0.0),
        # one conversation over its budget
        dict(name="evict, one row", op="evict", rows=1, kv_heads=8, dim=128, shortest=2111, longest=2111, keep=1024,
             sink=4, recent=64, page=16),
        # long prompts cut down after prefill
        dict(name="evict, batch", op="evict", rows=16, kv_heads=8, dim=128, shortest=4321, longest=16345, keep=4096,
             sink=4, recent=256, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["latent", "expanded", "decode_weights", "weights", "evict"])
    if op == "latent":
        rows, heads, new = _log(rng, 1, 64), rng.choice([1, 8, 16, 20, 32, 64, 96, 128]), rng.choice([1, 1, 1, 2, 3, 5])
        most = max(64, min(65521, 20_000_000 // (rows * max(heads, 16) * new)))
        longest = _log(rng, max(8, new), most)
        return dict(op=op, rows=rows, heads=heads, new=new, shortest=max(new, longest // rng.randint(1, 9)), longest=longest,
                    page=rng.choice([8, 16, 32, 64, 128]))
    if op == "expanded":
        rows, heads = rng.randint(1, 4), rng.choice([1, 4, 16, 20, 32])
        longest = _log(rng, 1, 4000)
        new = rng.choice([0, 0, min(longest, _log(rng, 1, 512))])
        return dict(op=op, rows=rows, heads=heads, new=new, shortest=max(new, 1, longest // rng.randint(1, 6)),
                    longest=longest)
    if op == "evict":
        rows, kv_heads, dim = _log(rng, 1, 16), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        longest = _log(rng, 40, 16000)
        sink, recent = rng.choice([0, 1, 4]), rng.randint(0, 30)
        return dict(op=op, rows=rows, kv_heads=kv_heads, dim=dim, shortest=max(1, longest // rng.randint(1, 9)),
                    longest=longest, keep=rng.randint(sink + recent + 1, longest - 1), sink=sink, recent=recent,
                    page=rng.choice([1, 8, 16, 32, 64]))
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
    heads, page = kv_heads * rng.choice([1, 2, 4, 5, 8]), rng.choice([8, 16, 32, 64])
    decay = rng.choice([0.0, 0.9, 1.0])
    if op == "decode_weights":
        rows = _log(rng, 1, 64)
        longest = _log(rng, 2, min(8000, 8000 * 1024 // (kv_heads * dim)))
        return dict(op=op, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim, page=page, decay=decay,
                    shortest=max(1, longest // rng.randint(1, 9)), longest=longest)
    rows, new = _log(rng, 1, 8), _log(rng, 1, 200)
    longest = _log(rng, new, 4000)
    return dict(op=op, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim, page=page, decay=decay, new=new,
                shortest=max(new, longest // rng.randint(1, 9)), longest=longest)


def _lens(c):
    """Row lengths from the longest to the shortest, evenly apart; they do not depend on the seed."""
    n = c["rows"]
    return [c["longest"] - (c["longest"] - c["shortest"]) * i // max(1, n - 1) for i in range(n)]


def work(c):
    lens = _lens(c)
    tokens = sum(lens)
    if c["op"] == "latent":
        H, n, W = c["heads"], c["new"], LATENT + ROPE
        T = n * len(lens)
        # the cached vectors and the new ones, q; the appended vectors, out and lse
        b = (tokens - T) * W * 2 + T * W * 2 + T * H * W * 2 + T * W * 2 + T * H * LATENT * 2 + T * H * 4
        seen = sum(n * L - n * (n - 1) // 2 for L in lens)
        return {"bytes": b, "flops": 2.0 * seen * H * (W + LATENT)}
    if c["op"] == "expanded":
        H = c["heads"]
        T = sum(c["new"] or L for L in lens)
        b = T * H * (NOPE + ROPE) * 2 + tokens * (H * (NOPE + VDIM) + ROPE) * 2 + T * H * (VDIM * 2 + 4)
        seen = sum(n * L - n * (n - 1) // 2 for n, L in ((c["new"] or L, L) for L in lens))
        return {"bytes": b, "flops": 2.0 * seen * H * (NOPE + ROPE + VDIM)}
    if c["op"] == "evict":
        moved = sum(min(c["keep"], L) for L in lens if L > c["keep"])
        kept = sum(min(c["keep"], L) for L in lens)
        judged = sum(L for L in lens if L > c["keep"])
        return {"bytes": judged * 4 + moved * (2 * 2 * c["kv_heads"] * c["dim"] * 2 + 4) + kept * 4, "flops": 0.0}
    H, Hkv, D = c["heads"], c["kv_heads"], c["dim"]
    n = c.get("new", 1)
    T = n * len(lens)
    old = 4 * (tokens - T) if c["decay"] else 0
    seen = sum(n * L - n * (n - 1) // 2 for L in lens)
    if c["op"] == "decode_weights":
        return {"bytes": tokens * Hkv * D * 4 + 2 * T * H * D * 2 + T * H * 4 + tokens * 4 + old,
                "flops": 4.0 * seen * H * D}
    return {"bytes": tokens * Hkv * D * 2 + T * H * D * 2 + T * H * 4 + tokens * 4 + old, "flops": 2.0 * seen * H * D}


def _paged(c, g, spare=0):
    """Page lists of the rows over a shuffled pool: host index arrays, and on the GPU the pool row of
    every (row, position) of a padded batch with the mask of the positions that exist."""
    P, lens = c["page"], _lens(c)
    pages = [-(-L // P) for L in lens]
    total = sum(pages) + spare + 3
    order = torch.randperm(total, generator=g)
    indptr = [0]
    for n in pages:
        indptr.append(indptr[-1] + n)
    ids = order[: indptr[-1]]
    most = max(lens)
    pos = torch.arange(most)
    at = torch.tensor(indptr[:-1])[:, None] + (pos // P)[None]
    L = torch.tensor(lens)
    valid = pos[None] < L[:, None]
    slot = torch.where(valid, ids[at.clamp(max=max(indptr[-1] - 1, 0))] * P + (pos % P)[None], 0)
    return dict(P=P, lens=L.to(DEV), valid=valid.to(DEV), slot=slot.to(DEV), pos=pos.to(DEV), pages=total,
                kv_indptr=torch.tensor(indptr, dtype=torch.int32).numpy(), kv_indices=ids.to(torch.int32).numpy(),
                last=torch.tensor([(n - 1) % P + 1 for n in lens], dtype=torch.int32).numpy(),
                free=order[indptr[-1]:])


def _workspace(h, *mode):
    return torch.empty(h.workspace_size(*mode), dtype=torch.uint8, device=DEV)


def prepare(c, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gd, device=DEV, dtype=torch.float32).to(dtype)

    s = {"c": c, "op": c["op"]}
    lens, rows = _lens(c), c["rows"]
    if own:
        from paged_kv_attention_gqa_gb300 import binding as B

    if c["op"] == "expanded":
        H = c["heads"]
        nq = [c["new"] or L for L in lens]
        cu_q = torch.tensor([0] + nq).cumsum(0)
        cu_k = torch.tensor([0] + lens).cumsum(0)
        T, K = int(cu_q[-1]), int(cu_k[-1])
        # keys and values of a prompt come out of one projection of the latent vectors, side by side
        kv = randn(K, H, NOPE + VDIM)
        s.update(q=randn(T, H, NOPE + ROPE), k_nope=kv[..., :NOPE], v=kv[..., NOPE:], k_rope=randn(K, ROPE),
                 out=torch.empty(T, H, VDIM, device=DEV, dtype=torch.bfloat16), lse=torch.empty(T, H, device=DEV))
        i, j = torch.arange(max(nq), device=DEV), torch.arange(max(lens), device=DEV)
        s.update(cu_q=cu_q.to(DEV), cu_k=cu_k.to(DEV), i=i, j=j)
        if own:
            h = B.LatentHandle(num_heads=H, page_size=64, max_batch=rows, max_total_tokens=T, max_num_pages=1, num_cache_pages=1)
            s.update(h=h, ws=_workspace(h, B.MODE_DENSE))
            h.plan_dense(cu_q.numpy(), cu_k.numpy(), workspace=s["ws"], causal=True, sm_scale=SCALE_LATENT)
        return s

    if c["op"] == "evict":
        P = c["page"]
        fresh = [-(-c["keep"] // P) if L > c["keep"] else 0 for L in lens]
        p = _paged(c, g, spare=sum(fresh))
        Hkv, D = c["kv_heads"], c["dim"]
        dst_indptr = torch.tensor([0] + fresh).cumsum(0)
        dst = p["free"][: sum(fresh)]
        # accumulated weights of a long conversation: a few heavy tokens, many near nothing, some never seen
        scores = torch.rand(p["pages"], P, generator=gd, device=DEV).pow(8) * 4.0
        scores[scores < 1e-6] = 0.0
        # where kept token i of row r goes: its slot in the row's fresh pages
        k = torch.arange(c["keep"])
        at = (dst_indptr[:-1][:, None] + (k // P)[None]).clamp(max=max(sum(fresh) - 1, 0))
        dst_slot = (dst[at] * P + (k % P)[None]) if sum(fresh) else torch.zeros(rows, c["keep"], dtype=torch.long)
        s.update(p=p, kv=randn(p["pages"], 2, P, Hkv, D), scores=scores, dst_slot=dst_slot.to(DEV))
        if own:
            h = B.Handle(num_qo_heads=Hkv, num_kv_heads=Hkv, head_dim=D, page_size=P, max_batch=rows,
                         max_num_pages=len(p["kv_indices"]), num_cache_pages=p["pages"])
            s.update(h=h, ws=_workspace(h, B.MODE_EVICT),
                     kept=torch.empty(sum(min(c["keep"], L) for L in lens), dtype=torch.int32, device=DEV))
            h.plan_evict(p["kv_indptr"], p["kv_indices"], p["last"], [c["keep"]] * rows, dst_indptr.numpy(),
                         dst.numpy(), num_sink=c["sink"], num_recent=c["recent"], workspace=s["ws"])
        return s

    p = _paged(c, g)
    n = c.get("new", 1)
    qo = [n * r for r in range(rows + 1)]
    s["p"] = p
    if c["op"] == "latent":
        H = c["heads"]
        s.update(cache=randn(p["pages"], p["P"], LATENT + ROPE), q=randn(rows * n, H, LATENT + ROPE),
                 c_new=randn(rows * n, LATENT), r_new=randn(rows * n, ROPE),
                 out=torch.empty(rows * n, H, LATENT, device=DEV, dtype=torch.bfloat16),
                 lse=torch.empty(rows * n, H, device=DEV))
        if own:
            h = B.LatentHandle(num_heads=H, page_size=p["P"], max_batch=rows, max_total_tokens=rows * n,
                               max_num_pages=len(p["kv_indices"]), num_cache_pages=p["pages"])
            s.update(h=h, ws=_workspace(h, B.MODE_PREFILL))
            h.plan(qo, p["kv_indptr"], p["kv_indices"], p["last"], workspace=s["ws"], sm_scale=SCALE_LATENT)
        return s

    H, Hkv, D = c["heads"], c["kv_heads"], c["dim"]
    s.update(kv=randn(p["pages"], 2, p["P"], Hkv, D), q=(1.5 * randn(rows * n, H, D, dtype=torch.float32)).to(torch.bfloat16),
             scores=torch.rand(p["pages"], p["P"], generator=gd, device=DEV), scale=1.0 / math.sqrt(D))
    if c["op"] == "decode_weights":
        s.update(out=torch.empty(rows, H, D, device=DEV, dtype=torch.bfloat16), lse=torch.empty(rows, H, device=DEV))
    else:
        k = _gather(s["kv"][:, 0].reshape(-1, Hkv * D), p)
        s["lse"] = _logits(s, k, n).logsumexp(-1).transpose(1, 2).reshape(rows * n, H).contiguous()
    if own:
        mode = B.MODE_DECODE_WEIGHTS if c["op"] == "decode_weights" else B.MODE_WEIGHTS
        h = B.Handle(num_qo_heads=H, num_kv_heads=Hkv, head_dim=D, page_size=p["P"], max_batch=rows,
                     max_total_tokens=rows * n, max_num_pages=len(p["kv_indices"]), num_cache_pages=p["pages"])
        s.update(h=h, ws=_workspace(h, mode))
        h.plan(mode, None if c["op"] == "decode_weights" else qo, p["kv_indptr"], p["kv_indices"], p["last"],
               workspace=s["ws"], sm_scale=s["scale"])
    return s


def _gather(rows_of_pool, p):
    """[rows, positions, width] in 32 bits; positions that do not exist are zero."""
    x = rows_of_pool[p["slot"]].float()
    return x.masked_fill_(~p["valid"][..., None], 0.0)


def _sees(p, n):
    """[rows, n, positions]: query token i of a row sits at position L - n + i and sees what is not after it."""
    at = p["lens"][:, None] - n + torch.arange(n, device=DEV)[None]
    return p["pos"][None, None] <= at[..., None]


def _logits(s, k, n):
    """[rows, heads, n, positions] of the grouped-query heads, -inf where a query does not see."""
    c, p = s["c"], s["p"]
    R, H, Hkv, D = c["rows"], c["heads"], c["kv_heads"], c["dim"]
    g = H // Hkv
    q = s["q"].float().view(R, n, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(R * Hkv, g * n, D)
    k = k.view(R, -1, Hkv, D).permute(0, 2, 3, 1).reshape(R * Hkv, D, -1)
    x = torch.bmm(q, k).view(R, Hkv * g, n, -1) * s["scale"]
    return x.masked_fill(~_sees(p, n)[:, None], -math.inf)


def _add_scores(s, w, n):
    """Every position's weight into its slot: the row's new tokens start from nothing."""
    p, decay = s["p"], s["c"]["decay"]
    flat = s["scores"].view(-1)
    old = flat[p["slot"]] * decay if decay else torch.zeros_like(w)
    old = torch.where(p["pos"][None] < p["lens"][:, None] - n, old, 0.0)
    flat[p["slot"][p["valid"]]] = (old + w)[p["valid"]]


def _plain_latent(s):
    c, p = s["c"], s["p"]
    R, H, n, W = c["rows"], c["heads"], c["new"], LATENT + ROPE
    pool = s["cache"].view(-1, W)
    new = (p["lens"][:, None] - n + torch.arange(n, device=DEV)[None]).view(R, n)
    pool[p["slot"].gather(1, new).view(-1)] = torch.cat([s["c_new"], s["r_new"]], -1)
    k = _gather(pool, p)
    x = torch.bmm(s["q"].float().view(R, n * H, W), k.transpose(1, 2)) * SCALE_LATENT
    x = x.view(R, n, H, -1).masked_fill(~_sees(p, n)[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    t = e.sum(-1, keepdim=True)
    o = torch.bmm(e.view(R, n * H, -1), k[..., :LATENT]).view(R, n, H, LATENT) / t
    return o.reshape(R * n, H, LATENT).to(torch.bfloat16), (m + t.log()).view(R * n, H), s["cache"]


def _plain_expanded(s):
    cu_q, cu_k, i, j = s["cu_q"], s["cu_k"], s["i"], s["j"]
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    in_q, in_k = i[None] < nq[:, None], j[None] < nk[:, None]
    at_q = torch.where(in_q, cu_q[:-1, None] + i[None], 0)
    at_k = torch.where(in_k, cu_k[:-1, None] + j[None], 0)
    H = s["q"].shape[1]
    q = s["q"].float()[at_q].transpose(1, 2)
    k = torch.cat([s["k_nope"].float(), s["k_rope"].float()[:, None].expand(-1, H, -1)], -1)[at_k].permute(0, 2, 3, 1)
    x = torch.matmul(q, k) * SCALE_LATENT
    at = (nk - nq)[:, None] + i[None]
    sees = (j[None, None] <= at[..., None]) & in_k[:, None]
    x = x.masked_fill(~sees[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    t = e.sum(-1, keepdim=True)
    o = torch.matmul(e, s["v"].float()[at_k].transpose(1, 2)) / t
    return o.transpose(1, 2)[in_q].to(torch.bfloat16), (m + t.log())[..., 0].transpose(1, 2)[in_q]


def _plain_decode_weights(s):
    c, p = s["c"], s["p"]
    R, H, Hkv, D = c["rows"], c["heads"], c["kv_heads"], c["dim"]
    x = _logits(s, _gather(s["kv"][:, 0].reshape(-1, Hkv * D), p), 1)[:, :, 0]
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    t = e.sum(-1, keepdim=True)
    v = _gather(s["kv"][:, 1].reshape(-1, Hkv * D), p).view(R, -1, Hkv, D).transpose(1, 2)
    o = torch.matmul(e.view(R, Hkv, H // Hkv, -1), v).view(R, H, D) / t
    _add_scores(s, (e / t).sum(1), 1)
    return o.to(torch.bfloat16), (m + t.log())[..., 0], s["scores"]


def _plain_weights(s):
    c, p = s["c"], s["p"]
    R, H, n = c["rows"], c["heads"], c["new"]
    k = _gather(s["kv"][:, 0].reshape(-1, c["kv_heads"] * c["dim"]), p)
    x = _logits(s, k, n) - s["lse"].view(R, n, H).transpose(1, 2)[..., None]
    _add_scores(s, x.exp().sum((1, 2)), n)
    return s["scores"]


def _plain_evict(s):
    c, p = s["c"], s["p"]
    keep, pos, lens, valid = c["keep"], p["pos"][None], p["lens"][:, None], p["valid"]
    flat = s["scores"].view(-1)
    forced = (pos < c["sink"]) | (pos >= lens - c["recent"]) | (lens <= keep)
    key = torch.where(forced, math.inf, flat[p["slot"]]).masked_fill(~valid, -math.inf)
    order = key.sort(dim=1, descending=True, stable=True).indices  # ties: the lowest position first
    rank = torch.empty_like(order).scatter_(1, order, p["pos"][None].expand_as(order).contiguous())
    kept = valid & ((rank < keep) | (lens <= keep))
    moved = kept & (lens > keep)
    row, at = moved.nonzero(as_tuple=True)
    to = s["dst_slot"][row, (moved.cumsum(1) - 1)[row, at]]
    src, P = p["slot"][row, at], p["P"]
    s["kv"][to // P, :, to % P] = s["kv"][src // P, :, src % P]
    flat[to] = flat[src]
    return p["pos"][None].expand_as(kept)[kept].to(torch.int32), s["scores"], s["kv"]


def run(s):
    op = s["op"]
    if not own:
        return {"latent": _plain_latent, "expanded": _plain_expanded, "decode_weights": _plain_decode_weights,
                "weights": _plain_weights, "evict": _plain_evict}[op](s)
    h, ws = s["h"], s["ws"]
    if op == "latent":
        h.append_planned(s["c_new"], s["r_new"], s["cache"], workspace=ws)
        h.run(s["q"], s["cache"], s["out"], s["lse"], workspace=ws)
        return s["out"], s["lse"], s["cache"]
    if op == "expanded":
        h.run_dense(s["q"], s["k_nope"], s["k_rope"], s["v"], s["out"], s["lse"], workspace=ws)
        return s["out"], s["lse"]
    if op == "decode_weights":
        h.run_decode_weights(s["q"], s["kv"], s["out"], s["lse"], s["scores"], decay=s["c"]["decay"], workspace=ws)
        return s["out"], s["lse"], s["scores"]
    if op == "weights":
        h.run_weights(s["q"], s["lse"], s["kv"], s["scores"], decay=s["c"]["decay"], workspace=ws)
        return s["scores"]
    h.run_evict(s["kv"], s["scores"], s["kept"], workspace=ws)
    return s["kept"], s["scores"], s["kv"]


def exact(c, seed):
    """The definitions in 64 bits, one row at a time."""
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    lens = _lens(c)
    if c["op"] == "expanded":
        outs, lses, q0, k0 = [], [], 0, 0
        for L in lens:
            n = c["new"] or L
            see = torch.ones(n, L, dtype=torch.bool, device=DEV).tril(L - n)
            o = torch.empty(n, c["heads"], VDIM, dtype=torch.float64, device=DEV)
            z = torch.empty(n, c["heads"], dtype=torch.float64, device=DEV)
            for h in range(c["heads"]):
                q = s["q"][q0:q0 + n, h].double()
                x = q[:, :NOPE] @ s["k_nope"][k0:k0 + L, h].double().T + q[:, NOPE:] @ s["k_rope"][k0:k0 + L].double().T
                x = torch.where(see, x * SCALE_LATENT, -math.inf)
                z[:, h] = torch.logsumexp(x, -1)
                o[:, h] = torch.softmax(x, -1) @ s["v"][k0:k0 + L, h].double()
            outs.append(o)
            lses.append(z)
            q0, k0 = q0 + n, k0 + L
        return torch.cat(outs), torch.cat(lses)
    p, P = s["p"], c["page"]
    table = [torch.tensor(p["kv_indices"][a:b], device=DEV).long()
             for a, b in zip(p["kv_indptr"][:-1].tolist(), p["kv_indptr"][1:].tolist())]
    if c["op"] == "evict":
        scores, kept = s["scores"].double(), []
        was = scores.clone()
        for r, L in enumerate(lens):
            mine = was[table[r]].view(-1)[:L]
            if L <= c["keep"]:
                kept += range(L)
                continue
            v = mine.tolist()
            head, tail = list(range(c["sink"])), list(range(L - c["recent"], L))
            mid = sorted(range(c["sink"], L - c["recent"]), key=lambda i: (-v[i], i))[: c["keep"] - c["sink"] - c["recent"]]
            best = head + sorted(mid) + tail
            kept += best
            scores.view(-1)[s["dst_slot"][r]] = mine[torch.tensor(best, device=DEV)]
        return torch.tensor(kept, dtype=torch.int32, device=DEV), scores, None
    if c["op"] == "latent":
        n, outs, lses = c["new"], [], []
        for r, L in enumerate(lens):
            k = torch.cat([s["cache"][table[r]].view(-1, LATENT + ROPE)[:L - n],
                           torch.cat([s["c_new"][r * n:(r + 1) * n], s["r_new"][r * n:(r + 1) * n]], 1)]).double()
            x = torch.einsum("thw,lw->thl", s["q"][r * n:(r + 1) * n].double(), k) * SCALE_LATENT
            for t in range(n):
                x[t, :, L - n + t + 1:] = -math.inf
            outs.append(torch.einsum("thl,lw->thw", torch.softmax(x, -1), k[:, :LATENT]))
            lses.append(torch.logsumexp(x, -1))
        return torch.cat(outs), torch.cat(lses), None
    n, g = c.get("new", 1), c["heads"] // c["kv_heads"]
    scores, outs, lses = s["scores"].double(), [], []
    for r, L in enumerate(lens):
        k = s["kv"][table[r], 0].reshape(-1, c["kv_heads"], c["dim"])[:L]
        v = s["kv"][table[r], 1].reshape(-1, c["kv_heads"], c["dim"])[:L]
        w = torch.zeros(L, dtype=torch.float64, device=DEV)
        see = torch.ones(n, L, dtype=torch.bool, device=DEV).tril(L - n)
        o = torch.empty(n, c["heads"], c["dim"], dtype=torch.float64, device=DEV)
        z = torch.empty(n, c["heads"], dtype=torch.float64, device=DEV)
        for h in range(c["heads"]):
            x = torch.where(see, s["q"][r * n:(r + 1) * n, h].double() @ k[:, h // g].double().T * s["scale"], -math.inf)
            z[:, h] = torch.logsumexp(x, -1)
            if c["op"] == "decode_weights":
                o[:, h] = torch.softmax(x, -1) @ v[:, h // g].double()
                w += torch.exp(x - z[:, h, None]).sum(0)
            else:
                w += torch.exp(x - s["lse"][r * n:(r + 1) * n, h, None].double()).sum(0)
        outs.append(o)
        lses.append(z)
        i = torch.arange(L, device=DEV)
        page, slot = table[r][i // P], i % P
        before = torch.where(i < L - n, scores[page, slot] * c["decay"], 0.0)
        scores[page, slot] = before + w
    return (torch.cat(outs), torch.cat(lses), scores) if c["op"] == "decode_weights" else scores
