"""Measured cases of the operators of a speculative decoding step over a paged KV cache.

Every row of a batch has some tokens in the cache and a tree of drafted tokens whose root is the token
chosen last.  One step takes three operators:

* "maps": from the rows' lengths and numbers of new tokens, on the GPU: pages taken from a stack of free
  ones (or given back to it), the block table, the index arrays of the paged attention calls, and the slot and
  position of every new token.
* "tree": attention of all drafted tokens in one pass: a token sees the row's cached tokens, its ancestors
  in the tree and itself.  K and V of the drafted tokens come from the step's own tensors.
* "accept": the longest path of drafted tokens that the model's own choices confirm, and its keys and
  values, of all layers, into the row's next slots.

Plain forms are elementary torch operations in 32 bits on padded batches; exact() computes the same row
by row in 64 bits (or in whole numbers).
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one conversation, a small tree: latency
        dict(name="tree, one row", op="tree", rows=1, heads=32, kv_heads=8, dim=128, page=16, shortest=517, longest=517,
             drafts=8, spread=3, window=-1),
        # a serving batch with trees of 16 tokens
        dict(name="tree, batch of 32", op="tree", rows=32, heads=32, kv_heads=8, dim=128, page=16, shortest=203, longest=8190,
             drafts=16, spread=4, window=-1),
        # wide trees of a large model's share of heads
        dict(name="tree, wide", op="tree", rows=16, heads=64, kv_heads=8, dim=128, page=64, shortest=611, longest=12001,
             drafts=61, spread=9, window=-1),
        # few long documents, chains of five tokens, an odd group size, small heads
        dict(name="tree, long chains", op="tree", rows=3, heads=20, kv_heads=4, dim=64, page=32, shortest=30011, longest=65521,
             drafts=5, spread=1, window=-1),
        # large heads under a sliding window
        dict(name="tree, window", op="tree", rows=24, heads=16, kv_heads=8, dim=256, page=16, shortest=1001, longest=9003,
             drafts=27, spread=5, window=2047),
        # one conversation's next step
        dict(name="maps, one row", op="maps", rows=1, page=16, shortest=517, longest=517, new=8),
        # a large batch of ordinary lengths
        dict(name="maps, batch of 200", op="maps", rows=200, page=16, shortest=33, longest=8190, new=17),
        # many long rows, small pages
        dict(name="maps, long rows", op="maps", rows=500, page=8, shortest=1009, longest=30011, new=5),
        # a batch of prompts that has no page yet
        dict(name="maps, prompts", op="maps", rows=48, page=16, shortest=0, longest=0, new=8111),
        # one conversation, all layers
        dict(name="accept, one row", op="accept", rows=1, layers=32, kv_heads=8, dim=128, page=16, shortest=129, longest=129,
             drafts=8, spread=3, bits=64),
        # a serving batch, all layers
        dict(name="accept, batch of 64", op="accept", rows=64, layers=32, kv_heads=8, dim=128, page=16, shortest=7,
             longest=131, drafts=16, spread=4, bits=64),
        # wide trees with long accepted paths, small heads
        dict(name="accept, long paths", op="accept", rows=40, layers=24, kv_heads=4, dim=64, page=32, shortest=0, longest=301,
             drafts=61, spread=2, bits=32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "maps", "accept"])
    if op == "maps":
        rows, page = _log(rng, 1, 500), rng.choice([1, 2, 8, 16, 32, 64])
        most = max(1, min(30000, 1_500_000 * page // rows))
        longest = _log(rng, 1, most)
        return dict(op=op, rows=rows, page=page, shortest=longest // rng.randint(1, 9), longest=longest,
                    new=_log(rng, 1, max(1, min(4000, 300_000 // rows))))
    drafts, spread = _log(rng, 1, 200), rng.choice([1, 2, 4, 9])
    if op == "accept":
        rows, layers, kv_heads, dim = _log(rng, 1, 64), _log(rng, 1, 32), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        most = max(1, min(1500, 280_000_000 // (rows * layers * kv_heads * dim) - drafts - 64))
        drafts = min(drafts, 64)
        longest = _log(rng, 1, most)
        return dict(op=op, rows=rows, layers=layers, kv_heads=kv_heads, dim=dim, page=rng.choice([8, 16, 32, 64]),
                    shortest=longest // rng.randint(1, 9), longest=longest, drafts=drafts, spread=spread, bits=rng.choice([32, 64]))
    rows, kv_heads, dim = _log(rng, 1, 64), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    most = max(8, min(65521, 130_000_000 // (rows * kv_heads * dim), 90_000_000_000 // (rows * heads * drafts * max(dim, 128))))
    longest = _log(rng, 1, most)
    return dict(op=op, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([8, 16, 32, 64, 128]),
                shortest=longest // rng.randint(1, 9), longest=longest, drafts=drafts, spread=spread,
                window=rng.choice([-1, -1, -1, 127, 1000]))


def _lens(c):
    """Row lengths from the longest to the shortest, evenly apart; they do not depend on the seed."""
    n = c["rows"]
    return [c["longest"] - (c["longest"] - c["shortest"]) * i // max(1, n - 1) for i in range(n)]


def _nodes(c):
    """Drafted tokens of each row, the root among them."""
    return [max(1, c["drafts"] - (r % 4) * (c["drafts"] // 5)) for r in range(c["rows"])]


def _parents(c, r, n):
    """A row's tree: the parent of every node, -1 for the root; spread 1 is a chain."""
    return [-1] + [max(0, i - 1 - (i * 7 + r * 3) % c["spread"]) for i in range(1, n)]


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _path(parents, r):
    """The accepted path of row r: from the root to a node in the tree's first two thirds."""
    n = len(parents)
    at, path = (r * 5 + n // 2) % max(1, (2 * n + 2) // 3), []
    while at >= 0:
        path.append(at)
        at = parents[at]
    return path[::-1]


def _map_rows(c):
    """(tokens before the step, new tokens, pages held) of each row: some rows hold a page too many, some
    have ended and give theirs back."""
    P, rows = c["page"], []
    for r, L in enumerate(_lens(c)):
        held = -(-L // P)
        if r % 17 == 5:
            rows.append((0, 0, held))
        else:
            rows.append((L, max(1, c["new"] - r % 7 * (c["new"] // 9)), held + (1 if r % 3 == 2 else 0)))
    return rows


def work(c):
    if c["op"] == "maps":
        rows, P = _map_rows(c), c["page"]
        need = [-(-(L + n) // P) for L, n, _ in rows]
        taken = sum(max(0, k - h) for k, (_, _, h) in zip(need, rows))
        back = sum(max(0, h - k) for k, (_, _, h) in zip(need, rows))
        T, R = sum(n for _, n, _ in rows), len(rows)
        ints = 3 * R + sum(need) + taken + back  # lengths, pages held; the entries that are kept, taken, given back
        ints += sum(need) + 2 * T + taken + back + 4 * R + 2  # kv_indices, slots, positions, table, stack, indptrs and fills, pages held
        return {"bytes": 4.0 * ints, "flops": 0.0}
    nodes = _nodes(c)
    trees = [_parents(c, r, n) for r, n in enumerate(nodes)]
    if c["op"] == "accept":
        acc, T = sum(len(_path(t, r)) for r, t in enumerate(trees)), sum(nodes)
        token = c["bits"] // 8
        return {"bytes": 2.0 * acc * c["layers"] * 2 * c["kv_heads"] * c["dim"] * 2 + T * (4 + 2 * token + 4) + c["rows"] * (8 + token),
                "flops": 0.0}
    H, Hkv, D, w = c["heads"], c["kv_heads"], c["dim"], c["window"]
    keys = pairs = 0
    for L, t in zip(_lens(c), trees):
        depth = _depths(t)
        first = [max(0, L + d - w) if w >= 0 else 0 for d in depth]
        keys += max(0, L - min(first))
        pairs += sum(max(0, L - f) + (min(d, w) if w >= 0 else d) + 1 for f, d in zip(first, depth))
    T = sum(nodes)
    return {"bytes": 2.0 * (keys + T) * Hkv * D * 2 + 2.0 * T * H * D * 2 + T * H * 4, "flops": 4.0 * pairs * H * D}


def prepare(c, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gd, device=DEV, dtype=torch.float32).to(torch.bfloat16)

    def i32(x):
        return torch.as_tensor(x, dtype=torch.int32).to(DEV)

    P, R = c["page"], c["rows"]
    s = {"c": c, "op": c["op"]}
    if c["op"] == "maps":
        rows = _map_rows(c)
        need = [-(-(L + n) // P) for L, n, _ in rows]
        held = [h for _, _, h in rows]
        width = max(max(need), max(held)) + 3
        taken = sum(max(0, k - h) for k, h in zip(need, held))
        free = taken + 5
        ids = torch.randperm(sum(held) + free, generator=g).to(torch.int32)
        table = torch.full((R, width), -1, dtype=torch.int32)
        table[torch.arange(width)[None] < torch.tensor(held)[:, None]] = ids[: sum(held)]
        T, nnz = sum(n for _, n, _ in rows), sum(need)
        new = lambda n: torch.full((n,), -1, dtype=torch.int32, device=DEV)
        s.update(seq=i32([L for L, _, _ in rows]), new=i32([n for _, n, _ in rows]), held=i32(held), table=table.to(DEV),
                 free=torch.cat([ids[sum(held):], torch.full((sum(held),), -1, dtype=torch.int32)]).to(DEV), count=i32([free]),
                 qo=new(R + 1), kvp=new(R + 1), kvi=new(nnz + 7), last=new(R), slots=new(T + 9), pos=new(T + 9), status=new(1),
                 held_out=new(R), count_out=new(1))
        if own:
            from paged_kv_attention_gqa_gb300 import binding as B
            s["h"] = B.Handle(num_qo_heads=8, num_kv_heads=8, head_dim=128, page_size=P, max_batch=R, max_total_tokens=T + 9,
                              max_num_pages=nnz + 7, num_cache_pages=len(ids))
        return s

    Hkv, D, lens, nodes = c["kv_heads"], c["dim"], _lens(c), _nodes(c)
    trees = [_parents(c, r, n) for r, n in enumerate(nodes)]
    T, most = sum(nodes), max(nodes)
    # the rows' pages, for the context and every drafted token, over a shuffled pool
    pages = [-(-(L + n) // P) for L, n in zip(lens, nodes)]
    ids = torch.randperm(sum(pages) + 3, generator=g)[: sum(pages)]
    qo, kvp = torch.tensor([0] + nodes).cumsum(0), torch.tensor([0] + pages).cumsum(0)
    last = [(L + n - 1) % P + 1 for L, n in zip(lens, nodes)]
    # padded: token of every (row, node), slot of every (row, position), who is whose ancestor (or itself)
    i = torch.arange(most)
    real = i[None] < torch.tensor(nodes)[:, None]
    token = torch.where(real, qo[:-1, None] + i[None], 0)
    j = torch.arange(max(L + n for L, n in zip(lens, nodes)))
    at = (kvp[:-1, None] + j[None] // P).clamp(max=max(sum(pages) - 1, 0))
    slot = torch.where(j[None] < (torch.tensor(lens) + torch.tensor(nodes))[:, None], ids[at] * P + j[None] % P, 0)
    parent = torch.full((R, most), -1)
    above = torch.zeros(R, most, most, dtype=torch.bool)
    for r, t in enumerate(trees):
        parent[r, : len(t)] = torch.tensor(t)
        for a, p in enumerate(t):
            if p >= 0:
                above[r, a] = above[r, p]
            above[r, a, a] = True
    s.update(lens=torch.tensor(lens).to(DEV), real=real.to(DEV), token=token.to(DEV), slot=slot.to(DEV), j=j.to(DEV),
             parent=parent.to(DEV), above=above.to(DEV), pages=sum(pages) + 3)
    chain = c["spread"] == 1
    index = dict(qo=i32(qo), kvp=i32(kvp), kvi=i32(ids), last=i32(last), parents=None if chain else i32(sum(trees, [])))

    if c["op"] == "tree":
        H = c["heads"]
        new = randn(T, 2, Hkv, D)  # the step's keys and values, side by side
        s.update(q=(1.5 * randn(T, H, D)).to(torch.bfloat16), k=new[:, 0], v=new[:, 1], kv=randn(s["pages"], 2, P, Hkv, D),
                 out=torch.empty(T, H, D, device=DEV, dtype=torch.bfloat16), lse=torch.empty(T, H, device=DEV))
    else:
        N, kind = c["layers"], torch.int64 if c["bits"] == 64 else torch.int32
        new = randn(N, T, 2, Hkv, D)
        # drafted tokens are even, what the model chooses elsewhere is odd: it agrees along one path
        draft = torch.randint(0, 60000, (T,), generator=g) * 2
        target = torch.randint(0, 60000, (T,), generator=g) * 2 + 1
        for r, t in enumerate(trees):
            path = _path(t, r)
            for a, b in zip(path, path[1:]):
                target[int(qo[r]) + a] = draft[int(qo[r]) + b]
        s.update(draft=draft.to(kind).to(DEV), target=target.to(kind).to(DEV), k=new[:, :, 0], v=new[:, :, 1],
                 cache=randn(N, s["pages"], 2, P, Hkv, D), accepted=torch.full((T,), -7, dtype=torch.int32, device=DEV),
                 count=torch.empty(R, dtype=torch.int32, device=DEV), next=torch.empty(R, dtype=kind, device=DEV),
                 seq=torch.empty(R, dtype=torch.int32, device=DEV))
    if own:
        from paged_kv_attention_gqa_gb300 import binding as B
        h = B.Handle(num_qo_heads=c.get("heads", Hkv), num_kv_heads=Hkv, head_dim=D, page_size=P, max_batch=R,
                     max_total_tokens=T, max_num_pages=sum(pages), num_cache_pages=s["pages"])
        ws = torch.empty(h.workspace_size(B.MODE_TREE), dtype=torch.uint8, device=DEV)
        s.update(h=h, ws=ws, index=index)
        h.plan_tree(index["qo"], index["kvp"], index["kvi"], index["last"], index["parents"], num_tokens=T, max_new=most,
                    workspace=ws, window_left=c.get("window", -1))
    return s


def _plain_tree(s):
    c = s["c"]
    R, H, Hkv, D, w = c["rows"], c["heads"], c["kv_heads"], c["dim"], c["window"]
    n, g = s["real"].shape[1], H // Hkv
    j, lens = s["j"][: c["longest"]], s["lens"][:, None]
    cached, slot = j[None] < lens, s["slot"][:, : c["longest"]]
    rows = lambda x, at, real: x[at].float().masked_fill_(~real[..., None, None], 0.0)
    P, page = c["page"], slot // c["page"]
    k = torch.cat([rows(s["kv"][:, 0].reshape(-1, Hkv, D), page * P + slot % P, cached), rows(s["k"], s["token"], s["real"])], 1)
    v = torch.cat([rows(s["kv"][:, 1].reshape(-1, Hkv, D), page * P + slot % P, cached), rows(s["v"], s["token"], s["real"])], 1)
    q = s["q"][s["token"]].float().view(R, n, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(R * Hkv, g * n, D)
    x = torch.bmm(q, k.permute(0, 2, 3, 1).reshape(R * Hkv, D, -1)).view(R, H, n, -1) * (1.0 / math.sqrt(D))
    place = lens + s["above"].sum(-1) - 1  # [R, n]
    sees, kin = cached[:, None].expand(R, n, -1), s["above"]
    if w >= 0:
        sees = sees & (j[None, None] >= place[..., None] - w)
        kin = kin & (place[:, None] >= place[..., None] - w)
    x = x.masked_fill(~torch.cat([sees, kin], -1)[:, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    e = (x - m).exp()
    t = e.sum(-1, keepdim=True)
    o = torch.bmm(e.view(R * Hkv, g * n, -1), v.transpose(1, 2).reshape(R * Hkv, -1, D)).view(R, H, n, D) / t
    return o.transpose(1, 2)[s["real"]].to(torch.bfloat16), (m + t.log())[..., 0].transpose(1, 2)[s["real"]]


def _plain_maps(s):
    P, table, held, R = s["c"]["page"], s["table"], s["held"].long(), s["c"]["rows"]
    seq, new, free, F = s["seq"].long(), s["new"].long(), s["free"], s["count"].long()
    need = (seq + new + P - 1) // P
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    b = torch.arange(table.shape[1], device=DEV)[None]
    # pages given back go on the stack, row by row; one slot more takes what is not written
    back, taken = (held - need).clamp(min=0), (need - held).clamp(min=0)
    at = F + (back.cumsum(0) - back)[:, None] + b - need[:, None]
    at = torch.where((b >= need[:, None]) & (b < held[:, None]), at, len(free))
    free.copy_(torch.cat([free, free[:1]]).scatter_(0, at.view(-1), table.view(-1))[:-1])
    F = F + back.sum()
    top = F - 1 - ((taken.cumsum(0) - taken)[:, None] + b - held[:, None])
    table.copy_(torch.where((b >= held[:, None]) & (b < need[:, None]), free[top.clamp(0, len(free) - 1)], table))
    qo, kvp = torch.cat([zero, new.cumsum(0)]), torch.cat([zero, need.cumsum(0)])
    e = torch.arange(len(s["kvi"]), device=DEV)
    r = torch.searchsorted(kvp, e, right=True).sub_(1).clamp_(0, R - 1)
    kvi = torch.where(e < kvp[-1], table[r, (e - kvp[r]).clamp(0, table.shape[1] - 1)], s["kvi"])
    t = torch.arange(len(s["slots"]), device=DEV)
    r = torch.searchsorted(qo, t, right=True).sub_(1).clamp_(0, R - 1)
    pos = torch.where(t < qo[-1], seq[r] + t - qo[r], 0)
    slots = torch.where(t < qo[-1], table[r, (pos // P).clamp(max=table.shape[1] - 1)] * P + pos % P, -1)
    last = torch.where(need > 0, (seq + new - 1) % P + 1, 0)
    i32 = lambda x: x.to(torch.int32)
    return i32(qo), i32(kvp), kvi, i32(last), i32(slots), i32(pos), i32(zero), i32(need), i32(F - taken.sum()), table, free


def _plain_accept(s):
    c, real, parent, T = s["c"], s["real"], s["parent"], len(s["draft"])
    n, P = real.shape[1], c["page"]
    draft, target = s["draft"][s["token"]], s["target"][s["token"]]
    hit = (draft == target.gather(1, parent.clamp(min=0))) & (parent >= 0) & real
    i = torch.arange(n, device=DEV)
    # of several such children the first one
    earlier = ((parent[:, None] == parent[..., None]) & hit[:, None] & (i[None] < i[:, None])).any(-1)
    goes = (hit & ~earlier) | (i == 0)
    path = real & ~(s["above"] & ~goes[:, None]).any(-1)
    rank = path.cumsum(1) - 1
    count = path.sum(1)
    accepted = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    row, node = path.nonzero(as_tuple=True)
    first = s["token"][:, 0]
    accepted[first[row] + rank[row, node]] = node.to(torch.int32)
    slot = s["slot"][row, s["lens"][row] + rank[row, node]]
    s["cache"][:, slot // P, 0, slot % P] = s["k"][:, first[row] + node]
    s["cache"][:, slot // P, 1, slot % P] = s["v"][:, first[row] + node]
    end = torch.where(path, i, 0).amax(1, keepdim=True)
    return accepted, count.to(torch.int32), target.gather(1, end)[:, 0], (s["lens"] + count).to(torch.int32), s["cache"]


def run(s):
    if not own:
        return {"tree": _plain_tree, "maps": _plain_maps, "accept": _plain_accept}[s["op"]](s)
    h = s["h"]
    if s["op"] == "tree":
        h.run_tree(s["q"], s["k"], s["v"], s["kv"], s["out"], s["lse"], workspace=s["ws"])
        return s["out"], s["lse"]
    if s["op"] == "maps":
        h.build_maps(s["seq"], s["new"], s["table"], s["held"], s["free"], s["count"], qo_indptr=s["qo"], kv_indptr=s["kvp"],
                     kv_indices=s["kvi"], last_page_len=s["last"], slots=s["slots"], positions=s["pos"], status=s["status"],
                     num_blocks_out=s["held_out"], free_count_out=s["count_out"])
        return (s["qo"], s["kvp"], s["kvi"], s["last"], s["slots"], s["pos"], s["status"], s["held_out"], s["count_out"],
                s["table"], s["free"])
    h.run_accept(s["draft"], s["target"], s["k"], s["v"], s["cache"], s["accepted"], s["count"], s["next"], s["seq"],
                 workspace=s["ws"])
    return s["accepted"], s["count"], s["next"], s["seq"], s["cache"]


def exact(c, seed):
    """The definitions, one row at a time."""
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    P, lens = c["page"], _lens(c)
    if c["op"] == "maps":
        table, free, kvi = s["table"].tolist(), s["free"].tolist(), s["kvi"].tolist()
        rows, F = _map_rows(c), int(s["count"])
        need = [-(-(L + n) // P) for L, n, _ in rows]
        for r, (_, _, h) in enumerate(rows):
            for b in range(need[r], h):
                free[F] = table[r][b]
                F += 1
        for r, (_, _, h) in enumerate(rows):
            for b in range(h, need[r]):
                F -= 1
                table[r][b] = free[F]
        qo, kvp, slots, pos, at = [0], [0], [], [], 0
        for r, (L, n, _) in enumerate(rows):
            for b in range(need[r]):
                kvi[at] = table[r][b]
                at += 1
            pos += range(L, L + n)
            slots += [table[r][p // P] * P + p % P for p in range(L, L + n)]
            qo.append(qo[-1] + n)
            kvp.append(at)
        rest = len(s["slots"]) - len(slots)
        last = [(L + n - 1) % P + 1 if L + n else 0 for L, n, _ in rows]
        out = (qo, kvp, kvi, last, slots + [-1] * rest, pos + [0] * rest, [0], need, [F], table, free)
        return tuple(torch.tensor(x, dtype=torch.int32) for x in out)
    trees = [_parents(c, r, n) for r, n in enumerate(_nodes(c))]
    if c["op"] == "accept":
        draft, target, cache = s["draft"].tolist(), s["target"].tolist(), s["cache"]
        accepted, count, following, seq, t0 = [], [], [], [], 0
        for r, t in enumerate(trees):
            path = [0]
            while True:
                more = [a for a in range(len(t)) if t[a] == path[-1] and draft[t0 + a] == target[t0 + path[-1]]]
                if not more:
                    break
                path.append(more[0])
            for i, a in enumerate(path):
                at = int(s["slot"][r, lens[r] + i])
                cache[:, at // P, 0, at % P] = s["k"][:, t0 + a]
                cache[:, at // P, 1, at % P] = s["v"][:, t0 + a]
            accepted += path + [-1] * (len(t) - len(path))
            count.append(len(path))
            following.append(target[t0 + path[-1]])
            seq.append(lens[r] + len(path))
            t0 += len(t)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32)
        return i32(accepted), i32(count), torch.tensor(following, dtype=s["next"].dtype), i32(seq), cache.double()
    H, Hkv, D, w = c["heads"], c["kv_heads"], c["dim"], c["window"]
    outs, lses, t0 = [], [], 0
    for r, t in enumerate(trees):
        L, n, depth = lens[r], len(t), torch.tensor(_depths(t), device=DEV)
        flat = s["kv"].transpose(0, 1).reshape(2, -1, Hkv, D)
        k, v = (torch.cat([flat[x, s["slot"][r, :L]], s[y][t0: t0 + n]]).double() for x, y in ((0, "k"), (1, "v")))
        place = torch.cat([torch.arange(L, device=DEV), L + depth])
        sees = torch.zeros(n, L + n, dtype=torch.bool, device=DEV)
        sees[:, :L] = True
        for a in range(n):
            b = a
            while b >= 0:
                sees[a, L + b] = True
                b = t[b]
        if w >= 0:
            sees &= place[None] >= (L + depth)[:, None] - w
        q = s["q"][t0: t0 + n].double().view(n, Hkv, H // Hkv, D)
        x = torch.einsum("nkgd,lkd->kgnl", q, k) / math.sqrt(D)
        x = x.masked_fill(~sees, -math.inf)
        z = torch.logsumexp(x, -1, keepdim=True)
        outs.append(torch.einsum("kgnl,lkd->nkgd", (x - z).exp(), v).reshape(n, H, D))
        lses.append(z[..., 0].permute(2, 0, 1).reshape(n, H))
        t0 += n
    return torch.cat(outs), torch.cat(lses)
