"""The speculative step from its definitions, on host tensors: trees, attention in 64 bits, page and slot maps,
acceptance."""
import math

import numpy as np
import torch


def tree(n, spread, salt=0):
    """Parents of n nodes: spread 1 is a chain, larger ones branch."""
    return [-1] + [max(0, i - 1 - (i * 7 + salt * 3) % spread) for i in range(1, n)] if n else []


def ancestors(parents):
    """[n, n]: whether node j is node i or above it; and the depths."""
    n = len(parents)
    up, depth = torch.zeros(n, n, dtype=torch.bool), []
    for i, p in enumerate(parents):
        if p >= 0:
            up[i] = up[p]
        up[i, i] = True
        depth.append(0 if p < 0 else depth[p] + 1)
    return up, torch.tensor(depth, dtype=torch.long)


def visible(ctx, parents, window=-1):
    """[n, ctx + n]: what each node sees of the row's cached tokens and of its nodes."""
    up, depth = ancestors(parents)
    n = len(parents)
    see = torch.cat([torch.ones(n, ctx, dtype=torch.bool), up], 1)
    if window >= 0 and n:
        place = torch.cat([torch.arange(ctx), ctx + depth])
        see &= place[None] >= (ctx + depth)[:, None] - window
    return see


def row_keys(kv_layer, kvp, kvi, r, ctx):
    """K and V of the first ctx tokens of row r: [ctx, Hkv, D] each."""
    x = kv_layer[torch.as_tensor(kvi[kvp[r]: kvp[r + 1]]).long()]
    return (x[:, i].reshape(-1, *x.shape[3:])[:ctx] for i in (0, 1))


def attend(q, k, v, see, scale):
    """q [n, H, D], k and v [L, Hkv, D], see [n, L]: out, lse, sum p|v|, and how far a score of 32-bit sums may be
    off, query by query over the keys it sees alone, in 64 bits."""
    H, g = q.shape[1], q.shape[1] // k.shape[1]
    q, k, v = q.double(), k.double().repeat_interleave(g, 1), v.double().repeat_interleave(g, 1)
    parts = []
    for i in range(len(q)):
        at = see[i].nonzero()[:, 0]
        x = torch.einsum("hd,lhd->hl", q[i], k[at]) * scale
        p = torch.softmax(x, -1)
        clean = v[at].nan_to_num(0, 0, 0)
        # where a value is not finite one by one: an einsum may sum in any order
        o = torch.einsum("hl,lhd->hd", p, v[at]) if torch.isfinite(v[at]).all() else (p.T[..., None] * v[at]).sum(0)
        most = k[at].nan_to_num(0, 0, 0).norm(dim=-1).max()
        parts.append((o, torch.logsumexp(x, -1), torch.einsum("hl,lhd->hd", p, clean.abs()),
                      q.shape[-1] * 2.0 ** -24 * q[i].norm(dim=-1) * most * scale))
    if not parts:
        e = torch.zeros(0, H, q.shape[-1], dtype=torch.float64)
        return e, e[..., 0], e, e[..., 0]
    return tuple(torch.stack(y) for y in zip(*parts))


def attention(q, k_new, v_new, kv_layer, qo, kvp, kvi, last, trees, scale, window=-1):
    """All rows; trees: the parents of each row's nodes."""
    P, parts = kv_layer.shape[2], []
    for r, parents in enumerate(trees):
        a, b = int(qo[r]), int(qo[r + 1])
        if a == b:
            continue
        ctx = int((kvp[r + 1] - kvp[r] - 1) * P + last[r]) - (b - a)
        k, v = row_keys(kv_layer, kvp, kvi, r, ctx)
        parts.append(attend(q[a:b], torch.cat([k, k_new[a:b]]), torch.cat([v, v_new[a:b]]), visible(ctx, parents, window), scale))
    return tuple(torch.cat(y) for y in zip(*parts))


def accept(parents, draft, target):
    """The accepted path of one row and the token that follows it."""
    if not parents:
        return [], -1
    path = [0]
    while True:
        more = [j for j in range(len(parents)) if parents[j] == path[-1] and draft[j] == target[path[-1]]]
        if not more:
            return path, target[path[-1]]
        path.append(more[0])


def maps(seq, new, table, held, free, count, P, kvi, tokens):
    """The step's maps by the definition, row by row; every argument a list (table a list of lists).  Returns a
    dict, or the status where nothing is done."""
    table, free, F = [list(x) for x in table], list(free), count
    width = len(table[0]) if table else 0
    need = [-(-(a + b) // P) for a, b in zip(seq, new)]
    if any(a < 0 or b < 0 or h < 0 or h > width or n > width for a, b, h, n in zip(seq, new, held, need)):
        return -1
    if sum(new) > tokens or sum(need) > len(kvi):
        return -2
    back, taken = sum(max(0, h - n) for h, n in zip(held, need)), sum(max(0, n - h) for h, n in zip(held, need))
    if F < 0 or F > len(free) or F + back > len(free):
        return -3
    if taken > F + back:
        return taken - F - back
    for r, (h, n) in enumerate(zip(held, need)):
        for b in range(n, h):
            free[F] = table[r][b]
            F += 1
    for r, (h, n) in enumerate(zip(held, need)):
        for b in range(h, n):
            F -= 1
            table[r][b] = free[F]
    qo = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
    kvp = np.concatenate([[0], np.cumsum(need)]).astype(int).tolist()
    pages = [p for r, n in enumerate(need) for p in table[r][:n]]
    where = [(r, p) for r in range(len(seq)) for p in range(seq[r], seq[r] + new[r])]
    return dict(qo=qo, kvp=kvp, kvi=pages + list(kvi[len(pages):]), last=[(a + b - 1) % P + 1 if a + b else 0 for a, b in zip(seq, new)],
                slots=[table[r][p // P] * P + p % P for r, p in where] + [-1] * (tokens - len(where)),
                positions=[p for _, p in where] + [0] * (tokens - len(where)), held=need, count=F, table=table, free=free)


def indices(lens, P, seed, spare=3):
    """kv_indptr, shuffled page ids, last_page_len and the pool's pages of rows of these lengths."""
    g = np.random.default_rng(seed)
    pages = [-(-L // P) for L in lens]
    order = g.permutation(sum(pages) + spare).astype(np.int32)
    kvp = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    last = np.array([(L - 1) % P + 1 if L else 0 for L in lens], np.int32)
    return kvp, order[: kvp[-1]], last, sum(pages) + spare


def default_scale(D):
    return 1.0 / math.sqrt(D)
