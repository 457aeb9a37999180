"""Accumulated attention weights and the eviction by them, from their definitions, on host tensors in
64 bits."""
import math

import torch

from latent_ref import attend, score_error, visible


def lengths(kvp, lpl, P):
    return [int((kvp[r + 1] - kvp[r] - 1) * P + lpl[r]) if kvp[r + 1] > kvp[r] else 0 for r in range(len(lpl))]


def rows_of(cache, kvp, kvi, r, L, kv):
    """K (0) or V (1) rows [L, Hkv, D] of row r out of [pages, 2, P, Hkv, D]."""
    ids = torch.as_tensor(kvi[kvp[r]: kvp[r + 1]]).long()
    return cache[ids, kv].reshape(-1, *cache.shape[3:])[:L]


def attention(q, cache, qo, kvp, kvi, lpl, scale, causal=True, window_left=-1):
    """out, lse, sum p|v|, score error of the grouped-query rows."""
    g, parts = q.shape[1] // cache.shape[3], []
    for r, L in enumerate(lengths(kvp, lpl, cache.shape[2])):
        a, b = int(qo[r]), int(qo[r + 1])
        if a == b:
            continue
        k = rows_of(cache, kvp, kvi, r, L, 0).repeat_interleave(g, 1)
        v = rows_of(cache, kvp, kvi, r, L, 1).repeat_interleave(g, 1)
        parts.append((*attend(q[a:b], k, v, visible(L, b - a, causal, window_left), scale), score_error(q[a:b], k, scale)))
    return tuple(torch.cat(x) for x in zip(*parts))


def add_weights(scores, q, lse, cache, qo, kvp, kvi, lpl, scale, decay, causal=True, window_left=-1):
    """The scores after a step, and for every slot sum over queries and heads of w * (its error), as
    [pages, P] in float64: (scores, error bound)."""
    P, g = cache.shape[2], q.shape[1] // cache.shape[3]
    new, bound = scores.double().clone(), torch.zeros(scores.shape, dtype=torch.float64)
    for r, L in enumerate(lengths(kvp, lpl, P)):
        a, b = int(qo[r]), int(qo[r + 1])
        w, e = torch.zeros(L, dtype=torch.float64), torch.zeros(L, dtype=torch.float64)
        if b > a:
            k = rows_of(cache, kvp, kvi, r, L, 0).repeat_interleave(g, 1).double()
            x = torch.einsum("nhd,lhd->nhl", q[a:b].double(), k) * scale - lse[a:b].double()[..., None]
            p = torch.exp(x.masked_fill(~visible(L, b - a, causal, window_left)[:, None], -math.inf))
            err = score_error(q[a:b], k, scale) + 2.0 ** -20 * (1 + lse[a:b].double().abs())
            w, e = p.sum((0, 1)), (p * err[..., None]).sum((0, 1))
        j = torch.arange(L)
        page, slot = torch.as_tensor(kvi[kvp[r]: kvp[r + 1]]).long()[j // P], j % P
        old = torch.where(j < L - (b - a), scores[page, slot].double() * decay, 0.0) if decay else torch.zeros(L).double()
        new[page, slot] = old + w
        # 32-bit sums: a rounding of 2^-24 of the running sum per term, in chains of at most 2^9 terms a level
        bound[page, slot] = e * 1.01 + (old.abs() + w) * 2.0 ** -14
    return new, bound


def select(scores, L, keep, sink, recent):
    """Positions kept of one row, ascending: a list of Python floats in, ties to the lowest position."""
    if L <= keep:
        return list(range(L))
    rank = lambda i: (1, 0.0, i) if math.isnan(scores[i]) else (0, -scores[i], i)
    mid = sorted(range(sink, L - recent), key=rank)[: keep - sink - recent]
    return list(range(sink)) + sorted(mid) + list(range(L - recent, L))
