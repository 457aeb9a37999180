"""Latent attention in 64 bits, from its definition, on host tensors: the plain implementation that
the GPU tests compare with."""
import math

import torch

LATENT, ROPE, NOPE, V = 512, 64, 128, 128


def visible(L, n, causal=True, window_left=-1):
    """[n, L]: whether new token i (position L - n + i) sees key j."""
    pos = L - n + torch.arange(n)[:, None]
    j = torch.arange(L)[None]
    see = (j <= pos) if causal else torch.ones(n, L, dtype=torch.bool)
    return see & (j >= pos - window_left) if window_left >= 0 else see


def attend(q, k, v, see, scale):
    """q [n, H, W], k [L, H or 1, W], v [L, H or 1, Dv] -> out [n, H, Dv], lse [n, H], and the sums
    sum_j p_j |v_j| that bound the output's rounding, in float64."""
    q, k, v = q.double(), k.double(), v.double()
    k, v = k.expand(-1, q.shape[1], -1), v.expand(-1, q.shape[1], -1)
    x = torch.einsum("nhw,lhw->nhl", q, k) * scale
    x = x.masked_fill(~see[:, None], -math.inf)
    p = torch.softmax(x, -1)
    return torch.einsum("nhl,lhd->nhd", p, v), torch.logsumexp(x, -1), torch.einsum("nhl,lhd->nhd", p, v.abs())


def score_error(q, k, scale):
    """How far a score of 32-bit sums may be off, per query row [n, H]: W terms, each at most |q||k|."""
    most = k.double().norm(dim=-1).max() if k.numel() else 0.0
    return q.shape[-1] * 2.0 ** -24 * q.double().norm(dim=-1) * most * scale


def _cat(parts, H, width):
    if not parts:
        e = torch.zeros(0, H, width, dtype=torch.float64)
        return e, e[..., 0], e, e[..., 0]
    return tuple(torch.cat(x) for x in zip(*parts))


def paged(q, cache, qo, kvp, kvi, lpl, scale, causal=True, window_left=-1):
    """Absorbed form over the pages: q [T, H, 576], cache [pages, P, 576] -> out, lse, sum p|v|, score error."""
    P, parts = cache.shape[1], []
    for r in range(len(kvp) - 1):
        a, b = int(qo[r]), int(qo[r + 1])
        if a == b:
            continue
        L = int((kvp[r + 1] - kvp[r] - 1) * P + lpl[r])
        x = cache[torch.as_tensor(kvi[kvp[r]: kvp[r + 1]]).long()].reshape(-1, LATENT + ROPE)[:L, None]
        parts.append((*attend(q[a:b], x, x[..., :LATENT], visible(L, b - a, causal, window_left), scale),
                      score_error(q[a:b], x, scale)))
    return _cat(parts, q.shape[1], LATENT)


def dense(q, k_nope, k_rope, v, cu_q, cu_k, scale, causal=True, window_left=-1):
    """Expanded form: q [T, H, 192], k_nope [K, H, 128], k_rope [K, 64], v [K, H, 128]."""
    H, parts = q.shape[1], []
    k = torch.cat([k_nope, k_rope[:, None].expand(-1, H, -1)], -1)
    for s in range(len(cu_q) - 1):
        a, b, c, d = int(cu_q[s]), int(cu_q[s + 1]), int(cu_k[s]), int(cu_k[s + 1])
        if a == b:
            continue
        parts.append((*attend(q[a:b], k[c:d], v[c:d], visible(d - c, b - a, causal, window_left), scale),
                      score_error(q[a:b], k[c:d], scale)))
    return _cat(parts, H, V)
