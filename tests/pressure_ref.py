"""Plain references, on CPU tensors and in 64 bits, of attention over shared prefixes, attention weights of cached keys
and eviction."""
import math

import torch


def rows_of(cache, table, b, n):
    """The first n positions of row b of a cache plane [N, Hkv, P, ...] -> [Hkv, n, ...] (table None: contiguous)."""
    if table is None:
        return cache[b, :, :n]
    P = cache.shape[2]
    j = torch.arange(n)
    return cache[table[b, j // P].long(), :, j % P].transpose(0, 1) if n else cache[:1, :, :0].reshape(cache.shape[1], 0, *cache.shape[3:])


def prefix(q, prefixes, own, lens, scale):
    """Attention over a prefix and own keys: q [B,Hq,Tq,D]; prefixes: (K, V) [Hkv,m,D] float64 for each prefix; own: (K, V)
    [Hkv,n,D] for each row; lens [B].  Returns (o, lse, spread, weight): spread = sum_j p_j |v_j|, what relative errors of
    the p_j are multiplied by; weight = max_j sum_d |q_d k_jd| scale, what errors of the scores are relative to."""
    B, Hq, Tq, D = q.shape
    Hkv = own[0][0].shape[0]
    o = torch.zeros(B, Hq, Tq, D, dtype=torch.float64)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64)
    spread, weight = torch.zeros_like(o), torch.zeros_like(lse)
    W = B // len(prefixes)
    for b in range(B):
        pk, pv = prefixes[b // W]
        K, V = torch.cat([pk, own[b][0]], 1), torch.cat([pv, own[b][1]], 1)
        for t in range(Tq):
            at = int(lens[b]) - Tq + t
            if at < 0:
                continue
            n = pk.shape[1] + at + 1
            x = q[b, :, t].double().reshape(Hkv, Hq // Hkv, D)
            s = torch.einsum("hgd,hkd->hgk", x, K[:, :n]) * scale
            lse[b, :, t] = torch.logsumexp(s, -1).flatten()
            p = torch.softmax(s, -1)
            o[b, :, t] = torch.einsum("hgk,hkd->hgd", p, V[:, :n]).reshape(Hq, D)
            spread[b, :, t] = torch.einsum("hgk,hkd->hgd", p, V[:, :n].abs()).reshape(Hq, D)
            weight[b, :, t] = torch.einsum("hgd,hkd->hgk", x.abs(), K[:, :n].abs()).amax(-1).flatten() * abs(scale)
    return o, lse, spread, weight


def prefix_tolerance(o, lse, spread, weight, D):
    """(of o, of lse).  A score: D products added in f32 in any order, off by at most D 2^-24 of sum |q k| (one rounding an
    addition), its factor and its exponent's argument by 2^-23 of the score and of the maximum each, exp2 by 2^-22, the
    sums of the p by 2^-20 (tens of thousands of terms in chains of at most a few hundred per thread, then trees): e.
    The p are rounded to bf16 (2^-8) before P V, o is rounded once (2^-8), and both meet e."""
    e = D * 2.0 ** -24 * weight + 2.0 ** -22 * (weight + lse.abs().clamp(max=1e30) + 1) + 2.0 ** -20
    tol_o = (2.0 ** -8 + 2 * e[..., None]) * spread + 2.0 ** -8 * (1 + 2.0 ** -7) * o.abs() + 1e-30
    return tol_o, e + 2.0 ** -22 * lse.abs().clamp(max=1e30)


def weights(q, K, lse, n, scale):
    """What one row's step adds: q [Hq,Tq,D], K [Hkv,n,D] float64, lse [Hq,Tq] -> (added [Hkv,n], tolerance of it)."""
    Hq, Tq, D = q.shape
    Hkv = K.shape[0]
    G = Hq // Hkv
    x = q.double().reshape(Hkv, G, Tq, D)
    s = torch.einsum("hgtd,hkd->hgtk", x, K) * scale
    big = torch.einsum("hgtd,hkd->hgtk", x.abs(), K.abs()) * abs(scale)
    seen = torch.arange(n)[None, :] <= (n - Tq + torch.arange(Tq))[:, None]
    e = lse.double().reshape(Hkv, G, Tq, 1)
    p = torch.where(seen & (e > -math.inf), torch.exp(s - e), torch.zeros_like(s))
    # a score: D additions in f32; its factor, the argument's rounding, exp2; G Tq additions of the sum
    rel = D * 2.0 ** -24 * big + 2.0 ** -22 * (s.abs() + torch.where(e > -math.inf, e.abs(), torch.zeros_like(e)) + 1) \
        + G * Tq * 2.0 ** -24
    return p.sum((1, 2)), (p * rel).sum((1, 2)) + 1e-38


def evict(weights, n, budget, recent, first):
    """Positions kept of one (row, head): weights [n] float32."""
    if n <= budget:
        return list(range(n))
    w = [math.inf if math.isnan(x) else x for x in weights.tolist()]
    nan = [math.isnan(x) for x in weights.tolist()]
    middle = sorted(range(first, n - recent), key=lambda j: (not nan[j], -w[j], j))
    return sorted([*range(first), *middle[:budget - first - recent], *range(n - recent, n)])
