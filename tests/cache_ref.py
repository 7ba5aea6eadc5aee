"""Plain references of the cache operators, on CPU tensors, in 64 bits (and in
float32 elementary operations where the operator is defined by them)."""
import math

import numpy as np
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def plan(lens, new, table, page, free, cursor, total):
    """(slots, positions, cu, lens_out, cursor_out, table, ok per request) by a loop over requests."""
    table = table.clone()
    mp = table.shape[1]
    slots, pos, cu, out, oks = [], [], [0], [], []
    at = at_all = cursor
    tokens, stop = 0, False
    for b, (n, a) in enumerate(zip(lens.tolist(), new.tolist())):
        valid = n >= 0 and a >= 0 and n + a <= mp * page
        have = -(-n // page) if valid else 0
        need = -(-(n + a) // page) - have if valid else 0
        at_all += need
        ok = valid and tokens + max(a, 0) <= total and (at_all == cursor or (0 <= cursor and at_all <= len(free)))
        oks.append(ok)
        if ok:
            for i in range(need):
                table[b, have + i] = free[at_all - need + i]
            at = at_all
        for i in range(max(a, 0)):
            if len(slots) < total:
                p = n + i
                pg = int(table[b, p // page]) if ok else -1
                slots.append(pg * page + p % page if pg >= 0 else -1)
                pos.append(p if ok else 0)
        tokens += max(a, 0)
        cu.append(min(tokens, total))
        out.append(n + a if ok else n)
    slots += [-1] * (total - len(slots))
    pos += [0] * (total - len(pos))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return i32(slots), i32(pos), i32(cu), i32(out), i32([at]), table, oks


def rope(x, pos, tab, inter, sign=1.0, dtype=torch.float64):
    """x [..., D] rotated at pos (broadcastable to x.shape[:-1]); elementary operations in dtype."""
    x, cs = x.to(dtype), tab.to(dtype)[pos.long()]
    R = tab.shape[1]
    h = R // 2
    c, s = cs[..., :h], cs[..., h:] * sign
    y = x.clone()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :h], x[..., h:R])
    u, v = a * c - b * s, b * c + a * s
    if inter:
        y[..., 0:R:2], y[..., 1:R:2] = u, v
    else:
        y[..., :h], y[..., h:R] = u, v
    return y


def e4m3(codes):
    return codes.view(torch.float8_e4m3fn).double()


def quantise(x, scale):
    """(packed codes, scale bytes) of float32 x [..., D]: the definition, in float32 elementary operations."""
    s = np.float32(scale)
    b = x.float().unflatten(-1, (-1, 16))
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    rc = float(np.float32(1) / (np.float32(6) * s))
    sf = (torch.where(bad, 0.0, amax) * rc).clamp(max=448.0).to(torch.float8_e4m3fn)
    prod = sf.float() * float(s)
    inv = torch.where(sf.float() > 0, 1.0 / prod, 0.0)
    y = (torch.where(bad[..., None], 0.0, b) * inv[..., None]).double()
    d = (y.abs().clamp(max=6)[..., None] - E2M1).abs()      # beyond the largest level: that level
    # the nearest level, of two equally near ones the even code
    near = (d * 16 + (torch.arange(8) % 2) * 2.0 ** -30).argmin(-1)
    codes = (near | (torch.signbit(y).long() << 3)).flatten(-2).to(torch.uint8)
    sf = torch.where(bad, torch.tensor(0x7F, dtype=torch.uint8), sf.view(torch.uint8))
    return codes[..., 0::2] | (codes[..., 1::2] << 4), sf


def values(packed, sf, scale):
    """float64 values of packed codes [..., D/2] with scale bytes [..., D/16]."""
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).long()
    v = E2M1[codes & 7] * (1 - 2 * (codes >> 3)).double()
    return (v.unflatten(-1, (-1, 16)) * e4m3(sf)[..., None]).flatten(-2) * float(np.float32(scale))


def decode(q, k, v, lens, scale, tab=None):
    """Cached attention in 64 bits, any 0 <= len: q [B,Hq,Tq,D], k, v [B,Hkv,S,D] float64 ->
    (o, lse, spread, weight): spread = sum_j (p_j + 2^-15) |v_j|, what a relative error 2^-10 of every p and an
    absolute one of 2^-25 is multiplied by (over 2^-10), and weight = max_j sum_d |q_d k_jd| scale, what the products'
    accumulation error is relative to."""
    B, Hq, Tq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    o = torch.zeros(B, Hq, Tq, D, dtype=torch.float64)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=torch.float64)
    spread, weight = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        n = int(lens[b])
        for t in range(Tq):
            seen = n - Tq + t + 1
            if seen <= 0:
                continue
            x = q[b, :, t].double()
            if tab is not None:
                x = rope(x, torch.tensor(seen - 1), tab, False)
            x = x.reshape(Hkv, G, D)
            kk, vv = k[b, :, :seen], v[b, :, :seen]
            s = torch.einsum("hgd,hkd->hgk", x, kk) * scale
            lse[b, :, t] = torch.logsumexp(s, -1).flatten()
            p = torch.softmax(s, -1)
            o[b, :, t] = torch.einsum("hgk,hkd->hgd", p, vv).reshape(Hq, D)
            spread[b, :, t] = torch.einsum("hgk,hkd->hgd", p + 2.0 ** -15, vv.abs()).reshape(Hq, D)
            weight[b, :, t] = torch.einsum("hgd,hkd->hgk", x.abs(), kk.abs()).amax(-1).flatten() * abs(scale)
    return o, lse, spread, weight


def pages_to_rows(pages, table):
    """[N,Hkv,P,w] pages through a block table [B,M] -> [B,Hkv,M*P,w] (entries outside the pool: zeros)."""
    out = pages[table.long().clamp(0, pages.shape[0] - 1)]
    ok = (table >= 0) & (table < pages.shape[0])
    out = torch.where(ok[..., None, None, None], out, torch.zeros_like(out))
    return out.transpose(1, 2).flatten(2, 3)
