"""The operators of a KV cache under pressure, as cases that can be timed and compared.

Three groups: attention of a batch over a prefix that its rows share and over each row's own cache (the prefix read once
for all of them), the attention weight each cached key has received (accumulated from a step's queries and log-sum-exps;
the step's own keys start at zero), and eviction (a cache cut down to a budget of keys by those weights, in place).  ``run`` computes each either with
elementary torch operations (``own`` false) or with the calls of causal_gqa_attention_fwd_gb300 (``own`` true); ``exact``
computes it in 64 bits.

A cache is [pages, Hkv, page_size, w]; a contiguous one is the case of one page a row, page_size = S.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# cache scales as a calibration over N(0, 1) keys gives them: the largest value seen / (6 * 448), and / 448 for E4M3
KS4, KS8 = 6.6873 / 2688, 6.6873 / 448


def listed():
    return [
        # a small model's decode step: 8 requests behind one system prompt
        dict(name="prefix_t2048_b8", op="prefix", B=8, P=1, Hq=14, Hkv=2, Tq=1, D=64, page=0, Sp=2048, plo=2048, phi=2048,
             S=256, lo=1, hi=256),
        # four samples of each of 8 prompts, ragged prompts, pages of 16
        dict(name="prefix_samples_p8", op="prefix", B=32, P=8, Hq=16, Hkv=8, Tq=1, D=128, page=16, Sp=4096, plo=1001,
             phi=4001, S=512, lo=5, hi=501),
        # several new tokens a row, odd lengths
        dict(name="prefix_tq4_ragged", op="prefix", B=5, P=1, Hq=16, Hkv=4, Tq=4, D=128, page=0, Sp=3001, plo=2999, phi=2999,
             S=777, lo=4, hi=777),
        # 64 conversations over one long system prompt
        dict(name="prefix_t8192_b64", op="prefix", B=64, P=1, Hq=32, Hkv=8, Tq=1, D=128, page=64, Sp=8192, plo=8192, phi=8192,
             S=1024, lo=16, hi=1024),
        # 256 questions about one long document
        dict(name="prefix_t32k_b256", op="prefix", B=256, P=1, Hq=32, Hkv=8, Tq=1, D=128, page=64, Sp=32768, plo=32768,
             phi=32768, S=512, lo=64, hi=512),
        # the weights that one decode step of a small model adds
        dict(name="weights_t2048_b8", op="weights", fmt="bf16", B=8, Hq=14, Hkv=2, Tq=1, D=64, page=0, S=2048, lo=2048, hi=2048),
        # the last 16 queries of each prompt look over it, before its cache is cut; E4M3 keys
        dict(name="weights_window_fp8", op="weights", fmt="fp8", B=5, Hq=16, Hkv=4, Tq=16, D=128, page=0, S=7001, lo=301, hi=7001),
        # a decode step over the long-context cache
        dict(name="weights_paged_s32k", op="weights", fmt="bf16", B=8, Hq=32, Hkv=8, Tq=1, D=128, page=64, S=32768, lo=16384,
             hi=32768),
        # the same keys in 4 bits
        dict(name="weights_q4_s32k", op="weights", fmt="q4", B=8, Hq=32, Hkv=8, Tq=1, D=128, page=64, S=32768, lo=16384, hi=32768),
        # many short requests cut to 256 keys, E4M3, pages of 16; some are short enough already
        dict(name="evict_fp8_b64", op="evict", fmt="fp8", B=64, Hkv=2, D=128, page=16, S=1024, lo=1, hi=1024, budget=256,
             recent=64, first=4),
        # a small model's caches cut by half
        dict(name="evict_t2048_b8", op="evict", fmt="bf16", B=8, Hkv=2, D=64, page=0, S=2048, lo=2048, hi=2048, budget=1024,
             recent=101, first=0),
        # long contexts cut to 4099 keys each
        dict(name="evict_paged_s32k", op="evict", fmt="bf16", B=4, Hkv=8, D=128, page=64, S=32768, lo=16384, hi=32768, budget=4099,
             recent=1024, first=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "weights", "evict"])
    D, Hkv, page = rng.choice([64, 128]), rng.choice([1, 2, 3, 8]), rng.choice([0, 16, 32, 64, 128])
    up = lambda s: -(-s // page) * page if page else s  # noqa: E731
    if op == "prefix":
        P, G, Tq = rng.choice([1, 1, 1, 2, 5]), rng.choice([1, 2, 4, 7, 8]), rng.choice([1, 1, 1, 2, 5])
        B = P * _log(rng, 1, 256 // P)
        Sp = _log(rng, 16, 32768)
        Sp = max(16, min(Sp, (1 << 28) // (B * Hkv * G * Tq)))
        S = max(Tq, min(_log(rng, 1, 2048), (1 << 19) // (B * Hkv)))
        return dict(op=op, B=B, P=P, Hq=Hkv * G, Hkv=Hkv, Tq=Tq, D=D, page=page, Sp=up(Sp), plo=rng.randint(1, Sp), phi=Sp,
                    S=up(S), lo=rng.randint(Tq, S), hi=S)
    B, S = _log(rng, 1, 64), _log(rng, 16, 32768)
    if op == "weights":
        G, Tq, fmt = rng.choice([1, 4, 7, 8]), rng.choice([1, 1, 1, 2, 5, 16]), rng.choice(["bf16", "bf16", "fp8", "q4"])
        S = max(Tq, min(S, 2000000 // (B * Hkv * max(1, G * Tq // 8))))
        return dict(op=op, fmt=fmt, B=B, Hq=Hkv * G, Hkv=Hkv, Tq=Tq, D=D, page=page, S=up(S), lo=rng.randint(Tq, S), hi=S)
    S = max(16, min(S, 1000000 // (B * Hkv)))
    budget = _log(rng, 4, max(4, S // 2))
    recent = rng.randint(0, budget // 2)
    return dict(op=op, fmt=rng.choice(["bf16", "fp8"]), B=B, Hkv=Hkv, D=D, page=page, S=up(S), lo=rng.randint(1, S), hi=S,
                budget=budget, recent=recent, first=rng.randint(0, min(4, budget - recent)))


# ---------------------------------------------------------------- inputs
def _spread(lo, hi, n, g):
    """n whole numbers spread evenly over [lo, hi], in an order drawn from g (so their sum is the case's alone)."""
    x = torch.linspace(lo, hi, n, dtype=torch.float64).round().to(torch.int32) if n > 1 else torch.tensor([hi], dtype=torch.int32)
    return x[torch.randperm(n, generator=g)]


def _lens(lo, hi, n):
    return _spread(lo, hi, n, torch.Generator().manual_seed(0)).tolist()


def _quant4(x, ks):
    """4-bit codes (packed) and block scales of float32 x [..., D]."""
    b = x.unflatten(-1, (-1, 16))
    sf = (b.abs().amax(-1) / (6 * ks)).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = b / (sf.float() * ks).clamp(min=1e-20)[..., None]
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    c = (torch.bucketize(y.abs(), mid).to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), sf.view(torch.uint8)


def _cache(fmt, rn, pages, H, page, D):
    """Planes of one side (keys, or values) of a cache of N(0, 1) entries, made a part at a time."""
    parts = []
    for m in torch.arange(pages).split(max(1, (1 << 25) // (H * page * D))):
        x = rn(len(m), H, page, D)
        parts.append(_quant4(x, KS4) if fmt == "q4" else (x.bfloat16(),) if fmt == "bf16" else
                     ((x / KS8).to(torch.float8_e4m3fn).view(torch.uint8),))
    return [torch.cat(p) for p in zip(*parts)]


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gd, device="cuda")  # noqa: E731
    st, op = dict(case), case["op"]
    B, Hkv, D, page, S = (case[n] for n in ("B", "Hkv", "D", "page", "S"))
    st.update(lens=_spread(case["lo"], case["hi"], B, g).cuda(), bt=None)
    extra = case["P"] * (case["Sp"] // page) if op == "prefix" and page else 0
    rows, per = (B, S) if not page else (B * (S // page) + extra + 3, page)
    if page:
        perm = torch.randperm(rows, generator=g).to(torch.int32).cuda()
        st["bt"] = perm[:B * (S // page)].reshape(B, -1).contiguous()
    if op != "evict":
        Hq, Tq = case["Hq"], case["Tq"]
        st.update(q=rn(B, Hq, Tq, D).bfloat16(), scale=1.0 / math.sqrt(D))
    if op == "prefix":
        P, Sp = case["P"], case["Sp"]
        st.update(k=_cache("bf16", rn, rows, Hkv, per, D)[0], v=_cache("bf16", rn, rows, Hkv, per, D)[0],
                  plens=_spread(case["plo"], case["phi"], P, g).cuda(),
                  o=torch.empty(B, Hq, Tq, D, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(B, Hq, Tq, device="cuda"))
        if page:
            st["pt"] = perm[B * (S // page):B * (S // page) + extra].reshape(P, -1).contiguous()
        else:
            st.update(kp=_cache("bf16", rn, P, Hkv, Sp, D)[0], vp=_cache("bf16", rn, P, Hkv, Sp, D)[0])
        return st
    if op == "weights":
        st.update(k=_cache(case["fmt"], rn, rows, Hkv, per, D), ks=dict(bf16=1.0, fp8=KS8, q4=KS4)[case["fmt"]],
                  # what an earlier step has left
                  weights=torch.rand(rows, Hkv, per, generator=gd, device="cuda") * (2.0 * Hq // Hkv * Tq / S))
        # the step's log-sum-exps, as its attention wrote them
        lse = torch.empty(B, Hq, Tq, device="cuda")
        for b in range(B):
            s, seen = _scores(st, b)
            lse[b] = torch.logsumexp(s.masked_fill(~seen, -math.inf), -1).reshape(Hq, Tq)
        st["lse"] = lse
        return st
    # accumulated attention weights are heavy-tailed: a few keys hold most
    st.update(k=_cache(case["fmt"], rn, rows, Hkv, per, D), v=_cache(case["fmt"], rn, rows, Hkv, per, D),
              weights=torch.exp(1.5 * rn(rows, Hkv, per)))
    return st


# ---------------------------------------------------------------- one pass
def _values(st, planes):
    """float32 values of a cache's planes, before its scale."""
    if st["fmt"] == "bf16":
        return planes[0].float()
    if st["fmt"] == "fp8":
        return planes[0].view(torch.float8_e4m3fn).float()
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=planes[0].device)
    c = torch.stack([planes[0] & 15, planes[0] >> 4], -1).flatten(-2)
    return (lut[c.int()].unflatten(-1, (-1, 16)) * planes[1].view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _row(x, bt, b):
    """Row b's entries of a plane [pages, Hkv, page, ...] as [Hkv, S, ...]."""
    return x[b] if bt is None else x[bt[b].long()].transpose(0, 1).flatten(1, 2)


def _rows(x, bt):
    """Every row's entries of a plane as [B, Hkv, S, ...]."""
    return x if bt is None else x[bt.long()].transpose(1, 2).flatten(2, 3)


def _scores(st, b):
    """Row b's scores [Hkv, G * Tq, S] in float32, and which are seen."""
    Hkv, Tq, D, S = st["Hkv"], st["Tq"], st["D"], st["S"]
    kk = _values(st, [_row(p, st["bt"], b) for p in st["k"]])
    s = torch.matmul(st["q"][b].float().reshape(Hkv, -1, D), kk.transpose(-1, -2)) * (st["scale"] * st["ks"])
    t = torch.arange(Tq, device=s.device).repeat(st["Hq"] // Hkv)
    return s, torch.arange(S, device=s.device) <= (st["lens"][b] - Tq + t)[:, None]


def _plain_prefix(st):
    B, P, Hq, Hkv, Tq, D = (st[n] for n in ("B", "P", "Hq", "Hkv", "Tq", "D"))
    G, W = Hq // Hkv, B // P
    kp, vp = (st["kp"], st["vp"]) if not st["page"] else (_rows(st["k"], st["pt"]), _rows(st["v"], st["pt"]))
    k, v = _rows(st["k"], st["bt"]).float(), _rows(st["v"], st["bt"]).float()
    q = st["q"].float().reshape(P, W, Hkv, G * Tq, D)
    dev = q.device
    # the prefix: all rows of a group in one product
    sp = torch.matmul(q.transpose(1, 2).reshape(P, Hkv, -1, D), kp.float().transpose(-1, -2)) * st["scale"]
    sp = sp.masked_fill(torch.arange(sp.shape[-1], device=dev) >= st["plens"].long()[:, None, None, None], -math.inf)
    # each row's own keys
    so = torch.matmul(q.reshape(B, Hkv, G * Tq, D), k.transpose(-1, -2)) * st["scale"]
    pos = st["lens"].long()[:, None] - Tq + torch.arange(Tq, device=dev).repeat(G)
    so = so.masked_fill(torch.arange(so.shape[-1], device=dev) > pos[:, None, :, None], -math.inf)
    own_rows = lambda x: x.reshape(P, Hkv, W, G * Tq, -1).transpose(1, 2).reshape(B, Hkv, G * Tq, -1)  # noqa: E731
    mp = sp.amax(-1, keepdim=True)
    m = torch.maximum(own_rows(mp), so.amax(-1, keepdim=True))
    pp, po = torch.exp(sp - mp), torch.exp(so - m)
    c = torch.exp(own_rows(mp) - m)
    l = own_rows(pp.sum(-1, keepdim=True)) * c + po.sum(-1, keepdim=True)
    o = (own_rows(torch.matmul(pp, vp.float())) * c + torch.matmul(po, v)) / l
    return o.reshape(B, Hq, Tq, D).bfloat16(), (m + torch.log(l)).reshape(B, Hq, Tq)


def _plain_weights(st):
    w, bt, page = st["weights"], st["bt"], st["page"]
    for b in range(st["B"]):
        s, seen = _scores(st, b)
        p = torch.exp(s - st["lse"][b].reshape(st["Hkv"], -1, 1)).masked_fill(~seen, 0.0).sum(-2)
        # the step's new keys had no weight before
        n = st["lens"][b]
        j = torch.arange(st["S"], device=w.device)
        old = _row(w, bt, b)
        p = torch.where(j < n - st["Tq"], old + p, torch.where(j < n, p, old))
        if bt is None:
            w[b] = p
        else:
            w[bt[b].long()] = p.unflatten(-1, (-1, page)).transpose(0, 1)
    return w


def _plain_evict(st):
    B, Hkv, S, budget, bt, page = (st[n] for n in ("B", "Hkv", "S", "budget", "bt", "page"))
    n = st["lens"].long()[:, None, None]
    j = torch.arange(S, device=n.device)
    key = _rows(st["weights"], bt)
    key = key.masked_fill((j < st["first"]) | (j >= n - st["recent"]), math.inf).masked_fill(j >= n, -math.inf)
    top = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]   # equal weights: the lowest position
    keep = torch.zeros(B, Hkv, S, dtype=torch.bool, device=n.device).scatter_(-1, top, True) & (j < n)
    src = torch.sort(torch.where(keep, j, S), dim=-1).values[..., :budget]
    live = src < S
    # the kept rows' places: (page or batch row, head, row in it)
    b = torch.arange(B, device=n.device)[:, None, None].expand_as(src)[live]
    h = torch.arange(Hkv, device=n.device)[None, :, None].expand_as(src)[live]
    at, to = src[live], torch.arange(src.shape[-1], device=n.device).expand_as(src)[live]
    place = (lambda x: (b, h, x)) if bt is None else (lambda x: (bt.long()[b, x // page], h, x % page))
    for x in (st["weights"], *st["k"], *st["v"]):
        x[place(to)] = x[place(at)]
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device=n.device)
    kept[..., :src.shape[-1]] = torch.where(live, src, -1).to(torch.int32)
    return kept, st["lens"].clamp(max=budget)


def _planes(st):
    """The cache's planes as values."""
    return [x.view(torch.float8_e4m3fn) if st["fmt"] == "fp8" else x for x in (*st["k"], *st["v"])]


def run(st):
    op = st["op"]
    if own:
        import causal_gqa_attention_fwd_gb300 as g
        if op == "prefix":
            kw = dict(scale=st["scale"], o=st["o"], lse=st["lse"])
            if st["page"]:
                return g.attn_decode_paged_prefix_fwd(st["q"], st["k"], st["v"], st["pt"], st["plens"], st["bt"], st["lens"], **kw)
            return g.attn_decode_prefix_fwd(st["q"], st["kp"], st["vp"], st["plens"], st["k"], st["v"], st["lens"], **kw)
        if op == "weights":
            kw = dict(block_table=st["bt"], scale=st["scale"])
            if st["fmt"] == "bf16":
                return g.attn_cache_weights(st["q"], *st["k"], st["lse"], st["lens"], st["weights"], **kw)
            f = g.attn_cache_weights_fp8 if st["fmt"] == "fp8" else g.attn_cache_weights_q4
            return f(st["q"], *st["k"], st["ks"], st["lse"], st["lens"], st["weights"], **kw)
        kept, lens = g.attn_cache_evict(st["weights"], (*st["k"], *st["v"]), st["lens"], st["budget"], recent=st["recent"],
                                        first=st["first"], block_table=st["bt"])
        return [kept, lens, st["weights"], *_planes(st)]
    if op == "prefix":
        return _plain_prefix(st)
    if op == "weights":
        return _plain_weights(st)
    return [*_plain_evict(st), st["weights"], *_planes(st)]


# ---------------------------------------------------------------- sizes
def work(case):
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    lens = _lens(case["lo"], case["hi"], case["B"])
    if op == "evict":
        wide = 2 * D * dict(bf16=2, fp8=1)[case["fmt"]]            # a position's keys and values of one head
        cut = [n for n in lens if n > case["budget"]]
        moved = len(cut) * (case["budget"] - case["first"])        # the first positions stay where they are
        kept = len(lens) * case["budget"]
        return dict(bytes=Hkv * (4 * sum(cut) + moved * (2 * wide + 4) + 4 * kept) + 8 * len(lens), flops=0)
    rows = case["B"] * case["Hq"] * case["Tq"]
    if op == "weights":
        wide = D * dict(bf16=2, fp8=1, q4=0.5625)[case["fmt"]]
        return dict(bytes=sum(lens) * Hkv * (wide + 8) + rows * (2 * D + 4), flops=2 * sum(lens) * case["Hq"] * case["Tq"] * D)
    pl = _lens(case["plo"], case["phi"], case["P"])
    return dict(bytes=(sum(lens) + sum(pl)) * Hkv * D * 4 + rows * (4 * D + 4),
                flops=4 * D * case["Hq"] * case["Tq"] * (sum(lens) + sum(pl) * (case["B"] // case["P"])))


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, B, Hkv, page = case["op"], case["B"], case["Hkv"], case["page"]
    dev = st["lens"].device
    lens = st["lens"].tolist()

    def slots(table, n):
        """(page, row in the page) of positions 0..n-1."""
        j = torch.arange(n, device=dev)
        return (table[j // page].long(), j % page)

    def keys(x, b, n):
        """Row b's first n entries of a plane, [n, Hkv, ...]."""
        if st["bt"] is None:
            return x[b, :, :n].transpose(0, 1)
        p, r = slots(st["bt"][b], n)
        return x[p, :, r]

    if op == "prefix":
        Hq, Tq, D, G, W = case["Hq"], case["Tq"], case["D"], case["Hq"] // Hkv, B // case["P"]
        o, lse = torch.zeros(B, Hq, Tq, D, dtype=torch.float64), torch.zeros(B, Hq, Tq, dtype=torch.float64)
        for b in range(B):
            n, m = lens[b], int(st["plens"][b // W])
            if page:
                p, r = slots(st["pt"][b // W], m)
                pk, pv = st["k"][p, :, r], st["v"][p, :, r]
            else:
                pk, pv = (st[x][b // W, :, :m].transpose(0, 1) for x in ("kp", "vp"))
            K = torch.cat([pk, keys(st["k"], b, n)]).double().transpose(0, 1).contiguous()
            V = torch.cat([pv, keys(st["v"], b, n)]).double().transpose(0, 1).contiguous()
            x = st["q"][b].double().reshape(Hkv, G, Tq, D)
            for t in range(Tq):
                seen = m + n - Tq + t + 1
                s = torch.einsum("hgd,hkd->hgk", x[:, :, t], K[:, :seen]) * st["scale"]
                lse[b, :, t] = torch.logsumexp(s, -1).flatten().cpu()
                o[b, :, t] = torch.einsum("hgk,hkd->hgd", torch.softmax(s, -1), V[:, :seen]).reshape(Hq, D).cpu()
        return o, lse
    if op == "weights":
        Hq, Tq, D, G = case["Hq"], case["Tq"], case["D"], case["Hq"] // Hkv
        grid = torch.tensor(E2M1, dtype=torch.float64, device=dev)
        grid = torch.cat([grid, -grid])
        w = st["weights"].double()
        for b in range(B):
            n = lens[b]
            K = keys(st["k"][0], b, n)
            if case["fmt"] == "bf16":
                K = K.double()
            elif case["fmt"] == "fp8":
                K = K.view(torch.float8_e4m3fn).double() * st["ks"]
            else:
                sf = keys(st["k"][1], b, n).contiguous().view(torch.float8_e4m3fn).double() * st["ks"]
                K = torch.stack([grid[(K & 15).long()], grid[(K >> 4).long()]], -1).flatten(-2) * sf.repeat_interleave(16, -1)
            add = torch.zeros(n, Hkv, dtype=torch.float64, device=dev)
            for t in range(Tq):
                seen = n - Tq + t + 1
                q = st["q"][b, :, t].double().reshape(Hkv, G, D)
                s = torch.einsum("hgd,khd->khg", q, K[:seen]) * st["scale"] - st["lse"][b, :, t].double().reshape(Hkv, G)
                add[:seen] += torch.exp(s).sum(-1)
            add[:max(n - Tq, 0)] += keys(w, b, n)[:max(n - Tq, 0)]       # what was there: of all but the Tq new keys
            if page:
                p, r = slots(st["bt"][b], n)
                w[p, :, r] = add
            else:
                w[b, :, :n] = add.t()
        return w
    budget, recent, first = case["budget"], case["recent"], case["first"]
    import numpy as np
    kept = np.full((B, Hkv, budget), -1, dtype=np.int32)
    for b in range(B):
        n = lens[b]
        weights = keys(st["weights"], b, n).t().cpu().numpy()
        for h in range(Hkv):
            if n <= budget:
                kept[b, h, :n] = np.arange(n)
                continue
            middle = np.arange(first, n - recent)
            order = np.lexsort((middle, -weights[h][middle].astype(np.float64)))    # by weight, then by position
            best = np.sort(middle[order[:budget - first - recent]])
            kept[b, h] = np.concatenate([np.arange(first), best, np.arange(n - recent, n)])
    planes = [st["weights"], *_planes(st)]
    for b in range(B):
        if lens[b] <= budget:
            continue
        p, r = slots(st["bt"][b], lens[b]) if page else (torch.full((lens[b],), b, device=dev), torch.arange(lens[b], device=dev))
        for h in range(Hkv):
            at = torch.from_numpy(kept[b, h]).long().to(dev)
            for x in planes:
                y = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
                y[p[:budget], h, r[:budget]] = y[p[at], h, r[at]].clone()
    return [torch.from_numpy(kept), torch.tensor([min(n, budget) for n in lens], dtype=torch.int32), *planes]
