"""The operators that fill and read a KV cache, as cases that can be timed and compared.

Four groups, in the order a serving step runs them: the cache plan (block table, slots and positions from request
lengths), rotary positions (forward, backward, scaled tables), appending keys and values to a cache (bf16, E4M3 or 4-bit)
and attention over a 4-bit cache.  ``run`` computes each either with elementary torch operations (``own`` false) or with
the calls of causal_gqa_attention_fwd_gb300 (``own`` true); ``exact`` computes it in 64 bits.

The 4-bit format: two E2M1 codes a byte (feature 2i in the low half), one E4M3 scale for 16 consecutive features, one
float32 scale for the cache; value = e2m1 * e4m3 * scale.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# cache scales as a calibration over N(0, 1) keys and values gives them: the largest value seen / (6 * 448)
KS, VS = 6.6873 / 2688, 5.4917 / 2688


def listed():
    return [
        # a decode step of 64 running requests, each one token further (most need no page)
        dict(name="plan_decode_b64", op="plan", B=64, page=64, max_pages=512, lo=1, hi=20000, new_lo=1, new_hi=1),
        # 512 requests admitted at once: ragged prompts, some of them continuing a cached prefix
        dict(name="plan_prompts_b512", op="plan", B=512, page=16, max_pages=256, lo=0, hi=1500, new_lo=1, new_hi=1000),
        # rotary positions of one decode step, small model
        dict(name="rope_decode_b8", op="rope", B=8, T=1, Hq=14, Hkv=2, D=64, R=64, inter=False, bwd=False, packed=True),
        # the long-context layer's prompt
        dict(name="rope_t4096", op="rope", B=2, T=4096, Hq=32, Hkv=8, D=128, R=128, inter=False, bwd=False, packed=False),
        # gradients of a packed batch; pairs of neighbours, half of the head rotated
        dict(name="rope_bwd_packed", op="rope", B=1, T=16411, Hq=16, Hkv=8, D=128, R=64, inter=True, bwd=True, packed=True),
        # table for a context extended 32-fold, by parts
        dict(name="rope_table_131072", op="table", n=131072, R=128, base=500000.0, factor=32.0, orig=4096, low=1.0,
             high=4.0, mscale=1.1),
        # new keys and values of a decode step, rotated on the way into the 4-bit cache
        dict(name="append_q4_b64", op="append", fmt="q4", tokens=64, Hkv=8, D=128, page=64, R=128, inter=False, pad=0),
        # packed prompts into 16-position pages, a padded tail
        dict(name="append_q4_prompts", op="append", fmt="q4", tokens=16411, Hkv=8, D=128, page=16, R=64, inter=True, pad=101),
        # cached attention: the batch-8 steady decode of a small model (context 2048)
        dict(name="decode_q4_t2048_b8", op="decode", B=8, Hq=14, Hkv=2, Tq=1, S=2048, D=64, page=0, lo=2048, hi=2048, rope=False),
        # several new tokens a row, odd and short lengths among them
        dict(name="decode_q4_tq4_ragged", op="decode", B=5, Hq=16, Hkv=4, Tq=4, S=3001, D=128, page=0, lo=4, hi=3001, rope=False),
        # many short requests over small pages
        dict(name="decode_q4_paged_b64", op="decode", B=64, Hq=32, Hkv=8, Tq=1, S=1024, D=128, page=16, lo=1, hi=1024, rope=True),
        # the long-context cache
        dict(name="decode_q4_paged_s32k", op="decode", B=8, Hq=32, Hkv=8, Tq=1, S=32768, D=128, page=64, lo=16384, hi=32768, rope=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "table", "append", "append", "decode", "decode", "decode"])
    if op == "plan":
        page, decode = rng.choice([16, 32, 64, 128]), rng.random() < 0.5
        hi = _log(rng, 1, 4000)
        return dict(op=op, B=_log(rng, 1, 512), page=page, max_pages=-(-6000 // page), lo=0, hi=hi, new_lo=1,
                    new_hi=1 if decode else _log(rng, 2, 1000))
    if op == "rope":
        D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 8])
        R = rng.choice([D, D, D // 2, D // 4])
        return dict(op=op, B=rng.randint(1, 4), T=_log(rng, 1, 4096), Hq=Hkv * rng.choice([1, 3, 4]), Hkv=Hkv, D=D, R=R,
                    inter=rng.random() < 0.5, bwd=rng.random() < 0.5, packed=rng.random() < 0.5)
    if op == "table":
        orig = rng.choice([0, 2048, 8192])
        return dict(op=op, n=_log(rng, 100, 131072), R=rng.choice([16, 32, 64, 128]), base=rng.choice([10000.0, 1000000.0]),
                    factor=round(rng.uniform(1.0, 40.0), 2), orig=orig, low=1.0, high=rng.choice([4.0, 32.0]),
                    mscale=round(rng.uniform(1.0, 1.4), 3))
    if op == "append":
        D, tokens = rng.choice([64, 128]), _log(rng, 1, 16000)
        return dict(op=op, fmt=rng.choice(["q4", "q4", "fp8", "bf16"]), tokens=tokens, Hkv=rng.choice([1, 2, 8]), D=D,
                    page=rng.choice([16, 32, 64, 256]), R=rng.choice([0, D, D // 2]), inter=rng.random() < 0.5,
                    pad=rng.choice([0, tokens // 5]))
    D, Hkv, Tq = rng.choice([64, 128]), rng.choice([1, 2, 8]), rng.choice([1, 1, 1, 2, 3, 5])
    B, S, G = _log(rng, 1, 64), _log(rng, 16, 32768), rng.choice([1, 4, 7, 8])
    S = max(Tq, min(S, 700000 // (B * Hkv * max(1, G * Tq // 8))))
    page = rng.choice([0, 16, 32, 64, 128])
    if page:
        S = -(-S // page) * page
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, Tq=Tq, S=S, D=D, page=page,
                lo=rng.randint(Tq, S), hi=S, rope=rng.random() < 0.4)


# ---------------------------------------------------------------- inputs
def _spread(lo, hi, n, g):
    """n whole numbers spread evenly over [lo, hi], in an order drawn from g (so their sum is the case's alone)."""
    x = torch.linspace(lo, hi, n, dtype=torch.float64).round().to(torch.int32) if n > 1 else torch.tensor([hi], dtype=torch.int32)
    return x[torch.randperm(n, generator=g)]


def _total(lo, hi, n):
    return int(_spread(lo, hi, n, torch.Generator().manual_seed(0)).sum())


def _table64(n, R, base=10000.0, device="cuda"):
    inv = base ** (-2.0 * torch.arange(R // 2, dtype=torch.float64, device=device) / R)
    ang = torch.arange(n, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([torch.cos(ang), torch.sin(ang)], 1)


def _levels(x):
    """Codes of the nearest E2M1 values of |x| (ties to the even code), then the sign bit."""
    a = x.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return c.to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)


def _quant(x, ks):
    """(codes uint8 [..., D], scales uint8 [..., D/16]) of float32 x."""
    b = x.unflatten(-1, (-1, 16))
    amax = b.abs().amax(-1)
    rc = float(torch.tensor(1.0) / (6.0 * torch.tensor(ks, dtype=torch.float32)))
    sf8 = (amax * rc).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = sf8.float()
    inv = torch.where(sf > 0, 1.0 / (sf * ks), torch.zeros_like(sf))
    return _levels(b * inv[..., None]).flatten(-2), sf8.view(torch.uint8)


def _pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _codes(p):
    return torch.stack([p & 15, p >> 4], -1).flatten(-2)


def _values(p, sf8):
    """e2m1 * e4m3 in float32 of packed codes and scale bytes."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=p.device)
    v = lut[_codes(p).int()].unflatten(-1, (-1, 16))
    return (v * sf8.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gd, device="cuda")  # noqa: E731
    st = dict(case)
    op = case["op"]
    if op == "plan":
        B, page, mp = case["B"], case["page"], case["max_pages"]
        lens, new = _spread(case["lo"], case["hi"], B, g), _spread(case["new_lo"], case["new_hi"], B, g)
        have = (lens + page - 1) // page
        need = (lens + new + page - 1) // page - have
        total = int(have.sum() + need.sum())
        perm = torch.randperm(total + 64, generator=g).to(torch.int32)
        table = torch.full((B, mp), -1, dtype=torch.int32)
        cut = torch.cumsum(have, 0)
        for b in range(B):
            table[b, :int(have[b])] = perm[int(cut[b]) - int(have[b]):int(cut[b])]
        st.update(lens=lens.cuda(), new=new.cuda(), table=table.cuda(), free=perm[int(have.sum()):].cuda(),
                  cursor=torch.zeros(1, dtype=torch.int32, device="cuda"), total=int(new.sum()) + 7)
    elif op == "rope":
        B, T, Hq, Hkv, D = (case[n] for n in ("B", "T", "Hq", "Hkv", "D"))
        if case["packed"]:      # views of one fused projection's output
            x = rn(B * T, Hq + 2 * Hkv, D).bfloat16()
            q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
            pos = torch.randint(0, 8192, (B * T,), generator=gd, device="cuda", dtype=torch.int32)
        else:
            q, k = rn(B, Hq, T, D).bfloat16(), rn(B, Hkv, T, D).bfloat16()
            pos = torch.randint(0, 8192 - T + 1, (B, 1), generator=gd, device="cuda", dtype=torch.int32) + \
                torch.arange(T, device="cuda", dtype=torch.int32)
        st.update(q=q, k=k, pos=pos.contiguous(), tab=_table64(8192, case["R"]).float(),
                  qo=torch.empty(q.shape, dtype=q.dtype, device="cuda"), ko=torch.empty(k.shape, dtype=k.dtype, device="cuda"))
    elif op == "table":
        st.update(base_=case["base"] * (1.0 + (seed % 1000) * 1e-4), out=torch.empty(case["n"], case["R"], device="cuda"))
    elif op == "append":
        n, H, D, page, R = case["tokens"], case["Hkv"], case["D"], case["page"], case["R"]
        pages = -(-n // page) + 3
        x = rn(n, 2 * H, D).bfloat16()
        slots = (torch.randperm(pages, generator=g)[:, None] * page + torch.arange(page)).flatten()[:n].to(torch.int32)
        if case["pad"]:
            slots[n - case["pad"]:] = -1
        z = lambda w: torch.zeros(pages, H, page, w, dtype=torch.uint8, device="cuda")  # noqa: E731
        cache = {"q4": lambda: [z(D // 2), z(D // 16), z(D // 2), z(D // 16)], "fp8": lambda: [z(D), z(D)],
                 "bf16": lambda: [z(D).bfloat16(), z(D).bfloat16()]}[case["fmt"]]()
        st.update(k=x[:, :H], v=x[:, H:], slots=slots.cuda(), cache=cache,
                  ks=KS if case["fmt"] == "q4" else 6 * KS, vs=VS if case["fmt"] == "q4" else 6 * VS,
                  pos=torch.randint(0, 8192, (n,), generator=gd, device="cuda", dtype=torch.int32),
                  tab=_table64(8192, R).float() if R else None)
    else:
        B, Hq, Hkv, Tq, S, D, page = (case[n] for n in ("B", "Hq", "Hkv", "Tq", "S", "D", "page"))
        lens = _spread(case["lo"], case["hi"], B, g)
        ks, vs = KS, VS
        rows = [(B, Hkv, S)] if not page else [(B * (S // page) + 3, Hkv, page)]
        cache = []
        for s in (ks, vs):
            p, f = [], []
            for m in torch.arange(rows[0][0]).split(max(1, (1 << 24) // (Hkv * rows[0][2] * D))):
                c, e = _quant(rn(len(m), Hkv, rows[0][2], D), s)
                p.append(_pack(c))
                f.append(e)
            cache += [torch.cat(p), torch.cat(f)]
        st.update(cache=cache, ks=ks, vs=vs, lens=lens.cuda(), q=rn(B, Hq, Tq, D).bfloat16(),
                  tab=_table64(S, D).float() if case["rope"] else None,
                  o=torch.empty(B, Hq, Tq, D, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.empty(B, Hq, Tq, device="cuda"), scale=1.0 / math.sqrt(D))
        if page:
            st["bt"] = torch.randperm(rows[0][0], generator=g)[:B * (S // page)].reshape(B, -1).to(torch.int32).cuda()
    return st


# ---------------------------------------------------------------- one pass
def _turn(x, c, s, R, inter, back=False):
    """x rotated: c, s broadcast against x[..., :R/2]; the features from R on stay."""
    if back:
        s = -s
    if inter:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., R:]], -1) if R < x.shape[-1] else y


def _plain_plan(st):
    page, B = st["page"], st["B"]
    lens, new, free, mp, N = st["lens"].long(), st["new"].long(), st["free"], st["max_pages"], st["total"]
    have = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - have
    end = torch.cumsum(need, 0)
    table = st["table"]
    col = torch.arange(mp, device=table.device)[None]
    at = (end - need + int(st["cursor"]))[:, None] + col - have[:, None]
    isnew = (col >= have[:, None]) & (col < (have + need)[:, None])
    table = torch.where(isnew, free[at.clamp(0, free.numel() - 1)], table)
    cu = torch.zeros(B + 1, dtype=torch.int64, device=table.device)
    cu[1:] = torch.cumsum(new, 0)
    tok = torch.arange(N, device=table.device)
    b = torch.searchsorted(cu, tok, right=True) - 1
    ok = b < B
    bb = b.clamp(max=B - 1)
    pos = torch.where(ok, lens[bb] + tok - cu[bb], 0)
    slot = torch.where(ok, table[bb, pos // page].long() * page + pos % page, -1)
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return [i32(slot), i32(pos), i32(cu), i32(lens + new), i32(st["cursor"] + end[-1]), table]


def _inv_freq(R, base, factor, orig, low, high, dtype, device):
    """Angle of each pair a position: scaled for wavelengths long against the original context, blended between."""
    inv = base ** (-2.0 * torch.arange(R // 2, dtype=dtype, device=device) / R)
    if not orig:
        return inv / factor
    turns = orig * inv / (2 * math.pi)
    keep = ((turns - low) / (high - low)).clamp(0, 1)
    return inv * keep + inv / factor * (1 - keep)


def _plain_append(st, k, v):
    fmt, slots, page = st["fmt"], st["slots"].long(), st["page"]
    if st["R"]:
        h = st["R"] // 2
        cs = st["tab"][st["pos"].long()][:, None]
        k = _turn(k, cs[..., :h], cs[..., h:], st["R"], st["inter"])
    live = slots >= 0
    pg, off = slots[live] // page, slots[live] % page
    if fmt == "bf16":
        for c, x in zip(st["cache"], (k, v)):
            c[pg, :, off] = x[live].bfloat16()
        return list(st["cache"])
    if fmt == "fp8":
        for c, x, s in zip(st["cache"], (k, v), (st["ks"], st["vs"])):
            r = float(torch.tensor(1.0) / torch.tensor(s, dtype=torch.float32))
            c[pg, :, off] = (x[live] * r).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return [c.view(torch.float8_e4m3fn) for c in st["cache"]]
    out = []
    for i, (x, s) in enumerate(((k, st["ks"]), (v, st["vs"]))):
        c, f = _quant(x, s)
        p = _pack(c)
        st["cache"][2 * i][pg, :, off] = p[live]
        st["cache"][2 * i + 1][pg, :, off] = f[live]
        out.append(torch.where(live[:, None, None], _values(p, f) * s, 0.0).bfloat16())
    return out


def _attend(q, kv, st, dtype):
    """Cached attention on a cache's values (K and V before their float32 scale), in `dtype`."""
    B, Hq, Tq, D = q.shape
    K, V = kv
    Hkv, S = K.shape[1], K.shape[2]
    lens = st["lens"].long()
    qpos = lens[:, None] - Tq + torch.arange(Tq, device=q.device)          # [B, Tq]
    q = q.to(dtype)
    if st["tab"] is not None:
        cs = st["tab"].to(dtype)[qpos][:, None]
        q = _turn(q, cs[..., :D // 2], cs[..., D // 2:], D, False)
    q = q.reshape(B, Hkv, Hq // Hkv * Tq, D)
    s = torch.matmul(q, K.transpose(-1, -2)).reshape(B, Hkv, Hq // Hkv, Tq, S) * (st["scale"] * st["ks"])
    seen = torch.arange(S, device=q.device) <= qpos[..., None]               # [B, Tq, S]
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul((p / l).reshape(B, Hkv, -1, S), V) * st["vs"]
    return o.reshape(B, Hq, Tq, D), (m + torch.log(l)).reshape(B, Hq, Tq)


def _rows(st, i):
    """The cache's tensor i as [B, Hkv, S, w]."""
    c = st["cache"][i]
    if st["page"]:
        c = c[st["bt"].long()].transpose(1, 2).flatten(2, 3)
    return c


def run(st):
    op = st["op"]
    if own:
        import causal_gqa_attention_fwd_gb300 as g
        if op == "plan":
            return list(g.attn_cache_plan(st["lens"], st["new"], st["table"], st["page"], st["free"], st["cursor"],
                                          st["total"])) + [st["table"]]
        if op == "rope":
            f = g.attn_rope_bwd if st["bwd"] else g.attn_rope
            return f(st["q"], st["k"], st["pos"], st["tab"], st["inter"], st["qo"], st["ko"])
        if op == "table":
            return g.attn_rope_table(st["n"], st["R"], base=st["base_"], factor=st["factor"], original_positions=st["orig"],
                                     low_turns=st["low"], high_turns=st["high"], mscale=st["mscale"], out=st["out"])
        if op == "append":
            kw = dict(positions=st["pos"], rope_cos_sin=st["tab"], interleaved=st["inter"]) if st["R"] else {}
            if st["fmt"] == "bf16":
                g.attn_cache_append(st["k"], st["v"], st["slots"], *st["cache"], **kw)
                return list(st["cache"])
            if st["fmt"] == "fp8":
                g.attn_cache_append_fp8(st["k"], st["v"], st["slots"], *st["cache"], st["ks"], st["vs"], **kw)
                return [c.view(torch.float8_e4m3fn) for c in st["cache"]]
            g.attn_cache_append_q4(st["k"], st["v"], st["slots"], *st["cache"], st["ks"], st["vs"], **kw)
            return g.attn_cache_gather_q4(st["slots"], *st["cache"], st["ks"], st["vs"])
        if st["page"]:
            return g.attn_decode_paged_q4_fwd(st["q"], *st["cache"], st["ks"], st["vs"], st["bt"], st["lens"],
                                              scale=st["scale"], o=st["o"], lse=st["lse"], rope_cos_sin=st["tab"])
        return g.attn_decode_q4_fwd(st["q"], *st["cache"], st["ks"], st["vs"], st["lens"], scale=st["scale"], o=st["o"],
                                    lse=st["lse"], rope_cos_sin=st["tab"])
    if op == "plan":
        return _plain_plan(st)
    if op == "rope":
        h = st["R"] // 2
        cs = st["tab"][st["pos"].long()]
        cs = cs[:, None]                                            # heads
        return tuple(_turn(x.float(), cs[..., :h], cs[..., h:], st["R"], st["inter"], st["bwd"]).bfloat16()
                     for x in (st["q"], st["k"]))
    if op == "table":
        inv = _inv_freq(st["R"], st["base_"], st["factor"], st["orig"], st["low"], st["high"], torch.float64, "cuda")
        ang = torch.arange(st["n"], dtype=torch.float64, device="cuda")[:, None] * inv
        return (torch.cat([torch.cos(ang), torch.sin(ang)], 1) * st["mscale"]).float()
    if op == "append":
        return _plain_append(st, st["k"].float(), st["v"].float())
    o, lse = _attend(st["q"], [_values(_rows(st, i), _rows(st, i + 1)) for i in (0, 2)], st, torch.float32)
    return o.bfloat16(), lse


# ---------------------------------------------------------------- sizes
def work(case):
    op = case["op"]
    if op == "plan":
        new = _total(case["new_lo"], case["new_hi"], case["B"])
        return dict(bytes=8 * (new + 7) + 20 * case["B"] + 8 * (new / case["page"]), flops=0)
    if op == "rope":
        n = case["B"] * case["T"]
        el = n * (case["Hq"] + case["Hkv"]) * case["D"]
        return dict(bytes=4 * el + n * 4 + min(n, 8192) * case["R"] * 4, flops=3 * el * case["R"] / case["D"])
    if op == "table":
        return dict(bytes=4 * case["n"] * case["R"], flops=case["n"] * case["R"] * 10)
    if op == "append":
        n = case["tokens"] - case["pad"]
        el = 2 * n * case["Hkv"] * case["D"]
        w = {"q4": 0.5625, "fp8": 1, "bf16": 2}[case["fmt"]]
        back = (w + 2) * el if case["fmt"] == "q4" else 0           # the rows are read back as bf16 values
        return dict(bytes=(2 + w) * el + back + 8 * case["tokens"] + min(n, 8192) * case["R"] * 4, flops=4 * el)
    keys = _total(case["lo"], case["hi"], case["B"])
    rows = case["B"] * case["Hq"] * case["Tq"]
    return dict(bytes=keys * case["Hkv"] * case["D"] * 2 * 0.5625 + rows * (case["D"] * 4 + 4),
                flops=4 * keys * case["Hq"] * case["Tq"] * case["D"])


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        page, lens, new = case["page"], st["lens"].tolist(), st["new"].tolist()
        table, free, at = st["table"].tolist(), st["free"].tolist(), int(st["cursor"])
        slots, pos, cu, out = [], [], [0], []
        for b in range(case["B"]):
            for p in range(-(-lens[b] // page), -(-(lens[b] + new[b]) // page)):
                table[b][p], at = free[at], at + 1
            for p in range(lens[b], lens[b] + new[b]):
                slots.append(table[b][p // page] * page + p % page)
                pos.append(p)
            cu.append(cu[-1] + new[b])
            out.append(lens[b] + new[b])
        slots += [-1] * (st["total"] - len(slots))
        pos += [0] * (st["total"] - len(pos))
        return [torch.tensor(x, dtype=torch.int32) for x in (slots, pos, cu, out, [at], table)]
    if op == "table":
        i = torch.arange(case["R"] // 2, dtype=torch.float64, device="cuda")
        w = torch.exp(-2.0 * i / case["R"] * math.log(st["base_"]))
        if case["orig"]:
            wave = 2 * math.pi / w
            mix = (case["orig"] / wave - case["low"]) / (case["high"] - case["low"])
            w = torch.where(mix >= 1, w, torch.where(mix <= 0, w / case["factor"], (1 - mix) * w / case["factor"] + mix * w))
        else:
            w = w / case["factor"]
        ang = torch.outer(torch.arange(case["n"], dtype=torch.float64, device="cuda"), w)
        return torch.cat([ang.cos(), ang.sin()], 1) * case["mscale"]

    def rot(x, pos, tab, R, inter, sign):
        """Each pair as a complex number times e^{i angle} (table rows broadcast over axis 1)."""
        cs = tab.double()[pos.long()].unsqueeze(1)
        w = torch.complex(cs[..., :R // 2].contiguous(), sign * cs[..., R // 2:].contiguous())
        x = x.double()
        y = x.clone()
        if inter:
            z = torch.view_as_complex(x[..., :R].unflatten(-1, (-1, 2)).contiguous()) * w
            y[..., :R] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * w
            y[..., :R] = torch.cat([z.real, z.imag], -1)
        return y

    if op == "rope":
        return tuple(rot(st[n], st["pos"], st["tab"], case["R"], case["inter"], -1.0 if case["bwd"] else 1.0) for n in ("q", "k"))
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    if op == "append":
        k, v = st["k"].double(), st["v"].double()
        if case["R"]:
            k = rot(k, st["pos"], st["tab"], case["R"], case["inter"], 1.0)
        out, slots = [], st["slots"].long()
        for i, (x, s) in enumerate(((k, st["ks"]), (v, st["vs"]))):
            s = float(torch.tensor(s, dtype=torch.float32))
            if case["fmt"] == "q4":
                b = x.unflatten(-1, (-1, 16))
                sf = (b.abs().amax(-1, keepdim=True) / (6 * s)).clamp(max=448).float().to(torch.float8_e4m3fn).double() * s
                a = b.abs() / sf.clamp(min=1e-300)
                mid = (grid[1:] + grid[:-1]) / 2
                near = torch.bucketize(a, mid)                    # halfway: the lower one, then the even one
                near = near + ((a == mid[near.clamp(max=6)]) & (near % 2 == 1) & (near < 7))
                val = (grid[near] * torch.sign(b) * sf).flatten(-2)
                out.append(torch.where((slots >= 0)[:, None, None], val, 0.0))
            else:
                c = torch.zeros(st["cache"][i].shape, dtype=torch.float64, device="cuda")
                live = slots >= 0
                y = x if case["fmt"] == "bf16" else (x / s).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
                pages = c.transpose(1, 2).contiguous().flatten(0, 1)
                pages[slots[live]] = y[live]
                out.append(pages.unflatten(0, (c.shape[0], c.shape[2])).transpose(1, 2).contiguous())
        return out
    B, Hq, Tq, D, G = case["B"], case["Hq"], case["Tq"], case["D"], case["Hq"] // case["Hkv"]
    signed = torch.cat([grid, -grid])
    os_, ls = torch.zeros(B, Hq, Tq, D, dtype=torch.float64), torch.zeros(B, Hq, Tq, dtype=torch.float64)
    for b in range(B):
        n = int(st["lens"][b])

        def val(i, scale):
            c, f = st["cache"][i], st["cache"][i + 1]
            if case["page"]:
                m = st["bt"][b, :-(-n // case["page"])].long()
                c, f = (t[m].transpose(0, 1).flatten(1, 2) for t in (c, f))
            else:
                c, f = c[b], f[b]
            c, f = c[:, :n], f[:, :n].view(torch.float8_e4m3fn).double() * scale
            both = torch.stack([signed[(c & 15).long()], signed[(c >> 4).long()]], -1).flatten(-2)
            return both * f.repeat_interleave(16, -1)

        K, V = val(0, st["ks"]), val(2, st["vs"])
        for t in range(Tq):
            seen = n - Tq + t + 1
            q = st["q"][b, :, t].double()
            if st["tab"] is not None:
                q = rot(q[None], torch.tensor([seen - 1], device="cuda"), st["tab"], D, False, 1.0)[0]
            s = torch.einsum("hgd,hkd->hgk", q.reshape(-1, G, D), K[:, :seen]) * st["scale"]
            ls[b, :, t] = torch.logsumexp(s, -1).flatten().cpu()
            os_[b, :, t] = torch.einsum("hgk,hkd->hgd", torch.softmax(s, -1), V[:, :seen]).reshape(Hq, D).cpu()
    return os_, ls
