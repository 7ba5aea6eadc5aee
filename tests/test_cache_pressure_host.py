"""Refusals of attention over shared prefixes, cached keys' weights and eviction at the C boundary, and their plain
references, on the CPU."""
import ctypes
import math

import pytest
import torch

import cache_ref as C
import pressure_ref as R

A = 256      # an aligned fake device address: refused calls never reach it
NULL = None


@pytest.fixture(scope="module")
def lib():
    from causal_gqa_attention_fwd_gb300 import build
    build.build()
    import causal_gqa_attention_fwd_gb300 as g
    return g.lib()


def test_prefix_refusals(lib):
    def f(q=A, kp=A, vp=A, pl=A, k=A, v=A, ln=A, o=A, lse=A, ws=A, wsb=1 << 40, B=4, Hq=8, Hkv=2, Tq=1, P=2, Sp=256, S=64,
          D=128, scale=0.1):
        return lib.attn_decode_prefix_fwd(q, kp, vp, pl, k, v, ln, o, lse, ws, wsb, B, Hq, Hkv, Tq, P, Sp, S, D, scale, None)
    assert f(B=-1) == 2 and f(P=0) == 2 and f(P=3) == 2 and f(Sp=-1) == 2 and f(S=-1) == 2 and f(Tq=65) == 2 and f(Hq=7) == 2
    assert f(D=96) == 3 and f(scale=math.inf) == 2 and f(scale=math.nan) == 2 and f(scale=3e38) == 2
    assert f(B=1 << 20, P=1 << 20, Hq=1 << 11, Hkv=1 << 11, S=1) == 2
    assert f(P=1, Sp=0x7fffffff, Hkv=128, Hq=128) == 2                         # the stream of blocks
    for name in ("q", "kp", "vp", "pl", "k", "v", "ln", "o", "lse"):
        assert f(**{name: NULL}) == 1, name
        assert f(**{name: A + 2}) == 4, name
    assert f(ws=NULL) == 6 and f(ws=A + 16) == 6
    need = lib.attn_decode_prefix_workspace_size(4, 8, 2, 1, 2, 256, 64, 128)
    assert need > 0 and f(wsb=need - 1) == 6
    assert f(B=0, q=NULL) == 0 and f(Tq=0, q=NULL) == 0
    assert lib.attn_decode_prefix_workspace_size(4, 8, 2, 1, 3, 256, 64, 128) == 0


def test_sizes_beyond_the_plans_are_refused(lib):
    """Sizes up to the largest integer, in every argument: a workspace that memory could hold, or a refusal."""
    import itertools
    top = 0x7fffffff
    vals = [1, 8, 255, 65535, 1 << 20, 1 << 30, top - 300, top - 255, top - 16, top]
    for B, Tq, Sp, S in itertools.product(vals, repeat=4):
        for P in (1, B):
            for Hq, Hkv in ((1, 1), (64, 8)):
                assert lib.attn_decode_prefix_workspace_size(B, Hq, Hkv, Tq, P, Sp, S, 64) < 1 << 44
    assert lib.attn_decode_prefix_workspace_size(1, 1, 1, top, 1, 0, top, 64) == 0
    w = [A] * 6
    assert lib.attn_cache_weights(*w, 1, 1, 1, top, top, 1, 1, 64, 0.1, None) == 2
    assert lib.attn_cache_weights(*w, top, 64, 64, top, 1, 1, 1, 64, 0.1, None) == 2


def test_paged_prefix_refusals(lib):
    def f(q=A, k=A, v=A, pt=A, pl=A, bt=A, ln=A, o=A, lse=A, ws=A, wsb=1 << 40, B=4, Hq=8, Hkv=2, Tq=1, P=2, ps=16, n=9, mpp=4,
          mp=4, D=128, scale=0.1):
        return lib.attn_decode_paged_prefix_fwd(q, k, v, pt, pl, bt, ln, o, lse, ws, wsb, B, Hq, Hkv, Tq, P, ps, n, mpp, mp, D,
                                                scale, None)
    assert f(ps=24) == 2 and f(ps=0) == 2 and f(n=0) == 2 and f(n=-1) == 2 and f(mpp=-1) == 2 and f(mp=0) == 2 and f(P=3) == 2
    assert f(ps=128, mpp=1 << 24) == 2 and f(ps=128, mp=1 << 24) == 2          # 2^31 positions
    for name in ("q", "k", "v", "pt", "pl", "bt", "ln", "o", "lse"):
        assert f(**{name: NULL}) == 1, name
        assert f(**{name: A + 2}) == 4, name
    assert f(wsb=0) == 6 and f(D=65) == 3 and f(B=0) == 0


def test_workspace_covers_every_cut(lib):
    """The workspace has a slot for each piece that any lengths can cut a unit into: the kernel's arithmetic, in Python."""
    import random
    r = random.Random(5)
    for _ in range(4000):
        P = r.choice([1, 1, 2, 5, 33])
        B, Hkv, G, Tq = P * r.randint(1, r.choice([2, 40, 256])), r.choice([1, 2, 3, 8]), r.choice([1, 2, 4, 7, 8]), r.choice([1, 2, 5])
        Sp = r.randint(1, r.choice([200, 5000, 40000]))
        Rp = B // P * G * Tq
        nrt = -(-Rp // 256)
        width = max(w for w in range(1, min(nrt, 38) + 1) if nrt % w == 0 and 152 // w * w * 100 >= 94 * 152)
        outer = nrt // width
        if (-(-Rp // 16) - 1) * P * Hkv * Sp * 64 * 4 <= (24 if P * Hkv * -(-Rp // 256) < 96 else 96) << 20:
            continue                # few rows: the prefix's pieces are the stream's, which needs no slots
        size = lib.attn_decode_prefix_workspace_size(B, Hkv * G, Hkv, Tq, P, Sp, 128, 64)
        R, block = G * Tq, 8 if G * Tq <= 8 else 16
        units = B * Hkv * -(-R // block)
        own = (units + 160 * 12) * min(R, block) * (64 * 4 + 8) + units * 8
        slots = (size - own) // (P * Hkv * Rp * (64 * 4 + 8))                   # and rounding, less than a slot
        ctas = r.choice([152, 148, 132])
        nb = [-(-m // 128) for m in (r.choice([0, Sp, r.randint(0, Sp)]) for _ in range(P))]
        total = Hkv * outer * sum(nb)
        T = min(ctas // width, total)
        at = 0
        for n in nb:
            for _ in range(Hkv * outer):
                if n:
                    pieces = ((at + n) * T - 1) // total - ((at + 1) * T - 1) // total + 1
                    assert pieces * (2 if (Rp - 1) % 256 < 128 else 1) <= slots
                at += n


def test_weights_refusals(lib):
    base = dict(q=A, k=A, lse=A, bt=A, ln=A, w=A, B=2, Hq=4, Hkv=2, Tq=1, ps=16, n=9, mp=4, D=64, scale=0.1)

    def f(kind="", ks=1.0, sf=A, **kw):
        x = dict(base, **kw)
        pre = {"": (x["q"], x["k"]), "_fp8": (x["q"], x["k"], ks), "_q4": (x["q"], x["k"], sf, ks)}[kind]
        return getattr(lib, "attn_cache_weights" + kind)(*pre, x["lse"], x["bt"], x["ln"], x["w"], x["B"], x["Hq"], x["Hkv"],
                                                         x["Tq"], x["ps"], x["n"], x["mp"], x["D"], x["scale"], None)
    for kind in ("", "_fp8", "_q4"):
        assert f(kind, B=-1) == 2 and f(kind, Tq=-1) == 2 and f(kind, ps=-1) == 2 and f(kind, n=-1) == 2 and f(kind, mp=-1) == 2
        assert f(kind, Hq=5) == 2 and f(kind, D=32) == 3 and f(kind, scale=math.nan) == 2 and f(kind, n=0) == 2
        assert f(kind, ps=1 << 16, mp=1 << 15) == 2 and f(kind, ps=1 << 16, n=1 << 15) == 2
        assert f(kind, bt=NULL) == 2                                            # contiguous: a row of the cache for each batch row
        for name in ("q", "k", "lse", "ln", "w"):
            assert f(kind, **{name: NULL}) == 1, name
            assert f(kind, **{name: A + 2}) == 4, name
        assert f(kind, bt=A + 2) == 4 and f(kind, B=0, n=0) == 0 and f(kind, Tq=0) == 0
    assert f("_q4", sf=NULL) == 1 and f("_q4", sf=A + 4) == 4
    assert f("_fp8", ks=math.inf) == 2 and f("_q4", ks=3e38, scale=10.0) == 2


def test_evict_refusals(lib):
    rows = lambda *v: (ctypes.c_int * len(v))(*v)  # noqa: E731
    ptrs = lambda *v: (ctypes.c_void_p * len(v))(*v)  # noqa: E731
    at = [1 << 20 | i << 16 for i in range(8)]     # far apart

    def f(w=at[0], planes=ptrs(at[1], at[2]), rb=rows(128, 128), n_planes=2, bt=at[3], ln=at[4], budget=8, recent=2, first=1,
          kept=at[5], out=at[6], B=2, Hkv=2, ps=4, n=9, mp=4):
        return lib.attn_cache_evict(w, planes, rb, n_planes, bt, ln, budget, recent, first, kept, out, B, Hkv, ps, n, mp, None)
    assert f(B=-1) == 2 and f(Hkv=0) == 2 and f(ps=-1) == 2 and f(n=-1) == 2 and f(mp=-1) == 2 and f(n_planes=9) == 2
    assert f(budget=0) == 2 and f(recent=-1) == 2 and f(first=-1) == 2 and f(recent=5, first=4) == 2
    assert f(recent=0x7fffffff, first=0x7fffffff) == 2
    assert f(rb=rows(128, 6)) == 2 and f(rb=rows(128, 0)) == 2 and f(rb=rows(4100, 128)) == 2
    assert f(bt=NULL) == 2                                                       # contiguous: a row of the cache a length
    for name in ("w", "planes", "rb", "ln", "kept", "out"):
        assert f(**{name: NULL}) == 1, name
    assert f(planes=ptrs(at[1], None)) == 1 and f(planes=ptrs(at[1], at[2] + 8)) == 4
    assert f(w=at[0] + 4) == 4 and f(ln=at[4] + 1) == 4 and f(bt=at[3] + 2) == 4
    # buffers that share memory: a plane with another or with the weights, an output with anything
    assert f(planes=ptrs(at[1], at[1])) == 2 and f(planes=ptrs(at[0], at[2])) == 2 and f(planes=ptrs(at[1], at[1] + 9 * 2 * 4 * 128 - 16)) == 2
    assert f(out=at[4]) == 2 and f(kept=at[6] - 4) == 2 and f(kept=at[3]) == 2 and f(out=at[2]) == 2 and f(kept=at[0]) == 2
    assert f(B=0) == 0
    if not torch.cuda.is_available():              # accepted by the checks: the call ends at the device
        assert f() in (7, 8) and f(planes=NULL, rb=NULL, n_planes=0) in (7, 8)
        assert f(planes=ptrs(at[1], at[1] + 9 * 2 * 4 * 128)) in (7, 8)


def test_prefix_reference_is_the_decode_over_the_joined_keys():
    g = torch.Generator().manual_seed(0)
    q = torch.randn(4, 4, 2, 16, generator=g)
    rn = lambda n: torch.randn(2, n, 16, generator=g, dtype=torch.float64)  # noqa: E731
    pre, own, lens = [(rn(7), rn(7)), (rn(0), rn(0))], [(rn(n), rn(n)) for n in (2, 5, 3, 4)], [2, 5, 3, 4]
    o, lse, _, _ = R.prefix(q, pre, own, lens, 0.3)
    for b in range(4):
        k, v = (torch.cat([pre[b // 2][i], own[b][i]], 1)[None] for i in range(2))
        ro, rl, _, _ = C.decode(q[b:b + 1], k, v, [k.shape[2]], 0.3)
        assert torch.allclose(o[b], ro[0], atol=1e-12) and torch.allclose(lse[b], rl[0], atol=1e-12)


def test_weights_reference_sums_to_the_queries():
    g = torch.Generator().manual_seed(1)
    q, K = torch.randn(6, 3, 16, generator=g), torch.randn(2, 9, 16, generator=g, dtype=torch.float64)
    x = torch.einsum("hgtd,hkd->hgtk", q.double().reshape(2, 3, 3, 16), K) * 0.2
    seen = torch.arange(9)[None] <= 6 + torch.arange(3)[:, None]
    lse = torch.logsumexp(x.masked_fill(~seen, -math.inf), -1).reshape(6, 3)
    add, _ = R.weights(q, K, lse, 9, 0.2)
    assert torch.allclose(add.sum(-1), torch.full((2,), 9.0, dtype=torch.float64), atol=1e-9)


def test_evict_reference():
    w = torch.tensor([5.0, 1.0, 3.0, 3.0, math.nan, 0.0, 3.0, 2.0, 9.0])
    assert R.evict(w, 9, 4, 1, 1) == [0, 2, 4, 8]      # NaN above all, then the first of the threes
    assert R.evict(w, 9, 9, 0, 0) == list(range(9)) and R.evict(w[:3], 3, 5, 5, 0) == [0, 1, 2]
    assert R.evict(w, 9, 3, 3, 0) == [6, 7, 8] and R.evict(w, 9, 2, 0, 2) == [0, 1]


def test_an_empty_batch_over_pages(lib):
    """A block table without rows is NULL for most allocators; that is no contiguous cache of another batch."""
    one = (ctypes.c_void_p * 1)(A << 12)
    wide = (ctypes.c_int * 1)(128)
    sizes = (0, 4, 2, 1, 16, 9, 4, 64, 0.1, None)
    for table in (NULL, A):
        assert lib.attn_cache_weights(A, A, A, table, NULL, A, *sizes) == 0
        assert lib.attn_cache_weights_fp8(A, A, 1.0, A, table, NULL, A, *sizes) == 0
        assert lib.attn_cache_weights_q4(A, A, A, 1.0, A, table, NULL, A, *sizes) == 0
        assert lib.attn_cache_evict(A, one, wide, 1, table, NULL, 8, 2, 1, NULL, NULL, 0, 2, 16, 9, 4, None) == 0
        assert lib.attn_cache_evict(A, one, wide, 1, table, NULL, 8, 8, 1, NULL, NULL, 0, 2, 16, 9, 4, None) == 2
