"""Cached attention over 4-bit caches on the GPU against 64 bits on the same codes and scales.

Tolerances.  O: one bf16 rounding (2^-8 of the value), P rounded to f16 (2^-11 of every term, times 2 for the f32
exponentials, sums and the merge of pieces): 2^-8 |o| + 2^-10 sum_j p_j |v_j|.  A P below 2^-14 of its row's largest is
subnormal in f16, whose rounding is absolute: half of its smallest step 2^-24, so up to 2^-25 |v_j| a key, over a sum of
exponentials of at least 1: 2^-25 sum_j |v_j| more (it also covers what is below the smallest f32 and bf16).  LSE: products of f16 values are exact
in f32, their sum over D <= 128 features (the remainder's too) is off by at most 2 D 2^-24 <= 2^-16 of sum_d |q_d k_d|;
the sum of exponentials by 2^-16 of itself (runs of up to 2^8 terms a lane)."""
import math

import pytest
import torch

import cache_ref as R
from causal_gqa_attention_fwd_gb300 import workloads as W

pytestmark = pytest.mark.gpu
KS, VS = 0.0031, 0.0023


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


def cache_of(n, H, P, D, seed, nan=False):
    """Codes and scales of N(0,1) values (drawn directly: any code, block scales around 2 / (6 * scale))."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for s in (KS, VS):
        c = torch.randint(0, 256, (n, H, P, D // 2), generator=g, dtype=torch.uint8)
        amax = 1.2 + 1.5 * torch.rand(n, H, P, D // 16, generator=g)
        out += [c, (amax / (6 * s) * 0.5).to(torch.float8_e4m3fn).view(torch.uint8)]
    return out


def close(o, lse, ref):
    ro, rl, spread, weight = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isnan(o), torch.isnan(ro)) and torch.equal(torch.isnan(lse), torch.isnan(rl))
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    ok = ~torch.isnan(ro)
    off = (o - ro).abs() - (2.0 ** -8 * ro.abs() + 2.0 ** -10 * spread)
    assert (off[ok] <= 0).all(), f"o off by {float(off[ok].max()):.2e} beyond its bound"
    fine = ~torch.isnan(rl) & ~empty
    off = (lse - rl).abs() - (2.0 ** -16 * weight + 2.0 ** -16 + 2.0 ** -22 * rl.abs())
    assert (off[fine] <= 0).all(), f"lse off by {float(off[fine].max()):.2e} beyond its bound"


def run(gq, q, cache, lens, scale, table=None, tab=None, **kw):
    dev = [c.cuda() for c in cache]
    args = (q.cuda(), *dev, KS, VS)
    if tab is not None:
        kw["rope_cos_sin"] = tab.cuda()
    if table is None:
        return gq.attn_decode_q4_fwd(*args, lens.cuda(), scale=scale, **kw)
    return gq.attn_decode_paged_q4_fwd(*args, table.cuda(), lens.cuda(), scale=scale, **kw)


def reference(q, cache, lens, scale, table=None, tab=None):
    k, v = (R.values(cache[i], cache[i + 1], s) for i, s in ((0, KS), (2, VS)))
    if table is not None:
        k, v = R.pages_to_rows(k, table), R.pages_to_rows(v, table)
    return R.decode(q, k, v, lens, scale, tab)


def queries(B, Hq, Tq, D, seed, std=1.0):
    return (torch.randn(B, Hq, Tq, D, generator=torch.Generator().manual_seed(seed)) * std).bfloat16()


def lens_of(x):
    return torch.tensor(x, dtype=torch.int32)


CASES = [  # B, Hq, Hkv, Tq, S, D, lens
    (1, 1, 1, 1, 1, 64, [1]),
    (3, 8, 2, 1, 701, 128, [701, 1, 389]),
    (4, 14, 2, 1, 513, 64, [513, 31, 32, 33]),
    (2, 16, 2, 4, 640, 128, [640, 385]),             # 32 query rows: two blocks
    (3, 9, 3, 3, 100, 64, [100, 3, 64]),             # 9 query rows
    (2, 24, 1, 1, 300, 128, [300, 17]),              # 24 query rows
    (6, 4, 4, 2, 97, 128, [97, 0, 1, 2, 96, 65]),    # rows shorter than their queries, an empty one
    (2, 5, 1, 7, 1111, 64, [1111, 5]),               # 35 query rows
    (4, 32, 8, 1, 4099, 128, [4099, 2000, 3, 1025]),
    (70, 4, 2, 1, 65, 64, None),
    (300, 2, 1, 1, 40, 128, None),
    (1, 8, 8, 1, 20000, 64, [20000]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_Hq%d_Hkv%d_Tq%d_S%d_D%d" % c[:6])
def test_decode_q4(gq, case):
    B, Hq, Hkv, Tq, S, D, lens = case
    lens = lens_of(lens) if lens else torch.randint(0, S + 1, (B,), generator=torch.Generator().manual_seed(B), dtype=torch.int32)
    q, cache = queries(B, Hq, Tq, D, 1), cache_of(B, Hkv, S, D, 2)
    o, lse = run(gq, q, cache, lens, 1 / math.sqrt(D))
    assert gq.get_device_status() == 0
    close(o, lse, reference(q, cache, lens, 1 / math.sqrt(D)))


@pytest.mark.parametrize("B,Hq,Hkv,D", [(1000, 2, 1, 128), (1300, 3, 3, 64), (700, 12, 1, 128), (2050, 2, 2, 128)])
def test_decode_q4_more_rows_than_a_block_scans_at_once(gq, B, Hq, Hkv, D):
    """The rows are counted in several passes; some are empty, two have lengths that are refused."""
    S, g = 70, torch.Generator().manual_seed(B)
    lens = torch.randint(0, S + 1, (B,), generator=g, dtype=torch.int32)
    lens[::7] = 0
    q, cache = queries(B, Hq, 1, D, 60), cache_of(B, Hkv, S, D, 61)
    o, lse = run(gq, q, cache, lens, 1 / math.sqrt(D))
    assert gq.get_device_status() == 0
    ref = reference(q, cache, lens, 1 / math.sqrt(D))
    close(o, lse, ref)
    bad = lens.clone()
    bad[1], bad[B - 1] = -1, S + 1
    o2, lse2 = (torch.full_like(t, 7.0) for t in (o, lse))
    run(gq, q, cache, bad, 1 / math.sqrt(D), o=o2, lse=lse2)
    assert gq.get_device_status() == 5
    for x, y in ((o, o2), (lse, lse2)):
        assert (y[1] == 7).all() and (y[B - 1] == 7).all()
        y[1], y[B - 1] = x[1], x[B - 1]
    close(o2, lse2, ref)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Tq", [1, 3])
def test_decode_q4_rope(gq, D, Tq):
    B, Hq, Hkv, S = 3, 8, 2, 3000
    lens, tab = lens_of([3000, 1501, 2]), W.rope_cos_sin_table(S, D)
    q, cache = queries(B, Hq, Tq, D, 3), cache_of(B, Hkv, S, D, 4)
    o, lse = run(gq, q, cache, lens, 0.09, tab=tab)
    assert gq.get_device_status() == 0
    close(o, lse, reference(q, cache, lens, 0.09, tab=tab))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Tq", [(3, 1, 1), (2, 2, 3), (6, 1, 1), (4, 2, 4), (20, 1, 1), (3, 1, 9)])
def test_decode_q4_rope_row_counts(gq, Hq, Hkv, Tq, D):
    """1 to 27 rotated query rows a K/V head: value and remainder in one score product (to 4 rows), in two, in blocks."""
    B, S = 2, 517
    lens, tab = lens_of([517, 64]), W.rope_cos_sin_table(S, D)
    q, cache = queries(B, Hq, Tq, D, 30, 3.0), cache_of(B, Hkv, S, D, 31)
    o, lse = run(gq, q, cache, lens, 0.08, tab=tab)
    assert gq.get_device_status() == 0
    close(o, lse, reference(q, cache, lens, 0.08, tab=tab))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,S", [(4, 1, 20001), (16, 1, 20001), (40, 1, 9000), (16, 2, 12345), (6, 3, 9000), (80, 5, 6000),
                                      (24, 12, 2500), (16, 16, 1300)])
def test_decode_q4_units_cut_between_many_ctas(gq, Hq, Hkv, S, D):
    """From a row whose only unit every CTA has a piece of, to units of a few pieces: each number of merging groups."""
    lens = lens_of([S])
    q, cache = queries(1, Hq, 1, D, 50), cache_of(1, Hkv, S, D, 51)
    o, lse = run(gq, q, cache, lens, 1 / math.sqrt(D))
    assert gq.get_device_status() == 0
    close(o, lse, reference(q, cache, lens, 1 / math.sqrt(D)))


def paged(B, Hkv, page, mp, D, lens, seed, spare=2):
    n = B * mp + spare
    table = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:B * mp].reshape(B, mp).to(torch.int32)
    for b in range(B):
        table[b, -(-int(lens[b]) // page):] = -1
    return table, cache_of(n, Hkv, page, D, seed)


@pytest.mark.parametrize("B,Hq,Hkv,Tq,page,mp,D,lens", [
    (3, 8, 2, 1, 16, 40, 128, [640, 1, 145]), (3, 8, 2, 2, 32, 20, 64, [640, 33, 200]),
    (2, 14, 2, 1, 64, 12, 64, [768, 257]), (2, 4, 4, 3, 128, 6, 128, [768, 130]),
    (3, 16, 2, 4, 256, 3, 128, [768, 300, 0]), (2, 8, 1, 1, 384, 3, 64, [1100, 385]),
    (64, 8, 2, 1, 16, 20, 128, None)])
def test_decode_paged_q4(gq, B, Hq, Hkv, Tq, page, mp, D, lens):
    lens = lens_of(lens) if lens else torch.randint(0, page * mp + 1, (B,), generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    table, cache = paged(B, Hkv, page, mp, D, lens, 21)
    q = queries(B, Hq, Tq, D, 5)
    tab = W.rope_cos_sin_table(page * mp, D)
    for t in (None, tab):
        o, lse = run(gq, q, cache, lens, 0.1, table, t)
        assert gq.get_device_status() == 0
        close(o, lse, reference(q, cache, lens, 0.1, table, t))


def test_decode_q4_paged_is_contiguous(gq):
    """The same cache laid out both ways gives the same bits."""
    B, Hq, Hkv, page, mp, D = 2, 8, 2, 64, 20, 128
    lens = lens_of([1280, 700])
    table, cache = paged(B, Hkv, page, mp, D, lens, 4)
    q = queries(B, Hq, 1, D, 6)
    a = run(gq, q, cache, lens, 0.1, table)
    b = run(gq, q, [R.pages_to_rows(c, table) for c in cache], lens, 0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_q4_ignores_what_is_past_the_length(gq):
    """NaN block scales past each row's length, and past a query's own position, must not leak."""
    B, Hq, Hkv, Tq, S, D = 4, 8, 2, 3, 500, 128
    lens = lens_of([500, 3, 261, 0])
    q, cache = queries(B, Hq, Tq, D, 8), cache_of(B, Hkv, S, D, 9)
    for b in range(B):
        n = int(lens[b])
        for i in (1, 3):
            cache[i][b, :, n:] = 0x7F
        if n:
            cache[3][b, 0, n - 1, 2] = 0xFF      # the newest key: visible to the last query only
            cache[1][b, 1, n - 1, 1] = 0x7F
            cache[3][b, 1, n - 2, 0] = 0x7F      # visible to the last two
    o, lse = run(gq, q, cache, lens, 0.1)
    assert gq.get_device_status() == 0
    ref = reference(q, cache, lens, 0.1)
    assert torch.isnan(ref[0]).any() and not torch.isnan(ref[0][0, 4, 0]).any()
    close(o, lse, ref)


def test_decode_q4_nan_inside_the_cache(gq):
    """A NaN block at a visible key: K's makes the rows that see it NaN, V's its 16 features."""
    B, Hq, Hkv, S, D = 2, 8, 2, 700, 128
    lens = lens_of([700, 300])
    q, cache = queries(B, Hq, 1, D, 10), cache_of(B, Hkv, S, D, 11)
    cache[3][0, 1, 400, 5] = 0x7F
    cache[3][1, 0, 17, 0] = 0xFF
    cache[1][1, 1, 250, 3] = 0x7F
    o, lse = run(gq, q, cache, lens, 0.1)
    assert gq.get_device_status() == 0
    close(o, lse, reference(q, cache, lens, 0.1))


@pytest.mark.parametrize("std", [1e-6, 1e-3, 30.0, 3e4, 1e30])
def test_decode_q4_query_magnitudes(gq, std):
    """Queries far outside f16's range: scaled by a power of two per row, the scores stay exact."""
    B, Hq, Hkv, S, D = 2, 8, 2, 333, 64
    lens = lens_of([333, 129])
    q, cache = queries(B, Hq, 1, D, 12, std), cache_of(B, Hkv, S, D, 13)
    scale = 0.125 / std
    o, lse = run(gq, q, cache, lens, scale)
    assert gq.get_device_status() == 0
    close(o, lse, reference(q, cache, lens, scale))


@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("Tq", [1, 3])
@pytest.mark.parametrize("big", [20, 30, 34])
def test_decode_q4_one_outlier_feature(gq, big, Tq, rope):
    """A query feature of 2^big where the keys are 0, beside others of N(0,1): rows are scaled by their largest, so the
    others lose bits.  In f16 a plain feature is off by at most 2^-39 of the row's largest, M (half of f16's smallest step,
    2^-25, against 2^14); a rotated one by that, by 2^-22 of itself (two f16 parts), and by the rotation's f32 roundings,
    3 2^-24 of its pair (|a| + |b|; a table of magnitude 1).  A score is off by delta = scale sum_d |k_d| (that), LSE by
    delta, a weight by a factor of e^(2 delta), beside the usual bounds."""
    B, Hq, Hkv, S, D = 2, 6, 2, 333, 64
    lens = lens_of([333, 129])
    q, cache = queries(B, Hq, Tq, D, 40), cache_of(B, Hkv, S, D, 41)
    q[..., 5] = 2.0 ** big
    cache[0][..., 2] &= 0x0f                       # features 5 and 37, its pair: code 0 (the high half bytes)
    cache[0][..., 18] &= 0x0f
    tab = W.rope_cos_sin_table(S, D) if rope else None
    ref = reference(q, cache, lens, 0.125, tab=tab)
    ka = R.values(cache[0], cache[1], KS).abs().repeat_interleave(Hq // Hkv, 1)[:, :, None]       # [B, Hq, 1, S, D]
    x = q.double()
    M = x.abs().amax(-1, keepdim=True) * (2 if rope else 1)
    off = 2.0 ** -39 * M
    if rope:
        pair = x.abs() + x.abs().roll(D // 2, -1)
        off = off + (2.0 ** -22 + 3 * 2.0 ** -24) * pair
    delta = 0.125 * (ka * off[..., None, :]).sum(-1).amax(-1)                                       # [B, Hq, Tq]
    o, lse = (t.double().cpu() for t in run(gq, q, cache, lens, 0.125, tab=tab))
    assert gq.get_device_status() == 0
    ro, rl, spread, weight = ref
    assert ((o - ro).abs() <= 2.0 ** -8 * ro.abs() + (2.0 ** -10 + torch.expm1(2 * delta)[..., None] * 1.01) * spread).all()
    assert ((lse - rl).abs() <= delta + 2.0 ** -16 * weight + 2.0 ** -16 + 2.0 ** -22 * rl.abs()).all()
    if big == 20 and not rope:                     # every bit is kept
        close(o, lse, ref)


def test_decode_q4_large_scores(gq):
    """Scores in the hundreds, either sign: one key takes almost all."""
    B, Hq, Hkv, S, D = 2, 8, 2, 2100, 128
    lens = lens_of([2100, 999])
    q, cache = queries(B, Hq, 2, D, 14, 20.0), cache_of(B, Hkv, S, D, 15)
    for scale in (1.0, -1.0):
        o, lse = run(gq, q, cache, lens, scale)
        assert gq.get_device_status() == 0
        close(o, lse, reference(q, cache, lens, scale))


def test_decode_q4_zero_and_infinite_queries(gq):
    B, Hq, Hkv, S, D = 1, 4, 2, 70, 64
    q, cache = queries(B, Hq, 1, D, 16), cache_of(B, Hkv, S, D, 17)
    q[0, 0] = 0
    q[0, 3, 0, 5] = float("inf")
    lens = lens_of([70])
    o, lse = run(gq, q, cache, lens, 0.1)
    ref = reference(q, cache, lens, 0.1)
    assert torch.isnan(o[0, 3]).all()
    close(o[:, :3], lse[:, :3], tuple(r[:, :3] for r in ref))


def test_decode_q4_reports_bad_lengths_and_pages(gq):
    """A length outside [0, S]: reported, that row unwritten, the others right.  A page outside the pool: reported."""
    B, Hq, Hkv, page, mp, D = 4, 4, 2, 32, 5, 64
    lens = lens_of([160, 161, 7, -1])
    table, cache = paged(B, Hkv, page, mp, D, lens.clamp(0, 160), 5)
    q = queries(B, Hq, 1, D, 18)
    o = torch.full((B, Hq, 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq, 1), 3.0, device="cuda")
    run(gq, q, cache, lens, 0.1, table, o=o, lse=lse)
    assert gq.get_device_status() == 5
    good = [0, 2]
    close(o[good], lse[good], reference(q[good], cache, lens[good], 0.1, table[good]))
    assert (o[[1, 3]] == 3).all() and (lse[[1, 3]] == 3).all()
    lens, bad = lens_of([160, 160, 7, 0]), table.clone()
    bad[1] = torch.tensor([0, 1, B * mp + 2, 3, 4])      # entry 2 is one past the pool
    o, lse = run(gq, q, cache, lens, 0.1, bad)
    assert gq.get_device_status() == 11
    close(o, lse, reference(q, cache, lens, 0.1, bad))   # its keys read as zeros


def test_decode_q4_is_deterministic(gq):
    lens = torch.randint(6000, 12000, (4,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    q, cache = queries(4, 32, 1, 128, 19), [c.cuda() for c in cache_of(4, 8, 12000, 128, 20)]
    first = run(gq, q, cache, lens, 0.09)
    for _ in range(3):
        again = run(gq, q, cache, lens, 0.09)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_decode_q4_two_captured_graphs_and_lengths_that_change(gq):
    """Two captured calls with workspaces of their own, replayed together on two streams, after the lengths changed."""
    S, D = 5000, 128
    cache = cache_of(2, 2, S, D, 23)
    dev = [c.cuda() for c in cache]
    qs = [queries(2, 8, 1, D, s) for s in (24, 25)]
    lens = [lens_of([S, 100]).cuda(), lens_of([3, 4000]).cuda()]
    graphs, outs = [], []
    qd = [x.cuda() for x in qs]
    for x, n in zip(qd, lens):
        gq.attn_decode_q4_fwd(x, *dev, KS, VS, n, scale=0.1)
    torch.cuda.synchronize()
    for x, n in zip(qd, lens):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gq.attn_decode_q4_fwd(x, *dev, KS, VS, n, scale=0.1))
        graphs.append(g)
    lens[0].copy_(lens_of([0, 4999]))
    lens[1].copy_(lens_of([777, 1]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert gq.get_device_status() == 0
    for x, n, (o, lse) in zip(qs, lens, outs):
        close(o, lse, reference(x, cache, n.cpu(), 0.1))


def test_decode_q4_agrees_with_the_bf16_cache(gq):
    """attn_decode_fwd over the gathered bf16 values: the values' rounding (2^-8 each) is all that differs; with scores
    of unit size the outputs agree to 4 2^-8 of their norm."""
    B, Hq, Hkv, S, D = 2, 8, 2, 900, 128
    lens = lens_of([900, 450])
    q, cache = queries(B, Hq, 1, D, 26), [c.cuda() for c in cache_of(B, Hkv, S, D, 27)]
    slots = torch.arange(B * S, dtype=torch.int32, device="cuda")
    k, v = (x.view(B, S, Hkv, D).transpose(1, 2).contiguous() for x in gq.attn_cache_gather_q4(slots, *cache, KS, VS))
    a, _ = run(gq, q, cache, lens, 0.05)
    b, _ = gq.attn_decode_fwd(q.cuda(), k, v, lens.cuda(), scale=0.05)
    assert float((a.float() - b.float()).norm() / b.float().norm()) < 4 * 2.0 ** -8
