"""The attention weight that cached keys receive, against the definition in 64 bits."""
import math

import pytest
import torch

import cache_ref as C
import pressure_ref as R

pytestmark = pytest.mark.gpu
KS = 0.0125


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


def make(fmt, B, Hq, Hkv, Tq, D, page, lens, seed, S=None, qs=1.0):
    """(planes, float64 keys of each plane slot, q, block table or None, weights), on the CPU.  Slots that hold no key of a
    row are NaN keys, and their weights are NaN, as are those of the rows' Tq new keys."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    S = S or max(*lens, 1)
    per = page or S
    M = -(-S // page) if page else 0
    N = B * M + 2 if page else B
    table = torch.randperm(N, generator=g)[:B * M].reshape(B, M).to(torch.int32) if page else None
    x = rn(N, Hkv, per, D)
    used, old = torch.zeros(N, per, dtype=torch.bool), torch.zeros(N, per, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            at = (int(table[b, j // page]), j % page) if page else (b, j)
            used[at], old[at] = True, j < n - Tq
    x = torch.where(used[:, None, :, None], x, torch.tensor(math.nan))
    if fmt == "bf16":
        planes, keys = [x.bfloat16()], x.bfloat16().double()
    elif fmt == "fp8":
        planes = [(x / KS).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)]
        keys = C.e4m3(planes[0]) * KS
    else:
        planes = list(C.quantise(x, KS))
        keys = C.values(*planes, KS)
    w = torch.where(old[:, None].expand(N, Hkv, per), torch.rand(N, Hkv, per, generator=g), torch.tensor(math.nan))
    if page:
        for b, n in enumerate(lens):
            table[b, -(-n // page):] = -9          # entries that no key needs may hold anything
    return planes, keys, (rn(B, Hq, Tq, D) * qs).bfloat16(), table, w


def call(gq, fmt, planes, q, lse, lens, w, table, scale, **kw):
    f = {"bf16": gq.attn_cache_weights, "fp8": gq.attn_cache_weights_fp8, "q4": gq.attn_cache_weights_q4}[fmt]
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    ks = () if fmt == "bf16" else (KS,)
    return f(q.cuda(), *(p.cuda() for p in planes), *ks, lse.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), w,
             block_table=cu(table), scale=scale, **kw)


def lse_of(q, keys, table, lens, scale):
    B, Hq, Tq, D = q.shape
    Hkv = keys.shape[1]
    lse = torch.full((B, Hq, Tq), -math.inf)
    for b, n in enumerate(lens):
        K = R.rows_of(keys, table, b, n).repeat_interleave(Hq // Hkv, 0)
        for t in range(Tq):
            if n - Tq + t >= 0:
                s = torch.einsum("hd,hkd->hk", q[b, :, t].double(), K[:, :n - Tq + t + 1]) * scale
                lse[b, :, t] = torch.logsumexp(s, -1).float()
    return lse


def check(got, w, q, keys, lse, table, lens, scale):
    got, want, tol = got.cpu().double(), w.double().clone(), torch.zeros_like(w, dtype=torch.float64)
    P = w.shape[2]
    for b, n in enumerate(lens):
        if n == 0:
            continue
        add, e = R.weights(q[b], R.rows_of(keys, table, b, n), lse[b], n, scale)
        j = torch.arange(n)
        at = (table[b, j // P].long(), slice(None), j % P) if table is not None else (b, slice(None), j)
        old = R.rows_of(w, table, b, n).double()
        old[:, max(n - q.shape[2], 0):] = 0                  # the Tq new keys
        want[at] = (old + add).t() if table is not None else old + add
        tol[at] = e.t() if table is not None else e
    tol = tol + 2.0 ** -23 * want.abs()      # the sum's rounding
    same = torch.isnan(want) & torch.isnan(got)
    off = ((got - want).abs() / tol.clamp(min=1e-300))[~same]
    assert bool((off <= 1).all()), float(off.max())


CASES = [
    # B, Hq, Hkv, Tq, D, page, lengths
    (1, 1, 1, 1, 64, 0, [1]),
    (8, 14, 2, 1, 64, 0, [300] * 8),
    (5, 16, 4, 16, 128, 0, [301, 16, 5, 257, 64]),        # 64 query rows; rows shorter than the window
    (3, 8, 1, 9, 128, 0, [40, 513, 9]),                   # 72 rows: two passes over the rows
    (2, 12, 4, 5, 64, 0, [0, 33]),
    (4, 8, 2, 1, 128, 16, [1, 16, 17, 255]),
    (3, 6, 3, 2, 64, 7, [50, 2, 1]),                      # any page size
    (2, 8, 8, 1, 128, 64, [64, 500]),
    (1, 8, 2, 1, 128, 128, [1031]),
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "q4"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{c[0]}H{c[1]}-{c[2]}T{c[3]}D{c[4]}p{c[5]}n{max(c[6])}")
def test_against_the_definition(gq, case, fmt):
    B, Hq, Hkv, Tq, D, page, lens = case
    planes, keys, q, table, w = make(fmt, *case, seed=1)
    scale = 1 / math.sqrt(D)
    lse = lse_of(q, keys, table, lens, scale)
    out = [w.cuda(), w.cuda()]
    for o in out:
        got = call(gq, fmt, planes, q, lse, lens, o, table, scale)
        assert got is o
    assert gq.get_device_status() == 0
    check(out[0], w, q, keys, lse, table, lens, scale)
    assert torch.equal(out[0].nan_to_num(-1), out[1].nan_to_num(-1))         # the same bits again


LONG = [
    # windows of many query rows: whole and partial blocks of 64 rows, chunks of 256 keys that all rows see and others
    (2, 8, 2, 9, 128, 0, [700, 257]),                     # 36 rows
    (2, 14, 2, 14, 64, 16, [513, 256]),                   # 98
    (3, 8, 2, 32, 128, 64, [1023, 31, 0]),                # 128; rows shorter than the window
    (1, 8, 1, 25, 64, 7, [300]),                          # 200
    (2, 16, 2, 40, 128, 16, [40, 900]),                   # 320
    (1, 32, 4, 67, 64, 0, [1500]),                        # 536
]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "q4"])
@pytest.mark.parametrize("case", LONG, ids=lambda c: f"B{c[0]}H{c[1]}-{c[2]}T{c[3]}D{c[4]}p{c[5]}n{max(c[6])}")
def test_long_windows(gq, case, fmt):
    B, Hq, Hkv, Tq, D, page, lens = case
    planes, keys, q, table, w = make(fmt, *case, seed=9)
    scale = -1 / math.sqrt(D) if B == 1 else 1 / math.sqrt(D)
    lse = lse_of(q, keys, table, lens, scale)
    lse[0, 1] = -math.inf                                                    # a head that the caller leaves out
    out = [w.cuda(), w.cuda()]
    for o in out:
        call(gq, fmt, planes, q, lse, lens, o, table, scale)
    assert gq.get_device_status() == 0
    check(out[0], w, q, keys, lse, table, lens, scale)
    assert torch.equal(out[0].nan_to_num(-1), out[1].nan_to_num(-1))


@pytest.mark.parametrize("B,Tq", [(3, 5), (3, 33), (40, 5), (70, 9), (130, 5)])
def test_ragged_rows_of_a_large_capacity(gq, B, Tq):
    """More chunks of the capacity than CTAs at once: CTAs find their keys by the lengths (up to 128 rows), also behind
    rows without keys, or by their place."""
    S = stream_capacity(B, 2)
    g = torch.Generator().manual_seed(B + Tq)
    lens = torch.randint(0, min(S, 600), (B,), generator=g).tolist()
    lens[0] = 0
    lens[B // 2] = min(S, 700)
    case = (B, 8, 2, Tq, 64, 64, lens)
    planes, keys, q, table, w = make("bf16", *case, seed=12, S=S)
    lse = lse_of(q, keys, table, lens, 0.125)
    out = call(gq, "bf16", planes, q, lse, lens, w.cuda(), table, 0.125)
    assert gq.get_device_status() == 0
    check(out, w, q, keys, lse, table, lens, 0.125)
    bad = list(lens)
    bad[B - 1] = -5
    out = call(gq, "bf16", planes, q, lse, bad, w.cuda(), table, 0.125)
    assert gq.get_device_status() == 5
    bad[B - 1] = 0
    check(out, w, q, keys, lse, table, bad, 0.125)


@pytest.mark.parametrize("qs", [1e-30, 30.0, 1e30])
def test_long_window_of_any_size(gq, qs):
    case = (2, 8, 2, 30, 128, 0, [400, 255])
    for fmt in ("bf16", "fp8", "q4"):
        planes, keys, q, table, w = make(fmt, *case, seed=10, qs=qs)
        scale = 0.05 / qs if qs > 1 else 0.05
        lse = lse_of(q, keys, table, case[6], scale)
        out = call(gq, fmt, planes, q, lse, case[6], w.cuda(), table, scale)
        check(out, w, q, keys, lse, table, case[6], scale)


def test_long_window_reports(gq):
    case = (3, 8, 2, 30, 64, 16, [320, 140, 333])
    planes, keys, q, table, w = make("bf16", *case, seed=11)
    lse = lse_of(q, keys, table, case[6], 0.125)
    for bad in (-1, 1000):
        out = call(gq, "bf16", planes, q, lse, [320, bad, 333], w.cuda(), table, 0.125)
        assert gq.get_device_status() == 5
        check(out, w, q, keys, lse, table, [320, 0, 333], 0.125)
    t = table.clone()
    t[1, 1] = -1
    out = call(gq, "bf16", planes, q, lse, case[6], w.cuda(), t, 0.125)
    assert gq.get_device_status() == 11
    assert torch.equal(out[int(table[1, 1])].cpu().nan_to_num(-1), w[int(table[1, 1])].nan_to_num(-1))


def stream_capacity(B, Hkv):
    """A capacity whose chunks of 256 positions are more than the CTAs that any GPU of this kind holds at once: few query
    rows then go by the stream of tiles whatever the lengths are."""
    return 256 * (3 * 160 // (B * Hkv) + 1)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "q4"])
@pytest.mark.parametrize("case", [c for c in CASES if c[1] // c[2] * c[3] <= 16] + [(3, 8, 4, 8, 128, 0, [3000, 7, 0])],
                         ids=lambda c: f"B{c[0]}H{c[1]}-{c[2]}T{c[3]}D{c[4]}p{c[5]}n{max(c[6])}")
def test_few_rows_of_a_large_capacity(gq, case, fmt):
    B, Hq, Hkv, Tq, D, page, lens = case
    planes, keys, q, table, w = make(fmt, *case, seed=7, S=stream_capacity(B, Hkv))
    scale = 1 / math.sqrt(D)
    lse = lse_of(q, keys, table, lens, scale)
    out = [w.cuda(), w.cuda()]
    for o in out:
        call(gq, fmt, planes, q, lse, lens, o, table, scale)
    assert gq.get_device_status() == 0
    check(out[0], w, q, keys, lse, table, lens, scale)
    assert torch.equal(out[0].nan_to_num(-1), out[1].nan_to_num(-1))


def test_a_large_capacity_reports_too(gq):
    case = (3, 4, 2, 1, 64, 16, [20, 40, 33])
    planes, keys, q, table, w = make("bf16", *case, seed=8, S=stream_capacity(3, 2))
    lse = lse_of(q, keys, table, case[6], 0.125)
    for bad in (-1, 1 << 30):
        out = call(gq, "bf16", planes, q, lse, [20, bad, 33], w.cuda(), table, 0.125)
        assert gq.get_device_status() == 5
        check(out, w, q, keys, lse, table, [20, 0, 33], 0.125)
    t = table.clone()
    t[1, 1] = planes[0].shape[0]
    out = call(gq, "bf16", planes, q, lse, case[6], w.cuda(), t, 0.125)
    assert gq.get_device_status() == 11
    assert torch.equal(out[int(table[1, 1])].cpu().nan_to_num(-1), w[int(table[1, 1])].nan_to_num(-1))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "q4"])
@pytest.mark.parametrize("qs", [1e-30, 1e-3, 30.0, 1e30])
def test_queries_of_any_size(gq, fmt, qs):
    case = (2, 4, 2, 2, 128, 0, [70, 33])
    planes, keys, q, table, w = make(fmt, *case, seed=2, qs=qs)
    scale = 0.05 / qs if qs > 1 else 0.05
    lse = lse_of(q, keys, table, case[6], scale)
    out = call(gq, fmt, planes, q, lse, case[6], w.cuda(), table, scale)
    check(out, w, q, keys, lse, table, case[6], scale)


def test_weights_of_a_row_sum_to_its_queries(gq):
    case = (3, 8, 2, 3, 64, 0, [400, 77, 3])
    planes, keys, q, table, _ = make("bf16", *case, seed=3)
    lse = lse_of(q, keys, None, case[6], 0.125)
    w = torch.zeros(3, 2, 400, device="cuda")
    w[0, :, 397:] = 5.0                              # slots of new keys, used before
    call(gq, "bf16", planes, q, lse, case[6], w, None, None)
    # 4 heads x 3 queries a K/V head, each summing to one: within the tolerance of every term, 1e-5 relative
    assert torch.allclose(w.sum(-1).cpu(), torch.full((3, 2), 12.0), rtol=1e-5, atol=0)
    for b, n in enumerate(case[6]):
        assert bool((w[b, :, n:] == 0).all())


def test_queries_that_saw_nothing_add_nothing(gq):
    case = (2, 4, 2, 4, 64, 0, [50, 2])
    planes, keys, q, table, w = make("bf16", *case, seed=4)
    lse = lse_of(q, keys, None, case[6], 0.125)
    lse[0, 1] = -math.inf                                                    # a head that the caller leaves out
    out = call(gq, "bf16", planes, q, lse, case[6], w.cuda(), None, 0.125)
    check(out, w, q, keys, lse, None, case[6], 0.125)


def test_bad_lengths_and_pages_are_reported(gq):
    case = (3, 4, 2, 1, 64, 16, [20, 40, 33])
    planes, keys, q, table, w = make("bf16", *case, seed=5)
    lse = lse_of(q, keys, table, case[6], 0.125)
    for bad in (-1, 1000):
        out = call(gq, "bf16", planes, q, lse, [20, bad, 33], w.cuda(), table, 0.125)
        assert gq.get_device_status() == 5
        # row 1 stays as it was
        check(out, w, q, keys, lse, table, [20, 0, 33], 0.125)
    t = table.clone()
    t[1, 1] = planes[0].shape[0]
    out = call(gq, "bf16", planes, q, lse, case[6], w.cuda(), t, 0.125)
    assert gq.get_device_status() == 11
    want = call(gq, "bf16", planes, q, lse, case[6], w.cuda(), table, 0.125)
    skip = int(table[1, 1])
    keep = [i for i in range(planes[0].shape[0]) if i != skip]
    assert torch.equal(out[keep].nan_to_num(-1), want[keep].nan_to_num(-1))
    assert torch.equal(out[skip].cpu().nan_to_num(-1), w[skip].nan_to_num(-1))


def test_arguments(gq):
    case = (2, 4, 2, 1, 64, 0, [9, 5])
    planes, keys, q, table, w = make("bf16", *case, seed=6)
    lse = torch.zeros(2, 4, 1)
    ok = lambda **k: call(gq, "bf16", k.get("planes", planes), k.get("q", q), k.get("lse", lse), k.get("lens", [9, 5]),  # noqa: E731
                          k.get("w", w.cuda()), k.get("table"), 0.1)
    ok()
    with pytest.raises(ValueError, match="weights"):
        ok(w=w[:, :, :8].contiguous().cuda())
    with pytest.raises(TypeError, match="float32"):
        ok(w=w.double().cuda())
    with pytest.raises(ValueError, match="lse"):
        ok(lse=torch.zeros(2, 4))
    with pytest.raises(ValueError, match="block_table"):
        ok(q=q[:1], lse=lse[:1], lens=[9])
    with pytest.raises(ValueError, match="cache_lens"):
        ok(lens=[9])
    with pytest.raises(ValueError, match="matching q"):
        ok(q=torch.cat([q, q], -1))
    with pytest.raises(TypeError, match="bfloat16"):
        ok(planes=[planes[0].float()])
    with pytest.raises(ValueError, match="contiguous"):
        ok(w=torch.zeros(2, 9, 2, device="cuda").transpose(1, 2))
    with pytest.raises(gq.AttnError, match="SHAPE"):
        ok(q=q[:, :3].contiguous(), lse=lse[:, :3].contiguous())
    # no page a row: nothing to add to
    none = torch.zeros(2, 0, dtype=torch.int32)
    before = w.cuda()
    assert torch.equal(ok(w=before, table=none, lens=[0, 0]).nan_to_num(-1), w.cuda().nan_to_num(-1))
