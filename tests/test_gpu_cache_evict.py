"""Eviction against a plain selection and copy: every byte is the expected one."""
import math

import pytest
import torch

import pressure_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


def draw(kind, shape, g):
    if kind == "heavy":
        return torch.exp(1.5 * torch.randn(*shape, generator=g))
    if kind == "ties":
        return torch.randint(0, 4, shape, generator=g).float()
    if kind == "equal":
        return torch.full(shape, 0.25)
    if kind == "signs":      # both zeros, both infinities, NaN, negative and tiny values
        v = torch.tensor([0.0, -0.0, 1.0, -1.0, math.inf, -math.inf, math.nan, 1e-42, -1e-42, 3.0])
        return v[torch.randint(0, len(v), shape, generator=g)]
    return torch.rand(*shape, generator=g) ** 8     # "steep": bits of every exponent


def widths(fmt, D):
    return {"bf16": [(torch.bfloat16, D)] * 2, "fp8": [(torch.uint8, D)] * 2,
            "q4": [(torch.uint8, D // 2), (torch.uint8, D // 16)] * 2, "none": [],
            "odd": [(torch.float32, 9), (torch.uint8, 12), (torch.int64, 33), (torch.uint8, 4)]}[fmt]


def make(fmt, B, Hkv, D, page, lens, seed, kind, S=None):
    g = torch.Generator().manual_seed(seed)
    S = S or max(*lens, 1)
    M = -(-S // page) if page else 0
    N, per = (B * M + 2, page) if page else (B, S)
    table = torch.randperm(N, generator=g)[:B * M].reshape(B, M).to(torch.int32) if page else None
    planes = []
    for dt, w in widths(fmt, D):
        raw = torch.randint(0, 256, (N, Hkv, per, w * dt.itemsize), dtype=torch.uint8, generator=g)
        planes.append(raw.view(dt))
    return planes, draw(kind, (N, Hkv, per), g), table


def reference(planes, w, table, lens, budget, recent, first):
    """(kept, lens_out, weights, planes as bytes) after the eviction."""
    B, Hkv, P = len(lens), w.shape[1], w.shape[2]
    raw = [w.view(torch.uint8).reshape(*w.shape, 4).clone()] + [p.view(torch.uint8).reshape(*p.shape[:3], -1).clone() for p in planes]
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    place = lambda b, j: (table[b, j // P].long(), j % P) if table is not None else (torch.full_like(j, b), j)  # noqa: E731
    for b, n in enumerate(lens):
        rows = R.rows_of(w, table, b, n)
        for h in range(Hkv):
            src = torch.tensor(R.evict(rows[h], n, budget, recent, first), dtype=torch.int64)
            kept[b, h, :len(src)] = src.int()
            if n > budget:
                (ps, rs), (pd, rd) = place(b, src), place(b, torch.arange(budget))
                for x in raw:
                    x[pd, h, rd] = x[ps, h, rs]
    return kept, torch.tensor([min(n, budget) for n in lens], dtype=torch.int32), raw


def run(gq, planes, w, table, lens, budget, recent, first, **kw):
    dev = [p.cuda() for p in planes]
    wd = w.cuda()
    kept, out = gq.attn_cache_evict(wd, dev, torch.tensor(lens, dtype=torch.int32).cuda(), budget, recent=recent, first=first,
                                    block_table=None if table is None else table.cuda(), **kw)
    raw = [x.view(torch.uint8).reshape(*x.shape[:3], -1).cpu() for x in (wd.unsqueeze(-1), *dev)]
    return kept.cpu(), out.cpu(), raw


def check(got, want):
    assert torch.equal(got[0], want[0]), "kept"
    assert torch.equal(got[1], want[1]), "lens_out"
    for i, (a, b) in enumerate(zip(got[2], want[2])):
        assert torch.equal(a, b), f"plane {i}"


CASES = [
    # B, Hkv, D, page, lengths, budget, recent, first
    (1, 1, 64, 0, [2], 1, 0, 0),
    (1, 1, 64, 0, [2], 1, 1, 0),
    (1, 1, 64, 0, [2], 1, 0, 1),
    (2, 2, 64, 0, [100, 99], 99, 10, 3),
    (4, 2, 128, 0, [300, 64, 65, 0], 64, 16, 4),
    (3, 3, 128, 16, [257, 33, 1000], 100, 30, 4),
    (2, 2, 64, 7, [150, 20], 13, 5, 8),                    # nothing but the first and the last ones
    (2, 1, 128, 64, [2500, 1025], 1024, 0, 0),
    (3, 2, 64, 1, [30, 5, 17], 6, 2, 1),
    (1, 2, 128, 128, [5000], 4097, 1000, 1),
]


@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "signs", "steep"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{c[0]}H{c[1]}D{c[2]}p{c[3]}n{max(c[4])}k{c[5]}")
def test_every_byte(gq, case, kind):
    B, Hkv, D, page, lens, budget, recent, first = case
    planes, w, table = make("bf16", B, Hkv, D, page, lens, 1, kind)
    got = run(gq, planes, w, table, lens, budget, recent, first)
    assert gq.get_device_status() == 0
    check(got, reference(planes, w, table, lens, budget, recent, first))


@pytest.mark.parametrize("kind", ["heavy", "ties", "signs"])
@pytest.mark.parametrize("S", [255, 2048, 2049, 9000])          # one CTA; CTAs that select alone, and together
@pytest.mark.parametrize("budget", [0.5, 0.97])
def test_capacities(gq, S, kind, budget):
    lens = [S, S - 1, S * 2 // 3]
    planes, w, table = make("bf16", 3, 2, 64, 0, lens, 6, kind)
    k = int(S * budget)
    got = run(gq, planes, w, table, lens, k, 11, 5)
    assert gq.get_device_status() == 0
    check(got, reference(planes, w, table, lens, k, 11, 5))


@pytest.mark.parametrize("fmt", ["fp8", "q4", "none", "odd"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16])
def test_planes_of_any_type(gq, fmt, D, page):
    lens = [130, 20, 333]
    planes, w, table = make(fmt, 3, 2, D, page, lens, 2, "heavy")
    got = run(gq, planes, w, table, lens, 50, 7, 3)
    assert gq.get_device_status() == 0
    check(got, reference(planes, w, table, lens, 50, 7, 3))


def test_long_row(gq):
    lens = [70001]
    planes, w, table = make("fp8", 1, 1, 64, 0, lens, 3, "ties")
    check(run(gq, planes, w, table, lens, 33333, 17, 2), reference(planes, w, table, lens, 33333, 17, 2))
    check(run(gq, planes, w, table, lens, 70000, 0, 0), reference(planes, w, table, lens, 70000, 0, 0))


@pytest.mark.parametrize("share", [18432, 18433, 20480, 20481])
@pytest.mark.parametrize("units,ctas", [(160, 1), (80, 2), (40, 4), (32, 8)])
def test_shares_up_to_what_shared_memory_holds(gq, units, ctas, share):
    """Capacities around the most that a CTA's part of a row takes in shared memory (18432 and 20480 positions), for each
    number of CTAs a row gets; most rows are short, for the capacity alone settles how the call is launched."""
    S = ctas * share
    lens = [S, S - 5] + [(i * 7) % 300 for i in range(units - 2)]
    planes, w, table = make("none", units, 1, 64, 0, lens, 8, "ties", S=S)
    got = run(gq, planes, w, table, lens, 257, 31, 4)
    assert gq.get_device_status() == 0
    check(got, reference(planes, w, table, lens, 257, 31, 4))


def test_budget_beyond_the_capacity(gq):
    lens = [20, 3]
    planes, w, table = make("bf16", 2, 2, 64, 0, lens, 4, "heavy")
    got = run(gq, planes, w, table, lens, 64, 10, 10)
    check(got, reference(planes, w, table, lens, 64, 10, 10))
    assert got[0][0, 0, 20:].eq(-1).all()


def test_bad_lengths_and_pages_are_reported(gq):
    lens = [100, 60, 90]
    planes, w, table = make("bf16", 3, 2, 64, 16, lens, 5, "heavy", S=112)
    for bad in (-3, 113):
        got = run(gq, planes, w, table, [100, bad, 90], 32, 4, 2)
        assert gq.get_device_status() == 5
        want = reference(planes, w, table, [100, 0, 90], 32, 4, 2)
        want[1][1] = bad
        check(got, want)
    t = table.clone()
    t[0, 3] = -1                                     # positions 48..63 of row 0: the smallest weights, not moved
    got = run(gq, planes, w, t, lens, 32, 4, 2)
    assert gq.get_device_status() == 11
    ref_w = w.clone()
    ref_w[table[0, 3].long()] = -math.inf
    want = reference(planes, ref_w, table, lens, 32, 4, 2)
    assert torch.equal(got[0], want[0])
    for a, b in zip(got[2][1:], want[2][1:]):
        assert torch.equal(a, b)


def test_given_outputs_and_a_stream(gq):
    lens = [500, 40]
    planes, w, table = make("bf16", 2, 2, 128, 0, lens, 6, "heavy")
    kept = torch.empty(2, 2, 64, dtype=torch.int32, device="cuda")
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    dev, wd, ln = [p.cuda() for p in planes], w.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    s.wait_stream(torch.cuda.current_stream())
    k, o = gq.attn_cache_evict(wd, dev, ln, 64, recent=8, kept=kept, lens_out=out, stream=s)
    s.synchronize()
    assert k is kept or k.data_ptr() == kept.data_ptr()
    want = reference(planes, w, table, lens, 64, 8, 0)
    check((k.cpu(), o.cpu(), [x.view(torch.uint8).reshape(*x.shape[:3], -1).cpu() for x in (wd.unsqueeze(-1), *dev)]), want)


def test_arguments(gq):
    planes, w, table = make("bf16", 2, 2, 64, 0, [50, 40], 7, "heavy")
    wd, dev, ln = w.cuda(), [p.cuda() for p in planes], torch.tensor([50, 40], dtype=torch.int32).cuda()
    f = gq.attn_cache_evict
    with pytest.raises(ValueError, match="budget"):
        f(wd, dev, ln, 0)
    with pytest.raises(gq.AttnError, match="SHAPE"):
        f(wd, dev, ln, 8, recent=5, first=4)
    with pytest.raises(gq.AttnError, match="SHAPE"):
        f(wd, dev, ln, 8, recent=-1)
    with pytest.raises(gq.AttnError, match="SHAPE"):                          # the same plane twice
        f(wd, [dev[0], dev[0]], ln, 8)
    with pytest.raises(gq.AttnError, match="SHAPE"):                          # in place: lengths are read while rows move
        f(wd, dev, ln, 8, lens_out=ln)
    with pytest.raises(gq.AttnError, match="SHAPE"):                          # rows of 3 bytes
        f(wd, [torch.zeros(2, 2, 50, 3, dtype=torch.uint8, device="cuda")], ln, 8)
    with pytest.raises(ValueError, match="as weights"):
        f(wd, [dev[0][:, :, :40].contiguous()], ln, 8)
    with pytest.raises(ValueError, match="contiguous"):
        f(wd, [dev[0].transpose(0, 1).contiguous().transpose(0, 1)], ln, 8)
    with pytest.raises(ValueError, match="block_table"):
        f(wd, dev, ln[:1].contiguous(), 8)
    with pytest.raises(ValueError, match="at most 8"):
        f(wd, dev * 5, ln, 8)
    with pytest.raises(TypeError, match="float32"):
        f(wd.double(), dev, ln, 8)
    with pytest.raises(ValueError, match="kept"):
        f(wd, dev, ln, 8, kept=torch.zeros(2, 2, 9, dtype=torch.int32, device="cuda"))
    assert torch.equal(wd.cpu(), w)
