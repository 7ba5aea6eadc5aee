"""4-bit cached attention on the same rows in caches of two capacities: few units of short rows go to a cluster of CTAs
each, in a cache of 13000 positions they are shared out as one stream.  Both against 64 bits, tolerances as there."""
import math

import pytest
import torch

import cache_ref as R
from causal_gqa_attention_fwd_gb300 import workloads as W
from test_gpu_decode_q4 import KS, VS, cache_of, close, lens_of, queries, reference, run

pytestmark = pytest.mark.gpu
S2 = 13000


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


def wide(cache, S2):
    """The caches with S2 positions a row, any bytes (NaN scales among them) behind the first S."""
    g = torch.Generator().manual_seed(70)
    out = []
    for c in cache:
        w = torch.randint(0, 256, (*c.shape[:2], S2, c.shape[3]), generator=g, dtype=torch.uint8)
        w[:, :, :c.shape[2]] = c
        out.append(w)
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,Tq,S,lens", [
    (3, 8, 2, 1, 701, [701, 1, 389]), (2, 16, 2, 4, 640, [640, 385]), (6, 4, 4, 2, 97, [97, 0, 1, 2, 96, 65]),
    (2, 5, 1, 7, 1111, [1111, 5]), (1, 3, 1, 1, 3000, [2999]), (5, 2, 1, 3, 300, [300, 33, 2, 0, 31]), (20, 6, 3, 1, 130, None),
    (1, 1, 1, 1, 5, [5]), (9, 14, 2, 1, 2100, None)])
def test_decode_q4_in_clusters_and_as_a_stream(gq, B, Hq, Hkv, Tq, S, lens, rope, D):
    lens = lens_of(lens) if lens else torch.randint(0, S + 1, (B,), generator=torch.Generator().manual_seed(B), dtype=torch.int32)
    tab = W.rope_cos_sin_table(S2, D) if rope else None
    q, cache = queries(B, Hq, Tq, D, 71), cache_of(B, Hkv, S, D, 72)
    cache[1].view(-1)[::997] = 0x7f                # NaN blocks here and there
    cache[3].view(-1)[5::1013] = 0xff
    ref = reference(q, cache, lens, 0.09, tab=tab)
    for c in (cache, wide(cache, S2)):
        o, lse = run(gq, q, c, lens, 0.09, tab=tab)
        assert gq.get_device_status() == 0
        close(o, lse, ref)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("Hq,Tq,rope", [(4, 1, True), (8, 3, False), (20, 2, True)])
def test_decode_paged_q4_in_clusters_and_as_a_stream(gq, page, Hq, Tq, rope):
    B, Hkv, D, S = 3, 2, 128, 768
    lens = lens_of([768, 411, 16])
    tab = W.rope_cos_sin_table(S2 + 256, D) if rope else None
    n = B * S // page + 3
    table = torch.randperm(n, generator=torch.Generator().manual_seed(page))[:B * S // page].reshape(B, -1).to(torch.int32)
    q, cache = queries(B, Hq, Tq, D, 73), cache_of(n, Hkv, page, D, 74)
    ref = reference(q, cache, lens, 0.08, table, tab=tab)
    long = torch.full((B, -(-S2 // page)), -1, dtype=torch.int32)
    long[:, :table.shape[1]] = table
    for t in (table, long):
        o, lse = run(gq, q, cache, lens, 0.08, t, tab)
        assert gq.get_device_status() == 0
        close(o, lse, ref)


@pytest.mark.parametrize("D,S,Hkv", [(128, 2048, 2), (64, 2048, 16), (128, 2048, 20), (64, 1500, 25), (128, 700, 40), (128, 256, 70), (128, 900, 128), (64, 12288, 1)])
def test_decode_q4_cluster_sizes(gq, D, S, Hkv):
    """One row: from a whole cluster for each of few units to a CTA a unit; lengths from one tile to the capacity."""
    for n in (1, 33, S // 2 + 1, S):
        q, cache = queries(1, Hkv * 2, 1, D, n), cache_of(1, Hkv, S, D, 75)
        o, lse = run(gq, q, cache, lens_of([n]), 1 / math.sqrt(D))
        assert gq.get_device_status() == 0
        close(o, lse, reference(q, cache, lens_of([n]), 1 / math.sqrt(D)))


def test_decode_q4_clusters_report_lengths_and_are_captured(gq):
    """Invalid lengths in some rows; a captured call that follows the lengths, and gives the same bits each time."""
    B, Hq, Hkv, D, S = 4, 4, 2, 128, 500
    q, cache = queries(B, Hq, 1, D, 76), cache_of(B, Hkv, S, D, 77)
    lens = lens_of([500, -1, 501, 77]).cuda()
    dev = [c.cuda() for c in cache]
    o, lse = torch.full((B, Hq, 1, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((B, Hq, 1), 7.0, device="cuda")
    qd = q.cuda()
    gq.attn_decode_q4_fwd(qd, *dev, KS, VS, lens, scale=0.1, o=o, lse=lse)
    assert gq.get_device_status() == 5
    assert (o[1:3] == 7).all() and (lse[1:3] == 7).all()
    ref = reference(q[[0, 3]], [c[[0, 3]] for c in cache], lens_of([500, 77]), 0.1)
    close(o[[0, 3]], lse[[0, 3]], ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gq.attn_decode_q4_fwd(qd, *dev, KS, VS, lens, scale=0.1, o=o, lse=lse)
    gq.get_device_status()
    for n in ([500, 1, 0, 64], [3, 499, 250, 128], [500, 1, 0, 64]):
        lens.copy_(lens_of(n))
        g.replay()
        first = o.clone(), lse.clone()
        g.replay()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
        assert gq.get_device_status() == 0
        close(o, lse, reference(q, cache, lens_of(n), 0.1))


@pytest.mark.parametrize("D,Hq,Hkv,Tq,rope", [(64, 14, 2, 1, False), (128, 16, 4, 4, False), (128, 4, 1, 1, True), (64, 8, 1, 2, True)])
def test_decode_q4_clusters_repeat_themselves(gq, D, Hq, Hkv, Tq, rope):
    """Every piece of every call is joined: 300 replays of four calls over other lengths give the first ones' bits."""
    B, S = 2, 2048
    q, cache = queries(B, Hq, Tq, D, 78).cuda(), [c.cuda() for c in cache_of(B, Hkv, S, D, 79)]
    tab = W.rope_cos_sin_table(S, D).cuda() if rope else None
    lens = [lens_of(n).cuda() for n in ([S, 1], [33, 700], [1500, 64], [97, 2000])]
    calls = lambda: [gq.attn_decode_q4_fwd(q, *cache, KS, VS, n, scale=0.1, rope_cos_sin=tab) for n in lens]  # noqa: E731
    want = calls()
    for n, (o, lse) in zip(lens, want):
        close(o, lse, reference(q.cpu(), [c.cpu() for c in cache], n.cpu(), 0.1, tab=None if tab is None else tab.cpu()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = calls()
    for _ in range(300):
        g.replay()
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    assert gq.get_device_status() == 0
