"""Appending to bf16, E4M3 and 4-bit caches, and gathering from 4-bit ones.

The stored bits are defined by float32 elementary operations (products and sums
rounded one by one), so they are compared for equality with a float32 reference."""
import numpy as np
import pytest
import torch

import cache_ref as R
from test_gpu_rope_ops import table

pytestmark = pytest.mark.gpu
KS, VS = 0.0031, 0.0023


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


def caches(fmt, pages, H, page, D, fill=0xA5):
    z = lambda w: torch.full((pages, H, page, w), fill, dtype=torch.uint8)  # noqa: E731
    if fmt == "q4":
        return [z(D // 2), z(D // 16), z(D // 2), z(D // 16)]
    return [z(D), z(D)] if fmt == "fp8" else [z(2 * D).view(torch.bfloat16), z(2 * D).view(torch.bfloat16)]


def append(gq, fmt, k, v, slots, cache, **kw):
    dev = [c.cuda() for c in cache]
    if fmt == "bf16":
        gq.attn_cache_append(k, v, slots, *dev, **kw)
    else:
        f = gq.attn_cache_append_fp8 if fmt == "fp8" else gq.attn_cache_append_q4
        f(k, v, slots, *dev, KS, VS, **kw)
    return [c.cpu() for c in dev]


def stored(fmt, k, v):
    """What the caches' rows hold for float32 k, v [n,H,D]."""
    if fmt == "bf16":
        return [k.bfloat16(), v.bfloat16()]
    if fmt == "fp8":
        return [(x * float(np.float32(1) / np.float32(s))).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for x, s in ((k, KS), (v, VS))]
    return [t for x, s in ((k, KS), (v, VS)) for t in R.quantise(x, s)]


def expect(cache, rows, slots, page):
    out = [c.clone() for c in cache]
    for i, s in enumerate(slots.flatten().tolist()):
        if s >= 0:
            for c, r in zip(out, rows):
                c[s // page, :, s % page] = r[i]
    return out


def same(a, b):
    for x, y in zip(a, b):
        x, y = (t.view(torch.int16) if t.dtype == torch.bfloat16 else t for t in (x, y))
        assert torch.equal(x, y)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "q4"])
@pytest.mark.parametrize("n,H,D,page,r,inter", [
    (1, 1, 64, 16, 0, False), (7, 8, 128, 64, 128, False), (33, 2, 64, 48, 16, True), (300, 3, 128, 16, 96, False),
    (1021, 2, 128, 256, 64, True), (130, 8, 64, 1, 64, False), (65, 1, 128, 32, 32, False)])
def test_append_packed(gq, fmt, n, H, D, page, r, inter):
    """Strided views, padded tokens (slot -1), shuffled slots; rows not named keep every byte."""
    g = torch.Generator().manual_seed(n * 7 + D)
    x = (torch.randn(n, 2 * H + 1, D, generator=g) * 1.3).bfloat16()
    k, v = x[:, :H], x[:, H:2 * H]
    pages = -(-n // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:n].to(torch.int32)
    slots[torch.rand(n, generator=g) < 0.1] = -1
    cache = caches(fmt, pages, H, page, D)
    kw, kf = {}, k.float()
    if r:
        tab, pos = table(500, r), torch.randint(0, 500, (n,), generator=g, dtype=torch.int32)
        kw = dict(positions=pos.cuda(), rope_cos_sin=tab.cuda(), interleaved=inter)
        kf = R.rope(k, pos[:, None], tab, inter, dtype=torch.float32)
    xd = x.cuda()
    got = append(gq, fmt, xd[:, :H], xd[:, H:2 * H], slots.cuda(), cache, **kw)
    assert gq.get_device_status() == 0
    same(got, expect(cache, stored(fmt, kf, v.float()), slots, page))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "q4"])
def test_append_contiguous_cache_of_odd_capacity(gq, fmt):
    """[B,Hkv,T,D] tokens into a [B,Hkv,S,D] cache: slot b*S + j."""
    B, H, T, D, S = 3, 2, 5, 64, 37
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(B, H, T, D, generator=g).bfloat16() for _ in range(2))
    at = torch.tensor([0, 32, 11])
    slots = (torch.arange(B)[:, None] * S + at[:, None] + torch.arange(T)).to(torch.int32)
    cache = caches(fmt, B, H, S, D)
    got = append(gq, fmt, k.cuda(), v.cuda(), slots.cuda(), cache)
    assert gq.get_device_status() == 0
    rows = stored(fmt, *(x.float().transpose(1, 2).reshape(B * T, H, D) for x in (k, v)))
    same(got, expect(cache, rows, slots, S))


def test_append_q4_edges(gq):
    """Ties, saturation, zeros, subnormal block scales, values no scale holds, NaN and infinities."""
    D = 64
    unit = float(np.float32(KS) * 16)            # block scale 16 when the block's largest is 6 units
    lv = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 0.1])
    rows = torch.zeros(12, 4, 16)
    rows[0] = lv * unit
    rows[1] = torch.randn(4, 16, generator=torch.Generator().manual_seed(0)) * 1e-5      # scale rounds to 0
    rows[2] = torch.randn(4, 16, generator=torch.Generator().manual_seed(1)) * 2e-4      # subnormal scale
    rows[3] = 1e30                                                                        # saturates
    rows[4, 1, 3] = float("nan")
    rows[5, 2, 9] = float("-inf")
    rows[6] = torch.randn(4, 16, generator=torch.Generator().manual_seed(2)) * 40
    rows[7, :, 5] = -3e38
    rows[8] = -0.0
    x = rows.reshape(12, 1, D).bfloat16()
    v = torch.randn(12, 1, D).bfloat16()
    slots = torch.arange(12, dtype=torch.int32)
    cache = caches("q4", 1, 1, 12, D)
    got = append(gq, "q4", x.cuda(), v.cuda(), slots.cuda(), cache)
    assert gq.get_device_status() == 0
    same(got, expect(cache, stored("q4", x.float(), v.float()), slots, 12))
    k2, v2 = gq.attn_cache_gather_q4(slots.cuda(), *[c.cuda() for c in got], KS, VS)
    assert gq.get_device_status() == 0
    ref = R.values(got[0], got[1], KS)[0, 0]
    assert torch.equal(torch.isnan(k2.cpu()[:, 0]), torch.isnan(ref))
    assert torch.isnan(ref[4, 16:32]).all() and torch.isnan(ref[5, 32:48]).all()


def test_append_q4_is_near(gq):
    """Ordinary values: off by at most half the widest step (1 unit between 4 and 6, or 6/16 where the block scale
    was rounded down by its half step 2^-4 and the largest saturates), unit = block scale * scale."""
    n, H, D = 200, 2, 128
    k = torch.randn(n, H, D, generator=torch.Generator().manual_seed(9)).bfloat16()
    slots = torch.arange(n, dtype=torch.int32)
    got = append(gq, "q4", k.cuda(), k.cuda(), slots.cuda(), caches("q4", 1, H, n, D))
    for i, s in ((0, KS), (2, VS)):
        val = R.values(got[i], got[i + 1], s)[0].transpose(0, 1)
        unit = (R.e4m3(got[i + 1]) * s)[0].transpose(0, 1).repeat_interleave(16, -1)
        assert ((val - k.double()).abs() <= unit * (1 + 1e-6)).all()


def test_append_fp8_edges(gq):
    x = torch.zeros(3, 1, 64)
    x[0, 0, :8] = torch.tensor([float("nan"), float("inf"), float("-inf"), 1e30, -1e30, 448 * KS * 1.01, 1e-9, -1e-9])
    x = x.bfloat16()
    slots = torch.arange(3, dtype=torch.int32)
    cache = caches("fp8", 1, 1, 3, 64)
    got = append(gq, "fp8", x.cuda(), x.cuda(), slots.cuda(), cache)
    a, b = R.e4m3(got[0]), R.e4m3(expect(cache, stored("fp8", x.float(), x.float()), slots, 3)[0])
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "q4"])
def test_append_reports_bad_slots_and_positions(gq, fmt):
    """A slot outside the cache or a position outside the table is reported; that token is not written, the rest is."""
    n, H, D, page = 6, 2, 64, 16
    k = torch.randn(n, H, D).bfloat16()
    slots = torch.tensor([0, 32, -2, 31, -1, 2 ** 31 - 1], dtype=torch.int32)
    cache = caches(fmt, 2, H, page, D)
    got = append(gq, fmt, k.cuda(), k.cuda(), slots.cuda(), cache)
    assert gq.get_device_status() == 11
    keep = torch.tensor([0, -1, -1, 31, -1, -1])
    same(got, expect(cache, stored(fmt, k.float(), k.float()), keep, page))
    tab, pos = table(9, 64), torch.tensor([9, 0, 0, 8, 0, 0], dtype=torch.int32)
    slots = torch.tensor([0, -1, -1, 31, -1, -1], dtype=torch.int32)
    got = append(gq, fmt, k.cuda(), k.cuda(), slots.cuda(), cache, positions=pos.cuda(), rope_cos_sin=tab.cuda())
    assert gq.get_device_status() == 5
    kf = R.rope(k, pos.clamp(max=8)[:, None], tab, False, dtype=torch.float32)
    same(got, expect(cache, stored(fmt, kf, k.float()), torch.tensor([-1, -1, -1, 31, -1, -1]), page))


@pytest.mark.parametrize("n,H,D,page", [(1, 1, 64, 16), (77, 3, 128, 32), (1000, 8, 64, 16)])
def test_gather_q4(gq, n, H, D, page):
    """Random codes and scales (NaN codes too): each value rounded once to f32, once to bf16."""
    g = torch.Generator().manual_seed(n)
    pages = -(-n // page) + 1
    cache = [torch.randint(0, 256, (pages, H, page, w), generator=g, dtype=torch.uint8) for w in (D // 2, D // 16) * 2]
    slots = torch.randint(0, pages * page, (n,), generator=g, dtype=torch.int32)
    slots[0] = -1
    k, v = gq.attn_cache_gather_q4(slots.cuda(), *[c.cuda() for c in cache], KS, VS)
    assert gq.get_device_status() == 0
    for y, i, s in ((k, 0, KS), (v, 2, VS)):
        ref = R.values(cache[i], cache[i + 1], s).transpose(1, 2).flatten(0, 1)[slots.long().clamp(min=0)]
        ref[0] = 0
        y = y.double().cpu()
        assert torch.equal(torch.isnan(y), torch.isnan(ref))
        ok = ~torch.isnan(ref)
        assert ((y - ref)[ok].abs() <= (2.0 ** -8 + 2.0 ** -24) * ref[ok].abs()).all()
    bad = torch.tensor([pages * page, -7], dtype=torch.int32)
    k, v = gq.attn_cache_gather_q4(bad.cuda(), *[c.cuda() for c in cache], KS, VS)
    assert gq.get_device_status() == 11
    assert (k == 0).all() and (v == 0).all()
