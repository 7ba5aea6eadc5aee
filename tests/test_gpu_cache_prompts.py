"""Rotary rows, append and gather at prompt sizes, where a thread takes several heads in turn: head counts that its
share does not divide, tokens that are not a block's worth, padded and bad tokens among them.  Tolerances as at the small
sizes."""
import pytest
import torch

import cache_ref as R
from test_gpu_cache_append import KS, VS, append, caches, expect, same, stored, table
from test_gpu_rope_ops import close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "q4"])
@pytest.mark.parametrize("n,H,D,page,r,inter", [
    (5003, 5, 128, 16, 0, False), (5003, 5, 128, 64, 128, False), (5003, 7, 128, 16, 96, False), (5003, 5, 128, 48, 16, False),
    (5003, 6, 128, 32, 64, True), (10007, 5, 64, 16, 64, False), (10007, 3, 64, 16, 32, True)])
def test_append_prompts(gq, fmt, n, H, D, page, r, inter):
    g = torch.Generator().manual_seed(n + D + r)
    x = (torch.randn(n, 2 * H, D, generator=g) * 1.3).bfloat16()
    pages = -(-n // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:n].to(torch.int32)
    slots[torch.rand(n, generator=g) < 0.1] = -1
    cache = caches(fmt, pages, H, page, D)
    kw, kf = {}, x[:, :H].float()
    if r:
        tab, pos = table(700, r), torch.randint(0, 700, (n,), generator=g, dtype=torch.int32)
        kw = dict(positions=pos.cuda(), rope_cos_sin=tab.cuda(), interleaved=inter)
        kf = R.rope(x[:, :H], pos[:, None], tab, inter, dtype=torch.float32)
    xd = x.cuda()
    got = append(gq, fmt, xd[:, :H], xd[:, H:], slots.cuda(), cache, **kw)
    assert gq.get_device_status() == 0
    want = expect(cache, stored(fmt, kf, x[:, H:].float()), slots, page)
    same(got, want)
    bad = slots.clone()
    bad[7], bad[n - 1] = pages * page, -5
    got = append(gq, fmt, xd[:, :H], xd[:, H:], bad.cuda(), cache, **kw)
    assert gq.get_device_status() == 11
    bad[7] = bad[n - 1] = -1
    same(got, expect(cache, stored(fmt, kf, x[:, H:].float()), bad, page))


@pytest.mark.parametrize("n,H,D", [(5003, 7, 128), (10007, 5, 64)])
def test_gather_prompts(gq, n, H, D):
    g = torch.Generator().manual_seed(n)
    page, pages = 16, n // 16 + 2
    cache = [torch.randint(0, 256, (pages, H, page, w), generator=g, dtype=torch.uint8) for w in (D // 2, D // 16) * 2]
    slots = torch.randint(-1, pages * page, (n,), generator=g, dtype=torch.int32)
    slots[3] = -1
    k, v = gq.attn_cache_gather_q4(slots.cuda(), *[c.cuda() for c in cache], KS, VS)
    assert gq.get_device_status() == 0
    for y, i, s in ((k, 0, KS), (v, 2, VS)):
        ref = R.values(cache[i], cache[i + 1], s).transpose(1, 2).flatten(0, 1)[slots.long().clamp(min=0)]
        ref[slots < 0] = 0
        y = y.double().cpu()
        assert torch.equal(torch.isnan(y), torch.isnan(ref))
        ok = ~torch.isnan(ref)
        assert ((y - ref)[ok].abs() <= (2.0 ** -8 + 2.0 ** -24) * ref[ok].abs()).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,Hq,Hkv,D,r", [(5003, 9, 2, 128, 128), (5003, 14, 3, 64, 64), (9001, 12, 4, 80, 48), (3001, 7, 2, 512, 256)])
def test_rope_prompts(gq, n, Hq, Hkv, D, r, inter):
    g = torch.Generator().manual_seed(n + D)
    q, k = (torch.randn(n, h, D, generator=g).bfloat16() for h in (Hq, Hkv))
    pos = torch.randint(0, 300, (n,), generator=g, dtype=torch.int32)
    tab = table(300, r)
    qd, kd = q.cuda(), k.cuda()
    for fn, sign in ((gq.attn_rope, 1.0), (gq.attn_rope_bwd, -1.0)):
        qo, ko = fn(qd, kd, pos.cuda(), tab.cuda(), inter)
        assert gq.get_device_status() == 0
        for x, y in ((q, qo), (k, ko)):
            close(y, R.rope(x, pos[:, None], tab, inter, sign), x, r)
    qo, ko = gq.attn_rope(qd, kd, pos.cuda(), tab.cuda(), inter)
    a, b = gq.attn_rope(qd, kd, pos.cuda(), tab.cuda(), inter, qd, kd)
    assert a is qd and torch.equal(a, qo) and torch.equal(b, ko)          # in place
    pos[11] = 300
    qo, ko = gq.attn_rope(q.cuda(), k.cuda(), pos.cuda(), tab.cuda(), inter)
    assert gq.get_device_status() == 5 and not qo[11].any() and not ko[11].any()
