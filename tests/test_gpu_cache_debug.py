"""The cache operators in the debug build (bounds checks on every cache offset and output row): odd sizes raise no check
and give the release build's bits."""
import pytest
import torch

import cache_ref as R
from test_gpu_decode_q4 import cache_of, close, paged, queries, reference
from test_gpu_rope_ops import table

pytestmark = pytest.mark.gpu
KS, VS = 0.0031, 0.0023


@pytest.fixture(scope="module")
def dbg():
    from causal_gqa_attention_fwd_gb300 import _binding, build
    path = build.build(debug=True)
    saved = (_binding._lib, _binding.LIB_PATH)
    _binding._lib, _binding.LIB_PATH = None, path
    assert _binding.lib().attn_is_debug_build() == 1
    import causal_gqa_attention_fwd_gb300 as g
    yield g
    _binding._lib, _binding.LIB_PATH = saved


def no_check_fired(g):
    assert g.get_device_status() == 0
    assert g.get_check_line() == 0


def test_the_native_module_calls_the_loaded_library(dbg):
    """The operators follow _binding to the debug library: its own status word records the error."""
    bad = torch.tensor([99], dtype=torch.int32).cuda()
    dbg.attn_rope(torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda"), None, bad, torch.zeros(4, 64, device="cuda"))
    assert dbg.get_device_status() == 5
    from causal_gqa_attention_fwd_gb300 import _binding, _cache
    assert _cache._bound is _binding._lib


@pytest.mark.parametrize("B,Hq,Hkv,Tq,S,D,lens", [(1, 1, 1, 1, 1, 64, [1]), (2, 12, 2, 3, 65, 128, [65, 2]),
                                                  (3, 8, 1, 1, 333, 128, [333, 0, 32]), (2, 20, 1, 1, 129, 64, [129, 97])])
def test_debug_decode(dbg, B, Hq, Hkv, Tq, S, D, lens):
    lens = torch.tensor(lens, dtype=torch.int32)
    q, cache = queries(B, Hq, Tq, D, 3), cache_of(B, Hkv, S, D, 4)
    o, lse = dbg.attn_decode_q4_fwd(q.cuda(), *[c.cuda() for c in cache], KS, VS, lens.cuda(), scale=0.1)
    no_check_fired(dbg)
    close(o, lse, reference(q, cache, lens, 0.1))


@pytest.mark.parametrize("page", [16, 32, 128])
def test_debug_decode_paged(dbg, page):
    B, Hq, Hkv, D, mp = 3, 8, 2, 128, 9
    lens = torch.tensor([page * mp, 1, page * 3 + 5], dtype=torch.int32)
    bt, cache = paged(B, Hkv, page, mp, D, lens, 5, spare=0)
    q = queries(B, Hq, 1, D, 6)
    o, lse = dbg.attn_decode_paged_q4_fwd(q.cuda(), *[c.cuda() for c in cache], KS, VS, bt.cuda(), lens.cuda(), scale=0.1)
    no_check_fired(dbg)
    close(o, lse, reference(q, cache, lens, 0.1, bt))


@pytest.mark.parametrize("D,H,page", [(64, 1, 16), (128, 5, 48)])
def test_debug_append(dbg, D, H, page):
    n, pages = 37, 4
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn(n, H, D, generator=g).bfloat16() for _ in range(2))
    slots = torch.randperm(pages * page, generator=g)[:n].to(torch.int32)
    slots[5] = pages * page - 1 if pages * page - 1 not in slots.tolist() else -1      # the cache's last row
    z = lambda w: torch.zeros(pages, H, page, w, dtype=torch.uint8)  # noqa: E731
    cache = [z(D // 2), z(D // 16), z(D // 2), z(D // 16)]
    tab, pos = table(50, 32), torch.randint(0, 50, (n,), generator=g, dtype=torch.int32)
    dev = [c.cuda() for c in cache]
    dbg.attn_cache_append_q4(k.cuda(), v.cuda(), slots.cuda(), *dev, KS, VS, positions=pos.cuda(), rope_cos_sin=tab.cuda())
    no_check_fired(dbg)
    want = [*R.quantise(R.rope(k, pos[:, None], tab, False, dtype=torch.float32), KS), *R.quantise(v.float(), VS)]
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            for c, w in zip(dev, want):
                assert torch.equal(c[s // page, :, s % page].cpu(), w[i])
