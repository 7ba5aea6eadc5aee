"""Caches larger than 2^32 bytes under shared prefixes, weights and eviction: offsets that pass 32 bits.  The memory is not
initialised; only the slots a test writes are read."""
import math

import pytest
import torch

import pressure_ref as R
from test_gpu_cache_evict import check as check_evict, reference as evict_reference
from test_gpu_cache_weights import check as check_weights, lse_of
from test_gpu_decode_prefix import check, tile_capacity

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    yield g
    torch.cuda.empty_cache()


PAGES, H, PAGE, D = 280_000, 2, 32, 128      # 4.6 GB of bf16 keys


def pool(dtype=torch.bfloat16, *w):
    return torch.empty(PAGES, H, PAGE, *w, dtype=dtype, device="cuda")


@pytest.mark.parametrize("tiles", [False, True])
def test_prefix_pages_beyond_4_gib(gq, tiles):
    B, Hq, m, lens = 3, 32, 70, [1, 40, 33]
    g = torch.Generator().manual_seed(1)
    k, v = pool(torch.bfloat16, D), pool(torch.bfloat16, D)
    assert k.numel() * 2 > 2 ** 32
    wide = tile_capacity(B, 1, Hq, H, 1, D) // PAGE if tiles else 3
    pt = torch.full((1, wide), -1, dtype=torch.int32)
    pt[0, :3] = torch.tensor([PAGES - 1, 262_145, PAGES - 7])
    bt = torch.tensor([[PAGES - 2, -1], [PAGES - 3, PAGES - 4], [270_000, PAGES - 5]], dtype=torch.int32)
    rn = lambda n: torch.randn(H, n, D, generator=g).bfloat16()  # noqa: E731
    pre, own = (rn(m), rn(m)), [(rn(n), rn(n)) for n in lens]
    for pairs, t in (([pre], pt), (own, bt)):
        for b, kv in enumerate(pairs):
            for pool_, x in zip((k, v), kv):
                for j0 in range(0, x.shape[1], PAGE):
                    c = min(PAGE, x.shape[1] - j0)
                    pool_[int(t[b, j0 // PAGE]), :, :c] = x[:, j0:j0 + c].cuda()
    q = torch.randn(B, Hq, 1, D, generator=g).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    got = gq.attn_decode_paged_prefix_fwd(q.cuda(), k, v, pt.cuda(), i32([m]), bt.cuda(), i32(lens))
    assert gq.get_device_status() == 0
    d64 = lambda kv: tuple(x.double() for x in kv)  # noqa: E731
    check(got, R.prefix(q, [d64(pre)], [d64(kv) for kv in own], lens, 1 / math.sqrt(D)), D)


def test_weights_and_eviction_beyond_4_gib(gq):
    """Rows whose pages lie at both ends of the pool, weighed and then cut; every page that no row names stays as it was."""
    lens, budget = [90, 33], 40
    g = torch.Generator().manual_seed(2)
    table = torch.tensor([[PAGES - 1, 3, PAGES - 9], [262_200, PAGES - 4, -1]], dtype=torch.int32)
    used = [int(x) for x in table.flatten() if x >= 0]
    k, v, w = pool(torch.bfloat16, D), pool(torch.bfloat16, D), pool(torch.float32)
    for p in used:
        k[p], v[p] = (torch.randn(H, PAGE, D, generator=g).bfloat16().cuda() for _ in range(2))
        w[p] = torch.rand(H, PAGE, generator=g).cuda()
    # the same pages as a small pool, for the references
    small = torch.tensor([[used.index(int(x)) if x >= 0 else -1 for x in row] for row in table], dtype=torch.int32)
    at = torch.tensor(used)
    sk, sv, sw = (x[at.cuda()].cpu() for x in (k, v, w))
    q = torch.randn(2, 8, 2, D, generator=g).bfloat16()
    lse = lse_of(q, sk.double(), small, lens, 0.09)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    gq.attn_cache_weights(q.cuda(), k, lse.cuda(), n, w, block_table=table.cuda(), scale=0.09)
    assert gq.get_device_status() == 0
    check_weights(w[at.cuda()], sw, q, sk.double(), lse, small, lens, 0.09)
    now = w[at.cuda()].cpu()
    kept, out = gq.attn_cache_evict(w, (k, v), n, budget, recent=7, first=2, block_table=table.cuda())
    assert gq.get_device_status() == 0
    raw = [x[at.cuda()].cpu() for x in (w.unsqueeze(-1), k, v)]
    check_evict((kept.cpu(), out.cpu(), [x.view(torch.uint8).reshape(*x.shape[:3], -1) for x in raw]),
                evict_reference([sk, sv], now, small, lens, budget, 7, 2))


def test_eviction_of_contiguous_rows_beyond_4_gib(gq):
    """[3, 2, 9M, 128] E4M3 codes: the last rows and heads lie past 2^32 bytes."""
    B, S, lens = 3, 9_000_000, [50, 20, 61]
    c = torch.empty(B, H, S, D, dtype=torch.uint8, device="cuda")
    w = torch.empty(B, H, S, device="cuda")
    assert c.numel() > 2 ** 32
    g = torch.Generator().manual_seed(3)
    sc, sw = torch.randint(0, 256, (B, H, 64, D), generator=g, dtype=torch.uint8), torch.rand(B, H, 64, generator=g)
    c[:, :, :64], w[:, :, :64] = sc.cuda(), sw.cuda()
    kept, out = gq.attn_cache_evict(w, (c,), torch.tensor(lens, dtype=torch.int32).cuda(), 24, recent=5)
    assert gq.get_device_status() == 0
    raw = [x[:, :, :64].cpu().contiguous() for x in (w.unsqueeze(-1), c)]
    check_evict((kept.cpu(), out.cpu(), [x.view(torch.uint8).reshape(*x.shape[:3], -1) for x in raw]),
                evict_reference([sc], sw, None, lens, 24, 5, 0))
