"""Caches larger than 2^32 bytes: offsets that pass 32 bits, in the page pool and in a contiguous cache's rows and heads.
The memory is not initialised; only the rows a test writes are read."""
import math

import pytest
import torch

import cache_ref as R
from test_gpu_decode_q4 import close, queries

pytestmark = pytest.mark.gpu
KS, VS = 0.0029, 0.0021


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    yield g
    torch.cuda.empty_cache()


def raw(*shape, dtype=torch.uint8):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def pool(pages, H, page, D):
    return [raw(pages, H, page, w) for w in (D // 2, D // 16) * 2]


def quantised(k, v):
    return [R.values(*R.quantise(x.float(), s), s) for x, s in ((k, KS), (v, VS))]


def test_q4_pages_beyond_4_gib(gq):
    """The last pages of a pool of 4.9 GB of codes: append, gather, attention."""
    pages, H, page, D, n = 300_000, 2, 128, 128, 300
    cache = pool(pages, H, page, D)
    assert cache[0].numel() > 2 ** 32
    table = torch.tensor([[pages - 1, pages - 3, 262_145]], dtype=torch.int32)
    slots = (table[0].long()[:, None] * page + torch.arange(page)).flatten()[:n].to(torch.int32).cuda()
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(n, H, D, generator=g).bfloat16() for _ in range(2))
    gq.attn_cache_append_q4(k.cuda(), v.cuda(), slots, *cache, KS, VS)
    kk, vv = gq.attn_cache_gather_q4(slots, *cache, KS, VS)
    K, V = quantised(k, v)
    for got, want in ((kk, K), (vv, V)):
        assert ((got.double().cpu() - want).abs() <= (2.0 ** -8 + 2.0 ** -24) * want.abs()).all()
    q = queries(1, 8, 1, D, 2)
    o, lse = gq.attn_decode_paged_q4_fwd(q.cuda(), *cache, KS, VS, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    assert gq.get_device_status() == 0
    close(o, lse, R.decode(q, K.transpose(0, 1)[None], V.transpose(0, 1)[None], [n], 1 / math.sqrt(D)))


def test_q4_contiguous_rows_beyond_4_gib(gq):
    """[3, 2, 24M, 64]: the rows of the last batch entries and heads lie past 2^32 bytes."""
    B, H, S, D = 3, 2, 24_000_000, 128
    cache = pool(B, H, S, D)
    assert (B - 1) * H * S * (D // 2) > 2 ** 32
    lens = [3, 0, 77]
    g = torch.Generator().manual_seed(3)
    K, V = (torch.zeros(B, H, 80, D, dtype=torch.float64) for _ in range(2))
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k, v = (torch.randn(n, H, D, generator=g).bfloat16() for _ in range(2))
        slots = (b * S + torch.arange(n)).to(torch.int32).cuda()
        gq.attn_cache_append_q4(k.cuda(), v.cuda(), slots, *cache, KS, VS)
        kq, vq = quantised(k, v)
        K[b, :, :n], V[b, :, :n] = kq.transpose(0, 1), vq.transpose(0, 1)
    q = queries(B, 4, 1, D, 4)
    o, lse = gq.attn_decode_q4_fwd(q.cuda(), *cache, KS, VS, torch.tensor(lens, dtype=torch.int32).cuda())
    assert gq.get_device_status() == 0
    close(o, lse, R.decode(q, K, V, lens, 1 / math.sqrt(D)))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_append_heads_beyond_4_gib(gq, fmt):
    """One row of 20M positions: the second and third K/V heads begin 2.5 to 10 GB further on."""
    H, S, D = 3, 20_000_000, 128
    cache = [raw(1, H, S, D, dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8) for _ in range(2)]
    k, v = (torch.randn(5, H, D).bfloat16() for _ in range(2))
    at = torch.tensor([0, 1, 16_777_217, S - 2, S - 1])
    slots = at.to(torch.int32).cuda()
    if fmt == "bf16":
        gq.attn_cache_append(k.cuda(), v.cuda(), slots, *cache)
        want = [k, v]
    else:
        gq.attn_cache_append_fp8(k.cuda(), v.cuda(), slots, *cache, KS * 6, VS * 6)
        want = [(x.float() * float(torch.tensor(1.0) / torch.tensor(s * 6))).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for x, s in ((k, KS), (v, VS))]
    assert gq.get_device_status() == 0
    for c, w in zip(cache, want):
        assert torch.equal(c[0][:, at.cuda()].transpose(0, 1).cpu(), w)


@pytest.mark.parametrize("D,rows", [(128, 2 ** 25), (64, 2 ** 26)])
def test_q4_one_page_of_a_whole_request(gq, D, rows):
    """A page of more rows than 2^31 bytes of codes hold, the request's only one, read to its end: all keys zero but the
    last ones; and the same page as a contiguous cache.  n0 zero keys add exp(0) each to the sum and nothing to O."""
    page, n, Hq = rows + 384, 300, 4
    cache = [torch.zeros(2, 1, page, w, dtype=torch.uint8, device="cuda") for w in (D // 2, D // 16) * 2]
    length = page - 7
    at = page + length - n                        # in the pool's second page
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn(n, 1, D, generator=g).bfloat16() for _ in range(2))
    gq.attn_cache_append_q4(k.cuda(), v.cuda(), torch.arange(at, at + n, dtype=torch.int32, device="cuda"), *cache, KS, VS)
    K, V = (x.transpose(0, 1)[None] for x in quantised(k, v))
    q, scale, n0 = queries(1, Hq, 1, D, 5), 6.0 / math.sqrt(D), length - n
    o, lse, spread, weight = R.decode(q, K, V, [n], scale)
    full = torch.logaddexp(lse, torch.tensor(math.log(n0), dtype=torch.float64))
    part = (lse - full).exp()[..., None]
    # spread is sum_j (p_j + 2^-15) |v_j|: its p shrink by `part`; as it is, it bounds that
    assert float(part.min()) > 0.02 and float(part.max()) < 0.98      # both kinds of keys count
    ref = (o * part, full, spread, weight)
    lens = torch.tensor([length], dtype=torch.int32).cuda()
    close(*gq.attn_decode_paged_q4_fwd(q.cuda(), *cache, KS, VS, torch.tensor([[1]], dtype=torch.int32).cuda(), lens, scale=scale), ref)
    close(*gq.attn_decode_q4_fwd(q.cuda(), *(c[1:] for c in cache), KS, VS, lens, scale=scale), ref)
    assert gq.get_device_status() == 0
