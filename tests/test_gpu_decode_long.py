"""Cached attention over rows of nearly 2^31 positions: lengths and page numbers at the end of 32 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_row_that_ends_within_a_page_of_2_31_positions(gq, fmt):
    """A row of 130055 pages of 16512 positions, all of them the same page of the pool: its attention is that over the one
    page, with a log-sum-exp larger by ln 130055.  A CTA of 152 takes 2^31 / 152 keys.  The weights' sum of a row is one
    addition a thread for each block of 128: 110376 < 2^17 of them, off by 2^-23 each, 2^-6.  O is accumulated by tensor-core
    steps of 16 keys, which may cut off what an f32 does not hold: 883012 < 2^20 of them, 2^-3.  The weights' rounding adds 2^-8
    (bf16) or less."""
    page, times = 16512, 130055
    n = page * times
    assert n < 2 ** 31 - 512 < n + page
    g = torch.Generator().manual_seed(8)
    k, v = torch.randn(1, 1, page, 64, generator=g), 1 + torch.randn(1, 1, page, 64, generator=g)
    q = torch.randn(1, 2, 1, 64, generator=g).bfloat16()
    table, lens = torch.zeros(1, times, dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32).cuda()
    if fmt == "bf16":
        k, v = k.bfloat16(), v.bfloat16()
        o, lse = gq.attn_decode_paged_fwd(q.cuda(), k.cuda(), v.cuda(), table, lens)
    else:
        k, v = ((x / s).clamp(-448, 448).to(torch.float8_e4m3fn) for x, s in ((k, 0.01), (v, 0.02)))
        o, lse = gq.attn_decode_paged_fp8_fwd(q.cuda(), k.view(torch.uint8).cuda(), v.view(torch.uint8).cuda(), 0.01, 0.02, table, lens)
        k, v = k.float() * 0.01, v.float() * 0.02
    assert gq.get_device_status() == 0
    s = q[0, :, 0].double() @ k[0, 0].double().t() / 8
    p, v = torch.softmax(s, -1), v[0, 0].double()
    assert float((lse[0, :, 0].cpu().double() - torch.logsumexp(s, -1) - math.log(times)).abs().max()) <= 2 * 2.0 ** -6
    assert bool(((o[0, :, 0].cpu().double() - p @ v).abs() <= (2.0 ** -3 + 2 * 2.0 ** -6 + 2 * 2.0 ** -8) * (p @ v.abs())).all())
