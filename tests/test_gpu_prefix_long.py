"""Shared-prefix attention over rows of nearly 2^31 positions: lengths and page numbers at the end of 32 bits."""
import math

import pytest
import torch

from test_gpu_decode_prefix import ran

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


@pytest.mark.parametrize("Hq,what", [(1, "own"), (1, "prefix"), (32, "prefix")], ids=["own", "stream", "tiles"])
def test_rows_that_end_within_a_page_of_2_31_positions(gq, Hq, what):
    """A row of 130055 pages of 16512 positions, less than a page from 2^31, and all of them the same page of the pool: its
    attention is that over the one page, with a log-sum-exp larger by ln 130055.  In the stream a warp of 152 * 12 takes 2^31
    / 1824 keys, in tensor-core steps and additions of 16 keys: 73585 < 2^17 of them, off by 2^-23 of the sum each, 2^-6.  With
    large tiles a tile of 302 takes 2^31 / 302: 55556 < 2^17 additions of 128 keys a thread, but 444443 < 2^19 tensor-core
    steps, 2^-4, for O.  The weights' rounding adds 2^-8."""
    page, times = 16512, 130055
    n = page * times
    assert n < 2 ** 31 - 512 < n + page
    g = torch.Generator().manual_seed(7)
    k, v = torch.randn(2, 1, page, 64, generator=g).bfloat16(), (1 + torch.randn(2, 1, page, 64, generator=g)).bfloat16()
    q = torch.randn(1, Hq, 1, 64, generator=g).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    long, short = torch.zeros(1, times, dtype=torch.int32, device="cuda"), i32([[1]])
    if what == "own":      # no prefix; every own key is in page 0
        args = (short, i32([0]), long, i32([n]))
        K, V, more = k[0], v[0], 0
    else:                  # one own key, in page 1: of no weight beside the others
        args = (long, i32([n]), short, i32([1]))
        K, V, more = k[0], v[0], 1
    got, names = ran(gq, lambda: gq.attn_decode_paged_prefix_fwd(q.cuda(), k.cuda(), v.cuda(), *args))
    assert gq.get_device_status() == 0 and ("prefix" in names) == (Hq == 32)
    s = torch.einsum("hd,kd->hk", q[0, :, 0].double(), K[0].double()) / 8
    lse = torch.logsumexp(s, -1) + math.log(times)
    o = torch.softmax(s, -1) @ V[0].double()
    size = torch.softmax(s, -1) @ V[0].double().abs()
    assert float((got[1][0, :, 0].cpu().double() - lse).abs().max()) <= 2 * 2.0 ** -6 + more * 2.0 ** -20
    tol = (2.0 ** -4 if Hq == 32 else 2.0 ** -6) + 2 * 2.0 ** -6 + 2 * 2.0 ** -8 + more * 2.0 ** -20
    assert bool(((got[0][0, :, 0].cpu().double() - o).abs() <= tol * size).all())
