"""attn_rope, attn_rope_bwd and attn_rope_table on the GPU against 64 bits.

Tolerance of a rotated row: its f32 value is a difference or sum of two rounded
products (three roundings of at most 2^-24 of |a| + |b| each), then one rounding
to bf16 of at most 2^-8 of the value.  Table entries: 2^-22 of the magnitude."""
import numpy as np
import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


def table(n, r, seed=1):
    """Any cos/sin of any magnitude: the rotation need not be orthogonal (scaled tables are not)."""
    g = torch.Generator().manual_seed(seed)
    a = torch.rand(n, r // 2, generator=g, dtype=torch.float64) * 100
    return (torch.cat([a.cos(), a.sin()], 1) * 1.25).float()


def close(y, ref, x, r):
    """|y - ref| <= 2^-8 |ref| + 3 2^-24 (sum over the pair) -- the pair bounded by the row's two largest entries."""
    y, ref = y.double().cpu(), ref.double()
    big = 1.25 * 2 * x.double().abs().amax(-1, keepdim=True)
    assert torch.isfinite(y).all()
    assert ((y - ref).abs() <= 2.0 ** -8 * ref.abs() + 3 * 2.0 ** -24 * big).all()
    if r < x.shape[-1]:
        assert torch.equal(y[..., r:], x.double()[..., r:])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,r", [(1, 1, 16, 16), (3, 1, 64, 16), (14, 2, 64, 64), (32, 8, 128, 96), (5, 5, 80, 48),
                                        (9, 1, 512, 512), (8, 8, 128, 32)])
@pytest.mark.parametrize("n", [1, 7, 1200])
def test_rope_packed(gq, Hq, Hkv, D, r, n, inter):
    g = torch.Generator().manual_seed(n + D)
    q, k = (torch.randn(n, h, D, generator=g).bfloat16() for h in (Hq, Hkv))
    pos = torch.randint(0, 300, (n,), generator=g, dtype=torch.int32)
    tab = table(300, r)
    for fn, sign in ((gq.attn_rope, 1.0), (gq.attn_rope_bwd, -1.0)):
        qo, ko = fn(q.cuda(), k.cuda(), pos.cuda(), tab.cuda(), inter)
        assert gq.get_device_status() == 0
        for x, y in ((q, qo), (k, ko)):
            close(y, R.rope(x, pos[:, None], tab, inter, sign), x, r)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_dense_views_and_in_place(gq, inter):
    """[B,H,T,D] views of a fused projection's output, positions per token and shared, q alone, and in place."""
    B, T, Hq, Hkv, D, r = 3, 65, 6, 2, 64, 32
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, T, Hq + 2 * Hkv, D, generator=g).bfloat16()
    xd = x.cuda()
    view = lambda t, a, b: t[:, :, a:b].transpose(1, 2)  # noqa: E731
    tab = table(200, r)
    pos = torch.randint(0, 200, (B, T), generator=g, dtype=torch.int32)
    refs = [R.rope(view(x, a, b), pos[:, None], tab, inter) for a, b in ((0, Hq), (Hq, Hq + Hkv))]
    q, k = view(xd, 0, Hq), view(xd, Hq, Hq + Hkv)
    qo, ko = gq.attn_rope(q, k, pos.cuda(), tab.cuda(), inter)
    close(qo, refs[0], view(x, 0, Hq), r)
    close(ko, refs[1], view(x, Hq, Hq + Hkv), r)
    only, none = gq.attn_rope(q, None, pos.cuda(), tab.cuda(), inter)
    assert none is None and torch.equal(only, qo)
    shared = gq.attn_rope(q, k, pos[0].contiguous().cuda(), tab.cuda(), inter)[0]
    close(shared, R.rope(view(x, 0, Hq), pos[0], tab, inter), view(x, 0, Hq), r)
    v0 = xd[:, :, Hq + Hkv:].clone()
    a, b = gq.attn_rope(q, k, pos.cuda(), tab.cuda(), inter, q, k)
    assert a is q and b is k and torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(xd[:, :, Hq + Hkv:], v0)          # the values beside them are untouched
    assert gq.get_device_status() == 0


def test_rope_gradient_is_the_formulas_and_the_differences(gq):
    """<g, R x> differentiated: attn_rope_bwd(g) against autograd in 64 bits and central differences (the map is linear,
    so a difference over any step is the derivative but for 64-bit rounding)."""
    n, H, D, r = 9, 2, 64, 48
    g = torch.Generator().manual_seed(8)
    x = torch.randn(n, H, D, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(n, H, D, generator=g).bfloat16()
    pos = torch.randint(0, 50, (n,), generator=g, dtype=torch.int32)
    tab = table(50, r)
    for inter in (False, True):
        f = lambda z: (R.rope(z, pos[:, None], tab, inter) * dy.double()).sum()  # noqa: E731
        grad, = torch.autograd.grad(f(x), x)
        dx, _ = gq.attn_rope_bwd(dy.cuda(), None, pos.cuda(), tab.cuda(), inter)
        close(dx, grad, dy, r)
        for i in range(0, D, 7):
            e = torch.zeros_like(x)
            e[4, 1, i] = 0.5
            with torch.no_grad():
                diff = float(f(x + e) - f(x - e))
            assert abs(diff - float(grad[4, 1, i])) < 1e-10


def test_rope_same_as_the_prefill_forward_takes(gq):
    """attn_fwd on rotated q and k against attn_fwd_rope on the unrotated: the same attention but for the rotated
    values' rounding (bf16 here, f16 there: 2^-8 of each score's terms; scores of N(0,1) features scaled to unit
    variance move by about 2^-8, outputs by less than 3 2^-8 of their norm)."""
    from causal_gqa_attention_fwd_gb300 import workloads as W
    x = W.dense_inputs(2, 8, 2, 300, 128, seed=5)
    q, k, v = (x[m].cuda() for m in ("q", "k", "v"))
    tab = gq.attn_rope_table(300, 128)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    qr, kr = gq.attn_rope(q, k, pos, tab)
    a, _ = gq.attn_fwd(qr, kr, v)
    b, _ = gq.attn_fwd_rope(q, k, v, tab)
    assert gq.get_device_status() == 0
    assert float((a.float() - b.float()).norm() / b.float().norm()) < 3 * 2.0 ** -8


@pytest.mark.parametrize("B,Hq,Hkv,T,D", [(1, 2, 1, 40, 64), (1, 8, 2, 300, 128), (2, 4, 4, 129, 128), (1, 14, 2, 200, 64)])
def test_rope_bwd_right_after_attn_bwd(gq, B, Hq, Hkv, T, D):
    """The backward of rotate-then-attend without a rest between, on small shapes, where the dK/dV kernel is the last to
    end: the gradients of each call alone, eager (the outputs take the memory of the workspace that was freed) and
    captured, and a forward behind it."""
    from causal_gqa_attention_fwd_gb300 import workloads as W
    x = W.dense_inputs(B, Hq, Hkv, T, D, seed=6)
    q, k, v, do = (x[m].cuda() for m in ("q", "k", "v", "do"))
    tab, pos = gq.attn_rope_table(T, D), torch.arange(T, dtype=torch.int32, device="cuda")

    def both(rest):
        qr, kr = gq.attn_rope(q, k, pos, tab)
        rest()
        o, lse = gq.attn_fwd(qr, kr, v)
        rest()
        dqr, dkr, dv = gq.attn_bwd(qr, kr, v, o, lse, do)
        rest()
        dq, dk = gq.attn_rope_bwd(dqr, dkr, pos, tab)
        rest()
        return dqr, dkr, dq, dk, dv, *gq.attn_fwd(q, k, v)

    want = both(torch.cuda.synchronize)
    for n, g in ((0, 2), (1, 3)):
        close(want[g], R.rope(want[n].cpu(), pos.cpu(), tab.cpu(), False, -1.0), want[n].cpu(), D)
    for _ in range(30):
        assert all(torch.equal(a, b) for a, b in zip(both(lambda: None), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(lambda: None)
    for _ in range(100):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert gq.get_device_status() == 0


def test_rope_positions_outside_the_table(gq):
    q = torch.randn(4, 2, 64).bfloat16()
    pos = torch.tensor([0, 10, -1, 9], dtype=torch.int32)
    tab = table(10, 32)
    qo, _ = gq.attn_rope(q.cuda(), None, pos.cuda(), tab.cuda())
    assert gq.get_device_status() == 5
    assert (qo[1:3] == 0).all()
    close(qo[[0, 3]], R.rope(q[[0, 3]], pos[[0, 3]][:, None], tab, False), q[[0, 3]], 32)


def test_rope_other_stream(gq):
    q = torch.randn(64, 4, 128, device="cuda").bfloat16()
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    tab = gq.attn_rope_table(64, 128)
    want, _ = gq.attn_rope(q, None, pos, tab)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = torch.empty_like(q)
    gq.attn_rope(q, None, pos, tab, q_out=got, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kw", [
    dict(),
    dict(base=500000.0, factor=8.0),
    dict(base=10000.0, factor=16.0, original_positions=4096, low_turns=1.0, high_turns=32.0, mscale=1.2772588722),
    dict(base=500000.0, factor=8.0, original_positions=8192, low_turns=1.0, high_turns=4.0),
    dict(base=10000.0, factor=0.25),
])
@pytest.mark.parametrize("n,r", [(1, 16), (1000, 80), (70001, 128)])
def test_rope_table(gq, n, r, kw):
    """Against 64 bits, to 2^-22 of the magnitude (the 64-bit angles themselves are off by 2^-53 of up to n turns)."""
    got = gq.attn_rope_table(n, r, **kw).double().cpu()
    theta = kw.get("base", 10000.0) ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)
    f, orig = kw.get("factor", 1.0), kw.get("original_positions", 0)
    if orig:
        lo, hi = kw["low_turns"], kw["high_turns"]
        g = ((orig * theta / (2 * np.pi) - lo) / (hi - lo)).clamp(0, 1)
        theta = theta * g + theta / f * (1 - g)
    else:
        theta = theta / f
    ang = torch.arange(n, dtype=torch.float64)[:, None] * theta
    m = kw.get("mscale", 1.0)
    ref = torch.cat([ang.cos(), ang.sin()], 1) * m
    assert float((got - ref).abs().max()) <= 2.0 ** -22 * m


def test_rope_table_is_the_workloads_table(gq):
    from causal_gqa_attention_fwd_gb300 import workloads as W
    a, b = gq.attn_rope_table(5000, 64).cpu(), W.rope_cos_sin_table(5000, 64)
    assert float((a - b).abs().max()) <= 2.0 ** -22 + 2.0 ** -24
