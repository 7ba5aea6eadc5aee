"""Shared prefix, attention weights and eviction as a serving loop runs them: plan, append, attend, weigh, evict, and on."""
import math

import pytest
import torch

import pressure_ref as R
from test_gpu_decode_prefix import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


class Loop:
    """Requests that share a prompt in the pool's first pages, with 16-position pages of their own."""

    def __init__(self, gq, B, Hq, Hkv, D, m, budget, seed):
        self.gq, self.B, self.Hq, self.Hkv, self.D, self.budget, self.page = gq, B, Hq, Hkv, D, budget, 16
        self.g = torch.Generator().manual_seed(seed)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        mp = -(-m // self.page)
        self.N = mp + B * 16 + 1
        z = lambda *s, dt=torch.bfloat16: torch.zeros(self.N, Hkv, self.page, *s, dtype=dt, device="cuda")  # noqa: E731
        self.k, self.v, self.w = z(D), z(D), z(dt=torch.float32)
        self.pt, self.pl = i32([list(range(mp))]), i32([m])
        self.pk, self.pv = (torch.randn(Hkv, m, D, generator=self.g).bfloat16() for _ in range(2))
        slots = torch.arange(m, dtype=torch.int32, device="cuda")
        gq.attn_cache_append(self.pk.transpose(0, 1).cuda(), self.pv.transpose(0, 1).cuda(), slots, self.k, self.v)
        self.bt = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
        self.free, self.cursor = torch.arange(mp, self.N, dtype=torch.int32, device="cuda"), i32([0])
        self.lens = i32([0] * B)
        # what the rows should hold, on the host
        self.own = [[torch.zeros(Hkv, 0, D) for _ in range(2)] for _ in range(B)]
        self.sums = [torch.zeros(Hkv, 0, dtype=torch.float64) for _ in range(B)]

    def step(self, T):
        """T new tokens in every request; their outputs."""
        B, gq = self.B, self.gq
        q, k, v = (torch.randn(B, h, T, self.D, generator=self.g).bfloat16() for h in (self.Hq, self.Hkv, self.Hkv))
        new = torch.full((B,), T, dtype=torch.int32, device="cuda")
        slots, _, _, self.lens, self.cursor = gq.attn_cache_plan(self.lens, new, self.bt, self.page, self.free, self.cursor, B * T)
        gq.attn_cache_append(k.cuda(), v.cuda(), slots, self.k, self.v)
        o, lse = gq.attn_decode_paged_prefix_fwd(q.cuda(), self.k, self.v, self.pt, self.pl, self.bt, self.lens)
        gq.attn_cache_weights(q.cuda(), self.k, lse, self.lens, self.w, block_table=self.bt)
        for b in range(B):
            self.own[b] = [torch.cat([c, x[b].float()], 1) for c, x in zip(self.own[b], (k, v))]
            self.sums[b] = torch.cat([self.sums[b], torch.zeros(self.Hkv, T, dtype=torch.float64)], 1)
        return q, o, lse

    def verify(self, q, o, lse):
        n = [c[0].shape[1] for c in self.own]
        assert self.lens.tolist() == n
        scale = 1 / math.sqrt(self.D)
        check((o, lse), R.prefix(q, [(self.pk.double(), self.pv.double())], [(c[0].double(), c[1].double()) for c in self.own], n,
                                 scale), self.D)
        for b in range(self.B):
            add, _ = R.weights(q[b], self.own[b][0].double(), lse[b].cpu(), n[b], scale)
            self.sums[b] += add
            got = R.rows_of(self.w.cpu(), self.bt.cpu(), b, n[b])
            assert torch.allclose(got.double(), self.sums[b], rtol=1e-4, atol=1e-9)

    def evict(self, recent, first):
        before = [R.rows_of(self.w.cpu(), self.bt.cpu(), b, int(n)).clone() for b, n in enumerate(self.lens.tolist())]
        n = self.lens.tolist()
        kept, self.lens = self.gq.attn_cache_evict(self.w, (self.k, self.v), self.lens, self.budget, recent=recent, first=first,
                                                   block_table=self.bt)
        for b in range(self.B):
            for h in range(self.Hkv):
                want = R.evict(before[b][h], n[b], self.budget, recent, first)
                assert kept[b, h, :len(want)].tolist() == want
            at = kept[b, :, :min(n[b], self.budget)].cpu().long()
            self.own[b] = [torch.gather(c, 1, at[..., None].expand(-1, -1, self.D)) for c in self.own[b]]
            self.sums[b] = torch.gather(self.sums[b], 1, at)
            for c, pool in zip(self.own[b], (self.k, self.v)):
                assert torch.equal(R.rows_of(pool.cpu(), self.bt.cpu(), b, at.shape[1]).float(), c)
        # the pages behind the budget are free again
        self.bt[:, -(-self.budget // self.page):] = -1


@pytest.mark.parametrize("B,Hq,Hkv,D,m,budget", [(3, 8, 2, 64, 150, 20), (5, 4, 4, 128, 16, 33)])
def test_serving_under_a_budget(gq, B, Hq, Hkv, D, m, budget):
    lp = Loop(gq, B, Hq, Hkv, D, m, budget, seed=1)
    for turn, T in enumerate((budget + 9, 1, 1, 3, 30, 1)):
        lp.verify(*lp.step(T))
        if turn in (0, 3, 4):
            lp.evict(recent=6, first=2)
    assert gq.get_device_status() == 0
    # the prompt is as it was
    assert torch.equal(R.rows_of(lp.k.cpu(), lp.pt.cpu(), 0, m), lp.pk)


def test_a_captured_loop(gq):
    """Attend, weigh and evict as one graph, replayed while the lengths stay at the budget plus the new token."""
    B, Hq, Hkv, D, S, budget = 4, 8, 2, 64, 96, 64
    g = torch.Generator().manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    kp, vp, pl = rn(1, Hkv, 200, D), rn(1, Hkv, 200, D), torch.tensor([200], dtype=torch.int32, device="cuda")
    q, k, v = rn(B, Hq, 1, D), rn(B, Hkv, 1, D), rn(B, Hkv, 1, D)
    lens = torch.full((B,), budget + 1, dtype=torch.int32, device="cuda")
    slots = torch.arange(B, dtype=torch.int32, device="cuda") * S + budget

    def step(kc, vc, w):
        gq.attn_cache_append(k, v, slots, kc, vc)
        o, lse = gq.attn_decode_prefix_fwd(q, kp, vp, pl, kc, vc, lens)
        gq.attn_cache_weights(q, kc, lse, lens, w)
        return o, lse, *gq.attn_cache_evict(w, (kc, vc), lens, budget, recent=8, first=4)

    start = [rn(B, Hkv, S, D), rn(B, Hkv, S, D), torch.rand(B, Hkv, S, generator=g).cuda()]
    eager, fixed = [x.clone() for x in start], [x.clone() for x in start]
    step(*[x.clone() for x in start])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*fixed)
    for i in range(5):
        for x in (q, k, v):
            x.copy_(rn(*x.shape))
        want = step(*eager)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*out, *fixed), (*want, *eager)):
            assert torch.equal(a, b), i
    assert gq.get_device_status() == 0


def test_two_streams_at_once(gq):
    """Calls on two streams, each with its own workspace, give what they give one after another."""
    from test_gpu_decode_prefix import make
    jobs = [make(8, 1, 8, 2, 1, 128, p, [1500], [1 + 30 * i for i in range(8)], seed=3 + p) for p in (0, 16)]
    want = [getattr(gq, f)(*a) for f, a, _ in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        got = [getattr(gq, f)(*a, stream=s) for (f, a, _), s in zip(jobs, streams)]
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("page", [0, 16])
def test_a_step_without_requests(gq, page):
    """An empty batch, over a pool of pages or contiguous: every call returns its empty outputs and touches nothing."""
    Hkv, D = 2, 64
    n, per = (9, page) if page else (0, 32)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    q, lse, lens = torch.zeros(0, 4, 1, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, 4, 1, device="cuda"), i32(0)
    bt = i32(0, 4) if page else None
    k, w = torch.randn(n, Hkv, per, D, device="cuda").bfloat16(), torch.rand(n, Hkv, per, device="cuda")
    k8, k4, sf = (torch.zeros(n, Hkv, per, x, dtype=torch.uint8, device="cuda") for x in (D, D // 2, D // 16))
    if page:
        o, out = gq.attn_decode_paged_prefix_fwd(q, k, k, i32(1, 2), i32(1), bt, lens)
    else:
        o, out = gq.attn_decode_prefix_fwd(q, *[torch.zeros(1, Hkv, 8, D, dtype=torch.bfloat16, device="cuda")] * 2, i32(1), k, k, lens)
    assert o.shape == q.shape and out.shape == lse.shape
    before = k.clone(), w.clone()
    assert gq.attn_cache_weights(q, k, lse, lens, w, block_table=bt) is w
    assert gq.attn_cache_weights_fp8(q, k8, 0.1, lse, lens, w, block_table=bt) is w
    assert gq.attn_cache_weights_q4(q, k4, sf, 0.1, lse, lens, w, block_table=bt) is w
    kept, lens_out = gq.attn_cache_evict(w, (k,), lens, 8, recent=2, block_table=bt)
    assert kept.shape == (0, Hkv, 8) and lens_out.shape == (0,)
    assert torch.equal(before[0], k) and torch.equal(before[1], w) and gq.get_device_status() == 0
