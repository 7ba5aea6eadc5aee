"""The loop of shared prefix, weights and eviction with rotary positions: an own key's position follows the prefix's, and a
row that was cut goes on at the positions it had reached, so the program keeps positions beside the lengths."""
import pytest
import torch

from test_gpu_cache_pressure_loop import Loop

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


def rotated(x, pos, base):
    """x [..., T, D] float64 rotated at pos [T] (pairs i, i + D/2)."""
    D = x.shape[-1]
    a = pos.double()[:, None] * base ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)
    c, s = a.cos(), a.sin()
    u, v = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([u * c - v * s, v * c + u * s], -1)


class RotaryLoop(Loop):
    BASE = 500.0

    def __init__(self, gq, B, Hq, Hkv, D, m, budget, seed):
        super().__init__(gq, B, Hq, Hkv, D, m, budget, seed)
        self.m, self.tab = m, gq.attn_rope_table(512, D, base=self.BASE)
        self.reached = torch.full((B,), m, dtype=torch.int32, device="cuda")      # each row's next position
        at = torch.arange(m, dtype=torch.int32, device="cuda")
        gq.attn_cache_append(self.pk.transpose(0, 1).cuda(), self.pv.transpose(0, 1).cuda(), at, self.k, self.v, positions=at,
                             rope_cos_sin=self.tab)
        rot = gq.attn_rope(self.pk.transpose(0, 1).contiguous().cuda(), None, at, self.tab)[0].transpose(0, 1).cpu()
        self.near(rot, self.pk, at.cpu())
        self.pk = rot

    def near(self, got, x, pos):
        """got is x rotated, in f32 (table entries within 2^-22, two products and a sum: 2^-21 of |x_i| + |x_j|) and rounded
        once to bf16 (2^-8 of the value)."""
        want = rotated(x.double(), pos, self.BASE)
        half = x.shape[-1] // 2
        size = x.double().abs() + torch.cat([x[..., half:], x[..., :half]], -1).double().abs()
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all())

    def step(self, T):
        B, gq = self.B, self.gq
        q, k, v = (torch.randn(B, h, T, self.D, generator=self.g).bfloat16() for h in (self.Hq, self.Hkv, self.Hkv))
        new = torch.full((B,), T, dtype=torch.int32, device="cuda")
        slots, _, _, self.lens, self.cursor = gq.attn_cache_plan(self.lens, new, self.bt, self.page, self.free, self.cursor, B * T)
        pos = self.reached[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")
        self.reached = self.reached + T
        qr, kr = (x.cpu() for x in gq.attn_rope(q.cuda(), k.cuda(), pos, self.tab))
        gq.attn_cache_append(k.cuda(), v.cuda(), slots, self.k, self.v, positions=pos.flatten(), rope_cos_sin=self.tab)
        o, lse = gq.attn_decode_paged_prefix_fwd(qr.cuda(), self.k, self.v, self.pt, self.pl, self.bt, self.lens)
        gq.attn_cache_weights(qr.cuda(), self.k, lse, self.lens, self.w, block_table=self.bt)
        for b in range(B):
            self.near(qr[b], q[b], pos[b].cpu())
            self.near(kr[b], k[b], pos[b].cpu())
            self.own[b] = [torch.cat([c, x[b].float()], 1) for c, x in zip(self.own[b], (kr, v))]
            self.sums[b] = torch.cat([self.sums[b], torch.zeros(self.Hkv, T, dtype=torch.float64)], 1)
        return qr, o, lse


@pytest.mark.parametrize("B,Hq,Hkv,D,m,budget", [(3, 8, 2, 64, 150, 20), (5, 4, 4, 128, 16, 33)])
def test_serving_under_a_budget_with_rotary_positions(gq, B, Hq, Hkv, D, m, budget):
    lp = RotaryLoop(gq, B, Hq, Hkv, D, m, budget, seed=4)
    for turn, T in enumerate((budget + 9, 1, 1, 3, 30, 1)):
        lp.verify(*lp.step(T))
        if turn in (0, 3, 4):
            lp.evict(recent=6, first=2)
    assert gq.get_device_status() == 0
    assert lp.reached.tolist() == [m + budget + 45] * B and max(lp.lens.tolist()) == budget + 1
