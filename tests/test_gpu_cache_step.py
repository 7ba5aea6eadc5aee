"""The cache operators together, as a serving loop runs them: requests of different lengths are admitted (plan, rotate,
append, whole-prompt attention), then decode step by step (plan, append with rotation, attention with rotated queries),
for 4-bit, E4M3 and bf16 caches; checked against 64 bits on what was appended.

Tolerances of the 4-bit steps as in test_gpu_decode_q4; the values attended to are those the reference quantises from the
same bf16 inputs (equal bits, see test_gpu_cache_append), so no quantisation error enters.  E4M3 and bf16 caches go
through attn_decode_paged_*: their bounds are those of their own tests (relative norm 5e-3)."""
import math

import pytest
import torch

import cache_ref as R
from test_gpu_decode_q4 import close

pytestmark = pytest.mark.gpu
KS, VS = 0.0027, 0.0024
SHAPE = dict(Hq=8, Hkv=2, D=128, page=16, mp=12)


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


class Loop:
    """What the program keeps: pages, block table, lengths, the free list's cursor."""

    def __init__(self, gq, fmt, B, seed):
        self.gq, self.fmt, self.B = gq, fmt, B
        s = SHAPE
        n = B * s["mp"]
        g = torch.Generator().manual_seed(seed)
        self.free = torch.randperm(n, generator=g).to(torch.int32).cuda()
        self.table = torch.full((B, s["mp"]), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.cursor = torch.zeros(1, dtype=torch.int32, device="cuda")
        z = lambda w, t=torch.uint8: torch.zeros(n, s["Hkv"], s["page"], w, dtype=t, device="cuda")  # noqa: E731
        D = s["D"]
        self.cache = {"q4": lambda: [z(D // 2), z(D // 16), z(D // 2), z(D // 16)], "fp8": lambda: [z(D), z(D)],
                      "bf16": lambda: [z(D, torch.bfloat16), z(D, torch.bfloat16)]}[fmt]()
        self.tab = gq.attn_rope_table(s["page"] * s["mp"], D)
        self.scales = () if fmt == "bf16" else (KS, VS)
        self.append = {"q4": gq.attn_cache_append_q4, "fp8": gq.attn_cache_append_fp8, "bf16": gq.attn_cache_append}[fmt]
        self.attend = {"q4": gq.attn_decode_paged_q4_fwd, "fp8": gq.attn_decode_paged_fp8_fwd,
                       "bf16": gq.attn_decode_paged_fwd}[fmt]

    def plan(self, new, total):
        slots, pos, cu, self.lens, self.cursor = self.gq.attn_cache_plan(self.lens, new, self.table, SHAPE["page"], self.free,
                                                                         self.cursor, total)
        return slots, pos, cu


def rows(loop, store, b):
    """Request b's keys and values as the reference has them, in float64 [Hkv, n, D]."""
    k, v = (torch.stack(x[b]).transpose(0, 1) for x in store)
    if loop.fmt == "bf16":
        return k.bfloat16().double(), v.bfloat16().double()
    if loop.fmt == "fp8":
        q = lambda x, s: (x * float(torch.tensor(1.0) / torch.tensor(s))).clamp(-448, 448).to(torch.float8_e4m3fn).double() * \
            float(torch.tensor(s, dtype=torch.float32))  # noqa: E731
        return q(k, KS), q(v, VS)
    return tuple(R.values(*R.quantise(x, s), s) for x, s in ((k, KS), (v, VS)))


@pytest.mark.parametrize("fmt", ["q4", "fp8", "bf16"])
def test_prompts_then_steps(gq, fmt):
    s = SHAPE
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    prompts = torch.tensor([17, 1, 64, 33], dtype=torch.int32)
    B, total, pad = len(prompts), int(prompts.sum()), 9
    loop = Loop(gq, fmt, B, 3)
    g = torch.Generator().manual_seed(4)
    scale = 1 / math.sqrt(D)
    store = [[[] for _ in range(B)] for _ in range(2)]      # rotated k and v of each request, float32 [Hkv, D] a position

    x = torch.randn(total + pad, Hq + 2 * Hkv, D, generator=g).bfloat16()       # one projection's output, padded tokens last
    xd = x.cuda()
    q, k, v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    slots, pos, cu = loop.plan(prompts.cuda(), total + pad)
    loop.append(k, v, slots, *loop.cache, *loop.scales, positions=pos, rope_cos_sin=loop.tab)
    qr, kr = gq.attn_rope(q[:total], k[:total], pos[:total].contiguous(), loop.tab)
    o, _ = gq.attn_varlen_fwd(qr, kr, v[:total].contiguous(), cu, int(prompts.max()), scale=scale)
    assert gq.get_device_status() == 0
    tab = loop.tab.cpu()
    kf = R.rope(x[:, Hq:Hq + Hkv], pos.cpu()[:, None], tab, False, dtype=torch.float32)
    n = 0
    for b in range(B):
        for i in range(int(prompts[b])):
            store[0][b].append(kf[n])
            store[1][b].append(x[n, Hq + Hkv:].float())
            n += 1
    # the last prompt token's attention, from the reference's unquantised rows
    for b in range(B):
        last = int(cu[b + 1]) - 1
        K, V = (torch.stack(z[b]).transpose(0, 1).double() for z in store)
        xq = R.rope(x[last, :Hq][None], torch.tensor([int(prompts[b]) - 1]), tab, False).reshape(Hkv, Hq // Hkv, D)
        p = torch.softmax(torch.einsum("hgd,hkd->hgk", xq, K) * scale, -1)
        want = torch.einsum("hgk,hkd->hgd", p, V).reshape(Hq, D)
        assert float((o[last].double().cpu() - want).norm() / want.norm()) < 4 * 2.0 ** -8    # q, k, p and o rounded to bf16

    for step in range(20):
        new = torch.ones(B, dtype=torch.int32)
        if step == 5:
            new[1] = 0                                       # a request that pauses
        qs, ks, vs = (torch.randn(B, h, 1, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
        slots, pos, _ = loop.plan(new.cuda(), B)
        live = [b for b in range(B) if new[b]]
        # packed order: the pausing request has no token
        kd, vd = ks[live, :, 0].cuda(), vs[live, :, 0].cuda()
        loop.append(kd, vd, slots[:len(live)].contiguous(), *loop.cache, *loop.scales,
                    positions=pos[:len(live)].contiguous(), rope_cos_sin=loop.tab)
        o, lse = loop.attend(qs.cuda(), *loop.cache, *loop.scales, loop.table, loop.lens, scale=scale, rope_cos_sin=loop.tab)
        assert gq.get_device_status() == 0
        for b in live:
            at = len(store[0][b])
            store[0][b].append(R.rope(ks[b, :, 0], torch.tensor(at), tab, False, dtype=torch.float32))
            store[1][b].append(vs[b, :, 0].float())
        assert loop.lens.tolist() == [len(z) for z in store[0]]
        if step in (0, 5, 19):
            for b in range(B):
                K, V = rows(loop, store, b)
                ref = R.decode(qs[b:b + 1], K[None], V[None], torch.tensor([K.shape[1]]), scale, tab)
                if fmt == "q4":
                    close(o[b:b + 1], lse[b:b + 1], ref)
                else:
                    assert float((o[b].double().cpu() - ref[0][0]).norm() / ref[0].norm()) < 5e-3
                    assert float((lse[b].double().cpu() - ref[1][0]).abs().max()) < 1e-3


def test_cached_prefix_read_back_for_a_later_chunk(gq):
    """The second chunk of a prompt attends to the first through the 4-bit cache read back as bf16: the gathered rows are
    the cache's values, and attention over [gathered, new] rows is that of the reference on them."""
    Hq, Hkv, D, n0, n1 = 4, 2, 64, 45, 19
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(n0 + n1, Hkv, D, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(n0 + n1, Hq, D, generator=g).bfloat16()
    z = lambda w: torch.zeros(5, Hkv, 16, w, dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = [z(D // 2), z(D // 16), z(D // 2), z(D // 16)]
    table = torch.full((1, 5), -1, dtype=torch.int32, device="cuda")
    free = torch.tensor([3, 0, 4, 1, 2], dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    s0, _, _, lens, cur = gq.attn_cache_plan(lens, torch.full_like(lens, n0), table, 16, free, None, n0)
    gq.attn_cache_append_q4(k[:n0].cuda(), v[:n0].cuda(), s0, *cache, KS, VS)
    kc, vc = gq.attn_cache_gather_q4(s0, *cache, KS, VS)
    K = torch.cat([kc, k[n0:].cuda()]).transpose(0, 1)[None].contiguous()
    V = torch.cat([vc, v[n0:].cuda()]).transpose(0, 1)[None].contiguous()
    Q = q.cuda().transpose(0, 1)[None].contiguous()
    o, lse = gq.attn_fwd(Q, K, V, scale=0.125)
    assert gq.get_device_status() == 0
    ref = R.decode(Q.cpu()[:, :, n0:], K.double().cpu(), V.double().cpu(), torch.tensor([n0 + n1]), 0.125)
    assert float((o[:, :, n0:].double().cpu() - ref[0]).norm() / ref[0].norm()) < 5e-3
    assert float((lse[:, :, n0:].double().cpu() - ref[1]).abs().max()) < 1e-3


def test_a_captured_step_replayed(gq):
    """One decode step (plan, append, attention) captured once and replayed: the lengths move on inside the graph."""
    s = SHAPE
    Hq, Hkv, D, B = s["Hq"], s["Hkv"], s["D"], 3
    loop = Loop(gq, "q4", B, 8)
    g = torch.Generator().manual_seed(9)
    loop.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.tensor([1, 1, 0], dtype=torch.int32, device="cuda")     # the last batch slot has no request
    q = torch.zeros(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(B, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        slots, pos, _, lens, cursor = gq.attn_cache_plan(loop.lens, new, loop.table, s["page"], loop.free, loop.cursor, B)
        gq.attn_cache_append_q4(k, v, slots, *loop.cache, KS, VS, positions=pos, rope_cos_sin=loop.tab)
        loop.lens.copy_(lens)
        loop.cursor.copy_(cursor)
        return gq.attn_decode_paged_q4_fwd(q, *loop.cache, KS, VS, loop.table, loop.lens, scale=0.1, rope_cos_sin=loop.tab)

    step()
    torch.cuda.synchronize()
    loop.lens.zero_()
    loop.cursor.zero_()
    loop.table.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    tab, store = loop.tab.cpu(), [[[] for _ in range(B)] for _ in range(2)]
    for i in range(40):
        qs, ks, vs = (torch.randn(B, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
        q.copy_(qs[:, :, None])
        k.copy_(ks)
        v.copy_(vs)
        graph.replay()
        for b in (0, 1):
            store[0][b].append(R.rope(ks[b], torch.tensor(i), tab, False, dtype=torch.float32))
            store[1][b].append(vs[b].float())
        if i in (0, 17, 39):
            assert gq.get_device_status() == 0
            assert loop.lens.tolist() == [i + 1, i + 1, 0]
            for b in (0, 1):
                K, V = rows(loop, store, b)
                close(o[b:b + 1], lse[b:b + 1], R.decode(qs[b:b + 1, :, None], K[None], V[None], torch.tensor([i + 1]), 0.1, tab))
            assert (o[2] == 0).all() and (lse[2] == -math.inf).all()


@pytest.mark.parametrize("fmt", ["q4", "fp8", "bf16"])
def test_a_captured_step_with_idle_rows_anywhere(gq, fmt):
    """k and v one row a request, idle rows among them: the plan packs its tokens, so a row's slot and position are entry
    cu_seqlens[b], if the request has a token.  The pattern changes between replays of one captured step."""
    s = SHAPE
    Hq, Hkv, D, B = s["Hq"], s["Hkv"], s["D"], 5
    loop = Loop(gq, fmt, B, 18)
    g = torch.Generator().manual_seed(19)
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(B, Hkv, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        slots, pos, cu, lens, cursor = gq.attn_cache_plan(loop.lens, new, loop.table, s["page"], loop.free, loop.cursor, B)
        first = cu[:-1].clamp(max=B - 1).long()
        slots = torch.where(cu[1:] > cu[:-1], slots[first], -1)
        loop.append(k, v, slots, *loop.cache, *loop.scales, positions=pos[first], rope_cos_sin=loop.tab)
        loop.lens.copy_(lens)
        loop.cursor.copy_(cursor)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    tab, store = loop.tab.cpu(), [[[] for _ in range(B)] for _ in range(2)]
    patterns = [[1, 1, 1, 1, 1], [0, 1, 1, 0, 1], [1, 0, 0, 1, 0], [0, 0, 0, 0, 0], [1, 0, 1, 0, 1], [0, 1, 0, 1, 1]]
    for i in range(36):
        on = patterns[i % 6]
        ks, vs = (torch.randn(B, Hkv, D, generator=g).bfloat16() for _ in range(2))
        k.copy_(ks[:, :, None])
        v.copy_(vs[:, :, None])
        new.copy_(torch.tensor(on, dtype=torch.int32))
        graph.replay()
        for b in range(B):
            if on[b]:
                store[0][b].append(R.rope(ks[b], torch.tensor(len(store[0][b])), tab, False, dtype=torch.float32))
                store[1][b].append(vs[b].float())
    assert gq.get_device_status() == 0
    n = [len(x) for x in store[0]]
    assert loop.lens.tolist() == n and len(set(n)) > 1
    qs = torch.randn(B, Hq, 1, D, generator=g).bfloat16()
    o, lse = loop.attend(qs.cuda(), *loop.cache, *loop.scales, loop.table, loop.lens, scale=0.1, rope_cos_sin=loop.tab)
    assert gq.get_device_status() == 0
    for b in range(B):
        K, V = rows(loop, store, b)
        ref = R.decode(qs[b:b + 1], K[None], V[None], torch.tensor([n[b]]), 0.1, tab)
        if fmt == "q4":
            close(o[b:b + 1], lse[b:b + 1], ref)
        else:
            assert float((o[b:b + 1].double().cpu() - ref[0]).norm() / ref[0].norm()) <= 5e-3
            assert float((lse[b:b + 1].double().cpu() - ref[1]).abs().max()) <= 1e-3


def test_on_another_stream_with_a_workspace_of_its_own(gq):
    """The same decode call on a side stream, workspace allocated by the call: the memory is that stream's."""
    B, Hq, Hkv, S, D = 2, 8, 2, 3000, 128
    from test_gpu_decode_q4 import cache_of, queries
    cache = [c.cuda() for c in cache_of(B, Hkv, S, D, 1)]
    q, lens = queries(B, Hq, 1, D, 2).cuda(), torch.tensor([S, 1234], dtype=torch.int32, device="cuda")
    want = gq.attn_decode_q4_fwd(q, *cache, KS, VS, lens, scale=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for i in range(8):
        for st in (side, side.cuda_stream):
            outs.append(gq.attn_decode_q4_fwd(q, *cache, KS, VS, lens, scale=0.1, stream=st))
        torch.empty(64 << 20, dtype=torch.uint8, device="cuda").fill_(255)      # the current stream's allocations meanwhile
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
