"""Refusals of the cache operators and their plain references, on the CPU."""
import math

import pytest
import torch

import cache_ref as R

A = 256      # an aligned fake device address: refused calls never reach it
NULL = None


@pytest.fixture(scope="module")
def lib():
    from causal_gqa_attention_fwd_gb300 import build
    build.build()
    import causal_gqa_attention_fwd_gb300 as g
    return g.lib()


def strides(*v):
    import ctypes
    return (ctypes.c_longlong * len(v))(*v)


def test_plan_refusals(lib):
    def f(lens=A, new=A, tab=A, free=A, cur=A, slots=A, pos=A, cu=A, lo=2 * A, co=2 * A, B=4, ps=16, mp=8, nf=9, n=5):
        return lib.attn_cache_plan(lens, new, tab, free, cur, slots, pos, cu, lo, co, B, ps, mp, nf, n, None)
    assert f(B=-1) == 2 and f(B=8193) == 2 and f(ps=0) == 2 and f(mp=-1) == 2 and f(nf=-1) == 2 and f(n=-1) == 2
    assert f(ps=1 << 20, mp=1 << 12) == 2 and f(B=8192, mp=1 << 19) == 2          # 2^31 positions, 2^32 entries
    for name in ("lens", "new", "tab", "free", "slots", "pos", "cu", "lo", "co"):
        assert f(**{name: NULL}) == 1, name
    assert f(pos=A + 2) == 4 and f(cur=A + 1) == 4
    assert f(lo=A) == 2 and f(co=A) == 2                                          # in place: several blocks read them


def test_plan_outputs_that_overlap_its_inputs(lib):
    """Every block reads the inputs while others write: an output that shares an entry with one is refused, whole or in
    part; outputs may lie side by side with them."""
    sizes = dict(lens=4, new=4, tab=32, free=9, cur=1, slots=5, pos=5, cu=5, lo=4, co=1)
    at, place = 1 << 20, {}
    for name, n in sizes.items():       # one after another in memory, no gap
        place[name] = at
        at += 4 * n

    def f(**kw):
        x = dict(place, **kw)
        return lib.attn_cache_plan(*(x[n] for n in sizes), 4, 16, 8, 9, 5, None)
    # accepted by the checks: without a GPU the call ends at the device (no device, status 7 or 8)
    import torch as t
    if not t.cuda.is_available():
        assert f() not in (0, 1, 2, 3, 4)
    for out in ("slots", "pos", "cu", "lo", "co"):
        for inp in ("lens", "new", "tab", "free", "cur"):
            first, last = place[inp], place[inp] + 4 * (sizes[inp] - 1)
            assert f(**{out: first}) == 2 and f(**{out: last}) == 2, (out, inp)
            if sizes[out] > 1:
                assert f(**{out: first - 4 * (sizes[out] - 1)}) == 2, (out, inp)


def test_rope_table_refusals(lib):
    def f(p=A, n=8, r=64, base=1e4, factor=1.0, orig=0, lo=1.0, hi=32.0, m=1.0):
        return lib.attn_rope_table(p, n, r, base, factor, orig, lo, hi, m, None)
    assert f(n=-1) == 2 and f(r=0) == 2 and f(r=24) == 2 and f(r=528) == 2 and f(orig=-1) == 2
    assert f(base=1.0) == 2 and f(base=math.inf) == 2 and f(factor=0.0) == 2 and f(factor=math.nan) == 2
    assert f(lo=2.0, hi=2.0) == 2 and f(m=math.nan) == 2
    assert f(p=NULL) == 1 and f(p=A + 4) == 4 and f(p=NULL, n=0) == 0


def test_rope_refusals(lib):
    good = strides(*[0, 256, 64] * 4)

    def f(q=A, k=A, qo=A, ko=A, pos=A, ps=3, tab=A, n=9, B=2, T=3, Hq=4, Hkv=2, D=64, r=32, st=good, fn=None):
        return (fn or lib.attn_rope)(q, k, qo, ko, pos, ps, tab, n, B, T, Hq, Hkv, D, r, 0, st, None)
    for fn in (lib.attn_rope, lib.attn_rope_bwd):
        assert f(B=-1, fn=fn) == 2 and f(T=-1, fn=fn) == 2 and f(Hq=65535, fn=fn) == 2 and f(B=1 << 20, T=1 << 11, fn=fn) == 2
        assert f(D=40, fn=fn) == 3 and f(D=528, fn=fn) == 3
        assert f(r=80, fn=fn) == 2 and f(r=24, fn=fn) == 2 and f(r=0, fn=fn) == 2 and f(ps=2, fn=fn) == 2
        for name in ("q", "k", "qo", "ko", "pos", "tab", "st"):
            assert f(**{name: NULL}, fn=fn) == 1, name
        for name in ("q", "k", "qo", "ko", "tab"):
            assert f(**{name: A + 8}, fn=fn) == 4, name
        assert f(st=strides(*[0, 256, 64] * 3, 0, 256, 60), fn=fn) == 4
        assert f(st=strides(-8, 256, 64, *[0, 256, 64] * 3), fn=fn) == 2
        assert f(q=NULL, T=0, ps=0, fn=fn) == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "q4"])
def test_append_refusals(lib, fmt):
    good = strides(0, 256, 64, 0, 256, 64)

    def f(k=A, v=A, slots=A, pos=A, tab=A, n=9, r=32, c=(A,) * 4, s=(0.1, 0.1), B=1, T=3, H=2, D=64, page=16, pages=4,
          st=good):
        fn = {"bf16": lib.attn_cache_append, "fp8": lib.attn_cache_append_fp8, "q4": lib.attn_cache_append_q4}[fmt]
        c, s = (c, s) if fmt == "q4" else (c[::2], s if fmt == "fp8" else ())
        return fn(k, v, slots, pos, tab, n, r, 0, *c, *s, B, T, H, D, page, pages, st, None)
    assert f(B=-1) == 2 and f(H=0) == 2 and f(D=96) == 3 and f(page=0) == 2 and f(pages=0) == 2
    assert f(page=1 << 16, pages=1 << 15) == 2                       # more than 2^31 - 1 slots
    assert f(r=24) == 2 and f(r=128) == 2 and f(n=-1) == 2
    for name in ("k", "v", "slots", "pos", "st"):
        assert f(**{name: NULL}) == 1, name
    assert f(c=(NULL, A, A, A)) == 1 and f(c=(A, A, NULL, A)) == 1 and f(c=(A + 8, A, A, A)) == 4
    assert f(k=A + 2) == 4 and f(tab=A + 4) == 4 and f(st=strides(0, 256, 64, 0, 256, 63)) == 4
    if fmt != "bf16":
        for bad in (0.0, -1.0, math.nan, math.inf, 1e-30):
            assert f(s=(bad, 0.1)) == 2 and f(s=(0.1, bad)) == 2
    if fmt == "q4":
        assert f(c=(A, NULL, A, A)) == 1 and f(c=(A, A, A, A + 4)) == 4
    assert f(k=NULL, T=0) == 0


def test_gather_refusals(lib):
    def f(slots=A, c=(A,) * 4, s=(0.1, 0.1), k=A, v=A, n=3, H=2, D=64, page=16, pages=4):
        return lib.attn_cache_gather_q4(slots, *c, *s, k, v, n, H, D, page, pages, None)
    assert f(n=-1) == 2 and f(H=0) == 2 and f(D=32) == 3 and f(page=0) == 2 and f(s=(math.nan, 1.0)) == 2
    assert f(slots=NULL) == 1 and f(k=NULL) == 1 and f(c=(A, A, A, NULL)) == 1 and f(v=A + 8) == 4
    assert f(slots=NULL, n=0) == 0


def test_decode_q4_refusals(lib):
    def f(q=A, c=(A,) * 4, ks=0.1, lens=A, o=A, lse=A, ws=A, wb=1 << 40, B=2, Hq=4, Hkv=2, Tq=1, S=4096, D=64, scale=0.1,
          rope=(None, 0)):
        return lib.attn_decode_q4_fwd(q, *c, ks, 0.1, lens, o, lse, ws, wb, B, Hq, Hkv, Tq, S, D, scale, *rope, None)
    assert f(Tq=5, S=4) == 2 and f(Hq=6, Hkv=4) == 2 and f(D=96) == 3 and f(B=-1) == 2
    assert f(scale=math.inf) == 2 and f(ks=math.nan) == 2
    for name in ("q", "lens", "o", "lse"):
        assert f(**{name: NULL}) == 1, name
    assert f(c=(A, NULL, A, A)) == 1 and f(c=(A, A, A + 8, A)) == 4 and f(lens=A + 2) == 4
    assert f(rope=(A + 4, 4096)) == 4 and f(rope=(A, 4095)) == 2
    assert f(q=NULL, B=0) == 0 and f(q=NULL, Tq=0) == 0
    need = lib.attn_decode_q4_workspace_size(2, 4, 2, 1, 4096, 64)
    if need:
        assert f(ws=NULL) == 6 and f(wb=need - 1) == 6 and f(ws=A + 16) == 6
    assert lib.attn_decode_q4_workspace_size(2, 4, 2, 1, 4096, 96) == 0

    def p(bt=A, ps=64, pages=8, mp=8, **kw):
        return lib.attn_decode_paged_q4_fwd(A, A, A, A, A, 0.1, 0.1, bt, A, A, A, A, 1 << 40, 2, 4, 2, 1, ps, pages, mp, 64,
                                            0.1, kw.get("tab"), kw.get("n", 0), None)
    assert p(ps=48) == 2 and p(ps=8) == 2 and p(ps=0) == 2 and p(pages=0) == 2 and p(mp=0) == 2 and p(bt=NULL) == 1
    assert p(bt=A + 2) == 4 and p(tab=A, n=511) == 2 and p(mp=1 << 26) == 2


def test_decode_q4_capacities_near_2_31(lib):
    """The kernel counts a row's keys in 32-key tiles with 32-bit positions, one tile past the last at most: capacities
    whose last tile would end past 2^31 - 1 are refused, the ones below are not."""
    most = 0x7fffffff - 32
    for D in (64, 128):
        assert lib.attn_decode_q4_workspace_size(1, 1, 1, 1, most, D) > 0
        for S in (most + 1, 0x7ffffffe, 0x7fffffff):
            assert lib.attn_decode_q4_workspace_size(1, 1, 1, 1, S, D) == 0
            assert lib.attn_decode_q4_fwd(A, A, A, A, A, 0.1, 0.1, A, A, A, A, 1 << 40, 1, 1, 1, 1, S, D, 0.1, None, 0, None) == 2

        def paged(page, max_pages):
            return lib.attn_decode_paged_q4_fwd(A, A, A, A, A, 0.1, 0.1, A, A, A, A, NULL, 0, 1, 1, 1, 1, page, 1, max_pages, D,
                                                0.1, None, 0, None)
        assert paged(16, (1 << 27) - 1) == 2 and paged(16, (1 << 27) - 2) == 2      # 2^31 - 16, 2^31 - 32
        assert paged(16, (1 << 27) - 3) == 6 and paged(0x7fffff80, 1) == 6          # 2^31 - 48, - 128: only the workspace lacks


def test_parameters_that_overflow_in_the_kernels_are_refused(lib):
    """Finite in what the call takes, infinite in what the kernel works with."""
    def table(factor=1.0, m=1.0):
        return lib.attn_rope_table(A, 8, 64, 1e4, factor, 0, 1.0, 32.0, m, None)
    for m in (1e39, -1e39, 3.5e38):                                  # mscale is applied in f32
        assert table(m=m) == 2
    assert table(factor=1e-310) == 2                                 # 1 / factor
    size = (2, 4, 2, 1, 4096, 64)
    for scale, ks in ((1e30, 1e30), (-1e30, 1e30), (3e38, 1.0), (1.0, 3e38)):       # scale * k_scale * log2(e) is one f32
        assert lib.attn_decode_q4_fwd(A, A, A, A, A, ks, 0.1, A, A, A, A, 1 << 40, *size, scale, None, 0, None) == 2
        assert lib.attn_decode_paged_q4_fwd(A, A, A, A, A, ks, 0.1, A, A, A, A, A, 1 << 40, 2, 4, 2, 1, 64, 8, 64, 64, scale,
                                            None, 0, None) == 2


def test_binding_refuses_cpu_tensors():
    import causal_gqa_attention_fwd_gb300 as g
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    tab = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        g.attn_rope(x, x, i, tab)
    with pytest.raises(ValueError, match="CUDA"):
        g.attn_cache_plan(i, i, torch.zeros(2, 4, dtype=torch.int32), 16, i, None, 4)
    with pytest.raises(ValueError, match="CUDA"):
        g.attn_cache_append(x, x, i, x, x)
    with pytest.raises(TypeError):
        g.attn_cache_gather_q4([1], x, x, x, x, 1.0, 1.0)


def test_workspace_size_is_the_c_functions():
    import causal_gqa_attention_fwd_gb300 as g
    for args in ((2, 8, 2, 1, 4096, 128), (1, 16, 1, 1, 64, 64), (3, 6, 2, 7, 100, 128)):
        assert g.attn_decode_q4_workspace_size(*args) == int(g.lib().attn_decode_q4_workspace_size(*args)) > 0


def test_native_module_fails_loudly_when_missing(monkeypatch):
    import sys

    from causal_gqa_attention_fwd_gb300 import _cache
    monkeypatch.setattr(_cache, "_bound", None)
    monkeypatch.setattr(_cache, "_mod", None)
    monkeypatch.setitem(sys.modules, "causal_gqa_attention_fwd_gb300._cache_ext", None)
    monkeypatch.delattr("causal_gqa_attention_fwd_gb300._cache_ext", raising=False)
    with pytest.raises(RuntimeError, match="no fallback"):
        _cache._ext()


class OnCuda1(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 1)


class FakeStream:
    def __init__(self, handle, device=None):
        self.handle, self.device = handle, device if device is None else torch.device(device)


@pytest.fixture
def streams(monkeypatch):
    """torch.cuda's streams without a GPU: the streams that calls were made on; cuda:0 is the current device."""
    import contextlib
    used = []

    @contextlib.contextmanager
    def use(s):
        used.append((s.handle, s.device))
        yield
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", type("FakeExternal", (FakeStream,), {}))
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return used


def test_a_call_runs_on_its_stream_of_the_tensors_device(streams):
    from causal_gqa_attention_fwd_gb300 import _cache
    x = torch.zeros(2).as_subclass(OnCuda1)
    dev = torch.device("cuda", 1)
    assert _cache._run(77, lambda *a: a, None, x) == (None, x)
    assert _cache._run(FakeStream(5, "cuda:1"), lambda *a: len(a), x) == 1
    assert streams == [(77, dev), (5, dev)]
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        _cache._run(FakeStream(6, "cuda:0"), lambda *a: 1, x)
    assert len(streams) == 2


def test_rope_table_runs_on_the_given_devices_stream(streams, monkeypatch):
    """Without `out` there is no tensor to tell the device of a handle."""
    import types

    from causal_gqa_attention_fwd_gb300 import _cache
    made = []
    monkeypatch.setattr(torch, "empty", lambda *s, dtype, device: made.append(device) or torch.zeros(*s, dtype=dtype))
    monkeypatch.setattr(_cache, "_ext", lambda: types.SimpleNamespace(rope_table=lambda out, *a: out))
    one = torch.device("cuda", 1)
    for device in (1, "cuda:1", one):
        _cache.attn_rope_table(4, 16, device=device, stream=77)
        assert streams.pop() == (77, one) and torch.device(made.pop()) == one
        _cache.attn_rope_table(4, 16, device=device, stream=FakeStream(5, one))
        assert streams.pop() == (5, one) and torch.device(made.pop()) == one
        with pytest.raises(ValueError, match="cuda:0"):
            _cache.attn_rope_table(4, 16, device=device, stream=FakeStream(5, "cuda:0"))
    for device in (None, "cuda"):                       # the current device's
        _cache.attn_rope_table(4, 16, device=device, stream=78)
        assert streams.pop() == (78, torch.device("cuda", 0)) and str(made.pop()).startswith("cuda")
    _cache.attn_rope_table(4, 16, stream=FakeStream(5, one))            # no device named: the stream's
    assert streams.pop() == (5, one) and torch.device(made.pop()) == one
    _cache.attn_rope_table(4, 16, out=torch.zeros(4, 16).as_subclass(OnCuda1), stream=79)
    assert streams.pop() == (79, one) and not made and not streams


# ------------------------------------------------------------ the references
def test_reference_quantisation_by_hand():
    """One block whose scale is exactly 1: amax 6; ties go to the even code; the sign is the top bit."""
    x = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5.1, 0, 0.3, 1.2, -1.3, 2.6])
    p, sf = R.quantise(x, 1.0)
    codes = torch.stack([p & 15, p >> 4], -1).flatten().tolist()
    assert sf.tolist() == [0x38]
    assert codes == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 15, 0, 1, 2, 11, 5]
    assert R.values(p, sf, 1.0).tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -6, 0, 0.5, 1, -1.5, 3]


def test_reference_rope_turns_and_turns_back():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 3, 64, generator=g, dtype=torch.float64)
    ang = torch.rand(9, 24, generator=g, dtype=torch.float64) * 7
    tab = torch.cat([ang.cos(), ang.sin()], 1)
    pos = torch.tensor([0, 8, 3, 3, 1])[:, None]
    for inter in (False, True):
        y = R.rope(x, pos, tab, inter)
        assert torch.allclose(R.rope(y, pos, tab, inter, -1.0), x, atol=1e-12)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1)) and torch.equal(y[..., 48:], x[..., 48:])
    # the two layouts are one another's reordering
    perm = torch.cat([torch.arange(0, 48, 2), torch.arange(1, 48, 2), torch.arange(48, 64)])
    assert torch.allclose(R.rope(x, pos, tab, True)[..., perm], R.rope(x[..., perm], pos, tab, False))


def test_reference_decode_is_the_oracles():
    import numpy as np
    import oracle
    oracle.build()
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(2, h, n, 64, generator=g, dtype=torch.float64) for h, n in ((4, 3), (2, 20), (2, 20)))
    lens = torch.tensor([20, 5], dtype=torch.int32)
    o, lse, _, _ = R.decode(q, k, v, lens, 0.2)
    ro, rl = oracle.decode_fwd(q.numpy(), k.numpy(), v.numpy(), lens.numpy(), scale=0.2)
    assert np.abs(o.numpy() - ro).max() < 1e-12 and np.abs(lse.numpy() - rl).max() < 1e-12


def test_reference_plan_by_hand():
    table = torch.tensor([[4, -1, -1], [-1, -1, -1], [7, 8, -1]], dtype=torch.int32)
    s, p, cu, n, c, t, ok = R.plan(torch.tensor([3, 0, 8]), torch.tensor([2, 5, 1]), table, 4, [9, 1, 2, 5], 0, 10)
    assert s.tolist() == [19, 36, 4, 5, 6, 7, 8, 20, -1, -1] and p.tolist() == [3, 4, 0, 1, 2, 3, 4, 8, 0, 0]
    assert cu.tolist() == [0, 2, 7, 8] and n.tolist() == [5, 5, 9] and c.tolist() == [4] and ok == [True] * 3
    assert t.tolist() == [[4, 9, -1], [1, 2, -1], [7, 8, 5]]
