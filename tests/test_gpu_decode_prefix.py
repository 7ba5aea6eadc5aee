"""Attention of rows that share prefixes against the definition in 64 bits."""
import math

import pytest
import torch

import pressure_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


def make(B, P, Hq, Hkv, Tq, D, page, plens, lens, seed, Sp=None, S=None, qs=1.0, junk=math.nan):
    """Inputs on the GPU; everything outside the lengths, and the pages of no row, is `junk`."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    Sp, S = Sp or max(*plens, 1), S or max(*lens, Tq)
    q = (rn(B, Hq, Tq, D).float() * qs).bfloat16()
    own = [(rn(Hkv, n, D), rn(Hkv, n, D)) for n in lens]
    pre = [(rn(Hkv, m, D), rn(Hkv, m, D)) for m in plens]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    d64 = lambda pairs: [(k.double(), v.double()) for k, v in pairs]  # noqa: E731
    if not page:
        bufs = []
        for pairs, cap in ((pre, Sp), (own, S)):
            for i in range(2):
                c = torch.full((len(pairs), Hkv, cap, D), junk, dtype=torch.bfloat16)
                for b, kv in enumerate(pairs):
                    c[b, :, :kv[i].shape[1]] = kv[i]
                bufs.append(c.cuda())
        args = (q.cuda(), bufs[0], bufs[1], i32(plens), bufs[2], bufs[3], i32(lens))
        return "attn_decode_prefix_fwd", args, (q, d64(pre), d64(own), lens)
    mp, mo = -(-Sp // page), -(-S // page)
    pages = P * mp + B * mo + 2
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    pt, bt = perm[:P * mp].reshape(P, mp).clone(), perm[P * mp:P * mp + B * mo].reshape(B, mo).clone()
    pools = [torch.full((pages, Hkv, page, D), junk, dtype=torch.bfloat16) for _ in range(2)]
    for pairs, t in ((pre, pt), (own, bt)):
        for b, kv in enumerate(pairs):
            n = kv[0].shape[1]
            for j0 in range(0, n, page):
                c = min(page, n - j0)
                for i in range(2):
                    pools[i][int(t[b, j0 // page]), :, :c] = kv[i][:, j0:j0 + c]
            t[b, -(-n // page):] = -7          # entries that no key needs may hold anything
    args = (q.cuda(), pools[0].cuda(), pools[1].cuda(), pt.cuda(), i32(plens), bt.cuda(), i32(lens))
    return "attn_decode_paged_prefix_fwd", args, (q, d64(pre), d64(own), lens)


def check(got, ref, D, what=""):
    o, lse = (x.cpu().double() for x in got)
    ro, rl, spread, weight = ref
    to, tl = R.prefix_tolerance(ro, rl, spread, weight, D)
    dead = rl == -math.inf
    assert torch.equal(lse == -math.inf, dead) and bool((o[dead] == 0).all()), what
    assert bool(torch.isfinite(o).all()), what
    assert bool(((lse - rl).abs()[~dead] <= tl[~dead]).all()), (what, float(((lse - rl).abs()[~dead] / tl[~dead]).max()))
    assert bool(((o - ro).abs() <= to).all()), (what, float(((o - ro).abs() / to).max()))


CASES = [
    # B, P, Hq, Hkv, Tq, D, page, prefix lengths, own lengths
    (1, 1, 1, 1, 1, 64, 0, [1], [1]),
    (1, 1, 4, 1, 1, 128, 0, [0], [1]),
    (2, 1, 14, 2, 1, 64, 0, [129], [1, 130]),
    (8, 1, 14, 2, 1, 64, 0, [2048], [1, 37, 128, 129, 200, 255, 256, 2]),
    (4, 2, 4, 4, 1, 128, 0, [300, 127], [5, 6, 300, 1]),
    (6, 3, 8, 2, 3, 128, 0, [128, 0, 513], [3, 9, 4, 3, 140, 7]),
    (5, 1, 16, 4, 4, 128, 0, [999], [4, 777, 128, 127, 60]),
    (33, 1, 8, 2, 1, 128, 0, [700], list(range(1, 34))),                       # 132 rows: both tiles, the second short
    (64, 1, 8, 2, 1, 64, 0, [257], [1 + i * 3 for i in range(64)]),            # 256 rows
    (65, 1, 12, 3, 1, 64, 0, [640], [1 + i for i in range(65)]),               # 260 rows: a unit of 4 more
    (40, 1, 8, 1, 2, 128, 0, [385], [2 + i for i in range(40)]),               # 640 rows, 3 units
    (10, 2, 7, 1, 5, 64, 0, [1500, 64], [5, 6, 7, 8, 9, 64, 128, 200, 12, 77]),
    (3, 1, 4, 2, 1, 64, 16, [100], [1, 17, 33]),
    (8, 2, 16, 8, 1, 128, 16, [1001, 16], [5, 16, 17, 64, 501, 1, 2, 128]),
    (4, 1, 8, 2, 2, 128, 32, [255], [2, 31, 32, 33]),
    (4, 4, 8, 2, 1, 64, 64, [64, 1, 200, 0], [1, 64, 65, 190]),
    (70, 1, 8, 2, 1, 128, 64, [1000], [1 + 5 * i for i in range(70)]),
    (4, 1, 8, 2, 1, 128, 128, [400], [1, 128, 129, 300]),
    (2, 1, 8, 2, 1, 64, 256, [700], [300, 10]),
]


def tile_capacity(B, P, Hq, Hkv, Tq, D):
    """The least prefix capacity (in steps of 1024) that sends prefixes of more than 16 query rows to the kernel of large
    tiles: it counts what the stream would read again, not how long the prefixes are."""
    again = -(-(B // P * Hq // Hkv * Tq) // 16) - 1
    return ((97 << 20) // (again * P * Hkv * D * 4) // 1024 + 1) * 1024 if again else None


def ran(gq, f):
    """f(), and which kernels it launched."""
    gq.profile_enable(True)
    gq.profile_reset()
    out = f()
    torch.cuda.synchronize()
    names = {k for k, (n, _) in gq.profile_read().items() if n}
    gq.profile_enable(False)
    return out, names


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{c[0]}P{c[1]}H{c[2]}-{c[3]}T{c[4]}D{c[5]}p{c[6]}m{max(c[7])}")
def test_against_the_definition(gq, case, tiles):
    """Both ways a prefix goes: in the stream of tiles beside the rows' own keys, and through the kernel of large tiles."""
    B, P, Hq, Hkv, Tq, D, page, plens, lens = case
    Sp = tile_capacity(B, P, Hq, Hkv, Tq, D) if tiles else None
    if tiles and Sp is None:
        pytest.skip("at most 16 query rows a key: always in the stream")
    f, args, ref = make(*case, seed=1, Sp=Sp)
    scale = 1 / math.sqrt(D)
    got, names = ran(gq, lambda: getattr(gq, f)(*args, scale=scale))
    assert names == ({"prefix", "prefix_merge"} if tiles else {"own_keys", "prefix_merge"})
    assert gq.get_device_status() == 0
    check(got, R.prefix(*ref, scale), D)
    again = getattr(gq, f)(*args, scale=scale)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("Hq", [8, 64])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("Tq,lens", [(1, [0, 5, 0, 1]), (4, [0, 1, 3, 4]), (3, [2, 2, 0, 0]), (2, [0, 0, 0, 0])])
def test_queries_at_negative_positions_see_nothing(gq, page, Tq, lens, Hq):
    f, args, ref = make(4, 2, Hq, 2, Tq, 128, page, [130, 0], lens, seed=2,
                        Sp=tile_capacity(4, 2, Hq, 2, Tq, 128) if Hq == 64 else None)
    got = getattr(gq, f)(*args, scale=0.1)
    assert gq.get_device_status() == 0
    check(got, R.prefix(*ref, 0.1), 128)


def test_capacities_beyond_the_lengths_and_default_scale(gq):
    for page in (0, 64):
        f, args, ref = make(3, 1, 6, 2, 2, 64, page, [77], [2, 40, 90], seed=3, Sp=640, S=448)
        got = getattr(gq, f)(*args)
        assert gq.get_device_status() == 0
        check(got, R.prefix(*ref, 1 / 8), 64)


@pytest.mark.parametrize("tiles", [False, True])
def test_large_scores_and_growing_maxima(gq, tiles):
    """Scores of tens, rising along the prefix, so that the running maximum moves in every block."""
    f, args, ref = make(9, 1, 8, 2, 1, 128, 0, [900], [1 + 20 * i for i in range(9)], seed=4, qs=6.0,
                        Sp=tile_capacity(9, 1, 8, 2, 1, 128) if tiles else None)
    k = args[1][:, :, :900]
    ramp = torch.linspace(0.1, 3.0, 900, device="cuda")
    k.copy_((k.float() * ramp[None, None, :, None]).bfloat16())
    pre = [(k[0].cpu().double(), ref[1][0][1])]
    got = getattr(gq, f)(*args, scale=0.2)
    check(got, R.prefix(ref[0], pre, ref[2], ref[3], 0.2), 128)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.11, 1e-30, 2.5])
def test_scales(gq, tiles, scale):
    f, args, ref = make(9, 1, 8, 2, 1, 128, 0, [300], [1 + 20 * i for i in range(9)], seed=14,
                        Sp=tile_capacity(9, 1, 8, 2, 1, 128) if tiles else None)
    got = getattr(gq, f)(*args, scale=scale)
    assert gq.get_device_status() == 0
    check(got, R.prefix(*ref, scale), 128)


@pytest.mark.parametrize("tiles", [False, True])
def test_a_prefix_that_is_not_finite(gq, tiles):
    """An infinite value and a NaN key of one prefix: its own rows are what the definition makes of them, others are whole."""
    B, P, Hq = 8, 2, 16
    f, args, ref = make(B, P, Hq, 2, 1, 64, 16, [200, 150], [3 + i for i in range(B)], seed=15, junk=0.0,
                        Sp=tile_capacity(B, P, Hq, 2, 1, 64) if tiles else None)
    page = int(args[3][0, 4])                       # keys 64..79 of prefix 0
    args[2][page, 1, 3, 7] = math.inf
    o, lse = getattr(gq, f)(*args, scale=0.125)
    assert gq.get_device_status() == 0
    want = R.prefix(*ref, 0.125)
    o[:4, 8:, :, 7] = want[0][:4, 8:, :, 7].bfloat16().cuda()          # infinity, where the definition says so
    check((o, lse), want, 64)
    args[1][page, 0, 9] = math.nan
    o, lse = getattr(gq, f)(*args, scale=0.125)
    assert bool(torch.isnan(o[:4, :8]).all()) and bool(torch.isnan(lse[:4, :8]).all())
    check((o[4:], lse[4:]), [x[4:] for x in want], 64)


def check_with_nan(got, ref, D):
    """As check, but where the definition gives a log-sum-exp of NaN both outputs are NaN; returns those queries."""
    lost = torch.isnan(ref[1])
    o, lse = (x.cpu().double() for x in got)
    assert torch.equal(torch.isnan(lse), lost) and torch.equal(torch.isnan(o).all(-1), lost)
    whole = lambda x: x.masked_fill(lost.reshape(lost.shape + (1,) * (x.dim() - 3)), 0.0)  # noqa: E731
    check((whole(o), whole(lse)), [whole(x) for x in ref], D)
    return lost


NAN_CASES = [
    # as CASES, and warps a row that join its pieces: 8, 16, 8 (heads of 64), 4, 1
    (2, 1, 8, 2, 1, 128, 0, [64], [1, 1]),
    (12, 1, 8, 1, 1, 128, 0, [9000], [1, 2, 17, 40, 1, 1, 1, 3, 16, 1, 700, 1]),
    (40, 2, 24, 1, 1, 64, 0, [500, 64], [1 + i % 33 for i in range(40)]),
    (20, 1, 16, 2, 3, 128, 0, [64], [3 + i % 20 for i in range(20)]),
    (60, 1, 32, 2, 1, 64, 0, [130], [1 + i % 3 for i in range(60)]),
]


@pytest.mark.parametrize("what", ["a row's newest key", "a row's keys", "a prefix", "a query"])
@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("case", NAN_CASES, ids=lambda c: f"B{c[0]}H{c[2]}-{c[3]}T{c[4]}D{c[5]}m{max(c[7])}")
def test_nan_scores_reach_the_outputs(gq, case, tiles, what):
    """A NaN score makes NaN of the output and of the log-sum-exp of the queries that see it, however the row's keys are cut
    into pieces (a piece of nothing but NaN scores has no maximum), and of no other."""
    B, P, Hq, Hkv, Tq, D, page, plens, lens = case
    Sp = tile_capacity(B, P, Hq, Hkv, Tq, D) if tiles else None
    if tiles and Sp is None:
        pytest.skip("at most 16 query rows a key: always in the stream")
    f, args, (q, pre, own, lens) = make(*case, seed=21, Sp=Sp)
    for b in (0,) if what == "a prefix" else (0, B // 2):
        h = (b + 1) % Hkv
        if what == "a query":
            q[b, h * (Hq // Hkv), 0] = math.nan
            args[0][b, h * (Hq // Hkv), 0] = math.nan
        elif what == "a prefix":
            pre[0][0][h] = math.nan
            args[1][0, h] = math.nan
        else:
            j = lens[b] - 1 if what == "a row's newest key" else 0
            own[b][0][h, j:] = math.nan
            args[4][b, h, j:] = math.nan
    o, lse = getattr(gq, f)(*args, scale=0.1)
    assert gq.get_device_status() == 0
    lost = check_with_nan((o, lse), R.prefix(q, pre, own, lens, 0.1), D)
    assert bool(lost.any()) and (what == "a prefix" or not bool(lost.all()))
    # a NaN log-sum-exp is not the -infinity of a query that saw nothing: the keys' weights are NaN too
    w = torch.zeros(args[4].shape[:3], device="cuda")
    gq.attn_cache_weights(args[0], args[4], lse, args[6], w, scale=0.1)
    if what == "a query":
        assert bool(torch.isnan(w[0, 1 % Hkv, :lens[0] - Tq + 1]).all())


def test_no_prefix_at_all(gq):
    f, args, ref = make(3, 1, 4, 2, 1, 64, 0, [0], [9, 200, 1], seed=5)
    empty = torch.empty(1, 2, 0, 64, dtype=torch.bfloat16, device="cuda")
    got = gq.attn_decode_prefix_fwd(args[0], empty, empty, *args[3:], scale=0.125)
    assert gq.get_device_status() == 0
    check(got, R.prefix(*ref, 0.125), 64)


def test_agrees_with_the_decode_over_the_joined_cache(gq):
    """The same keys as one cache a row: the outputs differ by the roundings alone."""
    B, D, m, lens = 6, 128, 500, [1, 12, 128, 129, 64, 33]
    f, args, ref = make(B, 1, 8, 2, 1, D, 0, [m], lens, seed=6)
    k, v = (torch.cat([args[1 + i].expand(B, -1, -1, -1)[:, :, :m], args[4 + i]], 2).nan_to_num().contiguous() for i in range(2))
    o, lse = gq.attn_decode_fwd(args[0], k, v, (args[6] + m).int(), scale=0.09)
    got = getattr(gq, f)(*args, scale=0.09)
    want = R.prefix(*ref, 0.09)
    check(got, want, D)
    check((o, lse), want, D)


@pytest.mark.parametrize("Hq", [4, 128])
def test_bad_lengths_and_pages_are_reported(gq, Hq):
    f, args, ref = make(4, 2, Hq, 2, 1, 64, 16, [40, 33], [3, 4, 5, 6], seed=7, junk=0.0,
                        Sp=tile_capacity(4, 2, Hq, 2, 1, 64) if Hq == 128 else None)
    for i, bad, rows in ((4, 1 << 20, [0, 1]), (4, -1, [0, 1]), (6, -2, [0]), (6, 1 << 20, [0])):
        a = list(args)
        a[i] = a[i].clone()
        a[i][0] = bad
        o, lse = torch.full_like(args[0], 7.0), torch.full(args[0].shape[:3], 7.0, device="cuda")
        gq.attn_decode_paged_prefix_fwd(*a, scale=0.1, o=o, lse=lse)
        assert gq.get_device_status() == 5
        live = [b for b in range(4) if b not in rows]
        assert bool((o[rows] == 7).all()) and bool((lse[rows] == 7).all())
        want = R.prefix(*ref, 0.1)
        check((o[live], lse[live]), [x[live] for x in want], 64)
    for i in (3, 5):
        a = list(args)
        a[i] = a[i].clone()
        a[i][0, 0] = args[1].shape[0]
        gq.attn_decode_paged_prefix_fwd(*a, scale=0.1)
        assert gq.get_device_status() == 11
    assert gq.get_device_status() == 0


@pytest.mark.parametrize("Hq", [2, 24])
def test_many_prefixes_of_one_row_each(gq, Hq):
    """More prefixes than a scan of 32 holds, lengths from none to several blocks."""
    P = 70
    plens = [(37 * i) % 400 for i in range(P)]
    f, args, ref = make(P, P, Hq, 1, 1, 64, 0, plens, [1 + i % 50 for i in range(P)], seed=8,
                        Sp=tile_capacity(P, P, Hq, 1, 1, 64) if Hq == 24 else None)
    got = getattr(gq, f)(*args, scale=0.125)
    assert gq.get_device_status() == 0
    check(got, R.prefix(*ref, 0.125), 64)


@pytest.mark.parametrize("Hq", [4, 40])
def test_more_rows_than_a_block_scans_at_once(gq, Hq):
    B = 500
    f, args, ref = make(B, 4, Hq, 1, 1, 64, 16, [5, 0, 300, 129], [(7 * i) % 40 for i in range(B)], seed=12,
                        Sp=tile_capacity(B, 4, Hq, 1, 1, 64) if Hq == 40 else None)
    got = getattr(gq, f)(*args, scale=0.125)
    assert gq.get_device_status() == 0
    check(got, R.prefix(*ref, 0.125), 64)


def test_workspace_and_streams(gq):
    f, args, ref = make(8, 1, 8, 2, 1, 128, 0, [1024], [1 + i for i in range(8)], seed=9)
    n = gq.attn_decode_prefix_workspace_size(8, 8, 2, 1, 1, 1024, 8, 128)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")           # nothing in it is relied on
    a = gq.attn_decode_prefix_fwd(*args, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = gq.attn_decode_prefix_fwd(*args, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(gq.AttnError, match="WORKSPACE"):
        gq.attn_decode_prefix_fwd(*args, workspace=ws[:n - 256])


@pytest.mark.parametrize("tiles", [False, True])
def test_replayed_with_other_lengths(gq, tiles):
    """A captured call reads the lengths on the device: replayed after they changed, it gives the eager call's bits."""
    f, args, ref = make(8, 1, 8, 2, 1, 128, 64, [900], [50 + 9 * i for i in range(8)], seed=10, junk=0.0,
                        Sp=tile_capacity(8, 1, 8, 2, 1, 128) if tiles else None)
    o, lse = torch.empty_like(args[0]), torch.empty(args[0].shape[:3], device="cuda")
    getattr(gq, f)(*args, o=o, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        getattr(gq, f)(*args, o=o, lse=lse)
    for m, cut in ((900, 0), (129, 3), (1, 40), (0, 50)):
        args[4].fill_(m)
        args[6].sub_(cut).clamp_(min=0)
        want = getattr(gq, f)(*args)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_arguments(gq):
    f, args, ref = make(4, 2, 4, 2, 1, 64, 0, [8, 9], [3, 4, 5, 6], seed=11)
    q, kp, vp, pl, k, v, ln = args
    call = gq.attn_decode_prefix_fwd
    with pytest.raises(ValueError, match="multiple of the prefixes"):
        call(q[:3].contiguous(), kp, vp, pl, k[:3].contiguous(), v[:3].contiguous(), ln[:3].contiguous())
    with pytest.raises(ValueError, match="k_prefix, v_prefix"):
        call(q, kp[:1], vp[:1], pl, k, v, ln)
    with pytest.raises(ValueError, match="k_cache, v_cache"):
        call(q, kp, vp, pl, k[..., :32].contiguous(), v, ln)
    with pytest.raises(TypeError, match="int32"):
        call(q, kp, vp, pl.long(), k, v, ln)
    with pytest.raises(TypeError, match="bfloat16"):
        call(q, kp.half(), vp, pl, k, v, ln)
    with pytest.raises(TypeError, match="k_prefix"):
        call(q, None, None, pl, k, v, ln)
    with pytest.raises(ValueError, match="contiguous"):
        call(q.expand(4, 4, 1, 64).transpose(1, 1)[:, ::2].repeat(1, 2, 1, 1)[:, ::2], kp, vp, pl, k, v, ln)
    with pytest.raises(ValueError, match="cache_lens"):
        call(q, kp, vp, pl, k, v, ln[:3])
    with pytest.raises(gq.AttnError, match="SHAPE"):
        call(q, kp, vp, pl, k, v, ln, scale=math.inf)
    with pytest.raises(ValueError, match="CUDA"):
        call(q.cpu(), kp, vp, pl, k, v, ln)
    f, args, ref = make(4, 2, 4, 2, 1, 64, 16, [8, 9], [3, 4, 5, 6], seed=11)
    q, k, v, pt, pl, bt, ln = args
    call = gq.attn_decode_paged_prefix_fwd
    with pytest.raises(ValueError, match="prefix_table"):
        call(q, k, v, pt[:1], pl, bt, ln)
    with pytest.raises(ValueError, match="block_table"):
        call(q, k, v, pt, pl, bt[:1], ln)
    with pytest.raises(TypeError, match="block_table"):
        call(q, k, v, pt, pl, None, ln)
    with pytest.raises(gq.AttnError, match="SHAPE"):                           # page sizes of the paged decode
        call(q, k[:, :, :8].contiguous(), v[:, :, :8].contiguous(), pt, pl, bt, ln)
