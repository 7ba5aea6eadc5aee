"""attn_cache_plan on the GPU against a loop over requests: all outputs are whole numbers and equal."""
import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


def problem(lens, new, page, mp, spare=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    lens, new = (torch.tensor(x, dtype=torch.int32) for x in (lens, new))
    B = len(lens)
    ids = torch.randperm(B * mp + 50, generator=g).to(torch.int32)
    table = torch.full((B, mp), -1, dtype=torch.int32)
    at = 0
    need = 0
    for b in range(B):
        n, a = int(lens[b]), int(new[b])
        if n < 0 or a < 0 or n + a > mp * page:
            continue
        have = -(-n // page)
        table[b, :have] = ids[at:at + have]
        at += have
        need += -(-(n + a) // page) - have
    return lens, new, table, ids[at:at + need + spare].clone()


def check(gq, lens, new, table, page, free, cursor, total, status=0):
    c = None if cursor is None else torch.tensor([cursor], dtype=torch.int32).cuda()
    t = table.cuda()
    got = gq.attn_cache_plan(lens.cuda(), new.cuda(), t, page, free.cuda(), c, total)
    assert gq.get_device_status() == status
    ref = R.plan(lens, new, table, page, free, cursor or 0, total)
    for name, a, b in zip(("slots", "positions", "cu_seqlens", "lens_out", "cursor_out"), got, ref):
        assert torch.equal(a.cpu(), b), name
    assert torch.equal(t.cpu(), ref[5]), "block_table"
    return ref


@pytest.mark.parametrize("page", [1, 16, 48, 128])
@pytest.mark.parametrize("B", [1, 5, 37, 700])
def test_plan_matches_loop(gq, B, page):
    g = torch.Generator().manual_seed(B * 1000 + page)
    mp = -(-400 // page)
    lens = torch.randint(0, 200, (B,), generator=g).tolist()
    new = torch.randint(0, 200, (B,), generator=g).tolist()
    lens[0], new[-1] = 0, 0                       # an empty request, one without new tokens
    if B > 2:
        lens[2], new[2] = mp * page - 7, 7        # fills its row to the last position
    x = problem(lens, new, page, mp)
    check(gq, x[0], x[1], x[2], page, x[3], None, sum(new) + 5)
    check(gq, x[0], x[1], x[2], page, torch.cat([torch.full((4,), -1, dtype=torch.int32), x[3]]), 4, sum(new))


def test_plan_nothing_to_do(gq):
    e = torch.zeros(0, dtype=torch.int32)
    x = problem([5, 0], [0, 0], 16, 4)
    check(gq, x[0], x[1], x[2], 16, e, None, 0)
    check(gq, x[0], x[1], x[2], 16, x[3], 1, 3)
    check(gq, e, e, torch.zeros(0, 4, dtype=torch.int32), 16, e, None, 2)


def test_plan_most_requests(gq):
    """8192 requests: the offsets fill more shared memory than the default."""
    x = problem([17] * 8192, [1, 0, 40] * 2730 + [2, 2], 32, 3)
    check(gq, x[0], x[1], x[2], 32, x[3], 0, int(x[1].sum()) + 1)


def test_plan_refuses_bad_lengths(gq):
    """A negative length or addition and a row that would overflow are refused one by one, the others served."""
    x = problem([3, -1, 40, 64, 9], [5, 6, -2, 1, 60], 16, 4)
    ref = check(gq, x[0], x[1], x[2], 16, x[3], 0, 80, status=5)
    assert ref[6] == [True, False, False, False, False]
    x = problem([3, -1, 40, 9], [5, 6, -2, 30], 16, 4)
    assert check(gq, x[0], x[1], x[2], 16, x[3], 0, 80, status=5)[6] == [True, False, False, True]


def test_plan_pages_run_out(gq):
    """The first request whose pages are not there and all after it keep their lengths; the earlier ones are served."""
    x = problem([10, 0, 31, 16], [10, 33, 1, 1], 16, 8)
    for k in range(len(x[3]) - 3 + 1):
        enough = k >= 1 + 3 + 0 + 1
        ref = check(gq, x[0], x[1], x[2], 16, x[3][:k], 0, 45, status=0 if enough else 11)
        assert ref[6] == [k >= 1, k >= 4, k >= 4, k >= 5]
    # a cursor outside the list: only requests before any that needs a page are served
    y = problem([10, 10], [1, 10], 16, 8)
    for cur in (-3, 99):
        assert check(gq, y[0], y[1], y[2], 16, y[3], cur, 11, status=11)[6] == [True, False]


def test_plan_tokens_beyond_the_total(gq):
    x = problem([4, 4, 4], [5, 6, 7], 16, 2)
    ref = check(gq, x[0], x[1], x[2], 16, x[3], 0, 12, status=5)
    assert ref[6] == [True, True, False]


def test_plan_negative_pages_give_no_slot(gq):
    x = problem([20, 3], [20, 4], 16, 4)
    x[2][0, 1] = -1                     # the page that holds request 0's position 20
    check(gq, x[0], x[1], x[2], 16, x[3], 0, 24, status=11)
    x = problem([20, 3], [20, 4], 16, 4)
    x[3][0] = -5
    table = x[2].cuda()
    s, *_ = gq.attn_cache_plan(x[0].cuda(), x[1].cuda(), table, 16, x[3].cuda(), None, 24)
    assert gq.get_device_status() == 11
    assert s.cpu()[:20].tolist()[12:] == [-1] * 8 and (s.cpu()[:12] >= 0).all()


def test_plan_in_a_graph_follows_new_lengths(gq):
    """A captured plan, replayed after its inputs changed, gives the plan of the new inputs."""
    x = problem([10, 0, 31], [3, 4, 5], 16, 8, spare=20)
    lens, new, table, free = (t.cuda() for t in x)
    cur = torch.zeros(1, dtype=torch.int32, device="cuda")
    gq.attn_cache_plan(lens, new, table.clone(), 16, free, cur, 40)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = gq.attn_cache_plan(lens, new, table, 16, free, cur, 40)
    table.copy_(x[2].cuda())
    new.copy_(torch.tensor([7, 20, 1], dtype=torch.int32))
    cur.fill_(2)
    g.replay()
    assert gq.get_device_status() == 0
    ref = R.plan(x[0], torch.tensor([7, 20, 1]), x[2], 16, x[3], 2, 40)
    for a, b in zip(out, ref):
        assert torch.equal(a.cpu(), b)
    assert torch.equal(table.cpu(), ref[5])
