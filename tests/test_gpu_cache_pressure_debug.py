"""Shared prefixes, weights and eviction in the debug build: odd sizes raise no bounds check and give the release build's
results."""
import math

import pytest
import torch

import pressure_ref as R
import test_gpu_cache_evict as E
import test_gpu_cache_weights as W
from test_gpu_cache_debug import dbg, no_check_fired  # noqa: F401
from test_gpu_decode_prefix import check, make, tile_capacity

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("case", [(9, 3, 14, 2, 1, 64, 0, [129, 0, 7], [0, 1, 2, 64, 65, 130, 3, 4, 5]),
                                  (10, 1, 32, 4, 3, 128, 16, [401], [3 * i for i in range(10)]),
                                  (70, 1, 8, 2, 1, 128, 64, [257], [1 + i for i in range(70)])])
def test_debug_prefix(dbg, case, tiles):  # noqa: F811
    B, P, Hq, Hkv, Tq, D = case[:6]
    f, args, ref = make(*case, seed=1, Sp=tile_capacity(B, P, Hq, Hkv, Tq, D) if tiles else None)
    got = getattr(dbg, f)(*args)
    no_check_fired(dbg)
    check(got, R.prefix(*ref, 1 / math.sqrt(D)), D)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "q4"])
@pytest.mark.parametrize("stream", [False, True])
def test_debug_weights(dbg, fmt, stream):  # noqa: F811
    case = (3, 12, 4, 5, 64, 7, [0, 33, 100])
    planes, keys, q, table, w = W.make(fmt, *case, seed=2, S=W.stream_capacity(3, 4) if stream else None)
    lse = W.lse_of(q, keys, table, case[6], 0.125)
    out = W.call(dbg, fmt, planes, q, lse, case[6], w.cuda(), table, 0.125)
    no_check_fired(dbg)
    W.check(out, w, q, keys, lse, table, case[6], 0.125)


def test_debug_evict(dbg):  # noqa: F811
    lens = [130, 20, 333]
    planes, w, table = E.make("odd", 3, 2, 64, 16, lens, 2, "ties")
    got = E.run(dbg, planes, w, table, lens, 50, 7, 3)
    no_check_fired(dbg)
    E.check(got, E.reference(planes, w, table, lens, 50, 7, 3))
