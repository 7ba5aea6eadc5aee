"""How attention over shared prefixes shares its CTAs out, as the kernel's own arithmetic built for the host."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_gqa_attention_fwd_gb300", "csrc")

SOURCE = """
#include "share_out.h"
static gqa::ShareWork work(const int* v) {
  return {v[0], v[1], v[2], v[3], v[4], v[5] != 0, v[6], v[7], v[8], v[9], v[10]};
}
extern "C" double time_of(const int* v, int own) { return gqa::share_time(work(v), own); }
extern "C" int choice(const int* v) {
  const gqa::ShareWork s = work(v);
  unsigned best = ~0u;
  for (int own = 1; own <= s.ctas - s.width; ++own) {
    const unsigned r = gqa::share_rank(gqa::share_time(s, own), own);
    best = r < best ? r : best;
  }
  return (int)(best & 255u);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("share")
    src, out = str(d / "share.cpp"), str(d / "share.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I" + CSRC, src, "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.time_of.restype = ctypes.c_double
    return lib


def work(B, P, Hkv, G, Tq, D, blocks_of, own_of, ctas=152):
    """The sizes of a call whose prefixes have blocks_of blocks of 128 keys and whose rows have own_of keys."""
    Rp, R = B // P * G * Tq, G * Tq
    nrt = -(-Rp // 256)
    width = max(w for w in range(1, min(nrt, 38) + 1) if nrt % w == 0 and 152 // w * w * 100 >= 94 * 152)
    runs = Hkv * (nrt // width)
    block = 8 if R <= 8 else 16
    tile = 16 if D == 128 else 32
    v = [ctas, width, runs, P, runs * P * blocks_of, nrt == 1 and Rp <= 128, Hkv * -(-R // block), B * -(-own_of // tile),
         B, 12 if block == 8 else 8, D]
    assert max(v) < 2 ** 31 and v[4] * width <= 2 ** 30
    return (ctypes.c_int * len(v))(*[int(x) for x in v])


def exact_time(v, own):
    """The estimate in whole numbers and 64 bits."""
    ctas, width, runs, P, blocks, split, heads, tiles, rows, warps, D = v
    byte = 1 / 41
    tile, block = (8192 * byte, 4 * 128 * D * byte) if split else (94, 1350)
    t_own = 6000 + max((tiles * tile + rows * (2000 / warps)) * heads / own, tiles * 1.25 * heads)
    teams = (ctas - own) // width
    most = -(-blocks // teams)
    whole = P == 1 and (teams % runs == 0 or runs % teams == 0)
    return max(t_own, (6000 if split else 10000) + most * block + (0 if whole else 5000 * (1 + most * runs * P // blocks)))


def sizes():
    r = random.Random(3)
    yield work(256, 1, 8, 8, 128, 128, 256, 1024)          # 20 ms at best: 128 new tokens of 256 rows over 32768 keys
    yield work(64, 1, 8, 4, 1, 128, 64, 520)
    yield work(256, 1, 8, 4, 1, 128, 256, 290)
    yield work(4096, 4096, 8, 64, 8, 64, 4000, 100)        # 2^15 runs, 2^27 blocks: their product passes 32 bits
    for _ in range(400):
        P = r.choice([1, 1, 2, 64, 1024])
        B, Hkv, G, Tq = P * r.choice([1, 3, 40, 256]), r.choice([1, 2, 8]), r.choice([1, 4, 8]), r.choice([1, 5, 64, 512])
        try:
            yield work(B, P, Hkv, G, Tq, r.choice([64, 128]), r.choice([1, 16, 300, 4096]), r.choice([1, 100, 5000]),
                       r.choice([152, 148]))
        except AssertionError:
            pass                                           # more than a call may have


def slack(v, own):
    """Between the estimate and exact_time: sums in 32 bits, and a piece more or less where their number is rounded."""
    ctas, width, runs, P, blocks = v[:5]
    pieces = -(-blocks // ((ctas - own) // width)) * runs * P
    return 2.0 ** -20 * exact_time(v, own) + (5000 * (1 + pieces // blocks * 2.0 ** -22) if pieces >= 1 << 24 else 0)


def test_the_choice_is_the_fastest_split_whatever_the_call_takes(lib):
    """The choice's estimated time is the least of all splits', but for the 2^-15 that the comparison leaves of a time: for
    calls of microseconds and of seconds."""
    slow = 0
    for v in sizes():
        times = {own: exact_time(v, own) for own in range(1, v[0] - v[1] + 1)}
        for own in (1, 7, max(times)):
            assert abs(lib.time_of(v, own) - times[own]) <= slack(v, own), (list(v), own)
        best, own = min(times, key=times.get), lib.choice(v)
        assert times[own] <= times[best] * (1 + 2.0 ** -14) + slack(v, own) + slack(v, best), (list(v), own, best)
        slow += times[best] > 1.6e7
    assert slow >= 20
