"""The tcgen05 kernel of the shared-prefix decode over many tiles per CTA: both of its forms (two streams of key
tiles over up to 128 rows; blocks of 256 rows), each checked to be the one that the sizes reach.  Bounds of the
differences as in test_shared_decode.py."""
import ctypes
import subprocess

import numpy as np
import pytest

import tiled_attention_26_b200 as fa
from tiled_attention_26_b200 import build
from test_kv_cache import built  # noqa: F401
from test_shared_decode import CASES, WIDE, Case

gpu = pytest.mark.gpu

PROGRAM = """
#include "shared_rule.h"
extern "C" int through_split(int D, long long R, int Hkv, long long keys) {
  return fa::shared_through_split(D, R, Hkv, keys);
}
extern "C" int own_splits(int B, int Hq, int Hkv, long long own) { return fa::shared_own_splits(B, Hq, Hkv, own); }
extern "C" int prefix_splits(int D, int B, int Hq, int Hkv, long long keys, int own_splits, long long own) {
  return fa::shared_prefix_splits(D, B, Hq, Hkv, keys, own_splits, own);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan(B, Hq, Hkv, D, table keys, table's own keys, num_splits) -> the prefix's kernel and its splits."""
    d = tmp_path_factory.mktemp("rule")
    src, out = str(d / "rule.cpp"), str(d / "rule.so")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", out], check=True)
    L = ctypes.CDLL(out)
    I, Q = ctypes.c_int, ctypes.c_longlong
    L.through_split.argtypes = [I, Q, I, Q]
    L.own_splits.argtypes = [I, I, I, Q]
    L.prefix_splits.argtypes = [I, I, I, I, Q, I, Q]

    def of(B, Hq, Hkv, D, keys, own, num_splits=0):
        R = B * (Hq // Hkv)
        n = num_splits or L.own_splits(B, Hq, Hkv, own)
        kernel = "split" if L.through_split(D, R, Hkv, keys) else "streams" if R <= 128 else "blocks"
        return kernel, L.prefix_splits(D, B, Hq, Hkv, keys, n, own)
    return of


def plan_of(plan, c):
    """Kernel, and tiles of a CTA at least."""
    kernel, splits = plan(c.B, c.Hq, c.Hkv, c.D, len(c.pt) * c.P, c.bt.shape[1] * c.P)
    return kernel, -(-c.prefix // 128) // splits


def sizes(case):
    bits, B, Hq, Hkv, D, P, prefix, lens, splits = case
    up = lambda n: -(-n // P)  # noqa: E731
    return B, Hq, Hkv, D, (up(prefix) + 2) * P, max([up(n) for n in lens] + [1]) * P, splits


def test_other_tests_reach_every_kernel(plan):
    """The cases of test_shared_decode.py: CASES go through the split kernel but for one, WIDE through both forms of
    the tcgen05 kernel."""
    kernels = [plan(*sizes(c))[0] for c in CASES]
    assert kernels.count("split") == len(CASES) - 1
    kernels = [plan(*sizes(c))[0] for c in WIDE]
    assert kernels.count("streams") >= 5 and kernels.count("blocks") >= 5


def test_the_smoke_run_reaches_the_tcgen05_kernel(plan):
    assert plan(3, 2400, 60, 128, 256, 64)[0] == "streams"


def long_case(bits, D, rows, kind="normal", seed=1):
    """75 KV heads: a CTA each, which takes the whole prefix of 10 tiles."""
    return Case(bits, 2, 75 * rows, 75, D, 64, 10 * 128 - 37, [70, 3], kind=kind, seed=seed)


LONG = [(bits, D, rows) for rows in (20, 65) for bits in (8, 4) for D in (128, 64)]  # R = 40 and 130


@gpu
@pytest.mark.parametrize("kind", ["normal", "scales", "peaked"])
@pytest.mark.parametrize("bits,D,rows", LONG)
def test_many_tiles_of_one_cta(built, plan, bits, D, rows, kind):
    """Barriers through several phases, and maxima and value scales that rise tile by tile."""
    c = long_case(bits, D, rows, kind)
    kernel, tiles = plan_of(plan, c)
    assert kernel == ("streams" if rows == 20 else "blocks") and tiles >= 9
    c.check(*c.call())
    assert fa.fa_device_status() == 0


@gpu
@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("bits,D", [(8, 128), (8, 64), (4, 128)])
def test_nan_of_a_stream_of_vanishing_weight(built, plan, bits, D, tile, which):
    """Keys of one stream outweigh the other's by more than 2^126; a NaN scale in the light one still makes every row
    that reads it NaN, and no other."""
    import torch
    c = long_case(bits, D, 20, seed=5)
    kernel, tiles = plan_of(plan, c)
    assert kernel == "streams" and tiles == 10
    d = c.dev
    pages = torch.from_numpy(np.ascontiguousarray(c.pt[:20])).cuda().long().view(10, 2)  # of each tile
    d["ks"][pages[1 - tile::2].flatten()] *= 200
    o, lse = c.call()
    assert torch.isfinite(o).all()
    d[which][int(pages[6 + tile, 1]), 3, 9] = float("nan")
    o2, lse2 = c.call()
    assert torch.isnan(o2[:, 0, 60:80]).all()
    assert torch.isnan(lse2[:, 60:80]).all() if which == "ks" else torch.equal(lse2, lse)
    o2[:, 0, 60:80] = o[:, 0, 60:80]
    assert torch.equal(o2, o)
