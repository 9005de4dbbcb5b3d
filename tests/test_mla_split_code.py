"""The latent decode's integer arithmetic itself (csrc/mla_split.h, compiled here for the host) against unbounded integers.

The kernels take tiles, workers, ranges, lists of pieces and pages from these functions. test_mla_split.py holds the
model of the split and its invariants; here the code has to agree with that model, up to the last totals that the
library accepts.
"""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from tests.test_mla_split import _split

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_layer_dsv3_gb300", "csrc")
CODE = """
#include "mla_split.h"
using namespace moe::mla;
extern "C" {
int tiles(int len, int tile) { return tiles_of(len, tile); }
int workers(int total, int W, int m) { return workers_of(total, W, m); }
int begin(int total, int w, int W) { return range_begin(total, w, W); }
int owner(int total, int t, int W) { return owner_of(total, t, W); }
void cut(int total, int W, int s0, int w, int* out) {
  const Cut c = cut_of(total, W, s0, w);
  out[0] = c.slot; out[1] = c.worker; out[2] = c.pieces;
}
int page(int size, unsigned tok) { const PageDiv d = page_div(size); return page_of(tok, d.mul, d.shift); }
}
"""
LAST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("split")
    (d / "split.cpp").write_text(CODE)
    so = str(d / "split.so")
    subprocess.run([gxx, "-std=c++17", "-O1", "-fwrapv", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-o", so,
                    str(d / "split.cpp")], check=True)
    return ctypes.CDLL(so)


def test_tiles(code):
    for tile in (64, 128):
        for n in (0, 1, tile - 1, tile, tile + 1, 2 ** 30, LAST - 64, LAST):
            assert code.tiles(n, tile) == -(-n // tile)


@pytest.mark.parametrize("min_tiles", [2, 3])
def test_workers_up_to_the_last_total(code, min_tiles):
    for total in list(range(0, 1000)) + [LAST - k for k in range(8)]:
        for W in (1, 76, 152, 160):
            assert code.workers(total, W, min_tiles) == max(1, min(W, -(-total // min_tiles))), (total, W)


def test_ranges_and_owners(code):
    r = random.Random(1)
    for _ in range(4000):
        W = r.randint(1, 160)
        total = r.choice([r.randrange(1, LAST + 1), r.randrange(W, 2000), W, LAST])
        w = r.randint(0, W)
        assert code.begin(total, w, W) == total * w // W
        t = r.choice([r.randrange(total), 0, total - 1])
        own = code.owner(total, t, W)
        assert total * own // W <= t < total * (own + 1) // W


@pytest.mark.parametrize("seed", range(40))
def test_split(code, seed):
    r = random.Random(100 + seed)
    tile, min_tiles = r.choice([(64, 3), (128, 2)])
    n = r.choice([1, 2, 7, 40, 300])
    lens = [r.choice([0, 1, tile, r.randint(1, 5000), r.randint(1, 100)]) for _ in range(n)]
    asked = r.choice([1, 2, 76, 152])
    tiles, pieces, entries = _split(lens, tile, asked, min_tiles)
    assert tiles == [code.tiles(k, tile) for k in lens]
    total = sum(tiles)
    W = code.workers(total, asked, min_tiles)
    assert W == len(pieces)
    out = (ctypes.c_int * 3)()
    for w, (mine, entry) in enumerate(zip(pieces, entries)):
        assert sum(k for _, _, k in mine) == code.begin(total, w + 1, W) - code.begin(total, w, W)
        if entry:
            code.cut(total, W, code.begin(total, w, W) - mine[0][1], w, out)
            assert tuple(out) == entry[1:]


def test_page_of_a_token(code):
    r = random.Random(2)
    pages = list(range(8, 1025, 8)) + [2 ** k + d for k in range(5, 31) for d in (-8, 0, 8)] + [2 ** 31 - 8]
    for page in pages:
        some = [r.randrange(2 ** 31 // page + 1) * page + d for d in (-1, 0, 1) for _ in range(8)]
        for tok in [0, 1, page - 1, page, LAST] + [t for t in some if 0 <= t <= LAST]:
            assert code.page(page, tok) == tok // page, (page, tok)


def test_the_kernels_use_this_code():
    text = "".join(open(os.path.join(CSRC, f)).read() for f in ("mla.cuh", "k_mla.cu", "k_mla_pair.cu"))
    for name in ("workers_of(", "range_begin(", "cut_of(", "page_of(", "page_div(", "tiles_of(len, TILE)"):
        assert name in text, name
    for name in ("workers_of", "range_begin", "owner_of", "cut_of", "page_of", "page_div"):
        assert "int %s(" % name not in text
