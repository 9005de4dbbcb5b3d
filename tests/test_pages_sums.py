"""The page plan's sums and verdict (csrc/pages_sums.h, compiled here for the host) against unbounded integers.

Lengths may be anything that the table is wide enough for, so sums over sequences pass 2^31 and 2^32. A step is made
only if its true sums allow it, and the sums are then exact, in whatever order they are added.
"""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

m = pytest.importorskip("moe_layer_dsv3_gb300")

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_layer_dsv3_gb300", "csrc")
CODE = """
#include "pages_sums.h"
using namespace moe::pages;
extern "C" int step(int n, const int* len, const int* want, int page, int count, int num_pages, int max_new, int group, unsigned* out) {
  Sums all{0, 0, 0};
  for (int b = 0; b < n; b += group) {     // sums of groups are added, as those of threads and warps are
    Sums part{0, 0, 0};
    for (int i = b; i < n && i < b + group; ++i) part += sums_of(len[i], want[i], page);
    all += part;
  }
  out[0] = all.add; out[1] = all.grow; out[2] = all.drop;
  return step_code(all, count, num_pages, max_new);
}
"""
MOST = 2 ** 30


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("pages")
    (d / "sums.cpp").write_text(CODE)
    so = str(d / "sums.so")
    subprocess.run([gxx, "-std=c++17", "-O1", "-fwrapv", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-o", so,
                    str(d / "sums.cpp")], check=True)
    return ctypes.CDLL(so)


def check(code, lens, want, page, count, num_pages, max_new):
    pages = lambda n: -(-n // page)
    add = sum(max(b - a, 0) for a, b in zip(lens, want))
    grow = sum(max(pages(b) - pages(a), 0) for a, b in zip(lens, want))
    drop = sum(max(pages(a) - pages(b), 0) for a, b in zip(lens, want))
    expect = m.MOE_OK
    if add > max_new or drop > num_pages - count:
        expect = m.MOE_ERR_BOUNDS
    elif grow > count + drop:
        expect = m.MOE_ERR_PAGES
    arr = ctypes.c_int * len(lens)
    out = (ctypes.c_uint * 3)()
    for group in (1, 2, 3, 32, len(lens)):
        got = code.step(len(lens), arr(*lens), arr(*want), page, count, num_pages, max_new, group, out)
        assert got == expect, (lens, want, page, group, list(out))
        assert list(out) == [min(v, MOST) for v in (add, grow, drop)]
    return expect


def test_sums_past_32_bits(code):
    """Sums that are negative, zero or small if they are kept in 32 bits."""
    last = 2 ** 31 - 3
    for n in (2, 3, 4, 5, 8, 64, 8192):
        for top in (MOST, MOST - 1, MOST + 1, last, 2 ** 31 // n, 2 ** 32 // n if n > 2 else last):
            for page in (1, 2, 8, 64):
                top = min(top, last - page)
                zero, big = [0] * n, [top] * n
                for count in (0, 5, 10):
                    assert check(code, zero, big, page, count, 10, 32) != m.MOE_OK
                    assert check(code, big, zero, page, count, 10, 32) == m.MOE_ERR_BOUNDS
                check(code, zero, big, page, MOST - 1, MOST - 1, MOST - 1)
                check(code, big, zero, page, 0, MOST - 1, 0)


def test_the_largest_steps(code):
    """At, and one past, the most pages and new tokens that the library takes."""
    for n in (1, 2, 7):
        each = (MOST - 1) // n
        want = [each] * (n - 1) + [MOST - 1 - each * (n - 1)]
        zero = [0] * n
        assert check(code, zero, want, 1, MOST - 1, MOST - 1, MOST - 1) == m.MOE_OK
        assert check(code, zero, want, 1, MOST - 2, MOST - 1, MOST - 1) == m.MOE_ERR_PAGES
        assert check(code, zero, want, 1, MOST - 1, MOST - 1, MOST - 2) == m.MOE_ERR_BOUNDS
        assert check(code, want, zero, 1, 0, MOST - 1, 0) == m.MOE_OK
        assert check(code, want, zero, 1, 1, MOST - 1, 0) == m.MOE_ERR_BOUNDS
        more = want[:-1] + [want[-1] + 1]
        assert check(code, zero, more, 1, MOST - 1, MOST - 1, MOST - 1) == m.MOE_ERR_BOUNDS


@pytest.mark.parametrize("seed", range(20))
def test_random_steps(code, seed):
    r = random.Random(seed)
    made = 0
    for _ in range(200):
        n, page = r.choice([1, 2, 5, 40, 300]), r.choice([1, 7, 16, 64, 1 << 20])
        top = r.choice([1, 100, 5000, 2 ** 24, MOST, 2 ** 31 - 2 - page])
        lens, want = ([r.choice([0, top, r.randint(0, top)]) for _ in range(n)] for _ in range(2))
        num = r.choice([1, 10, 1000, 2 ** 20, MOST - 1])
        made += check(code, lens, want, page, r.choice([0, num, r.randint(0, num)]), num, r.choice([0, 32, 2 ** 20, MOST - 1])) == m.MOE_OK
    assert made


def test_the_kernel_uses_this_code():
    text = open(os.path.join(CSRC, "k_pages.cu")).read()
    for name in ("pages::sums_of(", "pages::step_code(", "pages::pages_of("):
        assert name in text, name
    assert "struct Sums" not in text
