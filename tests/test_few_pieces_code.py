"""The few-token layer's list of pieces itself (csrc/few_pieces.h, compiled here for the host) against the model of test_few_pieces.py,
and the parts that the code makes against the room that the library gives them."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from tests import test_few_pieces as model

m = model.m
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_layer_dsv3_gb300", "csrc")
CODE = """
#include "few_pieces.h"
using namespace moe::few;
struct Args { int d, I; };
struct Plan { int slots; };
static Work list_of(int d, int I, int slots, int ctas) {
  Work w;
  work_of(w, Args{d, I}, Plan{slots}, ctas);
  return w;
}
extern "C" {
int consts(int i) { const int c[] = {kUpPieces, kDownPieces, kMinSteps}; return c[i]; }
void work(int d, int I, int slots, int ctas, int* out) {
  const Work w = list_of(d, I, slots, ctas);
  const int c[] = {w.KA, w.KI, w.NB, w.RP, w.PU, w.PD, w.nup, w.total};
  for (int i = 0; i < 8; ++i) out[i] = c[i];
}
void pieces(int d, int I, int slots, int ctas, int from, int n, int* out) {
  const Work w = list_of(d, I, slots, ctas);
  for (int i = 0; i < n; ++i) {
    const Piece p = piece_of(w, from + i);
    const int c[] = {p.up, p.s, p.b, p.part, p.k0, p.k1};
    for (int k = 0; k < 6; ++k) out[6 * i + k] = c[k];
  }
}
int slots_of(int N) { return acc_slots(N); }
int chunks(int up, int k0, int k1, int N, int* at) {
  const Piece p{up != 0, 0, 0, 0, k0, k1};
  const int n = chunks_of(p, N);
  for (int i = 0; i <= n; ++i) at[i] = chunk_at(p, i, n);
  return n;
}
long long room(long long T, long long picks, long long ctas, long long steps, long long blocks, long long want) {
  return parts_room(T, picks, ctas, steps, blocks, want);
}
}
"""


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("pieces")
    (d / "pieces.cpp").write_text(CODE)
    so = str(d / "pieces.so")
    subprocess.run([gxx, "-std=c++17", "-O1", "-fwrapv", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-o", so,
                    str(d / "pieces.cpp")], check=True)
    lib = ctypes.CDLL(so)
    lib.room.argtypes, lib.room.restype = [ctypes.c_longlong] * 6, ctypes.c_longlong
    return lib


def work(code, d, inner, slots, ctas):
    out = (ctypes.c_int * 8)()
    code.work(d, inner, slots, ctas, out)
    return dict(zip(("KA", "KI", "NB", "RP", "PU", "PD", "nup", "total"), out))


def test_constants(code):
    assert [code.consts(i) for i in range(3)] == [model.UP, model.DOWN, model.MIN_STEPS]


@pytest.mark.parametrize("seed", range(8))
def test_pieces_as_in_the_model(code, seed):
    r = random.Random(seed)
    for _ in range(12):
        slots, d, inner = r.choice([1, 2, 9, 38, 65, 513]), 128 * r.randint(1, 60), 128 * r.randint(1, 32)
        if slots * (d // 128) * (inner // 128) > 60000:
            slots = 2
        ctas = r.choice([1, 7, 148, 152, 160])
        want = list(model.pieces(slots, d, inner, ctas))
        n = work(code, d, inner, slots, ctas)["total"]
        assert n == len(want)
        out = (ctypes.c_int * (6 * n))()
        code.pieces(d, inner, slots, ctas, 0, n, out)
        got = [("up" if out[6 * i] else "down",) + tuple(out[6 * i + 1:6 * i + 6]) for i in range(n)]
        assert got == want


def test_ends_of_the_range(code):
    """The largest layers that the library takes: as many pieces as 32 bits hold, and the longest reductions that fit a GPU."""
    for slots, d, inner in ((513, 128 * 1000, 128 * 1000), (1, 128 * (1 << 17), 128), (1, 128, 128 * (1 << 17)), (2, 128 * 60000, 128 * 3)):
        for ctas in (1, 152, 160):
            w = work(code, d, inner, slots, ctas)
            KA, KI = d // 128, inner // 128
            pu, pd = model.parts_of(slots * KI, KA, ctas, model.UP), model.parts_of(slots * ((KA + 1) // 2), KI, ctas, model.DOWN)
            assert (w["PU"], w["PD"]) == (pu, pd)
            assert (w["nup"], w["total"]) == (slots * KI * pu, slots * KI * pu + slots * ((KA + 1) // 2) * pd) and w["total"] < 2 ** 31
            out = (ctypes.c_int * 6)()
            for first, parts, steps in ((0, pu, KA), (w["nup"], pd, KI)):
                end = 0
                for i in range(parts):
                    code.pieces(d, inner, slots, ctas, first + i, 1, out)
                    assert out[0] == (first == 0) and list(out)[1:4] == [0, 0, i] and out[4] == end < out[5]
                    end = out[5]
                assert end == steps
            code.pieces(d, inner, slots, ctas, w["total"] - 1, 1, out)
            assert list(out)[:4] == [0, slots - 1, (KA + 1) // 2 - 1, pd - 1] and out[5] == KI


def test_chunks_of_a_piece(code):
    """A piece's chunks are its steps in order, none empty, and leave an accumulator for the next piece's first one."""
    at = (ctypes.c_int * 8)()
    for N in (16, 32, 48, 64):
        slots = code.slots_of(N)
        assert slots * 2 * N <= 512 - 72 and slots <= 32    # (scales of six stages lie behind them; parities are bits)
        for k0 in (0, 2, 28):
            for steps in list(range(1, 60)) + [1000, 1 << 17]:
                n = code.chunks(1, k0, k0 + steps, N, at)
                assert 1 <= n <= min(4, slots - 1)
                cuts = list(at)[:n + 1]
                assert cuts[0] == k0 and cuts[-1] == k0 + steps and all(a < b for a, b in zip(cuts, cuts[1:]))
                assert n == 1 or min(b - a for a, b in zip(cuts, cuts[1:])) >= 14
                assert code.chunks(0, k0, k0 + steps, N, at) == 1 and list(at)[:2] == [k0, k0 + steps]
        assert code.chunks(1, 0, 56, N, at) == min(4, slots - 1)


def test_the_code_s_parts_fit(code):
    """With every number of experts in use and of CTAs, the parts that work_of makes fit the room, and that room is in the workspace."""
    r = random.Random(3)
    for _ in range(400):
        T, k, S = r.randint(1, 64), r.randint(1, 8), r.randint(0, 1)
        E = r.choice([k, r.randint(k, 40), r.randint(k, 512), 512])
        d, inner = 128 * r.choice([1, 2, 3, 7, 16, 56, 112]), 128 * r.choice([1, 2, 5, 6, 16, 31])
        gu = code.room(T, k + S, model.MAX_SMS, d // 128, inner // 128, code.consts(0))
        o = code.room(T, k + S, model.MAX_SMS, inner // 128, (d // 128 + 1) // 2, code.consts(1))
        total, gu_, o_ = model._room(T, d, E, k, inner, S)
        assert (gu, o) == (gu_, o_) and m.moe_few_workspace_size(m.config(T, d, E, k, 1, 1, inner, S)) == total
        most = min(T * k, E) + S
        for slots in range(1, most + 1):
            rows = min(T * (k + S), slots * T)
            for ctas in (model.MAX_SMS, 152, 1):
                w = work(code, d, inner, slots, ctas)
                assert (w["PU"] == 1 or rows * w["PU"] <= gu) and rows * w["PD"] <= o
                assert 2 + slots + slots * w["NB"] <= 2 + most + most * (inner // 128)


def test_the_kernel_uses_this_code():
    text = open(os.path.join(CSRC, "k_few.cu")).read()
    for name in ("few::work_of(", "few::piece_of(", "few::parts_room(", "few::kUpPieces", "few::kDownPieces"):
        assert name in text, name
    for name in ("parts_of(int", "cut_at(int", "struct Work", "struct Piece "):
        assert name not in text, name
