"""Refusals of moe_few_forward, moe_mla_decode_tree and moe_pages_update, checked on the host.

Argument checks run before the device check, so on a host without a GPU a bad
argument gives MOE_ERR_INVALID_ARG and a good call gets as far as
MOE_ERR_UNSUPPORTED_ARCH; nothing is launched or dereferenced. On a GPU only
the bad calls are made.
"""
import ctypes

import pytest

from tests.test_ops_refusals import A, CFG, _accepted, _refused, m

FEW_CFG = dict(T=4, d=256, E=8, k=2, n_groups=2, topk_groups=1, I=128, n_shared=1)
FEW = dict(x=A, w_router=A, bias=A, wq=A, idx=A, w=A, y=A, ws=A)


def test_few_accepts():
    cfg = m.config(**FEW_CFG)
    _accepted(m.moe_few_forward, cfg, *FEW.values())
    _accepted(m.moe_few_forward, cfg, *{**FEW, "bias": A + 4, "idx": A + 4, "w": A + 4}.values())
    _accepted(m.moe_few_forward, m.config(**{**FEW_CFG, "T": 64}), *FEW.values())
    _accepted(m.moe_few_forward, m.config(**{**FEW_CFG, "T": 0}), *{**FEW, "x": 0, "idx": 0, "w": 0, "y": 0}.values())
    _accepted(m.moe_few_forward, m.config(**FEW_CFG, flags=m.MOE_FLAG_LAP_LAUNCHES | m.MOE_FLAG_WGRAD_PAIR), *FEW.values())


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(T=65), dict(d=0), dict(d=192), dict(I=64), dict(E=0), dict(E=513), dict(E=7), dict(k=0), dict(k=9), dict(k=5),
    dict(n_groups=0), dict(n_groups=8), dict(topk_groups=3), dict(n_shared=2), dict(flags=4), dict(flags=8),
    dict(E=512, k=1, d=1 << 22, n_groups=1), dict(E=512, k=1, I=1 << 22, n_groups=1)])
def test_few_config_refused(change):
    cfg = m.config(**{**FEW_CFG, **change})
    _refused(m.moe_few_workspace_size, cfg)
    _refused(m.moe_few_forward, cfg, *FEW.values())
    _refused(m.moe_few_status, cfg, A)


@pytest.mark.parametrize("change", [dict([(k, 0)]) for k in FEW] +
                         [dict([(k, A + 8)]) for k in ("x", "w_router", "wq", "y", "ws")] +
                         [dict([(k, A + 2)]) for k in ("bias", "idx", "w")])
def test_few_refuses(change):
    _refused(m.moe_few_forward, m.config(**FEW_CFG), *{**FEW, **change}.values())


def test_few_workspace():
    size = lambda **c: m.moe_few_workspace_size(m.config(**{**FEW_CFG, **c}))
    sizes = [size(T=t) for t in range(65)]
    assert sizes == sorted(sizes)                          # that of more tokens serves fewer too
    assert m._lib.moe_few_workspace_size(ctypes.byref(m.config(**FEW_CFG)), ctypes.POINTER(ctypes.c_size_t)()) == \
        m.MOE_ERR_INVALID_ARG


TREE = dict(drafts=4, q=A, sb=4 * 16 * 576, sh=576, cache=A, table=A, lens=A, counts=A, tree=A, out=A, lse=A, ws=A)


def test_tree_accepts():
    cfg = m.mla_config(**CFG)
    _accepted(m.moe_mla_decode_tree, cfg, *TREE.values())
    for k in ("counts", "tree", "lse"):
        _accepted(m.moe_mla_decode_tree, cfg, *{**TREE, k: 0}.values())
    for n in (1, 64):
        _accepted(m.moe_mla_decode_tree, cfg, *{**TREE, "drafts": n}.values())


@pytest.mark.parametrize("change", [
    dict(drafts=0), dict(drafts=-1), dict(drafts=65), dict(drafts=1 << 33), dict(q=0), dict(cache=0), dict(table=0), dict(lens=0),
    dict(out=0), dict(ws=0), dict(sh=575), dict(sh=580), dict(sh=568), dict(sb=4 * 16 * 576 + 4), dict(sb=0), dict(sh=1 << 38),
    dict(q=A + 8), dict(cache=A + 8), dict(out=A + 8), dict(ws=A + 8), dict(lse=A + 2), dict(table=A + 2), dict(lens=A + 2),
    dict(counts=A + 2), dict(tree=A + 4)])
def test_tree_refuses(change):
    _refused(m.moe_mla_decode_tree, m.mla_config(**CFG), *{**TREE, **change}.values())


def test_tree_counts_tiles_of_all_row_groups_in_32_bits():
    cfg = dict(CFG, heads=128, page_size=64, max_pages=1 << 20)
    _accepted(m.moe_mla_decode, m.mla_config(**{**cfg, "batch": 1 << 10}), A, 128 * 576, 576, A, A, A, A, A, A)
    _refused(m.moe_mla_decode_tree, m.mla_config(**{**cfg, "batch": 1 << 10}), *TREE.values())


PAGES = dict(batch=4, page=16, num=10, maxp=8, new=32, lens=A, target=A, table=A, free=A, count=A, lens_out=A, count_out=A, seq=A,
             pos=A, slot=A, starts=A, ws=A)


def test_pages_accepts():
    _accepted(m.moe_pages_update, *PAGES.values())
    _accepted(m.moe_pages_update, *{**PAGES, "batch": 8192, "page": 1}.values())
    _accepted(m.moe_pages_update, *{**PAGES, "batch": 0, "lens": 0, "target": 0, "table": 0, "lens_out": 0}.values())
    _accepted(m.moe_pages_update, *{**PAGES, "new": 0, "seq": 0, "pos": 0, "slot": 0}.values())


@pytest.mark.parametrize("change", [
    dict(batch=-1), dict(batch=8193), dict(page=0), dict(num=0), dict(maxp=0), dict(new=-1), dict(new=1 << 30), dict(num=1 << 30, page=1),
    dict(num=1 << 28), dict(maxp=1 << 28), dict(batch=1 << 32), dict(new=1 << 32)] +
    [dict([(k, 0)]) for k in list(PAGES)[5:]] + [dict([(k, A + 8)]) for k in ("seq", "pos", "slot", "ws")] +
    [dict([(k, A + 2)]) for k in ("lens", "target", "table", "free", "count", "lens_out", "count_out", "starts")])
def test_pages_refuses(change):
    _refused(m.moe_pages_update, *{**PAGES, **change}.values())


def test_pages_status_refuses():
    _refused(m.moe_pages_status, 0)
