"""Refusals of the norm and latent-attention entry points, checked on the host.

Argument checks run before the device check, so on a host without a GPU a bad
argument gives MOE_ERR_INVALID_ARG and a good call gets as far as
MOE_ERR_UNSUPPORTED_ARCH; nothing is launched or dereferenced. On a GPU only
the bad calls are made.
"""
import ctypes

import pytest
import torch

m = pytest.importorskip("moe_layer_dsv3_gb300")

A = 1 << 20                     # a fake, aligned device address
HAS_GPU = torch.cuda.is_available()


def _rc(fn, *args):
    try:
        fn(*args)
        return m.MOE_OK
    except m.MoeError as e:
        return e.code


def _refused(fn, *args):
    assert _rc(fn, *args) == m.MOE_ERR_INVALID_ARG


def _accepted(fn, *args):
    if not HAS_GPU:
        assert _rc(fn, *args) == m.MOE_ERR_UNSUPPORTED_ARCH


NORM = dict(T=4, d=256, x=A, residual=A, gamma=A, eps=1e-6, h=A, y=A, rstd=A, codes=A, scales=A, scales_tiled=A)
NORM_BWD = dict(T=4, d=256, dy=A, dres=A, h=A, gamma=A, rstd=A, dx=A, dgamma=A, ws=A)


def test_norm_accepts():
    _accepted(m.moe_add_rmsnorm, *NORM.values())
    for k in ("residual", "h", "rstd", "scales", "scales_tiled"):
        _accepted(m.moe_add_rmsnorm, *{**NORM, k: 0}.values())
    _accepted(m.moe_add_rmsnorm, *{**NORM, "T": 0, "x": 0, "y": 0}.values())
    _accepted(m.moe_add_rmsnorm, *{**NORM, "d": 8, "codes": 0, "scales": 0, "scales_tiled": 0}.values())
    _accepted(m.moe_add_rmsnorm_backward, *NORM_BWD.values())
    _accepted(m.moe_add_rmsnorm_backward, *{**NORM_BWD, "dres": 0}.values())


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(d=0), dict(d=12), dict(d=16392), dict(eps=-1.0), dict(eps=float("nan")), dict(x=0), dict(gamma=0),
    dict(y=0), dict(x=A + 8), dict(residual=A + 8), dict(gamma=A + 8), dict(h=A + 8), dict(y=A + 8), dict(codes=A + 8),
    dict(rstd=A + 2), dict(codes=0), dict(scales=0, scales_tiled=0), dict(d=40, scales_tiled=0), dict(d=160)])
def test_norm_refuses(change):
    _refused(m.moe_add_rmsnorm, *{**NORM, **change}.values())


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(d=0), dict(d=20), dict(d=16392), dict(dy=0), dict(h=0), dict(gamma=0), dict(rstd=0), dict(dx=0),
    dict(dgamma=0), dict(ws=0), dict(dy=A + 8), dict(dres=A + 8), dict(h=A + 8), dict(dx=A + 8), dict(ws=A + 8),
    dict(dgamma=A + 2)])
def test_norm_backward_refuses(change):
    _refused(m.moe_add_rmsnorm_backward, *{**NORM_BWD, **change}.values())


def test_norm_workspace():
    assert m.moe_add_rmsnorm_backward_workspace(0, 64) == 0
    assert m.moe_add_rmsnorm_backward_workspace(1 << 20, 7168) >= 4 * 7168
    _refused(m.moe_add_rmsnorm_backward_workspace, 4, 12)
    assert m._lib.moe_add_rmsnorm_backward_workspace(4, 64, ctypes.POINTER(ctypes.c_size_t)()) == m.MOE_ERR_INVALID_ARG


CFG = dict(batch=4, heads=16, latent=512, rope=64, page_size=64, num_pages=10, max_pages=8, softmax_scale=0.1)
DECODE = dict(q=A, sb=16 * 576, sh=576, cache=A, table=A, lens=A, out=A, lse=A, ws=A)
APPEND = dict(n=4, kv=A, ld=576, gamma=A, eps=1e-6, cos_sin=A, max_pos=100, seq=A, pos=A, table=A, cache=A, ws=A)


@pytest.mark.parametrize("change", [
    dict(batch=-1), dict(heads=0), dict(heads=129), dict(latent=0), dict(latent=64), dict(latent=192), dict(latent=640),
    dict(rope=0), dict(rope=12), dict(rope=72), dict(page_size=0), dict(page_size=4), dict(page_size=20),
    dict(num_pages=0), dict(max_pages=0), dict(num_pages=1 << 25), dict(max_pages=1 << 25),
    dict(batch=1 << 20, max_pages=1 << 20), dict(softmax_scale=0.0), dict(softmax_scale=-1.0),
    dict(softmax_scale=float("nan")), dict(softmax_scale=float("inf"))])
def test_mla_config_refused(change):
    cfg = m.mla_config(**{**CFG, **change})
    _refused(m.moe_mla_workspace_size, cfg)
    _refused(m.moe_mla_decode, cfg, *DECODE.values())
    _refused(m.moe_mla_append, cfg, *APPEND.values())
    _refused(m.moe_mla_status, cfg, A)


def test_mla_accepts():
    cfg = m.mla_config(**CFG)
    assert m.moe_mla_workspace_size(cfg) > 0
    _accepted(m.moe_mla_decode, cfg, *DECODE.values())
    _accepted(m.moe_mla_decode, cfg, *{**DECODE, "lse": 0}.values())
    _accepted(m.moe_mla_append, cfg, *APPEND.values())
    _accepted(m.moe_mla_append, cfg, *{**APPEND, "gamma": 0, "cos_sin": 0, "max_pos": 0}.values())


@pytest.mark.parametrize("change", [
    dict(q=0), dict(cache=0), dict(table=0), dict(lens=0), dict(out=0), dict(ws=0), dict(sh=575), dict(sh=580),
    dict(sh=568), dict(sb=16 * 576 + 4), dict(sb=0), dict(sh=1 << 38), dict(q=A + 8), dict(cache=A + 8), dict(out=A + 8),
    dict(ws=A + 8), dict(lse=A + 2), dict(table=A + 2), dict(lens=A + 2)])
def test_mla_decode_refuses(change):
    _refused(m.moe_mla_decode, m.mla_config(**CFG), *{**DECODE, **change}.values())


@pytest.mark.parametrize("change", [
    dict(n=-1), dict(kv=0), dict(seq=0), dict(pos=0), dict(table=0), dict(cache=0), dict(ws=0), dict(ld=575),
    dict(ld=580), dict(ld=568), dict(eps=-1.0), dict(eps=float("nan")), dict(max_pos=0), dict(kv=A + 8),
    dict(gamma=A + 8), dict(cos_sin=A + 8), dict(cache=A + 8), dict(ws=A + 8), dict(seq=A + 2), dict(pos=A + 2),
    dict(table=A + 2)])
def test_mla_append_refuses(change):
    _refused(m.moe_mla_append, m.mla_config(**CFG), *{**APPEND, **change}.values())


def test_layer_flags():
    ok = m.config(256, 256, 8, 2, flags=m.MOE_FLAG_X_QUANTIZED)
    assert m.moe_workspace_size(ok) == m.moe_workspace_size(m.config(256, 256, 8, 2))
    _refused(m.moe_workspace_size, m.config(256, 256, 8, 2, flags=8))
