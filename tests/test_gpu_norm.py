"""moe_add_rmsnorm and its gradient against the formulas in 64 bits.

Tolerances. h, y and dx are rounded to bf16 once (relative 2^-8 at most); the
fp32 arithmetic before adds less than 2^-14 of that rounding except where terms
cancel, so those get 4e-6 (under 64 fp32 roundings) of the terms' size. rstd: a
chain of at most 44 fp32 operations on positive terms, halved by the root, plus
the root's own 2 ulp: 2e-6. dgamma: chains of at most 160 fp32 additions, 1e-5
of the terms' absolute sum. Codes and scales are the bytes of the MX oracle on
the bf16 y.
"""
import numpy as np
import pytest
import torch

import gen
from oracle import mxfp8
from tests.helpers import np_f64, np_u8, tile_scales

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
EPS = 1e-5


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


def _inputs(T, d, seed, residual=True, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    chan = 1.0 + 30.0 * (torch.rand(d, generator=g, device="cuda") < 0.02).float()
    x = (r(T, d) * scale).to(torch.bfloat16)
    res = (r(T, d) * chan * scale).to(torch.bfloat16) if residual else None
    gamma = (1.0 + 0.3 * r(d)).to(torch.bfloat16)
    return x, res, gamma, r(T, d).to(torch.bfloat16), r(T, d).to(torch.bfloat16)


def _within(got, want, tol, what):
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its tolerance" % (
        what, bad.sum(), bad.size, np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))


def _forward64(x, res, gamma, eps=EPS):
    h = np_f64(x) + (np_f64(res) if res is not None else 0.0)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * np_f64(gamma)


SHAPES = [(1, 8), (3, 24), (5, 32), (2, 256), (33, 264), (9, 512), (7, 520), (130, 1024), (17, 1032), (1, 2016),
          (300, 2048), (5, 4104), (1, 7168), (1000, 7168), (3, 16384)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward(lib, T, d, residual):
    from moe_layer_dsv3_gb300.norm import AddRMSNorm
    x, res, gamma, _, _ = _inputs(T, d, T + d, residual)
    mx = d % 32 == 0
    n = AddRMSNorm(T, d, eps=EPS, mx=mx)
    n.forward(x, gamma, res)
    torch.cuda.synchronize()
    h, rstd, y = _forward64(x, res, gamma)
    _within(np_f64(n.rstd), rstd, 2e-6 * rstd, "rstd")
    _within(np_f64(n.y), y, U * (1 + 2.0 ** -6) * np.abs(y) + 1e-30, "y")
    if residual:
        _within(np_f64(n.h), h, U * (1 + 2.0 ** -6) * np.abs(h), "h")
    if mx:
        codes, scales = mxfp8.quantize(np_f64(n.y))
        assert np.array_equal(np_u8(n.codes), codes) and np.array_equal(np_u8(n.scales), scales)


@pytest.mark.parametrize("T,d", [(1, 128), (127, 256), (128, 1024), (129, 1152), (200, 2048)])
def test_tiled_scales_and_padding_rows(lib, T, d):
    x, res, gamma, _, _ = _inputs(T, d, 7)
    Tp = (T + 127) // 128 * 128
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((Tp, d), 0xAB, dtype=torch.uint8, device="cuda")
    tiled = torch.full((Tp * d // 32,), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((T + 1, d // 32), 0xAB, dtype=torch.uint8, device="cuda")
    lib.moe_add_rmsnorm(T, d, x.data_ptr(), res.data_ptr(), gamma.data_ptr(), EPS, 0, y.data_ptr(), 0, codes.data_ptr(),
                        scales.data_ptr(), tiled.data_ptr())
    torch.cuda.synchronize()
    want_c, want_s = mxfp8.quantize(np_f64(y))
    pad = lambda a: np.concatenate([a, np.zeros((Tp - T, a.shape[1]), np.uint8)])
    assert np.array_equal(np_u8(codes), pad(want_c))
    assert np.array_equal(np_u8(tiled), tile_scales(pad(want_s), Tp, d))
    assert np.array_equal(np_u8(scales)[:T], want_s) and (np_u8(scales)[T] == 0xAB).all()


def test_in_place_sum_and_side_stream(lib):
    """h over the residual's own buffer, on a stream other than the default one."""
    T, d = 65, 1536
    x, res, gamma, _, _ = _inputs(T, d, 3)
    h, rstd, y = _forward64(x, res, gamma)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(x)
    lib.moe_add_rmsnorm(T, d, x.data_ptr(), res.data_ptr(), gamma.data_ptr(), EPS, res.data_ptr(), out.data_ptr(),
                        stream=s.cuda_stream)
    s.synchronize()
    _within(np_f64(res), h, U * (1 + 2.0 ** -6) * np.abs(h), "h")
    _within(np_f64(out), y, U * (1 + 2.0 ** -6) * np.abs(y), "y")


def test_zero_rows_and_special_values(lib):
    """A zero row gives zeros (eps > 0); NaN and inf stay in their own row."""
    from moe_layer_dsv3_gb300.norm import AddRMSNorm
    T, d = 6, 1280
    x, _, gamma, _, _ = _inputs(T, d, 4, residual=False)
    x[1] = 0
    x[3, 17] = float("nan")
    x[4, 5] = float("inf")
    n = AddRMSNorm(T, d, eps=EPS, mx=True)
    n.forward(x, gamma)
    torch.cuda.synchronize()
    assert not n.y[1].any() and not n.codes[1].any() and not n.scales[1].any()
    assert torch.isnan(n.y[3]).all()
    assert torch.isnan(n.y[4, 5]) and not n.y[4, 6:].any()
    keep = [0, 2, 5]
    _, _, y = _forward64(x[keep], None, gamma)
    _within(np_f64(n.y[keep]), y, U * (1 + 2.0 ** -6) * np.abs(y), "y")


def _backward64(dy, h, gamma, rstd, dres):
    dy, h, gamma, rstd = map(np_f64, (dy, h, gamma, rstd))
    xhat = h * rstd[:, None]
    g = dy * gamma
    dot = (g * xhat).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - xhat * dot)
    size = rstd[:, None] * (np.abs(g) + np.abs(xhat) * np.abs(g * xhat).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + np_f64(dres)
        size = size + np.abs(np_f64(dres))
    return dx, size, (dy * xhat).sum(0), np.abs(dy * xhat).sum(0)


@pytest.mark.parametrize("T,d", SHAPES + [(2500, 1024), (5000, 64)])
@pytest.mark.parametrize("residual", [True, False])
def test_backward(lib, T, d, residual):
    from moe_layer_dsv3_gb300.norm import AddRMSNorm
    x, res, gamma, dy, dres = _inputs(T, d, 2 * T + d)
    dres = dres if residual else None
    n = AddRMSNorm(T, d, eps=EPS)
    n.forward(x, gamma, res)
    n.backward(dy, gamma, dres)
    torch.cuda.synchronize()
    dx, size, dg, dg_size = _backward64(dy, n.h, gamma, n.rstd, dres)
    _within(np_f64(n.dx), dx, U * (1 + 2.0 ** -6) * np.abs(dx) + 4e-6 * size, "dx")
    _within(np_f64(n.dgamma), dg, 1e-5 * dg_size + 1e-30, "dgamma")


def test_backward_against_differences(lib):
    """dx and dgamma against central differences of the 64-bit forward along random directions."""
    from moe_layer_dsv3_gb300.norm import AddRMSNorm
    T, d = 12, 768
    x, res, gamma, dy, _ = _inputs(T, d, 11)
    n = AddRMSNorm(T, d, eps=EPS)
    n.forward(x, gamma, res)
    # the gradient's function: the norm of the saved (rounded) h, whose own statistics go with it
    n.backward(dy, gamma, rstd=(n.h.double().square().mean(1) + EPS).rsqrt().float())
    torch.cuda.synchronize()
    h, g, w = np_f64(n.h), np_f64(gamma), np_f64(dy)
    f = lambda h, g: float((h / np.sqrt((h * h).mean(1, keepdims=True) + EPS) * g * w).sum())
    rng = np.random.default_rng(0)
    step = 1e-5
    for _ in range(4):
        v, u = rng.standard_normal(h.shape), rng.standard_normal(g.shape)
        num = (f(h + step * v, g) - f(h - step * v, g)) / (2 * step)
        mine = float((np_f64(n.dx) * v).sum())
        # each dx carries a rounding of 2^-8 at most, independent in sign of v
        assert abs(num - mine) <= 6 * U * np.linalg.norm(np_f64(n.dx) * v) + 1e-6 * abs(num)
        num = (f(h, g + step * u) - f(h, g - step * u)) / (2 * step)
        mine = float((np_f64(n.dgamma) * u).sum())
        assert abs(num - mine) <= 1e-5 * float((np.abs(w * h / np.sqrt((h * h).mean(1, keepdims=True) + EPS)).sum(0)
                                               * np.abs(u)).sum())


def test_backward_in_place_is_deterministic(lib):
    T, d = 700, 3584
    x, res, gamma, dy, dres = _inputs(T, d, 5)
    from moe_layer_dsv3_gb300.norm import AddRMSNorm
    n = AddRMSNorm(T, d, eps=EPS)
    n.forward(x, gamma, res)
    runs = []
    for buf in (torch.empty_like(dy), dy.clone(), dres.clone(), n.h.clone()):
        src = dict(dy=dy, dres=dres, h=n.h)
        for k, v in src.items():               # dx may be any of its inputs' buffers
            if torch.equal(buf, v):
                src[k] = buf
        dg = torch.empty(d, dtype=torch.float32, device="cuda")
        lib.moe_add_rmsnorm_backward(T, d, src["dy"].data_ptr(), src["dres"].data_ptr(), src["h"].data_ptr(),
                                     gamma.data_ptr(), n.rstd.data_ptr(), buf.data_ptr(), dg.data_ptr(), n.ws.data_ptr())
        torch.cuda.synchronize()
        runs.append((buf, dg))
    for buf, dg in runs[1:]:
        assert torch.equal(buf, runs[0][0]) and torch.equal(dg, runs[0][1])


def test_no_tokens(lib):
    d = 256
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    dg = torch.full((d,), 7.0, device="cuda")
    lib.moe_add_rmsnorm(0, d, 0, 0, gamma.data_ptr(), EPS, 0, 0)
    lib.moe_add_rmsnorm_backward(0, d, 0, 0, 0, gamma.data_ptr(), 0, 0, dg.data_ptr(), 0)
    torch.cuda.synchronize()
    assert not dg.any()


@pytest.mark.parametrize("T", [300, 512])
def test_layer_reads_the_norms_codes(lib, T):
    """The layer with MOE_FLAG_X_QUANTIZED on the norm's codes gives the bytes of the layer on the bf16 rows."""
    from moe_layer_dsv3_gb300.layer import MoELayer
    from moe_layer_dsv3_gb300.norm import AddRMSNorm
    shape = gen.make_shape("normed", T, 256, 8, 2, 2, 1, 128, 1, "normal0.1", 0.05, C=128)
    inp = gen.make_inputs(shape, seed=3, device="cuda")
    x, res, gamma, _, _ = _inputs(shape.T, shape.d, 9)
    got = []
    for flags in (0, lib.MOE_FLAG_X_QUANTIZED):
        L = MoELayer.from_shape(shape, flags=flags)
        L.quantize_weights(inp["w_gu"], inp["w_d"], inp["ws_gu"], inp["ws_d"])
        n = AddRMSNorm(shape.T, shape.d, eps=EPS)
        y = n.forward(x, gamma, res, layer=L if flags else None)
        L.forward(y, inp["w_router"], inp["bias"])
        L.backward(inp["dy"])
        n.backward(L.dx, gamma)
        L.dispatch(y)
        torch.cuda.synchronize()
        L.check_status()
        got.append([t.clone() for t in (L.y, L.dx, L.dw_router, L.dw_gu, L.dw_d, L.dws_gu, n.dx, n.dgamma,
                                        L.ws_tensor("RING_X"), L.ws_tensor("XQ"), L.ws_tensor("XQ_SF"))])
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
