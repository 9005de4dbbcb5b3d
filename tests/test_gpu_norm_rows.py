"""moe_add_rmsnorm_backward where every row group walks its ring of stages more than once around.

Rows wait in a ring of 4 stages (2 for 513 to 1024 columns and beyond 8192). Each shape below gives every form of
the kernel (a warp a row up to 256, 512 and 1024 columns, a block a row up to 8192 and beyond) at least as many rows
a group as its stages and two more, with a number of rows that does not divide. The tolerances are those of the
gradient's other tests: the chains of dgamma are rows a group, warps a block, partial rows a thread, 5 shuffles, less
than 160 additions here too.
"""
import pytest
import torch

from tests.helpers import np_f64
from tests.test_gpu_norm import EPS, U, _backward64, _inputs, _within

pytestmark = pytest.mark.gpu

# a group per warp (16 a block) up to 1024 columns, per block beyond; 152 SMs, 1 to 4 blocks each
ROWS = [(30001, 64), (29999, 256), (15001, 264), (15001, 512), (10001, 520), (10001, 1024), (4001, 1032), (3701, 2048),
        (1001, 8192), (701, 8200), (701, 16384)]


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


@pytest.mark.parametrize("T,d", ROWS)
@pytest.mark.parametrize("residual", [True, False])
def test_many_rows_a_group(lib, T, d, residual):
    from moe_layer_dsv3_gb300.norm import AddRMSNorm
    x, res, gamma, dy, dres = _inputs(T, d, T + 3 * d)
    dres = dres if residual else None
    n = AddRMSNorm(T, d, eps=EPS)
    n.forward(x, gamma, res)
    n.backward(dy, gamma, dres)
    torch.cuda.synchronize()
    dx, size, dg, dg_size = _backward64(dy, n.h, gamma, n.rstd, dres)
    _within(np_f64(n.dx), dx, U * (1 + 2.0 ** -6) * abs(dx) + 4e-6 * size, "dx")
    _within(np_f64(n.dgamma), dg, 1e-5 * dg_size + 1e-30, "dgamma")


@pytest.mark.parametrize("T,d", [(30001, 200), (15001, 512), (10001, 1024), (4001, 1032), (701, 8200)])
def test_in_place_and_repeated(lib, T, d):
    """dx over dy, dres or h gives the bytes of a call with a buffer of its own, whichever the form."""
    from moe_layer_dsv3_gb300.norm import AddRMSNorm
    x, res, gamma, dy, dres = _inputs(T, d, 5)
    n = AddRMSNorm(T, d, eps=EPS)
    n.forward(x, gamma, res)
    torch.cuda.synchronize()
    runs = []
    for over in (None, None, "dy", "dres", "h"):
        src = dict(dy=dy, dres=dres, h=n.h)
        if over is None:
            dx = torch.empty_like(dy)
        else:
            dx = src[over] = src[over].clone()
        dg = torch.empty(d, dtype=torch.float32, device="cuda")
        lib.moe_add_rmsnorm_backward(T, d, src["dy"].data_ptr(), src["dres"].data_ptr(), src["h"].data_ptr(),
                                     gamma.data_ptr(), n.rstd.data_ptr(), dx.data_ptr(), dg.data_ptr(), n.ws.data_ptr())
        torch.cuda.synchronize()
        runs.append((dx, dg))
    for dx, dg in runs[1:]:
        assert torch.equal(dx, runs[0][0]) and torch.equal(dg, runs[0][1])
