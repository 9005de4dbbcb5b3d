"""moe_few_forward behind a router of 256 and 384 experts over 7168 columns, in each of its forms, against the formulas in 64 bits."""
import pytest
import torch

from tests.test_gpu_few import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


@pytest.mark.parametrize("T,E,G,kept,S", [
    (1, 256, 8, 4, 1), (2, 256, 8, 4, 1), (3, 256, 8, 4, 1), (16, 256, 8, 4, 1), (64, 256, 8, 4, 1), (1, 384, 1, 1, 1), (5, 384, 1, 1, 1),
    (64, 384, 12, 6, 0)])
def test_wide_router(lib, T, E, G, kept, S):
    Case(T, 7168, E, 8, G, kept, 128, S, seed=50 + T + E, xgain=0.25, bias=0.1).check()


def test_many_experts_in_use(lib):
    """64 tokens without groups: most of 256 experts, each with a few tokens."""
    c = Case(64, 2048, 256, 8, 1, 1, 256, 1, seed=51, xgain=0.25, bias=0.02)
    c.check()
    assert c.few.topk_idx.unique().numel() > 180
