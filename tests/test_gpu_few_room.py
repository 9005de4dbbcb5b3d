"""moe_few_forward writes nothing behind its workspace, at choices that fill the room for parts."""
import pytest
import torch

from tests.test_gpu_few import Case

pytestmark = pytest.mark.gpu

TAIL = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


# Few experts in use: both reductions in as many parts as they have, or as the room is made for
@pytest.mark.parametrize("T,d,E,k,I,S", [
    (64, 1024, 8, 1, 2048, 0), (64, 512, 8, 1, 512, 1), (33, 2048, 4, 2, 1024, 0), (1, 4096, 16, 8, 512, 1), (7, 128, 2, 1, 4096, 0),
    (64, 4096, 3, 1, 128, 1), (16, 384, 64, 8, 640, 1)])
def test_nothing_behind_the_workspace(lib, T, d, E, k, I, S):
    for same in (True, False):
        c = Case(T, d, E, k, 1, 1, I, S, seed=40 + T, same=same)
        n = c.few.ws.numel()
        buf = torch.zeros(n + TAIL, dtype=torch.uint8, device="cuda")
        tail = torch.arange(TAIL, device="cuda").remainder(251).to(torch.uint8)
        buf[n:] = tail
        c.few.ws = buf[:n]
        c.check()
        assert torch.equal(buf[n:], tail)
