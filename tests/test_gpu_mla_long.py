"""moe_mla_decode where its work is cut into long lists of pieces, and over page sizes, against the formulas in 64 bits.

The tolerances are those of the decode's other tests: its roundings, a row at a time.
"""
import pytest
import torch

from tests.test_gpu_mla import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


LONG = {
    "one_sequence": dict(lens=[30000], H=3),
    "one_sequence_48_heads": dict(lens=[70001], H=40, latent=384, page=48),
    "one_sequence_pair": dict(lens=[26000], H=128, latent=256),
    "two_long_one_short": dict(lens=[12000, 1, 9000], H=16, latent=256, page=16),
    "two_groups": dict(lens=[20000, 64], H=100, latent=384),
    "lists_fill_the_grid": dict(lens=[3000 + 17 * i for i in range(40)], H=20),
    "short_lists_of_a_pair": dict(lens=[700 + 13 * i for i in range(40)], H=127),
    "short_lists_of_64_heads": dict(lens=[800 + 7 * i for i in range(130)], H=63, latent=256, page=32),
    "long_lists_fill_the_grid": dict(lens=[9000, 9001, 9002, 9003, 9004, 9005, 9006], H=128),
}


@pytest.mark.parametrize("name", list(LONG))
def test_long_lists(name):
    Setup(seed=11, **LONG[name]).run().check()


@pytest.mark.parametrize("H", [3, 40])
def test_long_lists_repeat_the_same_bytes(H):
    s = Setup([40000], H).run()
    out, lse = s.att.out.clone(), s.att.lse.clone()
    for _ in range(3):
        s.run()
        assert torch.equal(out, s.att.out) and torch.equal(lse, s.att.lse)


@pytest.mark.parametrize("page", [8, 16, 24, 32, 48, 64, 128, 160, 256])
@pytest.mark.parametrize("H,latent,rope", [(16, 128, 32), (64, 384, 64), (100, 256, 64), (128, 512, 8)])
def test_pages(page, H, latent, rope):
    # 2100 tokens: the page table is read several batches of boxes long, and ends inside a batch
    Setup([5, 2100, 333, page, 2 * page - 1], H, latent=latent, rope=rope, page=page, seed=page).run().check()
