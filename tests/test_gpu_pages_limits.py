"""moe_pages_update at the limits of its numbers, and with pages that are out of range."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_dsv3_gb300 as m
    return m


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page,lens", [(1, [2 ** 30] * 2), (1, [2 ** 30, 2 ** 30 - 1]), (16, [2 ** 28] * 8), (16, [2 ** 28] * 16)])
def test_sums_past_32_bits_are_refused(lib, page, lens):
    """Lengths that the table is wide enough for, whose sums are not numbers of 32 bits: refused, and nothing changes."""
    from moe_layer_dsv3_gb300.pages import PagePlan
    B, wide = len(lens), max(lens)
    plan = PagePlan(B, page, 10, wide // page, 32)
    table = torch.empty((B, wide // page), dtype=torch.int32, device="cuda")   # (its entries are not read)
    free, count = i32([9, 8, 7, 6, 5, 4, 3, 2, 1, 0]), i32([5])
    for have, want in (([0] * B, lens), (lens, [0] * B), (lens, lens[:-1] + [0]), ([0] * (B - 1) + lens[-1:], lens[:-1] + [0])):
        now, target = i32(have), i32(want)
        seq, pos, slot = plan.update(now, target, table, free, count)
        torch.cuda.synchronize()
        assert plan.status()[0] == lib.MOE_ERR_BOUNDS
        assert now.tolist() == have and count.tolist() == [5] and free.tolist() == [9, 8, 7, 6, 5, 4, 3, 2, 1, 0]
        assert pos.tolist() == [-1] * 32 and slot.tolist() == [-1] * 32 and seq.tolist() == [0] * 32
        assert plan.starts.tolist() == [0] * (B + 1)
    # a good step of the same sequences after that
    now = i32([0] * B)
    plan.update(now, i32([1] + [0] * (B - 1)), table, free, count)
    torch.cuda.synchronize()
    assert plan.status() == (0, 0) and count.tolist() == [4] and table[0, 0].item() == 5 and plan.slot[0].item() == 5 * page
