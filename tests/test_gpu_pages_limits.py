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


def test_bad_pages_stay_and_are_told_again(lib):
    """A page out of range moves as it is, from the table to the pool and back, and every step that meets it says so."""
    from moe_layer_dsv3_gb300.pages import PagePlan
    for bad in (6, -1, 2 ** 31 - 1, -2 ** 31):
        plan = PagePlan(2, 8, 6, 4, 32)
        table, free, count, lens = plan.new_pool()

        def step(*target):
            plan.update(lens, i32(target), table, free, count)
            torch.cuda.synchronize()
            assert lens.tolist() == list(target)
            return plan.status()
        assert step(24, 3) == (0, 0) and table[0].tolist() == [0, 1, 2, -1] and table[1].tolist() == [3, -1, -1, -1]
        table[0, 2] = bad
        assert step(9, 3)[0] == lib.MOE_ERR_BOUNDS           # left by a sequence that shrinks: the pool holds it
        assert count.tolist() == [3] and free.tolist()[:3] == [5, 4, bad]
        assert step(9, 3) == (0, 0)                          # a step that does not meet it
        assert step(9, 20)[0] == lib.MOE_ERR_BOUNDS          # popped by the other sequence: the table holds it
        assert table[1].tolist() == [3, bad, 4, -1] and count.tolist() == [1]
        # the tokens of that page have no row, the others have theirs
        assert plan.slot.tolist()[:17] == [3 * 8 + i for i in range(3, 8)] + [-1] * 8 + [4 * 8 + i for i in range(4)]
        assert step(9, 20) == (0, 0)
        table[1, 1] = 2                                      # mended in the table, it serves again
        assert step(9, 0) == (0, 0) and sorted(free.tolist()[:4]) == [2, 3, 4, 5]
